"""What the waves of a workgroup share, in the kernels that train and adapt a block: pieces of the kernels' own source,
compiled for the host, run wave by wave with every touch of LDS and every barrier counted.  No GPU: a race seldom shows
there, and a barrier that some waves pass once more can hang it."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_29_amd", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def run(folder, text, *args, flags=("-O1",)):
    """The program's output lines; it is compiled once a folder."""
    cpp, exe = folder / "model.cpp", folder / "model"
    if not exe.exists():
        cpp.write_text(text)
        made = subprocess.run(["g++", "-std=c++20", *flags, "-w", str(cpp), "-o", str(exe)], capture_output=True, text=True)
        assert made.returncode == 0, made.stderr[-3000:]
    return subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, check=True, timeout=100).stdout.splitlines()


# ---------------------------------------------------------------- a norm's sums over a row

ROW_SUMS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
struct { int x; } threadIdx;
struct Touch { int wave, at; bool write; };
static std::vector<std::vector<Touch>> between;      // by the barriers passed so far
static int wave, epoch, highest;
static void touch(int at, bool write) {
  if ((int)between.size() <= epoch) between.resize(epoch + 1);
  between[epoch].push_back({wave, at, write});
  if (at > highest) highest = at;
}
static void __syncthreads() { ++epoch; }
struct Slot {
  int at;
  operator float() const { touch(at, false); return 1.0f; }
  void operator=(float) const { touch(at, true); }
};
struct Shared {
  int at;
  Slot operator[](int i) const { return {at + i}; }
  Shared operator+(int n) const { return {at + n}; }
};
static float wave_sum(float x) { return x; }
#define GPTQ_DEV static
@CONSTANTS@
@FUNCTION@
// args: waves of a row, waves of the workgroup, then the numbers of values of the calls in turn
int main(int n, char** v) {
  const int row = atoi(v[1]), waves = atoi(v[2]);
  for (wave = 0; wave < waves; ++wave) {
    threadIdx.x = 64 * wave;
    epoch = 0;
    int turn = 0;
    for (int c = 3; c < n; ++c) {
      float a[1] = {}, b[3] = {};
      if (atoi(v[c]) == 1) row_sums<1>(a, Shared{0}, turn, row);
      else row_sums<3>(b, Shared{0}, turn, row);
    }
  }
  int races = 0;
  for (const auto& e : between)
    for (const Touch& a : e)
      for (const Touch& b : e) races += a.wave < b.wave && a.at == b.at && (a.write || b.write);
  printf("%d %d %zu\n", races, highest, (size_t)(@SIZE@));
}
"""


@pytest.mark.parametrize("kernel,mixes", [("residual_norm_kernel", ["1 1 1 1 1"]),
                                          ("residual_norm_backward_kernel", ["3 3 3 3", "3 1 3 1 3 1", "3 1 1 3 3 1 1 1 3"])])
def test_row_sums_touch_nothing_that_is_still_read(tmp_path, kernel, mixes):
    """Between two barriers no wave writes what another one reads or writes, whatever the order of the calls, and all of it
    lies in the kernel's array."""
    text = source("norm.hip")
    function = re.search(r"template <int N>\nGPTQ_DEV void row_sums.*?\n}\n", text, re.S)[0].replace("float*", "Shared")
    body = text[text.index(f"void {kernel}("):]
    size = re.search(r"__shared__ float red\[([^\]]+)\]", body)[1]
    made = {int(x) for x in re.findall(r"row_sums<(\d)>", body[:body.index("\n}\n")])}
    assert made and made >= {int(x) for m in mixes for x in m.split()}
    constants = "\n".join(re.findall(r"^constexpr int \w+ = [^;]+;", text, re.M))
    program = ROW_SUMS.replace("@CONSTANTS@", constants).replace("@FUNCTION@", function).replace("@SIZE@", size)
    for row in range(1, 17):
        for mix in mixes:
            races, highest, room = map(int, run(tmp_path, program, row, 16 // row * row, *mix.split())[0].split())
            assert races == 0, f"{mix} with {row} waves a row: {races} pairs"
            assert highest < room



# ---------------------------------------------------------------- whole prompts: tiles and barriers

PROMPT = r"""
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>
using std::max; using std::min;
constexpr int HD = 64, kRows = 128, kKeys = 64;
constexpr uint32_t kTile = 1000, kBuf = 2 * kTile, kV = 3 * kTile, lds = 100000;
constexpr float kGrow = 4.0f, kFar = 65536.0f;
typedef int T; typedef int f32x16_t;
static std::mt19937 random_bits(1);
static bool some() { return random_bits() % 4 == 0; }
static bool __any(bool) { return some(); }
template <int N> void wait_copies() {}
static void wait_lds_reads() {}
static int wave, epoch;
static void ring_barrier() { ++epoch; }
struct Event { bool copy; uint32_t buf; int tile, epoch; };
static std::vector<Event> events[4];
static void copied(uint32_t buf, int tile) { events[wave].push_back({true, buf, tile, epoch}); }
static void read(uint32_t buf, int tile) { events[wave].push_back({false, buf, tile, epoch}); }
struct TileCopy { void go(int row0, uint32_t to) const { copied(to, row0 / kKeys); } };
static uint32_t looked_at;
template <typename A, int B> bool tile_has_none(uint32_t at) { looked_at = at; return some(); }
template <typename A, int B, typename... X> void add_none(X...) {}
template <typename A, int B, bool C, typename... X> void add_columns(X...) {}
template <typename A> int pack8(int, int) { return 0; }
struct { bool fits(int) { return !some(); } void apply(int) {} } sc;

@BODY@

static int bad, passed;
static void check(const char* what, int n, int level) {
  for (int w = 1; w < 4; ++w) {
    const auto barriers = [](int x) { int e = 0; for (const Event& v : events[x]) if (v.tile == -1) e = v.epoch; return e; };
    if (barriers(w) != barriers(0)) {
      if (++bad < 5) printf("%s n %d level %d: wave %d passes %d barriers, wave 0 %d\n", what, n, level, w, barriers(w), barriers(0));
    }
  }
  // a tile is read behind a barrier that all of its copies stand in front of, and before the buffer's next copies
  std::map<uint32_t, std::vector<Event>> copies;
  for (const auto& e : events) for (const Event& v : e) if (v.copy) copies[v.buf].push_back(v);
  for (int w = 0; w < 4; ++w)
    for (const Event& r : events[w]) {
      if (r.copy || r.tile == -1) continue;
      int parts = 0, newest = -1;
      bool over = false;
      for (const Event& c : copies[r.buf]) if (c.epoch <= r.epoch && c.epoch > newest) newest = c.epoch;
      for (const Event& c : copies[r.buf]) {
        if (c.epoch == newest && c.tile == r.tile) ++parts;
        if (c.epoch == r.epoch) over = true;
      }
      ++passed;
      if ((parts != 4 || over) && ++bad < 5)
        printf("%s n %d level %d: wave %d reads tile %d, where %d waves copied it%s\n", what, n, level, w, r.tile, parts, over ? ", while it is copied over" : "");
    }
  for (auto& e : events) e.clear();
}
int main() {
  for (int n = 1; n <= 460; ++n)
    for (int level = 0; level * kRows < n; ++level)
      for (int again = 0; again < 3; ++again) {
        for (wave = 0; wave < 4; ++wave) { epoch = 0; forward(n, level); read(0, -1); }
        check("forward", n, level);
        for (wave = 0; wave < 4; ++wave) { epoch = 0; queries(n, level); read(0, -1); }
        check("dq", n, level);
        const int rep = 1 + random_bits() % 3, splits = 1 + random_bits() % 4, split = random_bits() % splits;
        for (wave = 0; wave < 4; ++wave) { epoch = 0; keys_values(n, level, rep, splits, split); read(0, -1); }
        check("dkv", n, level);
      }
  printf("%d %d\n", bad, passed);
}
"""


def between(text, first, last, whole_line=False):
    """The text from `first` to in front of `last` (whole_line: to the end of its line)."""
    a = text.index(first)
    b = text.index(last, a)
    return text[a:text.index("\n", b) + 1] if whole_line else text[a:b]


def test_the_waves_of_a_prompt_tile_meet_at_every_barrier(tmp_path):
    """The loops over tiles, forward, dQ, dK and dV: every wave of a workgroup passes as many barriers, and reads a tile where
    all waves' copies of it have landed and before the next ones start, for every length, also where the workgroup's last
    tokens do not exist."""
    text = source("prompt.hip")
    kernel = lambda name: between(text, f"void {name}(", "\n}\n")  # noqa: E731
    f, q, kv = kernel("prompt_forward_kernel"), kernel("prompt_dq_kernel"), kernel("prompt_dkv_kernel")
    head = "  const int r0 = level * kRows, w0 = r0 + 32 * wave, row = w0;\n  TileCopy ck, cv;\n"
    forward = ["static void forward(int n, int level) {\n", head,
               between(f, "  const int tiles =", "\n", True), between(f, "  uint32_t keys = lds", "\n", True), "  ck.go(0, keys);\n  cv.go(0, values);\n",
               between(f, "  if (tiles > 1) ck.go", "\n", True), "  int o = 0, rd = 0;\n  float m = 0.0f, top = 0.0f;\n",
               between(f, "  int k = 0;\n", "  // raw scores"),
               """  auto tile_of = [&](uint32_t at) { return at == keys || at == values ? k : at == keys1 ? k + 1 : -2; };
  auto scores = [&](uint32_t from, int) { read(from, tile_of(from)); return 0; };
  auto top_of = [&](int) { return 0.0f; };
  auto any_block = [&]<bool FINITE>(int, int) { read(values, k); };
  auto whole_block = [&]<int KB>(uint32_t from, int&, int&) { read(from, tile_of(from)); read(values, k); };
""", between(f, "  const int last =", "\n", True), between(f, "  f32x16_t s0, s1;", "the other waves' tiles", True), "}\n"]
    dq = ["static void queries(int n, int level) {\n", head, "  ck.go(0, lds);\n  cv.go(0, lds + kTile);\n  int acc = 0, rd = 0;\n",
          between(q, "  const int tiles =", "  // ds of 32 keys"),
          """  auto slopes = [&](int, int& s) { s = 0; read(buf, k); read(buf + kTile, k); };
  auto any_tile = [&]<bool FINITE>(int) { read(buf, k); read(buf + kTile, k); };
""", between(q, "  const int whole =", "the other waves' tiles", True), "}\n"]
    dkv = ["static void keys_values(int n, int level, int rep, int splits, int split) {\n  struct { int rep, splits; } a{rep, splits};\n",
           between(kv, "  const int k0 =", ", key =").replace("\n", " ") + ";\n", between(kv, "  const int first =", "  TileCopy<HD> cq"),
           "  int dk = 0, dv = 0, rd = 0;\n  auto copy = [&](int t, uint32_t to) { copied(to, t); };\n",
           between(kv, "  uint32_t buf = lds", "  // p and ds of 32 tokens"),
           """  auto slopes = [&](int, int& s, int& ds) { s = ds = 0; read(buf, i); };
  auto any_tile = [&]<bool FINITE>(int) { read(buf, i); };
""", between(kv, "  const uint32_t whole =", "  if (key >= n) return;"), "}\n"]
    out = run(tmp_path, PROMPT.replace("@BODY@", "".join(forward + dq + dkv)))
    bad, passed = map(int, out[-1].split())
    assert passed > 100000
    assert bad == 0, "\n".join(out[:-1])


# ---------------------------------------------------------------- whole prompts: counts

def test_prompt_counts_at_the_end_of_32_bits(tmp_path):
    """How many tiles a batch may have and in how many parts a tile's tokens go, of bounds of nearly 2^31, with a trap at
    every overflow."""
    text = source("prompt.hip")
    body = between(text, "// tiles of 128 tokens that n_tokens", "static size_t rows_part")
    out = run(tmp_path, "#include <algorithm>\n#include <climits>\n#include <cstdint>\n#include <cstdio>\n"
              "constexpr int kRows = 128, kKeys = 64;\n" + body + """
int main() {
  for (int64_t most : {INT_MAX, INT_MAX - 1, INT_MAX - 62, INT_MAX - 63, INT_MAX - 126, INT_MAX - 127, 1 << 30, 700, 1})
    for (int64_t tokens : {(int64_t)INT_MAX, (int64_t)700, (int64_t)1}) {
      const int64_t tiles = tile_bound(tokens, 2, most);
      printf("%ld %ld %ld %d\\n", (long)most, (long)tokens, (long)tiles, key_splits(tiles, tokens, 1, 4, most));
    }
}
""", flags=("-ftrapv", "-O0"))
    assert len(out) == 27
    for most, tokens, tiles, splits in (map(int, line.split()) for line in out):
        assert tiles == min(-(-tokens // 128) + 1, 2 * -(-most // 128)) and 1 <= splits <= 8
