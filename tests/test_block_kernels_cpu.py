"""What the waves of a workgroup share, in the kernels that train and adapt a block: pieces of the kernels' own source,
compiled for the host, run wave by wave with every touch of LDS and every barrier counted.  No GPU: a race seldom shows
there, and a barrier that some waves pass once more can hang it."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_29_amd", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def run(folder, text, *args):
    """The program's output lines; it is compiled once a folder."""
    cpp, exe = folder / "model.cpp", folder / "model"
    if not exe.exists():
        cpp.write_text(text)
        made = subprocess.run(["g++", "-std=c++20", "-O1", "-w", str(cpp), "-o", str(exe)], capture_output=True, text=True)
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

