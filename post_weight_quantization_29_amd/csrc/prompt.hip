// Causal attention of whole prompts packed one behind the other, grouped heads,
// forward and backward, on v_mfma_f32_32x32x16.
//
// Forward: a workgroup takes 128 tokens of one head, 32 to each of four waves, and
// walks the sequence's keys in tiles of 64, copied HBM -> LDS a tile ahead (keys two).  The
// first product is made as S^T = K Q^T: a lane then holds scores of one token (its
// column), so maximum and sum are its own registers and one exchange with the
// other half of the wave, and the probabilities are, as they lie, the second
// operand of O^T = V^T P^T (k of that product in the order in which the registers
// hold the keys).  V^T is read out of V's rows by transposing LDS reads.
//
// Backward, without atomics: one kernel per 128 tokens for dQ (the forward's shape;
// it also leaves each row's lse and D = dout . out for the other), one per 128
// keys and kv head for dK and dV, which walks the query heads and their tokens.
// Both make the probabilities again from lse: seven products for five.
//
// p and ds are rounded once to 16 bits where they are an operand (ds of fp16 below a power
// of two, its own for each token or key): half a step of a term, so the outputs' errors are
// 1.2 to 1.3 (forward), 1.5 (bf16 gradients) and 1.6 times (fp16's dQ and dK) those of rounding the
// outputs alone, of which a tenth is D's, from the rounded out.  Two pieces instead would be two
// more products of the seven; of ds in dQ alone they took four sequences of 2048 from 618 to 681 us and
// 13 ragged ones from 182 to 195, for an error of dQ 1.2 times that of rounding it.  Sums, maxima
// and D are fp32.
//
// Tiles lie in LDS as rows of head_dim values whose 16-byte chunk c sits at c ^
// f(row): 16 consecutive rows' reads of one chunk, and the transposing reads of
// four rows by two groups of 16 channels, each fall into different banks.
//
// A row's zero probability times an infinity that it does not see would be NaN: in
// the tiles on the diagonal the operand that is summed over is looked at first,
// and if it has a value that is no number those count as zeros in the product and
// are added where they are seen.
#include "gemm16.h"
#include "w4_epilogue.h"

#include <climits>

namespace gptq {

constexpr int kRows = 128, kKeys = 64, kPromptWaves = 4;
constexpr float kNoScore = -1e30f;       // a running maximum that has seen nothing
constexpr float kGrow = 4.0f;            // log2 by which scores may pass the maximum before the sums are rescaled
constexpr float kFar = 65536.0f;         // a maximum whose half step is no longer nothing beside 1
constexpr int64_t kMaxPitch = (int64_t)1 << 22;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// fp16 has 5 exponent bits: probabilities are held times 2^kUp, so that those down
// to 2^-34 of the largest still count
template <typename T> constexpr float kUp = T16<T>::kType == GPTQ_F16 ? 10.0f : 0.0f;
template <typename T> constexpr bool kScaled = T16<T>::kType == GPTQ_F16;

struct PromptBatch {
  const int32_t* q_start;
  int64_t n_tokens;
  int n_seqs, max_len;
  // a sequence's first row and its tokens, cut to the rows that exist and to max_len
  GPTQ_DEV void span(int b, int64_t& t0, int& n) const {
    const int64_t a = max((int64_t)q_start[b], (int64_t)0), e = min((int64_t)q_start[b + 1], n_tokens);
    t0 = a;
    n = (int)min(max(e - a, (int64_t)0), (int64_t)max_len);
  }
  // the same for a sequence that is one for the whole wave, in scalar registers
  GPTQ_DEV void span_of(int b, int64_t& t0, int& n) const {
    span(b, t0, n);
    t0 = __builtin_amdgcn_readfirstlane((int)t0);       // rows fit 31 bits
    n = __builtin_amdgcn_readfirstlane(n);
  }
};

// The u-th tile (of kRows tokens) of the batch in the order of falling numbers of
// tiles behind (and with) it in its sequence, or before it: the longest work first, so that
// what is left for the end is short.  level: that number less one.  Tiles at
// level L or above number sum_b max(0, tiles_b - L): the level is found by halving.
GPTQ_DEV bool tile_at(const PromptBatch& q, int u, int& b, int& level) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int s) {
    int64_t t0;
    int n = 0;
    if (s < q.n_seqs) q.span(s, t0, n);
    return (n + kRows - 1) / kRows;
  };
  const int first = tiles_of(lane);
  auto from = [&](int L) {
    int64_t c = max(first - L, 0);
    for (int s = 64; s < q.n_seqs; s += 64) c += max(tiles_of(s + lane) - L, 0);
#pragma unroll
    for (int o = 32; o; o >>= 1) c += __shfl_xor(c, o);
    return c;
  };
  if (from(0) <= u) return false;
  int lo = 0, hi = (q.max_len + kRows - 1) / kRows;
  int64_t above = 0;                                    // from(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    const int64_t c = from(mid);
    if (c > u) lo = mid;
    else {
      hi = mid;
      above = c;
    }
  }
  level = lo;
  int left = (int)(u - above);                          // which of the sequences that reach this level
  for (int s = 0; s < q.n_seqs; s += 64) {
    const bool reach = (s ? tiles_of(s + lane) : first) > lo;
    const uint64_t m = __ballot(reach);
    const int c = __popcll(m);
    if (left < c) {
      const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
      b = s + __builtin_ctzll(__ballot(reach && rank == left));
      return true;
    }
    left -= c;
  }
  return false;
}

// Rows of a tile in LDS
template <int HD> GPTQ_DEV int chunk_flip(int row) {
  return HD == 128 ? ((row & 7) << 1) | ((row >> 3) & 1) : (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
}
template <int HD> constexpr uint32_t kTileBytes = kKeys * HD * 2;

// Copies of a tile of 64 rows: each wave its part.  The descriptor ends behind the
// last row that exists, so rows past it read zero.
template <int HD> struct TileCopy {
  static constexpr int kEach = (int)(kTileBytes<HD> / 1024) / kPromptWaves;   // copies a wave
  int voff[kEach];
  uint32_t at;
  uint64_t base;
  int64_t pitch;                                       // bytes
  int n;
  GPTQ_DEV void init(const uint16_t* p, int64_t ld, int n_rows, int wave) {
    const int lane = threadIdx.x & 63;
    constexpr int RC = HD / 8;                         // chunks a row
    base = reinterpret_cast<uint64_t>(p);
    pitch = 2 * ld;
    n = n_rows;
    at = 1024u * kEach * wave;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int row = (kEach * wave + k) * (64 / RC) + lane / RC;
      voff[k] = (int)(row * pitch) + 16 * ((lane % RC) ^ chunk_flip<HD>(row));
    }
  }
  // rows r0 .. r0 + 63 to lds
  GPTQ_DEV void go(int r0, uint32_t lds) const {
    const uint64_t p = base + (uint64_t)((int64_t)r0 * pitch);
    const int64_t left = max(n - r0, 0) * pitch;
    i32x4_t r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
    r[2] = __builtin_amdgcn_readfirstlane((int)min(left, (int64_t)0x7fffff00));
    r[3] = 0x00020000;
#pragma unroll
    for (int k = 0; k < kEach; ++k) copy16_lds(lds + at + 1024u * k, r, voff[k]);
  }
};

// Where a lane reads a tile.  Rows: row 32 b + lane % 32, chunk 2 s + lane / 32 (an
// operand whose k is the channels).  Columns: four rows 16 t + 8 j + 4 (lane / 32) ..
// by 16 channels (k is the rows): channels 16 (c + HD/32 (lane / 16 % 2)) ..
template <int HD> struct TileRead {
  uint32_t row, col;
  GPTQ_DEV void init() {
    const int lane = threadIdx.x & 63, h = lane >> 5, s = (lane >> 2) & 3;
    row = (lane & 31) * (2 * HD) + ((h ^ chunk_flip<HD>(lane & 15)) << 4);
    const int r = 4 * h + s, flip = HD == 128 ? r << 1 : (r >> 1) << 1;
    const int q0 = (lane >> 4) & 1;
    col = r * (2 * HD) + ((((q0 * (HD / 16)) | ((lane >> 1) & 1)) ^ flip) << 4) + 8 * (lane & 1);
  }
  template <typename V> GPTQ_DEV V rows(uint32_t tile, int b, int s) const {
    return *(LDS_AS const V*)(uintptr_t)((tile + (row ^ (s << 5))) + 64 * HD * b);
  }
  GPTQ_DEV uint2 four(uint32_t tile, int t, int j, int c) const {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    const uint32_t at = tile + (col ^ (c << 5) ^ (j << 4)) + (16 * t + 8 * j) * (2 * HD);
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(uintptr_t)at));
  }
};
// channel of row rho of a product whose rows are column block c's channels
template <int HD> GPTQ_DEV int channel_of(int c, int rho) { return 16 * (c + (rho >> 4) * (HD / 32)) + (rho & 15); }

// values that are no number as zeros, two 16-bit values at a time
template <typename T> GPTQ_DEV uint32_t finite_pair(uint32_t x) {
  constexpr uint32_t E = T16<T>::kType == GPTQ_F16 ? 0x7C00u : 0x7F80u;
  if ((x & E) == E) x &= 0xFFFF0000u;
  if ((x & (E << 16)) == E << 16) x &= 0xFFFFu;
  return x;
}
// does the tile have one (the same answer in all lanes)
template <typename T, int HD> GPTQ_DEV bool tile_has_none(uint32_t tile) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  constexpr uint32_t E = T16<T>::kType == GPTQ_F16 ? 0x7C00u : 0x7F80u;
  const int lane = threadIdx.x & 63;
  u16x2_t top = {0, 0};
#pragma unroll 4
  for (uint32_t at = 16 * lane; at < kTileBytes<HD>; at += 1024) {
    const i32x4_t v = *(LDS_AS const i32x4_t*)(uintptr_t)(tile + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[e] & 0x7FFF7FFF));
  }
  return __any(top[0] >= E || top[1] >= E);
}
// the larger of the two halves' values of a column
GPTQ_DEV float over_halves_max(float x) {
  const auto v = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)v[0]), __builtin_bit_cast(float, (uint32_t)v[1]));
}
GPTQ_DEV float over_halves_sum(float x) {
  const auto v = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)v[0]) + __builtin_bit_cast(float, (uint32_t)v[1]);
}

GPTQ_DEV f32x16_t zeros16() { return f32x16_t{}; }

// acc[c] += A^T B over 64 rows of the tile: A's columns by transposing reads, B the
// columns' registers in pairs (pk[t] the 16 rows 16 t ..)
template <typename T, int HD, bool FINITE>
GPTQ_DEV void add_columns(f32x16_t (&acc)[HD / 32], const TileRead<HD>& rd, uint32_t tile, int t, const typename T16<T>::v8& pk) {
  typedef typename T16<T>::v8 v8;
#pragma unroll
  for (int c = 0; c < HD / 32; ++c) {
    uint2 a = rd.four(tile, t, 0, c), b = rd.four(tile, t, 1, c);
    if constexpr (FINITE) {
      a.x = finite_pair<T>(a.x); a.y = finite_pair<T>(a.y);
      b.x = finite_pair<T>(b.x); b.y = finite_pair<T>(b.y);
    }
    acc[c] = T16<T>::mfma32(__builtin_bit_cast(v8, make_uint4(a.x, a.y, b.x, b.y)), pk, acc[c]);
  }
}
// A value that is no number as a small one that counts it: +inf 1, -inf 128, NaN 16384.
template <typename T> GPTQ_DEV uint32_t none_pair(uint32_t x) {
  constexpr uint32_t E = T16<T>::kType == GPTQ_F16 ? 0x7C00u : 0x7F80u;
  uint32_t r = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = (x >> (16 * h)) & 0xFFFFu;
    const float n = (v & E) != E ? 0.0f : (v & 0x7FFFu) != E ? 16384.0f : v >> 15 ? 128.0f : 1.0f;
    r |= (uint32_t)bits16<T>(n) << (16 * h);
  }
  return r;
}
// Adds the tile's values that are no number where the lane's column sees them
// (rows [lo, hi) of the tile): their numbers by channel are a product with ones.
template <typename T, int HD> GPTQ_DEV void add_none(f32x16_t (&acc)[HD / 32], const TileRead<HD>& rd, uint32_t tile, int lo, int hi) {
  typedef typename T16<T>::v8 v8;
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int c = 0; c < HD / 32; ++c) {
    f32x16_t n = zeros16();
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
      uint32_t see[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * t + 8 * (e >> 1) + 4 * h + 2 * (e & 1);
        see[e] = pack2<T>(k >= lo && k < hi ? 1.0f : 0.0f, k + 1 >= lo && k + 1 < hi ? 1.0f : 0.0f);
      }
      const uint2 a = rd.four(tile, t, 0, c), b = rd.four(tile, t, 1, c);
      n = T16<T>::mfma32(__builtin_bit_cast(v8, make_uint4(none_pair<T>(a.x), none_pair<T>(a.y), none_pair<T>(b.x), none_pair<T>(b.y))),
                         __builtin_bit_cast(v8, make_uint4(see[0], see[1], see[2], see[3])), n);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int x = (int)n[r];
      if (x & 127) acc[c][r] += INFINITY;
      if ((x >> 7) & 127) acc[c][r] -= INFINITY;
      if (x >> 14) acc[c][r] = NAN;
    }
  }
}
// eight registers of a block, 8 u .. 8 u + 7, as the operand of rows 16 (2 b + u) ..
template <typename T> GPTQ_DEV typename T16<T>::v8 pack8(const f32x16_t& p, int u) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack2<T>(p[8 * u + 2 * e], p[8 * u + 2 * e + 1]);
  return __builtin_bit_cast(typename T16<T>::v8, make_uint4(w[0], w[1], w[2], w[3]));
}

// a lane's row of a head: chunk 2 s + lane / 32 of each slice s
template <typename T, int HD> GPTQ_DEV void load_row(typename T16<T>::v8 (&v)[HD / 16], const uint16_t* p, uint32_t flip = 0) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int s = 0; s < HD / 16; ++s) {
    uint4 x = *reinterpret_cast<const uint4*>(p + 16 * s + 8 * h);
    x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
    v[s] = __builtin_bit_cast(typename T16<T>::v8, x);
  }
}
// the lane's column of a product whose rows are channels, times f, to a head's row
template <typename T, int HD> GPTQ_DEV void store_row(uint16_t* p, const f32x16_t (&acc)[HD / 32], float f) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int c = 0; c < HD / 32; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint2 w;
      w.x = pack2<T>(acc[c][4 * q] * f, acc[c][4 * q + 1] * f);
      w.y = pack2<T>(acc[c][4 * q + 2] * f, acc[c][4 * q + 3] * f);
      *reinterpret_cast<uint2*>(p + channel_of<HD>(c, 8 * q + 4 * h)) = w;
    }
}

struct PromptArgs {
  const uint16_t *Q, *K, *V, *dO, *O;
  uint16_t *out, *dQ, *dK, *dV;
  float* lse;              // forward: out; backward: in
  float* rows;             // backward: [2][n_heads][n_tokens]: lse in log2, D
  float* part;             // backward, splits > 1: [splits][dK, dV][n_tokens][n_kv][head_dim]
  int splits;              // workgroups that share the tokens of a tile of keys
  int64_t ldq, ldk, ldv, lddo, ldo, lddq, lddk, lddv;
  int n_heads, n_kv, rep;
  float scale, scale2;     // scale2 = scale * log2 e (forward: of its absolute value)
  uint32_t flip;           // forward: Q's sign bits, for a negative scale
};

// workgroup -> tile and head: a tile's heads next to each other, kv head by kv
// head, so that those of one kv head fall on few XCDs
GPTQ_DEV bool head_tile(const PromptArgs& a, const PromptBatch& q, int& b, int& level, int& head) {
  const int u = blockIdx.x / a.n_heads, x = blockIdx.x - u * a.n_heads;
  head = x % a.n_kv * a.rep + x / a.n_kv;
  return tile_at(q, u, b, level);
}

// Prompts of 4096, 2048, 2048 and 1371 tokens, 64 heads of 128 on 8 kv heads, bf16: 443
// GFLOP in 550 to 575 us back to back, 0.77 to 0.81 PFLOP/s, the matrix pipe busy in 35 % of the cycles,
// waves waiting in 40 %.  No single thing bounds it: in copies of the kernel the time under the
// profiler (655 to 690 as it is, with the box) was, of 690, 533 without the copies of tiles behind
// the first, 624 without LDS reads in the loop, some 640 without exponentials, 489 without any of
// them.  256 tokens a workgroup (half the copies) took as long, with tiles three ahead too, and so
// did a loop over pairs of tiles with constant addresses and half of the vector instructions.
template <typename T, int HD>
__global__ __launch_bounds__(64 * kPromptWaves, 2) void prompt_forward_kernel(PromptArgs a, PromptBatch q) {
  typedef typename T16<T>::v8 v8;
  constexpr int KS = HD / 16, NC = HD / 32;
  // LDS: three tiles of keys and two of values (two workgroups a CU take all of it)
  constexpr uint32_t kTile = kTileBytes<HD>, kV = 3 * kTile;
  __shared__ __attribute__((aligned(1024))) char smem[5 * kTile];
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int b, level, head;
  if (!head_tile(a, q, b, level, head)) return;
  int64_t t0;
  int n;
  q.span(b, t0, n);
  const int r0 = level * kRows, w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  const int kv = head / a.rep;
  const int tiles = (min(r0 + kRows, n) + kKeys - 1) / kKeys;
  TileCopy<HD> ck, cv;
  ck.init(a.K + t0 * a.ldk + (int64_t)kv * HD, a.ldk, n, wave);
  cv.init(a.V + t0 * a.ldv + (int64_t)kv * HD, a.ldv, n, wave);
  // where tile k's, k + 1's and k + 2's keys are, and tile k's values
  uint32_t keys = lds, keys1 = lds + kTile, keys2 = lds + 2 * kTile, values = lds + kV, values1 = lds + kV + kTile;
  ck.go(0, keys);
  cv.go(0, values);
  if (tiles > 1) ck.go(kKeys, keys1);
  v8 qv[KS];
  load_row<T, HD>(qv, a.Q + (t0 + min(row, n - 1)) * a.ldq + (int64_t)head * HD, a.flip);
  TileRead<HD> rd;
  rd.init();
  f32x16_t o[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) o[c] = zeros16();
  float m = kNoScore, l = 0.0f;
  int k = 0;
  // Tile k + 1's keys and tile k's values have landed, and everybody is done with tile
  // k - 1's of both.
  auto arrive = [&]() {
    wait_copies<0>();
    wait_lds_reads();
    ring_barrier();
    if (k + 2 < tiles) ck.go(kKeys * (k + 2), keys2);
    if (k + 1 < tiles) cv.go(kKeys * (k + 1), values1);
  };
  auto leave = [&]() {
    const uint32_t x = keys, y = values;
    keys = keys1;
    keys1 = keys2;
    keys2 = x;
    values = values1;
    values1 = y;
    ++k;
  };
  // raw scores of 32 keys: block kb of the tile at `from`
  auto scores = [&](uint32_t from, int kb) {
    f32x16_t s = zeros16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s = T16<T>::mfma32(rd.template rows<v8>(from, kb, ks), qv[ks], s);
    return s;
  };
  auto top_of = [&](const f32x16_t& s) {
    float top = -INFINITY;
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[r]);
    return over_halves_max(top) * a.scale2;
  };
  // This wave's tiles: w0 / 64 whole ones, then the one on the diagonal.  (A wave behind
  // the sequence's end has none.)
  const int last = w0 < n ? w0 / kKeys : -1;
  // Block kb, of scores s, of any tile: the last one, on the diagonal; one whose scores have
  // outgrown the maximum; one with a maximum so large that half a step of it counts.
  auto any_block = [&]<bool FINITE>(int kb, f32x16_t s) {
    const int k0 = kKeys * k + 32 * kb;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = k0 + 8 * (r >> 2) + 4 * h + (r & 3) <= row ? s[r] : -INFINITY;
    const float top = top_of(s);
    // only where it has grown: a token's rounding does not depend on its neighbours
    const float m_new = top > m + kGrow ? top : m, al = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    l *= al;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[c][r] *= al;
    // One fma a score sees the score times scale2 unrounded and the maximum rounded, half
    // a step apart, which is nothing until the maximum is large.
    const bool far = fabsf(m) > kFar;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
#pragma clang fp contract(off)
      const float x = s[r] * a.scale2;
      float p = __builtin_amdgcn_exp2f(far ? (x - m) + kUp<T> : __builtin_fmaf(s[r], a.scale2, kUp<T> - m));
      p = k0 + 8 * (r >> 2) + 4 * h + (r & 3) <= row ? p : 0.0f;
      l += p;
      s[r] = p;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) add_columns<T, HD, FINITE>(o, rd, values, 2 * kb + u, pack8<T>(s, u));
  };
  // Block KB of a whole tile: the next block's scores (of keys at `from`) are made while this
  // one's exponentials are, and their largest is looked for during the second product:
  // neither depends on what it stands beside, and the matrix pipe has as much to do as the
  // vector one.  Operands are read four products ahead; the order is the source's (left to
  // itself the compiler brings the reads together in front and spills, and a reload in the
  // loop waits for every copy under way).
  float top = 0.0f;                        // the largest of the next block's scores times scale2
  auto whole_block = [&]<int KB>(uint32_t from, f32x16_t& s, f32x16_t& next) {
    constexpr int EX = 16 / KS, NP = 2 * NC, MX = 16 / NP;
    const float sub = kUp<T> - m;
    auto value = [&](int y) {
      const uint2 u = rd.four(values, 2 * KB + y / NC, 0, y % NC), w = rd.four(values, 2 * KB + y / NC, 1, y % NC);
      return __builtin_bit_cast(v8, make_uint4(u.x, u.y, w.x, w.y));
    };
    v8 kf[4], vf[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) kf[x] = rd.template rows<v8>(from, 1 - KB, x);
    f32x16_t z = zeros16();
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      z = T16<T>::mfma32(kf[x & 3], qv[x], z);
      if (x + 4 < KS) kf[x & 3] = rd.template rows<v8>(from, 1 - KB, x + 4);
      else vf[x + 4 - KS] = value(x + 4 - KS);
#pragma unroll
      for (int e = EX * x; e < EX * (x + 1); ++e) {
        s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], a.scale2, sub));
        l += s[e];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    top = -INFINITY;
    v8 pk = pack8<T>(s, 0);
#pragma unroll
    for (int y = 0; y < NP; ++y) {
      o[y % NC] = T16<T>::mfma32(vf[y & 3], pk, o[y % NC]);
      if (y + 4 < NP) vf[y & 3] = value(y + 4);
      if (y == NC - 1) pk = pack8<T>(s, 1);
#pragma unroll
      for (int e = MX * y; e < MX * (y + 1); ++e) top = fmaxf(top, z[e]);
      __builtin_amdgcn_sched_barrier(0);
    }
    next = z;
    top = over_halves_max(top) * a.scale2;
  };
  // The sums are rescaled outside the inner loop, which stops at a block that asks for it: as a
  // branch inside, the compiler kept them in two sets of registers and spilled the rest.
  f32x16_t s0, s1;
  wait_copies<0>();
  ring_barrier();
  if (last >= 0) {
    s0 = scores(keys, 0);
    top = top_of(s0);
    if (last > 0 && top > m + kGrow) m = top;          // (nothing to rescale yet)
  }
  arrive();
  while (k <= last) {
    auto plain = [&]() { return !__any(top > m + kGrow || fabsf(m) > kFar); };
    int kb = 0;
    while (k < last) {
      if (!plain()) break;
      whole_block.template operator()<0>(keys, s0, s1);
      kb = 1;
      if (!plain()) break;
      whole_block.template operator()<1>(keys1, s1, s0);
      kb = 0;
      leave();
      arrive();
    }
    // the rest of the tile, block by block
    const bool none = k == last && tile_has_none<T, HD>(values);
    f32x16_t s = kb ? s1 : s0;
#pragma unroll 1
    for (;;) {
      if (none) any_block.template operator()<true>(kb, s);
      else any_block.template operator()<false>(kb, s);
      if (kb == 1 || kKeys * k + 32 > w0 + 31) break;  // (block 1 behind all of the wave's rows)
      s = scores(keys, 1);
      kb = 1;
    }
    if (none) add_none<T, HD>(o, rd, values, 0, row - kKeys * k + 1);
    if (k < last) {
      s0 = scores(keys1, 0);
      top = top_of(s0);
    }
    leave();
    if (k < tiles) arrive();
  }
  for (leave(); k < tiles; leave()) arrive();          // the other waves' tiles
  l = over_halves_sum(l);
  if (row >= n) return;
  // A score whose log2 is beyond fp32 leaves l 0 (or no number): then so is the row.  Scores that are all no
  // number leave m as it was, but not l.
  const bool none = m == kNoScore && l == l;
  const float inv = none ? 0.0f : 1.0f / l;
  store_row<T, HD>(a.out + (t0 + row) * a.ldo + (int64_t)head * HD, o, inv);
  if (a.lse && h == 0) a.lse[(t0 + row) * a.n_heads + head] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l) - kUp<T>) * kLn2;
}

// fp16: ds is rounded below a power of two of its own, so that small gradients keep
// their bits: `up` brings the lane's column into range and grows smaller when the
// column's values outgrow it, its sums with it.  (bf16 has fp32's range.)
template <typename T, int HD> struct Scaled {
  float up = kScaled<T> ? 0x1p126f : 1.0f, top = 0.0f;
  // whether a block's values are in range of `up` in all lanes
  GPTQ_DEV bool fits(const f32x16_t& ds) {
    if constexpr (!kScaled<T>) return true;
    top = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(ds[r]));
    top = over_halves_max(top);
    return !__any(top * up > 0x1p15f);
  }
  // a smaller `up` where they are not
  GPTQ_DEV void shrink(f32x16_t (&acc)[HD / 32]) {
    if constexpr (kScaled<T>) {
      const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23);
      // top to 2^8 .. 2^9; within what a float's exponent allows
      const float now = top * up > 0x1p15f ? __builtin_bit_cast(float, (uint32_t)min(max(262 - e, 1), 253) << 23) : up;
      const float f = now / up;
      up = now;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[c][r] *= f;
    }
  }
  GPTQ_DEV void apply(f32x16_t& ds) const {
    if constexpr (kScaled<T>) {
#pragma unroll
      for (int r = 0; r < 16; ++r) ds[r] *= up;
    }
  }
};

// dQ: per tile S^T and dP^T = V dO^T, then dQ^T += K^T dS^T.  Four sequences of 2048, 32 heads
// of 128 on 8 kv heads, bf16: 254 us under the profiler (dK and dV 408 there, together 661; the whole
// pass takes 618 back to back without it), 0.81 PFLOP/s, matrix pipe busy in 38 %.
template <typename T, int HD>
__global__ __launch_bounds__(64 * kPromptWaves, 2) void prompt_dq_kernel(PromptArgs a, PromptBatch q) {
  typedef typename T16<T>::v8 v8;
  constexpr int KS = HD / 16, NC = HD / 32;
  constexpr uint32_t kTile = kTileBytes<HD>, kBuf = 2 * kTile;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kBuf];
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int b, level, head;
  if (!head_tile(a, q, b, level, head)) return;
  int64_t t0;
  int n;
  q.span_of(b, t0, n);
  level = __builtin_amdgcn_readfirstlane(level);
  const int r0 = level * kRows, w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  const int kv = head / a.rep;
  const int64_t tok = t0 + min(row, n - 1);
  v8 qv[KS], dv[KS];
  load_row<T, HD>(qv, a.Q + tok * a.ldq + (int64_t)head * HD);
  load_row<T, HD>(dv, a.dO + tok * a.lddo + (int64_t)head * HD);
  TileCopy<HD> ck, cv;
  ck.init(a.K + t0 * a.ldk + (int64_t)kv * HD, a.ldk, n, wave);
  cv.init(a.V + t0 * a.ldv + (int64_t)kv * HD, a.ldv, n, wave);
  ck.go(0, lds);
  cv.go(0, lds + kTile);
  float D = 0.0f;
  {
    v8 ov[KS];
    load_row<T, HD>(ov, a.O + tok * a.ldo + (int64_t)head * HD);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) D = fmaf((float)dv[s][e], (float)ov[s][e], D);
    D = over_halves_sum(D);
  }
  float lse = a.lse[tok * a.n_heads + head] * kLog2e;
  if (lse == -INFINITY) lse = INFINITY;                 // a row that sees nothing: its probabilities are 0
  if (h == 0 && row < n) {
    a.rows[(int64_t)head * q.n_tokens + tok] = lse;
    a.rows[((int64_t)a.n_heads + head) * q.n_tokens + tok] = D;
  }
  TileRead<HD> rd;
  rd.init();
  f32x16_t acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = zeros16();
  Scaled<T, HD> sc;
  const int tiles = (min(r0 + kRows, n) + kKeys - 1) / kKeys;
  uint32_t buf = lds, other = lds + kBuf;
  int k = 0;
  auto arrive = [&]() {
    wait_copies<0>();
    wait_lds_reads();
    ring_barrier();
    if (k + 1 < tiles) {
      ck.go(kKeys * (k + 1), other);
      cv.go(kKeys * (k + 1), other + kTile);
    }
  };
  auto leave = [&]() {
    const uint32_t t = buf;
    buf = other;
    other = t;
    ++k;
  };
  // ds of 32 keys
  auto slopes = [&](int kb, f32x16_t& s) {
    f32x16_t dp = zeros16();
    s = zeros16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s = T16<T>::mfma32(rd.template rows<v8>(buf, kb, ks), qv[ks], s);
      dp = T16<T>::mfma32(rd.template rows<v8>(buf + kTile, kb, ks), dv[ks], dp);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.scale2, -lse)) * (dp[r] - D);
  };
  // blocks kb0 .. 1 of any tile
  auto any_tile = [&]<bool FINITE>(int kb0) {
    const int k0 = kKeys * k;
#pragma unroll 1
    for (int kb = kb0; kb < 2; ++kb) {
      f32x16_t s;
      slopes(kb, s);
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = k0 + 32 * kb + 8 * (r >> 2) + 4 * h + (r & 3) <= row ? s[r] : 0.0f;
      if (!sc.fits(s)) sc.shrink(acc);
      sc.apply(s);
#pragma unroll
      for (int u = 0; u < 2; ++u) add_columns<T, HD, FINITE>(acc, rd, buf, 2 * kb + u, pack8<T>(s, u));
    }
    if constexpr (FINITE) add_none<T, HD>(acc, rd, buf, 0, row - k0 + 1);
  };
  // w0 / 64 whole tiles, then the one on the diagonal.  (A wave behind the sequence's end has none: with its own
  // number of them it went one tile, and one barrier, beyond the others.)
  const int whole = w0 < n ? w0 / kKeys : -1;
  while (k <= whole) {
    arrive();
    int kb0 = 0;
    while (k < whole) {
      bool stop = false;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        f32x16_t s;
        slopes(kb, s);
        if (!sc.fits(s)) {
          kb0 = kb;
          stop = true;
          break;
        }
        sc.apply(s);
#pragma unroll
        for (int u = 0; u < 2; ++u) add_columns<T, HD, false>(acc, rd, buf, 2 * kb + u, pack8<T>(s, u));
      }
      if (stop) break;
      leave();
      arrive();
    }
    if (k == whole && tile_has_none<T, HD>(buf)) any_tile.template operator()<true>(kb0);
    else any_tile.template operator()<false>(kb0);
    leave();
  }
  for (; k < tiles; leave()) arrive();                 // the other waves' tiles
  if (row < n) store_row<T, HD>(a.dQ + (t0 + row) * a.lddq + (int64_t)head * HD, acc, a.scale / sc.up);
}

// dK and dV: a wave has 32 keys, in registers, and walks the tokens that see them in
// tiles of 64, of all query heads of its kv head: S = Q K^T and dP = dO V^T, so that
// a lane's registers are tokens of one key (its column), then dV^T += dO^T P and dK^T
// += Q^T dS.  One wave a SIMD at head_dim 128 (K, V and both sums are 192 registers): 408 us under
// the profiler for the batch above (455 on a slower box), 0.67 PFLOP/s, matrix pipe busy in 30 %.  In
// copies of the kernel on that box: 333 without the first products' LDS reads, 403 without
// exponentials, no less without copies.  Exponentials beside the other block's products, reads four
// products ahead, took as long (fp16, with its checks of range, twice as long).
template <typename T, int HD>
__global__ __launch_bounds__(64 * kPromptWaves, HD == 64 ? 2 : 1) void prompt_dkv_kernel(PromptArgs a, PromptBatch q) {
  typedef typename T16<T>::v8 v8;
  constexpr int KS = HD / 16, NC = HD / 32;
  constexpr uint32_t kTile = kTileBytes<HD>, kBuf = 2 * kTile + 512;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kBuf];
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % a.splits, u = blockIdx.x / a.splits / a.n_kv, kv = blockIdx.x / a.splits - u * a.n_kv;
  int b, level;
  if (!tile_at(q, u, b, level)) return;
  int64_t t0;
  int n;
  q.span_of(b, t0, n);
  level = __builtin_amdgcn_readfirstlane(level);
  // the levels count from the sequence's end here
  const int k0 = ((n + kRows - 1) / kRows - 1 - level) * kRows, w0 = k0 + 32 * wave, key = w0 + (lane & 31);
  const int64_t tok = t0 + min(key, n - 1);
  v8 kr[KS], vr[KS];
  load_row<T, HD>(kr, a.K + tok * a.ldk + (int64_t)kv * HD);
  load_row<T, HD>(vr, a.V + tok * a.ldv + (int64_t)kv * HD);
  TileRead<HD> rd;
  rd.init();
  f32x16_t dk[NC], dv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    dk[c] = zeros16();
    dv[c] = zeros16();
  }
  Scaled<T, HD> sc;
  constexpr float kShift = kScaled<T> ? 14.0f : 0.0f;
  // tiles of tokens, of one query head after the other; this workgroup's of them
  const int first = k0 / kKeys, per_head = (n + kKeys - 1) / kKeys - first, all = per_head * a.rep;
  const int share = (all + a.splits - 1) / a.splits, total = min((split + 1) * share, all);
  TileCopy<HD> cq, co;
  cq.init(a.Q + t0 * a.ldq + (int64_t)kv * a.rep * HD, a.ldq, n, wave);
  co.init(a.dO + t0 * a.lddo + (int64_t)kv * a.rep * HD, a.lddo, n, wave);
  const uint64_t q_base = cq.base, o_base = co.base;
  auto copy = [&](int i, uint32_t to) {
    const int r = i / per_head, row0 = (first + i - r * per_head) * kKeys;
    cq.base = q_base + (uint64_t)r * (HD * 2);
    co.base = o_base + (uint64_t)r * (HD * 2);
    cq.go(row0, to);
    co.go(row0, to + kTile);
    if (wave < 2) {
      // lse and D of the 64 tokens
      const float* p = a.rows + ((int64_t)wave * a.n_heads + kv * a.rep + r) * q.n_tokens + t0 + row0;
      i32x4_t d;
      const uint64_t at = reinterpret_cast<uint64_t>(p);
      d[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)at);
      d[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
      d[2] = __builtin_amdgcn_readfirstlane(4 * min(n - row0, kKeys));
      d[3] = 0x00020000;
      copy4_lds(to + 2 * kTile + 256 * wave, d, 4 * lane);
    }
  };
  uint32_t buf = lds, other = lds + kBuf;
  int i = split * share;
  if (i < total) copy(i, buf);
  int q0 = (first + i % per_head) * kKeys;
  auto arrive = [&]() {
    wait_copies<0>();
    wait_lds_reads();
    ring_barrier();
    if (i + 1 < total) copy(i + 1, other);
  };
  auto leave = [&]() {
    const uint32_t t = buf;
    buf = other;
    other = t;
    ++i;
    q0 += kKeys;
    if (q0 >= n) q0 = first * kKeys;
  };
  // p and ds of 32 tokens
  auto slopes = [&](int qb, f32x16_t& s, f32x16_t& ds) {
    s = zeros16();
    ds = zeros16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s = T16<T>::mfma32(rd.template rows<v8>(buf, qb, ks), kr[ks], s);
      ds = T16<T>::mfma32(rd.template rows<v8>(buf + kTile, qb, ks), vr[ks], ds);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t at = buf + 2 * kTile + 4 * (32 * qb + 8 * g + 4 * h);
      const f32x4_t lse = *(LDS_AS const f32x4_t*)(uintptr_t)at, D = *(LDS_AS const f32x4_t*)(uintptr_t)(at + 256);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * g + e;
        s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.scale2, kShift - lse[e]));
        ds[r] = s[r] * (ds[r] - D[e]);
      }
    }
  };
  // blocks qb0 .. 1 of any tile
  auto any_tile = [&]<bool FINITE>(int qb0) {
#pragma unroll 1
    for (int qb = qb0; qb < 2; ++qb) {
      f32x16_t s, ds;
      slopes(qb, s, ds);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        // from the key's own token to the sequence's end
        const bool seen = (uint32_t)(q0 + 32 * qb + 8 * (r >> 2) + 4 * h + (r & 3) - key) < (uint32_t)(n - key);
        s[r] = seen ? s[r] : 0.0f;
        ds[r] = seen ? ds[r] : 0.0f;
      }
      if (!sc.fits(ds)) sc.shrink(dk);
      sc.apply(ds);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        add_columns<T, HD, FINITE>(dv, rd, buf + kTile, 2 * qb + x, pack8<T>(s, x));
        add_columns<T, HD, FINITE>(dk, rd, buf, 2 * qb + x, pack8<T>(ds, x));
      }
    }
    if constexpr (FINITE) {
      add_none<T, HD>(dv, rd, buf + kTile, max(key - q0, 0), n - q0);
      add_none<T, HD>(dk, rd, buf, max(key - q0, 0), n - q0);
    }
  };
  // Tiles of 64 tokens that see all of the wave's keys: those from q0 = w0 + 31 on, but for one that the sequence ends
  // in.  (Rows behind it are zeros in LDS, but zero times a key that is no number is none.)  One comparison: with
  // two the compiler spilled in the loop (four sequences of 2048 618 -> 753 us).
  const uint32_t whole = max(n - kKeys - w0 - 30, 0);
  while (i < total) {
    arrive();
    int qb0 = 0;
    while (i < total && (uint32_t)(q0 - w0 - 31) < whole) {
      bool stop = false;
#pragma unroll
      for (int qb = 0; qb < 2; ++qb) {
        f32x16_t s, ds;
        slopes(qb, s, ds);
        if (!sc.fits(ds)) {
          qb0 = qb;
          stop = true;
          break;
        }
        sc.apply(ds);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          add_columns<T, HD, false>(dv, rd, buf + kTile, 2 * qb + x, pack8<T>(s, x));
          add_columns<T, HD, false>(dk, rd, buf, 2 * qb + x, pack8<T>(ds, x));
        }
      }
      if (stop) break;
      leave();
      if (i < total) arrive();
    }
    if (i >= total) break;
    if (q0 + kKeys > w0) {
      // on the diagonal, the last one, or out of range
      const bool none = q0 < w0 + 31 && (tile_has_none<T, HD>(buf) || tile_has_none<T, HD>(buf + kTile));
      if (none) any_tile.template operator()<true>(qb0);
      else any_tile.template operator()<false>(qb0);
    }
    leave();
  }
  if (key >= n) return;
  const float back = kScaled<T> ? 0x1p-14f : 1.0f;
  if (a.splits > 1) {
    const int64_t plane = q.n_tokens * a.n_kv * HD;
    float* to = a.part + 2 * split * plane + ((t0 + key) * a.n_kv + kv) * HD;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int ch = channel_of<HD>(c, 8 * g + 4 * h);
        const float f = a.scale * back / sc.up;
        f32x4_t x, y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = dk[c][4 * g + e] * f;
          y[e] = dv[c][4 * g + e] * back;
        }
        *reinterpret_cast<f32x4_t*>(to + ch) = x;
        *reinterpret_cast<f32x4_t*>(to + plane + ch) = y;
      }
    return;
  }
  store_row<T, HD>(a.dK + (t0 + key) * a.lddk + (int64_t)kv * HD, dk, a.scale * back / sc.up);
  store_row<T, HD>(a.dV + (t0 + key) * a.lddv + (int64_t)kv * HD, dv, back);
}

// dK and dV of a tile of keys: its splits' parts in order
template <typename T, int HD>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs a, PromptBatch q) {
  const int u = blockIdx.x / a.n_kv, kv = blockIdx.x - u * a.n_kv;
  int b, level;
  if (!tile_at(q, u, b, level)) return;
  int64_t t0;
  int n;
  q.span_of(b, t0, n);
  level = __builtin_amdgcn_readfirstlane(level);
  const int k0 = ((n + kRows - 1) / kRows - 1 - level) * kRows;
  const int64_t plane = q.n_tokens * a.n_kv * HD;
  for (int v = threadIdx.x; v < kRows * HD / 8; v += 256) {
    const int key = k0 + v / (HD / 8), ch = 8 * (v % (HD / 8));
    if (key >= n) break;
    const float* from = a.part + ((t0 + key) * a.n_kv + kv) * HD + ch;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float s[8], x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = 0.0f;
#pragma unroll 4
      for (int z = 0; z < a.splits; ++z) {
        load_f32<8>(from + (2 * z + y) * plane, true, 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += x[e];
      }
      uint16_t* out = y ? a.dV + (t0 + key) * a.lddv : a.dK + (t0 + key) * a.lddk;
      store_n<T, 8>(out + (int64_t)kv * HD + ch, true, 8, s);
    }
  }
}

// ---------------------------------------------------------------- host side
struct HeadRows {
  const void* p;
  int64_t ld;
  int heads;
};
static bool head_rows_ok(const HeadRows& r, int hd) {
  return r.p && (reinterpret_cast<uintptr_t>(r.p) & 15) == 0 && r.ld % 8 == 0 && r.ld < kMaxPitch && r.ld >= (int64_t)r.heads * hd;
}
// Do two arrays share a value?  Rows of one pitch that lie apart inside the pitch
// (queries, keys and values of one fused row) do not.
static bool heads_meet(const HeadRows& a, const HeadRows& b, int64_t m, int hd) {
  if (!a.p || !b.p) return false;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t na = rows_bytes(m, a.ld, (int64_t)a.heads * hd, 2), nb = rows_bytes(m, b.ld, (int64_t)b.heads * hd, 2);
  if (x >= y + nb || y >= x + na) return false;
  if (a.ld != b.ld) return true;
  const uint64_t pitch = 2 * a.ld, wa = 2ull * a.heads * hd, wb = 2ull * b.heads * hd;
  const uint64_t d = x >= y ? (x - y) % pitch : (pitch - (y - x) % pitch) % pitch;   // a's row behind b's
  return !(d >= wb && d + wa <= pitch);
}
static bool heads_meet(const HeadRows& a, int64_t m, int hd, const void* p, uint64_t bytes) {
  return share_bytes(a.p, rows_bytes(m, a.ld, (int64_t)a.heads * hd, 2), p, bytes);
}

static bool prompt_ok(gptq_dtype t, int64_t n_tokens, int n_heads, int n_kv, int hd, int n_seqs, int max_len, float scale) {
  if (t != GPTQ_F16 && t != GPTQ_BF16) return false;
  if (n_tokens < 0 || n_tokens > INT_MAX || n_heads <= 0 || n_kv <= 0 || n_heads % n_kv != 0 || (hd != 64 && hd != 128)) return false;
  if ((int64_t)n_heads * hd >= kMaxPitch || n_seqs <= 0 || n_seqs == INT_MAX || max_len < 0 || (max_len == 0 && n_tokens > 0)) return false;
  return fabsf(scale) <= 1e8f;
}
// tiles of 128 tokens that n_tokens in n_seqs sequences can have
static int64_t tile_bound(int64_t n_tokens, int n_seqs, int64_t max_len) {
  return std::min((n_tokens + kRows - 1) / kRows + n_seqs - 1, n_seqs * ((max_len + kRows - 1) / kRows));
}

// Workgroups that share the tokens of a tile of keys: up to four a CU in all, up to
// eight, with four tiles of tokens each at least.  A few long sequences of few kv heads
// leave most of the chip idle otherwise.  Whole passes, us, four query heads to a kv head, of 13 ragged
// sequences up to 2900 of 4 kv heads / one of 2048 of 2, 4 and 8 kv heads / one of 4096 of 1 / of 512 of 2:
// as here 179 / 143 166 242 / 224 / 76, unsplit 391 / 374 376 383 / 701 / 123; up to four parts 180 / 165 171
// 206 / 284 / 73, up to 16 179 / 167 214 243 / 228 / 76; up to two workgroups a CU 249 / 144 170 216 / 225 / 76,
// eight 170 / 143 166 248 / 224 / 76.  Two tiles a part at least, four and eight: 512 tokens 76, 76 and 73,
// 300 of 4 kv heads 70, 67 and 78, eight of 128 29, 33 and 35.  The parts hold a row for each row
// of the batch, in sequences or not, so
// their number is what kPartRows rows of one kv head's dK and dV leave room for.
constexpr int64_t kPartRows = 1024 * kRows;
static int key_splits(int64_t tiles, int64_t n_tokens, int n_kv, int rep, int64_t max_len) {
  const int64_t s = std::min<int64_t>(1023 / (tiles * n_kv), rep * ((max_len + kKeys - 1) / kKeys) / 4);
  return (int)std::max<int64_t>(1, std::min({s, (int64_t)8, kPartRows / (n_tokens * n_kv)}));
}
static size_t rows_part(int64_t n_tokens, int n_heads) { return align_up((size_t)2 * n_heads * n_tokens * sizeof(float)); }

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_prompt_attention(const void* Q, const void* K, const void* V, gptq_dtype dtype, int64_t n_tokens, int32_t n_heads,
                                     int32_t n_kv_heads, int32_t head_dim, int64_t ldq, int64_t ldk, int64_t ldv,
                                     const int32_t* q_start, int32_t n_seqs, int32_t max_len, float scale, void* out, int64_t ldo,
                                     float* lse, hipStream_t s) {
  if (!prompt_ok(dtype, n_tokens, n_heads, n_kv_heads, head_dim, n_seqs, max_len, scale)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  max_len = (int32_t)std::min<int64_t>(max_len, n_tokens);      // (the kernels round it up to whole tiles in 32 bits)
  const HeadRows q{Q, ldq, n_heads}, k{K, ldk, n_kv_heads}, v{V, ldv, n_kv_heads}, o{out, ldo, n_heads};
  for (const HeadRows& r : {q, k, v, o})
    if (!head_rows_ok(r, head_dim)) return GPTQ_ERR_INVALID_ARG;
  if (!q_start || ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(lse)) & 3)) return GPTQ_ERR_INVALID_ARG;
  const uint64_t lse_bytes = (uint64_t)n_tokens * n_heads * sizeof(float), start_bytes = ((uint64_t)n_seqs + 1) * sizeof(int32_t);
  for (const HeadRows& r : {q, k, v})
    if (heads_meet(o, r, n_tokens, head_dim)) return GPTQ_ERR_INVALID_ARG;
  for (const HeadRows& r : {q, k, v, o})
    if (heads_meet(r, n_tokens, head_dim, lse, lse_bytes)) return GPTQ_ERR_INVALID_ARG;
  if (heads_meet(o, n_tokens, head_dim, q_start, start_bytes) || share_bytes(lse, lse_bytes, q_start, start_bytes)) return GPTQ_ERR_INVALID_ARG;
  const int64_t grid = tile_bound(n_tokens, n_seqs, max_len) * n_heads;
  if (grid > (1 << 24) - 1) return GPTQ_ERR_INVALID_ARG;
  PromptArgs a{};
  a.Q = static_cast<const uint16_t*>(Q); a.K = static_cast<const uint16_t*>(K); a.V = static_cast<const uint16_t*>(V);
  a.out = static_cast<uint16_t*>(out); a.lse = lse;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldo = ldo;
  a.n_heads = n_heads; a.n_kv = n_kv_heads; a.rep = n_heads / n_kv_heads;
  a.scale = scale; a.scale2 = fabsf(scale) * kLog2e; a.flip = scale < 0.0f ? 0x80008000u : 0u;
  const PromptBatch b{q_start, n_tokens, n_seqs, max_len};
  auto go = [&]<typename T, int HD>() { prompt_forward_kernel<T, HD><<<(unsigned)grid, 64 * kPromptWaves, 0, s>>>(a, b); };
  if (dtype == GPTQ_BF16) head_dim == 128 ? go.template operator()<__bf16, 128>() : go.template operator()<__bf16, 64>();
  else head_dim == 128 ? go.template operator()<_Float16, 128>() : go.template operator()<_Float16, 64>();
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

extern "C" size_t gptq_prompt_attention_backward_workspace_size(int64_t n_tokens, int32_t n_heads) {
  if (n_tokens <= 0 || n_tokens > INT_MAX || n_heads <= 0 || n_heads >= kMaxPitch) return 0;
  return rows_part(n_tokens, n_heads) + align_up((size_t)std::min<int64_t>(8 * n_tokens * n_heads, kPartRows) * 2 * 128 * sizeof(float));
}

extern "C" int gptq_prompt_attention_backward(const void* dOut, int64_t lddo, const void* Q, const void* K, const void* V,
                                              gptq_dtype dtype, int64_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                                              int32_t head_dim, int64_t ldq, int64_t ldk, int64_t ldv, const void* out, int64_t ldo,
                                              const float* lse, const int32_t* q_start, int32_t n_seqs, int32_t max_len, float scale,
                                              void* dQ, int64_t lddq, void* dK, int64_t lddk, void* dV, int64_t lddv, void* ws,
                                              size_t ws_bytes, hipStream_t s) {
  if (!prompt_ok(dtype, n_tokens, n_heads, n_kv_heads, head_dim, n_seqs, max_len, scale)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  max_len = (int32_t)std::min<int64_t>(max_len, n_tokens);      // (the kernels round it up to whole tiles in 32 bits)
  const HeadRows ins[] = {{dOut, lddo, n_heads}, {Q, ldq, n_heads}, {K, ldk, n_kv_heads}, {V, ldv, n_kv_heads}, {out, ldo, n_heads}};
  const HeadRows outs[] = {{dQ, lddq, n_heads}, {dK, lddk, n_kv_heads}, {dV, lddv, n_kv_heads}};
  for (const HeadRows& r : ins)
    if (!head_rows_ok(r, head_dim)) return GPTQ_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (!head_rows_ok(outs[i], head_dim)) return GPTQ_ERR_INVALID_ARG;
    for (const HeadRows& r : ins)
      if (heads_meet(outs[i], r, n_tokens, head_dim)) return GPTQ_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (heads_meet(outs[i], outs[j], n_tokens, head_dim)) return GPTQ_ERR_INVALID_ARG;
  }
  if (!lse || !q_start || ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(lse)) & 3)) return GPTQ_ERR_INVALID_ARG;
  const uint64_t lse_bytes = (uint64_t)n_tokens * n_heads * sizeof(float), start_bytes = ((uint64_t)n_seqs + 1) * sizeof(int32_t);
  for (const HeadRows& r : outs)
    if (heads_meet(r, n_tokens, head_dim, lse, lse_bytes) || heads_meet(r, n_tokens, head_dim, q_start, start_bytes)) return GPTQ_ERR_INVALID_ARG;
  const int64_t tiles = tile_bound(n_tokens, n_seqs, max_len);
  if (tiles * n_heads > (1 << 24) - 1) return GPTQ_ERR_INVALID_ARG;
  const size_t need = gptq_prompt_attention_backward_workspace_size(n_tokens, n_heads);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  for (const HeadRows& r : ins)
    if (heads_meet(r, n_tokens, head_dim, ws, need)) return GPTQ_ERR_INVALID_ARG;
  for (const HeadRows& r : outs)
    if (heads_meet(r, n_tokens, head_dim, ws, need)) return GPTQ_ERR_INVALID_ARG;
  if (share_bytes(ws, need, lse, lse_bytes) || share_bytes(ws, need, q_start, start_bytes)) return GPTQ_ERR_INVALID_ARG;
  PromptArgs a{};
  auto c = [](const void* p) { return static_cast<const uint16_t*>(p); };
  a.Q = c(Q); a.K = c(K); a.V = c(V); a.dO = c(dOut); a.O = c(out);
  a.dQ = static_cast<uint16_t*>(dQ); a.dK = static_cast<uint16_t*>(dK); a.dV = static_cast<uint16_t*>(dV);
  a.lse = const_cast<float*>(lse); a.rows = static_cast<float*>(ws);
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.lddo = lddo; a.ldo = ldo; a.lddq = lddq; a.lddk = lddk; a.lddv = lddv;
  a.n_heads = n_heads; a.n_kv = n_kv_heads; a.rep = n_heads / n_kv_heads;
  a.scale = scale; a.scale2 = scale * kLog2e;
  a.splits = key_splits(tiles, n_tokens, n_kv_heads, a.rep, max_len);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + rows_part(n_tokens, n_heads));
  const PromptBatch b{q_start, n_tokens, n_seqs, max_len};
  auto go = [&]<typename T, int HD>() {
    prompt_dq_kernel<T, HD><<<(unsigned)(tiles * n_heads), 64 * kPromptWaves, 0, s>>>(a, b);
    prompt_dkv_kernel<T, HD><<<(unsigned)(tiles * n_kv_heads * a.splits), 64 * kPromptWaves, 0, s>>>(a, b);
    if (a.splits > 1) prompt_join_kernel<T, HD><<<(unsigned)(tiles * n_kv_heads), 256, 0, s>>>(a, b);
  };
  if (dtype == GPTQ_BF16) head_dim == 128 ? go.template operator()<__bf16, 128>() : go.template operator()<__bf16, 64>();
  else head_dim == 128 ? go.template operator()<_Float16, 128>() : go.template operator()<_Float16, 64>();
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}
