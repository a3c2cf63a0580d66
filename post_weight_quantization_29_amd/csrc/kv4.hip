// Attention over a paged cache held in 4 bits: gptq_kv4_append, gptq_kv4_read
// and gptq_kv4_attention.  A cached row (one token, one kv head) is head_dim
// 4-bit codes with a step and a minimum: x = lo + step * code.
#include "gemm16.h"
#include "kv4.h"
#include "w4_epilogue.h"

#include <climits>

namespace gptq {

// ---------------------------------------------------------------- append and read
// eight values of dtype DT at p as floats, and back
template <int DT> GPTQ_DEV void load8(const void* base, int64_t at, bool vec, float (&v)[8]) {
  if constexpr (DT == GPTQ_F32) load_f32<8>(static_cast<const float*>(base) + at, vec, 8, v);
  else if constexpr (DT == GPTQ_F16) load_n<_Float16, 8>(static_cast<const uint16_t*>(base) + at, vec, 8, v);
  else load_n<__bf16, 8>(static_cast<const uint16_t*>(base) + at, vec, 8, v);
}
template <int DT> GPTQ_DEV void store8(void* base, int64_t at, bool vec, const float (&v)[8]) {
  if constexpr (DT == GPTQ_F32) store_f32<8>(static_cast<float*>(base) + at, vec, 8, v);
  else if constexpr (DT == GPTQ_F16) store_n<_Float16, 8>(static_cast<uint16_t*>(base) + at, vec, 8, v);
  else store_n<__bf16, 8>(static_cast<uint16_t*>(base) + at, vec, 8, v);
}

constexpr float kF16Max = 65504.0f;

// f over the L (8 or 16) lanes of a row, by DPP: neighbours, pairs, mirrored
// halves of eight, mirrored rows of sixteen
template <int CTRL> GPTQ_DEV float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int L, typename F> GPTQ_DEV float row_fold(float v, F&& f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  if constexpr (L == 16) v = f(v, dpp<0x140>(v));
  return v;
}

// A wave takes one token: its rows of all kv heads, HD / 8 lanes per row (eight
// values each, 16 bytes), the row's minimum and maximum over those lanes.
// blockIdx.y: keys or values.  Bound by the chain of lookups (start, length, page)
// in front of the stores and by about 150 instructions a row: 4096 tokens of 8
// heads of 128 10 us, 4.3 us of them the bytes (12 us with an IEEE division per
// value and shuffles through LDS).
template <int DT, int HD>
__global__ __launch_bounds__(256) void kv4_append_kernel(KvDev c, KvBatch q, const void* __restrict__ K,
                                                         const void* __restrict__ V, int64_t ldk, int64_t ldv, bool vec) {
  constexpr int L = HD / 8, RPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= q.n_tokens) return;
  const void* src = blockIdx.y ? V : K;
  const int64_t ld = blockIdx.y ? ldv : ldk;
  const int b = seq_of_token(q.q_start, c.n_seqs, t);
  if (b < 0) return;                            // not the batch's: its row is not read either
  // the first rows are on their way while their place is looked up (two more
  // loads, each on the one before)
  float ahead[8];
  load8<DT>(src, t * ld + (int64_t)min(lane / L, c.n_kv - 1) * HD + 8 * (lane % L), vec, ahead);
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  const int64_t p = (int64_t)q.kv_len[b] - n_q + (t - t0);
  const int64_t row0 = kv_row(c, b, 0, p);
  if (row0 < 0) return;
  uint32_t* codes = blockIdx.y ? c.v_codes : c.k_codes;
  uint32_t* grid = blockIdx.y ? c.v_grid : c.k_grid;
  const int li = lane % L;
  for (int h0 = 0; h0 < c.n_kv; h0 += RPW) {
    const int h = h0 + lane / L;
    const bool in = h < c.n_kv;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ahead[e];
    if (h0 + RPW < c.n_kv) load8<DT>(src, t * ld + (int64_t)min(h + RPW, c.n_kv - 1) * HD + 8 * li, vec, ahead);
    // fmin and fmax pass NaNs over
    float mn = INFINITY, mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn = fminf(mn, x[e]);
      mx = fmaxf(mx, x[e]);
    }
    mn = row_fold<L>(mn, [](float u, float v) { return fminf(u, v); });
    mx = row_fold<L>(mx, [](float u, float v) { return fmaxf(u, v); });
    if (mn > mx) mn = mx = 0.0f;               // a row of NaNs
    // values beyond fp16 count as its largest
    mn = fminf(fmaxf(mn, -kF16Max), kF16Max);
    mx = fminf(fmaxf(mx, -kF16Max), kF16Max);
    const _Float16 lo16 = (_Float16)mn;
    const float lo = (float)lo16;
    const _Float16 st16 = (_Float16)(fmaxf(mx - lo, 0.0f) / 15.0f);
    const float st = (float)st16, inv = st > 0.0f ? 1.0f / st : 0.0f;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // a NaN clamps to the lowest value: code 0
      const float y = fminf(fmaxf(x[e], -kF16Max), kF16Max) - lo;
      // y / st correctly rounded: a quotient from the correctly rounded
      // reciprocal, corrected twice by its exact remainder (Markstein)
      float r = y * inv;
      r = fmaf(fmaf(-st, r, y), inv, r);
      r = fmaf(fmaf(-st, r, y), inv, r);
      w |= (uint32_t)fminf(fmaxf(rintf(r), 0.0f), 15.0f) << (4 * e);
    }
    if (in) {
      const int64_t row = row0 + (int64_t)h * c.page;
      codes[row * L + li] = w;
      if (li == 0)
        grid[row] = (uint32_t)__builtin_bit_cast(uint16_t, st16) | (uint32_t)__builtin_bit_cast(uint16_t, lo16) << 16;
    }
  }
}

template <int DT, int HD>
__global__ __launch_bounds__(256) void kv4_read_kernel(KvDev c, KvBatch q, void* __restrict__ K, void* __restrict__ V,
                                                       bool vec) {
  constexpr int L = HD / 8, RPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  void* dst = blockIdx.y ? V : K;
  if (t >= q.n_tokens || !dst) return;
  const int b = seq_of_token(q.q_start, c.n_seqs, t);
  if (b < 0) return;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  const int64_t row0 = kv_row(c, b, 0, (int64_t)q.kv_len[b] - n_q + (t - t0));
  const uint32_t* codes = blockIdx.y ? c.v_codes : c.k_codes;
  const uint32_t* grid = blockIdx.y ? c.v_grid : c.k_grid;
  const int li = lane % L;
  for (int h = lane / L; h < c.n_kv; h += RPW) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (row0 >= 0) {
      const int64_t row = row0 + (int64_t)h * c.page;
      const uint32_t w = codes[row * L + li], g = grid[row];
      const float st = grid_step(g), lo = grid_lo(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = lo + st * (float)((w >> (4 * e)) & 15u);
    }
    store8<DT>(dst, (t * c.n_kv + h) * HD + 8 * li, vec, x);
  }
}

// ---------------------------------------------------------------- attention
struct AttnArgs {
  const uint16_t* Q;
  uint16_t* out;
  int64_t ldq, ldo;
  int n_heads, rep;            // query heads, query heads per kv head
  int max_q, max_kv;
  float scale2;                // |scale| * log2(e), at least 1e-30
  float lazy;                  // kLazy in units of q . k
  uint32_t q_flip;             // sign bits to flip in Q (a negative scale)
  int chunk, n_chunks;         // keys per workgroup; 1 chunk: no partial results
  int row_tiles;
  float* part_o;               // [chunk][token][head][HD], not normalized
  float2* part_ml;             // [chunk][token][head]: maximum (log2 units), sum
};

constexpr float kNoMax = -1.0e30f;    // running maximum of a row that has seen nothing
constexpr float kMaxScale = 1.0e8f;   // kNoMax times scale2 stays finite
// A row's reference maximum follows the true one only when some row of the
// wave has outgrown its own by 2^8: the terms stay below 2^8 (2^9 with fp16's
// steps), and most tiles rescale nothing.
constexpr float kLazy = 8.0f;

// Few rows (a query row is one new token's one query head; a sequence has
// n_q * rep rows per kv head): a workgroup takes 16 rows against `chunk` keys,
// its four waves in turn 32 keys a step, all in registers.
//
// Scores are formed transposed, S^T[key][row] = K Q^T, on v_mfma_f32_16x16x32
// with the codes themselves as operand (16 + code, exact): operand lane l is
// key l % 16 with the eight codes of one packed word, and
//   q . k = step (D - 16 sum(q)) + lo sum(q),  D = sum_i q_i (16 + code_i).
// The result leaves lane l = 16 g + i with row i's keys 4g .. 4g + 3 of both
// 16-key tiles, which are the eight k-slots that the second product's operand
// wants of lane (i, g): O^T[d][row] = V^T P^T, with step_j folded into p_j and
// the keys of V's operand in the same order, so the softmax's numbers never
// change lanes.  p_j step_j goes in as two bf16 pieces (16 bits: the rounding
// stays far below an fp16 output's), sum_j p_j (lo_j - 16 step_j) is one number
// per row.  V's operand needs eight keys of one channel per lane: the lane
// loads the packed words of its eight keys, pairs of words are zipped by
// v_perm, and every code is then one shift and one and-or away.
//
// A step of 32 keys is 322 vector instructions, 374 with masks, which a tile of
// fewer than 16 rows always takes (its missing rows see nothing), and 4.3 KB of
// cache (head_dim 128); its loads are in flight while the step before is
// computed.  Measured, 64 query heads on 8: one sequence of 131072 positions 38 us
// (3.8 TB/s), 48 of 1 to 8192 31 us.  Neither bound is reached: the counters show
// 1.5 and 1.1 waves a SIMD on average, vector issue in 51 and 33 % of the cycles
// and waves waiting for 42 and 35 % of their time.  What costs the rest are the
// dependent loads in front of the first step (start, length, page, codes), a wave's
// few steps (four of a chunk of 512), and a second, partly filled round.
template <typename T, int HD>
__global__ __launch_bounds__(256, 3) void kv4_rows_kernel(AttnArgs a, KvDev c, KvBatch q) {
  typedef typename T16<T>::v8 v8;
  typedef typename T16<__bf16>::v8 b8;
  constexpr int KW = HD / 32;          // packed words of a key per lane
  constexpr int NJ = HD / 16;          // V products per step
  constexpr int RW = HD / 8;           // words per row
  __shared__ __attribute__((aligned(16))) float sO[4][16][HD + 4];
  __shared__ float sM[4][16], sL[4][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  // x: chunks, the row tiles and kv heads of one chunk next to each other
  const int per = c.n_kv * a.row_tiles;
  const int ch = blockIdx.x / per, b = blockIdx.y + 32768 * blockIdx.z;
  const int rt = (blockIdx.x % per) / c.n_kv, h = (blockIdx.x % per) % c.n_kv;
  if (b >= c.n_seqs) return;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  const int64_t first = (int64_t)q.kv_len[b] - n_q;       // position of the first new token
  n_q = min(n_q, a.max_q);
  const int rows = n_q * a.rep;
  if (rt * 16 >= rows) return;
  const int64_t most = min((int64_t)a.max_kv, (int64_t)c.max_pages * c.page);
  // this lane's row: token ti, head hq; it sees positions [0, seen)
  const int row = rt * 16 + i;
  const int ti = min(row, rows - 1) / a.rep, hq = h * a.rep + min(row, rows - 1) % a.rep;
  const int seen = row < rows ? (int)max(min(first + ti + 1, most), (int64_t)0) : 0;
  // the tile's longest row
  const int seen_max = (int)max(min(first + (min(rt * 16 + 15, rows - 1) / a.rep) + 1, most), (int64_t)0);
  const int c0 = ch * a.chunk;
  if (ch > 0 && c0 >= seen_max) return;

  // Q in the order of a word's codes, and the sum of its row
  v8 qv[KW];
  float qsum = 0.0f;
  {
    const uint16_t* qp = a.Q + (t0 + ti) * a.ldq + (int64_t)hq * HD + 8 * KW * g;
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      uint4 v = *reinterpret_cast<const uint4*>(qp + 8 * j);
      v.x ^= a.q_flip; v.y ^= a.q_flip; v.z ^= a.q_flip; v.w ^= a.q_flip;
      qsum += (lo16f<T>(v.x) + hi16f<T>(v.x)) + (lo16f<T>(v.y) + hi16f<T>(v.y)) +
              ((lo16f<T>(v.z) + hi16f<T>(v.z)) + (lo16f<T>(v.w) + hi16f<T>(v.w)));
      qv[j] = __builtin_bit_cast(v8, code_order(v));
    }
    qsum += __shfl_xor(qsum, 16);
    qsum += __shfl_xor(qsum, 32);
  }
  const float qbase = -kCodeBase * qsum;

  // wave w takes the steps of 32 keys w, w + 4, ...
  const int k_end = min(c0 + a.chunk, seen_max), kw0 = c0 + 32 * wave;
  const int steps = k_end > kw0 ? (k_end - kw0 + 127) >> 7 : 0;
  // lane l: the cache row of 16-key block l % 2 of this wave's step l / 2, -1 if there is none
  int tile_row = -1;
  {
    const int p = kw0 + 128 * (lane >> 1) + 16 * (lane & 1);
    if (p < k_end) tile_row = kv_row(c, b, h, p);
  }

  // a step's packed words and grids; each half is loaded again as soon as it
  // has been used, so its loads are in flight during the other half's work
  uint32_t kw[2][KW], vw[8];
  uint4 kg[2], vg[2];
  auto row_of = [&](int st, int u) { return (uint32_t)max(__builtin_amdgcn_readlane(tile_row, 2 * st + u), 0); };
  const uint32_t k_off = 4 * (i * RW + KW * g), v_off = 4 * (4 * g * RW + (i % RW));     // bytes
  auto load_k = [&](int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t r = row_of(st, u);
      const char* kp = reinterpret_cast<const char*>(c.k_codes + (size_t)r * RW);
      if constexpr (KW == 4) *reinterpret_cast<uint4*>(kw[u]) = *reinterpret_cast<const uint4*>(kp + k_off);
      else *reinterpret_cast<uint2*>(kw[u]) = *reinterpret_cast<const uint2*>(kp + k_off);
      kg[u] = *reinterpret_cast<const uint4*>(c.k_grid + r + 4 * g);
    }
  };
  auto load_v = [&](int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t r = row_of(st, u);
      const char* vp = reinterpret_cast<const char*>(c.v_codes + (size_t)r * RW);
#pragma unroll
      for (int e = 0; e < 4; ++e) vw[4 * u + e] = *reinterpret_cast<const uint32_t*>(vp + v_off + 4 * e * RW);
      vg[u] = *reinterpret_cast<const uint4*>(c.v_grid + r + 4 * g);
    }
  };

  f32x4_t o[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) o[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNoMax, l = 0.0f, base = 0.0f, sum_w = 0.0f;
  if (steps > 0) {
    load_k(0);
    load_v(0);
  }
  // Everything before the exponential is in units of q . k: the row's sum in
  // the accumulator's start takes 16 sum(q) off, and step and lo multiply as
  // the fp16 halves they are stored as (two mixed instructions a score).
  // WHOLE: every row sees all 32 keys.
  auto turn = [&]<bool WHOLE>(int st) {
    const int kb = kw0 + 128 * st;
    float s[8];
    bool ok[8];
    float mt = m;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t d = f32x4_t{qbase, qbase, qbase, qbase};
#pragma unroll
      for (int j = 0; j < KW; ++j) d = T16<T>::mfma16(__builtin_bit_cast(v8, code_word<T>(kw[u][j])), qv[j], d);
      const uint32_t gw[4] = {kg[u].x, kg[u].y, kg[u].z, kg[u].w};
      const bool there = WHOLE || __builtin_amdgcn_readlane(tile_row, 2 * st + u) >= 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = 4 * u + r;
        // what lies behind a row's end or on a missing page may be anything
        ok[e] = WHOLE || (there && kb + 16 * u + 4 * g + r < seen);
        s[e] = fma_lo(gw[r], d[r], fma_hi(gw[r], qsum, 0.0f));
        if constexpr (!WHOLE) s[e] = ok[e] ? s[e] : -INFINITY;
        mt = fmaxf(mt, s[e]);
      }
    }
    if (st + 1 < steps) load_k(st + 1);
    mt = fmaxf(mt, __shfl_xor(mt, 16));
    mt = fmaxf(mt, __shfl_xor(mt, 32));
    if (__any(mt > m + a.lazy)) {
      const float al = __builtin_amdgcn_exp2f((m - mt) * a.scale2);
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[j] *= al;
      l *= al;
      base *= al;
      sum_w *= al;
      m = mt;
    }
    const float off = -m * a.scale2;
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t gw[4] = {vg[u].x, vg[u].y, vg[u].z, vg[u].w};
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const int e = 4 * u + r;
        float p[2], w[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t gr = ok[e + y] ? gw[r + y] : 0u;
          p[y] = __builtin_amdgcn_exp2f(fmaf(s[e + y], a.scale2, off));
          l += p[y];
          base = fma_hi(gr, p[y], base);
          w[y] = fma_lo(gr, p[y], 0.0f);
          sum_w += w[y];
        }
        ph[e / 2] = pack2<__bf16>(w[0], w[1]);
        pl[e / 2] = pack2<__bf16>(w[0] - lo16f<__bf16>(ph[e / 2]), w[1] - hi16f<__bf16>(ph[e / 2]));
      }
    }
    const b8 hv = __builtin_bit_cast(b8, make_uint4(ph[0], ph[1], ph[2], ph[3]));
    const b8 lv = __builtin_bit_cast(b8, make_uint4(pl[0], pl[1], pl[2], pl[3]));
    // zipped words: halves of key pairs
    uint32_t z[HD == 128 ? 2 : 1][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (HD == 128) {
        z[0][e] = __builtin_amdgcn_perm(vw[2 * e + 1], vw[2 * e], 0x05040100u);
        z[HD == 128 ? 1 : 0][e] = __builtin_amdgcn_perm(vw[2 * e + 1], vw[2 * e], 0x07060302u);
      } else {
        z[0][e] = __builtin_amdgcn_perm(vw[2 * e + 1], vw[2 * e], i < 8 ? 0x05040100u : 0x07060302u);
      }
    }
    if (st + 1 < steps) load_v(st + 1);
    auto pv = [&]<int J>() {
      constexpr int zi = J / 4, K = J % 4;
      const b8 vv = __builtin_bit_cast(b8, make_uint4(code_pair<__bf16, K>(z[zi][0]), code_pair<__bf16, K>(z[zi][1]),
                                                      code_pair<__bf16, K>(z[zi][2]), code_pair<__bf16, K>(z[zi][3])));
      o[J] = T16<__bf16>::mfma16(vv, hv, o[J]);
      o[J] = T16<__bf16>::mfma16(vv, lv, o[J]);
    };
    [&]<int... J>(std::integer_sequence<int, J...>) { (pv.template operator()<J>(), ...); }(std::make_integer_sequence<int, NJ>{});
  };
  // the steps in front that need no masks (all their pages there, all their
  // keys seen by the tile's shortest row)
  const int seen_min = rt * 16 + 15 < rows ? (int)max(min(first + (rt * 16) / a.rep + 1, most), (int64_t)0) : 0;
  int plain = max(0, min(steps, (seen_min - kw0 + 96) >> 7));
  const uint64_t missing = __ballot(tile_row < 0);
  if (missing) plain = min(plain, (__ffsll((unsigned long long)missing) - 1) >> 1);
  for (int st = 0; st < plain; ++st) turn.template operator()<true>(st);
  for (int st = plain; st < steps; ++st) turn.template operator()<false>(st);
  base = fmaf(-kCodeBase, sum_w, base);
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  base += __shfl_xor(base, 16);
  base += __shfl_xor(base, 32);
  // lane (i, g), register r: operand row R = 4g + r of V, which is channels
  // 8R + j (head_dim 128), or 8 (R % 8) + 4 (R / 8) + j (64)
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int R = 4 * g + r;
#pragma unroll
    for (int j = 0; j < NJ; j += 4) {
      const f32x4_t v = {o[j][r] + base, o[j + 1][r] + base, o[j + 2][r] + base, o[j + 3][r] + base};
      *reinterpret_cast<f32x4_t*>(&sO[wave][i][HD == 128 ? 8 * R + j : 8 * (R & 7) + 4 * (R >> 3)]) = v;
    }
  }
  if (g == 0) {
    sM[wave][i] = m * a.scale2;
    sL[wave][i] = l;
  }
  __syncthreads();
  // join the waves: thread (row, 1/16 of the channels)
  const int jr = tid >> 4, row2 = rt * 16 + jr;
  if (row2 >= rows) return;
  const int64_t tok = t0 + row2 / a.rep;
  const int head = h * a.rep + row2 % a.rep;
  float mm = sM[0][jr];
#pragma unroll
  for (int w = 1; w < 4; ++w) mm = fmaxf(mm, sM[w][jr]);
  float ll = 0.0f, v[HD / 16];
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) v[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float al = __builtin_amdgcn_exp2f(sM[w][jr] - mm);
    ll = fmaf(al, sL[w][jr], ll);
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) v[e] = fmaf(al, sO[w][jr][(HD / 16) * (tid & 15) + e], v[e]);
  }
  // rows of one chunk need no joining
  const int64_t seen2 = min(first + row2 / a.rep + 1, most);
  if (seen2 > a.chunk) {
    if (c0 >= seen2) return;
    const int64_t at = ((int64_t)ch * q.n_tokens + tok) * a.n_heads + head;
#pragma unroll
    for (int e = 0; e < HD / 16; e += 4)
      *reinterpret_cast<float4*>(a.part_o + at * HD + (HD / 16) * (tid & 15) + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    if ((tid & 15) == 0) a.part_ml[at] = make_float2(mm, ll);
  } else if (ch == 0) {
    const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;       // a row that saw nothing is 0; NaN stays
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) v[e] *= inv;
    store_n<T, HD / 16>(a.out + tok * a.ldo + (int64_t)head * HD + (HD / 16) * (tid & 15), true, HD / 16, v);
  }
}

// Many rows (prompts): a workgroup takes 192 rows, 16 to each of twelve waves,
// and walks the keys in tiles of 64.  A tile's codes are unpacked once for the
// twelve: keys as 16 + code rows in the activations' type (waves 0..3), values
// transposed in bf16 (waves 4..7; channel rows, the keys of a 16-byte chunk in
// the order in which the softmax's registers hold them), double buffered; the packed words come three tiles ahead.  Products
// and register layouts are those of kv4_rows_kernel.
//
// w_j = p_j step_j is rounded to bf16 (fp16 has not the range: steps may differ
// by 2^37, and a scale that fits the widest row seen would leave the others few
// bits), for bf16 inputs in one piece, for fp16 in two (16 bits), and what the
// rounding is multiplied with has to be of the values' own size, not 16 + code:
//   out = sum_j w_j ((16 + code_j) + lo_j / step_j - 16) / sum_j w_j / step_j
// with the rounded w_j in all three sums: the error is p's own, as if p had been
// rounded.  The last two sums are six more rows of V^T (lo / step - 16 and 1 /
// step, each in three bf16 pieces, 24 bits), so they cost two products a tile
// and piece and no vector instructions; a step of 0 counts as 1e-20.  Measured,
// the prompts below: bf16 231 us, fp16 with its second piece 278 us (241 us with
// one fp16 piece and the widest step's exponent, which cost the rows next to a
// wide one up to seven bits).  At head_dim 128 the 168 registers that three waves a
// SIMD leave are all taken; the bf16 kernel spills two.
//
// 16-byte LDS accesses serve 16 lanes a cycle: the swizzles give 16 consecutive
// rows of one chunk 16 different 16-byte columns of the 64 banks.
//
// 32 rows a wave on the 32 x 32 products read LDS half as often, but their 96
// accumulators leave two waves per SIMD, and the loop then waits for LDS more
// than it computes (279 us against 230 for 2565 tokens of 32 heads over
// 4613 positions); 16 rows fit three.  0.46 PFLOP/s: the matrix pipe is busy in 19 %
// of the cycles, vector issue (exponentials, rounding, unpacking again for every
// 192 rows) fills 38 %, and the waves wait for 41 % of their time, as all twelve
// meet at a tile's one barrier and eight of them unpack in front of it.
constexpr float kNoStep = 1e-20f;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
constexpr int kTileWaves = 12;
constexpr uint32_t kRawSlots = 4, kRawBytes = 1024 + 128;

template <typename T, int HD>
__global__ __launch_bounds__(64 * kTileWaves, kTileWaves / 4) void kv4_tile_kernel(AttnArgs a, KvDev c, KvBatch q) {
  typedef typename T16<T>::v8 v8;
  typedef typename T16<__bf16>::v8 b8;
  constexpr int RW = HD / 8;           // packed words per row
  constexpr int KS = HD / 32;          // k-slices of the first product
  constexpr int NJ = HD / 16;          // 16-channel blocks of the second
  constexpr int kPieces = T16<T>::kType == GPTQ_F16 ? 2 : 1;     // of a weight
  constexpr int TR = 16 * kTileWaves;
  // LDS: [buffer][keys 64 x HD | values HD x 64 | six rows x 64 | ks, kl, vs | there]
  constexpr uint32_t kOffV = 64 * HD * 2, kOffX = 2 * kOffV, kOffG = kOffX + 8 * 128, kOffThere = kOffG + 3 * 256, kBuf = kOffThere + 256;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kBuf + 8 * kRawSlots * kRawBytes];
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  // Row tiles by falling length, so that what is left for the end is short; the
  // heads shift by one from length to length: workgroups go to the XCDs in
  // turn, and 32 CUs of one XCD on one head's keys at the same time wait for
  // the same few lines of its L2 (369 us instead of 250).
  const uint32_t wg = blockIdx.y * gridDim.x + blockIdx.x;
  const int ch = wg % a.n_chunks;
  const int heads = c.n_kv * c.n_seqs;
  if (wg / a.n_chunks >= (uint32_t)heads * a.row_tiles) return;    // the last of the launch's rows is not full
  int id = wg / a.n_chunks;
  const int rt = a.row_tiles - 1 - id / heads;
  id = (id + rt) % heads;
  const int h = id % c.n_kv, b = id / c.n_kv;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  const int64_t first = (int64_t)q.kv_len[b] - n_q;
  n_q = min(n_q, a.max_q);
  const int rows = n_q * a.rep;
  if (rt * TR >= rows) return;
  const int64_t most = min((int64_t)a.max_kv, (int64_t)c.max_pages * c.page);
  auto seen_of = [&](int row) { return (int)max(min(first + row / a.rep + 1, most), (int64_t)0); };
  const int seen_max = seen_of(min(rt * TR + TR - 1, rows - 1));
  const int c0 = ch * a.chunk, c1 = min(c0 + a.chunk, seen_max);
  if (ch > 0 && c0 >= seen_max) return;
  // this wave's shortest and longest row (none: nothing to compute)
  const int w0 = rt * TR + 16 * wave;
  const int wmin = w0 < rows ? seen_of(w0) : 0, wmax = w0 < rows ? seen_of(min(w0 + 15, rows - 1)) : 0;
  const int row = w0 + i;
  const int seen = row < rows ? seen_of(row) : 0;
  v8 qv[KS];
  float qs2 = 0.0f;
  {
    const int64_t tok = t0 + min(row, rows - 1) / a.rep;
    const int hq = h * a.rep + min(row, rows - 1) % a.rep;
    const uint16_t* qp = a.Q + tok * a.ldq + (int64_t)hq * HD + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint4 v = *reinterpret_cast<const uint4*>(qp + 32 * s);
      v.x ^= a.q_flip; v.y ^= a.q_flip; v.z ^= a.q_flip; v.w ^= a.q_flip;
      qs2 += (lo16f<T>(v.x) + hi16f<T>(v.x)) + (lo16f<T>(v.y) + hi16f<T>(v.y)) +
             ((lo16f<T>(v.z) + hi16f<T>(v.z)) + (lo16f<T>(v.w) + hi16f<T>(v.w)));
      qv[s] = __builtin_bit_cast(v8, code_order(v));
    }
    qs2 += __shfl_xor(qs2, 16);
    qs2 += __shfl_xor(qs2, 32);
    qs2 *= a.scale2;
  }

  // chunk swizzles: key rows of HD / 8 chunks (256 or 128 bytes), channel rows of 8
  auto swz_k = [](int key) { return HD == 128 ? key & 15 : (key >> 1) & 7; };
  auto swz_v = [](int chn) { return ((chn >> 1) ^ (chn >> 4)) & 7; };

  // Staging.  Wave w < 4: keys 16 w .. 16 w + 15, 16 bytes (four words) per
  // lane.  Wave 4 + u: chunks 2u and 2u + 1 of the values; chunk 4t + y is the
  // keys 32 t + 4 y + 0..3 and 16 further, a lane takes one word column of
  // them and unpacks four of its channels.  head_dim 64 takes half the lanes.
  const bool is_k = wave < 4, is_v = wave >= 4 && wave < 8;
  const int u = wave & 3;
  const int kkey = HD == 128 ? lane >> 2 : (lane & 31) >> 1, kq = HD == 128 ? lane & 3 : lane & 1;
  const int vb = lane & (RW - 1), vz = (lane >> (HD == 128 ? 4 : 3)) & 1, vc = 2 * u + ((lane >> (HD == 128 ? 5 : 4)) & 1);
  const bool busy = HD == 128 || lane < 32;
  const uint32_t v_sel = vz ? 0x07060302u : 0x05040100u;
  // LDS offsets of the lane's first chunk each; the others flip or add constants
  const int key_t = 16 * u + kkey, vchn = 8 * vb + 4 * vz;
  const uint32_t s_at = is_k ? key_t * (2 * HD) + (((4 * kq) ^ swz_k(key_t)) << 4)
                             : kOffV + vchn * 128 + ((vc ^ swz_v(vchn)) << 4);
  const uint32_t x_at = kOffX + ((4 * (u >> 1) + ((lane >> 2) & 3)) << 4) + 2 * ((lane & 3) + 4 * (u & 1));
  const uint32_t g_at = kOffG + 4 * (16 * u + i);
  const int n0 = c0 >> 6, n1 = (c1 + 63) >> 6;
  // lane l: cache rows of this wave's 16-key blocks of tile row_base + l: its
  // grids' block u (keys: all it needs), and the other block of its chunks
  int rows_u = -1, rows_o = -1;
  int row_base = n0;
  auto fetch_rows = [&](int n) {
    const int p = 64 * (n + lane) + 16 * u, po = p ^ 16;
    row_base = n;
    rows_u = p < c1 ? kv_row(c, b, h, p) : -1;
    if (is_v) rows_o = po < c1 ? kv_row(c, b, h, po) : -1;
  };
  // The packed words of a tile go HBM -> LDS without registers, kAhead tiles
  // ahead, each wave its own (a wave waits for nobody else's): a slot holds 1 KB
  // of codes (values: 8 rows each of two blocks), 16 grid words, a flag.
  const uint32_t raw = lds + 2 * kBuf + (is_k || is_v ? wave : 0) * kRawSlots * kRawBytes;
  const uint32_t code_off = is_k ? 16 * lane : 16 * (lane & (2 * HD / 8 - 1)) + 8 * (u & 1) * (HD / 2);
  auto copy_tile = [&](int n) {
    if (!is_k && !is_v) return;
    const int nn = min(n, n1 - 1);       // past the end: the last one again, so that the counts below hold
    if (nn - row_base >= 64) fetch_rows(nn);
    const int ru = __builtin_amdgcn_readlane(rows_u, nn - row_base);
    const uint32_t r = (uint32_t)max(ru, 0), slot = raw + (n % kRawSlots) * kRawBytes;
    if (lane == 0) *(LDS_AS int*)(uintptr_t)(slot + 1024 + 64) = ru >= 0;
    auto from = [&](const uint32_t* p) {
      return tile_rsrc(reinterpret_cast<uint64_t>(p), true);
    };
    if (is_k) {
      const i32x4_t rs = from(c.k_codes + (size_t)r * RW);
      if (HD == 128 || lane < 32) copy16_lds(slot, rs, code_off);
    } else {
      const uint32_t ro = (uint32_t)max(__builtin_amdgcn_readlane(rows_o, nn - row_base), 0);
      const i32x4_t r0 = from(c.v_codes + (size_t)(u & 1 ? ro : r) * RW), r1 = from(c.v_codes + (size_t)(u & 1 ? r : ro) * RW);
      if (lane < 2 * HD / 8) {
        copy16_lds(slot, r0, code_off);
        copy16_lds(slot + 512, r1, code_off);
      }
    }
    const i32x4_t rg = from((is_k ? c.k_grid : c.v_grid) + r);
    if (lane < 16) copy4_lds(slot + 1024, rg, 4 * lane);
  };
  // tile n into an unpacked buffer; `later` tiles' copies are still in flight
  auto store = [&](int n, uint32_t buf) {
    if (!is_k && !is_v) return;
    if (is_k) wait_copies<2 * (kRawSlots - 2)>();
    else wait_copies<3 * (kRawSlots - 2)>();
    asm volatile("" ::: "memory");
    const uint32_t slot = raw + (n % kRawSlots) * kRawBytes;
    const bool g_there = *(LDS_AS const int*)(uintptr_t)(slot + 1024 + 64);
    const bool in = g_there && 64 * n + 16 * u + i < seen_max;
    // a key past the rows' end or on a missing page stands for zeros
    const uint32_t gg = in ? *(LDS_AS const uint32_t*)(uintptr_t)(slot + 1024 + 4 * i) : 0u;
    uint32_t gw[8];
    if (is_k) {
      const u32x4_t v = *(LDS_AS const u32x4_t*)(uintptr_t)(slot + 16 * (HD == 128 ? lane : lane & 31));
#pragma unroll
      for (int e = 0; e < 4; ++e) gw[e] = v[e];
    } else {
      const LDS_AS uint32_t* p = (const LDS_AS uint32_t*)(uintptr_t)(slot + (4 * (vc & 1) * RW + vb) * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gw[e] = p[e * RW];
        gw[4 + e] = p[128 + e * RW];
      }
    }
    auto put = [&](uint32_t at, uint4 v) { *(LDS_AS u32x4_t*)(uintptr_t)at = u32x4_t{v.x, v.y, v.z, v.w}; };
    // opaque, so that the flipped addresses are formed where they are used
    // instead of being kept in two dozen registers through the loop
    uint32_t sa = buf + s_at, xa = buf + x_at, ga = buf + g_at;
    asm volatile("" : "+v"(sa), "+v"(xa), "+v"(ga));
    auto grid = [&](int plane) -> LDS_AS float& { return *(LDS_AS float*)(uintptr_t)(ga + 256 * plane); };
    if (is_k) {
      if (busy) {
#pragma unroll
        for (int j = 0; j < 4; ++j) put(sa ^ (j << 4), code_word<T>(gw[j]));
      }
      if (lane < 16) {
        const float ks = grid_step(gg);
        grid(0) = ks * a.scale2;
        grid(1) = fmaf(-kCodeBase, ks, grid_lo(gg));
        if (lane == 0) ((LDS_AS int*)(uintptr_t)(buf + kOffThere))[u] = g_there;
      }
    } else {
      if (busy) {
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = __builtin_amdgcn_perm(gw[2 * e + 1], gw[2 * e], v_sel);
        auto column = [&]<int K>() {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = code_pair<__bf16, K>(z[e]);
          put((sa ^ ((K >> 1) << 4)) + 128 * K, make_uint4(w[0], w[1], w[2], w[3]));
        };
        column.template operator()<0>();
        column.template operator()<1>();
        column.template operator()<2>();
        column.template operator()<3>();
      }
      if (lane < 16) {
        // a row with a step or minimum that is no number reaches those that see it
        // through its step alone, as 0 times such an operand would reach all
        const bool number = fabsf(grid_step(gg)) < INFINITY && fabsf(grid_lo(gg)) < INFINITY;
        const float vr = grid_step(gg), vs = vr != 0.0f ? vr : kNoStep;
        grid(2) = number ? vs : NAN;
        // three pieces each of lo / step - 16 and 1 / step: rows 0..5, this key's slot of its chunk
        const float inv = 1.0f / vs;
        float x[2] = {number ? grid_lo(gg) * inv - kCodeBase : 0.0f, number ? inv : 0.0f};
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const int rr = 3 * y + p;
            const uint16_t bits = bits16<__bf16>(x[y]);
            x[y] -= (float)__builtin_bit_cast(__bf16, bits);
            *(LDS_AS uint16_t*)(uintptr_t)((xa ^ (rr << 4)) + 128 * rr) = bits;
          }
      }
    }
  };

  // Operand reads: slice s of a key row is chunk 4 s + g; the swizzle of channel
  // row 16 j + i differs from row i's by j, so each read is the lane's first
  // address with some bits flipped and a constant added.
  const uint32_t k_rd = i * (2 * HD) + ((g ^ swz_k(i)) << 4);
  const uint32_t v_rd = kOffV + i * 128 + ((g ^ swz_v(i)) << 4);
  const uint32_t x_rd = kOffX + (i & 7) * 128 + ((g ^ (i & 7)) << 4);

  f32x4_t o[NJ], ox = {0.0f, 0.0f, 0.0f, 0.0f};   // ox: the sums of V^T's extra rows
  float m = kNoMax;
#pragma unroll
  for (int j = 0; j < NJ; ++j) o[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  if (n0 < n1) {
    if (is_k || is_v) fetch_rows(n0);
#pragma unroll
    for (int e = 0; e < kRawSlots - 1; ++e) copy_tile(n0 + e);
    store(n0, lds);
  }
  __syncthreads();
  uint32_t buf = lds, other = lds + kBuf;
  int n = n0;
  auto there = [&](int w) { return ((const LDS_AS int*)(uintptr_t)(buf + kOffThere))[w]; };
  auto next_tile = [&]() {
    if (n + 1 < n1) store(n + 1, other);
    __syncthreads();
    const uint32_t t = buf;
    buf = other;
    other = t;
    ++n;
  };
  // Tiles as long as `more` says so; WHOLE: every row of the wave sees all
  // their keys.  The accumulators are rescaled outside the inner loop, which
  // stops at a tile whose scores have outgrown the maximum and takes it again
  // afterwards: as a branch inside it, the rescaling made the compiler keep
  // them in two sets of registers and spill the rest.
  auto tiles = [&]<bool WHOLE>(auto&& more) {
    for (;;) {
      bool grow = false;
      float mt = m;
      while (n < n1 && more()) {
        auto rd = [&](uint32_t at) { return *(LDS_AS const v8*)(uintptr_t)at; };
        auto rdv = [&](uint32_t at) { return *(LDS_AS const b8*)(uintptr_t)at; };
        uint32_t kr = buf + k_rd, vr = buf + v_rd, xr = buf + x_rd, gr = buf + kOffG + 16 * g;
        asm volatile("" : "+v"(kr), "+v"(vr), "+v"(xr), "+v"(gr));
        // plane's values of keys 16 kt + 4 g + 0..3
        auto rd4 = [&](int plane, int kt) { return *(LDS_AS const f32x4_t*)(uintptr_t)(gr + 256 * plane + 64 * kt); };
        f32x4_t s[4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) s[kt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) s[kt] = T16<T>::mfma16(rd((kr ^ (ks << 6)) + kt * (32 * HD)), qv[ks], s[kt]);
        mt = m;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const f32x4_t ks = rd4(0, kt), kl = rd4(1, kt);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x = fmaf(ks[r], s[kt][r], kl[r] * qs2);
            if constexpr (!WHOLE) x = 64 * n + 16 * kt + 4 * g + r < seen && there(kt) ? x : -INFINITY;
            s[kt][r] = x;
            mt = fmaxf(mt, x);
          }
        }
        mt = fmaxf(mt, __shfl_xor(mt, 16));
        mt = fmaxf(mt, __shfl_xor(mt, 32));
        grow = __any(mt > m + kLazy);
        if (grow) break;
        copy_tile(n + kRawSlots - 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t pk[kPieces][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int kt = 2 * t + y;
            const f32x4_t vs = rd4(2, kt);
            float w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float p = __builtin_amdgcn_exp2f(s[kt][r] - m);
              // a key that this row does not see may hold anything
              w[r] = !WHOLE && s[kt][r] == -INFINITY ? 0.0f : p * vs[r];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t hi = pack2<__bf16>(w[2 * x], w[2 * x + 1]);
              pk[0][2 * y + x] = hi;
              if constexpr (kPieces == 2) pk[kPieces - 1][2 * y + x] = pack2<__bf16>(w[2 * x] - lo16f<__bf16>(hi), w[2 * x + 1] - hi16f<__bf16>(hi));
            }
          }
          b8 pv[kPieces];
#pragma unroll
          for (int x = 0; x < kPieces; ++x) pv[x] = __builtin_bit_cast(b8, make_uint4(pk[x][0], pk[x][1], pk[x][2], pk[x][3]));
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const b8 vv = rdv((vr ^ (((4 * t) ^ (j & 7)) << 4)) + 2048 * j);
#pragma unroll
            for (int x = 0; x < kPieces; ++x) o[j] = T16<__bf16>::mfma16(vv, pv[x], o[j]);
          }
          const b8 xv = rdv(xr ^ (t << 6));
#pragma unroll
          for (int x = 0; x < kPieces; ++x) ox = T16<__bf16>::mfma16(xv, pv[x], ox);
        }
        next_tile();
      }
      if (!grow) break;
      const float m_new = fmaxf(m, mt), al = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[j] *= al;
      ox *= al;
    }
  };
  // one after the other (the waves of a workgroup may be in different ones,
  // each turn of each has one barrier): tiles seen whole, tiles that need
  // their masks, tiles past the wave's rows, which it only helps to unpack
  tiles.template operator()<true>([&]() { return 64 * n + 64 <= wmin && (there(0) & there(1) & there(2) & there(3)); });
  tiles.template operator()<false>([&]() { return 64 * n < wmax; });
  while (n < n1) {
    copy_tile(n + kRawSlots - 1);
    next_tile();
  }
  wait_copies<0>();                      // no copy may land after the workgroup's end
  // rows 0..3 of the extra block are the registers of g = 0, 4 and 5 the first two of g = 1
  const float base = __shfl(ox[0] + (ox[1] + ox[2]), i);
  const float l = __shfl(ox[3], i) + __shfl(ox[0] + ox[1], 16 + i);
  if (row >= rows) return;
  const int64_t tok = t0 + row / a.rep;
  const int hq = h * a.rep + row % a.rep;
  if (seen > a.chunk) {                // rows of one chunk need no joining
    if (c0 >= seen) return;
    const int64_t at = ((int64_t)ch * q.n_tokens + tok) * a.n_heads + hq;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      *reinterpret_cast<float4*>(a.part_o + at * HD + 16 * j + 4 * g) =
          make_float4(o[j][0] + base, o[j][1] + base, o[j][2] + base, o[j][3] + base);
    if (g == 0) a.part_ml[at] = make_float2(m, l);
  } else if (ch == 0) {
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (o[j][r] + base) * inv;
      store_n<T, 4>(a.out + tok * a.ldo + (int64_t)hq * HD + 16 * j + 4 * g, true, 4, v);
    }
  }
}

// Joins the chunks of each row: a workgroup per (token, head), HD / 4 lanes
// across the channels and the chunks dealt to the groups of lanes, then the
// groups in order (the same sums every time).
template <typename T, int HD>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttnArgs a, KvDev c, KvBatch q) {
  constexpr int L = HD / 4, NG = 256 / L;
  __shared__ f32x4_t sv[NG][L];
  __shared__ float sl[NG], sm[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, tok = wg / a.n_heads;
  const int head = (int)(wg % a.n_heads);
  if (tok >= q.n_tokens) return;
  const int b = seq_of_token(q.q_start, c.n_seqs, tok);
  if (b < 0) return;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  if (tok - t0 >= a.max_q) return;
  const int64_t most = min((int64_t)a.max_kv, (int64_t)c.max_pages * c.page);
  const int64_t seen = max(min((int64_t)q.kv_len[b] - n_q + (tok - t0) + 1, most), (int64_t)0);
  if (seen <= a.chunk) return;               // written by its only chunk
  const int n = (int)((seen + a.chunk - 1) / a.chunk);
  const int64_t at = tok * a.n_heads + head, step = q.n_tokens * a.n_heads;
  float m = kNoMax;
  for (int k = tid; k < n; k += 256) m = fmaxf(m, a.part_ml[at + k * step].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if (lane == 0) sm[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const int grp = tid / L, li = tid % L;
  float l = 0.0f;
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int k = grp; k < n; k += NG) {
    const float2 ml = a.part_ml[at + k * step];
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(a.part_o + (at + k * step) * HD + 4 * li);
    const float al = __builtin_amdgcn_exp2f(ml.x - m);
    l = fmaf(al, ml.y, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaf(al, x[e], v[e]);
  }
  sv[grp][li] = v;
  if (li == 0) sl[grp] = l;
  __syncthreads();
  if (tid >= L) return;
  l = sl[0];
  v = sv[0][tid];
#pragma unroll
  for (int g = 1; g < NG; ++g) {
    l += sl[g];
    v += sv[g][tid];
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  float r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = v[e] * inv;
  store_n<T, 4>(a.out + tok * a.ldo + (int64_t)head * HD + 4 * tid, true, 4, r);
}

// ---------------------------------------------------------------- host side
static bool cache_ok(const gptq_kv4_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_grid || !c->v_grid || !c->page_table) return false;
  if (c->n_pages <= 0 || c->n_kv_heads <= 0 || c->n_seqs <= 0 || c->max_pages <= 0) return false;
  if (c->page_size <= 0 || (c->page_size % 16) != 0 || (c->head_dim != 64 && c->head_dim != 128)) return false;
  if ((int64_t)c->max_pages * c->page_size > INT_MAX - 65536) return false;
  // rows are counted in 32 bits (their addresses are not)
  if ((int64_t)c->n_pages * c->n_kv_heads > INT_MAX / c->page_size) return false;
  const uintptr_t al = reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes) |
                       reinterpret_cast<uintptr_t>(c->k_grid) | reinterpret_cast<uintptr_t>(c->v_grid);
  return (al & 15) == 0 && (reinterpret_cast<uintptr_t>(c->page_table) & 3) == 0;
}
static KvDev dev_of(const gptq_kv4_cache* c) {
  return KvDev{c->k_codes, c->v_codes, static_cast<uint32_t*>(c->k_grid), static_cast<uint32_t*>(c->v_grid), c->page_table,
               c->n_pages, c->n_kv_heads, c->page_size, c->n_seqs, c->max_pages,
               (c->page_size & (c->page_size - 1)) == 0 ? __builtin_ctz((unsigned)c->page_size) : -1};
}
static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static bool elem_al(const void* p, gptq_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == GPTQ_F32 ? 3 : 1)) == 0; }

template <typename F> static int with_kind(gptq_dtype t, int hd, F&& f) {
  auto by_hd = [&]<int DT>() {
    if (hd == 128) f.template operator()<DT, 128>();
    else f.template operator()<DT, 64>();
  };
  if (t == GPTQ_F32) by_hd.template operator()<GPTQ_F32>();
  else if (t == GPTQ_F16) by_hd.template operator()<GPTQ_F16>();
  else by_hd.template operator()<GPTQ_BF16>();
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// Keys per workgroup of few rows: at least 512 workgroups where the keys allow
// it, and at least 16 pieces of the longest sequence, so that a batch of many
// lengths has no long tail (lengths are on the device: the host knows only
// their bound).  Measured, chunks of 256, 512, 1024, 2048: 48 sequences of 1 to
// 8192 positions 41, 37, 39, 50 us; one of 131072 57, 48, 45, 43 us.
static int chunk_of(int64_t groups, int max_kv) {
  if (max_kv <= 512) return 512;
  int c = groups * max_kv < (int64_t)256 * 512 ? 256 : 512;
  while (c < 4096 && 32 * c <= max_kv && groups * max_kv >= (int64_t)2 * c * 512) c *= 2;
  return c;
}

// Many rows: the keys are split only where there are too few row tiles for the
// 256 workgroups that the chip holds.  Measured for 256 and 512 workgroups:
// 192 rows of 8 sequences of 4096 positions 65, 76 us; of one of 32768 54, 66 us.
static int tile_chunk_of(int64_t groups, int max_kv) {
  const int all = (max_kv + 63) / 64 * 64;
  if (groups >= 256) return all;
  const int64_t want = ((int64_t)max_kv * groups / 256 + 63) / 64 * 64;
  return (int)std::min<int64_t>(all, std::max<int64_t>(want, 512));
}

// Rows of a sequence and kv head from which the unpacked tiles pay.  Measured,
// 48 and 64 rows, 16 at a time against in tiles: 8 sequences of 4096 positions
// 33 against 40, 41 against 41 us; 64 of 2048 116 against 114, 152 against 114;
// one of 32768 27 against 37, 33 against 38.
constexpr int kTileRows = 49;

// A launch has fewer than 2^32 threads along x: more workgroups than this go on
// along y (one long prompt beside many short sequences has that many, most of them
// without rows).
constexpr int64_t kGridX = 1 << 22;
static dim3 grid_of(int64_t n) {
  const int64_t x = std::min(n, kGridX);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

struct AttnPlan {
  int per;                   // rows per workgroup: 16, or the unpacked tiles' 192
  int chunk, n_chunks, row_tiles;
  int64_t grid;
  size_t off_ml, total;
};
static bool attn_plan(int64_t n_tokens, int n_heads, const gptq_kv4_cache* c, int max_q, int max_kv, AttnPlan& p) {
  if (!cache_ok(c) || n_tokens < 0 || n_tokens > INT_MAX || n_heads <= 0 || n_heads % c->n_kv_heads != 0) return false;
  if (max_q <= 0 || max_kv <= 0) return false;
  max_kv = (int)std::min<int64_t>(max_kv, (int64_t)c->max_pages * c->page_size);
  const int64_t rows = (int64_t)max_q * (n_heads / c->n_kv_heads);
  if (rows > INT_MAX - 16) return false;
  const int64_t seqs = (int64_t)c->n_seqs * c->n_kv_heads;
  p.per = rows < kTileRows ? 16 : 16 * kTileWaves;
  p.row_tiles = (int)((rows + p.per - 1) / p.per);
  const int64_t groups = seqs * p.row_tiles;
  p.chunk = p.per > 16 ? tile_chunk_of(groups, max_kv) : chunk_of(groups, max_kv);
  p.n_chunks = (max_kv + p.chunk - 1) / p.chunk;
  p.grid = groups * p.n_chunks;
  if (p.grid > INT_MAX || n_tokens * n_heads > INT_MAX) return false;
  if (p.per == 16 && p.grid / c->n_seqs > UINT32_MAX / 256) return false;     // sequences go along y
  const size_t n = p.n_chunks > 1 ? (size_t)p.n_chunks * n_tokens * n_heads : 0;
  p.off_ml = align_up(n * c->head_dim * sizeof(float));
  p.total = p.off_ml + align_up(n * sizeof(float2));
  return true;
}

template <typename T>
static int attend(const AttnArgs& a, const KvDev& c, const KvBatch& q, const AttnPlan& p, int hd, hipStream_t s) {
  if (p.per > 16) {
    if (hd == 128) kv4_tile_kernel<T, 128><<<grid_of(p.grid), 64 * kTileWaves, 0, s>>>(a, c, q);
    else kv4_tile_kernel<T, 64><<<grid_of(p.grid), 64 * kTileWaves, 0, s>>>(a, c, q);
  } else {
    const dim3 grid((unsigned)(p.grid / c.n_seqs), (unsigned)std::min(c.n_seqs, 32768), (unsigned)((c.n_seqs + 32767) / 32768));
    if (hd == 128) kv4_rows_kernel<T, 128><<<grid, 256, 0, s>>>(a, c, q);
    else kv4_rows_kernel<T, 64><<<grid, 256, 0, s>>>(a, c, q);
  }
  GPTQ_LAUNCH_CHECK();
  if (p.n_chunks > 1) {
    const dim3 grid = grid_of(q.n_tokens * a.n_heads);
    if (hd == 128) kv4_join_kernel<T, 128><<<grid, 256, 0, s>>>(a, c, q);
    else kv4_join_kernel<T, 64><<<grid, 256, 0, s>>>(a, c, q);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_kv4_append(const gptq_kv4_cache* cache, const void* K, const void* V, gptq_dtype dtype, int64_t n_tokens,
                               int64_t ldk, int64_t ldv, const int32_t* q_start, const int32_t* kv_len, hipStream_t s) {
  if (!cache_ok(cache) || n_tokens < 0 || n_tokens > INT_MAX || !q_start || !kv_len) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F32 && dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
  if (!K || !V || ldk < row || ldv < row || !elem_al(K, dtype) || !elem_al(V, dtype)) return GPTQ_ERR_INVALID_ARG;
  const int64_t step = dtype == GPTQ_F32 ? 4 : 8;
  const bool vec = al16(K) && al16(V) && ldk % step == 0 && ldv % step == 0;
  const KvDev c = dev_of(cache);
  const KvBatch q{q_start, kv_len, n_tokens};
  return with_kind(dtype, cache->head_dim, [&]<int DT, int HD>() {
    kv4_append_kernel<DT, HD><<<dim3((unsigned)((n_tokens + 3) / 4), 2), 256, 0, s>>>(c, q, K, V, ldk, ldv, vec);
  });
}

extern "C" int gptq_kv4_read(const gptq_kv4_cache* cache, void* K, void* V, gptq_dtype dtype, int64_t n_tokens,
                             const int32_t* q_start, const int32_t* kv_len, hipStream_t s) {
  if (!cache_ok(cache) || n_tokens < 0 || n_tokens > INT_MAX || !q_start || !kv_len) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F32 && dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (!elem_al(K, dtype) || !elem_al(V, dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || (!K && !V)) return GPTQ_OK;
  const bool vec = al16(K) && al16(V);
  const KvDev c = dev_of(cache);
  const KvBatch q{q_start, kv_len, n_tokens};
  return with_kind(dtype, cache->head_dim, [&]<int DT, int HD>() {
    kv4_read_kernel<DT, HD><<<dim3((unsigned)((n_tokens + 3) / 4), 2), 256, 0, s>>>(c, q, K, V, vec);
  });
}

extern "C" size_t gptq_kv4_attention_workspace_size(int64_t n_tokens, int32_t n_heads, const gptq_kv4_cache* cache,
                                                    int32_t max_q_len, int32_t max_kv_len) {
  AttnPlan p;
  return attn_plan(n_tokens, n_heads, cache, max_q_len, max_kv_len, p) ? p.total : 0;
}

extern "C" int gptq_kv4_attention(const void* Q, gptq_dtype dtype, int64_t n_tokens, int32_t n_heads, int64_t ldq,
                                  const gptq_kv4_cache* cache, const int32_t* q_start, const int32_t* kv_len,
                                  int32_t max_q_len, int32_t max_kv_len, float scale, void* out, int64_t ldo, void* ws,
                                  size_t ws_bytes, hipStream_t s) {
  AttnPlan p;
  if (n_tokens == 0) {                    // no tokens may have bounds of 0
    max_q_len += max_q_len == 0;
    max_kv_len += max_kv_len == 0;
  }
  if (!attn_plan(n_tokens, n_heads, cache, max_q_len, max_kv_len, p) || !q_start || !kv_len) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (!(std::fabs(scale) <= kMaxScale)) return GPTQ_ERR_INVALID_ARG;      // nor NaN
  if (n_tokens == 0) return GPTQ_OK;
  const int64_t row = (int64_t)n_heads * cache->head_dim;
  if (!Q || !out || ldq < row || ldo < row || ldq % 8 != 0 || ldo % 8 != 0 || !al16(Q) || !al16(out)) return GPTQ_ERR_INVALID_ARG;
  if (p.total && (!ws || ws_bytes < p.total || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)))) return GPTQ_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  const float scale2 = std::max(std::fabs(scale) * 1.44269504088896341f, 1.0e-30f);
  AttnArgs a{static_cast<const uint16_t*>(Q), static_cast<uint16_t*>(out), ldq, ldo, n_heads, n_heads / cache->n_kv_heads,
             max_q_len, (int)std::min<int64_t>(max_kv_len, (int64_t)cache->max_pages * cache->page_size),
             scale2, std::min(kLazy / scale2, 1.0e29f), scale < 0.0f ? 0x80008000u : 0u, p.chunk, p.n_chunks, p.row_tiles, reinterpret_cast<float*>(w),
             reinterpret_cast<float2*>(w + p.off_ml)};
  const KvDev c = dev_of(cache);
  const KvBatch q{q_start, kv_len, n_tokens};
  if (dtype == GPTQ_BF16) return attend<__bf16>(a, c, q, p, cache->head_dim, s);
  return attend<_Float16>(a, c, q, p, cache->head_dim, s);
}
