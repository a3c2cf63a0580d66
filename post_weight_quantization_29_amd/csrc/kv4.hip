// Attention over a paged cache held in 4 bits: gptq_kv4_append, gptq_kv4_read
// and gptq_kv4_attention.  A cached row (one token, one kv head) is head_dim
// 4-bit codes with a step and a minimum: x = lo + step * code.
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

// A wave takes one token: its rows of all kv heads, HD / 8 lanes per row (eight
// values each, 16 bytes), the row's minimum and maximum over those lanes.
// blockIdx.y: keys or values.  Bound by reading the 16-bit rows.
template <int DT, int HD>
__global__ __launch_bounds__(256) void kv4_append_kernel(KvDev c, KvBatch q, const void* __restrict__ K,
                                                         const void* __restrict__ V, int64_t ldk, int64_t ldv, bool vec) {
  constexpr int L = HD / 8, RPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= q.n_tokens) return;
  const int b = seq_of_token(q.q_start, c.n_seqs, t);
  if (b < 0) return;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  const int64_t p = (int64_t)q.kv_len[b] - n_q + (t - t0);
  const int64_t row0 = kv_row(c, b, 0, p);
  if (row0 < 0) return;
  const void* src = blockIdx.y ? V : K;
  const int64_t ld = blockIdx.y ? ldv : ldk;
  uint32_t* codes = blockIdx.y ? c.v_codes : c.k_codes;
  uint32_t* grid = blockIdx.y ? c.v_grid : c.k_grid;
  const int li = lane % L;
  for (int h0 = 0; h0 < c.n_kv; h0 += RPW) {
    const int h = h0 + lane / L;
    const bool in = h < c.n_kv;
    float x[8];
    load8<DT>(src, t * ld + (int64_t)min(h, c.n_kv - 1) * HD + 8 * li, vec, x);
    // values beyond fp16 count as its largest; fmin and fmax pass NaNs over
    float mn = kF16Max + 1.0f, mx = -kF16Max - 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = fminf(fmaxf(x[e], -kF16Max), kF16Max);
      const bool num = x[e] == x[e];
      mn = num ? fminf(mn, y) : mn;
      mx = num ? fmaxf(mx, y) : mx;
      x[e] = num ? y : -kF16Max;               // a NaN gets code 0
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      mn = fminf(mn, __shfl_xor(mn, o));
      mx = fmaxf(mx, __shfl_xor(mx, o));
    }
    if (mn > mx) mn = mx = 0.0f;               // a row of NaNs
    const _Float16 lo16 = (_Float16)mn;
    const float lo = (float)lo16;
    const _Float16 st16 = (_Float16)(fmaxf(mx - lo, 0.0f) / 15.0f);
    const float st = (float)st16;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = st > 0.0f ? rintf((x[e] - lo) / st) : 0.0f;
      w |= (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f) << (4 * e);
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
  float scale2;                // scale * log2(e)
  int chunk, n_chunks;         // keys per workgroup; 1 chunk: no partial results
  int row_tiles;
  float* part_o;               // [chunk][token][head][HD], not normalized
  float2* part_ml;             // [chunk][token][head]: maximum (log2 units), sum
};

constexpr float kNoMax = -3.0e38f;   // running maximum of a row that has seen nothing

// Few rows (a query row is one new token's one query head; a sequence has
// n_q * rep rows per kv head): a workgroup takes 16 rows against `chunk` keys,
// each of its four waves a quarter of them, 32 keys a step, all in registers.
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
// Bound by reading the cache: 136 bytes per key (head_dim 128) against about
// 330 vector instructions per 32 keys.  A step's loads are in flight while the
// step before is computed.
template <typename T, int HD>
__global__ __launch_bounds__(256) void kv4_rows_kernel(AttnArgs a, KvDev c, KvBatch q) {
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
  int id = blockIdx.x;
  const int ch = id % a.n_chunks;
  id /= a.n_chunks;
  const int rt = id % a.row_tiles;
  id /= a.row_tiles;
  const int h = id % c.n_kv, b = id / c.n_kv;
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
  // the tile's longest and shortest row
  const int seen_max = (int)max(min(first + (min(rt * 16 + 15, rows - 1) / a.rep) + 1, most), (int64_t)0);
  const int seen_min = (int)max(min(first + (rt * 16) / a.rep + 1, most), (int64_t)0);
  const int c0 = ch * a.chunk;
  if (ch > 0 && c0 >= seen_max) return;

  // Q in the order of a word's codes, and the sum of its row
  v8 qv[KW];
  float qsum = 0.0f;
  {
    const uint16_t* qp = a.Q + (t0 + ti) * a.ldq + (int64_t)hq * HD + 8 * KW * g;
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(qp + 8 * j);
      qsum += (lo16f<T>(v.x) + hi16f<T>(v.x)) + (lo16f<T>(v.y) + hi16f<T>(v.y)) +
              ((lo16f<T>(v.z) + hi16f<T>(v.z)) + (lo16f<T>(v.w) + hi16f<T>(v.w)));
      qv[j] = __builtin_bit_cast(v8, code_order(v));
    }
    qsum += __shfl_xor(qsum, 16);
    qsum += __shfl_xor(qsum, 32);
  }
  const float qs2 = qsum * a.scale2;

  const int quarter = a.chunk >> 2;
  const int kb0 = c0 + wave * quarter, kb1 = min(kb0 + quarter, seen_max);
  const int steps = kb1 > kb0 ? (kb1 - kb0 + 31) >> 5 : 0;
  // lane l: the cache row of 16-key tile l of this wave's keys, -1 if there is none
  int tile_row = -1;
  if (kb0 + 16 * lane < kb1) tile_row = (int)kv_row(c, b, h, kb0 + 16 * lane);

  struct Step {
    uint32_t k[2][KW];
    uint32_t v[8];
    uint4 kg[2], vg[2];
  };
  auto load = [&](int st, Step& s) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t r = max(__builtin_amdgcn_readlane(tile_row, 2 * st + u), 0);
      const uint32_t* kp = c.k_codes + (r + i) * RW + KW * g;
      if constexpr (KW == 4) *reinterpret_cast<uint4*>(s.k[u]) = *reinterpret_cast<const uint4*>(kp);
      else *reinterpret_cast<uint2*>(s.k[u]) = *reinterpret_cast<const uint2*>(kp);
      s.kg[u] = *reinterpret_cast<const uint4*>(c.k_grid + r + 4 * g);
      s.vg[u] = *reinterpret_cast<const uint4*>(c.v_grid + r + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) s.v[4 * u + e] = c.v_codes[(r + 4 * g + e) * RW + (i % RW)];
    }
  };

  f32x4_t o[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) o[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNoMax, l = 0.0f, base = 0.0f;
  Step cur, nxt;
  if (steps > 0) load(0, cur);
  for (int st = 0; st < steps; ++st) {
    if (st + 1 < steps) load(st + 1, nxt);
    const int kb = kb0 + 32 * st;
    float s[8], vs[8], vl[8];
    float mt = m;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t d = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KW; ++j) d = T16<T>::mfma16(__builtin_bit_cast(v8, code_word<T>(cur.k[u][j])), qv[j], d);
      const uint32_t kg[4] = {cur.kg[u].x, cur.kg[u].y, cur.kg[u].z, cur.kg[u].w};
      const uint32_t vg[4] = {cur.vg[u].x, cur.vg[u].y, cur.vg[u].z, cur.vg[u].w};
      const bool there = __builtin_amdgcn_readlane(tile_row, 2 * st + u) >= 0;
      const bool whole = there && kb + 16 * u + 16 <= seen_min;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = 4 * u + r;
        uint32_t kw = kg[r], vw = vg[r];
        bool ok = true;
        if (!whole) {
          // what lies behind a row's end or on a missing page may be anything
          ok = there && kb + 16 * u + 4 * g + r < seen;
          kw = ok ? kw : 0u;
          vw = ok ? vw : 0u;
        }
        const float ks = grid_step(kw), kl = grid_lo(kw);
        const float sc = fmaf(ks * a.scale2, d[r], fmaf(-kCodeBase, ks, kl) * qs2);
        s[e] = ok ? sc : -INFINITY;
        vs[e] = grid_step(vw);
        vl[e] = fmaf(-kCodeBase, vs[e], grid_lo(vw));
        mt = fmaxf(mt, s[e]);
      }
    }
    mt = fmaxf(mt, __shfl_xor(mt, 16));
    mt = fmaxf(mt, __shfl_xor(mt, 32));
    if (__any(mt > m)) {
      const float al = __builtin_amdgcn_exp2f(m - mt);
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[j] *= al;
      l *= al;
      base *= al;
      m = mt;
    }
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float p0 = __builtin_amdgcn_exp2f(s[e] - m), p1 = __builtin_amdgcn_exp2f(s[e + 1] - m);
      l += p0 + p1;
      base = fmaf(p0, vl[e], fmaf(p1, vl[e + 1], base));
      const float w0 = p0 * vs[e], w1 = p1 * vs[e + 1];
      ph[e / 2] = pack2<__bf16>(w0, w1);
      pl[e / 2] = pack2<__bf16>(w0 - lo16f<__bf16>(ph[e / 2]), w1 - hi16f<__bf16>(ph[e / 2]));
    }
    const b8 hv = __builtin_bit_cast(b8, make_uint4(ph[0], ph[1], ph[2], ph[3]));
    const b8 lv = __builtin_bit_cast(b8, make_uint4(pl[0], pl[1], pl[2], pl[3]));
    // zipped words: halves of key pairs
    uint32_t z[HD == 128 ? 2 : 1][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (HD == 128) {
        z[0][e] = __builtin_amdgcn_perm(cur.v[2 * e + 1], cur.v[2 * e], 0x05040100u);
        z[HD == 128 ? 1 : 0][e] = __builtin_amdgcn_perm(cur.v[2 * e + 1], cur.v[2 * e], 0x07060302u);
      } else {
        z[0][e] = __builtin_amdgcn_perm(cur.v[2 * e + 1], cur.v[2 * e], i < 8 ? 0x05040100u : 0x07060302u);
      }
    }
    auto pv = [&]<int J>() {
      constexpr int zi = J / 4, K = J % 4;
      const b8 vv = __builtin_bit_cast(b8, make_uint4(code_pair<__bf16, K>(z[zi][0]), code_pair<__bf16, K>(z[zi][1]),
                                                      code_pair<__bf16, K>(z[zi][2]), code_pair<__bf16, K>(z[zi][3])));
      o[J] = T16<__bf16>::mfma16(vv, hv, o[J]);
      o[J] = T16<__bf16>::mfma16(vv, lv, o[J]);
    };
    [&]<int... J>(std::integer_sequence<int, J...>) { (pv.template operator()<J>(), ...); }(std::make_integer_sequence<int, NJ>{});
    cur = nxt;
  }
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
    sM[wave][i] = m;
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
  if (a.n_chunks > 1) {
    const int64_t at = ((int64_t)ch * q.n_tokens + tok) * a.n_heads + head;
#pragma unroll
    for (int e = 0; e < HD / 16; e += 4)
      *reinterpret_cast<float4*>(a.part_o + at * HD + (HD / 16) * (tid & 15) + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    if ((tid & 15) == 0) a.part_ml[at] = make_float2(mm, ll);
  } else {
    const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;       // a row that saw nothing is 0; NaN stays
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) v[e] *= inv;
    store_n<T, HD / 16>(a.out + tok * a.ldo + (int64_t)head * HD + (HD / 16) * (tid & 15), true, HD / 16, v);
  }
}

// Joins the chunks of each row in their order: a wave per (token, head).
template <typename T, int HD>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttnArgs a, KvDev c, KvBatch q) {
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t tok = id / a.n_heads;
  const int head = (int)(id % a.n_heads);
  if (tok >= q.n_tokens) return;
  const int b = seq_of_token(q.q_start, c.n_seqs, tok);
  if (b < 0) return;
  int64_t t0;
  int n_q;
  q.span(b, t0, n_q);
  if (tok - t0 >= a.max_q) return;
  const int64_t most = min((int64_t)a.max_kv, (int64_t)c.max_pages * c.page);
  const int64_t seen = max(min((int64_t)q.kv_len[b] - n_q + (tok - t0) + 1, most), (int64_t)0);
  const int n = (int)((seen + a.chunk - 1) / a.chunk);
  const int64_t at = tok * a.n_heads + head, step = q.n_tokens * a.n_heads;
  float m = kNoMax;
  for (int k = lane; k < n; k += 64) m = fmaxf(m, a.part_ml[at + k * step].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  constexpr int E = HD / 64;
  float l = 0.0f, v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.0f;
  for (int k = 0; k < n; ++k) {
    const float2 ml = a.part_ml[at + k * step];
    const float al = __builtin_amdgcn_exp2f(ml.x - m);
    l = fmaf(al, ml.y, l);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(al, a.part_o[(at + k * step) * HD + E * lane + e], v[e]);
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[tok * a.ldo + (int64_t)head * HD + E * lane + e] = bits16<T>(v[e] * inv);
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
               c->n_pages, c->n_kv_heads, c->page_size, c->n_seqs, c->max_pages};
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

// Keys per workgroup.
static int chunk_of(int64_t groups, int max_kv) {
  if (max_kv <= 512) return 512;
  int64_t want = (int64_t)max_kv * groups / 2048;
  int c = 512;
  while (c < 4096 && c < want) c *= 2;
  return c;
}

struct AttnPlan {
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
  p.row_tiles = (int)((rows + 15) / 16);
  const int64_t groups = (int64_t)c->n_seqs * c->n_kv_heads * p.row_tiles;
  p.chunk = chunk_of(groups, max_kv);
  p.n_chunks = (max_kv + p.chunk - 1) / p.chunk;
  p.grid = groups * p.n_chunks;
  if (p.grid > INT_MAX) return false;
  const size_t n = p.n_chunks > 1 ? (size_t)p.n_chunks * n_tokens * n_heads : 0;
  p.off_ml = align_up(n * c->head_dim * sizeof(float));
  p.total = p.off_ml + align_up(n * sizeof(float2));
  return true;
}

template <typename T>
static int attend(const AttnArgs& a, const KvDev& c, const KvBatch& q, const AttnPlan& p, int hd, hipStream_t s) {
  if (hd == 128) kv4_rows_kernel<T, 128><<<(unsigned)p.grid, 256, 0, s>>>(a, c, q);
  else kv4_rows_kernel<T, 64><<<(unsigned)p.grid, 256, 0, s>>>(a, c, q);
  GPTQ_LAUNCH_CHECK();
  if (p.n_chunks > 1) {
    const unsigned grid = (unsigned)((q.n_tokens * a.n_heads + 3) / 4);
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
  if (!attn_plan(n_tokens, n_heads, cache, max_q_len, max_kv_len, p) || !q_start || !kv_len) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (!(scale == scale) || std::isinf(scale)) return GPTQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return GPTQ_OK;
  const int64_t row = (int64_t)n_heads * cache->head_dim;
  if (!Q || !out || ldq < row || ldo < row || ldq % 8 != 0 || ldo % 8 != 0 || !al16(Q) || !al16(out)) return GPTQ_ERR_INVALID_ARG;
  if (p.total && (!ws || ws_bytes < p.total || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)))) return GPTQ_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  AttnArgs a{static_cast<const uint16_t*>(Q), static_cast<uint16_t*>(out), ldq, ldo, n_heads, n_heads / cache->n_kv_heads,
             max_q_len, (int)std::min<int64_t>(max_kv_len, (int64_t)cache->max_pages * cache->page_size),
             scale * 1.44269504088896341f, p.chunk, p.n_chunks, p.row_tiles, reinterpret_cast<float*>(w),
             reinterpret_cast<float2*>(w + p.off_ml)};
  const KvDev c = dev_of(cache);
  const KvBatch q{q_start, kv_len, n_tokens};
  if (dtype == GPTQ_BF16) return attend<__bf16>(a, c, q, p, cache->head_dim, s);
  return attend<_Float16>(a, c, q, p, cache->head_dim, s);
}
