// Operators on the packed 4-bit layer: the product with bias, activation and
// residual (gptq_w4_linear), the gated feed-forward block's first half
// (gptq_w4_gated) and its backward pass (gptq_w4_gated_backward).  GPTQ
// practice page m.lqnn.cn/news/117696, section 4.3: at inference the 4-bit
// weights are dequantized to a 16-bit type and then multiplied.
//
//  few tokens     w4_skinny_kernel, w4_mid_kernel (to kMidMax): packed words go
//                 straight into matrix-instruction operands; bound by reading
//                 the codes
//  more           w4_dense_kernel writes the 16-bit weight to the workspace
//                 once, then gemm16_kernel; bound by the matrix pipe
//  backward       dG, dU elementwise, the 16-bit weights transposed to the
//                 workspace, one product over both contractions
#include "gemm16.h"
#include "w4_epilogue.h"

#include <climits>

namespace gptq {

struct W4Dev {
  const uint32_t* packed;
  const float* scales;
  const int32_t* zeros;
};
static W4Dev dev_of(const gptq_w4_weight* w) { return W4Dev{w->packed, w->scales, w->zeros}; }

// ---------------------------------------------------------------- few tokens
// A wave holds 16 weight rows (of each of NMAT matrices) against 16 NT
// tokens on v_mfma_f32_16x16x32: operand lane l is row l % 16 with eight k of
// k-group l / 16, which is exactly one packed word, so a word is dequantized
// in registers where it is consumed and nothing goes through LDS.  A lane's
// 16-byte load is four words, 32 k; a chunk (64 lanes) covers 16 rows x 128 k.
// The NW waves of a workgroup split k in chunk pairs (256 k: one 128-byte line
// per row), each with the next pair's loads in flight while one is multiplied,
// and their sums are joined through LDS in wave order.
// GRID 0: any layout (a (scale, zero) pair loaded for each word: 4104 -> 4096 in
// groups of 24 12.4 us for one token, 13 for 16, 21 for 64, where 4096 -> 4096 in
// groups of 128 takes 7.9, 7.8 and, by w4_mid_kernel, 17).  1: rows allow 16-byte loads and a lane's 32 k share a
// group.  2: as 1, and the rows' scales and zero points fit LDS, where the
// workgroup puts them first, in one coalesced sweep: loaded where they are
// used, each touches 16 cache lines for 16 numbers, which cost more than the
// codes themselves (11008 x 4096 gate and up, one token: 26 us, 17 from LDS).
template <typename T, int NT, int NMAT, int NW, int GRID, typename Epi>
__global__ __launch_bounds__(64 * NW) void w4_skinny_kernel(const uint16_t* __restrict__ X, int64_t ldx, int m, W4Dev wa,
                                                            W4Dev wb, int d_out, int d_in, int G, int ng, Epi epi) {
  typedef typename T16<T>::v8 v8;
  constexpr bool FAST = GRID > 0;
  constexpr int MT = 1;
  constexpr int NG = FAST ? 1 : 4;          // (scale, zero) pairs per lane and chunk
  extern __shared__ float2 sgrid[];         // [NMAT][16][ng + 1] (scale, zero) when GRID == 2
  __shared__ f32x4_t red[NW][NMAT * MT * NT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r0 = blockIdx.x * 16 * MT;
  const int lr = lane & 15, lg = lane >> 4;
  const int nw = d_in >> 3, pairs = (d_in + 255) >> 8;
  const float invG = 1.0f / (float)G;

  struct Chunk {
    uint32_t p[4];
    float s[NG], z[NG];
  };
  Chunk cur[2][NMAT][MT], nxt[2][NMAT][MT];
  auto load = [&](int pair, Chunk (&c)[2][NMAT][MT]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k0 = 256 * pair + 128 * u + 32 * lg;
#pragma unroll
      for (int a = 0; a < NMAT; ++a)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const W4Dev& w = a ? wb : wa;
          const int r = min(r0 + 16 * t + lr, d_out - 1);   // rows past the end: computed, not stored
          const uint32_t* prow = w.packed + (size_t)r * nw;
          const float* srow = w.scales + (size_t)r * ng;
          const int32_t* zrow = w.zeros + (size_t)r * ng;
          Chunk& o = c[u][a][t];
          if constexpr (FAST) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            o.s[0] = o.z[0] = 0.0f;                          // past the end: weights of 0
            if (k0 < d_in) {
              v = *reinterpret_cast<const uint4*>(prow + (k0 >> 3));
              if constexpr (GRID == 1) {
                const int g = group_of(k0, G, invG);
                o.s[0] = srow[g];
                o.z[0] = (float)zrow[g];
              }
            }
            o.p[0] = v.x; o.p[1] = v.y; o.p[2] = v.z; o.p[3] = v.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = k0 + 8 * j;
              o.p[j] = 0u;
              o.s[j] = o.z[j] = 0.0f;
              if (k < d_in) {
                const int g = group_of(k, G, invG);
                o.p[j] = prow[k >> 3];
                o.s[j] = srow[g];
                o.z[j] = (float)zrow[g];
              }
            }
          }
        }
    }
  };

  f32x4_t acc[NMAT][MT][NT];
#pragma unroll
  for (int a = 0; a < NMAT; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[a][t][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const uint16_t* xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xrow[n] = X + (int64_t)min(16 * n + lr, m - 1) * ldx;   // tokens past the end: likewise

  if (wave < pairs) load(wave, cur);
  if constexpr (GRID == 2) {
    const int have = min(16, d_out - r0) * ng;
#pragma unroll
    for (int a = 0; a < NMAT; ++a) {
      const W4Dev& w = a ? wb : wa;
      for (int e = tid; e < have; e += 64 * NW) {
        const int row = group_of(e, ng, 1.0f / (float)ng);
        sgrid[(a * 16 + row) * (ng + 1) + e - row * ng] =
            make_float2(w.scales[(size_t)r0 * ng + e], (float)w.zeros[(size_t)r0 * ng + e]);
      }
    }
    __syncthreads();
  }
  for (int pair = wave; pair < pairs; pair += NW) {
    if (pair + NW < pairs) load(pair + NW, nxt);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k0 = 256 * pair + 128 * u + 32 * lg;
      uint4 xv[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xv[n][j] = k0 + 8 * j < d_in ? *reinterpret_cast<const uint4*>(xrow[n] + k0 + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int a = 0; a < NMAT; ++a)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          Chunk& c = cur[u][a][t];
          if constexpr (GRID == 2) {
            if (k0 < d_in) {
              const float2 sz = sgrid[(a * 16 + min(lr, d_out - 1 - r0)) * (ng + 1) + group_of(k0, G, invG)];
              c.s[0] = sz.x;
              c.z[0] = sz.y;
            }
          }
          bool far = false;
#pragma unroll
          for (int q = 0; q < NG; ++q) far |= fabsf(c.z[q]) > kZeroFast;
          uint32_t w[4][4];
          if (!__any(far)) {
            uint32_t zp[NG];
#pragma unroll
            for (int q = 0; q < NG; ++q) zp[q] = zero_pair(c.z[q]);
#pragma unroll
            for (int j = 0; j < 4; ++j) dequant_fast<T>(c.p[j], c.s[FAST ? 0 : j], zp[FAST ? 0 : j], w[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) dequant_any<T>(c.p[j], c.s[FAST ? 0 : j], c.z[FAST ? 0 : j], w[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const v8 wv = __builtin_bit_cast(v8, make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[a][t][n] = T16<T>::mfma16(wv, __builtin_bit_cast(v8, xv[n][j]), acc[a][t][n]);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int a = 0; a < NMAT; ++a)
#pragma unroll
        for (int t = 0; t < MT; ++t) cur[u][a][t] = nxt[u][a][t];
  }

#pragma unroll
  for (int a = 0; a < NMAT; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) red[wave][(a * MT + t) * NT + n][lane] = acc[a][t][n];
  __syncthreads();
  // lane l of a tile holds rows 4 (l / 16) + 0..3 of token l % 16
  for (int e = tid; e < MT * NT * 64; e += 64 * NW) {
    const int tile = e >> 6, l = e & 63;
    float v[NMAT][4];
#pragma unroll
    for (int a = 0; a < NMAT; ++a) {
      f32x4_t sum = red[0][a * MT * NT + tile][l];
#pragma unroll
      for (int w = 1; w < NW; ++w) sum += red[w][a * MT * NT + tile][l];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[a][q] = sum[q];
    }
    const int tok = 16 * (tile % NT) + (l & 15);
    if (tok < m) epi.template finish<4>(v, tok, r0 + 16 * (tile / NT) + 4 * (l >> 4));
  }
}

// ---------------------------------------------------------------- some tokens
// Up to 128 tokens (blocks of 64): the activations no longer are a small part
// of what a CU reads, so eight waves of 16 weight rows share them.  A workgroup
// takes 128 rows (64 of gate and 64 of up) against its block's tokens over a
// slice of k; stages of 256 k of the activations are copied HBM -> LDS
// (buffer_load ... lds, 16 bytes a lane, three slots, two stages ahead), the
// codes go to registers two stages ahead, the slice's scales and zero points to
// LDS first.  Slices' sums go to the workspace and w4_join_kernel adds them in
// order and finishes them.  Measured, 24 tokens, 28672 -> 8192: 50 us (2.4 TB/s of
// codes; and 5 to join) against 129 us with every 16 rows reading the activations
// themselves.  Vector issue (dequantizing) fills half of the cycles, at 2.8 waves a
// SIMD that wait for 46 % of their time: a barrier every 256 k, scales read from
// LDS right before their use, and at up to 32 tokens five spilled registers (24
// bytes a lane) for the 128 that let four waves share a SIMD.
// A token's row in LDS is 512 bytes; the 16-byte chunk c of its half y sits at
// c ^ (token % 16): 16 tokens' reads of one chunk hit 16 columns of the banks.
constexpr int kMidK = 256;          // k per stage
constexpr int kMidSlots = 3;
constexpr int kMidWaves = 8;

template <typename T, int NT, int NMAT>
__global__ __launch_bounds__(64 * kMidWaves, NT <= 2 ? 4 : 2) void w4_mid_kernel(const uint16_t* __restrict__ X, int64_t ldx, int m, W4Dev wa,
                                                                   W4Dev wb, int d_out, int d_in, int G, int ng, int slice_k,
                                                                   int slice_groups, float* __restrict__ part) {
  typedef typename T16<T>::v8 v8;
  constexpr uint32_t kSlot = NT * 16 * 2 * kMidK;
  constexpr int RB = 16 * kMidWaves / NMAT;          // rows of a matrix per workgroup
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  float2* sgrid = reinterpret_cast<float2*>(smem + kMidSlots * kSlot);   // [wave][16][slice_groups + 1]
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int mat = NMAT == 2 ? wave / (kMidWaves / 2) : 0;
  const int r0 = blockIdx.x * RB + 16 * (wave % (RB / 16));
  const W4Dev& w = mat ? wb : wa;
  const int nw = d_in >> 3;
  const float invG = 1.0f / (float)G;
  X += (int64_t)blockIdx.z * (16 * NT) * ldx;
  const int t0 = blockIdx.z * 16 * NT, tokens = m - t0;
  const int k_lo = blockIdx.y * slice_k, k_hi = min(k_lo + slice_k, d_in);
  const int stages = (k_hi - k_lo + kMidK - 1) / kMidK;
  const int g_lo = group_of(k_lo, G, invG);

  // copy i of a stage: tokens 2 (wave + 8 i) + lane / 32, half (lane / 16) % 2, chunk lane % 16
  const uint64_t xb = reinterpret_cast<uint64_t>(X);
  int x_off[NT];
  int x_k;
  {
    const int tl = 2 * wave + (lane >> 5);
    x_k = 128 * ((lane >> 4) & 1) + 8 * ((lane & 15) ^ (tl & 15));
#pragma unroll
    for (int i = 0; i < NT; ++i) x_off[i] = (int)(min(tl + 16 * i, tokens - 1) * ldx + x_k) * 2;
  }
  auto copy_x = [&](int st) {
    const int k0 = k_lo + st * kMidK;
    const i32x4_t rs = tile_rsrc(xb + (uint64_t)k0 * 2, st < stages);
    const bool in = k0 + x_k < k_hi;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      copy16_lds(lds + (st % kMidSlots) * kSlot + 1024u * (wave + kMidWaves * i), rs, in ? x_off[i] : kPastEnd);
  };
  // Codes of stage st: 32 k at k0 + 32 lg and at 128 further.  Past the slice's
  // end the last ones again, with scale 0: always two loads, as the waits count.
  const uint32_t* prow = w.packed + (size_t)min(r0 + lr, d_out - 1) * nw;
  uint4 p[3][2];
  auto load_p = [&](int st, uint4 (&o)[2]) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
      o[y] = *reinterpret_cast<const uint4*>(prow + (min(k_lo + st * kMidK + 128 * y + 32 * lg, k_hi - 32) >> 3));
  };
  f32x4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  load_p(0, p[0]);
  copy_x(0);
  load_p(1, p[1]);
  copy_x(1);
  // this wave's scales and zero points; 0, 0 past the ends
  {
    const int n = 16 * slice_groups;
    for (int e = lane; e < n; e += 64) {
      const int row = e / slice_groups, g = e - row * slice_groups;
      const bool in = r0 + row < d_out && g_lo + g < ng;
      const size_t at = (size_t)(r0 + row) * ng + g_lo + g;
      sgrid[(wave * 16 + row) * (slice_groups + 1) + g] = in ? make_float2(w.scales[at], (float)w.zeros[at]) : make_float2(0.0f, 0.0f);
    }
  }
  const float2* grow = sgrid + (wave * 16 + lr) * (slice_groups + 1);
  wait_copies<0>();
  __syncthreads();

  // RING: stages follow whose copies and codes are to be issued.  The last one
  // or two stages issue nothing and wait for everything: the codes that they
  // would load nobody uses, so the compiler drops such loads, and a wait that
  // counts them lets copies pass that the next stage reads.
  auto stage = [&]<int S, bool RING>(int st) {
    if constexpr (RING) {
      load_p(st + 2, p[(S + 2) % 3]);
      copy_x(st + 2);
    }
    const uint32_t xs = lds + S * kSlot + lr * (2 * kMidK);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int k = k_lo + st * kMidK + 128 * y + 32 * lg;
      float2 sz = make_float2(0.0f, 0.0f);
      if (k < k_hi) sz = grow[group_of(k, G, invG) - g_lo];
      const uint32_t c[4] = {p[S][y].x, p[S][y].y, p[S][y].z, p[S][y].w};
      uint32_t wv[4][4];
      if (!__any(fabsf(sz.y) > kZeroFast)) {
        const uint32_t zp = zero_pair(sz.y);
#pragma unroll
        for (int j = 0; j < 4; ++j) dequant_fast<T>(c[j], sz.x, zp, wv[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) dequant_any<T>(c[j], sz.x, sz.y, wv[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v8 a = __builtin_bit_cast(v8, make_uint4(wv[j][0], wv[j][1], wv[j][2], wv[j][3]));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const v8 b = *(LDS_AS const v8*)(uintptr_t)(xs + n * (16 * 2 * kMidK) + 256 * y + (((4 * lg + j) ^ lr) << 4));
          acc[n] = T16<T>::mfma16(a, b, acc[n]);
        }
      }
    }
    // the next stage's copies are older than this stage's NT copies and two code loads
    if constexpr (RING) wait_copies<NT + 2>();
    else wait_copies<0>();
    wait_lds_reads();
    ring_barrier();
  };
  int st = 0;
  for (; st + 3 <= stages; st += 3) {
    stage.template operator()<0, true>(st);
    stage.template operator()<1, true>(st + 1);
    stage.template operator()<2, true>(st + 2);
  }
  if (st < stages) stage.template operator()<0, false>(st++);
  if (st < stages) stage.template operator()<1, false>(st++);
  wait_copies<0>();                     // no copy may land after the workgroup's end

  // lane l: rows r0 + 4 (l / 16) + 0..3 of token 16 n + l % 16
  const int dp = (d_out + 3) & ~3;
  if (r0 + 4 * lg < dp) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (16 * n + lr < tokens)
        *reinterpret_cast<f32x4_t*>(part + ((size_t)(blockIdx.y * NMAT + mat) * m + t0 + 16 * n + lr) * dp + r0 + 4 * lg) = acc[n];
  }
}

// The slices' sums in order, and the epilogue: four outputs of a token per thread.
template <typename Epi>
__global__ __launch_bounds__(256) void w4_join_kernel(const float* __restrict__ part, int slices, int m, int d_out, Epi epi) {
  constexpr int PL = Epi::kPlanes;
  const int dp = (d_out + 3) & ~3;
  const int c = 4 * (blockIdx.x * 256 + threadIdx.x), tok = blockIdx.y;
  if (c >= dp) return;
  float v[PL][4];
#pragma unroll
  for (int a = 0; a < PL; ++a) {
    f32x4_t sum = *reinterpret_cast<const f32x4_t*>(part + ((size_t)a * m + tok) * dp + c);
#pragma unroll 8
    for (int s = 1; s < slices; ++s) sum += *reinterpret_cast<const f32x4_t*>(part + ((size_t)(s * PL + a) * m + tok) * dp + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[a][e] = sum[e];
  }
  epi.template finish<4>(v, tok, c);
}

// ---------------------------------------------------------------- operands of the large products
// out[t][k] = X[t][perm[k]] (perm NULL: k), zeros from d_in to Kp; Kp a
// multiple of 8.  One thread per eight values.
__global__ __launch_bounds__(256) void x_order_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t m, int d_in,
                                                      const int32_t* __restrict__ perm, int Kp, uint16_t* __restrict__ out) {
  const int k = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (k >= Kp) return;
  int at[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = min(k + e, d_in - 1);
    at[e] = perm ? min(max(perm[c], 0), d_in - 1) : c;
  }
  for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < d_in ? X[t * ldx + at[e]] : (uint16_t)0;
    uint4 o;
    o.x = v[0] | (uint32_t)v[1] << 16;
    o.y = v[2] | (uint32_t)v[3] << 16;
    o.z = v[4] | (uint32_t)v[5] << 16;
    o.w = v[6] | (uint32_t)v[7] << 16;
    *reinterpret_cast<uint4*>(out + t * Kp + k) = o;
  }
}

// The same for a row that fits LDS and a perm: loaded whole and in order, its
// values are then picked from LDS.  blockIdx.x: shares of a row's groups of eight.
// Measured, against x_order_kernel's picks through L1: 8192 rows of 4096 22 and 82
// us, 24 of 28672 5.4 and 8.0 us.
constexpr int kGatherMax = 32768;
__global__ __launch_bounds__(256) void x_gather_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t m, int d_in,
                                                       const int32_t* __restrict__ perm, int Kp, bool vec, bool pvec,
                                                       uint16_t* __restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) uint16_t row[];
  const int tid = threadIdx.x;
  for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
    const uint16_t* x = X + t * ldx;
    if (vec) {
#pragma unroll 4
      for (int c = 8 * tid; c < d_in; c += 8 * 256) *reinterpret_cast<uint4*>(row + c) = *reinterpret_cast<const uint4*>(x + c);
    } else {
#pragma unroll 4
      for (int c = tid; c < d_in; c += 256) row[c] = x[c];
    }
    __syncthreads();
    for (int k = 8 * (blockIdx.x * 256 + tid); k < Kp; k += 8 * 256 * gridDim.x) {
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (k < d_in) {
        int at[8];
        if (pvec) {
          *reinterpret_cast<int4*>(at) = *reinterpret_cast<const int4*>(perm + k);
          *reinterpret_cast<int4*>(at + 4) = *reinterpret_cast<const int4*>(perm + k + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) at[e] = perm[k + e];
        }
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = row[min(max(at[e], 0), d_in - 1)];
        o = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
      *reinterpret_cast<uint4*>(out + t * Kp + k) = o;
    }
    __syncthreads();
  }
}

template <typename T>
GPTQ_DEV void dequant_word16(uint32_t p, float s, float z, uint32_t (&w)[4]) {
  if (!__any(fabsf(z) > kZeroFast)) dequant_fast<T>(p, s, zero_pair(z), w);
  else dequant_any<T>(p, s, z, w);
}

// The 16-bit weight, rows of Kp (zeros from d_in on).  Row r goes to row
// r of out, or with two matrices (wb.packed not NULL, blockIdx.z picks one) to
// 64 (r / 32) + 32 z + r % 32: gate and up alternate in blocks of 32 rows, so a
// wave of the product holds both sums of the same outputs.  One thread per
// word: 4 bytes in, 16 out; bound by those writes (5120 x 13824 38 us, 4.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void w4_dense_kernel(W4Dev wa, W4Dev wb, int d_out, int d_in, int G, int ng, int Kp,
                                                       uint16_t* __restrict__ out) {
  const int q = blockIdx.x * 256 + threadIdx.x;
  if (8 * q >= Kp) return;
  const W4Dev& w = blockIdx.z ? wb : wa;
  const int nw = d_in >> 3;
  const bool in = q < nw;
  const int g = in ? group_of(8 * q, G, 1.0f / (float)G) : 0;
  for (int r = blockIdx.y; r < d_out; r += gridDim.y) {
    const size_t ro = wb.packed ? (size_t)64 * (r >> 5) + 32 * blockIdx.z + (r & 31) : (size_t)r;
    const uint32_t p = in ? w.packed[(size_t)r * nw + q] : 0u;
    const float s = in ? w.scales[(size_t)r * ng + g] : 0.0f, z = in ? (float)w.zeros[(size_t)r * ng + g] : 0.0f;
    uint32_t v[4];
    dequant_word16<T>(p, s, z, v);
    *reinterpret_cast<uint4*>(out + ro * Kp + 8 * q) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// The transposed 16-bit weights: out[channel c][k], row pitch Fp for each matrix, k = r for
// the first's row r and Fp + r for the second's; zeros from d_out to Fp.  Column q
// of the packed layer goes to row perm[q].  A workgroup turns 64 rows x 16
// words (128 columns) through LDS, two rows to a 4-byte write: 128-byte pieces
// out.  A column's eight 16-byte chunks (eight rows each) sit at chunk ^ (column
// / 8) % 8, so the 16 words' writes spread over the banks.  Bound by the writes: 2 x
// 11008 x 4096 59 us (3.8 TB/s), with unspread writes 87 us.
template <typename T>
__global__ __launch_bounds__(256) void w4_dense_t_kernel(W4Dev wa, W4Dev wb, int d_out, int d_in, int G, int ng,
                                                         const int32_t* __restrict__ perm, int Fp, uint16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[128 * 64];
  const W4Dev& w = blockIdx.z ? wb : wa;
  const int nw = d_in >> 3, tid = threadIdx.x;
  const int ql = tid & 15, q = blockIdx.x * 16 + ql;
  const int gq = q < nw ? group_of(8 * q, G, 1.0f / (float)G) : 0;
  for (int rb = blockIdx.y; rb * 64 < Fp; rb += gridDim.y) {
    const int r0 = rb * 64;
    uint32_t v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 2 * (tid >> 4) + 32 * (i >> 1) + (i & 1);
      const bool in = q < nw && r < d_out;
      const uint32_t p = in ? w.packed[(size_t)r * nw + q] : 0u;
      const float s = in ? w.scales[(size_t)r * ng + gq] : 0.0f, z = in ? (float)w.zeros[(size_t)r * ng + gq] : 0.0f;
      dequant_word16<T>(p, s, z, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rl = 2 * (tid >> 4) + 32 * i;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t two = __builtin_amdgcn_perm(v[2 * i + 1][e >> 1], v[2 * i][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
        *reinterpret_cast<uint32_t*>(tile + (8 * ql + e) * 64 + (((rl >> 3) ^ (ql & 7)) << 3) + (rl & 7)) = two;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cl = (tid >> 3) + 32 * i, c = 128 * blockIdx.x + cl, k = r0 + 8 * (tid & 7);
      if (c < d_in && k < Fp) {
        const int ch = perm ? min(max(perm[c], 0), d_in - 1) : c;
        *reinterpret_cast<uint4*>(out + ((size_t)ch * gridDim.z + blockIdx.z) * Fp + k) =
            *reinterpret_cast<const uint4*>(tile + cl * 64 + (((tid & 7) ^ ((cl >> 3) & 7)) << 3));
      }
    }
    __syncthreads();
  }
}

// dU = dM act(G), dG = dM U act'(G): eight values per thread, to the outputs
// (each may be NULL) and, where the product cannot take them from there, to
// copies with rows of Fp (zeros from f on; NULL otherwise).  Bound by memory: 4096 x
// 11008 79 us, 5.7 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void gated_slopes_kernel(const uint16_t* dM, const uint16_t* G, const uint16_t* U,
                                                           int64_t m, int f, int Fp, int act, bool vec, uint16_t* dG,
                                                           uint16_t* dU, uint16_t* cG, uint16_t* cU) {
  const int c = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (c >= Fp) return;
  const int have = max(0, min(8, f - c));
  const bool full = vec && have == 8;
  for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
    const int64_t at = t * f + c;
    float dm[8], g[8], u[8], a[8], b[8];
    load_n<T, 8>(dM + at, full, have, dm);
    load_n<T, 8>(G + at, full, have, g);
    load_n<T, 8>(U + at, full, have, u);
    with_act(act, [&]<int ACT>() {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = e < have ? dm[e] * u[e] * act_slope<ACT>(g[e]) : 0.0f;
        b[e] = e < have ? dm[e] * act_fn<ACT>(g[e]) : 0.0f;
      }
    });
    if (dG) store_n<T, 8>(dG + at, full, have, a);
    if (dU) store_n<T, 8>(dU + at, full, have, b);
    if (cG) store_n<T, 8>(cG + t * Fp + c, true, 8, a);
    if (cU) store_n<T, 8>(cU + t * Fp + c, true, 8, b);
  }
}

// ---------------------------------------------------------------- host side
// Tokens up to which the packed words are multiplied directly, by the 16-row
// waves and by w4_mid_kernel.  Measured, w4_mid_kernel and through memory, 65 and
// 128 tokens (one layer, its codes in the last-level cache; from HBM 28672 ->
// 8192 takes 157 and 163): 4096 -> 4096 18 and 25, 19 and 26 us; 5120 -> 13824 62 and 61, 68 and
// 64 us; 28672 -> 8192 141 and 245, 147 and 252 us; 192 tokens in three blocks 29 and
// 31, 100 and 79, 217 and 261 us.
constexpr int kSkinnyMax = 64, kMidMax = 128;

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static int pad_k(int d) { return (d + kGk - 1) / kGk * kGk; }
static unsigned grid_rows(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 32768); }

static size_t x_copy_bytes(int64_t m, int d_in) { return align_up((size_t)m * pad_k(d_in) * 2); }

// X's rows in the order perm (NULL: as they are), padded to whole stages
static int order_x(const void* X, int64_t ldx, int64_t m, int d_in, const int32_t* perm, uint16_t* out, hipStream_t s) {
  const int Kp = pad_k(d_in);
  if (perm && d_in <= kGatherMax) {
    const bool vec = aligned16(X) && ldx % 8 == 0;
    // every share of a row loads all of it: as many as fill the chip
    const int64_t shares = std::min<int64_t>(std::max<int64_t>(512 / m, 1), (Kp / 8 + 255) / 256);
    x_gather_kernel<<<dim3((unsigned)shares, (unsigned)std::min<int64_t>(m, 4096)), 256, (size_t)d_in * 2, s>>>(
        static_cast<const uint16_t*>(X), ldx, m, d_in, perm, Kp, vec, aligned16(perm), out);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  x_order_kernel<<<dim3((unsigned)((Kp / 8 + 255) / 256), grid_rows(m)), 256, 0, s>>>(
      static_cast<const uint16_t*>(X), ldx, m, d_in, perm, Kp, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// The slices of k that w4_mid_kernel takes for m tokens; no slices: it does not
// (few tokens, or rows or groups that its loads do not fit).
struct MidPlan {
  int slices, slice_k, slice_groups;
  size_t bytes;
};
// Tokens x d_in x d_out from which it pays with at most 16 tokens, too: what
// the 16-row workgroups read of the activations outweighs the second launch.
// Measured, 16-row and this, 8 and 16 tokens: 4096 -> 4096 7 and 11, 7 and 12 us;
// 5120 -> 13824 19 and 19, 26 and 20 us; 28672 -> 8192 50 and 39, 68 and 40 us.
// Two matrices share the reading: 4096 -> 2 x 11008 21 and 26, 22 and 26 us; 8192
// -> 2 x 28672 81 and 79, 90 and 80 us.
constexpr double kMidWork = 6.0e8;
constexpr size_t kMidGridBytes = 48 << 10;      // LDS for the scales and zero points
static MidPlan mid_plan(int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  MidPlan p{0, 0, 0, 0};
  const int G = w4_group(wa);
  if (m > kMidMax || (m <= 16 && (double)m * wa->d_in * wa->d_out < (wb ? 3.0 : 1.0) * kMidWork) || wa->d_in % 32 != 0 || G % 32 != 0) return p;
  if (!aligned16(wa->packed) || (wb && !aligned16(wb->packed))) return p;
  const int64_t blocks = (wa->d_out + (wb ? 64 : 128) - 1) / (wb ? 64 : 128);
  // two workgroups a CU, four stages a slice at least, scales that fit LDS
  int64_t k = ((int64_t)wa->d_in * blocks / 512 + kMidK - 1) / kMidK * kMidK;
  const int64_t groups = kMidGridBytes / (16 * kMidWaves * sizeof(float2)) - 2;
  k = std::max<int64_t>(k, 4 * kMidK);
  k = std::min<int64_t>(k, std::max<int64_t>((groups - 1) * G / kMidK * kMidK, kMidK));
  // as many slices of even length
  const int64_t stages = (wa->d_in + kMidK - 1) / kMidK, n = (wa->d_in + k - 1) / k;
  p.slice_k = (int)((stages + n - 1) / n * kMidK);
  p.slices = (wa->d_in + p.slice_k - 1) / p.slice_k;
  p.slice_groups = std::min(p.slice_k / G + 2, wa->n_groups);
  p.bytes = align_up((size_t)p.slices * (wb ? 2 : 1) * m * ((wa->d_out + 3) & ~3) * sizeof(float));
  return p;
}

// the 16-bit weight goes through memory
static bool is_dense(int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  return m > kSkinnyMax && !mid_plan(m, wa, wb).slices;
}

// X has to be copied (and brought into processing order)
static bool copies_x(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* w, const gptq_w4_weight* wb) {
  if (w->perm || !aligned16(X) || (ldx % 8) != 0 || ldx * 2 > kMaxRowBytes) return true;
  return is_dense(m, w, wb) && w->d_in % kGk != 0;
}

template <typename T, typename Epi>
static int launch_mid(const uint16_t* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb,
                      const MidPlan& p, const Epi& epi, float* part, hipStream_t s) {
  constexpr int NMAT = Epi::kPlanes;
  const int d_out = wa->d_out, rb = 128 / NMAT;
  auto go = [&]<int NT>() {
    const dim3 grid((unsigned)((d_out + rb - 1) / rb), (unsigned)p.slices, (unsigned)((m + 16 * NT - 1) / (16 * NT)));
    const size_t lds = (size_t)kMidSlots * NT * 16 * 2 * kMidK + (size_t)kMidWaves * 16 * (p.slice_groups + 1) * sizeof(float2);
    w4_mid_kernel<T, NT, NMAT><<<grid, 64 * kMidWaves, lds, s>>>(X, ldx, (int)m, dev_of(wa), dev_of(wb), d_out, wa->d_in,
                                                                 w4_group(wa), wa->n_groups, p.slice_k, p.slice_groups, part);
  };
  if (m <= 16) go.template operator()<1>();
  else if (m <= 32) go.template operator()<2>();
  else go.template operator()<4>();
  GPTQ_LAUNCH_CHECK();
  w4_join_kernel<Epi><<<dim3((unsigned)((d_out + 1023) / 1024), (unsigned)m), 256, 0, s>>>(part, p.slices, (int)m, d_out, epi);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T, int NMAT, typename Epi>
static int launch_skinny(const uint16_t* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb,
                         const Epi& epi, hipStream_t s) {
  const int G = w4_group(wa), d_out = wa->d_out, d_in = wa->d_in, ng = wa->n_groups;
  const W4Dev a = dev_of(wa), b = dev_of(wb);
  const bool fast = (d_in % 32) == 0 && (G % 32) == 0 && aligned16(a.packed) && aligned16(b.packed);
  // scales in LDS beside the sums of 8 waves (a workgroup may have 64 KB without further ado)
  const size_t grid_bytes = (size_t)NMAT * 16 * (ng + 1) * sizeof(float2);
  auto go = [&]<int NT, int GRID>() {
    w4_skinny_kernel<T, NT, NMAT, 8, GRID, Epi><<<(unsigned)((d_out + 15) / 16), 512, GRID == 2 ? grid_bytes : 0, s>>>(
        X, ldx, (int)m, a, b, d_out, d_in, G, ng, epi);
  };
  if (m <= 16) {
    if (fast && grid_bytes <= 40 * 1024) go.template operator()<1, 2>();
    else if (fast) go.template operator()<1, 1>();
    else go.template operator()<1, 0>();
  } else if (m <= 32) {
    go.template operator()<2, 0>();
  } else {
    go.template operator()<4, 0>();
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// Tiles of the large products.  256 workgroups of 256 x 256 tiles fill the chip,
// or 512 of 128 x 128 (two a CU).  What is left after the full rounds leaves part
// of it idle, so those tiles' k is split where that pays.  The model: a round of
// large tiles takes 28 ns per k (1.18 PFLOP/s), of small ones 2/3 of that, and
// slices' sums pass memory at a copy's rate.  Measured whole and split: 8192 x
// 13824 x 5120 1050 and 982 us; 577 x 5120 x 13824 146 and 126 us; gated 4096 ->
// 2 x 11008, 1024 tokens 239 and 216 us, 4096 tokens 700 and 692 us.
struct GemmPlan {
  int edge, whole, slices, slice_pairs;
  size_t bytes;
};
constexpr int kMinSlicePairs = 4;
static GemmPlan gemm_plan(int64_t m, int64_t n, int pairs) {
  GemmPlan best{0, 0, 0, 0, 0};
  double best_us = 0.0;
  for (const int e : {256, 128}) {
    const int64_t tiles = ((m + e - 1) / e) * ((n + e - 1) / e), slots = e == 256 ? 256 : 512;
    const double round_us = pairs * kGk * (e == 256 ? 0.028 : 0.019);
    const int64_t rest = tiles % slots;
    for (int s = 1; s <= 8; ++s) {
      if (s > 1 && (rest * s > slots || pairs < s * kMinSlicePairs)) break;
      const int per = (pairs + s - 1) / s;
      if (s > 1 && (pairs + per - 1) / per != s) continue;
      const size_t bytes = s > 1 ? (size_t)rest * s * e * e * sizeof(float) : 0;
      const double us = round_us * (double)(tiles / slots) + (rest ? round_us / s : 0.0) + (s > 1 ? 5.0 + 2.0 * (double)bytes / 4.9e6 : 0.0);
      if (!best.edge || us < best_us) {
        best = GemmPlan{e, (int)std::min<int64_t>(s > 1 ? tiles - rest : tiles, INT_MAX), s, per, align_up(bytes)};
        best_us = us;
      }
      if (!rest) break;
    }
  }
  return best;
}

template <typename T, int MB, int NB, int WM, int WN, typename Epi>
static int launch_tiles(const Gemm16Args& g, const Epi& epi, hipStream_t s) {
  const int64_t rest = (int64_t)g.tiles_m * g.tiles_n - g.whole;
  const int64_t grid = ((int64_t)g.whole + 7) / 8 * 8 + (rest * g.slices + 7) / 8 * 8;
  gemm16_kernel<T, MB, NB, WM, WN, Epi><<<(unsigned)grid, 64 * WM * WN, 0, s>>>(g, epi);
  GPTQ_LAUNCH_CHECK();
  if (rest) {
    const int64_t waves = rest * WM * WN * (NB * MB / Epi::kPlanes);
    gemm16_join_kernel<MB, NB, WM, WN, Epi><<<(unsigned)((waves + 3) / 4), 256, 0, s>>>(g, epi);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

// part: gemm_plan(g.m, g.n, g.n_pairs).bytes
template <typename T, typename Epi>
static int launch_gemm16(Gemm16Args g, const Epi& epi, void* part, hipStream_t s) {
  const GemmPlan p = gemm_plan(g.m, g.n, g.n_pairs);
  const int64_t tm = (g.m + p.edge - 1) / p.edge, tn = (g.n + p.edge - 1) / p.edge;
  if (tm * tn > INT_MAX / 16) return GPTQ_ERR_INVALID_ARG;
  g.tiles_m = (int)tm;
  g.tiles_n = (int)tn;
  g.whole = p.whole;
  g.slices = p.slices;
  g.slice_pairs = p.slice_pairs;
  g.part = static_cast<float*>(part);
  return p.edge == 256 ? launch_tiles<T, 4, 2, 2, 4>(g, epi, s) : launch_tiles<T, 2, 2, 2, 2>(g, epi, s);
}

template <typename T>
static int launch_dense(const gptq_w4_weight* wa, const gptq_w4_weight* wb, uint16_t* out, hipStream_t s) {
  const int Kp = pad_k(wa->d_in);
  w4_dense_kernel<T><<<dim3((unsigned)((Kp / 8 + 255) / 256), grid_rows(wa->d_out), wb ? 2 : 1), 256, 0, s>>>(
      dev_of(wa), wb ? dev_of(wb) : W4Dev{nullptr, nullptr, nullptr}, wa->d_out, wa->d_in, w4_group(wa), wa->n_groups, Kp, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// rows of the 16-bit weight, both matrices' in blocks of 32
static int weight_rows(const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  return wb ? 2 * ((wa->d_out + 31) / 32 * 32) : wa->d_out;
}
static size_t dense_bytes(const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  return align_up((size_t)weight_rows(wa, wb) * pad_k(wa->d_in) * 2);
}

// one or both products of X with packed weights, and the epilogue
template <typename T, typename Epi>
static int forward(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb, const Epi& epi,
                   void* ws, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  const uint16_t* x = static_cast<const uint16_t*>(X);
  if (copies_x(X, ldx, m, wa, wb)) {
    uint16_t* xc = reinterpret_cast<uint16_t*>(base);
    const int st = order_x(X, ldx, m, wa->d_in, wa->perm, xc, s);
    if (st != GPTQ_OK) return st;
    x = xc;
    ldx = pad_k(wa->d_in);
  }
  if (const MidPlan p = mid_plan(m, wa, wb); p.slices) {
    return launch_mid<T>(x, ldx, m, wa, wb ? wb : wa, p, epi, reinterpret_cast<float*>(base + x_copy_bytes(m, wa->d_in)), s);
  } else if (m <= kSkinnyMax) {
    return launch_skinny<T, Epi::kPlanes>(x, ldx, m, wa, wb ? wb : wa, epi, s);
  } else {
    uint16_t* w16 = reinterpret_cast<uint16_t*>(base + x_copy_bytes(m, wa->d_in));
    const int st = launch_dense<T>(wa, wb, w16, s);
    if (st != GPTQ_OK) return st;
    const int Kp = pad_k(wa->d_in), n = weight_rows(wa, wb);
    return launch_gemm16<T>(Gemm16Args{x, x, ldx, w16, Kp, m, n, Kp / kGk, Kp / kGk}, epi,
                            base + x_copy_bytes(m, wa->d_in) + dense_bytes(wa, wb), s);
  }
}

static size_t forward_bytes(int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  if (!is_dense(m, wa, wb)) return x_copy_bytes(m, wa->d_in) + mid_plan(m, wa, wb).bytes;
  return x_copy_bytes(m, wa->d_in) + dense_bytes(wa, wb) +
         gemm_plan(m, weight_rows(wa, wb), pad_k(wa->d_in) / kGk).bytes;
}
// what this call touches of it
static size_t forward_needs(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  if (!is_dense(m, wa, wb) && !copies_x(X, ldx, m, wa, wb) && !mid_plan(m, wa, wb).slices) return 0;
  return forward_bytes(m, wa, wb);
}

static bool pair_ok(const gptq_w4_weight* a, const gptq_w4_weight* b) {
  return w4_ok(a) && w4_ok(b) && a->d_out == b->d_out && a->d_in == b->d_in && w4_group(a) == w4_group(b) && a->perm == b->perm;
}
static bool is16(gptq_dtype t) { return t == GPTQ_F16 || t == GPTQ_BF16; }
static bool is_gate(gptq_act a) { return a == GPTQ_ACT_SILU || a == GPTQ_ACT_GELU || a == GPTQ_ACT_GELU_TANH; }
// 2-byte (4-byte for fp32) alignment of every element pointer
static bool elem_ok(const void* p, gptq_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == GPTQ_F32 ? 3 : 1)) == 0; }

// two arrays (each may be NULL) share a byte
static bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uint64_t)b_bytes && y < x + (uint64_t)a_bytes;
}

struct BackLayout {
  size_t off_g, off_u, off_part, total;
  int Fp;
};
static BackLayout back_layout(int64_t m, const gptq_w4_weight* w) {
  BackLayout L;
  L.Fp = pad_k(w->d_out);
  L.off_g = align_up((size_t)w->d_in * 2 * L.Fp * 2);
  L.off_u = L.off_g + align_up((size_t)m * L.Fp * 2);
  L.off_part = L.off_u + align_up((size_t)m * L.Fp * 2);
  L.total = L.off_part + gemm_plan(m, w->d_in, 2 * L.Fp / kGk).bytes;
  return L;
}

template <typename T>
static int backward(const void* dM, const void* G, const void* U, int64_t m, const gptq_w4_weight* gate,
                    const gptq_w4_weight* up, int act, void* dG, void* dU, void* dX, void* ws, hipStream_t s) {
  const int f = gate->d_out, d = gate->d_in;
  const BackLayout L = back_layout(m, gate);
  char* base = static_cast<char*>(ws);
  uint16_t* wt = reinterpret_cast<uint16_t*>(base);
  // the product takes dG and dU from the outputs where their rows fit its stages
  const bool direct = dG && dU && L.Fp == f && aligned16(dG) && aligned16(dU);
  uint16_t* cg = direct ? nullptr : reinterpret_cast<uint16_t*>(base + L.off_g);
  uint16_t* cu = direct ? nullptr : reinterpret_cast<uint16_t*>(base + L.off_u);
  const bool vec = (f % 8) == 0 && aligned16(dM) && aligned16(G) && aligned16(U) && aligned16(dG) && aligned16(dU);
  gated_slopes_kernel<T><<<dim3((unsigned)((L.Fp / 8 + 255) / 256), grid_rows(m)), 256, 0, s>>>(
      static_cast<const uint16_t*>(dM), static_cast<const uint16_t*>(G), static_cast<const uint16_t*>(U), m, f, L.Fp, act, vec,
      static_cast<uint16_t*>(dG), static_cast<uint16_t*>(dU), cg, cu);
  GPTQ_LAUNCH_CHECK();
  w4_dense_t_kernel<T><<<dim3((unsigned)((d + 127) / 128), grid_rows((L.Fp + 63) / 64), 2), 256, 0, s>>>(
      dev_of(gate), dev_of(up), f, d, w4_group(gate), gate->n_groups, gate->perm, L.Fp, wt);
  GPTQ_LAUNCH_CHECK();
  const uint16_t* a0 = direct ? static_cast<const uint16_t*>(dG) : cg;
  const uint16_t* a1 = direct ? static_cast<const uint16_t*>(dU) : cu;
  const LinearEpi<T> epi{nullptr, nullptr, dX, 0, d, d, GPTQ_ACT_NONE, T16<T>::kType, (d % 8) == 0 && aligned16(dX)};
  return launch_gemm16<T>(Gemm16Args{a0, a1, L.Fp, wt, 2 * L.Fp, m, d, L.Fp / kGk, 2 * L.Fp / kGk}, epi, base + L.off_part, s);
}

struct LinearBackLayout {
  size_t off_y, off_part, total;
  int Fp;
};
static LinearBackLayout linear_back_layout(int64_t m, const gptq_w4_weight* w) {
  LinearBackLayout L;
  L.Fp = pad_k(w->d_out);
  L.off_y = align_up((size_t)w->d_in * L.Fp * 2);
  L.off_part = L.off_y + align_up((size_t)m * L.Fp * 2);
  L.total = L.off_part + gemm_plan(m, w->d_in, L.Fp / kGk).bytes;
  return L;
}

// dX = dY W + R: the transposed 16-bit weight once into the workspace, then the 16-bit
// product, which takes dY from where it is if its rows fit its stages.  4096 tokens, 4096 -> 11008:
// weight 36 us (written at 2.5 TB/s), product 320 (1.15 PFLOP/s); 577 tokens, 5120 -> 5120 in
// act order: 20 and 41, and 8 for the last round's slices of k.
template <typename T>
static int linear_backward(const void* dY, int64_t lddy, int64_t m, const gptq_w4_weight* w, const LinearEpi<T>& epi, void* ws,
                           hipStream_t s) {
  const LinearBackLayout L = linear_back_layout(m, w);
  char* base = static_cast<char*>(ws);
  uint16_t* wt = reinterpret_cast<uint16_t*>(base);
  const uint16_t* a = static_cast<const uint16_t*>(dY);
  if (L.Fp != w->d_out || !aligned16(dY) || lddy % 8 != 0 || lddy * 2 > kMaxRowBytes) {
    uint16_t* c = reinterpret_cast<uint16_t*>(base + L.off_y);
    const int st = order_x(dY, lddy, m, w->d_out, nullptr, c, s);
    if (st != GPTQ_OK) return st;
    a = c;
    lddy = L.Fp;
  }
  w4_dense_t_kernel<T><<<dim3((unsigned)((w->d_in + 127) / 128), grid_rows((L.Fp + 63) / 64), 1), 256, 0, s>>>(
      dev_of(w), dev_of(w), w->d_out, w->d_in, w4_group(w), w->n_groups, w->perm, L.Fp, wt);
  GPTQ_LAUNCH_CHECK();
  return launch_gemm16<T>(Gemm16Args{a, a, lddy, wt, L.Fp, m, w->d_in, L.Fp / kGk, L.Fp / kGk}, epi, base + L.off_part, s);
}

}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_w4_linear_workspace_size(int64_t m, const gptq_w4_weight* w) {
  if (m <= 0 || m > INT_MAX || !w4_ok(w)) return 0;
  return forward_bytes(m, w, nullptr);
}

extern "C" int gptq_w4_linear(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_w4_weight* w,
                              const void* bias, gptq_act act, const void* R, int64_t ldr, void* Y, gptq_dtype y_dtype,
                              int64_t ldy, void* ws, size_t ws_bytes, hipStream_t s) {
  if (!w4_ok(w) || m < 0 || m > INT_MAX || !is16(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (y_dtype != GPTQ_F32 && !is16(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (act < GPTQ_ACT_NONE || act > GPTQ_ACT_GELU_TANH) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!X || !Y || ldx < w->d_in || ldy < w->d_out || (R && ldr < w->d_out)) return GPTQ_ERR_INVALID_ARG;
  if (!elem_ok(X, x_dtype) || !elem_ok(bias, x_dtype) || !elem_ok(R, y_dtype) || !elem_ok(Y, y_dtype)) return GPTQ_ERR_INVALID_ARG;
  const size_t need = forward_needs(X, ldx, m, w, nullptr);
  if (need && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)))) return GPTQ_ERR_WORKSPACE;
  const int64_t step = y_dtype == GPTQ_F32 ? 4 : 8;
  const bool vec = aligned16(Y) && (ldy % step) == 0 && (!R || (aligned16(R) && (ldr % step) == 0));
  if (x_dtype == GPTQ_BF16)
    return forward<__bf16>(X, ldx, m, w, nullptr,
                           LinearEpi<__bf16>{static_cast<const uint16_t*>(bias), R, Y, ldr, ldy, w->d_out, act, y_dtype, vec}, ws, s);
  return forward<_Float16>(X, ldx, m, w, nullptr,
                           LinearEpi<_Float16>{static_cast<const uint16_t*>(bias), R, Y, ldr, ldy, w->d_out, act, y_dtype, vec}, ws, s);
}

extern "C" size_t gptq_w4_gated_workspace_size(int64_t m, const gptq_w4_weight* gate, const gptq_w4_weight* up) {
  if (m <= 0 || m > INT_MAX || !pair_ok(gate, up)) return 0;
  return forward_bytes(m, gate, up);
}

extern "C" int gptq_w4_gated(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_w4_weight* gate,
                             const gptq_w4_weight* up, gptq_act act, void* G, void* U, void* M, void* ws, size_t ws_bytes,
                             hipStream_t s) {
  if (!pair_ok(gate, up) || m < 0 || m > INT_MAX || !is16(x_dtype) || !is_gate(act)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!X || !M || !G != !U || ldx < gate->d_in) return GPTQ_ERR_INVALID_ARG;
  if (!elem_ok(X, x_dtype) || !elem_ok(G, x_dtype) || !elem_ok(U, x_dtype) || !elem_ok(M, x_dtype)) return GPTQ_ERR_INVALID_ARG;
  const size_t need = forward_needs(X, ldx, m, gate, up);
  if (need && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)))) return GPTQ_ERR_WORKSPACE;
  const bool vec = (gate->d_out % 8) == 0 && aligned16(M) && aligned16(G) && aligned16(U);
  uint16_t *g = static_cast<uint16_t*>(G), *u = static_cast<uint16_t*>(U), *o = static_cast<uint16_t*>(M);
  if (x_dtype == GPTQ_BF16) return forward<__bf16>(X, ldx, m, gate, up, GatedEpi<__bf16>{g, u, o, gate->d_out, act, vec}, ws, s);
  return forward<_Float16>(X, ldx, m, gate, up, GatedEpi<_Float16>{g, u, o, gate->d_out, act, vec}, ws, s);
}

extern "C" size_t gptq_w4_gated_backward_workspace_size(int64_t m, const gptq_w4_weight* gate, const gptq_w4_weight* up) {
  if (m <= 0 || m > INT_MAX || !pair_ok(gate, up)) return 0;
  return back_layout(m, gate).total;
}

extern "C" int gptq_w4_gated_backward(const void* dM, const void* G, const void* U, gptq_dtype dtype, int64_t m,
                                      const gptq_w4_weight* gate, const gptq_w4_weight* up, gptq_act act, void* dG, void* dU,
                                      void* dX, void* ws, size_t ws_bytes, hipStream_t s) {
  if (!pair_ok(gate, up) || m < 0 || m > INT_MAX || !is16(dtype) || !is_gate(act)) return GPTQ_ERR_INVALID_ARG;
  if (gate->d_out > kW4MaxCols) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!dM || !G || !U || !dX) return GPTQ_ERR_INVALID_ARG;
  for (const void* p : {dM, G, U, (const void*)dG, (const void*)dU, (const void*)dX})
    if (!elem_ok(p, dtype)) return GPTQ_ERR_INVALID_ARG;
  // the product writes dX while it reads dG and dU
  const int64_t xb = m * gate->d_in * 2, gb = m * gate->d_out * 2;
  if (overlap(dX, xb, dG, gb) || overlap(dX, xb, dU, gb) || overlap(dG, gb, dU, gb)) return GPTQ_ERR_INVALID_ARG;
  if (!ws || ws_bytes < back_layout(m, gate).total || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  if (dtype == GPTQ_BF16) return backward<__bf16>(dM, G, U, m, gate, up, act, dG, dU, dX, ws, s);
  return backward<_Float16>(dM, G, U, m, gate, up, act, dG, dU, dX, ws, s);
}

extern "C" size_t gptq_w4_linear_backward_workspace_size(int64_t m, const gptq_w4_weight* w) {
  if (m <= 0 || m > INT_MAX || !w4_ok(w) || w->d_out > kW4MaxCols) return 0;
  return linear_back_layout(m, w).total;
}

extern "C" int gptq_w4_linear_backward(const void* dY, gptq_dtype dtype, int64_t m, int64_t lddy, const gptq_w4_weight* w,
                                       const void* R, int64_t ldr, void* dX, gptq_dtype x_dtype, int64_t lddx, void* ws,
                                       size_t ws_bytes, hipStream_t s) {
  if (!w4_ok(w) || w->d_out > kW4MaxCols || m < 0 || m > INT_MAX || !is16(dtype)) return GPTQ_ERR_INVALID_ARG;
  if (x_dtype != GPTQ_F32 && !is16(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!dY || !dX || lddy < w->d_out || lddx < w->d_in || (R && ldr < w->d_in)) return GPTQ_ERR_INVALID_ARG;
  if (!elem_ok(dY, dtype) || !elem_ok(R, x_dtype) || !elem_ok(dX, x_dtype)) return GPTQ_ERR_INVALID_ARG;
  const int64_t xe = x_dtype == GPTQ_F32 ? 4 : 2;
  const int64_t xb = rows_bytes(m, lddx, w->d_in, xe);
  if (overlap(dX, xb, dY, rows_bytes(m, lddy, w->d_out, 2))) return GPTQ_ERR_INVALID_ARG;
  if (R && !(R == dX && ldr == lddx) && overlap(dX, xb, R, rows_bytes(m, ldr, w->d_in, xe))) return GPTQ_ERR_INVALID_ARG;
  if (!ws || ws_bytes < linear_back_layout(m, w).total || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  const int64_t step = x_dtype == GPTQ_F32 ? 4 : 8;
  const bool vec = aligned16(dX) && (lddx % step) == 0 && (!R || (aligned16(R) && (ldr % step) == 0));
  if (dtype == GPTQ_BF16)
    return linear_backward<__bf16>(dY, lddy, m, w, LinearEpi<__bf16>{nullptr, R, dX, ldr, lddx, w->d_in, GPTQ_ACT_NONE, x_dtype, vec}, ws, s);
  return linear_backward<_Float16>(dY, lddy, m, w, LinearEpi<_Float16>{nullptr, R, dX, ldr, lddx, w->d_in, GPTQ_ACT_NONE, x_dtype, vec}, ws, s);
}
