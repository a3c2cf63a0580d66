// Operators on the packed 4-bit layer: the product with bias, activation and
// residual (gptq_w4_linear), the gated feed-forward block's first half
// (gptq_w4_gated) and its backward pass (gptq_w4_gated_backward).  GPTQ
// practice page m.lqnn.cn/news/117696, section 4.3: at inference the 4-bit
// weights are dequantized to a 16-bit type and then multiplied.
//
//  few tokens (m <= kSkinnyMax)  w4_skinny_kernel: packed words go straight
//                 into matrix-instruction operands; bound by reading the codes
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
// A wave holds 16 MT weight rows (of each of NMAT matrices) against 16 NT
// tokens on v_mfma_f32_16x16x32: operand lane l is row l % 16 with eight k of
// k-group l / 16, which is exactly one packed word, so a word is dequantized
// in registers where it is consumed and nothing goes through LDS.  A lane's
// 16-byte load is four words, 32 k; a chunk (64 lanes) covers 16 rows x 128 k.
// The NW waves of a workgroup split k in chunk pairs (256 k: one 128-byte line
// per row), each with the next pair's loads in flight while one is multiplied,
// and their sums are joined through LDS in wave order.  FAST: rows allow
// 16-byte loads and a lane's 32 k share a group.
template <typename T, int MT, int NT, int NMAT, int NW, bool FAST, typename Epi>
__global__ __launch_bounds__(64 * NW) void w4_skinny_kernel(const uint16_t* __restrict__ X, int64_t ldx, int m, W4Dev wa,
                                                            W4Dev wb, int d_out, int d_in, int G, int ng, Epi epi) {
  typedef typename T16<T>::v8 v8;
  constexpr int NG = FAST ? 1 : 4;          // (scale, zero) pairs per lane and chunk
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
              const int g = group_of(k0, G, invG);
              o.s[0] = srow[g];
              o.z[0] = (float)zrow[g];
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
          const Chunk& c = cur[u][a][t];
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

template <typename T>
GPTQ_DEV void dequant_word16(uint32_t p, float s, float z, uint32_t (&w)[4]) {
  if (!__any(fabsf(z) > kZeroFast)) dequant_fast<T>(p, s, zero_pair(z), w);
  else dequant_any<T>(p, s, z, w);
}

// The 16-bit weight, rows of Kp (zeros from d_in on).  Row r goes to row
// r of out, or with two matrices (wb.packed not NULL, blockIdx.z picks one) to
// 64 (r / 32) + 32 z + r % 32: gate and up alternate in blocks of 32 rows, so a
// wave of the product holds both sums of the same outputs.  One thread per
// word: 4 bytes in, 16 out; bound by those writes.
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

// The transposed 16-bit weights: out[channel c][k], row pitch 2 Fp, k = r for
// the gate's row r and Fp + r for the up's; zeros from d_out to Fp.  Column q
// of the packed layer goes to row perm[q].  A workgroup turns 64 rows x 16
// words (128 columns) through LDS: 128-byte pieces out.
constexpr int kTPitch = 64 + 8;
template <typename T>
__global__ __launch_bounds__(256) void w4_dense_t_kernel(W4Dev wa, W4Dev wb, int d_out, int d_in, int G, int ng,
                                                         const int32_t* __restrict__ perm, int Fp, uint16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[128 * kTPitch];
  const W4Dev& w = blockIdx.z ? wb : wa;
  const int nw = d_in >> 3, tid = threadIdx.x;
  const int q = blockIdx.x * 16 + (tid & 15);
  const int gq = q < nw ? group_of(8 * q, G, 1.0f / (float)G) : 0;
  for (int rb = blockIdx.y; rb * 64 < Fp; rb += gridDim.y) {
    const int r0 = rb * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rl = (tid >> 4) + 16 * i, r = r0 + rl;
      const bool in = q < nw && r < d_out;
      const uint32_t p = in ? w.packed[(size_t)r * nw + q] : 0u;
      const float s = in ? w.scales[(size_t)r * ng + gq] : 0.0f, z = in ? (float)w.zeros[(size_t)r * ng + gq] : 0.0f;
      uint32_t v[4];
      dequant_word16<T>(p, s, z, v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        tile[(8 * (tid & 15) + e) * kTPitch + rl] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cl = (tid >> 3) + 32 * i, c = 128 * blockIdx.x + cl, k = r0 + 8 * (tid & 7);
      if (c < d_in && k < Fp) {
        const int ch = perm ? min(max(perm[c], 0), d_in - 1) : c;
        *reinterpret_cast<uint4*>(out + (size_t)ch * 2 * Fp + (size_t)blockIdx.z * Fp + k) =
            *reinterpret_cast<const uint4*>(tile + cl * kTPitch + 8 * (tid & 7));
      }
    }
    __syncthreads();
  }
}

// dU = dM act(G), dG = dM U act'(G): eight values per thread, to the outputs
// (each may be NULL) and, where the product cannot take them from there, to
// copies with rows of Fp (zeros from f on; NULL otherwise).
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
// tokens up to which the packed words are multiplied directly
constexpr int kSkinnyMax = 64;

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static int pad_k(int d) { return (d + kGk - 1) / kGk * kGk; }
static unsigned grid_rows(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 32768); }

// X has to be copied (and brought into processing order)
static bool copies_x(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* w) {
  if (w->perm || !aligned16(X) || (ldx % 8) != 0) return true;
  return m > kSkinnyMax && (w->d_in % kGk != 0 || ldx * 2 > kMaxRowBytes);
}
static size_t x_copy_bytes(int64_t m, int d_in) { return align_up((size_t)m * pad_k(d_in) * 2); }

static int order_x(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* w, uint16_t* out, hipStream_t s) {
  const int Kp = pad_k(w->d_in);
  x_order_kernel<<<dim3((unsigned)((Kp / 8 + 255) / 256), grid_rows(m)), 256, 0, s>>>(
      static_cast<const uint16_t*>(X), ldx, m, w->d_in, w->perm, Kp, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T, int NMAT, typename Epi>
static int launch_skinny(const uint16_t* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb,
                         const Epi& epi, hipStream_t s) {
  const int G = w4_group(wa), d_out = wa->d_out, d_in = wa->d_in, ng = wa->n_groups;
  const W4Dev a = dev_of(wa), b = dev_of(wb);
  const bool fast = (d_in % 32) == 0 && (G % 32) == 0 && aligned16(a.packed) && aligned16(b.packed);
  auto go = [&]<int MT, int NT, bool FAST>() {
    w4_skinny_kernel<T, MT, NT, NMAT, 8, FAST, Epi><<<(unsigned)((d_out + 16 * MT - 1) / (16 * MT)), 512, 0, s>>>(
        X, ldx, (int)m, a, b, d_out, d_in, G, ng, epi);
  };
  if (fast) {
    if (m <= 16) go.template operator()<1, 1, true>();
    else if (m <= 32) go.template operator()<1, 2, true>();
    else go.template operator()<1, 4, true>();
  } else {
    if (m <= 16) go.template operator()<1, 1, false>();
    else if (m <= 32) go.template operator()<1, 2, false>();
    else go.template operator()<1, 4, false>();
  }
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T, typename Epi>
static int launch_gemm16(Gemm16Args g, const Epi& epi, hipStream_t s) {
  auto tiles = [&](int tm, int tn) { return ((g.m + tm - 1) / tm) * (int64_t)((g.n + tn - 1) / tn); };
  // A round of 256 large tiles takes 1, one of 512 small ones (two a CU) 2/3.
  const int64_t r256 = (tiles(256, 256) + 255) / 256, r128 = (tiles(128, 128) + 511) / 512;
  const bool big = 3 * r256 <= 2 * r128;
  const int64_t t = big ? tiles(256, 256) : tiles(128, 128);
  if (t > INT_MAX / 16) return GPTQ_ERR_INVALID_ARG;
  const int e = big ? 256 : 128;
  g.tiles_m = (int)((g.m + e - 1) / e);
  g.tiles_n = (g.n + e - 1) / e;
  const unsigned grid = (unsigned)(8 * ((t + 7) / 8));
  if (big) gemm16_kernel<T, 4, 2, 2, 4, Epi><<<grid, 512, 0, s>>>(g, epi);
  else gemm16_kernel<T, 2, 2, 2, 2, Epi><<<grid, 256, 0, s>>>(g, epi);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <typename T>
static int launch_dense(const gptq_w4_weight* wa, const gptq_w4_weight* wb, uint16_t* out, hipStream_t s) {
  const int Kp = pad_k(wa->d_in);
  w4_dense_kernel<T><<<dim3((unsigned)((Kp / 8 + 255) / 256), grid_rows(wa->d_out), wb ? 2 : 1), 256, 0, s>>>(
      dev_of(wa), wb ? dev_of(wb) : W4Dev{nullptr, nullptr, nullptr}, wa->d_out, wa->d_in, w4_group(wa), wa->n_groups, Kp, out);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

// one or both products of X with packed weights, and the epilogue
template <typename T, typename Epi>
static int forward(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb, const Epi& epi,
                   void* ws, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  const uint16_t* x = static_cast<const uint16_t*>(X);
  if (copies_x(X, ldx, m, wa)) {
    uint16_t* xc = reinterpret_cast<uint16_t*>(base);
    const int st = order_x(X, ldx, m, wa, xc, s);
    if (st != GPTQ_OK) return st;
    x = xc;
    ldx = pad_k(wa->d_in);
  }
  if (m <= kSkinnyMax) {
    return launch_skinny<T, Epi::kPlanes>(x, ldx, m, wa, wb ? wb : wa, epi, s);
  } else {
    uint16_t* w16 = reinterpret_cast<uint16_t*>(base + x_copy_bytes(m, wa->d_in));
    const int st = launch_dense<T>(wa, wb, w16, s);
    if (st != GPTQ_OK) return st;
    const int Kp = pad_k(wa->d_in), n = wb ? 2 * ((wa->d_out + 31) / 32 * 32) : wa->d_out;
    return launch_gemm16<T>(Gemm16Args{x, x, ldx, w16, Kp, m, n, Kp / kGk, Kp / kGk, 0, 0}, epi, s);
  }
}

static size_t forward_bytes(int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  const size_t rows = wb ? 2 * (size_t)((wa->d_out + 31) / 32 * 32) : (size_t)wa->d_out;
  return x_copy_bytes(m, wa->d_in) + (m > kSkinnyMax ? align_up(rows * pad_k(wa->d_in) * 2) : 0);
}
// what this call touches of it
static size_t forward_needs(const void* X, int64_t ldx, int64_t m, const gptq_w4_weight* wa, const gptq_w4_weight* wb) {
  if (m <= kSkinnyMax && !copies_x(X, ldx, m, wa)) return 0;
  return forward_bytes(m, wa, wb);
}

static bool pair_ok(const gptq_w4_weight* a, const gptq_w4_weight* b) {
  return w4_ok(a) && w4_ok(b) && a->d_out == b->d_out && a->d_in == b->d_in && w4_group(a) == w4_group(b) && a->perm == b->perm;
}
static bool is16(gptq_dtype t) { return t == GPTQ_F16 || t == GPTQ_BF16; }
static bool is_gate(gptq_act a) { return a == GPTQ_ACT_SILU || a == GPTQ_ACT_GELU || a == GPTQ_ACT_GELU_TANH; }
// 2-byte (4-byte for fp32) alignment of every element pointer
static bool elem_ok(const void* p, gptq_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == GPTQ_F32 ? 3 : 1)) == 0; }

struct BackLayout {
  size_t off_g, off_u, total;
  int Fp;
};
static BackLayout back_layout(int64_t m, const gptq_w4_weight* w) {
  BackLayout L;
  L.Fp = pad_k(w->d_out);
  L.off_g = align_up((size_t)w->d_in * 2 * L.Fp * 2);
  L.off_u = L.off_g + align_up((size_t)m * L.Fp * 2);
  L.total = L.off_u + align_up((size_t)m * L.Fp * 2);
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
  return launch_gemm16<T>(Gemm16Args{a0, a1, L.Fp, wt, 2 * L.Fp, m, d, L.Fp / kGk, 2 * L.Fp / kGk, 0, 0}, epi, s);
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
  if (!ws || ws_bytes < back_layout(m, gate).total || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  if (dtype == GPTQ_BF16) return backward<__bf16>(dM, G, U, m, gate, up, act, dG, dU, dX, ws, s);
  return backward<_Float16>(dM, G, U, m, gate, up, act, dG, dU, dX, ws, s);
}
