// The residual stream between two sub-layers and its norms, forward and
// backward, a row (token) at a time:
//
//   b = B, or unit(B) * post_gamma          unit(x) = x / sqrt(mean x^2 + eps)
//   h = R + alpha * gate * b
//   y = unit(h) * gamma
//
// and, from dY and what reaches the stream from elsewhere (dH), at the stored h:
//
//   n = unit(h) = r h,  g = dY gamma,  dh = dH + r (g - n mean(g n)),  dgamma = sum_t dY n
//   db = alpha gate dh,  dgate = alpha sum_t dh b
//   with a norm behind the sub-layer: u = unit(B) = q B,  g' = db post_gamma,
//   dB = q (g' - u mean(g' u)),  dpost_gamma = sum_t db u
//
// Bound by memory: each array passes once.  A group of T threads (whole waves)
// takes a row and holds it in registers, eight values a thread and chunk, so
// that a row is read once whatever its reductions; a workgroup of up to 1024
// threads has as many groups as fit, and keeps the column sums of the rows that
// it walks in registers.
#include "w4_epilogue.h"

#include <climits>

namespace gptq {

constexpr int kNormMax = 16384;        // two chunks of eight for each of 1024 threads
// Workgroups of the backward pass, each with its column sums: one a CU.  128, 256 and 512, us, 16-bit with
// all gradients: 4095 rows of 4096 81, 56 and 69, 512 of them 23, 21 and 21, 16384 of 1024 72, 52 and 62,
// 1024 of 16384 259, 180 and 219.
constexpr int kNormParts = 256;

struct NormArgs {
  const void *R, *B;          // forward: stream in, branch; backward: R is dH
  const void *H;              // backward: the stored stream
  const void *dY;
  const float *gamma, *post, *gate;
  void *Hout, *Y;             // forward: stream out, normed; backward: dR, dB
  float *part;                // backward: [workgroup][sum][d]
  int64_t ldr, ldb, ldh, ldy, ldho, ldyo;
  int64_t m;
  int d, T, groups;           // threads of a row, rows of a workgroup at a time
  float alpha, eps;
  bool vec, wvec;             // every row, every vector allows 16-byte loads
  bool want_gamma, want_post, want_gate;
};

// eight values of a 16-bit or 32-bit type
template <typename T> GPTQ_DEV void load8(const void* p, int64_t at, bool vec, int have, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) load_f32<8>(static_cast<const float*>(p) + at, vec, have, v);
  else load_n<T, 8>(static_cast<const uint16_t*>(p) + at, vec, have, v);
}
template <typename T> GPTQ_DEV void store8(void* p, int64_t at, bool vec, int have, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) store_f32<8>(static_cast<float*>(p) + at, vec, have, v);
  else store_n<T, 8>(static_cast<uint16_t*>(p) + at, vec, have, v);
}

// The same as they lie, for loads that are to be under way for a while
template <typename T> struct Raw8 {
  uint4 v[sizeof(T) / 2];
  GPTQ_DEV void load(const void* p, int64_t at) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (int64_t)sizeof(T));
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) v[k] = q[k];
  }
  GPTQ_DEV void get(float (&x)[8]) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          x[4 * k + e] = __builtin_bit_cast(float, w[e]);
        } else {
          x[2 * e] = lo16f<T>(w[e]);
          x[2 * e + 1] = hi16f<T>(w[e]);
        }
      }
    }
  }
};

// the sum of a wave's lanes, in all of them: inside rows of 16 by DPP, then across
GPTQ_DEV float wave_sum(float x) {
  auto add = [&]<int CTRL>() {
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
  };
  add.template operator()<0xB1>();       // quad_perm 1, 0, 3, 2
  add.template operator()<0x4E>();       // quad_perm 2, 3, 0, 1
  add.template operator()<0x141>();      // row_half_mirror
  add.template operator()<0x140>();      // row_mirror
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto v = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  x = __builtin_bit_cast(float, (uint32_t)v[0]) + __builtin_bit_cast(float, (uint32_t)v[1]);
  const uint32_t c = __builtin_bit_cast(uint32_t, x);
  const auto w = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return __builtin_bit_cast(float, (uint32_t)w[0]) + __builtin_bit_cast(float, (uint32_t)w[1]);
}

// Sums of N values over a row's threads, the same in all of them: over a wave's
// lanes, then over its waves in order.  `red` is two halves of kRowSums; a call takes
// the half that the one before it did not, so one barrier a call is enough (both halves hold
// the most values that a call sums: with halves of 16 N, one value's second half lay in three
// values' first, which a slower wave was still reading).
constexpr int kRowSums = 16 * 3;
template <int N>
GPTQ_DEV void row_sums(float (&v)[N], float* red, int& turn, int waves) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  const int w = threadIdx.x >> 6, first = w / waves * waves;
  static_assert(16 * N <= kRowSums);
  float* r = red + turn * kRowSums;
  turn ^= 1;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[w * N + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.0f;
  for (int i = first; i < first + waves; ++i)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += r[i * N + k];
}

// One pass, the next row's loads under way while this one's sums are made.  8192 rows of
// 5120 with an fp32 stream and norms before and behind: 503 MB in 107 us, 4.7 TB/s, the rate of
// a large copy within 10 %.
template <typename TH, typename TB, int NC>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a) {
  __shared__ float red[2 * kRowSums];
  const int group = threadIdx.x / a.T, t = threadIdx.x - group * a.T, waves = a.T >> 6;
  int turn = 0;
  // the vectors stay in registers for all the rows that the workgroup walks (1 past the row's end)
  float wp[NC][8], wg[NC][8], wy[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = 8 * (t + k * a.T), have = a.d - c;
#pragma unroll
    for (int e = 0; e < 8; ++e) wp[k][e] = wg[k][e] = wy[k][e] = 1.0f;
    if (have > 0) {
      if (a.post) load_f32<8>(a.post + c, a.wvec && have >= 8, have, wp[k]);
      if (a.gate) load_f32<8>(a.gate + c, a.wvec && have >= 8, have, wg[k]);
      if (a.gamma && a.Y) load_f32<8>(a.gamma + c, a.wvec && have >= 8, have, wy[k]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) wg[k][e] *= a.alpha;
  }
  // the next row's values are on their way while a row is worked on
  Raw8<TH> rh[NC];
  Raw8<TB> rb[NC];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T);
      if (row < a.m && a.vec && a.d - c >= 8) {
        rh[k].load(a.R, row * a.ldr + c);
        if (a.B) rb[k].load(a.B, row * a.ldb + c);
      }
    }
  };
  fetch((int64_t)blockIdx.x * a.groups + group);
  for (int64_t row0 = (int64_t)blockIdx.x * a.groups; row0 < a.m; row0 += (int64_t)gridDim.x * a.groups) {
    const int64_t row = row0 + group;
    const bool in = row < a.m;
    float h[NC][8], b[NC][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = b[k][e] = 0.0f;          // and 0 past the row's end
      if (a.vec && have >= 8) {
        rh[k].get(h[k]);
        if (a.B) rb[k].get(b[k]);
      } else if (have > 0) {
        load8<TH>(a.R, row * a.ldr + c, false, have, h[k]);
        if (a.B) load8<TB>(a.B, row * a.ldb + c, false, have, b[k]);
      }
    }
    fetch(row + (int64_t)gridDim.x * a.groups);
    if (a.B) {
      float q = 1.0f;
      if (a.post) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[0] += b[k][e] * b[k][e];
        row_sums<1>(sum, red, turn, waves);
        q = 1.0f / sqrtf(sum[0] / (float)a.d + a.eps);
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] = fmaf(b[k][e] * (q * wp[k][e]), wg[k][e], h[k][e]);
        if (a.Hout && have > 0) store8<TH>(a.Hout, row * a.ldho + c, a.vec && have >= 8, have, h[k]);
      }
    }
    if (!a.Y) continue;
    sum[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += h[k][e] * h[k][e];
    row_sums<1>(sum, red, turn, waves);
    const float r = 1.0f / sqrtf(sum[0] / (float)a.d + a.eps);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] *= r * wy[k][e];
      if (have > 0) store8<TB>(a.Y, row * a.ldyo + c, a.vec && have >= 8, have, h[k]);
    }
  }
}

// The rows of a workgroup one after the other, their column sums in registers (one chunk a
// thread: the vectors and the next row's loads too).  MORE: there is a gate or a norm
// behind the sub-layer, whose column sums take registers that the plain residual does not spend.
// 4095 rows of 4096, 16-bit, all gradients: 201 MB in 62 us, 3.2 TB/s: three sums over a row
// that wait for each other, at two rows a CU under way.
template <typename TH, typename TB, int NC, bool MORE>
__global__ __launch_bounds__(1024) void residual_norm_backward_kernel(NormArgs a) {
  __shared__ float red[2 * kRowSums];
  extern __shared__ float cols[];
  const int group = threadIdx.x / a.T, t = threadIdx.x - group * a.T, waves = a.T >> 6;
  int turn = 0;
  float sg[NC][8], sp[MORE ? NC : 1][8], sq[MORE ? NC : 1][8];
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sg[k][e] = 0.0f;
      if constexpr (MORE) sp[k][e] = sq[k][e] = 0.0f;
    }
  // the next row's values are on their way while a row is worked on (one chunk a
  // thread: with two there are no registers for it)
  constexpr bool kAhead = NC == 1;
  Raw8<TH> rh[NC], rx[NC];
  Raw8<TB> rg[NC], rb[NC];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T);
      if (row < a.m && a.vec && a.d - c >= 8) {
        rh[k].load(a.H, row * a.ldh + c);
        rg[k].load(a.dY, row * a.ldy + c);
        if (a.R) rx[k].load(a.R, row * a.ldr + c);
        if constexpr (MORE) rb[k].load(a.B, row * a.ldb + c);
      }
    }
  };
  // the vectors (1 where there is none) stay in registers likewise: loaded where they
  // are used, four times a row, they cost as much as the rows did
  float vg[kAhead ? NC : 1][8], vp[kAhead && MORE ? NC : 1][8], vw[kAhead && MORE ? NC : 1][8];
  auto vector = [&](const float* v, int c, float (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    if (v && c < a.d) load_f32<8>(v + c, a.wvec && a.d - c >= 8, a.d - c, w);
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T);
      vector(a.gamma, c, vg[k]);
      if constexpr (MORE) {
        vector(a.post, c, vp[k]);
        vector(a.gate, c, vw[k]);
      }
    }
    fetch((int64_t)blockIdx.x * a.groups + group);
  }
  for (int64_t row0 = (int64_t)blockIdx.x * a.groups; row0 < a.m; row0 += (int64_t)gridDim.x * a.groups) {
    const int64_t row = row0 + group;
    const bool in = row < a.m;
    float h[NC][8], g[NC][8], b[NC][8], x[NC][8];
    float sum[3] = {0.0f, 0.0f, 0.0f};
    if constexpr (!kAhead) fetch(row);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = g[k][e] = b[k][e] = x[k][e] = 0.0f;
      if (a.vec && have >= 8) {
        rh[k].get(h[k]);
        rg[k].get(g[k]);
        if (a.R) rx[k].get(x[k]);
        if constexpr (MORE) rb[k].get(b[k]);
      } else if (have > 0) {
        load8<TH>(a.H, row * a.ldh + c, false, have, h[k]);
        load8<TB>(a.dY, row * a.ldy + c, false, have, g[k]);
        if (a.R) load8<TH>(a.R, row * a.ldr + c, false, have, x[k]);
        if constexpr (MORE) load8<TB>(a.B, row * a.ldb + c, false, have, b[k]);
      }
    }
    if constexpr (kAhead) fetch(row + (int64_t)gridDim.x * a.groups);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      float other[8];
      if constexpr (!kAhead) vector(a.gamma, 8 * (t + k * a.T), other);
      const float (&w)[8] = kAhead ? vg[kAhead ? k : 0] : other;
#pragma unroll
      for (int e = 0; e < 8; ++e) {          // all 0 past the row's end
        sum[0] += h[k][e] * h[k][e];
        sum[1] += g[k][e] * w[e] * h[k][e];
        if constexpr (MORE) sum[2] += b[k][e] * b[k][e];
      }
    }
    row_sums<3>(sum, red, turn, waves);
    // (0 in a row that does not exist: with eps 0 its zeros' root has no inverse, and the column sums take all rows)
    const float r = in ? 1.0f / sqrtf(sum[0] / (float)a.d + a.eps) : 0.0f;
    const float mean = sum[1] * r / (float)a.d;            // mean(g n)
    const float q = !in ? 0.0f : MORE && a.post ? 1.0f / sqrtf(sum[2] / (float)a.d + a.eps) : 1.0f;
    float dot[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
      float other[8];
      if constexpr (!kAhead) vector(a.gamma, c, other);
      const float (&w)[8] = kAhead ? vg[kAhead ? k : 0] : other;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[k][e] * r;
        sg[k][e] += g[k][e] * n;
        x[k][e] += r * (g[k][e] * w[e] - n * mean);        // dh
      }
      if (have > 0 && a.Hout) store8<TH>(a.Hout, row * a.ldho + c, a.vec && have >= 8, have, x[k]);
      if (!a.Y && !a.want_post && !a.want_gate) continue;
      if constexpr (MORE) {
        float other_p[8], other_g[8];
        if constexpr (!kAhead) {
          vector(a.post, c, other_p);
          vector(a.gate, c, other_g);
        }
        const float (&wp)[8] = kAhead ? vp[kAhead ? k : 0] : other_p;
        const float (&wg)[8] = kAhead ? vw[kAhead ? k : 0] : other_g;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          b[k][e] *= q;
          x[k][e] *= a.alpha;
          sq[k][e] += x[k][e] * (b[k][e] * wp[e]);
          const float db = wg[e] * x[k][e];
          sp[k][e] += db * b[k][e];
          x[k][e] = db * wp[e];
          dot[0] += x[k][e] * b[k][e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= a.alpha;
      }
    }
    if (!a.Y) continue;
    if constexpr (MORE) {
      if (a.post) {
        row_sums<1>(dot, red, turn, waves);
        const float mean_u = dot[0] / (float)a.d;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = q * (x[k][e] - b[k][e] * mean_u);
      }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T), have = in ? a.d - c : 0;
      if (have > 0) store8<TB>(a.Y, row * a.ldyo + c, a.vec && have >= 8, have, x[k]);
    }
  }
  // the workgroup's column sums: its groups' in order
  auto put = [&](float (&s)[NC][8], int plane) {
    __syncthreads();
    if (a.groups > 1) {
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) cols[(group * 8 + e) * (NC * a.T) + t + k * a.T] = s[k][e];
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = 8 * (t + k * a.T);
      for (int o = 1; o < a.groups; ++o)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[k][e] += cols[(o * 8 + e) * (NC * a.T) + t + k * a.T];
      if (c < a.d)
        store_f32<8>(a.part + ((int64_t)blockIdx.x * 3 + plane) * ((a.d + 3) & ~3) + c, a.d - c >= 8, a.d - c, s[k]);
    }
  };
  if (a.want_gamma) put(sg, 0);
  if constexpr (MORE) {
    if (a.want_post) put(sp, 1);
    if (a.want_gate) put(sq, 2);
  }
}

// The workgroups' column sums, 64 columns a workgroup: sixteen threads to a column
// take every sixteenth part each, and their sums are added in order (5 us for three sums of
// 4096 columns of 256 parts).
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* __restrict__ part, int parts, int d, float* o0, float* o1,
                                                            float* o2) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int x = threadIdx.x & 63, c = blockIdx.x * 64 + x, k = threadIdx.x >> 6;
  const int64_t pitch = (d + 3) & ~3;
  float v = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int p = k; p < parts; p += 16) v += part[((int64_t)p * 3 + blockIdx.y) * pitch + c];
  }
  s[k][x] = v;
  __syncthreads();
  if (k == 0 && c < d) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += s[w][x];
    out[c] = v;
  }
}

// Threads of a row: whole waves, one chunk of eight values each up to 8192 values, then two (in the
// backward pass two chunks leave no registers for the vectors and the next row: 4095 rows of 4096 in
// half as many threads 189 us for 56, without post-norm and gate 36 for 34).
struct NormShape {
  int T, groups, nc;
};
static NormShape norm_shape(int d) {
  NormShape s;
  s.nc = d > 8192 ? 2 : 1;
  s.T = (d + 512 * s.nc - 1) / (512 * s.nc) * 64;
  s.groups = 1024 / s.T;
  return s;
}
// Forward, where there are rows enough: two chunks a thread and one row a
// workgroup, so that more rows are under way in a CU and fewer waves meet at a barrier.  One
// chunk and two, fp32 stream, norms before and behind: 1024 rows of 5120 19.2 and 17.4 us, 2048
// 32.1 and 27.7, 8192 112 and 106 (of 8192 values 162 and 167, of 4096 84 and 84, of 2048 43 and 37,
// of 1000 24.3 and 22.5, of 512, where the second chunk is behind every row's end, 14.6 and 13.9, of 128
// and 64 both the launch's 9); below 1024 rows the same within 4 %, and a single row has more threads.
static NormShape forward_shape(int64_t m, int d) {
  NormShape s = norm_shape(d);
  if (m < 1024) return s;
  s.nc = 2;
  s.T = (d + 512 * s.nc - 1) / (512 * s.nc) * 64;
  s.groups = 1;
  return s;
}
static int norm_parts(int64_t m, int groups) { return (int)std::min<int64_t>(kNormParts, (m + groups - 1) / groups); }

static bool norm_types_ok(gptq_dtype h, gptq_dtype b) {
  if (h != GPTQ_F32 && h != GPTQ_F16 && h != GPTQ_BF16) return false;
  if (b != GPTQ_F32 && b != GPTQ_F16 && b != GPTQ_BF16) return false;
  return h == b || h == GPTQ_F32;
}
static bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
static int norm_bytes(gptq_dtype t) { return t == GPTQ_F32 ? 4 : 2; }
// a row of this type and pitch allows 16-byte loads
static bool wide(const void* p, int64_t ld, gptq_dtype t) { return !p || (on(p, 16) && ld % (16 / norm_bytes(t)) == 0); }
// Whether an output may lie where another array does: apart from it, or, for an
// input that each thread reads before it writes the same place, on the whole of it.
struct NormRows {
  const void* p;
  int64_t ld;
  gptq_dtype t;
};
static bool apart(NormRows a, NormRows b, int64_t m, int d) {
  if (!a.p || !b.p) return true;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t na = rows_bytes(m, a.ld, d, norm_bytes(a.t)), nb = rows_bytes(m, b.ld, d, norm_bytes(b.t));
  return x >= y + nb || y >= x + na;
}
// an array that is a vector or scratch, against rows
static bool rows_meet(NormRows a, int64_t m, int d, const void* p, uint64_t bytes) {
  return share_bytes(a.p, rows_bytes(m, a.ld, d, norm_bytes(a.t)), p, bytes);
}
static bool same_or_apart(NormRows a, NormRows b, int64_t m, int d) {
  return (a.p == b.p && a.ld == b.ld && a.t == b.t) || apart(a, b, m, d);
}
static bool rows_ok(NormRows a, int d) { return !a.p || (a.ld >= d && on(a.p, norm_bytes(a.t))); }

// the kernel for the stream's and the branch's types
template <typename F> static void with_types(gptq_dtype h, gptq_dtype b, F&& f) {
  if (b == GPTQ_F32) f.template operator()<float, float>();
  else if (b == GPTQ_BF16 && h == GPTQ_BF16) f.template operator()<__bf16, __bf16>();
  else if (b == GPTQ_BF16) f.template operator()<float, __bf16>();
  else if (h == GPTQ_F16) f.template operator()<_Float16, _Float16>();
  else f.template operator()<float, _Float16>();
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_residual_rmsnorm(const void* R, gptq_dtype h_dtype, int64_t ldr, const void* B, gptq_dtype dtype, int64_t ldb,
                                     int64_t m, int32_t d, const float* post_gamma, const float* gate, float alpha,
                                     const float* gamma, float eps, void* H, int64_t ldh, void* Y, int64_t ldy, hipStream_t s) {
  if (!norm_types_ok(h_dtype, dtype) || m < 0 || m > INT_MAX || d <= 0 || d > kNormMax) return GPTQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(fabsf(alpha) < INFINITY) || !(eps < INFINITY)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!B && (post_gamma || gate || H)) return GPTQ_ERR_INVALID_ARG;
  const NormRows r{R, ldr, h_dtype}, b{B, ldb, dtype}, h{H, ldh, h_dtype}, y{Y, ldy, dtype};
  if (!R || (!H && !Y) || !rows_ok(r, d) || !rows_ok(b, d) || !rows_ok(h, d) || !rows_ok(y, d)) return GPTQ_ERR_INVALID_ARG;
  if (!on(gamma, 4) || !on(post_gamma, 4) || !on(gate, 4)) return GPTQ_ERR_INVALID_ARG;
  if (!apart(h, y, m, d) || !same_or_apart(h, r, m, d) || !same_or_apart(h, b, m, d) || !same_or_apart(y, r, m, d) ||
      !same_or_apart(y, b, m, d)) return GPTQ_ERR_INVALID_ARG;
  for (const float* p : {gamma, post_gamma, gate})
    if (rows_meet(h, m, d, p, (uint64_t)d * 4) || rows_meet(y, m, d, p, (uint64_t)d * 4)) return GPTQ_ERR_INVALID_ARG;
  const NormShape n = forward_shape(m, d);
  NormArgs a{};
  a.R = R; a.B = B; a.gamma = gamma; a.post = post_gamma; a.gate = gate; a.Hout = H; a.Y = Y;
  a.ldr = ldr; a.ldb = ldb; a.ldho = ldh; a.ldyo = ldy;
  a.m = m; a.d = d; a.T = n.T; a.groups = n.groups; a.alpha = alpha; a.eps = eps;
  a.vec = wide(R, ldr, h_dtype) && wide(B, ldb, dtype) && wide(H, ldh, h_dtype) && wide(Y, ldy, dtype);
  a.wvec = on(gamma, 16) && on(post_gamma, 16) && on(gate, 16);
  const unsigned grid = (unsigned)std::min<int64_t>((m + n.groups - 1) / n.groups, 256 * std::max(1, 12 / (n.T * n.groups / 64)));
  with_types(h_dtype, dtype, [&]<typename TH, typename TB>() {
    if (n.nc == 1) residual_norm_kernel<TH, TB, 1><<<grid, n.T * n.groups, 0, s>>>(a);
    else residual_norm_kernel<TH, TB, 2><<<grid, n.T * n.groups, 0, s>>>(a);
  });
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

extern "C" size_t gptq_residual_rmsnorm_backward_workspace_size(int64_t m, int32_t d) {
  if (m <= 0 || m > INT_MAX || d <= 0 || d > kNormMax) return 0;
  return align_up((size_t)norm_parts(m, norm_shape(d).groups) * 3 * ((d + 3) & ~3) * sizeof(float));
}

extern "C" int gptq_residual_rmsnorm_backward(const void* dY, gptq_dtype dtype, int64_t lddy, const void* H, gptq_dtype h_dtype,
                                              int64_t ldh, const void* dH, int64_t lddh, const void* B, int64_t ldb, int64_t m,
                                              int32_t d, const float* post_gamma, const float* gate, float alpha,
                                              const float* gamma, float eps, void* dR, int64_t lddr, void* dB, int64_t lddb,
                                              float* dgamma, float* dpost_gamma, float* dgate, void* ws, size_t ws_bytes,
                                              hipStream_t s) {
  if (!norm_types_ok(h_dtype, dtype) || m < 0 || m > INT_MAX || d <= 0 || d > kNormMax) return GPTQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(fabsf(alpha) < INFINITY) || !(eps < INFINITY)) return GPTQ_ERR_INVALID_ARG;
  const bool more = post_gamma || gate;
  if ((dpost_gamma && !post_gamma) || (dgate && !gate)) return GPTQ_ERR_INVALID_ARG;
  if (!on(dgamma, 4) || !on(dpost_gamma, 4) || !on(dgate, 4)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) {
    // sums over no rows
    norm_columns_kernel<<<dim3((unsigned)((d + 63) / 64), 3), 1024, 0, s>>>(nullptr, 0, d, dgamma, dpost_gamma, dgate);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  const NormRows y{dY, lddy, dtype}, h{H, ldh, h_dtype}, x{dH, lddh, h_dtype}, b{B, ldb, dtype}, r{dR, lddr, h_dtype}, o{dB, lddb, dtype};
  if (!dY || !H || (!B && more) || (!dR && !dB && !dgamma && !dpost_gamma && !dgate)) return GPTQ_ERR_INVALID_ARG;
  for (const NormRows& t : {y, h, x, b, r, o})
    if (!rows_ok(t, d)) return GPTQ_ERR_INVALID_ARG;
  for (const float* p : {gamma, post_gamma, gate})
    if (!on(p, 4)) return GPTQ_ERR_INVALID_ARG;
  if (!apart(r, o, m, d)) return GPTQ_ERR_INVALID_ARG;
  for (const NormRows& t : {y, h, x, b})
    if (!same_or_apart(r, t, m, d) || !same_or_apart(o, t, m, d)) return GPTQ_ERR_INVALID_ARG;
  // the sums, the vectors and the scratch: vectors may be one another, nothing else meets
  const uint64_t vb = (uint64_t)d * 4;
  const float *const vectors[] = {gamma, post_gamma, gate}, *const totals[] = {dgamma, dpost_gamma, dgate};
  for (const float* v : vectors)
    if (rows_meet(r, m, d, v, vb) || rows_meet(o, m, d, v, vb)) return GPTQ_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    for (const NormRows& t : {y, h, x, b, r, o})
      if (rows_meet(t, m, d, totals[i], vb)) return GPTQ_ERR_INVALID_ARG;
    for (const float* v : vectors)
      if (share_bytes(totals[i], vb, v, vb)) return GPTQ_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (share_bytes(totals[i], vb, totals[j], vb)) return GPTQ_ERR_INVALID_ARG;
  }
  const bool sums = dgamma || dpost_gamma || dgate;
  const size_t need = gptq_residual_rmsnorm_backward_workspace_size(m, d);
  if (sums && (!ws || ws_bytes < need || !on(ws, kAlign))) return GPTQ_ERR_WORKSPACE;
  if (sums) {
    for (const NormRows& t : {y, h, x, b, r, o})
      if (rows_meet(t, m, d, ws, need)) return GPTQ_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (share_bytes(vectors[i], vb, ws, need) || share_bytes(totals[i], vb, ws, need)) return GPTQ_ERR_INVALID_ARG;
  }
  const NormShape n = norm_shape(d);
  const int parts = norm_parts(m, n.groups);
  NormArgs a{};
  a.R = dH; a.B = B; a.H = H; a.dY = dY; a.gamma = gamma; a.post = post_gamma; a.gate = gate; a.Hout = dR; a.Y = dB;
  a.part = static_cast<float*>(ws);
  a.ldr = lddh; a.ldb = ldb; a.ldh = ldh; a.ldy = lddy; a.ldho = lddr; a.ldyo = lddb;
  a.m = m; a.d = d; a.T = n.T; a.groups = n.groups; a.alpha = alpha; a.eps = eps;
  a.vec = wide(dH, lddh, h_dtype) && wide(H, ldh, h_dtype) && wide(dY, lddy, dtype) && wide(dR, lddr, h_dtype) && wide(dB, lddb, dtype) &&
          (!more || wide(B, ldb, dtype));
  a.wvec = on(gamma, 16) && on(post_gamma, 16) && on(gate, 16);
  a.want_gamma = dgamma; a.want_post = dpost_gamma; a.want_gate = dgate;
  const size_t lds = n.groups > 1 ? (size_t)n.groups * 8 * n.nc * n.T * sizeof(float) : 0;
  with_types(h_dtype, dtype, [&]<typename TH, typename TB>() {
    auto go = [&]<int NC, bool MORE>() { residual_norm_backward_kernel<TH, TB, NC, MORE><<<parts, n.T * n.groups, lds, s>>>(a); };
    if (n.nc == 1) more ? go.template operator()<1, true>() : go.template operator()<1, false>();
    else more ? go.template operator()<2, true>() : go.template operator()<2, false>();
  });
  GPTQ_LAUNCH_CHECK();
  if (sums) {
    norm_columns_kernel<<<dim3((unsigned)((d + 63) / 64), 3), 1024, 0, s>>>(a.part, parts, d, dgamma, dpost_gamma, dgate);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}
