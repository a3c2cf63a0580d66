// What happens to the fp32 sums of a product on the packed layer: N
// neighbouring outputs of one token at a time (N = 4 or 8), bias, activation
// and residual (or activation(gate) * up) in fp32, one rounding to the
// output's type.
#pragma once
#include "w4.h"

namespace gptq {

// N 16-bit values at p as floats / from floats; vec: p is 2N-byte aligned and
// all N exist, else the first `have` are touched one by one
template <typename T, int N> GPTQ_DEV void load_n(const uint16_t* p, bool vec, int have, float (&v)[N]) {
  if (vec) {
    uint32_t w[N / 2];
    if constexpr (N == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      v[2 * e] = lo16f<T>(w[e]);
      v[2 * e + 1] = hi16f<T>(w[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < have ? (float)__builtin_bit_cast(T, p[e]) : 0.0f;
  }
}
template <typename T, int N> GPTQ_DEV void store_n(uint16_t* p, bool vec, int have, const float (&v)[N]) {
  if (vec) {
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) w[e] = pack2<T>(v[2 * e], v[2 * e + 1]);
    if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(w);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < have) p[e] = bits16<T>(v[e]);
  }
}
template <int N> GPTQ_DEV void load_f32(const float* p, bool vec, int have, float (&v)[N]) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    if (vec) {
      const float4 t = reinterpret_cast<const float4*>(p)[q];
      v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
    } else {
#pragma unroll
      for (int e = 4 * q; e < 4 * q + 4; ++e) v[e] = e < have ? p[e] : 0.0f;
    }
  }
}
template <int N> GPTQ_DEV void store_f32(float* p, bool vec, int have, const float (&v)[N]) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    if (vec) {
      reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
      for (int e = 4 * q; e < 4 * q + 4; ++e)
        if (e < have) p[e] = v[e];
    }
  }
}

// Y = act(sum + bias) + R
template <typename T> struct LinearEpi {
  static constexpr int kPlanes = 1;
  const uint16_t* bias;
  const void* R;
  void* Y;
  int64_t ldr, ldy;
  int n;
  int act, y_type;
  bool vec;               // rows of Y and R allow whole stores of N values

  template <int N> GPTQ_DEV void finish(float (&v)[1][N], int64_t tok, int c) const {
    const int have = n - c;
    if (have <= 0) return;
    const bool full = vec && have >= N;
    float (&x)[N] = v[0];
    if (bias) {
      float b[N];
      load_n<T, N>(bias + c, false, have, b);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] += b[e];
    }
    with_act(act, [&]<int ACT>() {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = act_fn<ACT>(x[e]);
    });
    if (R) {
      float r[N];
      if (y_type == GPTQ_F32) load_f32<N>(static_cast<const float*>(R) + tok * ldr + c, full, have, r);
      else if (y_type == GPTQ_BF16) load_n<__bf16, N>(static_cast<const uint16_t*>(R) + tok * ldr + c, full, have, r);
      else load_n<_Float16, N>(static_cast<const uint16_t*>(R) + tok * ldr + c, full, have, r);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] += r[e];
    }
    if (y_type == GPTQ_F32) store_f32<N>(static_cast<float*>(Y) + tok * ldy + c, full, have, x);
    else if (y_type == GPTQ_BF16) store_n<__bf16, N>(static_cast<uint16_t*>(Y) + tok * ldy + c, full, have, x);
    else store_n<_Float16, N>(static_cast<uint16_t*>(Y) + tok * ldy + c, full, have, x);
  }
};

// M = act(gate sum) * up sum, and the rounded sums where they are kept
template <typename T> struct GatedEpi {
  static constexpr int kPlanes = 2;
  uint16_t *G, *U, *M;    // G and U: both or neither
  int n;
  int act;
  bool vec;

  template <int N> GPTQ_DEV void finish(float (&v)[2][N], int64_t tok, int c) const {
    const int have = n - c;
    if (have <= 0) return;
    const bool full = vec && have >= N;
    const int64_t at = tok * n + c;
    if (G) {
      store_n<T, N>(G + at, full, have, v[0]);
      store_n<T, N>(U + at, full, have, v[1]);
    }
    with_act(act, [&]<int ACT>() {
#pragma unroll
      for (int e = 0; e < N; ++e) v[0][e] = act_fn<ACT>(v[0][e]) * v[1][e];
    });
    store_n<T, N>(M + at, full, have, v[0]);
  }
};

}  // namespace gptq
