// Shared pieces of the operators on the packed 4-bit layer: 16-bit type
// traits, the exact dequantization of a word of codes, activations and their
// slopes, and the argument checks of a packed weight.
#pragma once
#include "common.h"

namespace gptq {

typedef float f32x2w_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2w_t __attribute__((ext_vector_type(2)));

// 16-bit activation types: conversions, the matrix instructions and a packed
// conversion of two floats (round to nearest, ties to even).
template <typename T> struct T16;
template <> struct T16<__bf16> {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  static constexpr gptq_dtype kType = GPTQ_BF16;
  static GPTQ_DEV f32x4_t mfma16(v8 a, v8 b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static GPTQ_DEV f32x16_t mfma32(v8 a, v8 b, f32x16_t c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <> struct T16<_Float16> {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  static constexpr gptq_dtype kType = GPTQ_F16;
  static GPTQ_DEV f32x4_t mfma16(v8 a, v8 b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static GPTQ_DEV f32x16_t mfma32(v8 a, v8 b, f32x16_t c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};

template <typename T> GPTQ_DEV uint32_t pack2(float a, float b) {
  const f32x2w_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename T16<T>::v2));
}
template <typename T> GPTQ_DEV uint16_t bits16(float a) { return __builtin_bit_cast(uint16_t, (T)a); }
template <typename T> GPTQ_DEV float lo16f(uint32_t p) { return (float)__builtin_bit_cast(T, (uint16_t)p); }
template <typename T> GPTQ_DEV float hi16f(uint32_t p) { return (float)__builtin_bit_cast(T, (uint16_t)(p >> 16)); }

// (v & mask) | base in one instruction: it takes one scalar operand, so the
// mask is held in a scalar and the base in a vector register (left to itself
// the compiler folds both as literals into two instructions)
GPTQ_DEV uint32_t and_or(uint32_t v, uint32_t mask, uint32_t base) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(mask), "v"(base));
  return r;
}

// ---------------------------------------------------------------- dequantization
// The eight weights of word p in order, as four packed pairs: w = RN16(RN32(
// scale * (code - zero))), bit for bit gptq_w4a16_gemm's.
//
// Two codes at a time: code k and code k + 4 of the word land in the low bits
// of the two halves of a register; or-ed onto 0x6400 they are the fp16
// numbers 1024 + code, and one packed fp16 addition of -(1024 + zero) makes
// the exact integers code - zero (exact while |zero| <= kZeroFast).  A mixed
// multiply reads an fp16 half as fp32, so a weight costs 2.9 vector
// instructions instead of the 3.9 of byte conversion, subtraction and
// multiplication; single-token products feel that count next to HBM (4096 -> 2 x
// 11008, one token: vector issue in 42 % of the cycles).
constexpr float kZeroFast = 1000.0f;

// an fp16 half of n, as fp32, times s plus a: one mixed instruction.  (Left to
// the compiler, not asm: it also places the waits that an operand fresh from a
// matrix instruction or an exponential needs.)
GPTQ_DEV float fma_lo(uint32_t n, float s, float a) {
  return __builtin_fmaf((float)__builtin_bit_cast(_Float16, (uint16_t)n), s, a);
}
GPTQ_DEV float fma_hi(uint32_t n, float s, float a) {
  return __builtin_fmaf((float)__builtin_bit_cast(_Float16, (uint16_t)(n >> 16)), s, a);
}

// -(1024 + zero) in both halves, for |zero| <= kZeroFast
GPTQ_DEV uint32_t zero_pair(float z) {
  const _Float16 h = (_Float16)(-1024.0f - z);
  const f16x2w_t v = {h, h};
  return __builtin_bit_cast(uint32_t, v);
}

template <typename T>
GPTQ_DEV void dequant_fast(uint32_t p, float s, uint32_t zp, uint32_t (&w)[4]) {
  float a[4], b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t c = and_or(p >> (4 * k), 0x000F000Fu, 0x64006400u);
    const f16x2w_t n = __builtin_bit_cast(f16x2w_t, c) + __builtin_bit_cast(f16x2w_t, zp);
    a[k] = fma_lo(__builtin_bit_cast(uint32_t, n), s, 0.0f);
    b[k] = fma_hi(__builtin_bit_cast(uint32_t, n), s, 0.0f);
  }
  w[0] = pack2<T>(a[0], a[1]);
  w[1] = pack2<T>(a[2], a[3]);
  w[2] = pack2<T>(b[0], b[1]);
  w[3] = pack2<T>(b[2], b[3]);
}

// any zero point
template <typename T>
GPTQ_DEV void dequant_any(uint32_t p, float s, float z, uint32_t (&w)[4]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = s * ((float)((p >> (4 * k)) & 15u) - z);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
}

// c / G for c >= 0, exact for c < 2^24 and any G >= 1 (the quotient of floats
// is off by at most one)
GPTQ_DEV int group_of(int c, int G, float invG) {
  int g = (int)((float)c * invG);
  if (g * G > c) --g;
  if ((g + 1) * G <= c) ++g;
  return g;
}

// ---------------------------------------------------------------- activations
// GELU with tanh: (1 + tanh z) / 2 = 1 / (1 + exp(-2z)), no cancellation.
constexpr float kGeluA = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <int ACT> GPTQ_DEV float act_fn(float x) {
  if constexpr (ACT == GPTQ_ACT_RELU) return x > 0.0f ? x : (x != x ? x : 0.0f);
  if constexpr (ACT == GPTQ_ACT_SILU) return x / (1.0f + expf(-x));
  if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * x * erfcf(-x * 0.70710678118654752f);
  if constexpr (ACT == GPTQ_ACT_GELU_TANH) return x / (1.0f + expf(-kGeluA * (x + kGeluB * x * x * x)));
  return x;
}
// d act / dx
template <int ACT> GPTQ_DEV float act_slope(float x) {
  if constexpr (ACT == GPTQ_ACT_SILU) {
    const float sg = 1.0f / (1.0f + expf(-x));
    return sg * (1.0f + x * (1.0f - sg));
  }
  if constexpr (ACT == GPTQ_ACT_GELU)
    return 0.5f * erfcf(-x * 0.70710678118654752f) + x * expf(-0.5f * x * x) * 0.39894228040143268f;
  if constexpr (ACT == GPTQ_ACT_GELU_TANH) {
    const float sg = 1.0f / (1.0f + expf(-kGeluA * (x + kGeluB * x * x * x)));
    // x^2 cut to where sg is 0 or 1 anyway: 0 times an overflow would be NaN
    return sg + x * sg * (1.0f - sg) * kGeluA * (1.0f + 3.0f * kGeluB * fminf(x * x, 1.0e4f));
  }
  return 1.0f;
}
// The activation is a run-time argument; callers apply it to a whole array of
// accumulators at once so that the choice is made once, not per element.
template <typename F> GPTQ_DEV void with_act(int act, F&& f) {
  switch (act) {
    case GPTQ_ACT_RELU: f.template operator()<GPTQ_ACT_RELU>(); break;
    case GPTQ_ACT_SILU: f.template operator()<GPTQ_ACT_SILU>(); break;
    case GPTQ_ACT_GELU: f.template operator()<GPTQ_ACT_GELU>(); break;
    case GPTQ_ACT_GELU_TANH: f.template operator()<GPTQ_ACT_GELU_TANH>(); break;
    default: break;
  }
}

// ---------------------------------------------------------------- host checks
constexpr int kW4MaxCols = 1 << 20;      // group_of() and the tiles' 32-bit row offsets hold to here
constexpr int kW4MaxRows = (1 << 27) - 32;   // so many rows' threads, 32 a row at most, can be launched (2^32 - 1)

inline bool w4_ok(const gptq_w4_weight* w) {
  if (!w || !w->packed || !w->scales || !w->zeros) return false;
  if (w->d_out <= 0 || w->d_in <= 0 || (w->d_in % 8) != 0 || w->d_in > kW4MaxCols || w->d_out > kW4MaxRows) return false;
  const int G = w->group_size == -1 ? w->d_in : w->group_size;
  if (G <= 0 || (G % 8) != 0) return false;
  if (w->n_groups != (w->d_in + (int64_t)G - 1) / G) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(w->packed) | reinterpret_cast<uintptr_t>(w->scales) |
                      reinterpret_cast<uintptr_t>(w->zeros) | reinterpret_cast<uintptr_t>(w->perm);
  return (a & 3) == 0;
}
inline int w4_group(const gptq_w4_weight* w) { return w->group_size == -1 ? w->d_in : w->group_size; }

}  // namespace gptq
