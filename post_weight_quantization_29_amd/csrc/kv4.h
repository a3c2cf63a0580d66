// Shared pieces of the 4-bit cache: where a token's rows are, and the parts of
// an attention call.
#pragma once
#include "w4.h"

namespace gptq {

struct KvDev {
  uint32_t* k_codes;
  uint32_t* v_codes;
  uint32_t* k_grid;        // a row's (step, lo) as one word
  uint32_t* v_grid;
  const int32_t* table;
  int n_pages, n_kv, page, n_seqs, max_pages;
  int page_shift;          // log2(page), or -1
};

// One batch: where a sequence's new tokens are and how long it is.
struct KvBatch {
  const int32_t* q_start;
  const int32_t* kv_len;
  int64_t n_tokens;
  // first new token and their number, cut to the rows that exist
  GPTQ_DEV void span(int b, int64_t& t0, int& n_q) const {
    const int64_t a = max((int64_t)q_start[b], (int64_t)0), e = min((int64_t)q_start[b + 1], n_tokens);
    t0 = a;
    n_q = (int)max(e - a, (int64_t)0);
  }
};

// The sequence that token t belongs to, or -1 (t wave-uniform, all lanes
// active): q_start does not decrease, so it is the number of starts <= t,
// less one; sequences without new tokens have their successor's start and are
// passed over.
GPTQ_DEV int seq_of_token(const int32_t* q_start, int n_seqs, int64_t t) {
  const int lane = threadIdx.x & 63;
  int count = 0;
  for (int i0 = 0; i0 <= n_seqs; i0 += 64) {
    const bool le = i0 + lane <= n_seqs && (int64_t)q_start[i0 + lane] <= t;
    const int c = __popcll(__ballot(le));
    count += c;
    if (c < 64) break;
  }
  return count >= 1 && count <= n_seqs ? count - 1 : -1;
}

// Row of position p of sequence b, kv head h; -1 where there is none.  Rows
// and positions are counted in 32 bits (the host checks that they fit).
GPTQ_DEV int kv_row(const KvDev& c, int b, int h, int64_t p) {
  if (p < 0 || p >= (int64_t)c.max_pages * c.page) return -1;
  const uint32_t q = (uint32_t)p;
  const uint32_t i = c.page_shift >= 0 ? q >> c.page_shift : q / (uint32_t)c.page;
  const int pg = c.table[(int64_t)b * c.max_pages + i];
  if (pg < 0 || pg >= c.n_pages) return -1;
  return (pg * c.n_kv + h) * c.page + (int)(q - i * (uint32_t)c.page);
}

GPTQ_DEV float grid_step(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
GPTQ_DEV float grid_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }

// Codes as exact 16-bit numbers 16 + code, two at a time: a number in [16, 32)
// has steps of 2^-6 in fp16 and 2^-3 in bf16, so a code shifted to bit 6 (bit
// 3) of a half and or-ed onto 16.0 is 16 + code.  kBit is that bit.
template <typename T> struct Code16;
template <> struct Code16<__bf16> {
  static constexpr int kBit = 3;
  static constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
};
template <> struct Code16<_Float16> {
  static constexpr int kBit = 6;
  static constexpr uint32_t kMask = 0x03C003C0u, kBase = 0x4C004C00u;
};
constexpr float kCodeBase = 16.0f;

// 16 + the codes at bits 4k and 4k + 16 of w (k = 0..3)
template <typename T, int K> GPTQ_DEV uint32_t code_pair(uint32_t w) {
  constexpr int sh = 4 * K - Code16<T>::kBit;
  const uint32_t v = sh >= 0 ? w >> (sh >= 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
  return and_or(v, Code16<T>::kMask, Code16<T>::kBase);
}
// a word's eight codes: elements in the order 0 4 1 5 2 6 3 7
template <typename T> GPTQ_DEV uint4 code_word(uint32_t w) {
  return make_uint4(code_pair<T, 0>(w), code_pair<T, 1>(w), code_pair<T, 2>(w), code_pair<T, 3>(w));
}
// eight 16-bit values brought into that order
GPTQ_DEV uint4 code_order(uint4 v) {
  return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                    __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

}  // namespace gptq
