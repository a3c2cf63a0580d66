// Low-rank adapters of many requests beside a shared projection, forward and
// backward.  Token t of a sequence with adapter a:
//
//   s_t = A_a x_t                              [rank]
//   y_t = r_t + scale_a B_a s_t                [d_out]
//   dS_t = B_a' dy_t (unscaled),  dx_t = r_t + scale_a A_a' dS_t
//   dA_a = scale_a sum_t dS_t x_t',  dB_a = scale_a sum_t dy_t s_t'
//
// A batch mixes adapters token by token (a decode step) or in long runs
// (prompts), so the kernels go by blocks of 16 tokens and, inside one, by the
// adapters that occur in it: a product with one adapter's matrix is made for all
// 16 columns of the matrix instruction, and each token keeps the one of its own
// adapter (kept by selection, not by zeros: another request's infinities do not
// reach it).
//
// s and dS are fp32.  Where they are an operand of a matrix instruction they go in
// two pieces of the operands' 16-bit type (16 bits for bf16, 22 for fp16), whose error
// stays below that of rounding an output to this type; an fp32 Y or dX is as exact as the
// pieces, not as fp32 sums (a third piece would be half as much again of that product).  In
// dA and dB, always fp32, three bf16 ones.
#include "w4_epilogue.h"

#include <climits>

namespace gptq {

constexpr int kLoraMaxRank = 128, kLoraMaxDim = 1 << 20, kLoraMaxSets = 65535;
constexpr int kUpWaves = 4;

struct LoraBatch {
  const int32_t* q_start;
  const int32_t* adapter;
  int n_seqs, n_adapters;
  int64_t m;
};

constexpr int kNoAdapter = -1, kNoToken = -2;

// The adapters of tokens t0 .. t0 + 15 (lane i: token i % 16's): a token's
// sequence is the number of starts up to it, less one, so sequences without
// tokens are passed over.
GPTQ_DEV int adapter_of(const LoraBatch& b, int64_t t0) {
  const int lane = threadIdx.x & 63;
  int count = 0;
  for (int i0 = 0; i0 <= b.n_seqs; i0 += 64) {
    const int v = i0 + lane <= b.n_seqs ? b.q_start[i0 + lane] : INT_MAX;      // tokens are below 2^24
    int c = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      c = __popcll(__ballot(v <= (int)t0 + i));
      if ((lane & 15) == i) count += c;
    }
    if (c < 64) break;
  }
  if (count < 1 || count > b.n_seqs || t0 + (lane & 15) >= b.m) return kNoToken;
  const int a = b.adapter[count - 1];
  return a >= 0 && a < b.n_adapters ? a : kNoAdapter;
}

// Tile u of `tok` tokens of the batch, where tiles end with their sequences: its
// first row, tokens and adapter (or kNoAdapter); false if there are fewer.  By a
// running sum of the sequences' tiles; the same in all of a wave's lanes.
GPTQ_DEV bool run_tile(const LoraBatch& batch, uint32_t u, int tok, int64_t& t0, int& n, int& a) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < batch.n_seqs; s0 += 64) {
    const int b = s0 + lane;
    int lo = 0, hi = 0;                                // rows are below 2^24
    if (b < batch.n_seqs) {
      lo = max(batch.q_start[b], 0);
      hi = (int)min((int64_t)batch.q_start[b + 1], batch.m);
    }
    const int tiles = hi > lo ? (hi - lo + tok - 1) / tok : 0;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    upto += before;
    const uint64_t past = __ballot((int)u < upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int tile = (int)u - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l));
      const int first = __builtin_amdgcn_readlane(lo, l) + tile * tok;
      t0 = first;
      n = min(__builtin_amdgcn_readlane(hi, l) - first, tok);
      a = batch.adapter[s0 + l];
      a = a >= 0 && a < batch.n_adapters ? a : kNoAdapter;
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// the first of the adapters (or kNoAdapter) among the lanes of `left`, which loses its lanes
GPTQ_DEV int next_adapter(int id, uint64_t& left) {
  const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
  left &= ~__ballot(id == a);
  return a;
}

// eight 16-bit values at p; VEC: 16-byte loads, all eight or none
template <bool VEC> GPTQ_DEV uint4 load_chunk(const uint16_t* p, int have) {
  if constexpr (VEC) return have > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = (2 * e < have ? p[2 * e] : 0u) | (2 * e + 1 < have ? (uint32_t)p[2 * e + 1] << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct LowArgs {
  const uint16_t* X;      // [m x K], pitch ldx
  const uint16_t* A;      // [adapters][rank x K], row pitch lda
  int64_t ldx, lda, set;  // set: from one adapter's matrix to the next's
  int K, rank, slice_k;   // a workgroup's share of k, a multiple of 64 times its waves
  float* part;            // [slice][m][16 NB]
  int32_t* ids;           // [m], written by the first slice
};

// one adapter's product: X rows of 16 MT tokens by all ranks over this wave's share of [k_lo, k_hi)
template <typename T, int NB, int MT, int W, bool VEC>
GPTQ_DEV void low_product(const LowArgs& p, const uint16_t* const (&x)[MT], int a, int k_lo, int k_hi, f32x4_t (&acc)[MT][NB]) {
  typedef typename T16<T>::v8 v8;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t* A = p.A + a * p.set;
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[j][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = k_lo + 64 * wave; k0 < k_hi; k0 += 64 * W) {
    uint4 xv[MT][2], av[NB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h + 8 * g, have = k_hi - k;
#pragma unroll
      for (int j = 0; j < MT; ++j) xv[j][h] = load_chunk<VEC>(x[j] + k, have);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int r = 16 * n + i;
        av[n][h] = load_chunk<VEC>(A + r * p.lda + k, r < p.rank ? have : 0);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          acc[j][n] = T16<T>::mfma16(__builtin_bit_cast(v8, av[n][h]), __builtin_bit_cast(v8, xv[j][h]), acc[j][n]);
  }
}

// Partial sums of X A^T: k dealt to a workgroup's waves by 64 and joined through LDS
// in order.  A is the first operand, so that a lane has four neighbouring ranks of
// one token.
//
// Runs: a workgroup takes 16 MT tokens of one sequence, so of one adapter (tiles that
// end with their sequences: taken from the rows as they lie, a tile of two adapters
// went through k twice, and the launch waited for it: 50 us instead of 27 for 4096 tokens
// of rank 64 and 5120 channels in four sequences).  Neither memory (42 MB of X in those 27 us)
// nor issue (9 %) bounds it: eight waves a CU here, one step of loads a wave in flight.
template <typename T, int NB, int MT, int W, bool VEC>
__global__ __launch_bounds__(64 * W, 4) void lora_low_runs_kernel(LowArgs p, LoraBatch batch) {
  constexpr int TOK = 16 * MT;
  __shared__ f32x4_t red[W][MT][NB][64];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // rows that no sequence has: the last workgroup says so
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) {
      const int64_t lo = min(max((int64_t)batch.q_start[0], (int64_t)0), batch.m), hi = min(max((int64_t)batch.q_start[batch.n_seqs], lo), batch.m);
      for (int64_t t = threadIdx.x; t < lo; t += 64 * W) p.ids[t] = kNoToken;
      for (int64_t t = hi + threadIdx.x; t < batch.m; t += 64 * W) p.ids[t] = kNoToken;
    }
    return;
  }
  int64_t t0;
  int n, a;
  if (!run_tile(batch, blockIdx.x, TOK, t0, n, a)) return;
  if (blockIdx.y == 0 && (int)threadIdx.x < n) p.ids[t0 + threadIdx.x] = a;
  const int k_lo = blockIdx.y * p.slice_k, k_hi = min(k_lo + p.slice_k, p.K);
  if (a >= 0) {
    const uint16_t* x[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = p.X + (t0 + min(16 * j + i, n - 1)) * p.ldx;
    f32x4_t acc[MT][NB];
    low_product<T, NB, MT, W, VEC>(p, x, a, k_lo, k_hi, acc);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave][j][b][lane] = acc[j][b];
  }
  __syncthreads();
  for (int u = wave; u < MT * NB; u += W) {
    const int j = u / NB, b = u % NB;
    if (16 * j + i >= n) continue;
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[w][j][b][lane];
    }
    *reinterpret_cast<f32x4_t*>(p.part + ((int64_t)blockIdx.y * batch.m + t0 + 16 * j + i) * (16 * NB) + 16 * b + 4 * g) = s;
  }
}

// Steps of mixed adapters: 16 tokens, whatever their sequences; blockIdx.z takes every
// gridDim.z-th of the tile's adapters (one after the other they would be a chain of
// memory latencies).  48 requests of rank 16, 8192 channels: 6.9 us, of which some 4 are the
// launch and the first loads.
template <typename T, int NB, bool VEC>
__global__ __launch_bounds__(256) void lora_low_steps_kernel(LowArgs p, LoraBatch batch) {
  constexpr int W = 4;
  __shared__ f32x4_t red[W][NB][64];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * 16, t = t0 + i;
  const int id = adapter_of(batch, t0);
  const uint16_t* const x[1] = {p.X + min(t, batch.m - 1) * p.ldx};
  if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 16 && t < batch.m) p.ids[t] = id;
  uint64_t left = __ballot(lane < 16 && id >= 0);
  bool mine = false;           // this workgroup sums the lane's token
  const int k_lo = blockIdx.y * p.slice_k, k_hi = min(k_lo + p.slice_k, p.K);
  for (uint32_t n_set = 0; left; ++n_set) {
    const int a = next_adapter(id, left);
    if (n_set % gridDim.z != blockIdx.z) continue;
    f32x4_t acc[1][NB];
    low_product<T, NB, 1, W, VEC>(p, x, a, k_lo, k_hi, acc);
    if (id == a) {
      mine = true;
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave][b][lane] = acc[0][b];
    }
  }
  __syncthreads();
  if (t >= batch.m || !(mine || (id < 0 && blockIdx.z == 0))) return;
  for (int b = wave; b < NB; b += W) {
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mine) {
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[w][b][lane];
    }
    *reinterpret_cast<f32x4_t*>(p.part + ((int64_t)blockIdx.y * batch.m + t) * (16 * NB) + 16 * b + 4 * g) = s;
  }
}

// Rows of s as an operand: in two pieces of T, [hi ranks | lo ranks], below the
// row's power of two (fp16 has not the range of fp32), which `row` takes: that of its
// largest finite value, so that an infinity does not make the others infinite.
GPTQ_DEV float finite_top(float top, float v) { return fabsf(v) < INFINITY ? fmaxf(top, fabsf(v)) : top; }
template <typename T> GPTQ_DEV float piece_scale(float top, float& row) {
  int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23);
  ex = ex == 0 ? 127 : min(ex, 252);
  row = __builtin_bit_cast(float, (uint32_t)ex << 23);
  return __builtin_bit_cast(float, (uint32_t)(254 - ex) << 23);
}
template <typename T> GPTQ_DEV uint4 piece_of(const float (&s)[8], float inv, bool low) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a0 = s[2 * e] * inv, a1 = s[2 * e + 1] * inv;
    w[e] = pack2<T>(a0, a1);
    if (low) {
      const float h0 = lo16f<T>(w[e]), h1 = hi16f<T>(w[e]);
      w[e] = pack2<T>(fabsf(h0) < INFINITY ? a0 - h0 : 0.0f, fabsf(h1) < INFINITY ? a1 - h1 : 0.0f);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The slices' sums in order: s (fp32, where it is wanted), its pieces and their
// rows' scales.  2 NB threads to a token, eight ranks each.  (In long runs every one
// of a token's channel groups would add the slices again.)
template <typename T>
__global__ __launch_bounds__(256) void lora_pieces_kernel(const float* __restrict__ part, int slices, const int32_t* __restrict__ ids, int64_t m,
                                                          int nb, int rank, float* __restrict__ S, uint16_t* __restrict__ pieces,
                                                          float* __restrict__ rows) {
  const int per = 2 * nb, c = threadIdx.x % per;
  const int64_t t = (int64_t)blockIdx.x * (256 / per) + threadIdx.x / per;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  if (t < m) {
#pragma unroll 4
    for (int z = 0; z < slices; ++z) {
      const f32x4_t* from = reinterpret_cast<const f32x4_t*>(part + ((int64_t)z * m + t) * (16 * nb) + 8 * c);
      const f32x4_t lo = from[0], hi = from[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] += lo[e];
        s[4 + e] += hi[e];
      }
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = finite_top(top, s[e]);
  for (int o = 1; o < per; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (t >= m) return;
  float row;
  const float inv = piece_scale<T>(top, row);
  uint4* to = reinterpret_cast<uint4*>(pieces + t * (32 * nb));
  to[c] = piece_of<T>(s, inv, false);
  to[per + c] = piece_of<T>(s, inv, true);
  if (c == 0) rows[t] = row;
  if (S && ids[t] != kNoToken) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * c + e < rank) S[t * rank + 8 * c + e] = s[e];
  }
}

struct UpArgs {
  const float* part;      // [slices][m][16 NB]
  const uint16_t* pieces; // [m][32 NB], where lora_pieces_kernel has made them
  const float* rows;      // [m]
  const int32_t* ids;
  const uint16_t* B;      // [adapters][d x rank], row pitch ldb
  const float* scale;
  const void* R;          // [m x d] of y_type, or NULL
  void* Y;                // or NULL: only S
  float* S;               // [m x rank], or NULL
  int64_t ldb, set, ldr, ldy;
  int64_t m;
  int slices, rank, d;
  int y_type;
  bool vec;               // rows of Y and R allow 16-byte accesses
  int blocks;             // token blocks of a workgroup
};

// Row rho of matrix block b stands for this channel of the wave's 64: a lane then has
// eight neighbouring channels twice, 8 g .. and 32 + 8 g ..
GPTQ_DEV int up_channel(int rho, int b) { return 32 * (b >> 1) + 8 * (rho >> 2) + 4 * (b & 1) + (rho & 3); }

// Eight channels of one token: Y = R + add, R's load done by the caller where it is
// wide.  BITS32: fp32 values, else 16-bit ones (of bf16 or fp16: `bf`).
template <bool BITS32> struct UpRow {
  static constexpr int kLoads = BITS32 ? 2 : 1;
  uint4 raw[kLoads];
  GPTQ_DEV static bool wide(const UpArgs& p, int c) { return p.vec && c + 8 <= p.d; }
  GPTQ_DEV void load(const UpArgs& p, int64_t t, int c) {
    if (!p.R || !wide(p, c)) return;
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const char*>(p.R) + (t * p.ldr + c) * (BITS32 ? 4 : 2));
#pragma unroll
    for (int q = 0; q < kLoads; ++q) raw[q] = r[q];
  }
  GPTQ_DEV void finish(const UpArgs& p, int64_t t, int c, bool bf, const float (&add)[8]) const {
    const int have = p.d - c;
    const bool full = wide(p, c);
    if (have <= 0) return;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = 0.0f;
    if (p.R) {
      if constexpr (BITS32) {
        if (full) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const f32x4_t v = __builtin_bit_cast(f32x4_t, raw[BITS32 ? q : 0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[4 * q + e] = v[e];
          }
        } else {
          load_f32<8>(static_cast<const float*>(p.R) + t * p.ldr + c, false, have, r);
        }
      } else if (full) {
        const uint32_t v[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
        auto values = [&]<typename T>() {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[2 * e] = lo16f<T>(v[e]);
            r[2 * e + 1] = hi16f<T>(v[e]);
          }
        };
        if (bf) values.template operator()<__bf16>();
        else values.template operator()<_Float16>();
      } else if (bf) {
        load_n<__bf16, 8>(static_cast<const uint16_t*>(p.R) + t * p.ldr + c, false, have, r);
      } else {
        load_n<_Float16, 8>(static_cast<const uint16_t*>(p.R) + t * p.ldr + c, false, have, r);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] += add[e];
    if constexpr (BITS32) store_f32<8>(static_cast<float*>(p.Y) + t * p.ldy + c, full, have, r);
    else if (bf) store_n<__bf16, 8>(static_cast<uint16_t*>(p.Y) + t * p.ldy + c, full, have, r);
    else store_n<_Float16, 8>(static_cast<uint16_t*>(p.Y) + t * p.ldy + c, full, have, r);
  }
};

// Y = R + scale S B^T in runs: 256 channels, 64 a wave with B's rows in registers, by a
// tile of up to 16 p.blocks tokens of one sequence, so of one adapter.  32 tokens at a
// time the sums go through LDS, so that residual and output pass in pieces of 512
// bytes (fp32 1 KB) of a row: stored as the matrix instruction leaves them, in pieces
// of 64 or 128 bytes, the stores alone went at 2 TB/s.  A step's residual and pieces of
// s are on their way while the one before it is multiplied and stored.  4096 tokens of rank
// 64 by 13824 channels, 226 MB: 85 us, 2.7 TB/s; two thirds of the waves' time are waits for
// loads and for the two barriers of a step.
template <typename T, int NB, bool VEC, bool BITS32>
__global__ __launch_bounds__(64 * kUpWaves, NB == 8 ? 1 : (NB == 4 ? 3 : 4) - BITS32) void lora_up_runs_kernel(UpArgs p, LoraBatch batch) {
  typedef typename T16<T>::v8 v8;
  constexpr int kPitch = 256 + 4;                      // floats of a token's sums in LDS
  constexpr int kRow = 32 * NB + 8;                    // 16-bit values of its pieces there
  constexpr int kEach = 32 * 32 / (64 * kUpWaves);     // eight-channel pieces of 32 tokens, a thread
  constexpr int kLoads = 32 * 4 * NB / (64 * kUpWaves) > 0 ? 32 * 4 * NB / (64 * kUpWaves) : 1;
  __shared__ __attribute__((aligned(16))) float out[32 * kPitch];
  __shared__ __attribute__((aligned(16))) uint16_t low[32 * kRow];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = (p.d + 255) / 256;
  const int c0 = 256 * (int)(blockIdx.x % groups);
  int64_t t0;
  int n, a;
  if (!run_tile(batch, blockIdx.x / groups, 16 * p.blocks, t0, n, a)) return;
  const bool bf = p.y_type == GPTQ_BF16, has = a >= 0;
  float scale = 0.0f;
  v8 bo[4][NB];
  if (has) {
    scale = p.scale[a];
    const uint16_t* B = p.B + a * p.set;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int ch = c0 + 64 * wave + up_channel(i, b);
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) {
        const int r = 8 * ((4 * kb + g) % (2 * NB));
        bo[b][kb] = __builtin_bit_cast(v8, load_chunk<VEC>(B + ch * p.ldb + r, ch < p.d ? p.rank - r : 0));
      }
    }
  }
  const int c = c0 + 8 * (tid & 31);                   // this thread's channels of the rows tid / 32 + 8 k
  UpRow<BITS32> res[2][kEach];
  float f[2][kEach];
  uint4 sv[kLoads];
  auto fetch = [&]<int TO>(int k0) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int64_t t = t0 + min(k0 + (tid >> 5) + 8 * k, n - 1);
      res[TO][k].load(p, t, c);
      f[TO][k] = has ? p.rows[t] : 0.0f;
    }
    if (has) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int u = tid + 64 * kUpWaves * k, row = u / (4 * NB);
        sv[k] = *reinterpret_cast<const uint4*>(p.pieces + (t0 + min(k0 + row, n - 1)) * (32 * NB) + 8 * (u % (4 * NB)));
      }
    }
  };
  fetch.template operator()<0>(0);
  auto step = [&]<int CUR>(int k0) {
    if (has) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int u = tid + 64 * kUpWaves * k, row = u / (4 * NB);
        if (row < 32) *reinterpret_cast<uint4*>(low + row * kRow + 8 * (u % (4 * NB))) = sv[k];
      }
    }
    __syncthreads();
    if (k0 + 32 < n) fetch.template operator()<CUR ^ 1>(k0 + 32);
    if (has) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        f32x4_t acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
          const v8 so = *reinterpret_cast<const v8*>(low + (16 * x + i) * kRow + 8 * (4 * kb + g));
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[b] = T16<T>::mfma16(bo[b][kb], so, acc[b]);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<f32x4_t*>(out + (16 * x + i) * kPitch + 64 * wave + up_channel(4 * g, b)) = acc[b];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int row = (tid >> 5) + 8 * k;
      if (k0 + row >= n) continue;
      float add[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) add[e] = 0.0f;
      if (has) {
        load_f32<8>(out + row * kPitch + 8 * (tid & 31), true, 8, add);
#pragma unroll
        for (int e = 0; e < 8; ++e) add[e] *= scale * f[CUR][k];
      }
      res[CUR][k].finish(p, t0 + k0 + row, c, bf, add);
    }
  };
  for (int k0 = 0; k0 < n; k0 += 64) {
    step.template operator()<0>(k0);
    if (k0 + 32 < n) step.template operator()<1>(k0 + 32);
  }
}

// The same where a block of tokens has several adapters: a unit is a block of 16
// tokens and one of the adapters in it, a workgroup's waves share the units of 64
// channels, and s's pieces are made here, from up to eight slices.  48 requests of rank 16 by
// 8192 channels: 8.8 us, the latency of three loads that wait for each other.
template <typename T, int NB, bool VEC, bool BITS32>
__global__ __launch_bounds__(64 * kUpWaves) void lora_up_steps_kernel(UpArgs p) {
  typedef typename T16<T>::v8 v8;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (p.d + 63) / 64;
  const int64_t t = (int64_t)(blockIdx.x / groups) * 16 + i;
  const int c0 = 64 * (int)(blockIdx.x % groups), c = c0 + 8 * g;
  const bool writes_s = p.S && c0 == 0 && wave == 0, bf = p.y_type == GPTQ_BF16;
  const int64_t at = min(t, p.m - 1);
  const int id = t < p.m ? p.ids[t] : kNoToken;
  UpRow<BITS32> res[2];
  if (p.Y) {
    res[0].load(p, at, c);
    res[1].load(p, at, c + 32);
  }
  // the lane's chunks of its token's pieces
  v8 so[NB];
  float row = 1.0f;
  {
    float s[NB][8], top = 0.0f;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      const int rc = (4 * kb + g) % (2 * NB);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[kb][e] = 0.0f;
#pragma unroll 8
      for (int z = 0; z < p.slices; ++z) {
        const f32x4_t* from = reinterpret_cast<const f32x4_t*>(p.part + ((int64_t)z * p.m + at) * (16 * NB) + 8 * rc);
        const f32x4_t lo = from[0], hi = from[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[kb][e] += lo[e];
          s[kb][4 + e] += hi[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = finite_top(top, s[kb][e]);
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float inv = piece_scale<T>(top, row);
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      const bool low = (4 * kb + g) / (2 * NB) != 0;
      so[kb] = __builtin_bit_cast(v8, piece_of<T>(s[kb], inv, low));
      if (writes_s && !low && id != kNoToken) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 8 * ((4 * kb + g) % (2 * NB)) + e;
          if (r < p.rank) p.S[t * p.rank + r] = s[kb][e];
        }
      }
    }
  }
  if (!p.Y) return;
  uint64_t left = __ballot(id != kNoToken && lane < 16);
  for (int unit = 0; left; ++unit) {
    const int a = next_adapter(id, left);
    if (unit % kUpWaves != wave) continue;
    f32x4_t acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float f = 0.0f;
    if (a >= 0) {
      f = p.scale[a] * row;
      const uint16_t* B = p.B + a * p.set;
#pragma unroll
      for (int kb = 0; kb < NB; ++kb)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int ch = c0 + up_channel(i, b), r = 8 * ((4 * kb + g) % (2 * NB));
          const v8 bo = __builtin_bit_cast(v8, load_chunk<VEC>(B + ch * p.ldb + r, ch < p.d ? p.rank - r : 0));
          acc[b] = T16<T>::mfma16(bo, so[kb], acc[b]);
        }
    }
    if (id != a) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float add[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) add[e] = a >= 0 ? f * acc[2 * h + (e >> 2)][e & 3] : 0.0f;
      res[h].finish(p, t, c + 32 * h, bf, add);
    }
  }
}

// ---------------------------------------------------------------- backward

// [n][rows x cols] -> [n][cols x rows], row pitch `pitch` (a multiple of 8, zeros from
// rows on), of one or two matrices a set: 64 x 64 tiles through LDS
struct TransposeSide {
  const uint16_t* in;
  uint16_t* out;
  int rows, cols, pitch;
  int tiles_c, tiles;      // tiles of 64 columns, all tiles (0: nothing to do)
};
__global__ __launch_bounds__(256) void lora_transpose_kernel(TransposeSide s0, TransposeSide s1) {
  __shared__ uint16_t tile[64][66];
  const bool second = (int)blockIdx.x >= s0.tiles;
  const TransposeSide& s = second ? s1 : s0;
  const int u = blockIdx.x - (second ? s0.tiles : 0);
  const int64_t set = blockIdx.y;
  const int r0 = u / s.tiles_c * 64, c0 = u % s.tiles_c * 64, x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const uint16_t* from = s.in + set * s.rows * s.cols;
  uint16_t* to = s.out + set * s.cols * s.pitch;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int r = r0 + y + 4 * k, c = c0 + x;
    tile[y + 4 * k][x] = r < s.rows && c < s.cols ? from[(int64_t)r * s.cols + c] : (uint16_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int c = c0 + y + 4 * k, r = r0 + x;
    if (c < s.cols && r < s.pitch) to[(int64_t)c * s.pitch + r] = tile[x][y + 4 * k];
  }
}

// One of the two products over tokens: dA (X: the inputs, S: dS) or dB (X: dY, S: s)
struct OuterSide {
  const uint16_t* X;
  const float* S;         // [m x rank]
  int64_t ldx;
  float* out;             // [adapters][rank x d] or [adapters][d x rank]; with splits the first one's part
  int64_t split;          // from one split's part to the next's
  int d, tiles;           // tiles of 128 channels
  bool vec;
};
struct OuterArgs {
  OuterSide side[2];
  const int32_t* ids;
  const float* scale;
  int64_t m, slice;       // tokens of a split, a multiple of 32
  int rank;
};

typedef short i16x4_t __attribute__((ext_vector_type(4)));
// Four rows of 16 channels of 16-bit values become four values of one channel a
// lane: in each group of 16 lanes, lane l names 8 bytes of row l / 4 (channels 4 (l %
// 4) ..), and gets channel l of the four rows.
GPTQ_DEV uint2 read_transposed(uint32_t at) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(uintptr_t)at));
}

// scale sum_t X[t][c] S[t][r] over one adapter's tokens: 128 channels by all ranks
// a workgroup, 32 tokens a step.  Both operands want the tokens next to each
// other: X goes to LDS as it lies and is read transposed, S in three bf16 pieces
// (24 bits; two cost an error twice that of fp32 sums) with tokens innermost.  fp16 channels
// are two bf16 values exactly; the second one's product with the third piece, 2^-27 of
// the whole, is left out.  8192 tokens of two adapters of rank 32, 4096 by 4096 channels:
// 51 us for 136 MB and 4.3 GFLOP (three times with the pieces); vector work (making the
// pieces) fills a third of the issue slots, the rest waits for the next step's loads.
template <typename T, int NB>
__global__ __launch_bounds__(256) void lora_outer_kernel(OuterArgs p) {
  typedef typename T16<__bf16>::v8 b8;
  constexpr bool kSplitX = T16<T>::kType == GPTQ_F16;
  constexpr int kPitch = 40;                         // tokens of a rank's row in LDS: 80 bytes
  __shared__ __attribute__((aligned(1024))) uint16_t xs[2 * 32 * 128];
  __shared__ __attribute__((aligned(16))) uint16_t ss[2 * 3 * 16 * NB * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool is_b = (int)blockIdx.x >= p.side[0].tiles;
  const OuterSide& o = p.side[is_b];
  const int c0 = 128 * ((int)blockIdx.x - (is_b ? p.side[0].tiles : 0)), a = blockIdx.z;
  const int64_t t_lo = blockIdx.y * p.slice, t_hi = min(t_lo + p.slice, p.m);
  const float scale = p.scale[a];
  const uint32_t xl0 = (uint32_t)(uintptr_t)(LDS_AS const char*)(const char*)xs;
  // 32-byte pairs of chunks of row t sit at pair ^ (t % 4 + 4 (t / 8 % 2)): the rows that a read takes differ in it
  auto swz = [](int t) { return (t & 3) | ((t >> 1) & 4); };
  f32x4_t acc[2][NB];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[b][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // One step ahead: a step's values are on their way while the one before it is
  // multiplied, its tokens' adapters one step longer.
  uint4 xv[2];
  float sv[2 * NB];
  auto load_ids = [&](int64_t t0) {
    const int64_t t = t0 + (lane & 31);
    return t < t_hi ? p.ids[t] : kNoToken;
  };
  // another adapter's tokens count as zeros, whatever they hold
  auto load = [&](int64_t t0, uint32_t some) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = (tid >> 4) + 16 * h, c = c0 + 8 * (tid & 15);
      const int have = (some >> t) & 1 ? o.d - c : 0;
      const uint16_t* x = o.X + (t0 + t) * o.ldx + c;
      xv[h] = o.vec && have >= 8 ? load_chunk<true>(x, have) : load_chunk<false>(x, have);
    }
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) {
      const int u = tid + 256 * k, t = u / (16 * NB), r = u % (16 * NB);
      sv[k] = ((some >> t) & 1) && r < p.rank ? o.S[(t0 + t) * p.rank + r] : 0.0f;
    }
  };
  uint32_t now = (uint32_t)__ballot(load_ids(t_lo) == a);
  if (now) load(t_lo, now);
  int next_ids = load_ids(t_lo + 32);
  uint32_t turn = 0;
  for (int64_t t0 = t_lo; t0 < t_hi; t0 += 32) {
    const uint32_t next = (uint32_t)__ballot(next_ids == a), some = now;
    uint16_t* xb = xs + (turn & 1) * (32 * 128);
    uint16_t* sb = ss + (turn & 1) * (3 * 16 * NB * kPitch);
    if (some) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = (tid >> 4) + 16 * h, ch = tid & 15;
        *reinterpret_cast<uint4*>(xb + t * 128 + (((ch >> 1) ^ swz(t)) << 4) + 8 * (ch & 1)) = xv[h];
      }
#pragma unroll
      for (int k = 0; k < 2 * NB; ++k) {
        const int u = tid + 256 * k, t = u / (16 * NB), r = u % (16 * NB);
        float v = (some >> t) & 1 ? scale * sv[k] : 0.0f;
#pragma unroll
        for (int z = 0; z < 3; ++z) {
          const uint16_t piece = bits16<__bf16>(v);
          const float f = (float)__builtin_bit_cast(__bf16, piece);
          sb[(16 * NB * z + r) * kPitch + t] = piece;
          v = fabsf(f) < INFINITY ? v - f : 0.0f;
        }
      }
    }
    if (next) load(t0 + 32, next);
    next_ids = load_ids(t0 + 64);
    now = next;
    if (!some) continue;
    const uint32_t xl = xl0 + (turn & 1) * (32 * 128 * 2);
    ++turn;
    // (two buffers: a wave that is behind still reads the other one)
    __syncthreads();
    b8 xo[2][kSplitX ? 2 : 1];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 8 * g + 4 * h + (i >> 2), pair = 2 * wave + b;
        const uint2 v = read_transposed(xl + t * 256 + ((pair ^ swz(t)) << 5) + 8 * (i & 3));
        w[2 * h] = v.x;
        w[2 * h + 1] = v.y;
      }
      if constexpr (kSplitX) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f0 = lo16f<_Float16>(w[e]), f1 = hi16f<_Float16>(w[e]);
          hi[e] = pack2<__bf16>(f0, f1);
          const float h0 = lo16f<__bf16>(hi[e]), h1 = hi16f<__bf16>(hi[e]);
          lo[e] = pack2<__bf16>(fabsf(h0) < INFINITY ? f0 - h0 : 0.0f, fabsf(h1) < INFINITY ? f1 - h1 : 0.0f);
        }
        xo[b][0] = __builtin_bit_cast(b8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        xo[b][kSplitX ? 1 : 0] = __builtin_bit_cast(b8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      } else {
        xo[b][0] = __builtin_bit_cast(b8, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      b8 so[3];
#pragma unroll
      for (int z = 0; z < 3; ++z) so[z] = *reinterpret_cast<const b8*>(sb + (16 * NB * z + 16 * n + i) * kPitch + 8 * g);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        auto product = [&](const b8& x, const b8& s) {
          // dA: rows are channels, so that a lane has four channels of one rank; dB: four ranks of one channel
          acc[b][n] = is_b ? T16<__bf16>::mfma16(s, x, acc[b][n]) : T16<__bf16>::mfma16(x, s, acc[b][n]);
        };
        product(xo[b][0], so[2]);
        product(xo[b][0], so[1]);
        product(xo[b][0], so[0]);
        if constexpr (kSplitX) {
          product(xo[b][kSplitX ? 1 : 0], so[0]);
          product(xo[b][kSplitX ? 1 : 0], so[1]);
        }
      }
    }
  }
  float* out = o.out + blockIdx.y * o.split + (int64_t)a * p.rank * o.d;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int c = c0 + 16 * (2 * wave + b) + (is_b ? i : 4 * g), r = 16 * n + (is_b ? 4 * g : i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ce = is_b ? c : c + e, re = is_b ? r + e : r;
        if (ce < o.d && re < p.rank) out[is_b ? (int64_t)ce * p.rank + re : (int64_t)re * o.d + ce] = acc[b][n][e];
      }
    }
}

// the splits' parts in order: the first n0 values of a part are o0's, the others o1's (each may be NULL)
__global__ __launch_bounds__(256) void lora_join_kernel(const float* __restrict__ part, int64_t split, int splits, int64_t n0, int64_t n,
                                                        float* __restrict__ o0, float* __restrict__ o1) {
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < n; u += (int64_t)gridDim.x * 256) {
    float* out = u < n0 ? o0 : o1;
    if (!out) continue;
    float v = 0.0f;
#pragma unroll 8
    for (int z = 0; z < splits; ++z) v += part[z * split + u];
    out[u < n0 ? u : u - n0] = v;
  }
}

// ---------------------------------------------------------------- host side
static bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static int rank_blocks(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

static bool lora_ok(const gptq_lora_set* a) {
  if (!a || !a->A || !a->B || !a->scale) return false;
  if (a->n_adapters <= 0 || a->n_adapters > kLoraMaxSets || a->rank <= 0 || a->rank > kLoraMaxRank) return false;
  if (a->d_in <= 0 || a->d_in > kLoraMaxDim || a->d_out <= 0 || a->d_out > kLoraMaxDim) return false;
  return ((reinterpret_cast<uintptr_t>(a->A) | reinterpret_cast<uintptr_t>(a->B)) & 1) == 0 && (reinterpret_cast<uintptr_t>(a->scale) & 3) == 0;
}
constexpr int64_t kLoraMaxTokens = 1 << 24;
// whether an array shares a byte with the set's matrices and scales or with the batch's description
static bool meets_set(const void* p, uint64_t n, const gptq_lora_set* a, const int32_t* q_start, const int32_t* adapter, int n_seqs) {
  const uint64_t pairs = (uint64_t)a->n_adapters * a->rank * 2;
  return share_bytes(p, n, a->A, pairs * a->d_in) || share_bytes(p, n, a->B, pairs * a->d_out) ||
         share_bytes(p, n, a->scale, (uint64_t)a->n_adapters * 4) || share_bytes(p, n, q_start, ((uint64_t)n_seqs + 1) * 4) ||
         share_bytes(p, n, adapter, (uint64_t)n_seqs * 4);
}

// How X A^T is dealt out.  Runs: 32 tokens a workgroup of eight waves (at rank 128
// 16), k in slices until there are two workgroups a CU.  Steps of mixed adapters: 16
// tokens a workgroup of four waves, one of the adapters each, up to 8 slices (which the
// second product adds itself).  One slice against these, whole calls of 8192 channels: 48
// requests 22.8 and 11.9 us, 512 tokens of rank 64 70 and 37, 4096 of them 98 and 85.  Half and twice
// as many workgroups: 4096 tokens of rank 64, 5120 -> 13824, 115, 110 (these) and 112, of rank 16, 4096
// channels, 38, 36 and 35, smaller batches the same within 3 %.  Up to 8, 16 and 32 slices: 40 tokens of
// rank 64 23.8, 22.3 and 22.3, more of them the same.  Steps, up to 4 and 8: 48 requests of rank 16 13.3 and
// 12.0, 8 of them 12.1 and 11.4, 256 of 4096 channels 16.6 and 20.0.
struct LowPlan {
  bool mix;
  int mt, tiles, slices, slice_k, shares;
};
// Whether the batch counts as steps, whose blocks have several adapters.  Both ways, 16
// adapters, steps first: 48 tokens of rank 16 in sequences of one 15.5 and 17.1 us, of six 11.1
// and 14.2 (a launch fewer); 512 tokens in ones 51 and 71, in twos 35 and 35, in sixes 25 and 19;
// of rank 64 in ones 167 and 172, in twos 117 and 90, in sixes 97 and 45.
static bool mixed(int64_t m, int n_seqs) { return m < (m <= 128 ? 16 : 2) * (int64_t)n_seqs; }
static LowPlan low_plan(int64_t m, int n_seqs, int K, int nb) {
  LowPlan p;
  p.mix = mixed(m, n_seqs);
  p.mt = p.mix || nb == 8 ? 1 : 2;
  p.tiles = (int)((m + 16 * p.mt - 1) / (16 * p.mt));
  p.shares = p.mix ? 16 : 1;
  const int step = 64 * (p.mix ? 4 : 8), most = (K + step - 1) / step;
  const int n = (int)std::max<int64_t>(1, std::min<int64_t>(512 / (p.mix ? (p.tiles + 7) / 8 * 8 : p.tiles), std::min(most, p.mix ? 8 : 16)));
  p.slice_k = (most + n - 1) / n * step;
  p.slices = (K + p.slice_k - 1) / p.slice_k;
  if (!p.mix) p.tiles += n_seqs;       // tiles that end with their sequences, and one workgroup more
  return p;
}
// The partial sums' part of the workspace: token ids, sums, and s's pieces with their rows' scales; room for every
// batch of m tokens, whatever its sequences.
struct LowLayout {
  size_t off_part, off_pieces, off_rows, total;
};
static LowLayout low_layout(int64_t m, int K, int nb) {
  LowLayout L;
  const int slices = std::max(low_plan(m, 1, K, nb).slices, low_plan(m, (int)m + 1, K, nb).slices);
  L.off_part = align_up((size_t)m * sizeof(int32_t));
  L.off_pieces = L.off_part + align_up((size_t)slices * m * 16 * nb * sizeof(float));
  L.off_rows = L.off_pieces + align_up((size_t)m * 32 * nb * 2);
  L.total = L.off_rows + align_up((size_t)m * sizeof(float));
  return L;
}

// How the second product by d channels is dealt out: tiles of 16 `blocks` tokens by `groups` of channels
struct UpPlan {
  int blocks;
  int64_t groups, tiles;
};
static UpPlan up_plan(const LowPlan& lp, int64_t m, int n_seqs, int d) {
  UpPlan p;
  const int width = lp.mix ? 64 : 256;
  p.groups = (d + width - 1) / width;
  // A run's tiles as long as leave four workgroups a CU, up to 128 tokens (B's rows serve them all): 32
  // and 128 tokens, whole calls of rank 64: 2048 tokens by 4096 channels 44.0 and 46.8 us, 4096 by 4096 60
  // and 56, 8192 by 13824 206 and 184.
  p.blocks = lp.mix ? 1 : m * p.groups >= 128 * 1024 ? 8 : m * p.groups >= 64 * 1024 ? 4 : 2;
  p.tiles = (m + 16 * p.blocks - 1) / (16 * p.blocks) + (lp.mix ? 0 : n_seqs - 1);
  return p;
}
// whether both products' launches are within the hardware's limits
static bool plans_fit(const LowPlan& lp, const UpPlan& up) {
  return (int64_t)lp.tiles * 512 <= UINT32_MAX && up.tiles * up.groups <= (1 << 24) - 1;
}

// s of every token into the workspace at base; where they are runs, as pieces
template <typename T>
static int launch_low(const LowPlan& p, const LowLayout& L, int nb, bool vec, LowArgs a, const LoraBatch& b, char* base, float* S, hipStream_t s) {
  const dim3 grid((unsigned)p.tiles, (unsigned)p.slices, (unsigned)p.shares);
  a.slice_k = p.slice_k;
  a.ids = reinterpret_cast<int32_t*>(base);
  a.part = reinterpret_cast<float*>(base + L.off_part);
  auto go = [&]<int NB>() {
    constexpr int MT = NB == 8 ? 1 : 2;
    if (p.mix) {
      if (vec) lora_low_steps_kernel<T, NB, true><<<grid, 256, 0, s>>>(a, b);
      else lora_low_steps_kernel<T, NB, false><<<grid, 256, 0, s>>>(a, b);
    } else {
      if (vec) lora_low_runs_kernel<T, NB, MT, 8, true><<<grid, 512, 0, s>>>(a, b);
      else lora_low_runs_kernel<T, NB, MT, 8, false><<<grid, 512, 0, s>>>(a, b);
    }
  };
  if (nb == 1) go.template operator()<1>();
  else if (nb == 2) go.template operator()<2>();
  else if (nb == 4) go.template operator()<4>();
  else go.template operator()<8>();
  GPTQ_LAUNCH_CHECK();
  if (!p.mix) {
    lora_pieces_kernel<T><<<(unsigned)((b.m * 2 * nb + 255) / 256), 256, 0, s>>>(a.part, p.slices, a.ids, b.m, nb, a.rank, S,
                                                                              reinterpret_cast<uint16_t*>(base + L.off_pieces),
                                                                              reinterpret_cast<float*>(base + L.off_rows));
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

// The second product (a.Y; a.S where the pieces are made here), from what launch_low left at base.
template <typename T>
static int launch_up(UpArgs a, const LowPlan& lp, const UpPlan& up, const LowLayout& L, int nb, const LoraBatch& b, char* base, hipStream_t s) {
  a.part = reinterpret_cast<float*>(base + L.off_part);
  a.pieces = reinterpret_cast<uint16_t*>(base + L.off_pieces);
  a.rows = reinterpret_cast<float*>(base + L.off_rows);
  a.ids = reinterpret_cast<int32_t*>(base);
  a.slices = lp.slices;
  a.blocks = up.blocks;
  const bool vec = at16(a.B) && a.rank % 8 == 0 && a.ldb % 8 == 0 && a.set % 8 == 0;
  const unsigned grid = (unsigned)(up.tiles * up.groups);
  auto go = [&]<int NB>() {
    auto on = [&]<bool VEC, bool BITS32>() {
      if (lp.mix) lora_up_steps_kernel<T, NB, VEC, BITS32><<<grid, 64 * kUpWaves, 0, s>>>(a);
      else lora_up_runs_kernel<T, NB, VEC, BITS32><<<grid, 64 * kUpWaves, 0, s>>>(a, b);
    };
    if (a.y_type == GPTQ_F32) vec ? on.template operator()<true, true>() : on.template operator()<false, true>();
    else vec ? on.template operator()<true, false>() : on.template operator()<false, false>();
  };
  if (nb == 1) go.template operator()<1>();
  else if (nb == 2) go.template operator()<2>();
  else if (nb == 4) go.template operator()<4>();
  else go.template operator()<8>();
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

static bool is_16(gptq_dtype t) { return t == GPTQ_F16 || t == GPTQ_BF16; }
static bool elem_at(const void* p, gptq_dtype t) { return (reinterpret_cast<uintptr_t>(p) & (t == GPTQ_F32 ? 3 : 1)) == 0; }
static bool rows_vec(const void* p, int64_t ld, gptq_dtype t) { return !p || (at16(p) && ld % (t == GPTQ_F32 ? 4 : 8) == 0); }

struct LoraBackLayout {
  LowLayout low;
  size_t off_ds, off_at, off_bt, off_outer, total;
  int nb, splits;
  int64_t slice, out_pitch;
};
static LoraBackLayout lora_back_layout(int64_t m, const gptq_lora_set* a) {
  LoraBackLayout L;
  L.nb = rank_blocks(a->rank);
  const int64_t sets = a->n_adapters, r = a->rank, pitch = (r + 7) & ~7;
  L.low = low_layout(m, a->d_out, L.nb);
  L.off_ds = L.low.total;
  L.off_at = L.off_ds + align_up((size_t)m * r * 4);
  L.off_bt = L.off_at + align_up((size_t)sets * a->d_in * pitch * 2);
  L.off_outer = L.off_bt + align_up((size_t)sets * r * ((a->d_out + 7) & ~7) * 2);
  // Splits of the tokens until there are four workgroups a CU, 256 tokens each at least.  Whole calls of
  // two adapters of rank 32 by 4096 channels: 512 tokens 33.0 us whole, 31.9 so, 42.8 in parts of 64; 8192
  // tokens 224 whole, 108 so, 138 in four times as many parts.
  const int64_t tiles = ((a->d_in + 127) / 128 + (a->d_out + 127) / 128) * sets;
  int64_t n = std::max<int64_t>(1, std::min<int64_t>({1024 / tiles, (m + 255) / 256, 16}));
  L.slice = ((m + n - 1) / n + 31) / 32 * 32;
  L.splits = (int)((m + L.slice - 1) / L.slice);
  L.out_pitch = sets * r * (a->d_in + a->d_out);
  L.total = L.off_outer + (L.splits > 1 ? align_up((size_t)L.splits * L.out_pitch * 4) : 0);
  return L;
}

template <typename T>
static int lora_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const float* S, const gptq_lora_set* a,
                         const LoraBatch& b, const void* R, int64_t ldr, void* dX, gptq_dtype x_dtype, int64_t lddx, float* dA,
                         float* dB, char* base, hipStream_t s) {
  const LoraBackLayout L = lora_back_layout(b.m, a);
  const LowPlan lp = low_plan(b.m, b.n_seqs, a->d_out, L.nb);
  const UpPlan up = up_plan(lp, b.m, b.n_seqs, dX ? a->d_in : 1);
  if (!plans_fit(lp, up)) return GPTQ_ERR_INVALID_ARG;
  const int sets = a->n_adapters, r = a->rank, pitch = (r + 7) & ~7, kp = (a->d_out + 7) & ~7;
  const int32_t* ids = reinterpret_cast<const int32_t*>(base);
  float* ds = reinterpret_cast<float*>(base + L.off_ds);
  uint16_t *at = reinterpret_cast<uint16_t*>(base + L.off_at), *bt = reinterpret_cast<uint16_t*>(base + L.off_bt);
  auto side = [](const void* in, uint16_t* out, int rows, int cols, int out_pitch) {
    const int tc = (cols + 63) / 64;
    return TransposeSide{static_cast<const uint16_t*>(in), out, rows, cols, out_pitch, tc, tc * ((out_pitch + 63) / 64)};
  };
  const TransposeSide tb = side(a->B, bt, a->d_out, r, kp);
  TransposeSide ta = side(a->A, at, r, a->d_in, pitch);
  if (!dX) ta.tiles = 0;
  lora_transpose_kernel<<<dim3((unsigned)(tb.tiles + ta.tiles), (unsigned)sets), 256, 0, s>>>(tb, ta);
  GPTQ_LAUNCH_CHECK();
  const bool vec = rows_vec(dY, lddy, GPTQ_BF16) && a->d_out % 8 == 0;
  LowArgs low{static_cast<const uint16_t*>(dY), bt, lddy, kp, (int64_t)r * kp, a->d_out, r};
  int st = launch_low<T>(lp, L.low, L.nb, vec, low, b, base, dA ? ds : nullptr, s);
  if (st != GPTQ_OK) return st;
  if (dX || (dA && lp.mix)) {
    UpArgs u{};
    u.B = at; u.scale = a->scale; u.R = R; u.Y = dX; u.S = dA ? ds : nullptr;
    u.ldb = pitch; u.set = (int64_t)a->d_in * pitch; u.ldr = ldr; u.ldy = lddx; u.m = b.m; u.rank = r; u.d = dX ? a->d_in : 1; u.y_type = x_dtype;
    u.vec = rows_vec(R, ldr, x_dtype) && rows_vec(dX, lddx, x_dtype);
    st = launch_up<T>(u, lp, up, L.low, L.nb, b, base, s);
    if (st != GPTQ_OK) return st;
  }
  if (!dA && !dB) return GPTQ_OK;
  float* outer = reinterpret_cast<float*>(base + L.off_outer);
  const int64_t na = (int64_t)sets * r * a->d_in, nb = (int64_t)sets * r * a->d_out;
  const bool split = L.splits > 1;
  OuterArgs o{};
  o.side[0] = OuterSide{static_cast<const uint16_t*>(X), ds, ldx, split ? outer : dA, split ? L.out_pitch : 0, a->d_in,
                        dA ? (a->d_in + 127) / 128 : 0, rows_vec(X, ldx, GPTQ_BF16)};
  o.side[1] = OuterSide{static_cast<const uint16_t*>(dY), S, lddy, split ? outer + na : dB, split ? L.out_pitch : 0, a->d_out,
                        dB ? (a->d_out + 127) / 128 : 0, rows_vec(dY, lddy, GPTQ_BF16)};
  o.ids = ids;
  o.scale = a->scale;
  o.m = b.m;
  o.slice = L.slice;
  o.rank = r;
  const dim3 grid((unsigned)(o.side[0].tiles + o.side[1].tiles), (unsigned)L.splits, (unsigned)sets);
  if (L.nb == 1) lora_outer_kernel<T, 1><<<grid, 256, 0, s>>>(o);
  else if (L.nb == 2) lora_outer_kernel<T, 2><<<grid, 256, 0, s>>>(o);
  else if (L.nb == 4) lora_outer_kernel<T, 4><<<grid, 256, 0, s>>>(o);
  else lora_outer_kernel<T, 8><<<grid, 256, 0, s>>>(o);
  GPTQ_LAUNCH_CHECK();
  if (split) {
    lora_join_kernel<<<(unsigned)std::min<int64_t>((na + nb + 255) / 256, 8192), 256, 0, s>>>(outer, L.out_pitch, L.splits, na, na + nb, dA, dB);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_lora_workspace_size(int64_t m, const gptq_lora_set* a) {
  if (m <= 0 || m > kLoraMaxTokens || !lora_ok(a)) return 0;
  return low_layout(m, a->d_in, rank_blocks(a->rank)).total;
}

extern "C" int gptq_lora(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_lora_set* a, const int32_t* q_start,
                         const int32_t* adapter, int32_t n_seqs, const void* R, int64_t ldr, void* Y, gptq_dtype y_dtype, int64_t ldy,
                         float* S, void* ws, size_t ws_bytes, hipStream_t s) {
  if (!lora_ok(a) || m < 0 || m > kLoraMaxTokens || n_seqs <= 0 || n_seqs == INT_MAX || !is_16(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (y_dtype != GPTQ_F32 && !is_16(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) return GPTQ_OK;
  if (!X || !Y || !q_start || !adapter || ldx < a->d_in || ldy < a->d_out || (R && ldr < a->d_out)) return GPTQ_ERR_INVALID_ARG;
  if (!elem_at(X, x_dtype) || !elem_at(R, y_dtype) || !elem_at(Y, y_dtype) || !elem_at(S, GPTQ_F32) || !elem_at(q_start, GPTQ_F32) ||
      !elem_at(adapter, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  const uint64_t e = y_dtype == GPTQ_F32 ? 4 : 2, yb = rows_bytes(m, ldy, a->d_out, e), xb = rows_bytes(m, ldx, a->d_in, 2), sb = (uint64_t)m * a->rank * 4;
  if (share_bytes(Y, yb, X, xb) || share_bytes(Y, yb, S, sb) || share_bytes(S, sb, X, xb)) return GPTQ_ERR_INVALID_ARG;
  if (R && !(R == Y && ldr == ldy) && share_bytes(Y, yb, R, rows_bytes(m, ldr, a->d_out, e))) return GPTQ_ERR_INVALID_ARG;
  if (R && share_bytes(S, sb, R, rows_bytes(m, ldr, a->d_out, e))) return GPTQ_ERR_INVALID_ARG;
  if (meets_set(Y, yb, a, q_start, adapter, n_seqs) || meets_set(S, sb, a, q_start, adapter, n_seqs)) return GPTQ_ERR_INVALID_ARG;
  const size_t need = gptq_lora_workspace_size(m, a);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  if (meets_set(ws, need, a, q_start, adapter, n_seqs) || share_bytes(ws, need, X, xb) || share_bytes(ws, need, Y, yb) || share_bytes(ws, need, S, sb) ||
      (R && share_bytes(ws, need, R, rows_bytes(m, ldr, a->d_out, e)))) return GPTQ_ERR_INVALID_ARG;
  const int nb = rank_blocks(a->rank);
  const LowPlan lp = low_plan(m, n_seqs, a->d_in, nb);
  const UpPlan upp = up_plan(lp, m, n_seqs, a->d_out);
  if (!plans_fit(lp, upp)) return GPTQ_ERR_INVALID_ARG;
  const LowLayout L = low_layout(m, a->d_in, nb);
  const LoraBatch b{q_start, adapter, n_seqs, a->n_adapters, m};
  char* base = static_cast<char*>(ws);
  const bool vec = rows_vec(X, ldx, x_dtype) && at16(a->A) && a->d_in % 8 == 0;
  const LowArgs low{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(a->A), ldx, a->d_in, (int64_t)a->rank * a->d_in, a->d_in, a->rank};
  UpArgs up{};
  up.B = static_cast<const uint16_t*>(a->B); up.scale = a->scale; up.R = R; up.Y = Y; up.S = S;
  up.ldb = a->rank; up.set = (int64_t)a->d_out * a->rank; up.ldr = ldr; up.ldy = ldy; up.m = m; up.rank = a->rank; up.d = a->d_out; up.y_type = y_dtype;
  up.vec = rows_vec(R, ldr, y_dtype) && rows_vec(Y, ldy, y_dtype);
  auto go = [&]<typename T>() {
    const int st = launch_low<T>(lp, L, nb, vec, low, b, base, S, s);
    return st != GPTQ_OK ? st : launch_up<T>(up, lp, upp, L, nb, b, base, s);
  };
  return x_dtype == GPTQ_BF16 ? go.template operator()<__bf16>() : go.template operator()<_Float16>();
}

extern "C" size_t gptq_lora_backward_workspace_size(int64_t m, const gptq_lora_set* a) {
  if (m <= 0 || m > kLoraMaxTokens || !lora_ok(a)) return 0;
  return lora_back_layout(m, a).total;
}

extern "C" int gptq_lora_backward(const void* dY, gptq_dtype dtype, int64_t m, int64_t lddy, const void* X, int64_t ldx, const float* S,
                                  const gptq_lora_set* a, const int32_t* q_start, const int32_t* adapter, int32_t n_seqs,
                                  const void* R, int64_t ldr, void* dX, gptq_dtype x_dtype, int64_t lddx, float* dA, float* dB,
                                  void* ws, size_t ws_bytes, hipStream_t s) {
  if (!lora_ok(a) || m < 0 || m > kLoraMaxTokens || n_seqs <= 0 || n_seqs == INT_MAX || !is_16(dtype)) return GPTQ_ERR_INVALID_ARG;
  if (x_dtype != GPTQ_F32 && !is_16(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dA) | reinterpret_cast<uintptr_t>(dB)) & 3) return GPTQ_ERR_INVALID_ARG;
  const uint64_t na = (uint64_t)a->n_adapters * a->rank * a->d_in * 4, nb = (uint64_t)a->n_adapters * a->rank * a->d_out * 4;
  if (share_bytes(dA, na, dB, nb)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0) {
    // sums over no tokens
    const int64_t n0 = na / 4, n = n0 + nb / 4;
    if (!dA && !dB) return GPTQ_OK;
    lora_join_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 8192), 256, 0, s>>>(nullptr, 0, 0, n0, n, dA, dB);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  if (!dY || !q_start || !adapter || (!dX && !dA && !dB) || (R && !dX) || (dA && !X) || (dB && !S)) return GPTQ_ERR_INVALID_ARG;
  if (lddy < a->d_out || (dA && ldx < a->d_in) || (dX && lddx < a->d_in) || (R && ldr < a->d_in)) return GPTQ_ERR_INVALID_ARG;
  if (!elem_at(dY, dtype) || !elem_at(X, dtype) || !elem_at(R, x_dtype) || !elem_at(dX, x_dtype) || !elem_at(S, GPTQ_F32) ||
      !elem_at(q_start, GPTQ_F32) || !elem_at(adapter, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  const uint64_t e = x_dtype == GPTQ_F32 ? 4 : 2, dxb = rows_bytes(m, lddx, a->d_in, e), dyb = rows_bytes(m, lddy, a->d_out, 2);
  const uint64_t xb = dA ? rows_bytes(m, ldx, a->d_in, 2) : 0, sb = (uint64_t)m * a->rank * 4;
  const struct {
    const void* p;
    uint64_t n;
  } outs[] = {{dX, dxb}, {dA, na}, {dB, nb}}, ins[] = {{dY, dyb}, {dA ? X : nullptr, xb}, {dB ? S : nullptr, sb}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (share_bytes(o.p, o.n, i.p, i.n)) return GPTQ_ERR_INVALID_ARG;
  if (share_bytes(dX, dxb, dA, na) || share_bytes(dX, dxb, dB, nb)) return GPTQ_ERR_INVALID_ARG;
  if (R) {
    const uint64_t rb = rows_bytes(m, ldr, a->d_in, e);
    if (!(R == dX && ldr == lddx) && share_bytes(dX, dxb, R, rb)) return GPTQ_ERR_INVALID_ARG;
    if (share_bytes(dA, na, R, rb) || share_bytes(dB, nb, R, rb)) return GPTQ_ERR_INVALID_ARG;
  }
  for (const auto& o : outs)
    if (meets_set(o.p, o.n, a, q_start, adapter, n_seqs)) return GPTQ_ERR_INVALID_ARG;
  const size_t need = lora_back_layout(m, a).total;
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return GPTQ_ERR_WORKSPACE;
  for (const auto& o : outs)
    if (share_bytes(ws, need, o.p, o.n)) return GPTQ_ERR_INVALID_ARG;
  for (const auto& i : ins)
    if (share_bytes(ws, need, i.p, i.n)) return GPTQ_ERR_INVALID_ARG;
  if (meets_set(ws, need, a, q_start, adapter, n_seqs) || (R && share_bytes(ws, need, R, rows_bytes(m, ldr, a->d_in, e)))) return GPTQ_ERR_INVALID_ARG;
  const LoraBatch b{q_start, adapter, n_seqs, a->n_adapters, m};
  char* base = static_cast<char*>(ws);
  if (dtype == GPTQ_BF16) return lora_backward<__bf16>(dY, lddy, X, ldx, S, a, b, R, ldr, dX, x_dtype, lddx, dA, dB, base, s);
  return lora_backward<_Float16>(dY, lddy, X, ldx, S, a, b, R, ldr, dX, x_dtype, lddx, dA, dB, base, s);
}
