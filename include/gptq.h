/*
 * gptq.h -- C ABI of the MI355X (gfx950) GPTQ layer quantizer, libgptq.so.
 *
 * The library quantizes the weights of one linear layer W [d_out x d_in] with
 * GPTQ: a Hessian from calibration activations, damping of its diagonal, an
 * optional column order by descending diag(H), the upper Cholesky factor of
 * H^-1, and a column-by-column min-max group quantization whose rounding
 * error is pushed onto the columns not yet quantized, 128 columns at a time
 * with one lazy update of the rest.
 *
 * Sources: the GPTQ practice page at m.lqnn.cn/news/117696, section 2.1 (the
 * OBQ step and the Hessian from calibration activations), section 2.2 (fixed
 * order, lazy batch updates, Cholesky of H^-1), section 3.3 (bits,
 * group_size, desc_act, damp_percent); the tutorial page "大模型压缩量化技术：
 * GPTQ 与 AWQ 原理详解 + Python 实战教程", section 二 (the min-max grid).
 *
 * Conventions shared by every call:
 *  - Pointers are device pointers owned by the caller, except out_host in
 *    gptq_layer_error, which is host memory.  The library allocates no device
 *    memory; scratch memory comes in through ws/ws_bytes, sized by the
 *    matching *_workspace_size query.  Workspaces need 256-byte alignment
 *    (any hipMalloc / torch allocation satisfies this).
 *  - The library keeps no state between calls (no handles, no globals) and
 *    reads no environment variables: every option is an argument.  The one
 *    exception is gptq_hessian_accumulate_noalloc, which keeps per device the
 *    address of its static scratch array.
 *  - All work is enqueued on stream s, in stream order: it starts after the
 *    work already on s and is complete, as seen from s, before anything
 *    enqueued on s later.  Only gptq_prepare_hinv and gptq_layer_error
 *    synchronize s (to read one device flag or scalar).
 *  - Argument errors return GPTQ_ERR_INVALID_ARG (or GPTQ_ERR_WORKSPACE)
 *    before anything is enqueued.  HIP failures return GPTQ_ERR_HIP.
 *  - Layouts are row-major.  Columns of W are input channels.  X is
 *    token-major [n_tokens x d_in].
 *  - Calls on distinct buffers and streams are independent (reentrant).
 */
#ifndef GPTQ_MI355X_H
#define GPTQ_MI355X_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GPTQ_F32 = 0, GPTQ_F16 = 1, GPTQ_BF16 = 2 } gptq_dtype;

typedef enum {
  GPTQ_OK = 0,
  GPTQ_ERR_INVALID_ARG = -1,
  GPTQ_ERR_NOT_PD = -2,      /* damped Hessian not positive definite: raise damp_percent */
  GPTQ_ERR_HIP = -3,
  GPTQ_ERR_WORKSPACE = -4,   /* workspace missing or smaller than the query returns */
  GPTQ_ERR_UNSUPPORTED = -5  /* a valid option this library does not implement */
} gptq_status;

/* The quantizer's options, as the pages' config objects name them
 * (practice page section 3.3; the ms-swift review page's GptqConfig).
 *  bits          2..8 (the code range is [0, 2^bits - 1])
 *  group_size    columns sharing one scale/zero (consecutive in processing
 *                order); -1 = one group per row.  Must divide block_size, or
 *                be a multiple of it, or be -1; in-block groups must be a
 *                multiple of 4.
 *  block_size    lazy-batch width; this library supports 128 only.
 *  damp_percent  lambda = damp_percent * mean(diag H) is added to diag(H).
 *  desc_act      0/1: process columns by descending diag(H).
 *  sym           0 = asymmetric min-max grid: scale = (max - min)/maxq,
 *                zero = rint(-min/scale).  1 = symmetric grid (the ms-swift
 *                review page's sym=True; no formula is given, the plainest
 *                reading is used): m = max(|min|, |max|), scale = 2m/maxq,
 *                zero = (maxq + 1)/2 (scale 1 for an all-zero group).
 *  per_block_steps  0 (default): with groups inside the block, each block's
 *                column loop runs in the same launch as the previous block's
 *                lazy update of the later columns.  1: one launch per step
 *                (column loop, then lazy update).  The results are the same
 *                bit for bit; 1 exists to show that. */
typedef struct {
  int32_t bits;
  int32_t group_size;
  int32_t block_size;
  float damp_percent;
  int32_t desc_act;
  int32_t sym;
  int32_t per_block_steps;
} gptq_config;

/* ---------------------------------------------------------------- Hessian
 * H += 2 * X^T X over n_tokens calibration tokens (practice page 2.1: the
 * Hessian is built from the layer's input activations).
 *  H        [d_in x d_in] fp32, full symmetric, accumulated into (the caller
 *           zero-fills it once; further calls add more tokens).
 *  hdiag    [d_in] fp64, nullable, accumulated like H: diag(H) summed in fp64
 *           (the squares of bf16/fp16 values are exact).  gptq_prepare_hinv
 *           orders columns by these keys when given, so the desc_act order is
 *           the exact one and does not depend on fp32 accumulation rounding.
 *           NULL: the 16-bit kernels do none of this work (H is the same).
 *  X        [n_tokens x d_in], token-major, of x_dtype (bf16/fp16 multiply
 *           exactly in fp32 on MFMA; fp32 inputs use the fp32 MFMA), 16-byte
 *           aligned (the kernels load 16 bytes at a time; INVALID_ARG else).
 *  d_in     1..65536, multiple of 8.  n_tokens >= 0 (0 leaves H unchanged).
 *  ws       scratch of gptq_hessian_workspace_size(n_tokens, d_in) bytes
 *           (partial sums of the split token range; the result does not
 *           depend on timing: every partial is reduced in a fixed order). */
size_t gptq_hessian_workspace_size(int64_t n_tokens, int32_t d_in);
int gptq_hessian_accumulate(float* H, double* hdiag, const void* X, gptq_dtype x_dtype,
                            int64_t n_tokens, int32_t d_in, void* ws, size_t ws_bytes,
                            hipStream_t s);

/* gptq_hessian_accumulate for callers that cannot allocate device memory
 * (code under HIP graph capture, tight calibration loops, harnesses that forbid
 * hipMalloc): the same H and hdiag (same kernels; H within fp32 accumulation
 * order of the other call, since the token range may be split differently),
 * with the partial sums in a static device array of
 * gptq_hessian_noalloc_scratch_bytes() = 256 MiB that each GPU the library
 * runs on holds until the process ends.  It calls no allocator.
 *  d_in up to 11,264 (one token split's partial tiles must fit the array);
 *  larger d_in returns GPTQ_ERR_WORKSPACE before anything is enqueued.
 *  The first call on a device looks up the array's device address (kept per
 *  device).  Every call on one GPU shares its array, so calls that overlap on
 *  one GPU (different streams, or host threads) race: order them on one
 *  stream.  Nothing in the array needs clearing (every partial is written
 *  before it is read). */
size_t gptq_hessian_noalloc_scratch_bytes(void);
int gptq_hessian_accumulate_noalloc(float* H, double* hdiag, const void* X, gptq_dtype x_dtype,
                                    int64_t n_tokens, int32_t d_in, hipStream_t s);

/* ---------------------------------------------------------------- H^-1 factor
 * From H (undamped, as accumulated): lambda = damp_percent * mean(diag H);
 * perm = processing order -> original column (identity, or stable descending
 * diag(H) when desc_act); U [d_in x d_in] fp32 upper triangular (zeros below)
 * with U^T U = (H[perm][:,perm] + lambda I)^-1 -- the triangular factor of the
 * inverse Hessian of practice page section 2.2 ("third").  The page calls it
 * lower-triangular; that factor is U^T.
 *  H        [d_in x d_in] fp32 input, unchanged.
 *  hdiag    [d_in] fp64 diagonal keys from gptq_hessian_accumulate, or NULL
 *           to take diag(H): used for lambda and for the desc_act order.
 *  U        [d_in x d_in] fp32 output.  perm [d_in] int32 output.
 *  ws       scratch of gptq_prepare_hinv_workspace_size(d_in) bytes.
 * Synchronizes s.  Returns GPTQ_ERR_NOT_PD when a pivot of the factorization
 * is <= 0 or NaN (the pages' remedy: a larger damp_percent); U is then
 * undefined. */
size_t gptq_prepare_hinv_workspace_size(int32_t d_in);
int gptq_prepare_hinv(const float* H, const double* hdiag, int32_t d_in, float damp_percent,
                      int32_t desc_act, float* U, int32_t* perm, void* ws, size_t ws_bytes,
                      hipStream_t s);

/* ---------------------------------------------------------------- quantize
 * GPTQ column loop (practice page 2.1 / 2.2; min-max grid of the tutorial
 * page section 二).  In processing order k (column perm[k]) and per row r:
 * at each group start, scale = (max - min)/maxq and zero = rint(-min/scale)
 * over the group's current (already compensated) weights; code =
 * clamp(rint(w/scale) + zero, 0, maxq); q = scale*(code - zero);
 * e = (w - q)/U[k][k]; the later columns of the 128-column block take
 * w -= e * U[k][.] at once, the columns after the block take one lazy update
 * W -= Err * U[block rows][after] at the block's end.  The block's running
 * weights, the grid and every integer decision (zero point, code) are fp64;
 * the work copy of W, U and the lazy update are fp32.  scales are the fp64
 * scales rounded to fp32.
 *  W       [d_out x d_in] of w_dtype, original column order, unchanged.
 *  U, perm as produced by gptq_prepare_hinv (processing order).
 *  codes   [d_out x d_in] uint8 output, original column order.
 *  scales  [d_out x n_groups] fp32, zeros [d_out x n_groups] int32 outputs,
 *          indexed by processing-order group; n_groups = ceil(d_in / G).
 *  g_idx   [d_in] int32 output: original column -> group.
 *  Q       [d_out x d_in] fp32 dequantized weights, original order; may be NULL.
 *  ws      scratch of gptq_quantize_workspace_size(d_out, d_in, cfg) bytes (cfg
 *          NULL: a size that suffices for every configuration at this shape).
 *  d_out >= 1, d_in >= 1 (any width; packing needs d_in % 8 == 0). */
size_t gptq_quantize_workspace_size(int32_t d_out, int32_t d_in, const gptq_config* cfg);
int gptq_quantize_layer(const void* W, gptq_dtype w_dtype, int32_t d_out, int32_t d_in,
                        const float* U, const int32_t* perm, const gptq_config* cfg,
                        uint8_t* codes, float* scales, int32_t* zeros, int32_t* g_idx,
                        float* Q, void* ws, size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- pack
 * Eight 4-bit codes per uint32 (practice page section 1.1: half a byte per
 * weight at 4 bits): packed[r][m] = sum_k (codes[r][8m+k] & 15) << 4k.
 *  codes [rows x cols] uint8, packed [rows x cols/8] uint32; cols % 8 == 0.
 *  3-bit codes are stored as nibbles too. */
int gptq_pack_int4(const uint8_t* codes, int64_t rows, int64_t cols, uint32_t* packed,
                   hipStream_t s);

/* Dense packing for 2, 3, 4 or 8 bits (practice page section 1.1 counts
 * bits/8 byte per weight): each row is one bit stream, code k at bits
 * [k*bits, (k+1)*bits) from the least significant bit of the row's word 0; a
 * 3-bit code may straddle two words.  At 4 bits the layout equals
 * gptq_pack_int4's.  Each code is masked to its low `bits` bits.
 *  codes [rows x cols] uint8, packed [rows x cols*bits/32] uint32.
 *  INVALID_ARG: bits not in {2, 3, 4, 8}, (cols * bits) % 32 != 0, null
 *  pointers, negative sizes. */
int gptq_pack_dense(const uint8_t* codes, int64_t rows, int64_t cols, int32_t bits,
                    uint32_t* packed, hipStream_t s);

/* ---------------------------------------------------------------- using the packed layer
 * Y = X W^T with W dequantized from the packed 4-bit layer (practice page
 * section 4.3: at inference the 4-bit weights are dequantized to a 16-bit type,
 * then multiplied).  W[r][c] = round16(scales[r][g] * (code[r][c] - zeros[r][g])),
 * the product taken in fp32 and rounded (ties to even) to x_dtype (the weight of
 * gptq_w4_linear too, which is the faster product where codes are packed in
 * processing order), with
 * code[r][c] = (packed[r][c/8] >> 4(c%8)) & 15 and g = g_idx[c] (clamped to
 * [0, n_groups)), or, with g_idx NULL, g = c / group_size (group_size a
 * multiple of 8, or -1 for one group per row).  Products accumulate in fp32;
 * Y is rounded once to y_dtype.
 *  X [m x d_in] f16/bf16 row-major, 16-byte aligned; packed [d_out x d_in/8]
 *  uint32; scales [d_out x n_groups] fp32; zeros [d_out x n_groups] int32;
 *  Y [m x d_out] of y_dtype (F32, F16 or BF16).  d_in % 8 == 0.
 *  INVALID_ARG: null pointers, bad sizes or dtypes, misaligned X, with g_idx
 *  NULL a group size that is not a multiple of 8 or an n_groups that does not
 *  match it. */
int gptq_w4a16_gemm(const void* X, gptq_dtype x_dtype, int64_t m, int32_t d_in,
                    const uint32_t* packed, const float* scales, const int32_t* zeros,
                    const int32_t* g_idx, int32_t group_size, int32_t n_groups, int32_t d_out,
                    void* Y, gptq_dtype y_dtype, hipStream_t s);

/* ---------------------------------------------------------------- layer error
 * out_host[0] = ||(W - Q) X^T||_F^2 = 1/2 tr((W - Q) H (W - Q)^T) with the
 * undamped H (practice page section 5.5: measure the loss, do not eyeball it).
 * fp32 products, fp64 final sum.  Synchronizes s.
 *  H [d_in x d_in] fp32, W [d_out x d_in] of w_dtype, Q [d_out x d_in] fp32.
 *  ws: gptq_layer_error_workspace_size(d_out, d_in) bytes. */
size_t gptq_layer_error_workspace_size(int32_t d_out, int32_t d_in);
int gptq_layer_error(const float* H, const void* W, gptq_dtype w_dtype, const float* Q,
                     int32_t d_out, int32_t d_in, double* out_host, void* ws, size_t ws_bytes,
                     hipStream_t s);

/* ---------------------------------------------------------------- AWQ
 * Activation-aware weight quantization, the second method of the pages
 * ("GPTQ/AWQ量化导出：让大模型在消费级显卡上跑起来", its AWQ steps: per-channel RMS
 * of the calibration activations, the top 5 % of channels get a larger factor,
 * the factor is undone at inference; "大模型压缩量化技术：GPTQ 与 AWQ 原理详解 +
 * Python 实战教程" section 四: weights of the large-activation channels times
 * s > 1, quantize, activations divided by s, the best factor chosen; no
 * Hessian).  The grid is the asymmetric min-max grid of the GPTQ calls, with
 * correctly rounded fp32 divisions. */

/* a[j] += sum_t X[t][j]^2 in fp64 (exact squares; the token splits are added
 * in a fixed order), the square of the RMS times n_tokens.  Accumulates, like
 * the Hessian: zero a before the first chunk.
 *  a   [d_in] fp64 (device).  X [n_tokens x d_in] of x_dtype.
 *  ws  scratch of gptq_awq_sumsq_workspace_size(n_tokens, d_in) bytes.
 *  n_tokens == 0 leaves a untouched. */
size_t gptq_awq_sumsq_workspace_size(int64_t n_tokens, int32_t d_in);
int gptq_awq_act_sumsq(double* a, const void* X, gptq_dtype x_dtype, int64_t n_tokens,
                       int32_t d_in, void* ws, size_t ws_bytes, hipStream_t s);

/* The factor search.  Salient channels: the k = floor(top_frac * d_in + 0.5)
 * channels with the largest a[j] (ties to the lower index).  For each
 * candidate sigma = grid[i]: s_j = sigma on salient channels, 1 elsewhere;
 * per group of group_size consecutive columns (-1: the whole row) the grid of
 * fp32(W[r][j] * s_j); Qhat = scale * (code - zero) / s_j (fp64); and
 * scores[i] = sum_j a[j] sum_r (W[r][j] - Qhat[r][j])^2 (fp64, rows added in a
 * fixed order).  The first smallest score wins: s_out[j] = its sigma on
 * salient channels, 1 elsewhere; *best = its index (best may be NULL).
 *  W [d_out x d_in] of w_dtype; a [d_in] fp64 from gptq_awq_act_sumsq;
 *  grid: HOST array of n_grid (1..32) finite factors > 0;
 *  s_out [d_in] fp32, scores [n_grid] fp64, best [1] int32 (device).
 *  ws  scratch of gptq_awq_search_workspace_size(d_out, d_in, group_size) bytes.
 *  INVALID_ARG: bits outside 2..8, group_size 0 or < -1, top_frac outside
 *  [0, 1], a bad grid, null pointers, non-positive sizes. */
size_t gptq_awq_search_workspace_size(int32_t d_out, int32_t d_in, int32_t group_size);
int gptq_awq_search(const void* W, gptq_dtype w_dtype, int32_t d_out, int32_t d_in,
                    const double* a, int32_t bits, int32_t group_size, float top_frac,
                    const float* grid, int32_t n_grid, float* s_out, double* scores,
                    int32_t* best, void* ws, size_t ws_bytes, hipStream_t s);

/* Quantize with given channel factors: per group the grid of
 * fp32(W[r][j] * s[j]); codes [d_out x d_in] uint8; scales/zeros
 * [d_out x n_groups] fp32/int32 (the grid of the scaled weights; at inference
 * the activations are divided by s); Qhat (may be NULL) [d_out x d_in] fp32,
 * the effective weights scale * (code - zero) / s[j] rounded from fp64. */
int gptq_awq_quantize(const void* W, gptq_dtype w_dtype, int32_t d_out, int32_t d_in,
                      const float* s, int32_t bits, int32_t group_size, uint8_t* codes,
                      float* scales, int32_t* zeros, float* Qhat, hipStream_t s_stream);

/* ---------------------------------------------------------------- one decoder block
 * The forward pieces that layer-by-layer quantization needs between the
 * sub-layers of a Llama decoder block ("GPTQ/AWQ量化导出：让大模型在消费级显卡上
 * 跑起来": a calibration forward pass collects each layer's inputs and the
 * layers are quantized one after another; "大模型压缩量化技术：GPTQ 与 AWQ 原理
 * 详解 + Python 实战教程": one layer at a time, its curvature from running the
 * calibration data through it).  fp32 throughout; token-major [T x d]. */

/* Y[t] = X[t] / sqrt(mean_j X[t][j]^2 + eps) * gamma (gamma NULL: 1).
 *  X [n_tokens x d] of x_dtype; Y [n_tokens x d] fp32. */
int gptq_rmsnorm(const void* X, gptq_dtype x_dtype, int64_t n_tokens, int32_t d,
                 const float* gamma, float eps, float* Y, hipStream_t s);

/* Y = X W^T (+ R): X [n_tokens x d_in], W [d_out x d_in] (e.g. the dequantized
 * Q of gptq_quantize_layer), R and Y [n_tokens x d_out]; R may be NULL or
 * equal to Y (then Y is accumulated into).  n_tokens <= INT_MAX.
 *  ws  scratch of gptq_linear_workspace_size(d_out, d_in) bytes (W^T). */
size_t gptq_linear_workspace_size(int32_t d_out, int32_t d_in);
int gptq_linear(const float* X, int64_t n_tokens, int32_t d_in, const float* W, int32_t d_out,
                const float* R, float* Y, void* ws, size_t ws_bytes, hipStream_t s);

/* Causal self-attention of the block: q = x1 Wq^T, k = x1 Wk^T, v = x1 Wv^T
 * ([d x d] each); q and k rotated per head (pairs (i, i + hd/2) by
 * p * rope_base^(-2i/hd), p = t % seq_len); per sequence of seq_len tokens and
 * per head: softmax(q_h k_h^T / sqrt(hd)) over positions <= the query's,
 * times v_h; out [n_tokens x d] is the heads side by side (the o projection's
 * input).  hd = d / n_heads must be even; n_tokens a multiple of seq_len and
 * at most 65535 * 32.
 *  ws  scratch of gptq_block_attention_workspace_size(...) bytes (W^T, q, k,
 *      v, k^T, one sequence's scores per head, the rotation table). */
size_t gptq_block_attention_workspace_size(int64_t n_tokens, int32_t d, int32_t n_heads,
                                           int32_t seq_len);
int gptq_block_attention(const float* x1, int64_t n_tokens, int32_t d, int32_t n_heads,
                         int32_t seq_len, const float* Wq, const float* Wk, const float* Wv,
                         float rope_base, float* out, void* ws, size_t ws_bytes, hipStream_t s);

/* M = silu(G) * U elementwise, silu(x) = x / (1 + exp(-x)); n elements. */
int gptq_swiglu(const float* G, const float* U, int64_t n, float* M, hipStream_t s);

/* ---------------------------------------------------------------- running the packed layer
 * Operators for running and fine-tuning a block whose layers are packed to 4
 * bits.  They share one description of a packed weight:
 *  packed     [d_out x d_in/8] uint32, gptq_pack_int4's layout, columns in
 *             processing order (codes[:, perm] for desc_act, else as they are).
 *             gptq_quantize_layer writes codes in channel order: a desc_act
 *             layer's are brought into this order before they are packed.
 *  scales, zeros  [d_out x n_groups] fp32 / int32, as gptq_quantize_layer
 *             writes them; group_size a multiple of 8, or -1 for one group per
 *             row; n_groups = ceil(d_in / group_size).
 *  perm       NULL, or the [d_in] int32 processing order (a permutation):
 *             packed column k belongs to channel perm[k].
 * The weight is W[r][perm[k]] = round16(scales[r][k/G] * (code[r][k] - zeros[r][k/G])),
 * the product in fp32, rounded (ties to even) to the activations' type, as in
 * gptq_w4a16_gemm.  d_in is a multiple of 8, at most 2^20; d_out is at most
 * 2^27 - 32 (the backward pass: 2^20).  Sums are fp32.
 * The struct itself is host memory and is read before the call returns. */
typedef struct {
  const uint32_t* packed;
  const float* scales;
  const int32_t* zeros;
  const int32_t* perm;
  int32_t d_out;
  int32_t d_in;
  int32_t group_size;
  int32_t n_groups;
} gptq_w4_weight;

/* SILU x / (1 + exp(-x)); GELU x Phi(x); GELU_TANH its tanh approximation
 * x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2. */
typedef enum {
  GPTQ_ACT_NONE = 0,
  GPTQ_ACT_RELU = 1,
  GPTQ_ACT_SILU = 2,
  GPTQ_ACT_GELU = 3,
  GPTQ_ACT_GELU_TANH = 4
} gptq_act;

/* Y = act(X W^T + bias) + R.  bias, activation and residual are applied to the
 * fp32 sums, which are rounded once, to y_dtype.
 *  X [m x d_in] f16/bf16, row t at X + t*ldx elements (ldx >= d_in).
 *  bias [d_out] of x_dtype, or NULL.  R [m x d_out] of y_dtype, row pitch ldr,
 *  or NULL; R may be Y itself (with ldr = ldy), else they do not overlap.  Y [m x d_out] of y_dtype
 *  (F32, F16 or BF16), row pitch ldy; elements between rows stay as they are.
 *  Y may overlap neither X nor bias.
 *  ws  scratch of gptq_w4_linear_workspace_size(m, w) bytes, 256-byte aligned:
 *      X's copy (for perm, or rows that are not 16-byte aligned), and from 17
 *      tokens on (with large weights from a few on) partial sums or the 16-bit
 *      weight.  A call that needs none of these takes ws NULL.  Calls that may
 *      run at the same time need workspaces of their own, as captured graphs do.
 *  m == 0 is a no-op.  INVALID_ARG: null pointers, bad sizes, types, pitches
 *  or group sizes. */
size_t gptq_w4_linear_workspace_size(int64_t m, const gptq_w4_weight* w);
int gptq_w4_linear(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_w4_weight* w,
                   const void* bias, gptq_act act, const void* R, int64_t ldr, void* Y,
                   gptq_dtype y_dtype, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t s);

/* The gated feed-forward block's first half in one product: G = X Wg^T,
 * U = X Wu^T, M = act(G) * U, from the fp32 sums of both.
 *  gate, up: packed weights of one shape, with the same group_size and the
 *  same perm pointer (they share one Hessian, so one order).
 *  X [m x d_in], row pitch ldx.  M [m x d_out] of x_dtype, contiguous.  G and
 *  U (both or neither; NULL when no backward pass follows): [m x d_out] of
 *  x_dtype, contiguous.  act: SILU, GELU or GELU_TANH.  M, G and U overlap
 *  neither X nor each other. */
size_t gptq_w4_gated_workspace_size(int64_t m, const gptq_w4_weight* gate, const gptq_w4_weight* up);
int gptq_w4_gated(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_w4_weight* gate,
                  const gptq_w4_weight* up, gptq_act act, void* G, void* U, void* M, void* ws,
                  size_t ws_bytes, hipStream_t s);

/* Its backward pass through the frozen packed weights: from dM, G and U
 *   dU = dM * act(G),  dG = dM * U * act'(G),  dX = dG Wg + dU Wu.
 * All [m x d_out] (dX: [m x d_in]) of one 16-bit type, contiguous.  dG and dU
 * are rounded to that type (what an adapter's gradient needs; each may be
 * NULL), and dX's products take the rounded values: one rounding more than
 * exact, of the size of dX's own.  dX is written whole, in channel order.
 * dG may be G (or dM, or U) and dU may be U (or dM, or G), whole; apart from that
 * no output overlaps another array, and dX, dG and dU that overlap each other
 * are refused. */
size_t gptq_w4_gated_backward_workspace_size(int64_t m, const gptq_w4_weight* gate,
                                             const gptq_w4_weight* up);
int gptq_w4_gated_backward(const void* dM, const void* G, const void* U, gptq_dtype dtype, int64_t m,
                           const gptq_w4_weight* gate, const gptq_w4_weight* up, gptq_act act, void* dG,
                           void* dU, void* dX, void* ws, size_t ws_bytes, hipStream_t s);

/* dX = dY W + R, the product's gradient through the frozen packed weight (a
 * bias's and an activation's are the caller's).
 *  dY [m x d_out] f16/bf16, row pitch lddy.  dX [m x d_in] of x_dtype (F32, F16 or
 *  BF16), row pitch lddx, in channel order, written whole.  R [m x d_in] of
 *  x_dtype, row pitch ldr, or NULL: what reaches X from elsewhere (the other
 *  projections of the same input, an adapter); R may be dX itself (with ldr = lddx),
 *  else they do not overlap, nor do dX and dY.
 *  The weight counts as rounded to dtype.  d_out is at most 2^20.
 *  ws  scratch of gptq_w4_linear_backward_workspace_size(m, w) bytes (the
 *      transposed 16-bit weight, dY's copy, partial sums). */
size_t gptq_w4_linear_backward_workspace_size(int64_t m, const gptq_w4_weight* w);
int gptq_w4_linear_backward(const void* dY, gptq_dtype dtype, int64_t m, int64_t lddy, const gptq_w4_weight* w,
                            const void* R, int64_t ldr, void* dX, gptq_dtype x_dtype, int64_t lddx, void* ws,
                            size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- adapters
 * Low-rank adapters of many requests beside a shared projection
 * (gptq_w4_linear's): a set holds n_adapters pairs of matrices of one 16-bit type,
 *  A      [n_adapters x rank x d_in], B [n_adapters x d_out x rank], contiguous,
 *  scale  [n_adapters] fp32,
 * rank 1..128 (a smaller one's rows and columns are filled with zeros), d_in and
 * d_out up to 2^20, channels in the layer's own order (whatever its perm).
 * A batch is described on the device: sequence b's tokens are rows q_start[b] ..
 * q_start[b+1]-1 ([n_seqs + 1] int32, not decreasing) and go through adapter[b]
 * ([n_seqs] int32; a number outside [0, n_adapters): through none).  Rows outside
 * [q_start[0], q_start[n_seqs]) are neither read nor written.
 * The struct itself is host memory and is read before the call returns. */
typedef struct {
  const void* A;
  const void* B;
  const float* scale;
  int32_t n_adapters;
  int32_t rank;
  int32_t d_in;
  int32_t d_out;
} gptq_lora_set;

/* Y = R + scale_a (X A_a^T) B_a^T; a token without an adapter has Y = R.
 *  X [m x d_in] of the set's type, row pitch ldx.  R [m x d_out] of y_dtype, row
 *  pitch ldr, or NULL (0); R may be Y itself (with ldr = ldy: the adapters are
 *  added to the shared projection's output), else they do not overlap.  Y [m x d_out]
 *  of y_dtype (F32, F16 or BF16), row pitch ldy, rounded once.
 *  S [m x rank] fp32, contiguous, or NULL: X A_a^T, for the backward pass (0 for a
 *  token without an adapter).  Sums are fp32; X A_a^T enters the second product in
 *  two 16-bit pieces (16 bits for bf16, 22 for fp16, for an F32 output too; an infinity
 *  in B may then come out as NaN).
 *  Y, S and the scratch overlap no input (the set's and the batch's among them; but Y
 *  may be R), nor each other.  m is at most 2^24, and so are the
 *  workgroups that the batch needs, some (m / 128 + n_seqs) * d_out / 256 (sequences of
 *  one token: m / 16 * d_out / 64); more are refused.
 *  ws  scratch of gptq_lora_workspace_size(m, set) bytes. */
size_t gptq_lora_workspace_size(int64_t m, const gptq_lora_set* set);
int gptq_lora(const void* X, gptq_dtype x_dtype, int64_t m, int64_t ldx, const gptq_lora_set* set,
              const int32_t* q_start, const int32_t* adapter, int32_t n_seqs, const void* R, int64_t ldr,
              void* Y, gptq_dtype y_dtype, int64_t ldy, float* S, void* ws, size_t ws_bytes, hipStream_t s);

/* Its backward pass, from dY, X and the forward pass's S, with dS = dY B_a:
 *   dX = R + scale_a dS A_a,  dA_a = scale_a sum_t dS_t^T X_t,
 *   dB_a = scale_a sum_t dY_t^T S_t,
 * the sums over all of an adapter's tokens (0 for one without any; both are
 * written whole).  Each of dX, dA and dB may be NULL; X is needed for dA, S for dB.
 *  dY [m x d_out] and X [m x d_in] of dtype, the set's; dX [m x d_in] and R (NULL:
 *  0; or dX itself) of x_dtype (F32, F16 or BF16): the shared projection's dX, say.
 *  dA [n_adapters x rank x d_in], dB [n_adapters x d_out x rank] fp32.
 *  Sums are fp32, added in a fixed order; dS enters dX's product in two 16-bit
 *  pieces as in the forward pass, dS and S those of dA and dB in three.  Outputs overlap neither inputs nor each other.
 *  ws  scratch of gptq_lora_backward_workspace_size(m, set) bytes (NULL if m is 0). */
size_t gptq_lora_backward_workspace_size(int64_t m, const gptq_lora_set* set);
int gptq_lora_backward(const void* dY, gptq_dtype dtype, int64_t m, int64_t lddy, const void* X, int64_t ldx,
                       const float* S, const gptq_lora_set* set, const int32_t* q_start, const int32_t* adapter,
                       int32_t n_seqs, const void* R, int64_t ldr, void* dX, gptq_dtype x_dtype, int64_t lddx,
                       float* dA, float* dB, void* ws, size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- the residual stream and its norms
 * What stands between two sub-layers, in one pass:
 *   b = B, or with post_gamma its norm: unit(B) * post_gamma,
 *   H = R + alpha * gate * b,   Y = unit(H) * gamma,
 * unit(x) = x / sqrt(mean_j x_j^2 + eps).  Y is the norm of the unrounded H.
 *  R, H   [m x d] of h_dtype, row pitches ldr, ldh: the stream before and after.
 *         H may be R (with ldh = ldr).
 *  B, Y   [m x d] of dtype, row pitches ldb, ldy.  h_dtype is dtype or F32.
 *         B NULL: H = R, only Y is written (post_gamma, gate and H are NULL).
 *         Y or H may be NULL; either may be B (same type and pitch).
 *  post_gamma, gate, gamma  [d] fp32, each NULL for 1 (post_gamma NULL: no norm).
 * Outputs overlap nothing else.  d is at most 16384.  Statistics are fp32. */
int gptq_residual_rmsnorm(const void* R, gptq_dtype h_dtype, int64_t ldr, const void* B, gptq_dtype dtype,
                          int64_t ldb, int64_t m, int32_t d, const float* post_gamma, const float* gate,
                          float alpha, const float* gamma, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                          hipStream_t s);

/* Its backward pass, at the stored stream H: with n = unit(H),
 *   dh = dH + (dY gamma - n mean(dY gamma n)) / sqrt(mean H^2 + eps),
 *   dR = dh,   dB = alpha gate dh, through unit(B) post_gamma where there is one,
 *   dgamma = sum_t dY n,   dgate = alpha sum_t dh b,
 *   dpost_gamma = sum_t alpha gate dh unit(B).
 *  dH  [m x d] of h_dtype, what reaches the stream behind the norm, or NULL (0).
 *  B   as in the forward pass; read only with post_gamma or gate (else it may be
 *      NULL).  dR of h_dtype, dB of dtype, dgamma, dpost_gamma and dgate [d] fp32:
 *      each may be NULL.  The sums are written, not added to (0 if m is 0), and do not
 *      depend on timing.
 *  dR and dB may each be one of dY, H, dH, B whole (same type and pitch); outputs and
 *  the scratch overlap nothing else, nor each other.
 *  ws  scratch of gptq_residual_rmsnorm_backward_workspace_size(m, d) bytes (NULL
 *      without dgamma, dpost_gamma and dgate). */
size_t gptq_residual_rmsnorm_backward_workspace_size(int64_t m, int32_t d);
int gptq_residual_rmsnorm_backward(const void* dY, gptq_dtype dtype, int64_t lddy, const void* H,
                                   gptq_dtype h_dtype, int64_t ldh, const void* dH, int64_t lddh, const void* B,
                                   int64_t ldb, int64_t m, int32_t d, const float* post_gamma, const float* gate,
                                   float alpha, const float* gamma, float eps, void* dR, int64_t lddr, void* dB,
                                   int64_t lddb, float* dgamma, float* dpost_gamma, float* dgate, void* ws,
                                   size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- a cache held in 4 bits
 * Keys and values of a decoder block in pages of 4-bit rows.  A row is one
 * token's head_dim values of one kv head, on its own min-max grid:
 *   lo = fp16(min), step = fp16(max(max - lo, 0) / 15) (fp32 arithmetic),
 *   code = clamp(rint((x - lo) / step), 0, 15) (0 when step is 0),
 * and stands for lo + step * code.  Inputs beyond +-65504 count as +-65504, a
 * NaN as the row's minimum (0 in a row of NaNs).
 *  k_codes, v_codes  [n_pages x n_kv_heads x page_size x head_dim/8] uint32,
 *                    code i of a row in bits 4(i%8) of word i/8; 16-byte aligned.
 *  k_grid, v_grid    [n_pages x n_kv_heads x page_size x 2] fp16: step, lo;
 *                    16-byte aligned.
 *  page_table        [n_seqs x max_pages] int32: token j of sequence b is row
 *                    j % page_size of page page_table[b][j / page_size].
 *  head_dim 64 or 128; page_size a multiple of 16.
 * A batch is described on the device: sequence b's new tokens are rows
 * q_start[b] .. q_start[b+1]-1 of the token-major inputs and outputs
 * ([n_seqs + 1] int32, not decreasing), and kv_len[b] ([n_seqs] int32) is its
 * length in the cache with them: its new token i sits at position
 * kv_len[b] - n_q + i.  Rows outside [q_start[0], q_start[n_seqs]) are neither
 * read nor written.  Tokens at positions below 0 or on a page whose number is
 * outside [0, n_pages) or past max_pages are not there: append skips them,
 * read gives zeros, attention does not see them.  Pages of one batch's
 * sequences may be shared (a common prefix) as long as no call appends to
 * them through two sequences. */
typedef struct {
  uint32_t* k_codes;
  uint32_t* v_codes;
  void* k_grid;
  void* v_grid;
  const int32_t* page_table;
  int32_t n_pages;
  int32_t n_kv_heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t n_seqs;
  int32_t max_pages;
} gptq_kv4_cache;

/* Quantize the new tokens' keys and values into their places.
 *  K, V: token t's row of head h at K + t*ldk + h*head_dim elements (f16, bf16
 *  or f32), ldk, ldv >= n_kv_heads * head_dim.  n_tokens: rows that K and V
 *  have (q_start is cut to it). */
int gptq_kv4_append(const gptq_kv4_cache* cache, const void* K, const void* V, gptq_dtype dtype,
                    int64_t n_tokens, int64_t ldk, int64_t ldv, const int32_t* q_start,
                    const int32_t* kv_len, hipStream_t s);

/* The values that the cache holds for the batch's tokens, in append's layout
 * (contiguous rows [n_tokens x n_kv_heads x head_dim]); K or V may be NULL. */
int gptq_kv4_read(const gptq_kv4_cache* cache, void* K, void* V, gptq_dtype dtype, int64_t n_tokens,
                  const int32_t* q_start, const int32_t* kv_len, hipStream_t s);

/* Causal attention of the batch's tokens over the cache: new token i of
 * sequence b, query head h, sees the positions j <= kv_len[b] - n_q + i of kv
 * head h / (n_heads / n_kv_heads):
 *   out = softmax_j(scale * q . k_j) v_j,
 * sums and statistics in fp32.  A row that sees nothing is 0.  |scale| is at
 * most 1e8; a key whose q . k or score is below -1e30 counts as not seen.
 *  Q: token t, head h at Q + t*ldq + h*head_dim (f16/bf16, 16-byte aligned
 *  rows); out likewise with ldo, not overlapping Q.
 *  max_q_len, max_kv_len: host bounds on n_q and kv_len, at least 1 (0 too
 *  where n_tokens is 0, which is a no-op in every call here); tokens past
 *  max_q_len of a sequence are left alone, positions past max_kv_len unseen.
 *  ws  scratch of gptq_kv4_attention_workspace_size(...) bytes (partial
 *      results of long sequences, joined in a fixed order). */
size_t gptq_kv4_attention_workspace_size(int64_t n_tokens, int32_t n_heads, const gptq_kv4_cache* cache,
                                         int32_t max_q_len, int32_t max_kv_len);
int gptq_kv4_attention(const void* Q, gptq_dtype dtype, int64_t n_tokens, int32_t n_heads, int64_t ldq,
                       const gptq_kv4_cache* cache, const int32_t* q_start, const int32_t* kv_len,
                       int32_t max_q_len, int32_t max_kv_len, float scale, void* out, int64_t ldo,
                       void* ws, size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- whole prompts
 * Causal attention of whole sequences packed one behind the other, before their
 * keys and values go into a cache, or in training: token i of a sequence, query
 * head h, sees the sequence's tokens j <= i of kv head h / (n_heads / n_kv_heads):
 *   out = softmax_j(scale * q . k_j) v_j,   lse = log sum_j exp(scale * q . k_j).
 *  Q, out  token t, head h at Q + t*ldq + h*head_dim elements; K, V likewise with
 *          n_kv_heads heads: rows of a fused projection as they are.  f16 or bf16,
 *          rows 16-byte aligned; pitches below 2^22 elements.  head_dim 64 or 128;
 *          n_heads a multiple of n_kv_heads.  out and lse overlap no input, nor each other.
 *  q_start [n_seqs + 1] int32 (device, not decreasing): sequence b is rows
 *          q_start[b] .. q_start[b+1]-1.  Rows outside [q_start[0], q_start[n_seqs])
 *          are left as they are, and so are a sequence's tokens past max_len
 *          (a host bound on the lengths, at least 1), which nobody sees.
 *  lse     [n_tokens x n_heads] fp32, or NULL: what the backward pass needs.
 * Scores and statistics are fp32; the probabilities are rounded to 16 bits for the
 * second product.  What comes behind a token or belongs to another sequence, infinities
 * and NaN too, does not reach it.  Tiles of 128 tokens (n_tokens / 128 + n_seqs at most)
 * times n_heads are below 2^24, more are refused.  |scale| is at most 1e8; a key whose
 * score is below -6e29 has no weight (but a value of it that is no number still makes
 * the row none), and a row of such keys alone is 0 (its lse -inf); a score above 1e38 may
 * count as infinite (the row is then no number). */
int gptq_prompt_attention(const void* Q, const void* K, const void* V, gptq_dtype dtype, int64_t n_tokens,
                          int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int64_t ldq, int64_t ldk,
                          int64_t ldv, const int32_t* q_start, int32_t n_seqs, int32_t max_len, float scale,
                          void* out, int64_t ldo, float* lse, hipStream_t s);

/* Its backward pass, from dOut and the forward pass's out and lse: with
 * p_ij = exp(scale q_i . k_j - lse_i) and ds_ij = p_ij (dout_i . v_j - dout_i . out_i),
 *   dV_j = sum p_ij dout_i,  dK_j = scale sum ds_ij q_i,  dQ_i = scale sum_j ds_ij k_j,
 * the sums over i >= j and over the query heads of a kv head.  (lse is fp32: p is
 * off by up to 2^-23 |lse| relatively.)
 *  dOut, out and dQ are laid out as Q, dK and dV as K and V, each with its own
 *  pitch (gradients of one fused row are written in place).  p and ds are rounded
 *  to 16 bits for the products (fp16: below a power of two that follows ds); sums are
 *  fp32, in a fixed order.
 *  dQ, dK and dV overlap no input (lse and q_start among them) and, row by row, not each
 *  other.
 *  ws  scratch of gptq_prompt_attention_backward_workspace_size(n_tokens, n_heads)
 *      bytes, apart from all arrays. */
size_t gptq_prompt_attention_backward_workspace_size(int64_t n_tokens, int32_t n_heads);
int gptq_prompt_attention_backward(const void* dOut, int64_t lddo, const void* Q, const void* K, const void* V,
                                   gptq_dtype dtype, int64_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                                   int32_t head_dim, int64_t ldq, int64_t ldk, int64_t ldv, const void* out,
                                   int64_t ldo, const float* lse, const int32_t* q_start, int32_t n_seqs,
                                   int32_t max_len, float scale, void* dQ, int64_t lddq, void* dK, int64_t lddk,
                                   void* dV, int64_t lddv, void* ws, size_t ws_bytes, hipStream_t s);

/* ---------------------------------------------------------------- misc */
const char* gptq_status_string(int status);
int gptq_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_MI355X_H */
