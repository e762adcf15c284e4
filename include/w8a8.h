/*
 * w8a8.h -- C ABI of the MI355X (gfx950) W8A8 INT8 projection library.
 *
 * The operation is the INT8 projection GEMM inside each block of a
 * MiniMax-H3-style audio/video diffusion transformer: Q, K, V, attention
 * output, FC1 and FC2 run with INT8 weights and per-token INT8 activations
 * at the model's native hidden width (5376), without padding K and without
 * dequantizing the weights ("feat(mps): support MiniMax-H3 INT8 inference
 * on Apple M5", LightX2V pull request #1672: description, commit notes and
 * "Changes" table).
 *
 * Conventions shared by every entry point:
 *   - All tensors are dense and row-major, with no leading-dimension
 *     arguments.  BF16 values are passed as their 16-bit patterns.
 *   - Device pointers only (memory the caller allocated on the current HIP
 *     device); the caller owns every buffer, including any workspace.  The
 *     library never allocates, frees or synchronizes.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Calls enqueue
 *     kernels on it and return without waiting.
 *   - Arguments are validated on the host before anything is enqueued; on
 *     error nothing is launched and no output is touched.  A launch failure
 *     returns W8A8_ERR_HIP; a device fault surfaces at the caller's next
 *     synchronization.
 *   - The current device must be a gfx950 GPU; otherwise W8A8_ERR_DEVICE
 *     (there is no other code path).
 *   - Calls on one stream are ordered; concurrent calls on different
 *     streams are safe as long as their output buffers do not overlap.
 *   - Not checked on the device (documented preconditions): activations are
 *     finite; weight scales are finite and > 0 (the converter on the
 *     LightX2V page validates exactly this, "Validation").
 */
#ifndef W8A8_H
#define W8A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  W8A8_OUT_BF16 = 0, /* y: uint16 BF16 bits [M,N]                        */
  W8A8_OUT_FP32 = 1, /* y: float [M,N], the epilogue before BF16 rounding */
  W8A8_OUT_I32 = 2   /* y: int32 [M,N], the raw INT32 accumulators        */
} w8a8_out_t;

typedef enum {
  W8A8_OK = 0,
  W8A8_ERR_NULL = 1,      /* a required pointer is NULL                  */
  W8A8_ERR_SHAPE = 2,     /* a size violates the shape contract          */
  W8A8_ERR_ALIGN = 3,     /* a pointer is not aligned as required        */
  W8A8_ERR_WORKSPACE = 4, /* workspace missing or smaller than required  */
  W8A8_ERR_OUT_DTYPE = 5, /* unknown output type                         */
  W8A8_ERR_ALIAS = 6,     /* an output overlaps an input or other output */
  W8A8_ERR_DEVICE = 7,    /* no HIP device, or it is not gfx950          */
  W8A8_ERR_HIP = 8,       /* a HIP call or kernel launch failed          */
  W8A8_ERR_ARG = 9        /* an option is unknown or out of range        */
} w8a8_status_t;

/* Largest K accepted by w8a8_gemm / w8a8_linear: with INT8 operands every
 * product is at most 128*128 = 2^14 in magnitude, so the INT32 accumulator
 * cannot overflow while K*2^14 <= 2^31 - 1; 130944 is the largest multiple
 * of 128 below that bound. */
#define W8A8_MAX_K 130944

/*
 * Per-token activation quantization.
 *   x        BF16 [M,K], 16-byte aligned.
 *   a_q      INT8 [M,K] out, 8-byte aligned.
 *   a_scale  FP32 [M] out, 4-byte aligned.
 * For each row m: amax = max_k |x[m,k]|; a_scale[m] = amax / 127 (binary32
 * division, round to nearest even); a_q[m,k] = x[m,k] / a_scale[m] divided
 * in binary32 and rounded to the nearest integer, ties to even, clamped to
 * [-127, 127].  A row of zeros gives a_scale = 0 and zero codes.  FP32
 * subnormals are kept.
 * Shape: 1 <= M <= 2^24 - 1 (a launch holds fewer than 2^32 work-items,
 * up to 256 per row), 8 <= K <= W8A8_MAX_K and K % 8 == 0 (16-byte rows
 * of BF16; up to K = 90112 a row stays in registers and is read once,
 * longer rows are read twice); rows whose length is not a multiple of the
 * kernel's chunk width are handled by masking the partial chunk, as the
 * LightX2V page's quantizer does (commit notes, "Changes" table).
 * Errors: NULL, SHAPE, ALIGN, ALIAS (a_q or a_scale overlapping x or each
 * other), DEVICE, HIP.
 */
int w8a8_quantize_act(const uint16_t *x, int64_t M, int64_t K, int8_t *a_q,
                      float *a_scale, void *stream);

/*
 * INT8 GEMM with fused dequantization epilogue.
 *   a_q       INT8 [M,K] activation codes, 16-byte aligned.
 *   a_scale   FP32 [M] per-token scales, 4-byte aligned.
 *   w_q       INT8 [N,K] weights in a Linear's stored layout (one row per
 *             output channel), 16-byte aligned, consumed as stored.
 *   w_scale   FP32 [N] per-output-channel scales (finite, > 0), 4-byte
 *             aligned (16-byte alignment lets the epilogue use vector
 *             loads; a channel slice of a larger array is accepted).
 *   bias      BF16 [N] or NULL (no bias), 2-byte aligned (8-byte: vector
 *             loads).
 *   out       [M,N] of the type selected by out_dtype, 16-byte aligned.
 *   out_dtype W8A8_OUT_BF16, W8A8_OUT_FP32 or W8A8_OUT_I32.
 *   workspace device scratch of at least w8a8_gemm_workspace_bytes(M, N,
 *             K) bytes (w8a8_workspace_bytes is always enough; may be NULL
 *             when the former is 0), 16-byte aligned.  It holds INT32
 *             partial sums of split-K launches; its contents before and
 *             after the call do not matter.
 * acc[m,n] = sum_k a_q[m,k] * w_q[n,k] exactly in INT32;
 * t = ((float)acc * a_scale[m]) * w_scale[n] + bf16->f32(bias[n]), each
 * operation rounded in binary32 with no fused multiply-add; BF16 output is
 * t rounded once to nearest even.  Adding the bias before the one rounding
 * follows "MLX implementation and experiment report" (MiniMax-H3-Image-mlx),
 * "What the default preserves".
 * Shape: 1 <= M < 2^31; N and K positive multiples of 128 (the LightX2V
 * page's shape contract, commit notes); N < 2^31; K <= W8A8_MAX_K; and the
 * tile grid (256 x 256 tiles of 512 work-items, or 64 x 128 tiles of 256)
 * below 2^32 work-items: M * N up to about 2^39 (M <= 25.6 million at
 * N = 21504).
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, OUT_DTYPE, ALIAS, DEVICE, HIP.
 */
int w8a8_gemm(const int8_t *a_q, const float *a_scale, const int8_t *w_q,
              const float *w_scale, const uint16_t *bias, void *out,
              int out_dtype, int64_t M, int64_t N, int64_t K,
              void *workspace, size_t workspace_bytes, void *stream);

/*
 * w8a8_gemm without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation).  Arguments, results and errors as w8a8_gemm;
 * the split-K partial sums go to a device array the library holds, one
 * copy of W8A8_NOALLOC_SCRATCH_BYTES per GPU for the life of the process
 * (no call allocates or frees anything).  Every shape w8a8_gemm accepts
 * fits: its partial sums never exceed that size (W8A8_ERR_WORKSPACE
 * otherwise).  Calls of this entry point that overlap in time on one GPU
 * (on different streams, or from different threads) share that array and
 * race: order them on one stream.  The array's contents between calls do
 * not matter (nothing in it needs clearing).  The array's address is
 * looked up once per GPU at the first call of any entry point there.
 */
#define W8A8_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int w8a8_gemm_noalloc(const int8_t *a_q, const float *a_scale,
                      const int8_t *w_q, const float *w_scale,
                      const uint16_t *bias, void *out, int out_dtype,
                      int64_t M, int64_t N, int64_t K, void *stream);

/*
 * Whole projection, the quantized Linear that replaces a BF16 Linear on
 * each of the six block projections ("feat(mps): support MiniMax-H3 INT8
 * inference on Apple M5", LightX2V pull request #1672, description: W8A8
 * on Q, K, V, attention output, FC1 and FC2; commit notes: per-token
 * activation quantization feeding the INT8 GEMM at native K): per-token
 * quantization of x (as w8a8_quantize_act) into the workspace, then the
 * INT8 GEMM with BF16 output (as w8a8_gemm), y = bf16(((float)acc*sa[m]) *
 * sw[n] + bias[n]) with the bias added before the one rounding ("MLX
 * implementation and experiment report", "What the default preserves").
 *   x   BF16 [M,K] (16-byte aligned); y BF16 [M,N] (16-byte aligned);
 *   the other arguments as for w8a8_gemm.
 * Workspace: at least w8a8_workspace_bytes(M, N, K) bytes, 16-byte
 * aligned, not overlapping any argument (the INT8 codes, their scales and
 * the GEMM's partial sums).  M <= 2^24 - 1 (the quantizer's bound).
 * Errors: as w8a8_gemm.
 */
int w8a8_linear(const uint16_t *x, const int8_t *w_q, const float *w_scale,
                const uint16_t *bias, uint16_t *y, int64_t M, int64_t N,
                int64_t K, void *workspace, size_t workspace_bytes,
                void *stream);

/*
 * Per-output-channel weight quantization (the converter side of the
 * GEMM: "feat(mps): support MiniMax-H3 INT8 inference on Apple M5",
 * LightX2V pull request #1672, "Validation" and "Changes": weights become
 * INT8 one row per output channel with a finite, positive FP32 scale).
 *   w        BF16 [N,K] in a Linear's layout, 16-byte aligned.
 *   w_q      INT8 [N,K] out, 8-byte aligned.
 *   w_scale  FP32 [N] out, 4-byte aligned.
 * Each row is quantized exactly as w8a8_quantize_act quantizes a token
 * row, except that an all-zero row takes the scale 1 (its codes are 0), so
 * every scale is finite and positive.  Shape, alignment and errors as
 * w8a8_quantize_act with M = N.
 */
int w8a8_quantize_weight(const uint16_t *w, int64_t N, int64_t K,
                         int8_t *w_q, float *w_scale, void *stream);

/*
 * Scale contract check: *bad_count (a device int32, 4-byte aligned)
 * receives the number of entries of w_scale [N] that are not finite and
 * > 0 (NaN, +-Inf, zero or negative), for weights produced elsewhere.
 * 0 <= N < 2^31.  Errors: NULL, SHAPE, ALIGN, DEVICE, HIP.
 */
int w8a8_check_scales(const float *w_scale, int64_t N, int32_t *bad_count,
                      void *stream);

/* Workspace bytes that serve both w8a8_linear and w8a8_gemm for this
 * shape: the INT8 activation codes [M,K] and their scales [M] that
 * w8a8_linear stages, plus the INT32 split-K partial sums of the GEMM, each
 * part starting at a 256-byte offset.  0 for shapes the contract rejects. */
size_t w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* The smaller workspace w8a8_gemm alone needs (only its split-K partial
 * sums; 0 when the plan for this shape splits nothing, and for shapes the
 * contract rejects). */
size_t w8a8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Static description of a status code (never NULL). */
const char *w8a8_status_string(int status);

/* hipError_t code of the last W8A8_ERR_HIP returned on this thread (0 if
 * none yet), for diagnostics. */
int w8a8_last_hip_error(void);

/* SHA-256 (64 hex digits) of the sources this library was compiled from
 * (its kernels, API layer and this header), so a caller can refuse a build
 * that no longer matches the sources beside it. */
const char *w8a8_build_id(void);

/*
 * Glue between projections (not part of the W8A8 method; it produces the
 * inputs a DiT block feeds to FC2 and to the next block).
 *
 * w8a8_silu_bf16: y[i] = x / (1 + exp(-x)) correctly rounded to BF16, for
 *   n elements, read from a table of all 65536 BF16 inputs that a small
 *   kernel fills on the device (FP32 evaluation, FP64 for the rare inputs
 *   whose FP32 value lies too close to a BF16 rounding midpoint) on the
 *   caller's stream ahead of every call; x and y 16-byte aligned, n >= 0
 *   and n % 8 == 0; x and y may be the same buffer (in place) but must not
 *   partially overlap.
 *   Between FC1 and FC2 the block applies SiLU to the BF16 output of FC1
 *   ("MLX implementation and experiment report", "What the default
 *   preserves": SiLU rounding follows the original recipe).
 *
 * w8a8_pow2_renorm: each row of x [M,K] is multiplied by 2^-e, where
 *   e = floor(log2(max_k |x[m,k]|)), and rounded to BF16 (all-zero rows
 *   are copied).  Per-token symmetric quantization is exactly invariant to
 *   such a scaling, so chaining blocks through it changes no INT8 code
 *   while keeping BF16 activations finite.  K % 8 == 0, 16-byte aligned;
 *   in place allowed.
 *
 * w8a8_pow2_renorm_quantize: w8a8_pow2_renorm of x into y followed by
 *   w8a8_quantize_act of y, in one pass over x: y BF16 [M,K] is written
 *   and a_q INT8 [M,K], a_scale FP32 [M] are exactly what
 *   w8a8_quantize_act(y) produces.  x, y 16-byte aligned, a_q 8-byte,
 *   a_scale 4-byte; 8 <= K <= 90112, K % 8 == 0; y may be x (in place) but
 *   must not partially overlap it; a_q and a_scale overlap nothing.
 *   Errors as w8a8_quantize_act.
 *
 * w8a8_quantize_act_silu: w8a8_silu_bf16 followed by w8a8_quantize_act in
 *   one pass over x (the SiLU values are rounded to BF16 before they are
 *   quantized, exactly as the two separate calls do); the BF16 SiLU output
 *   is not written.  Arguments and errors as w8a8_quantize_act, with
 *   8 <= K <= 90112.
 */
int w8a8_silu_bf16(const uint16_t *x, uint16_t *y, int64_t n, void *stream);

/*
 * Gated-MLP glue for the fused gate/up projection of the pages' H3 shapes
 * ("MLX implementation and experiment report", "Operator tuning": a fused
 * gate/up GEMM 5376 -> 28672 feeding a down GEMM 14336 -> 5376; "What the
 * default preserves": BF16 products and SiLU rounding as in the original).
 *
 * w8a8_swiglu_bf16: h BF16 [M, 2F] holds the gate g in its first F columns
 *   and the up value u in the next F; y BF16 [M, F] = BF16(BF16(silu(g)) *
 *   u), the SiLU as w8a8_silu_bf16 and the product (exact in FP32) rounded
 *   once to nearest even.  h and y 16-byte aligned, F % 8 == 0, M >= 1; y
 *   must not overlap h.
 *
 * w8a8_quantize_act_swiglu: w8a8_swiglu_bf16 followed by
 *   w8a8_quantize_act of the [M, F] result in one pass over h (the SwiGLU
 *   output is not written).  a_q INT8 [M, F] (8-byte aligned), a_scale
 *   FP32 [M] (4-byte aligned); 8 <= F <= 90112.  Errors as
 *   w8a8_quantize_act.
 */
int w8a8_swiglu_bf16(const uint16_t *h, uint16_t *y, int64_t M, int64_t F,
                     void *stream);
int w8a8_quantize_act_swiglu(const uint16_t *h, int64_t M, int64_t F,
                             int8_t *a_q, float *a_scale, void *stream);
int w8a8_pow2_renorm(const uint16_t *x, uint16_t *y, int64_t M, int64_t K,
                     void *stream);
int w8a8_pow2_renorm_quantize(const uint16_t *x, int64_t M, int64_t K,
                              uint16_t *y, int8_t *a_q, float *a_scale,
                              void *stream);
int w8a8_quantize_act_silu(const uint16_t *x, int64_t M, int64_t K,
                           int8_t *a_q, float *a_scale, void *stream);

/*
 * Block norms: what stands between a block's projections.
 *
 * In front of a projection the block normalizes its input row and modulates
 * it (a shift and a scale per token or per group of tokens); behind the
 * attention output and the MLP it may normalize the branch, gates it and adds
 * it to the residual.  With r the residual row after the addition:
 *
 *   norm(v)  RMS:    v * rsqrt(mean(v^2) + eps) * weight
 *            LAYER:  (v - mean(v)) * rsqrt(mean((v - mean(v))^2) + eps)
 *                    * weight + bias
 *            NONE:   v
 *   r = residual_scale * x + gate[i] * post(branch)
 *   y = pre(r) * (1 + scale[i]) + shift[i]
 *
 * all in binary32 (sums and statistics included).  r is rounded to BF16 where
 * it is written; the norm behind it reads r before that rounding, and the
 * quantizing forms take y before any rounding to BF16: the scale is
 * max|y| / 127 and the codes are the integers nearest to y / scale in [-127,
 * 127] (taken as y times the reciprocal: either neighbour where y / scale lies
 * within 2^-16 of a half; a row of zeros has scale 0 and codes 0).
 * (norm_modulate followed by quantize_act quantizes the rounded y instead, and
 * may differ by a code.)
 *
 * i is the token's modulation row: row[m] when `row` is given, else m when
 * rows == M, else 0 (rows must then be 1).  A row[m] outside [0, rows) marks
 * token m as padding: what its branch row holds does not count, r is x
 * unchanged bit for bit, y and its codes and scale are zero.  `row` needs
 * rows >= 1 also where no vector is given.
 *
 * Rows are independent: a row that holds Inf or NaN spoils only itself.
 * Behind an RMS or layer norm the sum of squares must stay below the binary32
 * range (|v| below about 2^56); where it does not, or v holds Inf or NaN, the
 * norm's whole row is NaN.  A NaN anywhere in y, from x, the branch or a
 * vector, makes the row's scale NaN, and an Inf makes it Inf (or NaN); codes
 * under such a scale mean nothing.  Padding tokens stay as they are said to be.
 */
typedef enum {
  W8A8_NORM_NONE = 0,
  W8A8_NORM_RMS = 1,
  W8A8_NORM_LAYER = 2
} w8a8_norm_kind_t;

typedef struct {
  int kind;               /* w8a8_norm_kind_t                               */
  float eps;              /* 2^-126 <= eps < Inf (ignored for NONE)          */
  const uint16_t *weight; /* BF16 [H], 16-byte aligned, or NULL (ones)       */
  const uint16_t *bias;   /* BF16 [H], 16-byte aligned, or NULL (zeros);
                             LAYER only.  NONE takes neither.               */
} w8a8_norm_t;

/* Modulation vectors: each is NULL (scale and shift 0, gate 1) or `rows` rows
 * of H BF16 values at its own row stride in elements (so that the parts of
 * one [rows, 6 H] table can be passed as they are): 16-byte aligned, strides
 * multiples of 8, H or more and below 2^30, or 0 (one row for all).  The
 * residual alone reads no scale and shift, the norm alone no gate. */
typedef struct {
  const uint16_t *scale, *shift, *gate;
  int64_t scale_stride, shift_stride, gate_stride;
  int64_t rows;           /* 1 <= rows < 2^31 (0 without any vector)         */
  const int32_t *row;     /* int32 [M], 4-byte aligned, or NULL              */
} w8a8_modulation_t;

/* Largest row the block norms take (it stays in registers). */
#define W8A8_NORM_MAX_H 32768

/*
 * w8a8_norm_modulate            x -> y.
 * w8a8_norm_modulate_quantize   x -> codes and scales of y.
 * w8a8_gated_residual           x, branch -> r.
 * w8a8_gated_residual_norm      x, branch -> r, y.
 * w8a8_gated_residual_norm_quantize
 *                               x, branch -> r, codes and scales of y.
 *   x, branch, r, y  BF16 [M,H], 16-byte aligned; r may be x itself (in
 *             place), no other overlap of an output with anything.
 *   a_q       INT8 [M,H], 8-byte aligned; a_scale FP32 [M], 4-byte aligned.
 *   post, pre the norms; NULL means NONE.  mod NULL means no modulation.
 *   residual_scale  finite.
 * The structs are read during the call only.
 * Shape: 1 <= M <= 2^24 - 1, 8 <= H <= W8A8_NORM_MAX_H, H % 8 == 0,
 * M * H < 2^36.
 * Errors: NULL, SHAPE (M, H, rows, strides), ARG (kind, eps, residual_scale, a
 * weight or bias that the kind does not take), ALIGN, ALIAS, DEVICE, HIP.
 */
int w8a8_norm_modulate(const uint16_t *x, int64_t M, int64_t H,
                       const w8a8_norm_t *pre, const w8a8_modulation_t *mod,
                       uint16_t *y, void *stream);
int w8a8_norm_modulate_quantize(const uint16_t *x, int64_t M, int64_t H,
                                const w8a8_norm_t *pre,
                                const w8a8_modulation_t *mod, int8_t *a_q,
                                float *a_scale, void *stream);
int w8a8_gated_residual(const uint16_t *x, const uint16_t *branch, int64_t M,
                        int64_t H, const w8a8_norm_t *post,
                        const w8a8_modulation_t *mod, float residual_scale,
                        uint16_t *r, void *stream);
int w8a8_gated_residual_norm(const uint16_t *x, const uint16_t *branch,
                             int64_t M, int64_t H, const w8a8_norm_t *post,
                             const w8a8_norm_t *pre,
                             const w8a8_modulation_t *mod,
                             float residual_scale, uint16_t *r, uint16_t *y,
                             void *stream);
int w8a8_gated_residual_norm_quantize(
    const uint16_t *x, const uint16_t *branch, int64_t M, int64_t H,
    const w8a8_norm_t *post, const w8a8_norm_t *pre,
    const w8a8_modulation_t *mod, float residual_scale, uint16_t *r,
    int8_t *a_q, float *a_scale, void *stream);

/*
 * Linear over few tokens with packed 4-bit weights and group scales.
 *
 * A weight is (u - 8) * s, u its 4-bit code and s the BF16 scale of its group:
 * `group` (32, 64 or 128) consecutive inputs of one output channel.  The
 * activations stay BF16: y[m,n] = bf16(sum_k x[m,k] * w[n,k] + bias[n]), each
 * group's sum of x * (u - 8) and the sum over groups in binary32.  At few
 * tokens the weights are the bytes a Linear moves; half of the INT8 ones.
 *
 * Packed layout (N % 16 == 0, K % 128 == 0), written by the two converters
 * below, contiguous, one block per 16 channels x 128 inputs:
 *   w4       uint8 [N/16][K/128][64][16]: byte b of lane l holds the codes of
 *            channel 16 i + l % 16 at input 128 j + 32 (b / 4) + 8 (l / 16) +
 *            b % 4 (low four bits) and at the input 4 further (high bits);
 *   w4_scale BF16 [N/16][K/128][16][128/group]: the scale of channel 16 i + c
 *            for the inputs from 128 j + group * t on.
 * Any content of w4 is valid.
 */

/*
 * Converts a BF16 weight [N,K] in a Linear's layout: per group, scale =
 * bf16(max|w| / 7) (1 for a group of zeros, at least the smallest BF16 above
 * zero otherwise) and code = clamp(round_half_even(w / scale), -7, 7), the
 * divisions in binary32.  A group that holds NaN has a NaN scale, one that holds
 * Inf an infinite one (their codes mean nothing): w8a8_w4_linear gives NaN or
 * Inf for such a channel.
 *   w 16-byte aligned; w4 and w4_scale 16-byte aligned, overlapping nothing.
 * Shape: 16 <= N < 2^26, N % 16 == 0; 128 <= K <= W8A8_MAX_K, K % 128 == 0;
 * N * K < 2^37 (a launch holds fewer than 2^32 work-items).  Errors: NULL,
 * SHAPE, ARG (group), ALIGN, ALIAS, DEVICE, HIP.
 */
int w8a8_w4_quantize_weight(const uint16_t *w, int64_t N, int64_t K,
                            int64_t group, uint8_t *w4, uint16_t *w4_scale,
                            void *stream);

/*
 * Packs codes and scales that were made elsewhere: codes INT8 [N,K] (values
 * outside [-8, 7] are clamped), scales BF16 [N, K/group], both row-major and
 * 16-byte aligned.  Shape and errors as w8a8_w4_quantize_weight.
 */
int w8a8_w4_pack_weight(const int8_t *codes, const uint16_t *scales,
                        int64_t N, int64_t K, int64_t group, uint8_t *w4,
                        uint16_t *w4_scale, void *stream);

/*
 * The product.  x BF16 [M,K] and y BF16 [M,N], 16-byte aligned; w4 and
 * w4_scale as above; bias BF16 [N], 2-byte aligned, or NULL.  No workspace.
 * A token that holds Inf or NaN spoils only its own outputs.  Nothing overflows
 * on the way to a finite y while the magnitudes of x in a group sum to less than
 * the binary32 range and the sums over groups stay below 16 times that range.
 * The codes' offset is taken off by groups (the sum of 8 x from that of u x), so
 * that each input costs a few binary32 roundings of |x| (|u - 8| + 16) s, also
 * where its weight is zero.
 * Made for a few tokens: beyond 32 the weights are read again for every 32
 * (from there on w8a8_linear is faster where N or K is large).
 * Shape: 1 <= M <= 32 * 65535; N and K as above.
 * Errors: NULL, SHAPE, ARG (group), ALIGN, ALIAS (y overlapping an input),
 * DEVICE, HIP.
 */
int w8a8_w4_linear(const uint16_t *x, const uint8_t *w4,
                   const uint16_t *w4_scale, const uint16_t *bias,
                   uint16_t *y, int64_t M, int64_t N, int64_t K,
                   int64_t group, void *stream);

/*
 * Heads: what stands between a block's Q, K and V and its output projection.
 * A row holds the heads of one token behind each other, D values each; rows lie
 * at any stride (in elements), so that the parts of a fused Q, K, V output can
 * be passed as they are.
 */

/*
 * Rotary table: cosines and sines of a token's positions.
 *   positions  INT32 or FP32 [T, axes], 4-byte aligned (frame, row and column
 *              of a token, or its place alone).
 *   table      FP32 [T, 2, P] out, 16-byte aligned: the P cosines of a token,
 *              then its P sines; P is the sum of pairs[0 .. axes - 1].
 * Pair i of axis a turns by position * f(a, i), with p = pairs[a]:
 *   NONE    f = theta^(-i / p)
 *   LINEAR  f = theta^(-i / p) / factor
 *   NTK     f = (theta * factor^(p / (p - 1)))^(-i / p)   (p = 1: f = 1)
 *   YARN    f = theta^(-i / p) * (ramp / factor + 1 - ramp), ramp = clamp((i -
 *           low) / (high - low), 0, 1), low = max(floor(at(beta_fast)), 0),
 *           high = min(ceil(at(beta_slow)), 2 p - 1), at(b) = p *
 *           ln(original / (2 pi b)) / ln(theta); a high - low below 0.001
 *           counts as 0.001 ("YaRN", Peng et al., 2023)
 * and the table holds amplitude * cos and amplitude * sin.  Frequencies (off by
 * 1.25 * 2^-52 of themselves at most) and their products with positions are rounded
 * to binary64, so an angle is off by |angle| * 1.75 * 2^-52 at most; the result is
 * rounded to binary32 (6 * 2^-24 of the amplitude off at most).  A position that is NaN or
 * Inf gives NaN.
 * Shape: 1 <= T <= 2^24 - 1; 1 <= axes <= 4, each with 1 or more pairs, 256 in
 * all.  theta finite and > 1, factor finite and >= 1 (and what NTK makes of them
 * finite), amplitude finite in binary32; for YARN original finite and > 0,
 * beta_fast and beta_slow finite and > 0.
 * Errors: NULL, SHAPE, ARG, ALIGN, ALIAS, DEVICE, HIP.
 */
#define W8A8_ROPE_MAX_AXES 4
#define W8A8_ROPE_MAX_PAIRS 256

typedef enum {
  W8A8_ROPE_NONE = 0,
  W8A8_ROPE_LINEAR = 1,
  W8A8_ROPE_NTK = 2,
  W8A8_ROPE_YARN = 3
} w8a8_rope_scaling_t;

typedef enum {
  W8A8_POSITIONS_I32 = 0,
  W8A8_POSITIONS_F32 = 1
} w8a8_positions_t;

typedef struct {
  int axes;
  int pairs[W8A8_ROPE_MAX_AXES];
  int scaling;            /* w8a8_rope_scaling_t                            */
  double theta, factor;   /* factor is not read for NONE                    */
  double original, beta_fast, beta_slow; /* read for YARN only              */
  double amplitude;
} w8a8_rope_t;

int w8a8_rope_table(const void *positions, int position_type, int64_t T,
                    const w8a8_rope_t *rope, float *table, void *stream);

/*
 * Norms of queries and keys for each head, with the rotation in the same pass.
 * Every head of a token is normalized over its D values (the norm of
 * w8a8_norm_t, with NONE for the rotation alone), then its first 2 P values are
 * turned by the token's row of a rotary table: pair i's values (a, b) become
 *   (a cos_i - b sin_i, b cos_i + a sin_i)
 * all in binary32, rounded to BF16 once.  The pair is (2 i, 2 i + 1) where
 * `interleaved`, else (i, i + P); values from 2 P on are not turned.
 *
 *   q, k     one side each; k may be NULL.
 *   table    FP32 [rows, 2, P] as above, 16-byte aligned, or NULL (no
 *            rotation; pairs, rows and row are then not read).
 *   row      INT32 [M], 4-byte aligned: each token's row of the table; NULL:
 *            row m (rows == M), or row 0 for all (rows == 1).  A row outside
 *            [0, rows) marks a padding token: its outputs are zero, whatever
 *            it holds.
 * A head that holds Inf or NaN spoils only itself (behind RMS or LAYER all of
 * it is NaN; without a norm only the pair that holds it).
 * y may be x itself with the same stride (in place); else no output overlaps
 * anything (parts of one row that interleave at one stride do not).
 * Shape: 1 <= M <= 2^24 - 1; 8 <= D <= 256, D % 8 == 0; 1 <= heads <= 4096;
 * strides multiples of 8, heads * D or more and below 2^30; P % 4 == 0,
 * 2 P <= D; 1 <= rows < 2^31; M * heads * D < 2^36 for each side, and a launch
 * of fewer than 2^32 work-items.
 * Errors: NULL, SHAPE, ARG (norm), ALIGN (x, y, weight, bias, table: 16 bytes),
 * ALIAS, DEVICE, HIP.
 */
typedef struct {
  const uint16_t *x;  /* BF16 [M] rows of heads * D                         */
  uint16_t *y;        /* BF16 out, likewise                                  */
  int64_t heads, x_stride, y_stride;
  w8a8_norm_t norm;   /* weight and bias BF16 [D], or [heads, D] where        */
  int per_head;       /* this is not 0                                       */
} w8a8_heads_t;

int w8a8_head_norm_rope(const w8a8_heads_t *q, const w8a8_heads_t *k,
                        int64_t M, int64_t D, const float *table,
                        int64_t pairs, int64_t rows, const int32_t *row,
                        int interleaved, void *stream);

/*
 * Attention of queries to keys and values of another length (an encoder's
 * states, or the block's own tokens), for B sequences at once:
 *   out = softmax(scale * q k^T) v
 * for each sequence and head, over all of the sequence's keys.  Query head h
 * reads key head h / (q_heads / k_heads).
 *   q, out  BF16, Tq rows of q_heads * D;  k, v  BF16, Tk rows of k_heads * D.
 *   q_offsets, k_offsets  INT32 [B + 1], 4-byte aligned: sequence b's rows are
 *           those from offsets[b] to offsets[b + 1] - 1; NULL: B sequences of
 *           T / B rows each (T % B == 0).
 *   k_lens  INT32 [B], 4-byte aligned, or NULL: only the first k_lens[b] of a
 *           sequence's keys count (padding behind; none if not positive).
 * Offsets do not decrease (where they do, or leave [0, T], rows of out may be
 * written with any values, but nothing outside of q, k, v and out is touched).
 * Query rows outside of all sequences are left as they were.  What k and v hold
 * at keys that do not count does not matter.  A sequence without keys gives
 * zeros.  Scores, maxima, sums and outputs are held in binary32; weights are
 * rounded to BF16 for the product with v, and their sum is taken of the rounded
 * ones.  Inf or NaN in q spoils its own row and head; in k or v that counts,
 * the rows of its sequence and heads; a row all of whose scores are -Inf is
 * NaN.
 * Workspace: w8a8_attention_workspace_bytes of the same sizes, 16-byte aligned,
 * of this call alone until it is done (it holds the parts of a call whose keys
 * are split; 0 where they are not).  Every row of a part that is read is
 * written before, by the same call.
 * out overlaps nothing (parts of one row that interleave at one stride do not).
 * Results do not depend on other calls, nor on how work groups run.
 * Shape: 1 <= B <= 2^20; 1 <= Tq, Tk (0 <= Tk: k and v may then be NULL) and
 * T * heads < 2^31; 8 <= D <= 128, D % 8 == 0; q_heads a multiple of k_heads;
 * strides multiples of 8, heads * D or more and below 2^22; a launch of fewer
 * than 2^32 work-items.  0 < scale, and scale * log2(e) finite in binary32; the
 * sums of q k^T, and scale * log2(e) times them, within the binary32 range.
 * Errors: NULL, SHAPE, ARG (scale), ALIGN (q, k, v, out: 16 bytes), WORKSPACE,
 * ALIAS, DEVICE, HIP.
 */
typedef struct {
  const uint16_t *q, *k, *v;
  uint16_t *out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  int64_t Tq, Tk, B;
  int64_t q_heads, k_heads, D;
  const int32_t *q_offsets, *k_offsets, *k_lens;
  float scale;
} w8a8_attention_t;

size_t w8a8_attention_workspace_bytes(const w8a8_attention_t *a);
int w8a8_attention(const w8a8_attention_t *a, void *workspace,
                   size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
