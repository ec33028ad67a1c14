/*
 * nf4.h -- C ABI of libnf4 (package dequant_gemm_amd): NF4 blockwise weight
 * quantization with double quantization, and the fused NF4-dequant GEMMs,
 * for AMD Instinct MI355X (gfx950).
 *
 * What the calls compute (sources cited by page title and passage):
 *
 *  - "Zenbit" (PyPI project page), section "What's inside", bullet zenbit.nf4:
 *    NF4 blockwise quantization with double quantization of the scale
 *    factors, QLoRA-style.  Bullet zenbit.pallas_nf4: a fused NF4
 *    dequant+matmul whose weight streams compressed and is dequantized on
 *    chip, never materialised at full precision in device memory; a fused
 *    backward that forms dL/dX without materialising the weight, and no dL/dW
 *    (the quantized base weight is frozen).
 *  - "bitsandbytes" (unfragile.ai artifact page), NF4 data-type paragraph:
 *    16 levels from the inverse normal CDF, more of them near zero; weights
 *    map to levels through lookup tables after per-block scaling.
 *    Double-quantization paragraph: one absmax per 64-weight block, the absmax
 *    values themselves quantized to 8 bits with their own meta-scales; the
 *    scales are dequantized first, then used to dequantize the weights.
 *    Quantized-GEMM paragraph: weights dequantized on the fly, float32
 *    multiply, float32 outputs.  QuantState paragraph: the quantized data,
 *    absmax, data type and shape travel together (here: nf4_qtensor).
 *    4-bit training paragraph: the 4-bit data type is NF4 or FP4, standard
 *    floating-point 4-bit (quant_type NF4_QT_FP4 here).
 *
 * Exact semantics (the readings where the pages are silent):
 *  - weight W is logical [rows, cols] row-major, flattened e = r*cols + c;
 *    with B weights per block (64 by default; 32, 128 or 256), block b holds
 *    elements Bb .. Bb+B-1 (the last block may be partial);
 *  - a_b = max|x| over the block (fp32); n = fp32(x / a_b) (IEEE division);
 *    code = index of the nearest level, ties to the lower index; an all-zero
 *    block codes every element as the +0 level (NF4 code 7, FP4 code 0);
 *  - NF4 levels ascend with the code (nf4_codebook).  FP4 codes are the bit
 *    patterns of the E2M1 4-bit float (bit 3 the sign, bits 2-1 the exponent
 *    with bias 1, bit 0 the mantissa: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6)
 *    and a level is the value over 6, rounded once to fp32; ties to the lower
 *    code then go toward zero, and zero takes code 0;
 *  - packed byte j = code[2j] | code[2j+1] << 4 (odd count: high nibble 0);
 *  - double quantization: mu = exact mean of all a_b rounded once to fp32;
 *    a'_b = fp32(a_b - mu); per group of 256 consecutive blocks
 *    s_g = fp32(max|a'| / 127); q_b = clamp(rint_even(fp32(a'_b / s_g)),
 *    -127, 127) as int8; an all-zero group has s_g = 0 and q = 0;
 *  - dequantized absmax a^_b = fp32(fp32(q_b * s_g) + mu) with double
 *    quantization (two roundings, no fused multiply-add), else a^_b = a_b;
 *  - W^_e = bf16_rne(fp32(level[code_e] * a^_b)); the fp32 variant returns
 *    fp32(level * a^) unrounded;
 *  - GEMMs: Y = X W^T and dX = dY W^ with bf16 operands, fp32 accumulation
 *    and fp32 (or, on request, bf16-rounded) outputs; W^ is formed on chip.
 *
 * Conventions for every call:
 *  - Device pointers point to memory of the current HIP device; every device
 *    pointer must be 16-byte aligned (NF4_ERR_ALIGN otherwise).
 *  - The caller owns and frees every buffer.  The library never allocates or
 *    frees device memory and never synchronises; work is queued on `stream`
 *    (a hipStream_t; NULL means the default stream) and outputs are valid once
 *    the stream has reached that point.  No global mutable state.
 *  - Every problem the host can see (NULL pointer, bad size, bad blocksize,
 *    bad dtype enum, misalignment, short workspace, unsupported shape) is
 *    returned before anything is launched, and outputs are left untouched.
 *    A failed launch returns NF4_ERR_HIP.
 *  - Non-finite weights are outside the method's domain (precondition); if
 *    `d_status` is given, the quantizer ORs bit 0 into it when it sees a
 *    non-finite block absmax.
 *  - Dense tensors are row-major and contiguous: X [M,K], Y [M,N],
 *    dY [M,N], dX [M,K], where the weight is [N,K] (nn.Linear's [out,in]).
 */
#ifndef NF4_H_
#define NF4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum nf4_status {
  NF4_OK = 0,
  NF4_ERR_NULL = 1,         /* a required pointer is NULL */
  NF4_ERR_SHAPE = 2,        /* a size is negative, zero where it may not be, or too large */
  NF4_ERR_BLOCKSIZE = 3,    /* blocksize is not 32, 64, 128 or 256 */
  NF4_ERR_DTYPE = 4,        /* unknown nf4_dtype value */
  NF4_ERR_ALIGN = 5,        /* a device pointer is not 16-byte aligned */
  NF4_ERR_WORKSPACE = 6,    /* workspace smaller than nf4_sizes reports */
  NF4_ERR_UNSUPPORTED = 7,  /* valid but not supported, e.g. a GEMM with cols % 64 != 0 */
  NF4_ERR_HIP = 8,          /* a HIP launch failed */
  NF4_ERR_QUANT_TYPE = 9,   /* unknown nf4_quant_type value */
  NF4_ERR_SCRATCH = 10      /* the tensor needs more than the fixed scratch of nf4_quantize_noalloc */
};

enum nf4_dtype {
  NF4_F32 = 0,
  NF4_BF16 = 1
};

/* The 4-bit data type of a quantized weight: its level table. */
enum nf4_quant_type {
  NF4_QT_NF4 = 0,   /* the NF4 levels (default) */
  NF4_QT_FP4 = 1    /* E2M1 values over 6 */
};

/* Largest element count a quantized tensor may hold (2^36; a weight that size
 * is 128 GiB in bf16, and its block count fits 32 bits at every block size). */
#define NF4_MAX_NUMEL ((int64_t)1 << 36)
/* The GEMMs take weights with fewer columns than this (32-bit tile offsets). */
#define NF4_GEMM_COLS_LIMIT ((int64_t)1 << 24)
/* Weights per absmax block: the default (and the workloads' size) is 64;
 * 32, 128 and 256 are accepted as well (any power of two in that range). */
#define NF4_BLOCKSIZE 64
#define NF4_BLOCKSIZE_MIN 32
#define NF4_BLOCKSIZE_MAX 256
/* Absmax values per double-quantization group. */
#define NF4_DQ_GROUP 256
/* Low-rank adapter ranks: a multiple of this step, at most the maximum. */
#define NF4_LORA_RANK_STEP 16
#define NF4_LORA_MAX_RANK 1024

/*
 * A quantized weight: host struct, device buffers (the QuantState analogue).
 * Blocks run over the row-major flattening: block b holds elements
 * b*blocksize .. b*blocksize + blocksize - 1 (it may span rows when blocksize
 * does not divide cols; the last one may be partial).  Sizes for rows x cols
 * (numel = rows*cols, nblocks = ceil(numel/blocksize), ngroups =
 * ceil(nblocks/256)):
 *   packed        ceil(numel/2) bytes
 *   absmax        nblocks fp32     (double_quant == 0; NULL otherwise)
 *   absmax_q      nblocks int8     (double_quant == 1)
 *   absmax_scale  ngroups fp32     (double_quant == 1)
 *   absmax_mean   1 fp32           (double_quant == 1)
 * quant_type (an nf4_quant_type) names the level table; every call that
 * reads the struct rejects other values with NF4_ERR_QUANT_TYPE.  It is the
 * last field so that a zero-initialised tail means NF4.
 * The struct is read during a call only; the library keeps no pointer to it.
 */
typedef struct nf4_qtensor {
  int64_t rows;
  int64_t cols;
  int32_t blocksize;
  int32_t double_quant;
  uint8_t *packed;
  float *absmax;
  int8_t *absmax_q;
  float *absmax_scale;
  float *absmax_mean;
  int32_t quant_type;
} nf4_qtensor;

/* A short English description of a status code (static storage). */
const char *nf4_status_string(int status);

/*
 * Copies the 16 NF4 levels, ascending (level 0 = -1, level 7 = 0,
 * level 15 = +1), into host memory `levels16`.  Source: "bitsandbytes" page,
 * NF4 data-type paragraph (levels from the inverse normal CDF); construction:
 * QLoRA's 8 positive / 7 negative normal quantiles with offset 0.9677083,
 * normalised by the largest, rounded once to fp32.
 */
int nf4_codebook(float *levels16);

/*
 * Copies the 16 levels of `quant_type` (an nf4_quant_type), indexed by code,
 * into host memory `levels16`: NF4 as nf4_codebook; FP4 c[0] = +0 .. c[7] = 1
 * and c[8 + i] = -c[i].  Errors: NF4_ERR_NULL, NF4_ERR_QUANT_TYPE.
 */
int nf4_levels(int quant_type, float *levels16);

/*
 * Copies into host memory `thresholds15` the 15 decision thresholds the
 * quantizer uses: t_i is the smallest fp32 n that codes to i+1, so that
 * code(n) = #{i : n >= t_i} equals the nearest level with ties to the lower
 * index.  Exposed so the derivation can be checked against an independent
 * nearest-level search.
 */
int nf4_thresholds(float *thresholds15);

/*
 * Buffer sizes for a rows x cols weight.  Any output pointer may be NULL.
 * workspace_bytes is the device workspace nf4_quantize needs (0 without
 * double quantization).  Errors: NF4_ERR_SHAPE (rows or cols < 1, or
 * numel > NF4_MAX_NUMEL), NF4_ERR_BLOCKSIZE.
 */
int nf4_sizes(int64_t rows, int64_t cols, int blocksize, int double_quant,
              int64_t *packed_bytes, int64_t *nblocks, int64_t *ngroups,
              size_t *workspace_bytes);

/*
 * Quantizes W (device, [rows, cols] row-major, dtype w_dtype = NF4_F32 or
 * NF4_BF16) into `out`, whose rows/cols/blocksize/double_quant must match the
 * arguments and whose buffers are sized per nf4_sizes; out->quant_type picks
 * the level table (NF4 or FP4).  "Zenbit" page,
 * zenbit.nf4 bullet; "bitsandbytes" page, NF4 and double-quantization
 * paragraphs.  `workspace` (device, >= workspace_bytes from nf4_sizes, may be
 * NULL when that is 0) is scratch for the fp32 absmax and the exact-mean
 * accumulators; its contents on entry do not matter.  `d_status` (device
 * uint32, may be NULL): bit 0 is ORed in if a block absmax is non-finite.
 * Bit-exact and deterministic: the mean is formed from integer sums, so the
 * result does not depend on launch order.
 */
int nf4_quantize(const void *W, int w_dtype, int64_t rows, int64_t cols,
                 int blocksize, int double_quant, const nf4_qtensor *out,
                 void *workspace, size_t workspace_bytes, uint32_t *d_status,
                 void *stream);

/*
 * nf4_quantize without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation).  Same arguments, results and errors as
 * nf4_quantize; the double-quantization scratch (exact-mean rows and the fp32
 * absmax of every block) lives in a fixed buffer inside the library, one per
 * GPU, sized for NF4_NOALLOC_MAX_BLOCKS blocks (about 16.3 MiB), held until
 * the process ends.  A tensor with more blocks, with double_quant set, is
 * refused with NF4_ERR_SCRATCH before anything is launched; without double
 * quantization no scratch is used and every size nf4_quantize takes is
 * accepted.  Calls no allocating routine.  The buffer is shared by every call
 * on a GPU and keeps the last call's contents (the kernels overwrite every
 * byte they later read, so nothing needs clearing between calls); calls whose
 * execution overlaps on one GPU (different streams, different threads) race
 * on it and must be serialised by the caller.  The first call on each device
 * looks the buffer's device address up (thread-safe); NF4_ERR_HIP if that
 * fails.
 */
#define NF4_NOALLOC_MAX_BLOCKS ((int64_t)1 << 22)
int nf4_quantize_noalloc(const void *W, int w_dtype, int64_t rows, int64_t cols,
                         int blocksize, int double_quant, const nf4_qtensor *out,
                         uint32_t *d_status, void *stream);

/*
 * Writes the dequantized weight W^ (device, [rows, cols] row-major) in
 * out_dtype: NF4_BF16 gives bf16_rne(level * a^) (the operand the GEMMs
 * use), NF4_F32 gives fp32(level * a^).  "bitsandbytes" page,
 * double-quantization paragraph: absmax first, then the weights.
 */
int nf4_dequantize(const nf4_qtensor *q, void *out, int out_dtype, void *stream);

/*
 * Y = X W^T.  X: device bf16 [M, K] with K = q->cols; Y: device [M, N] with
 * N = q->rows, in y_dtype (NF4_F32, or NF4_BF16 = one rounding of the fp32
 * accumulator).  W^ is dequantized on chip to bf16 and never written to
 * memory.  Requires K % 64 == 0 and K < NF4_GEMM_COLS_LIMIT
 * (NF4_ERR_UNSUPPORTED otherwise).  M == 0 is a successful no-op.  "Zenbit" page, zenbit.pallas_nf4 bullet (fused
 * forward); "bitsandbytes" page, quantized-GEMM paragraph (fp32 output).
 */
int nf4_matmul_fwd(const void *X, int64_t M, const nf4_qtensor *q, void *Y,
                   int y_dtype, void *stream);

/*
 * dX = dY W^ (the backward pass with respect to the input of Y = X W^T; no
 * gradient for the frozen weight).  dY: device bf16 [M, N] with N = q->rows;
 * dX: device [M, K] with K = q->cols, in dx_dtype (NF4_F32 or NF4_BF16).
 * Requires K % 64 == 0 and K < NF4_GEMM_COLS_LIMIT (NF4_ERR_UNSUPPORTED
 * otherwise).  M == 0 is a successful no-op.  "Zenbit" page,
 * zenbit.pallas_nf4 bullet (fused backward, dL/dX only).
 */
int nf4_matmul_bwd_dx(const void *dY, int64_t M, const nf4_qtensor *q, void *dX,
                      int dx_dtype, void *stream);

/*
 * Y = X W^T + U B^T: the fused forward with a low-rank adapter term added in
 * the same fp32 accumulators before the single store.  "bitsandbytes" page,
 * 4-bit/LoRA paragraph (frozen 4-bit base weight plus small trainable
 * adapters); "Zenbit" page, NF4DenseFused.  For an adapter with down
 * projection A [r, K] and up projection B [N, r] (nn.Linear layouts), U is the
 * down-projected activation X A^T.  U: device bf16 [M, r]; B: device bf16
 * [N, r] with N = q->rows (any adapter scaling folded in); both row-major.
 * X, Y, y_dtype and the shape rules as nf4_matmul_fwd.  r must be a multiple
 * of NF4_LORA_RANK_STEP in [NF4_LORA_RANK_STEP, NF4_LORA_MAX_RANK]
 * (NF4_ERR_UNSUPPORTED otherwise); U and B must be 16-byte aligned.  The
 * adapter product runs on the same bf16 matrix cores with fp32 accumulation.
 */
int nf4_matmul_fwd_lora(const void *X, int64_t M, const nf4_qtensor *q,
                        const void *U, const void *B, int64_t r, void *Y,
                        int y_dtype, void *stream);

/*
 * dX = dY W^ + V A: the fused backward with respect to the input, with the
 * adapter's contribution added in the same accumulators.  For the adapter of
 * nf4_matmul_fwd_lora, V = dY B (device bf16 [M, r]) and At = A^T (device
 * bf16 [K, r] with K = q->cols), both row-major.  dY, dX, dx_dtype and the
 * shape rules as nf4_matmul_bwd_dx; r as nf4_matmul_fwd_lora.  The
 * adapter's own products (U, V and its gradients) are nf4_adapter_matmul.
 */
int nf4_matmul_bwd_dx_lora(const void *dY, int64_t M, const nf4_qtensor *q,
                           const void *V, const void *At, int64_t r, void *dX,
                           int dx_dtype, void *stream);

/*
 * C = alpha op(A) op(B): the dense products of a low-rank adapter on the
 * frozen 4-bit weight ("bitsandbytes" page, 4-bit/LoRA paragraph: a frozen
 * 4-bit base weight with small trainable adapters).  For an adapter with down
 * projection Ad [r, K] and up projection Bu [N, r] (scale s) on input X [M, K]
 * and output gradient dY [M, N]:
 *   U  = s X Ad^T  (trans_a 0, trans_b 1)   the activation nf4_matmul_fwd_lora adds
 *   V  = s dY Bu   (trans_a 0, trans_b 0)   the activation nf4_matmul_bwd_dx_lora adds
 *   dAd = V^T X    (trans_a 1, trans_b 0)   gradient of the down projection
 *   dBu = dY^T U   (trans_a 1, trans_b 0)   gradient of the up projection
 * op(A) is [M, K]: A (trans_a = 0, stored [M, K]) or A^T (trans_a = 1, stored
 * [K, M]); op(B) is [K, N]: B (trans_b = 0, stored [K, N]) or B^T (trans_b =
 * 1, stored [N, K]).  A and B are device bf16, row-major with row strides lda
 * and ldb elements (at least the stored row length); C is device [M, N] with
 * row stride ldc >= N in c_dtype: NF4_F32, or NF4_BF16 = one round-to-nearest-
 * even rounding of the fp32 value.  Products accumulate in fp32 on the bf16
 * matrix cores; alpha multiplies the fp32 sum once.  M or N == 0 is a
 * successful no-op; K >= 1.  Errors: NF4_ERR_UNSUPPORTED (trans flag not 0 or
 * 1, a stored operand of 2^31 bytes or more), NF4_ERR_SHAPE (negative size,
 * K < 1, a stride shorter than its row), NF4_ERR_DTYPE, NF4_ERR_NULL,
 * NF4_ERR_ALIGN (A, B and C 16-byte aligned).
 */
int nf4_adapter_matmul(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K,
                       float alpha, const void *A, int64_t lda, const void *B,
                       int64_t ldb, void *C, int c_dtype, int64_t ldc, void *stream);

/* ------------------------------------------------------------------------
 * Operators around the frozen linear layers of a training or serving step:
 * an 8-bit weight and activation format with its matrix product, the RMS norm
 * that feeds it, and the AdamW step of what is trained beside the frozen
 * weights ("bitsandbytes" page, 4-bit/LoRA paragraph: small trainable adapters;
 * its 8-bit optimizers).  The conventions above hold: device pointers 16-byte
 * aligned, caller-owned buffers, work queued on `stream`, every visible error
 * returned before a launch.  Matrices described as having a leading dimension
 * have contiguous rows, `ld` elements apart (ld >= the row's length).
 * ------------------------------------------------------------------------ */

enum nf4_fp8_format {
  NF4_E4M3 = 0,   /* 4 exponent bits, 3 mantissa bits, largest value 448 */
  NF4_E5M2 = 1    /* 5 exponent bits, 2 mantissa bits, largest value 57344 */
};

/* Columns (and, for weights, rows) per scale of an 8-bit tensor. */
#define NF4_FP8_BLOCK 128

/*
 * An 8-bit tensor [rows, cols]: host struct, device buffers.  Element (r, c)
 * is data[r * pitch + c] (an 8-bit float of `format`) times
 * scale[(r / block_rows) * spitch + c / 128].  pitch is cols rounded up to 128
 * bytes, spitch is pitch / 128 rounded up to 4; data past cols and scales past
 * pitch / 128 are zeros (the quantizers write them; a caller that lays data
 * out itself must too).  block_rows is 1 (activations) or 128 (weights).
 */
typedef struct nf4_fp8_tensor {
  int64_t rows;
  int64_t cols;
  int32_t block_rows;
  int32_t format;        /* an nf4_fp8_format */
  uint8_t *data;         /* rows x pitch */
  float *scale;          /* ceil(rows / block_rows) x spitch */
} nf4_fp8_tensor;

/*
 * Buffer sizes of an 8-bit tensor.  Any output pointer may be NULL.  Errors:
 * NF4_ERR_SHAPE (rows < 0, cols < 1, or too large: cols must stay below
 * NF4_GEMM_COLS_LIMIT), NF4_ERR_BLOCKSIZE (block_rows not 1 or 128).
 */
int nf4_fp8_sizes(int64_t rows, int64_t cols, int block_rows, int64_t *pitch, int64_t *scale_rows,
                  int64_t *spitch);

/*
 * Quantizes x (device, [rows, cols], x_dtype, leading dimension ldx) into
 * `out` of the same shape.  Per block: amax = max|x|, scale = fp32(amax fp32(1 /
 * top)), factor = fp32(fp32(1 / amax) top), code = nearest-even 8-bit float of
 * fp32(x factor), top the format's largest value.  A block with amax below 2^-100 is held as
 * zeros.  A NaN becomes the NaN code; an infinity makes its block's scale
 * infinite, so that the whole block reads back as NaN.  rows == 0 is a no-op.
 */
int nf4_fp8_quantize(const void *x, int x_dtype, int64_t ldx, const nf4_fp8_tensor *out, void *stream);

/*
 * Y = X W^T: X an 8-bit tensor with block_rows 1 [M, K] in either format, W one
 * with block_rows 128 [N, K] in e4m3; Y device [M, N] in y_dtype.  Each
 * block of 128 products is summed in fp32, multiplied by the two scales' fp32
 * product and added in fp32; Y is rounded once.  (A product of scales below
 * 2^-126 is a subnormal number: its rounding is worth at most 2^-125 of Y a
 * block, 2^-118 with an e5m2 X.  One of 2^128 or more makes the block an infinity, or a NaN where its
 * sum is zero.)  A bf16 Y is formed on the fp8
 * matrix cores, which keep 13 bits below the largest of the products they add
 * at once (about 1e-5 of a block's sum); an fp32 Y on the bf16 matrix cores,
 * with every product and sum in fp32.  Any
 * M, N, K (K below NF4_GEMM_COLS_LIMIT, N below 2^26).  M == 0 or
 * N == 0 is a no-op.  Errors: NF4_ERR_NULL, NF4_ERR_SHAPE (K differs),
 * NF4_ERR_BLOCKSIZE, NF4_ERR_UNSUPPORTED (W not in e4m3; too many tiles),
 * NF4_ERR_DTYPE, NF4_ERR_ALIGN.
 */
int nf4_fp8_matmul(const nf4_fp8_tensor *x, const nf4_fp8_tensor *w, void *Y, int y_dtype, void *stream);

/*
 * RMS norm with the residual's addition.  x, and res if not NULL, are device
 * [rows, cols] in x_dtype (leading dimensions ldx, ldr); w is device [cols] in
 * w_dtype.  h = x + res rounded once to x_dtype (h = x without res), rstd =
 * 1 / sqrt(mean(h^2) + eps), y = h rstd w, all in fp32.  Outputs: h [rows, cols]
 * (required with res, unused without), rstd fp32 [rows], and either y [rows,
 * cols] in y_dtype or, with yq not NULL (block_rows 1, e4m3; y must then be
 * NULL), y quantized as by nf4_fp8_quantize from its fp32 values.  eps >= 0.
 * rows == 0 is a no-op.
 */
int nf4_rmsnorm_fwd(const void *x, int x_dtype, int64_t ldx, const void *res, int64_t ldr, const void *w,
                    int w_dtype, int64_t rows, int64_t cols, float eps, void *h, void *y, int y_dtype,
                    const nf4_fp8_tensor *yq, float *rstd, void *stream);

/*
 * Gradient of nf4_rmsnorm_fwd: with g = dy w, dx = rstd (g - h rstd^2 mean(g h))
 * + dh and dw = sum over rows of dy h rstd.  dy [rows, cols] in dy_dtype; h and
 * the optional dh (the gradient that reaches h along the residual stream) in
 * h_dtype; dx [rows, cols] in h_dtype is the gradient of x and of res; dw [cols]
 * in w_dtype, summed in fp32 in a fixed order.  `workspace`: at least
 * nf4_rmsnorm_bwd_workspace bytes (NULL when that is 0); its contents on entry
 * do not matter.  rows == 0 writes zeros to dw.
 */
int nf4_rmsnorm_bwd_workspace(int64_t rows, int64_t cols, size_t *bytes);
int nf4_rmsnorm_bwd(const void *dy, int dy_dtype, int64_t lddy, const void *h, int h_dtype, int64_t ldh,
                    const void *w, int w_dtype, const float *rstd, const void *dh, int64_t lddh, int64_t rows,
                    int64_t cols, void *dx, void *dw, void *workspace, size_t workspace_bytes, void *stream);

/* Elements per scale of an 8-bit optimizer state, and the largest tensor. */
#define NF4_ADAM_BLOCK 256
#define NF4_ADAM_MAX_NUMEL ((int64_t)1 << 34)

/*
 * One tensor of an AdamW step: n elements of parameter and gradient and their
 * two moments (device).  fp32 states: exp_avg and exp_avg_sq are fp32 [n] and
 * the scales are not read.  8-bit states: n rounded up to 256 e4m3 codes each (zeros
 * past n) with one fp32 scale per 256; exp_avg_sq holds the square root.
 */
typedef struct nf4_adamw_tensor {
  void *param;
  const void *grad;
  void *exp_avg;
  void *exp_avg_sq;
  float *exp_avg_scale;
  float *exp_avg_sq_scale;
  int64_t n;
} nf4_adamw_tensor;

typedef struct nf4_adamw_config {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;              /* 1 for the first step */
  const float *grad_scale;   /* device scalar that multiplies every gradient, or NULL */
  uint32_t seed;             /* of the random rounding of 8-bit states: another one each step */
  int32_t state_bits;        /* 32 or 8 */
  int32_t param_dtype;       /* nf4_dtype of every param */
  int32_t grad_dtype;        /* nf4_dtype of every grad */
  const void *layout;        /* device copy of what nf4_adamw_layout wrote, or NULL */
} nf4_adamw_config;

/*
 * The layout of a state whose tensors lie one after another in flat buffers,
 * each at a multiple of NF4_ADAM_BLOCK elements (and 8-bit scales likewise, one
 * per block): with it many tensors take fewer launches.  nf4_adamw_layout
 * writes it to `out` (host, 8-byte aligned, nf4_adamw_layout_bytes of it) for
 * tensors of n[0 .. count) elements; it depends on the sizes only.  The caller
 * copies it to 8-byte aligned device memory once.  Errors: NF4_ERR_NULL,
 * NF4_ERR_SHAPE, NF4_ERR_ALIGN, NF4_ERR_WORKSPACE (`bytes` too small).
 */
int nf4_adamw_layout_bytes(const int64_t *n, int64_t count, size_t *bytes);
int nf4_adamw_layout(const int64_t *n, int64_t count, void *out, size_t bytes);

/*
 * g = grad grad_scale; m = b1 m + (1 - b1) g; v = b2 v + (1 - b2) g^2;
 * p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps) in
 * fp32, p rounded once to its type.  8-bit states are rounded to one of the two
 * neighbouring codes by 16 random bits per value: with mix(x) = { x ^= x >> 16;
 * x *= 0x983B6369; x ^= x >> 15; x *= 0xC1F49415; x ^= x >> 16 } and the key
 * mix(number of the tensor + seed), element i takes mix(i + key) (for
 * i >= 2^32 the key is mix(key + (i >> 32) 0x11D5D725)), the low half for the
 * first moment, the high half for the second.  A root that is not zero takes at
 * least the smallest code (2^-9 of the scale): a step never divides a moment by
 * a root that rounding took away.  Non-finite moments become NaN
 * codes and do not enter their block's scale.  `tensors` (host, `count`
 * entries) is read during the call only; entries with n == 0 are passed over.
 * Tensors must not overlap.  With config->layout the states of all `count`
 * entries must lie as it says, and the layout be that of their sizes.  Errors:
 * NF4_ERR_NULL, NF4_ERR_SHAPE (n out of range, step < 1, states that do not
 * lie flat), NF4_ERR_DTYPE, NF4_ERR_ALIGN, NF4_ERR_UNSUPPORTED
 * (state_bits; a hyperparameter that is not finite or out of range: lr, eps or
 * weight_decay negative, betas outside [0, 1)).
 */
int nf4_adamw_step(const nf4_adamw_tensor *tensors, int64_t count, const nf4_adamw_config *config, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_H_ */
