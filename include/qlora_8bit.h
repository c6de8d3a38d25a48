/*
 * qlora_8bit.h -- C ABI of the 8-bit operators beside the NF4 layer of
 * qlora.h, in the same library: a matrix in 8-bit floating point with a scale
 * for each block of 128, the product of two such matrices, and an AdamW step
 * over many tensors at once with moments in 32 or 8 bits.
 *
 * Together they train or serve a linear layer whose weight W [N, K] is held
 * in 8 bits (tokens x [M, K]):
 *     y  = fp8_matmul(x, W)             x in rows, W in 128 x 128 tiles
 *     dx = fp8_matmul(dy, W transposed) dy in rows
 *     dW = fp8_matmul(dy transposed, x transposed), added into fp32
 * where fp8_quantize gives a matrix and its transpose from one reading of the
 * input, and ql_adamw_step_many updates the master weights (or the adapters)
 * from the gradients.
 *
 * Conventions, status codes and element types are those of qlora.h: device
 * pointers, a hipStream_t passed as void *, nothing allocated, kept or
 * synchronised, every argument checked on the host before anything is
 * enqueued.  Unlike there, infinities and NaN have defined results here.
 */
#ifndef QLORA_8BIT_H
#define QLORA_8BIT_H

#include "qlora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit floating-point formats: sign, exponent and mantissa bits 1-4-3
 * (largest value 448, smallest 2^-9; no infinity, NaN is 0x7F / 0xFF) and
 * 1-5-2 (largest value 57344, smallest 2^-16). */
#define QL_E4M3 3
#define QL_E5M2 4

/* Values that share a scale: 128 of a row (or a 128 x 128 tile) of a matrix,
 * 256 consecutive ones of a tensor's moments. */
#define QL_FP8_BLOCK 128
#define QL_STATE_BLOCK 256

/*
 * A matrix [rows, cols] in 8-bit floating point.  ld = cols rounded up to a
 * multiple of 128, rp = rows rounded up to a multiple of 16.
 *
 *  codes   uint8 [rows][ld] in `format`; bytes cols .. ld - 1 of a row are 0.
 *  scales  uint8 [ld / 128][rp]: scales[b][i] belongs to elements 128 b ..
 *          128 b + 127 of row i.  A byte s stands for 2^(s - 127); 255 makes
 *          the whole block NaN.  Bytes rows .. rp - 1 are never used.
 *
 * Element (i, j) is  codes[i][j] * 2^(scales[j / 128][i] - 127).  Scales are
 * powers of two because the matrix cores apply those themselves, for every
 * 32 products; the codes lose nothing by it (they are floating-point values)
 * except in the lowest octave of the format.  A weight in 128 x 128 tiles
 * holds one value 128 times: 1/128 of a byte per element buys one layout.
 * Both pointers 16-byte aligned; the struct itself lives in host memory.
 */
typedef struct ql_fp8 {
  uint8_t *codes;
  uint8_t *scales;
  int64_t rows;
  int64_t cols;
  int32_t format;   /* QL_E4M3 or QL_E5M2 */
  int32_t reserved; /* must be 0 */
} ql_fp8;

/* Host only.  bytes_out[0..1] = bytes of codes and scales of a rows x cols
 * matrix.  Returns QL_OK or QL_EINVAL (sizes below 1 or above 2^31 - 256). */
int ql_fp8_sizes(int64_t rows, int64_t cols, size_t bytes_out[2]);

/*
 * Quantise x [R, C] (row-major, densely packed, x_dtype QL_F32, QL_BF16 or
 * QL_F16), and its transpose, in one launch that reads x once.
 *   block_rows  1: one scale per 128 elements of a row (activations,
 *               gradients); 128: one per 128 x 128 tile (weights)
 *   q           receives x:   rows = R, cols = C; or NULL
 *   qt          receives x^T: rows = C, cols = R; or NULL (not both NULL)
 * Each takes its own format.  With block_rows 128 the two hold the same
 * values (the tiles are the same ones) if the formats are equal; with 1, qt's
 * scales are those of 128 consecutive rows of x in one column.
 *   scale  the smallest 2^e, -127 <= e, with  max |block| <= top 2^e,
 *          top = 448 (E4M3) or 57344 (E5M2); a block of zeros has e = -127
 *   code   x 2^-e rounded to the nearest value, ties to even
 * A block that holds a NaN or an infinity has scale byte 255, as far as that
 * block reaches.  Padding bytes of codes and scales are written as 0.
 * Errors: QL_EINVAL (null pointers, sizes, dtype, block_rows, format,
 * reserved, x, q and qt sharing memory), QL_ESHAPE (q and qt do not describe x
 * and its transpose), QL_EUNSUPPORTED (2^24 tiles of 128 x 128 or more),
 * QL_EALIGN (x, codes, scales: 16 bytes), QL_EHIP.
 */
int fp8_quantize(const void *x, int32_t x_dtype, int32_t block_rows, const ql_fp8 *q,
                 const ql_fp8 *qt, void *stream);

/* Host only.  Workspace bytes of fp8_matmul for a [M, K] and b [N, K], any
 * output type (a multiple of 256, may be 0); 0 for invalid sizes. */
size_t ql_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * out [M, N] = a b^T over the K blocked elements of both (out += a b^T with
 * accumulate = 1, fp32 only): a [M, K] in either format, b [N, K] in E4M3.
 *   out       device [M, N], out_dtype QL_F32, QL_BF16 or QL_F16, 16-byte
 *             aligned; rounded once (to nearest, ties to even)
 *   ws        device workspace of ql_fp8_workspace_bytes(M, N, K), 256-byte
 *             aligned (NULL with ws_bytes 0 if that is 0).  Calls that can
 *             run at the same time need workspaces of their own.
 * 16-bit outputs multiply the codes on the 8-bit matrix cores, which add 8
 * consecutive products at a time and drop of each what is below 2^-13 of the
 * largest of them, then add in fp32 (measured on normal data: an error of
 * 1.4e-5 of the result's root mean square, 1/140 of a bf16 rounding).  Where
 * that is too much, or terms cancel, take fp32 and round it.
 * fp32 outputs multiply the exact values in bf16 (a code times a power of two
 * is a bf16 value) and accumulate in fp32, at half the rate.  Values below
 * 2^-126 may count as 0 there, and values from 2^128 on are infinite.  The
 * order of all sums is fixed: equal calls give equal bits.
 * Errors: QL_EINVAL (null pointers, sizes, formats, dtype, accumulate, out or
 * ws sharing memory with each other or with a or b), QL_ESHAPE (a and b differ
 * in cols), QL_EUNSUPPORTED (b in E5M2, accumulate into 16 bits, K > 2^22,
 * 2^24 output tiles of 128 x 128 or more), QL_EALIGN, QL_EWORKSPACE, QL_EHIP.
 */
int fp8_matmul(const ql_fp8 *a, const ql_fp8 *b, void *out, int32_t out_dtype, int32_t accumulate,
               void *ws, size_t ws_bytes, void *stream);

/*
 * One tensor of an AdamW step over many: n parameters and what belongs to
 * them, contiguous device arrays.  nb = ceil(n / 256).
 *   param             fp32 [n], updated
 *   grad              [n] of the call's grad_dtype, read
 *   exp_avg           fp32 [n], or E4M3 codes [n], updated
 *   exp_avg_sq        fp32 [n], or E5M2 codes [n], updated
 *   exp_avg_scale     fp32 [nb] (8-bit moments only, else NULL), updated
 *   exp_avg_sq_scale  fp32 [nb] (8-bit moments only, else NULL), updated
 *   copy              [n] of the call's copy_dtype: receives param rounded to
 *                     16 bits, what a layer reads; or NULL
 * Alignment: 16 bytes for fp32 arrays of n, 8 for 16-bit ones, 4 for codes
 * and scales.  n may be 0.
 */
typedef struct ql_adamw_tensor {
  float *param;
  const void *grad;
  void *exp_avg;
  void *exp_avg_sq;
  float *exp_avg_scale;
  float *exp_avg_sq_scale;
  void *copy;
  int64_t n;
} ql_adamw_tensor;

/*
 * One AdamW step over `count` tensors, in place, up to 960 in one launch: for
 * each the update of ql_adamw_step, bit for bit with 32-bit moments and no
 * grad_scale.
 *   t           host array of count structs; no two may share memory.  It is
 *               what is checked, and its n make the grid
 *   t_device    the same array in device memory, byte for byte, n included,
 *               16-byte aligned (uploaded once, it serves every step), left
 *               unchanged until the step is done.  The kernel reads a tensor's
 *               pointers and its n from here; a struct that differs from t's is
 *               not found out, and its tensor is updated in part, or written
 *               past its end
 *   grad_dtype  QL_F32, QL_BF16 or QL_F16
 *   state_bits  32 or 8
 *   copy_dtype  QL_BF16 or QL_F16 (ignored where no tensor has a copy)
 *   grad_scale  device fp32 [1]: every gradient is multiplied by it first
 *               (a clipping factor, the inverse of a loss scale); or NULL
 *   seed        any value: draws the rounding of 8-bit moments
 * 8-bit moments: a block of 256 consecutive values of a tensor is held as
 * codes and a scale S (value = code * S); the moments' arithmetic is fp32, one
 * rounding for each operation, and a parameter's step is within 2^-21 of
 * itself (eps below 2^-126 counts as that, 2^126 or more as infinite).  With
 * the new moments x of a block and big = max |x|, top = 448 (exp_avg) or 57344
 * (exp_avg_sq):
 *     S = big * fp32(1 / top),   t = min(|x| * (top * (1 / big)), top)
 * and t, between the neighbouring codes lo and hi, becomes hi with the
 * probability (t - lo) / (hi - lo), to 16 bits: rounded to the nearest code,
 * a moving average whose steps are smaller than half a code's distance would
 * stand still.  The 16 bits are the low (exp_avg) and high (exp_avg_sq) half
 * of word i % 4 of Philox4x32 (Salmon et al., SC'11) with 7 rounds at counter
 * (i / 4 low word, i / 4 high word, index of the tensor in t, step low word)
 * under the key `seed`, i the element's index.  A value of exp_avg_sq above 0
 * keeps a code above 0 wherever its block keeps any: a block with big < 2^-100
 * becomes zeros with S = 0.  Each moment's block is judged by itself, so that of
 * gradients below 2^-45 or so the second moment can go while the first one
 * stays, which the next gradient's square and eps alone then divide.  What that
 * changes is at most 2^-50 / (eps sqrt(1 - beta2^step)) of a step, below 3e-6 at
 * an eps of 1e-8; under one below 1e-10 such gradients want 32-bit moments.  A
 * block that holds a NaN or infinity becomes NaN as a whole.  The parameters are
 * updated from the moments before these are rounded to 8 bits.
 * Scalars are passed by value: a captured step replays its own lr, step and
 * seed, and only grad_scale is read anew; t_device has to outlive the graph.
 * Errors: QL_EINVAL (count < 0, step < 1, null pointers, dtypes, state_bits,
 * n < 0, hyperparameters as for ql_adamw_step), QL_EUNSUPPORTED (n > 2^33),
 * QL_EALIGN, QL_EHIP.  Every tensor is checked before anything is enqueued.
 */
int ql_adamw_step_many(int32_t count, const ql_adamw_tensor *t, const ql_adamw_tensor *t_device,
                       int32_t grad_dtype, int32_t state_bits, int32_t copy_dtype, const float *grad_scale, double lr,
                       double beta1, double beta2, double eps, double weight_decay, int64_t step,
                       uint64_t seed, void *stream);

/* Host only: version of this header (major * 100 + minor).  The minor version
 * grows whenever an entry point is added or a workspace size changes. */
int ql_8bit_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_8BIT_H */
