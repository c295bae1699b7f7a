/*
 * fp8.h — C ABI of the 8-bit floating point operators of libgptq_b200.so.
 *
 * Beside the integer formats of gptq.h, a linear layer can be held, and multiplied, in e4m3
 * (1 sign, 4 exponent, 3 mantissa bits, bias 7, largest value 448, no infinities) with one fp32
 * scale for each block of 128:
 *   fp8_quantize      a matrix into the format: activations (blocks of 1 x 128) or weights
 *                     (blocks of 128 x 128)
 *   fp8_add_rmsnorm   h = x + r, and the root-mean-square norm of h in the format (1 x 128)
 *   fp8_gemm          Y = X W^T of activations and weights in the format
 *   fp8_gated_gemm    silu(X Wg^T) * (X Wu^T) in the format (1 x 128): the two products of a
 *                     gated feed-forward block, its activation and the quantization in one kernel
 * Run one after the other they are the feed-forward half of a decoder block: norm -> gated pair ->
 * product (down projection) -> the next norm, which adds the residual.
 *
 * The format. value(i, j) = e4m3(i, j) * s(block of (i, j)), the block's scale being
 *   s = fl(amax / 448), amax the largest magnitude in the block;
 *       at least 2^-126 (so that 1 / s is finite), and 1 for a block of zeros;
 *   e4m3 = round-to-nearest-even of y * fl(1 / s), so that the largest value becomes +-448.
 * A block that holds a NaN or an infinity gets the scale NaN and e4m3 NaNs, so that every product
 * with it is NaN. The last block of a row (column) holds what is left when the length is not
 * a multiple of 128.
 *
 * Conventions are those of gptq.h: device pointers owned by the caller, no allocation and no
 * scratch, asynchronous on `stream`, host-side argument errors returned before anything is
 * launched, dev_status (where taken) as described there. Leading dimensions are in elements.
 * m (rows of activations) may be 0: the call then returns GPTQ_OK and writes nothing. Outputs
 * may not overlap inputs or one another, except as stated. Results are bitwise repeatable.
 */
#ifndef GPTQ_B200_FP8_H
#define GPTQ_B200_FP8_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types here: GPTQ_BF16, GPTQ_F32 (gptq.h) and */
enum { GPTQ_F16 = 2 };

/*
 * fp8_quantize — Q, scales = X in the format.
 *
 *   X           [m, ldx] of x_dtype (GPTQ_BF16, GPTQ_F16, GPTQ_F32); ldx >= k
 *   block_rows  1: one scale per row and 128 columns (activations);
 *               128: one per 128 rows and 128 columns (weights)
 *   Q           e4m3 [m, ldq], ldq >= k. Bytes behind column k are not written. For the tensor
 *               cores (fp8_gemm) give Q a 16-byte aligned base and ldq a multiple of 16.
 *   scales      fp32 [ceil(m / block_rows), lds], lds >= ceil(k / 128)
 * Errors: INVALID_ARG for a null pointer, m < 0, k < 1, m or k > 2^30, a short leading dimension,
 * a block_rows other than 1 and 128, a pointer that is not aligned to its element;
 * UNSUPPORTED for another x_dtype.
 */
int fp8_quantize(const void* X, int x_dtype, int64_t ldx, int64_t m, int64_t k, int block_rows,
                 uint8_t* Q, int64_t ldq, float* scales, int64_t lds, gptq_stream_t stream);

/*
 * fp8_add_rmsnorm — the residual's addition, the root-mean-square norm and the quantization:
 *   h = x + r            in fp32 (h = x when R is NULL)
 *   H = h                rounded to dtype (not written when H is NULL)
 *   y = h / sqrt(mean_j(h_j^2) + eps) * gamma      in fp32, in this order, from the unrounded h
 *   Q, scales = y in the format, one scale per row and 128 columns
 *
 *   X, R, H     [m, ld] of `dtype` (GPTQ_BF16, GPTQ_F16, GPTQ_F32). H may be X or R itself (the
 *               same pointer and leading dimension): each element is read before it is written.
 *   gamma       [k] of gamma_dtype: `dtype` or GPTQ_F32
 *   eps         finite, >= 0
 *   Q, scales   as in fp8_quantize with block_rows 1
 * Errors: as fp8_quantize; UNSUPPORTED for another dtype or gamma_dtype. Squares are summed in
 * fp32: a row whose sum of h^2 passes 3.4e38 is divided by infinity, as in the formula in fp32.
 */
int fp8_add_rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, int dtype,
                    const void* gamma, int gamma_dtype, float eps, int64_t m, int64_t k, void* H,
                    int64_t ldh, uint8_t* Q, int64_t ldq, float* scales, int64_t lds,
                    gptq_stream_t stream);

/*
 * fp8_gemm — Y = X W^T of matrices in the format:
 *   Y[i, j] = sum_g sx[i, g] * sw[j / 128, g] * sum_{c in block g} X[i, c] * W[j, c]
 * with exact products, the sum over each block of 128 columns in the tensor core's fp32
 * accumulator and the scaled sums added in fp32; rounded once to y_dtype (a value beyond fp16's
 * range becomes an infinity). sx * sw is formed first, in fp32: beyond 3.4e38 it is an infinity, and
 * below 2^-126 it has fewer bits.
 *
 *   X           e4m3 [m, ldx], sx fp32 [m, ldsx]                (blocks of 1 x 128)
 *   W           e4m3 [n, ldw], sw fp32 [ceil(n / 128), ldsw]    (blocks of 128 x 128)
 *   Y           [m, ldy] of y_dtype (GPTQ_BF16, GPTQ_F16, GPTQ_F32), ldy >= n; written, not added to
 *   dev_status  as in gptq.h: work is skipped while it holds an error; a wait that runs out
 *               records GPTQ_ERR_TIMEOUT (then Y holds no result); may be NULL
 * X and W whose base is 16-byte aligned and whose leading dimension is a multiple of 16 run on
 * the tensor cores. Any other alignment is taken too, by a kernel on the CUDA cores that is
 * about a hundred times slower at large sizes. Bytes behind column k are never used.
 * Errors: INVALID_ARG for a null pointer, m < 0, n < 1, k < 1, sizes > 2^30, a short leading
 * dimension, a misaligned scale or Y pointer; UNSUPPORTED for another y_dtype.
 */
int fp8_gemm(const uint8_t* X, int64_t ldx, const float* sx, int64_t ldsx, const uint8_t* W,
             int64_t ldw, const float* sw, int64_t ldsw, int64_t m, int64_t n, int64_t k, void* Y,
             int y_dtype, int64_t ldy, int32_t* dev_status, gptq_stream_t stream);

/*
 * fp8_gated_gemm — the gated pair of products of a feed-forward block, from the format to the
 * format:
 *   g = X Wg^T, u = X Wu^T (as fp8_gemm, kept in fp32), h = g / (1 + exp(-g)) * u
 *   (the sigmoid in fp32: a subnormal number for g below -87.3, zero below -104)
 *   Q, scales = h in the format, one scale per row and 128 columns
 *
 *   X, sx       as in fp8_gemm
 *   Wg, sg      e4m3 [n, ldwg] and fp32 [ceil(n / 128), ldsg]; Wu, su likewise. They may be the
 *               two halves of one stacked weight.
 *   Q           e4m3 [m, ldq], ldq >= n; scales fp32 [m, lds], lds >= ceil(n / 128)
 * Alignment, dev_status and errors as in fp8_gemm.
 */
int fp8_gated_gemm(const uint8_t* X, int64_t ldx, const float* sx, int64_t ldsx,
                   const uint8_t* Wg, int64_t ldwg, const float* sg, int64_t ldsg,
                   const uint8_t* Wu, int64_t ldwu, const float* su, int64_t ldsu, int64_t m,
                   int64_t n, int64_t k, uint8_t* Q, int64_t ldq, float* scales, int64_t lds,
                   int32_t* dev_status, gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_B200_FP8_H */
