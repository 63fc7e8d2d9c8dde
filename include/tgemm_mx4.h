/*
 * tgemm_mx4 — matrices in 4-bit floating point with block scales: quantising,
 * reading back, and products on one NVIDIA GB300 (sm_103a).
 *
 * Part of libtgemm.so; a C ABI like tgemm.h, with its status codes, its rules
 * on streams, CUDA graphs and threads, and its bounded waits
 * (gemm_device_status). No entry point here draws on the device allocator
 * unless its description says so; all buffers are the caller's.
 *
 * A 4-bit matrix. R rows of C columns, the rows the matrix is quantised
 * along (a product sums over its columns). Each value is
 *
 *     code x scale of its block [x g]
 *
 *   code   an E2M1 number: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
 *          (bits: sign, two of exponent, one of mantissa);
 *   scale  one byte for each block of consecutive columns of a row:
 *            TGEMM_MXFP4  blocks of 32, E8M0: 2^(byte - 127), 255 is NaN
 *            TGEMM_NVFP4  blocks of 16, E4M3 (sign bit 0), 0x7F is NaN
 *   g      TGEMM_NVFP4 only: one FP32 number for the whole matrix, > 0, in
 *          device memory (NULL: 1). The NVFP4 scales span 2^-9 .. 448, so g
 *          brings a matrix into that range. TGEMM_MXFP4 takes NULL.
 *
 * Layout in memory:
 *   codes   rows of gemm_mx4_codes_pitch(C) = 16 ceil(C / 32) bytes, column
 *           2i in the low and 2i + 1 in the high half of byte i; the codes
 *           from column C to the row's end are zero.
 *   scales  tiles of 128 rows x 4 blocks, 512 bytes each, as the tensor core
 *           takes them: tile (r / 128, b / 4) holds the byte of row r and
 *           block b at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4. The tiles
 *           of 128 rows follow each other along the row, and a row of tiles
 *           covers whole spans of 256 columns; gemm_mx4_scales_bytes gives
 *           the size. Bytes of rows and blocks outside the matrix are zero.
 * Both buffers start on 16-byte boundaries (TGEMM_ERR_ALIGNMENT otherwise).
 * gemm_mx4_pack makes this layout from row-major codes and scales. Rows,
 * columns, M, N and K are at most TGEMM_MX4_MAX_DIM
 * (TGEMM_ERR_INVALID_ARG beyond).
 *
 * Quantising a block whose largest magnitude is m:
 *   TGEMM_MXFP4: scale = 2^clamp(floor(log2 m) - 2, -127, 127)
 *   TGEMM_NVFP4: scale = E4M3(m / (6 g)), to nearest even, at most 448
 * and each code is the E2M1 number nearest to x / (scale [x g]), ties to the
 * even code, magnitudes above 6 to 6 (0 when the scale is 0). A block that
 * holds an infinity or a NaN gets a NaN scale: all its values read back as
 * NaN, and a product that uses it gives NaN.
 */
#ifndef TGEMM_MX4_H
#define TGEMM_MX4_H

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of rows or columns: tiles' ends stay in an int. */
#define TGEMM_MX4_MAX_DIM 2147482624

/* Formats of a 4-bit matrix. */
#define TGEMM_MXFP4 1
#define TGEMM_NVFP4 2

/* Element types of the matrices that are not in 4 bits. */
#define TGEMM_TYPE_F32  0
#define TGEMM_TYPE_BF16 1

/* Bytes between the rows of codes of a matrix with `cols` columns (a multiple
 * of 16), or a negative status code. */
TGEMM_API long long gemm_mx4_codes_pitch(int cols);

/* Bytes of the scales of a rows x cols matrix in format `fmt`, or a negative
 * status code. */
TGEMM_API long long gemm_mx4_scales_bytes(int rows, int cols, int fmt);

/*
 * gemm_mx4_tensor_scale — the FP32 scale g of an NVFP4 matrix.
 *
 * Writes to *g (device memory) the smallest power of two, from 2^-100 to
 * 2^117, with 2688 g >= |x| for every finite x of the rows x cols matrix X
 * (2688 = 6 x 448, the largest code times the largest scale); 2^-100 for a
 * matrix of zeros or with no elements. As a power of two it costs the values
 * no rounding of their own. The same g serves X and its transpose.
 *
 * X holds `x_type` elements (TGEMM_TYPE_*), ldx >= cols, any alignment to its
 * element size. Returns TGEMM_OK, TGEMM_ERR_INVALID_ARG, TGEMM_ERR_UNSUPPORTED
 * or TGEMM_ERR_CUDA.
 */
TGEMM_API int gemm_mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type,
                                    float* g, cudaStream_t stream);

/* Flag of gemm_mx4_quantize: write g first, as gemm_mx4_tensor_scale does. */
#define TGEMM_MX4_SET_G 1

/*
 * gemm_mx4_quantize — X (rows x cols, ldx >= cols, TGEMM_TYPE_F32 or _BF16) in
 * 4 bits along its rows (codes, scales: a rows x cols matrix), along its
 * columns (codes_t, scales_t: the cols x rows matrix of its transpose), or
 * both in one reading of X. A pair that is not wanted is NULL, NULL.
 *
 * g: see above; with flags TGEMM_MX4_SET_G (TGEMM_NVFP4 only) it is computed
 * from X and written, otherwise it is read, say one of an earlier step. A g
 * that is not finite or lies outside [2^-100, 2^117] makes every scale NaN.
 * Returns as gemm_mx4_tensor_scale, and TGEMM_ERR_INVALID_ARG for half a
 * pair, no pair, an unknown format or flag, a g with TGEMM_MXFP4 or a flag
 * without one.
 */
TGEMM_API int gemm_mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                                float* g, int flags, void* codes, void* scales, void* codes_t,
                                void* scales_t, cudaStream_t stream);

/*
 * gemm_mx4_dequantize — the values a rows x cols 4-bit matrix stands for, as
 * FP32 or BF16 (code x scale, then x g, rounded once each; BF16 to nearest
 * even), to X (ldx >= cols). Errors as above.
 */
TGEMM_API int gemm_mx4_dequantize(int rows, int cols, const void* codes, const void* scales,
                                  int fmt, const float* g, void* X, long ldx, int x_type,
                                  cudaStream_t stream);

/*
 * gemm_mx4_pack — codes and scales kept row-major (as a checkpoint keeps
 * them) to the layout above. src_codes: rows of at least ceil(cols / 2)
 * bytes, src_ldc bytes apart; src_scales: rows of at least one byte for each
 * block, src_lds bytes apart; neither needs any alignment. A code past the
 * last column in its byte is ignored. Errors as above.
 */
TGEMM_API int gemm_mx4_pack(int rows, int cols, int fmt, const void* src_codes, long src_ldc,
                            const void* src_scales, long src_lds, void* codes, void* scales,
                            cudaStream_t stream);

/*
 * gemm_mx4 — product of two 4-bit matrices of one format on the tensor cores:
 *
 *     C = alpha * A * B^T + beta * C + bias
 *
 * A is M x K and B is N x K, both quantised along K; C is M x N (ldc >= N),
 * TGEMM_TYPE_F32 or _BF16, any alignment to its element size. Products of
 * codes and scales are exact and are summed in FP32: on the tensor cores, which
 * cut low bits off at every step of 64 columns, up to 4096 columns; with an FP32
 * C longer sums are made of such parts, added with rounding to nearest. `bias`
 * is NULL or N floats; C is not read when beta == 0. Each output is
 *     v = acc * ga * gb * alpha;  if (beta != 0) v = fmaf(beta, C_old, v);
 *     v += bias[j]
 * in FP32, rounded once for a BF16 C. K == 0 gives acc = 0; M == 0 or
 * N == 0 is a no-op. C must not overlap an operand.
 *
 * Returns TGEMM_OK, TGEMM_ERR_INVALID_ARG (a negative size, ldc < N, a null
 * pointer, an unknown format or type, a g with TGEMM_MXFP4, C or bias not
 * aligned to its elements), TGEMM_ERR_ALIGNMENT (codes or scales off 16
 * bytes), TGEMM_ERR_UNSUPPORTED or TGEMM_ERR_CUDA.
 */
TGEMM_API int gemm_mx4(int M, int N, int K,
                       const void* a_codes, const void* a_scales, const float* ga,
                       const void* b_codes, const void* b_scales, const float* gb,
                       int fmt, void* C, long ldc, int c_type,
                       float alpha, float beta, const float* bias, cudaStream_t stream);

/*
 * gemm_w4 — the same product with A in BF16 (M x K, lda >= K, any alignment
 * to 2 bytes) and B a kept 4-bit matrix: activations that stay in 16 bits
 * with weights in 4. Products of A with code x scale are exact; they are summed
 * in FP32 (with an FP32 C in parts of 1024 columns, as above) and
 *     v = acc * gb * alpha, then beta and bias as in gemm_mx4.
 * The sums are held times 2^-16 (TGEMM_NVFP4) or 2^-2 (TGEMM_MXFP4), so that
 * terms below 2^-110 or 2^-124 may lose bits. An A whose rows do not start on
 * 16-byte boundaries is copied first, to 2 M round_up(K, 64) bytes of
 * stream-ordered scratch from the library's pool (see tgemm.h), where M > 24,
 * where M > 8 and N K >= 2^24, and where K >= 2^27.
 *
 * Errors as gemm_mx4, and TGEMM_ERR_INVALID_ARG for lda < K or A off 2 bytes.
 */
TGEMM_API int gemm_w4(int M, int N, int K, const void* A, long lda,
                      const void* b_codes, const void* b_scales, const float* gb,
                      int fmt, void* C, long ldc, int c_type,
                      float alpha, float beta, const float* bias, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_MX4_H */
