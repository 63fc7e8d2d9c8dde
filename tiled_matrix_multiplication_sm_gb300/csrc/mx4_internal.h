// Internal interface of the 4-bit operators: the matrix layout, number
// formats and output rule that their kernels share. The public contract is in
// include/tgemm_mx4.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/tgemm_mx4.h"
#include "tgemm_internal.h"

namespace tgemm {

constexpr int MX4_SPAN = 256;            // columns covered by whole scale tiles
constexpr int MX4_TILE_ROWS = 128;       // rows of a scale tile
constexpr int MX4_TILE_BYTES = 512;      // 128 rows x 4 blocks

__host__ __device__ constexpr int mx4_block(int fmt) { return fmt == TGEMM_MXFP4 ? 32 : 16; }
// Scale tiles along a row of `cols` columns.
__host__ __device__ constexpr long mx4_tiles_k(int cols, int fmt) {
    return ((long)cols + MX4_SPAN - 1) / MX4_SPAN * (MX4_SPAN / mx4_block(fmt) / 4);
}
__host__ __device__ constexpr long mx4_pitch(int cols) { return ((long)cols + 31) / 32 * 16; }
__host__ __device__ constexpr size_t mx4_scale_bytes(int rows, int cols, int fmt) {
    return (size_t)(((long)rows + MX4_TILE_ROWS - 1) / MX4_TILE_ROWS) * mx4_tiles_k(cols, fmt) *
           MX4_TILE_BYTES;
}
// Offset of the scale of row r, block b; tiles_k tiles along a row.
__host__ __device__ constexpr size_t mx4_scale_at(long r, long b, long tiles_k) {
    return (size_t)(r / 128 * tiles_k + b / 4) * MX4_TILE_BYTES + (size_t)(r % 32 * 16) +
           (size_t)(r % 128 / 32 * 4) + (size_t)(b % 4);
}

// The tensor cores cut what does not fit into an FP32 sum off at every step of
// K, always towards zero: over 14336 columns BF16 products lose 8e-6 of the
// result's norm, four times what an FP32 library product does; products of
// two 4-bit matrices, whose steps are four times as long, nothing while all terms
// are multiples of 2^-24 of the sum, but 5.5e-6 with NVFP4 scales over 16
// octaves and 2.5e-5 over 65536 columns. So where C keeps 32 bits, a sum of more
// than SUM_STEPS steps is made of sums over SUM_STEPS, added with rounding to
// nearest. (A BF16 C rounds by 2e-3 itself.)
constexpr int SUM_STEPS = 64;
constexpr int SUM_K = 16 * SUM_STEPS;                 // of BF16 products

// A 4-bit operand of a product.
struct Mx4Operand {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* g;       // device; nullptr: 1
};

// Output of a product: C = acc * ga * gb * alpha + beta * C_old + bias[col].
struct Mx4Out {
    void* C;
    long ldc;
    int c_type;           // TGEMM_TYPE_*
    float alpha, beta;
    const float* bias;
};

#ifdef __CUDACC__
// E8M0: 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}
// E4M3 without its sign: 4 bits of exponent (bias 7), 3 of mantissa; 0x7F is NaN.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const float v = (byte & 0x78) ? __uint_as_float(((byte >> 3) + 120) << 23 | (byte & 7) << 20)
                                  : (float)byte * 0.001953125f;
    return byte == 0x7F ? __uint_as_float(0x7FC00000u) : v;
}
template <int FMT>
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
    return FMT == TGEMM_MXFP4 ? e8m0_value(byte) : e4m3_value(byte & 0x7F);
}
// E2M1 code (4 bits) to FP32.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7;
    const float v = m < 2 ? 0.5f * (float)m : __uint_as_float((m >> 1) + 126 << 23 | (m & 1) << 22);
    return (c & 8) ? -v : v;
}

// (Operands are read by plain loads: the read-only path takes what nothing writes
// while a kernel runs, and with programmatic dependent launch a kernel runs
// while the one before it still writes them. Nor may such loads move above
// pdl_wait, as read-only ones may.)
__device__ __forceinline__ float mx4_g(const float* g) { return g != nullptr ? *g : 1.0f; }

// One output under the rule; C_old is read only when beta != 0.
template <typename T>
__device__ __forceinline__ void mx4_store(T* c, float acc, float ga, float gb, const Mx4Out& o,
                                          int col) {
    float v = acc * ga * gb * o.alpha;
    if (o.beta != 0.0f) v = fmaf(o.beta, (float)*c, v);
    if (o.bias != nullptr) v += o.bias[col];
    *c = (T)v;
}
#endif

// ---- quantising (mx4_quantize.cu)
cudaError_t mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type, float* g,
                             int num_sms, cudaStream_t s);
cudaError_t mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                         const float* g, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                         uint8_t* scales_t, int num_sms, cudaStream_t s);
cudaError_t mx4_dequantize(int rows, int cols, const uint8_t* codes, const uint8_t* scales,
                           int fmt, const float* g, void* X, long ldx, int x_type, cudaStream_t s);
cudaError_t mx4_pack(int rows, int cols, int fmt, const uint8_t* src_codes, long src_ldc,
                     const uint8_t* src_scales, long src_lds, uint8_t* codes, uint8_t* scales,
                     cudaStream_t s);

// ---- products (mx4_gemm.cu, mx4_weights.cu)
cudaError_t mx4_gemm(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, int fmt,
                     const Mx4Out& out, int num_sms, cudaStream_t s);
// The K == 0 product: C = beta * C_old + bias.
cudaError_t mx4_empty_sum(int M, int N, const Mx4Out& out, cudaStream_t s);
// The device address of these kernels' status word on the current device.
cudaError_t mx4_status_word(int** word);
cudaError_t mx4_read_and_clear_status(int* status, cudaStream_t s);
cudaError_t mx4_weights(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt,
                        const Mx4Out& out, int num_sms, cudaStream_t s);

// At most MX4_FEW_ROWS rows of A (mx4_weights_rows.cu): all products with up to
// 8, and small ones with more, where its shorter start counts. There, and in
// mx4_weights_tmem.cu (us, BF16 C):
//     MXFP4   8 x 1024 x 1024    2.4   4.3      NVFP4   9 x 1024 x 4096    5.3   5.5
//             8 x 4096 x 14336  13.3  15.0             24 x 1024 x 4096    6.0   5.7
//             8 x 65536 x 4096  48.9  59.6             16 x 4096 x 4096    7.3   7.3
//            24 x 1024 x 1024    4.0   4.5             24 x 4096 x 4096    9.0   7.7
//            16 x 14336 x 4096  14.6  15.2             16 x 14336 x 4096  16.1  14.8
//            24 x 14336 x 4096  22.9  15.5             16 x 65536 x 4096  66.2  59.0
constexpr int MX4_FEW_ROWS = 24;
inline bool mx4_few_rows(int M, int N, int K) { return M <= 8 || (M <= MX4_FEW_ROWS && (long)N * K < 1L << 24); }
cudaError_t mx4_weights_rows(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt,
                             const Mx4Out& out, int num_sms, cudaStream_t s);

// C of few tiles (mx4_weights_tmem.cu); X's rows on 16-byte boundaries.
cudaError_t mx4_weights_tmem(int M, int N, int K, const void* X, long ldx, const Mx4Operand& W, int fmt,
                             const Mx4Out& out, cudaStream_t s);

}  // namespace tgemm
