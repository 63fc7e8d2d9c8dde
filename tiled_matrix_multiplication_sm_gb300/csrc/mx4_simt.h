// Product with a 4-bit B on the CUDA cores: 64 x 64 tiles of C, both operands
// decoded to FP32 in shared memory.
#pragma once

#include "mx4_internal.h"

namespace tgemm {
namespace mx4_simt {

constexpr int BT = 64, BK = 32, THREADS = 256;

template <int FMT>
__device__ __forceinline__ float value_at(const Mx4Operand& m, long r, int k, int K) {
    const uint32_t pair = m.codes[r * mx4_pitch(K) + k / 2];
    const float s = mx4_scale_value<FMT>(m.scales[mx4_scale_at(r, k / mx4_block(FMT), mx4_tiles_k(K, FMT))]);
    return e2m1_value((k & 1) ? pair >> 4 : pair & 15) * s;
}

// A4: A is a 4-bit matrix; otherwise BF16 at `a16`, rows lda apart.
template <int FMT, bool A4, typename TC>
__global__ void __launch_bounds__(THREADS)
product_kernel(int M, int N, int K, Mx4Operand A, const __nv_bfloat16* a16, long lda, Mx4Operand B,
               Mx4Out out) {
    __shared__ float as[BK][BT + 1], bs[BK][BT + 1];
    pdl_launch_dependents();
    pdl_wait();
    const long m0 = (long)blockIdx.y * BT, n0 = (long)blockIdx.x * BT;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += BK) {
        for (int i = threadIdx.x; i < BT * BK; i += THREADS) {
            const int r = i / BK, k = i % BK;
            float a = 0.0f, b = 0.0f;
            if (k0 + k < K) {
                if (m0 + r < M)
                    a = A4 ? value_at<FMT>(A, m0 + r, k0 + k, K) : (float)a16[(m0 + r) * lda + k0 + k];
                if (n0 + r < N) b = value_at<FMT>(B, n0 + r, k0 + k, K);
            }
            as[k][r] = a;
            bs[k][r] = b;
        }
        __syncthreads();
        for (int k = 0; k < BK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    const float ga = A4 ? mx4_g(A.g) : 1.0f, gb = mx4_g(B.g);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long r = m0 + ty * 4 + i, c = n0 + tx + 16 * j;
            if (r < M && c < N)
                mx4_store(static_cast<TC*>(out.C) + r * out.ldc + c, acc[i][j], ga, gb, out, (int)c);
        }
}

template <int FMT, bool A4>
cudaError_t launch(int M, int N, int K, const Mx4Operand& A, const void* a16, long lda,
                   const Mx4Operand& B, const Mx4Out& out, cudaStream_t s) {
    const dim3 grid((unsigned)(((long)N + BT - 1) / BT), (unsigned)(((long)M + BT - 1) / BT));
    if (grid.y > 65535) return cudaErrorInvalidValue;
    const auto a = static_cast<const __nv_bfloat16*>(a16);
    return out.c_type == TGEMM_TYPE_F32
               ? launch_pdl(product_kernel<FMT, A4, float>, grid, dim3(THREADS), 0, s, M, N, K, A, a, lda, B, out)
               : launch_pdl(product_kernel<FMT, A4, __nv_bfloat16>, grid, dim3(THREADS), 0, s, M, N, K, A, a, lda, B, out);
}

}  // namespace mx4_simt
}  // namespace tgemm
