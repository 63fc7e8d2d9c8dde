// The small kernels beside the fused products: joining column sums and the
// cross entropy's maxima and sums, and keeping the rows that count.

#include "fused_act.h"

namespace tgemm {
namespace {

using fused_act::exp2_fast;
using fused_act::LOG2E;

// A block takes 32 columns; its 8 warps take every eighth block of rows each
// and are added in their order.
__global__ void __launch_bounds__(256) join_sums_kernel(const float* sums, long blocks, long cols, float* db) {
    pdl_launch_dependents();
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long c = (long)blockIdx.x * 32 + lane;
    pdl_wait();
    float v = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (long b = warp; b < blocks; b += 8) v += sums[b * cols + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += part[w][lane];
        db[c] = v;
    }
}

// Two shares of a sum of exponentials, each a maximum m and the sum s of
// exp(z - m): joined.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
    s = s * exp2_fast((m - base) * LOG2E) + s2 * exp2_fast((m2 - base) * LOG2E);
    m = top;
}

// A block takes `rows` rows (a power of two, up to 32); its threads, a row each,
// take every (1024 / rows)th block of columns and are joined in a fixed order:
// a warp's lanes, then the warps.
__global__ void __launch_bounds__(1024)
join_ce_kernel(const float2* parts, const float* picked, const long long* target, int T, long V, long blocks, int rows,
               float* loss, float* lse) {
    pdl_launch_dependents();
    __shared__ float2 part[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long row = (long)blockIdx.x * rows + (threadIdx.x & (rows - 1));
    const int slices = 1024 / rows;
    pdl_wait();
    float m = -INFINITY, s = 0.0f;
    if (row < T) {
        long b = threadIdx.x / rows;
        for (; b + 3L * slices < blocks; b += 4L * slices) {
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = parts[(b + (long)j * slices) * T + row];
#pragma unroll
            for (int j = 0; j < 4; ++j) join(m, s, v[j].x, v[j].y);
        }
        for (; b < blocks; b += slices) {
            const float2 v = parts[b * T + row];
            join(m, s, v.x, v.y);
        }
    }
    for (int w = 16; w >= rows; w >>= 1) join(m, s, __shfl_xor_sync(~0u, m, w), __shfl_xor_sync(~0u, s, w));
    if (lane < rows) part[lane][warp] = make_float2(m, s);
    __syncthreads();
    // A warp a row, a lane a warp's share.
    if (warp < rows) {
        const float2 v = part[warp][lane];
        m = v.x;
        s = v.y;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) join(m, s, __shfl_xor_sync(~0u, m, w), __shfl_xor_sync(~0u, s, w));
        const long i = (long)blockIdx.x * rows + warp;
        if (lane == 0 && i < T) {
            // The target's logit is taken from the maximum, not from lse: a loss near
            // zero keeps its digits.
            const float l = logf(s);
            lse[i] = m + l;
            const long long t = target[i];
            loss[i] = t >= 0 && t < V ? (m - picked[i]) + l : 0.0f;
        }
    }
}

__global__ void __launch_bounds__(256)
keep_rows_kernel(const __nv_bfloat16* X, long ldx, __nv_bfloat16* Y, long ldy, int T, int D, const long long* target,
                 long V, int wide) {
    pdl_launch_dependents();
    pdl_wait();
    for (long row = blockIdx.x; row < T; row += gridDim.x) {
        const long long t = target[row];
        const bool kept = t >= 0 && t < V;
        const __nv_bfloat16* x = X + row * ldx;
        __nv_bfloat16* y = Y + row * ldy;
        if (wide) {
            for (int c = threadIdx.x * 8; c < D; c += 256 * 8)
                *reinterpret_cast<uint4*>(y + c) = kept ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
        } else {
            for (int c = threadIdx.x; c < D; c += 256) y[c] = kept ? x[c] : __float2bfloat16(0.0f);
        }
    }
}

}  // namespace

cudaError_t fused_join_sums(const float* sums, long blocks, long cols, float* db, cudaStream_t s) {
    return launch_pdl(join_sums_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, sums, blocks, cols, db);
}

cudaError_t fused_join_ce(const float2* parts, const float* picked, const long long* target, int T, long V, long blocks,
                          float* loss, float* lse, cudaStream_t s) {
    // Fewer rows a block where there are few: 16 x 65536 x 4096 spent 49 of 135 us
    // here with 32 (and 8 warps).
    int rows = 32;
    while (rows > 1 && (long)T < 128L * rows) rows /= 2;
    return launch_pdl(join_ce_kernel, dim3((unsigned)(((long)T + rows - 1) / rows)), dim3(1024), 0, s, parts, picked, target, T, V,
                      blocks, rows, loss, lse);
}

cudaError_t fused_keep_rows(const void* X, long ldx, void* Y, long ldy, int T, int D, const long long* target, long V,
                            cudaStream_t s) {
    // Whole 16-byte pieces of both rows.
    const int wide = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0 && ldy % 8 == 0 && D % 8 == 0 ? 1 : 0;
    return launch_pdl(keep_rows_kernel, dim3((unsigned)(T < 4096 ? T : 4096)), dim3(256), 0, s,
                      static_cast<const __nv_bfloat16*>(X), ldx, static_cast<__nv_bfloat16*>(Y), ldy, T, D, target, V, wide);
}

}  // namespace tgemm
