// The small kernels beside the fused products: joining column sums, slices of a
// sum and the cross entropy's maxima and sums; copies of operands.

#include "fused_act.h"

namespace tgemm {
namespace {

using fused_act::exp2_fast;
using fused_act::LOG2E;

// A block takes 32 columns; its 8 warps take every eighth block of rows each, add
// them up 64 at a time, and are added in their order. (One after the other the roundings
// of a million rows' additions took 1.0e-6 of db's norm.)
__global__ void __launch_bounds__(256) join_sums_kernel(const float* sums, long blocks, long cols, float* db) {
    pdl_launch_dependents();
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long c = (long)blockIdx.x * 32 + lane;
    pdl_wait();
    float v = 0.0f;
    if (c < cols)
        for (long b = warp; b < blocks;) {
            const long end = b + 8 * 64 < blocks ? b + 8 * 64 : blocks;
            float some = 0.0f;
#pragma unroll 4
            for (; b < end; b += 8) some += sums[b * cols + c];
            v += some;
        }
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

// out[i][j] = the sum of `slices` matrices of rows x cols. A block takes 32 elements;
// its 8 warps take every eighth slice each and are added in their order (76 slices
// of 56 x 170: 11 us a thread an element).
template <typename T>
__global__ void __launch_bounds__(256)
join_slices_kernel(const float* parts, int slices, long size, int cols, T* out, long ld) {
    pdl_launch_dependents();
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long i = (long)blockIdx.x * 32 + lane;
    pdl_wait();
    float v = 0.0f;
    if (i < size)
#pragma unroll 8
        for (int s = warp; s < slices; s += 8) v += parts[s * size + i];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && i < size) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += part[w][lane];
        const long row = i / cols;
        out[row * ld + (i - row * cols)] = (T)v;
    }
}

// Copies of matrices with rows off 16 bytes, and of rows that count. A warp takes
// four rows at a time, so that narrow ones keep it as busy as wide ones (59871 x 170:
// 34 us a row at a time), of 512 columns at most, two columns a lane; rows on 16 bytes
// go eight columns a lane.
struct Copies {
    CopyJob job[3];
    long blocks[3];               // up to and with each job's
};
constexpr int COPY_ROWS = 4, COPY_WARPS = 8, COPY_COLS = 512;

__global__ void __launch_bounds__(32 * COPY_WARPS) copy_rows_kernel(const Copies c) {
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int which = (long)blockIdx.x < c.blocks[0] ? 0 : (long)blockIdx.x < c.blocks[1] ? 1 : 2;
    const CopyJob j = c.job[which];
    const long block = (long)blockIdx.x - (which > 0 ? c.blocks[which - 1] : 0);
    const long across = (j.cols + COPY_COLS - 1) / COPY_COLS;
    const long row0 = (block / across * COPY_WARPS + (threadIdx.x >> 5)) * COPY_ROWS;
    const int first = (int)(block % across) * COPY_COLS, cols = min(j.cols, first + COPY_COLS);
    const __nv_bfloat16 zero = __float2bfloat16(0.0f);
    pdl_wait();
    const __nv_bfloat16* from[COPY_ROWS];
    bool kept[COPY_ROWS];
#pragma unroll
    for (int r = 0; r < COPY_ROWS; ++r) {
        const long row = row0 + r;
        kept[r] = row < j.rows;
        if (kept[r] && j.target != nullptr) {
            const long long t = j.target[row];
            kept[r] = t >= 0 && t < j.V;
        }
        from[r] = static_cast<const __nv_bfloat16*>(j.src) + row * j.ld_src;
    }
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(j.dst) + row0 * j.ld_dst;
    if (j.wide) {
        for (int c0 = first + lane * 8; c0 < cols; c0 += 256) {
            uint4 v[COPY_ROWS];
#pragma unroll
            for (int r = 0; r < COPY_ROWS; ++r)
                v[r] = kept[r] ? *reinterpret_cast<const uint4*>(from[r] + c0) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < COPY_ROWS; ++r)
                if (row0 + r < j.rows) *reinterpret_cast<uint4*>(to + r * j.ld_dst + c0) = v[r];
        }
        return;
    }
    for (int c0 = first + lane * 2; c0 < cols; c0 += 128) {
        __nv_bfloat16 v[COPY_ROWS][2][2];
#pragma unroll
        for (int r = 0; r < COPY_ROWS; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) v[r][u][k] = kept[r] && c0 + u * 64 + k < cols ? from[r][c0 + u * 64 + k] : zero;
        // (Rows of the copy hold whole 64 columns.)
#pragma unroll
        for (int r = 0; r < COPY_ROWS; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (row0 + r < j.rows && c0 + u * 64 < cols)
                    *reinterpret_cast<__nv_bfloat162*>(to + r * j.ld_dst + c0 + u * 64) = __nv_bfloat162(v[r][u][0], v[r][u][1]);
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

cudaError_t fused_join_slices(const float* parts, int slices, int rows, int cols, void* out, long ld, bool f32, cudaStream_t s) {
    const long size = (long)rows * cols;
    const dim3 grid((unsigned)((size + 31) / 32));
    return f32 ? launch_pdl(join_slices_kernel<float>, grid, dim3(256), 0, s, parts, slices, size, cols, static_cast<float*>(out), ld)
               : launch_pdl(join_slices_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, parts, slices, size, cols,
                            static_cast<__nv_bfloat16*>(out), ld);
}

cudaError_t fused_copy_rows(const CopyJob* jobs, int count, cudaStream_t s) {
    Copies c = {};
    long blocks = 0;
    int n = 0;
    for (int i = 0; i < count; ++i) {
        if (jobs[i].rows <= 0 || jobs[i].cols <= 0) continue;
        c.job[n] = jobs[i];
        c.job[n].wide = reinterpret_cast<uintptr_t>(jobs[i].src) % 16 == 0 && jobs[i].ld_src % 8 == 0 && jobs[i].cols % 8 == 0;
        blocks += ((long)jobs[i].rows + COPY_ROWS * COPY_WARPS - 1) / (COPY_ROWS * COPY_WARPS) *
                  (((long)jobs[i].cols + COPY_COLS - 1) / COPY_COLS);
        c.blocks[n++] = blocks;
    }
    if (n == 0) return cudaSuccess;
    if (blocks > 2147483647L) return cudaErrorInvalidValue;
    for (int i = n; i < 3; ++i) c.blocks[i] = blocks;
    return launch_pdl(copy_rows_kernel, dim3((unsigned)blocks), dim3(32 * COPY_WARPS), 0, s, c);
}

}  // namespace tgemm
