// What the fused products' kernels share: sums out of tensor memory, and the
// epilogue of a column of C, a lane a column, for any alignment.
#pragma once

#include "fused_act.h"
#include "mx4_tile.h"

namespace tgemm {
namespace fused_column {

using namespace mx4_ptx;
using namespace fused_act;
typedef __nv_bfloat16 bf16;

template <bool PAIR>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 sums of this thread's lane (zeros where K is 0).
__device__ __forceinline__ void load_sums(uint32_t tmem, float (&v)[32], int kblocks) {
    uint32_t r[32];
    tmem_ld32(tmem, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (kblocks == 0)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
}

// The rows that count (FusedEpilogue::keep), by warp `mine` of `warps`: while the
// first tile's sums are made (a kernel of its own before the product: 10 us on 4096 x
// 4096, and a launch).
__device__ __forceinline__ void keep_rows(const FusedEpilogue& e, long rows, long mine, long warps) {
    const int lane = threadIdx.x & 31;
    for (long row = mine; row < rows; row += warps) {
        const long long t = e.target[row];
        const bool counts = t >= 0 && t < e.vocabulary;
        const bf16* from = static_cast<const bf16*>(e.keep) + row * e.ld_keep;
        bf16* to = static_cast<bf16*>(e.kept) + row * e.ld_kept;
#pragma unroll 4
        for (int c = lane * 8; c < e.keep_cols; c += 256)
            *reinterpret_cast<uint4*>(to + c) = counts ? *reinterpret_cast<const uint4*>(from + c) : make_uint4(0, 0, 0, 0);
    }
}

// Column c of C, below N columns (gated: and column N + c of what has 2 N), rows
// in groups of eight, whose loads come before their stores.
template <int KIND, bool GATED>
struct Column {
    static constexpr bool TWO = KIND == FUSED_ACT && GATED;      // sums of g and of u
    const FusedEpilogue& e;
    const long N;
    const int c;
    float b = 0.0f, b2 = 0.0f;                                   // bias
    float sum = 0.0f, sum2 = 0.0f;                               // GRAD: of this thread's rows

    const long shift;                                            // ACT: of C, in elements

    __device__ __forceinline__ Column(const FusedEpilogue& e_, long N_, int c_, long shift_ = 0)
        : e(e_), N(N_), c(c_), shift(shift_) {
        if (KIND == FUSED_ACT && e.bias != nullptr) {
            b = e.bias[c];
            if constexpr (TWO) b2 = e.bias[N + c];
        }
    }

    // Rows of R or Z on their way to L2: row, row + 32, .. below `end` (a warp's
    // lanes ask for a row each, of the 32 columns that they are).
    __device__ __forceinline__ void ask(long row, long end) const {
        const char* from = nullptr;
        long pitch = 0, second = 0;
        if (KIND == FUSED_ACT && e.R != nullptr) {
            const long size = e.r_f32 ? 4 : 2;
            from = static_cast<const char*>(e.R) + c * size;
            pitch = e.ldr * size;
        } else if (KIND == FUSED_GRAD) {
            from = static_cast<const char*>(e.Z) + c * 2L;
            pitch = e.ldz * 2;
            second = GATED ? N * 2 : 0;
        }
        if (from == nullptr) return;
        for (; row < end; row += 32) {
            asm volatile("prefetch.global.L2 [%0];" :: "l"(from + row * pitch));
            if (GATED && KIND == FUSED_GRAD) asm volatile("prefetch.global.L2 [%0];" :: "l"(from + row * pitch + second));
        }
    }

    // What rows row .. row + 7, of which the first n are C's (FULL: all), take beside
    // their sums: R, or Z (gated: and its second half).
    template <bool FULL>
    __device__ __forceinline__ void load(long row, int n, float (&z)[8], float (&w)[8]) const {
        if (KIND == FUSED_ACT && e.R != nullptr) {
            if (e.r_f32) {
                const float* R = static_cast<const float*>(e.R) + row * e.ldr + c;
#pragma unroll
                for (int j = 0; j < 8; ++j, R += e.ldr) z[j] = FULL || j < n ? *R : 0.0f;
            } else {
                const bf16* R = static_cast<const bf16*>(e.R) + row * e.ldr + c;
#pragma unroll
                for (int j = 0; j < 8; ++j, R += e.ldr) z[j] = FULL || j < n ? __bfloat162float(*R) : 0.0f;
            }
        }
        if (KIND == FUSED_GRAD) {
            const bf16* Z = static_cast<const bf16*>(e.Z) + row * e.ldz + c;
#pragma unroll
            for (int j = 0; j < 8; ++j, Z += e.ldz) {
                z[j] = FULL || j < n ? __bfloat162float(*Z) : 0.0f;
                if constexpr (GATED) w[j] = FULL || j < n ? __bfloat162float(Z[N]) : 0.0f;
            }
        }
    }

    // Those rows, from their sums x (TWO: g's, y u's) and what load gave.
    template <bool FULL>
    __device__ __forceinline__ void finish(long row, int n, float (&x)[8], float (&y)[8], float (&z)[8], float (&w)[8]) {
        if constexpr (KIND == FUSED_ACT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] += b;
                if constexpr (TWO) y[j] += b2;
            }
            if (e.Z != nullptr) {
                bf16* Z = static_cast<bf16*>(e.Z) + row * e.ldz + c;
#pragma unroll
                for (int j = 0; j < 8; ++j, Z += e.ldz)
                    if (FULL || j < n) {
                        Z[0] = __float2bfloat16(x[j]);
                        if constexpr (TWO) Z[N] = __float2bfloat16(y[j]);
                    }
            }
            apply(e.act, x);
            if constexpr (TWO)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= y[j];
            if (e.R != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(e.r_scale, z[j], x[j]);
        } else if constexpr (KIND == FUSED_GRAD) {
            if constexpr (GATED) {
                gated_grad(e.act, x, z, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = z[j];
                    y[j] = w[j];
                }
            } else {
                times_slope(e.act, x, z);
            }
            if (e.sums != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (FULL || j < n) {
                        sum += x[j];
                        if constexpr (GATED) sum2 += y[j];
                    }
        } else if constexpr (KIND == FUSED_CE_GRAD) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (FULL || j < n) {
                    const long long t = e.target[row + j];
                    const float d = fmaf(x[j], e.alpha, -e.lse[row + j]);
                    const float p = t - e.first == c ? expm1f(d) : exp2_fast(d * LOG2E);
                    // (A row left out may hold infinities.)
                    x[j] = t >= 0 && t < e.vocabulary ? p * (e.alpha * e.dloss[row + j]) : 0.0f;
                }
        }
        const long at = row * e.ldc + c + (KIND == FUSED_ACT && !GATED ? shift : 0);
        if (e.c_f32) {
            float* C = static_cast<float*>(e.C) + at;
#pragma unroll
            for (int j = 0; j < 8; ++j, C += e.ldc)
                if (FULL || j < n) *C = x[j];
        } else {
            bf16* C = static_cast<bf16*>(e.C) + at;
#pragma unroll
            for (int j = 0; j < 8; ++j, C += e.ldc)
                if (FULL || j < n) {
                    C[0] = __float2bfloat16(x[j]);
                    if constexpr (KIND == FUSED_GRAD && GATED) C[N] = __float2bfloat16(y[j]);
                }
        }
    }

    // Rows row + first, row + first + step, .. below row + end in groups of eight, sums
    // by sums(k, x, y); a group's loads are on their way while the one before is
    // finished, the first group's while before() runs. All lanes of a warp (`in`: this
    // one has a column).
    template <typename Before, typename Sums>
    __device__ __forceinline__ void rows(long row, int first, int end, int step, bool in, Before before, Sums sums) {
        float z[8], w[8];
        if (in && end - first >= 8) load<true>(row + first, 8, z, w);
        else if (in && first < end) load<false>(row + first, end - first, z, w);
        before();
#pragma unroll 1
        for (int k = first; k < end; k += step) {
            float x[8], y[8], next_z[8], next_w[8];
            const int left = end - k - step;
            if (in && left >= 8) load<true>(row + k + step, 8, next_z, next_w);
            else if (in && left > 0) load<false>(row + k + step, left, next_z, next_w);
            sums(k, x, y);
            if (in && end - k >= 8) finish<true>(row + k, 8, x, y, z, w);
            else if (in) finish<false>(row + k, end - k, x, y, z, w);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = next_z[j];
                w[j] = next_w[j];
            }
        }
    }

    // The sums, as entry `block` of what fused_join_sums adds up.
    __device__ __forceinline__ void leave(long block) {
        if (KIND == FUSED_GRAD && e.sums != nullptr) {
            float* to = e.sums + block * (GATED ? 2 * N : N) + c;
            to[0] = sum;
            if constexpr (GATED) to[N] = sum2;
        }
    }
};

}  // namespace fused_column
}  // namespace tgemm
