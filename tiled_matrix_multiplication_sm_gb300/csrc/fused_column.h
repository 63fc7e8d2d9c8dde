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
    for (int j = 0; j < 32; ++j) v[j] = kblocks > 0 ? __uint_as_float(r[j]) : 0.0f;
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

    __device__ __forceinline__ Column(const FusedEpilogue& e_, long N_, int c_) : e(e_), N(N_), c(c_) {
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

    // Rows row .. row + 7, of which the first n are C's, from their sums x (TWO: g's, y u's).
    __device__ __forceinline__ void finish(long row, int n, float (&x)[8], float (&y)[8]) {
        float z[8];
        bf16* Z = static_cast<bf16*>(e.Z) + row * e.ldz + c;
        if constexpr (KIND == FUSED_ACT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] += b;
                if constexpr (TWO) y[j] += b2;
            }
            if (e.R != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[j] = j >= n      ? 0.0f
                           : e.r_f32 ? static_cast<const float*>(e.R)[(row + j) * e.ldr + c]
                                     : __bfloat162float(static_cast<const bf16*>(e.R)[(row + j) * e.ldr + c]);
            if (e.Z != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) {
                        Z[j * e.ldz] = __float2bfloat16(x[j]);
                        if constexpr (TWO) Z[j * e.ldz + N] = __float2bfloat16(y[j]);
                    }
            apply(e.act, x);
            if constexpr (TWO)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= y[j];
            if (e.R != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(e.r_scale, z[j], x[j]);
        } else if constexpr (KIND == FUSED_GRAD) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = j < n ? __bfloat162float(Z[j * e.ldz]) : 0.0f;
                if constexpr (GATED) y[j] = j < n ? __bfloat162float(Z[j * e.ldz + N]) : 0.0f;
            }
            if constexpr (GATED) {
                gated_grad(e.act, x, z, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = z[j];
            } else {
                times_slope(e.act, x, z);
            }
            if (e.sums != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) {
                        sum += x[j];
                        if constexpr (GATED) sum2 += y[j];
                    }
        } else if constexpr (KIND == FUSED_CE_GRAD) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) {
                    const long long t = e.target[row + j];
                    const float p = exp2_fast((x[j] * e.alpha - e.lse[row + j]) * LOG2E) - (t - e.first == c ? 1.0f : 0.0f);
                    // (A row left out may hold infinities.)
                    x[j] = t >= 0 && t < e.vocabulary ? p * (e.alpha * e.dloss[row + j]) : 0.0f;
                }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                const long at = (row + j) * e.ldc + c;
                if (e.c_f32) static_cast<float*>(e.C)[at] = x[j];
                else static_cast<bf16*>(e.C)[at] = __float2bfloat16(x[j]);
                if constexpr (KIND == FUSED_GRAD && GATED) static_cast<bf16*>(e.C)[at + N] = __float2bfloat16(y[j]);
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
