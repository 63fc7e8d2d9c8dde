// Few BF16 rows times a kept 4-bit matrix, C = alpha X W^T + beta C + bias
// with at most MX4_FEW_ROWS rows of X: bound by reading W once.
//
// A warp multiplies 32 rows of W (RW times the 16-row side of mma.sync
// m16n8k16) with 8 NT rows of X. A lane takes 16 bytes of codes of two rows -- 32
// columns of K, four lanes side by side 128 -- and uses them as the K
// positions that the instruction gives it: a sum over K may take its terms in
// any order as long as X's fragments follow the same one. So codes go from
// memory to registers to the tensor core, with no exchange between lanes.
// Eight warps of a block take every eighth 128 columns; their sums meet in
// shared memory, and those of up to eight blocks of a cluster, which split K
// further when W has few rows, through distributed shared memory, always in
// the same order. Where C keeps 32 bits a warp's sum is made of sums over
// SUM_K columns, as in the other kernels.

#include "mx4_decode.h"

#include <type_traits>

namespace tgemm {
namespace {

using namespace mx4_decode;

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int UNIT_K = 128;
constexpr int RW = 2, TN = 16 * RW;                  // 16-row tiles of W a warp, and their rows

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive values of X of which the row has `left` more; 0 past them.
__device__ __forceinline__ uint4 load_x(const __nv_bfloat16* x, int left) {
    uint32_t w[4];
    const uint16_t* p = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? p[2 * i] : 0, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0;
        w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 128-column unit of a lane: codes of its 2 RW rows and the words that
// hold their scales. A lane copies what it will use itself (cp.async) into
// slots of its own, DEPTH units ahead, so the copies need no registers and no
// barrier.
constexpr int DEPTH = 2;
struct Unit {
    uint4 codes[2 * RW];
    uint32_t scales[2 * RW];
};
struct Slots {
    uint4 codes[WARPS][DEPTH][2 * RW][32];
    uint32_t scales[WARPS][DEPTH][2 * RW][32];
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(d), "l"(src) : "memory");
}

// BLOCKS: how many blocks are resident on an SM, 2 (up to 128 registers a
// thread) or 3 (80). LONG: a warp's sum is made of parts (for sums of one part,
// 1 x 14336 x 4096 MXFP4 with FP32 C, the registers of a second sum cost 6 %).
template <int FMT, int NT, int BLOCKS, bool LONG, typename TC>
__global__ void __launch_bounds__(THREADS, BLOCKS)
weights_rows_kernel(int M, int N, int K, const __nv_bfloat16* X, long ldx, bool vec, Mx4Operand W,
                    Mx4Out out, int split) {
    constexpr int TM = 8 * NT;
    __shared__ uint32_t factors[256];
    extern __shared__ __align__(16) uint8_t slots_raw[];
    Slots& slots = *reinterpret_cast<Slots*>(slots_raw);
    // The sums, once every warp is done with its slots.
    float (&part)[WARPS][TN][TM + 1] = *reinterpret_cast<float (*)[WARPS][TN][TM + 1]>(slots_raw);
    __shared__ float total[TN * TM];
    static_assert(sizeof(part) <= sizeof(Slots), "sums in place of the slots");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = split > 1 ? (int)(blockIdx.x % split) : 0;
    const long n0 = (long)(blockIdx.x / split) * TN;
    factors[threadIdx.x] = factor<FMT>(threadIdx.x);
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();

    const int units = (K + UNIT_K - 1) / UNIT_K;
    // Addresses are a base of the block's and 32-bit offsets. Rows past N and
    // past M repeat the last one: their sums are not stored.
    const uint32_t pitch = (uint32_t)mx4_pitch(K);
    const uint8_t* code_base = W.codes + n0 * pitch;
    const uint8_t* scale_base = W.scales + mx4_scale_at(n0, 0, mx4_tiles_k(K, FMT));
    uint32_t code_at[2 * RW], scale_at[2 * RW];
#pragma unroll
    for (int i = 0; i < 2 * RW; ++i) {
        const uint32_t r = (uint32_t)min((long)(i * 8 + g), N - 1 - n0);
        code_at[i] = r * pitch;
        scale_at[i] = r * 16 + (FMT == TGEMM_MXFP4 ? 0 : (t >> 1) * MX4_TILE_BYTES);     // 32 rows in one column of a tile
    }
    const __nv_bfloat16* x_row[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x_row[i] = X + (long)min(i * 8 + g, M - 1) * ldx + t * 32;

    // A unit's copies, one group; past the last unit an empty one.
    auto fetch = [&](int unit, int slot) {
        if (unit < units) {
            // Past the row's end any codes do: X is 0 there.
            const uint32_t at = min((uint32_t)unit * 64 + t * 16, pitch - 16);
            const uint32_t sc = (uint32_t)unit * (FMT == TGEMM_MXFP4 ? MX4_TILE_BYTES : 2 * MX4_TILE_BYTES);
#pragma unroll
            for (int i = 0; i < 2 * RW; ++i) {
                copy_async<16>(&slots.codes[warp][slot][i][lane], code_base + (code_at[i] + at));
                copy_async<4>(&slots.scales[warp][slot][i][lane], scale_base + (scale_at[i] + sc));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](Unit& u, int slot) {
#pragma unroll
        for (int i = 0; i < 2 * RW; ++i) {
            u.codes[i] = slots.codes[warp][slot][i][lane];
            const uint32_t w = slots.scales[warp][slot][i][lane];
            u.scales[i] = FMT == TGEMM_MXFP4 ? w >> t * 8 & 0xFF : w >> (t & 1) * 16 & 0xFFFF;
        }
    };

    float acc[RW][NT][4] = {};
    // Columns j * 8 .. j * 8 + 7 of a lane's 32: X's fragments, and the product.
    auto step8 = [&](const Unit& u, int j, const uint4 (&xs)[NT], const uint32_t (&f)[2 * RW][2], auto is_wide) {
        uint32_t b[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            b[i][0] = __byte_perm(xs[i].x, xs[i].z, 0x5410);       // columns 0 and 4
            b[i][1] = __byte_perm(xs[i].x, xs[i].z, 0x7632);       // 1 and 5
            b[i][2] = __byte_perm(xs[i].y, xs[i].w, 0x5410);       // 2 and 6
            b[i][3] = __byte_perm(xs[i].y, xs[i].w, 0x7632);       // 3 and 7
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            uint32_t v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 c = u.codes[2 * r + h];
                values<decltype(is_wide)::value>(j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w,
                                                 f[2 * r + h][j / 2], v[h]);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma_bf16(acc[r][i], v[0][0], v[1][0], v[0][1], v[1][1], b[i][0], b[i][1]);
                mma_bf16(acc[r][i], v[0][2], v[1][2], v[0][3], v[1][3], b[i][2], b[i][3]);
            }
        }
    };
    // X comes from the caches: loaded when its unit is due, not ahead.
    auto run = [&](const Unit& u, int unit) {
        uint32_t f[2 * RW][2];                     // the factors of a row's first and last 16 codes
        bool w = false;
#pragma unroll
        for (int i = 0; i < 2 * RW; ++i) {
            if (FMT == TGEMM_NVFP4) {
                f[i][0] = factors[u.scales[i] & 0xFF];
                f[i][1] = factors[u.scales[i] >> 8];
            } else {
                f[i][0] = f[i][1] = (u.scales[i] + 124) * 0x00800080u;
                w |= wide(u.scales[i]);
            }
        }
        const int k0 = unit * UNIT_K;
        if (vec && K - k0 >= UNIT_K && !(FMT == TGEMM_MXFP4 && __any_sync(~0u, w))) {
            uint4 xs[4][NT];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i) xs[j][i] = reinterpret_cast<const uint4*>(x_row[i] + k0)[j];
#pragma unroll
            for (int j = 0; j < 4; ++j) step8(u, j, xs[j], f, std::false_type());
            return;
        }
        // The last columns, rows off 16 bytes, wide scales.
        if (FMT == TGEMM_MXFP4) {
            w = __any_sync(~0u, w);
#pragma unroll
            for (int i = 0; i < 2 * RW; ++i) {
                // Beside a wide block the others take their scale alone too.
                const uint32_t c = u.scales[i];
                f[i][0] = f[i][1] = !w ? f[i][0] : c == 255 ? 0x7FC07FC0u : c == 0 ? 0x00400040u : c * 0x00800080u;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 xs[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) xs[i] = load_x(x_row[i] + k0 + j * 8, K - k0 - t * 32 - j * 8);
            if (FMT == TGEMM_MXFP4 && w) step8(u, j, xs, f, std::true_type());
            else step8(u, j, xs, f, std::false_type());
        }
    };

    // The parts of a long sum are added with rounding to nearest.
    float parts[RW][NT][4] = {};
    auto end_part = [&]() {
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    parts[r][i][k] += acc[r][i][k];
                    acc[r][i][k] = 0.0f;
                }
    };

    const int step = WARPS * split;
    int unit = rank * WARPS + warp, slot = 0, in_part = 0;
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) fetch(unit + i * step, i);
#pragma unroll 1
    for (; unit < units; unit += step) {
        asm volatile("cp.async.wait_group %0;" :: "n"(DEPTH - 1) : "memory");
        Unit u;
        take(u, slot);
        fetch(unit + DEPTH * step, slot);            // the lane's own slot, read just before
        run(u, unit);
        if (LONG && ++in_part == SUM_K / UNIT_K) {
            in_part = 0;
            end_part();
        }
        if (++slot == DEPTH) slot = 0;
    }
    if (LONG) end_part();
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                part[warp][r * 16 + (k >> 1) * 8 + g][i * 8 + 2 * t + (k & 1)] = LONG ? parts[r][i][k] : acc[r][i][k];
    __syncthreads();
    const float gb = mx4_g(W.g);
    auto store = [&](int i, float v) {
        const int m = i / TN;
        const long n = n0 + i % TN;
        if (m < M && n < N)
            mx4_store(static_cast<TC*>(out.C) + (long)m * out.ldc + n, v * unscale<FMT>(), 1.0f, gb, out, (int)n);
    };
    for (int i = threadIdx.x; i < TN * TM; i += THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w][i % TN][i / TN];
        if (split == 1) store(i, v); else total[i] = v;
    }
    if (split == 1) return;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // Block `rank` adds its share of the outputs over the cluster.
    for (int i = rank * THREADS + threadIdx.x; i < TN * TM; i += split * THREADS) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&total[i]));
        float v = 0.0f;
        for (int r = 0; r < split; ++r) {
            uint32_t remote;
            float w;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(remote) : "memory");
            v += w;
        }
        store(i, v);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int FMT, int NT, int BLOCKS, bool LONG, typename TC>
cudaError_t launch_kernel(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W, const Mx4Out& out,
                   int split, cudaStream_t s) {
    const long tiles = ((long)N + TN - 1) / TN;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sizeof(Slots);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    const cudaError_t e = set_smem_limit_once<weights_rows_kernel<FMT, NT, BLOCKS, LONG, TC>>(sizeof(Slots));
    if (e != cudaSuccess) return e;
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
    return cudaLaunchKernelEx(&cfg, weights_rows_kernel<FMT, NT, BLOCKS, LONG, TC>, M, N, K, X, ldx, vec, W, out, split);
}

template <int FMT, int NT, int BLOCKS, typename TC>
cudaError_t launch(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W, const Mx4Out& out,
                   int split, cudaStream_t s) {
    if constexpr (sizeof(TC) == 4)
        if (((long)K + UNIT_K - 1) / UNIT_K > (long)WARPS * split * (SUM_K / UNIT_K))
            return launch_kernel<FMT, NT, BLOCKS, true, TC>(M, N, K, X, ldx, W, out, split, s);
    return launch_kernel<FMT, NT, BLOCKS, false, TC>(M, N, K, X, ldx, W, out, split, s);
}

// Resident blocks (2 or 3) and the blocks of a cluster that split K. A round of
// resident blocks is taken to last as long as there are blocks on an SM, times a
// warp's units and about three units' worth of start and end. Two against three,
// MXFP4, us (* the choice): 1 x 1024 x 4096 3.9* and 4.5, 8 x 4096 x 4096 5.5* and 7.3,
// 1 x 4096 x 14336 12.9* and 13.9, 8 x 14336 x 4096 14.8 and 11.5*, 8 x 8192 x 28672
// 38.6* and 46.0; with many rounds it errs, 1 x 65536 x 4096 43.5* and 39.9.
struct Choice {
    int blocks, split;
};
Choice choose(long tiles, int K, int num_sms, int most = 3) {
    const int units = (K + UNIT_K - 1) / UNIT_K;
    Choice best{2, 1};
    long least = -1;
    for (int blocks = 2; blocks <= most; ++blocks)
        for (int c = 1; c <= 8; ++c) {
            const long slots = (long)blocks * num_sms;
            const long cost = (tiles * c + slots - 1) / slots * ((units + WARPS * c - 1) / (WARPS * c) + 3) * blocks;
            if (least < 0 || cost < least) {
                least = cost;
                best = {blocks, c};
            }
        }
    return best;
}

template <int FMT, int NT, typename TC>
cudaError_t launch_blocks(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W,
                          const Mx4Out& out, int num_sms, cudaStream_t s) {
    const Choice c = choose(((long)N + TN - 1) / TN, K, num_sms);
    return c.blocks == 2 ? launch<FMT, NT, 2, TC>(M, N, K, X, ldx, W, out, c.split, s)
                         : launch<FMT, NT, 3, TC>(M, N, K, X, ldx, W, out, c.split, s);
}

template <int FMT, typename TC>
cudaError_t launch_rows(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W,
                        const Mx4Out& out, int num_sms, cudaStream_t s) {
    if (M <= 8) return launch_blocks<FMT, 1, TC>(M, N, K, X, ldx, W, out, num_sms, s);
    if (M <= 16) return launch_blocks<FMT, 2, TC>(M, N, K, X, ldx, W, out, num_sms, s);
    return launch<FMT, 3, 2, TC>(M, N, K, X, ldx, W, out, choose(((long)N + TN - 1) / TN, K, num_sms, 2).split, s);
}

}  // namespace

cudaError_t mx4_weights_rows(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt,
                             const Mx4Out& out, int num_sms, cudaStream_t s) {
    const auto X = static_cast<const __nv_bfloat16*>(A);
    if (out.c_type == TGEMM_TYPE_F32)
        return fmt == TGEMM_MXFP4 ? launch_rows<TGEMM_MXFP4, float>(M, N, K, X, lda, B, out, num_sms, s)
                                  : launch_rows<TGEMM_NVFP4, float>(M, N, K, X, lda, B, out, num_sms, s);
    return fmt == TGEMM_MXFP4 ? launch_rows<TGEMM_MXFP4, __nv_bfloat16>(M, N, K, X, lda, B, out, num_sms, s)
                              : launch_rows<TGEMM_NVFP4, __nv_bfloat16>(M, N, K, X, lda, B, out, num_sms, s);
}

}  // namespace tgemm
