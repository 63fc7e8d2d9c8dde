// Few BF16 rows times a kept 4-bit matrix, C = alpha X W^T + beta C + bias
// with at most 16 rows of X: bound by reading W once.
//
// A warp multiplies 16 RW rows of W (the 16-row side of mma.sync m16n8k16)
// with 8 NT rows of X. A lane takes 16 bytes of codes of two rows -- 32
// columns of K, four lanes side by side 128 -- and uses them as the K
// positions that the instruction gives it: a sum over K may take its terms in
// any order as long as X's fragments follow the same one. So codes go from
// memory to registers to the tensor core, with no exchange between lanes.
// Eight warps of a block take every eighth 128 columns; their sums meet in
// shared memory, and those of up to eight blocks of a cluster, which split K
// further when W has few rows, through distributed shared memory, always in
// the same order.

#include "mx4_decode.h"

#include <type_traits>

namespace tgemm {
namespace {

using namespace mx4_decode;

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int UNIT_K = 128;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive values of a row of X from column k on, 0 past K.
__device__ __forceinline__ uint4 load_x(const __nv_bfloat16* row, long k, int K, bool vec) {
    if (vec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4];
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + k;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = k + 2 * i < K ? p[2 * i] : 0, hi = k + 2 * i + 1 < K ? p[2 * i + 1] : 0;
        w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 128-column unit of a lane: codes of its 2 RW rows and their scales.
template <int RW>
struct Unit {
    uint4 codes[2 * RW];
    uint32_t scales[2 * RW];        // one byte (MXFP4) or two (NVFP4)
};

template <int FMT, int NT, int RW, typename TC>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 3 : 2)
weights_rows_kernel(int M, int N, int K, const __nv_bfloat16* X, long ldx, bool vec, Mx4Operand W,
                    Mx4Out out, int split) {
    constexpr int TN = 16 * RW, TM = 8 * NT;
    __shared__ uint32_t factors[256];
    __shared__ float part[WARPS][TN][TM + 1];
    __shared__ float total[TN * TM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = split > 1 ? (int)(blockIdx.x % split) : 0;
    const long n0 = (long)(blockIdx.x / split) * TN;
    factors[threadIdx.x] = factor<FMT>(threadIdx.x);
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();

    const long pitch = mx4_pitch(K), tiles_k = mx4_tiles_k(K, FMT);
    const int units = (K + UNIT_K - 1) / UNIT_K;
    const uint8_t* code_row[2 * RW];
    const uint8_t* scale_row[2 * RW];
#pragma unroll
    for (int i = 0; i < 2 * RW; ++i) {
        const long r = min(n0 + i * 8 + g, (long)N - 1);     // rows past N: read, not stored
        code_row[i] = W.codes + r * pitch + t * 16;
        scale_row[i] = W.scales + mx4_scale_at(r, 0, tiles_k) +
                       (FMT == TGEMM_MXFP4 ? t : (t >> 1) * MX4_TILE_BYTES + (t & 1) * 2);
    }
    const __nv_bfloat16* x_row[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x_row[i] = i * 8 + g < M ? X + (long)(i * 8 + g) * ldx : nullptr;

    using U = Unit<RW>;
    auto load = [&](U& u, int unit) {
        const bool in = (long)unit * 64 + t * 16 < pitch;
#pragma unroll
        for (int i = 0; i < 2 * RW; ++i) {
            u.codes[i] = in ? __ldg(reinterpret_cast<const uint4*>(code_row[i] + (long)unit * 64)) : make_uint4(0, 0, 0, 0);
            if (FMT == TGEMM_MXFP4) u.scales[i] = __ldg(scale_row[i] + (long)unit * MX4_TILE_BYTES);
            else u.scales[i] = __ldg(reinterpret_cast<const uint16_t*>(scale_row[i] + (long)unit * 2 * MX4_TILE_BYTES));
        }
    };

    float acc[RW][NT][4] = {};
    auto multiply = [&](const U& u, const uint4 (&xs)[NT][4], auto is_wide) {
        constexpr bool WIDE = decltype(is_wide)::value;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t b[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 x = xs[i][j];
                b[i][0] = __byte_perm(x.x, x.z, 0x5410);       // columns 0 and 4
                b[i][1] = __byte_perm(x.x, x.z, 0x7632);       // 1 and 5
                b[i][2] = __byte_perm(x.y, x.w, 0x5410);       // 2 and 6
                b[i][3] = __byte_perm(x.y, x.w, 0x7632);       // 3 and 7
            }
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                uint32_t v[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 c = u.codes[2 * r + h];
                    const uint32_t s = u.scales[2 * r + h];
                    const uint32_t byte = FMT == TGEMM_MXFP4 ? s : j < 2 ? s & 0xFF : s >> 8;
                    uint32_t f = factors[byte];
                    // Beside a wide block the others take their scale alone too.
                    if (WIDE && byte != 255) f = byte == 0 ? 0x00400040u : byte << 7 | byte << 23;
                    values<WIDE>(j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w, f, v[h]);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma_bf16(acc[r][i], v[0][0], v[1][0], v[0][1], v[1][1], b[i][0], b[i][1]);
                    mma_bf16(acc[r][i], v[0][2], v[1][2], v[0][3], v[1][3], b[i][2], b[i][3]);
                }
            }
        }
    };
    // X comes from the caches: loaded when its unit is due, not ahead.
    auto run = [&](const U& u, int unit) {
        uint4 xs[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xs[i][j] = x_row[i] != nullptr ? load_x(x_row[i], (long)unit * UNIT_K + t * 32 + j * 8, K, vec)
                                               : make_uint4(0, 0, 0, 0);
        bool w = false;
        if (FMT == TGEMM_MXFP4)
#pragma unroll
            for (int i = 0; i < 2 * RW; ++i) w |= wide(u.scales[i]);
        if (FMT == TGEMM_MXFP4 && __any_sync(~0u, w)) multiply(u, xs, std::true_type());
        else multiply(u, xs, std::false_type());
    };

    // Two units in flight.
    const int step = WARPS * split;
    int unit = rank * WARPS + warp;
    U u0, u1;
    if (unit < units) load(u0, unit);
    while (unit < units) {
        if (unit + step < units) load(u1, unit + step);
        run(u0, unit);
        unit += step;
        if (unit >= units) break;
        if (unit + step < units) load(u0, unit + step);
        run(u1, unit);
        unit += step;
    }

#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                part[warp][r * 16 + (k >> 1) * 8 + g][i * 8 + 2 * t + (k & 1)] = acc[r][i][k];
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

template <int FMT, int NT, int RW, typename TC>
cudaError_t launch(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W, const Mx4Out& out,
                   int num_sms, cudaStream_t s) {
    const long tiles = ((long)N + 16 * RW - 1) / (16 * RW);
    // Blocks of a cluster split K while there are too few blocks to fill the
    // SMs and each keeps two units a warp.
    const int units = (K + UNIT_K - 1) / UNIT_K;
    int split = 1;
    while (split < 8 && tiles * split < 2L * num_sms && units >= 2 * WARPS * (split + 1)) ++split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(THREADS);
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
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
    return cudaLaunchKernelEx(&cfg, weights_rows_kernel<FMT, NT, RW, TC>, M, N, K, X, ldx, vec, W, out, split);
}

template <int FMT, typename TC>
cudaError_t launch_rows(int M, int N, int K, const __nv_bfloat16* X, long ldx, const Mx4Operand& W,
                        const Mx4Out& out, int num_sms, cudaStream_t s) {
    return M <= 8 ? launch<FMT, 1, 2, TC>(M, N, K, X, ldx, W, out, num_sms, s)
                  : launch<FMT, 2, 2, TC>(M, N, K, X, ldx, W, out, num_sms, s);
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
