// Product of two 4-bit matrices, C = alpha A B^T + beta C + bias, on the
// tensor cores' block-scaled MMA (tcgen05, kind mxf4 / mxf4nvf4).
//
// The instruction multiplies E2M1 codes, sums 16 or 32 of them exactly,
// scales the sum by the two blocks' scales and adds it to an FP32 accumulator
// in tensor memory: 64 columns of K an instruction. Both operands are read as
// they are kept: rows of codes, K contiguous, two to a byte, copied by TMA in
// boxes of 128 rows x 128 bytes (256 columns of K, one pipeline stage) into
// the 128-byte swizzle; and tiles of scales, which the MMA wants in tensor
// memory, copied from shared memory by the thread that issues the MMAs
// (tcgen05.cp; it runs in order with them).
//
// Two forms, both persistent, one block on an SM, six or ten warps (0: TMA,
// 1: MMA, from 2 on: epilogue):
//   pair    256 x 256 tiles on an SM pair (cta_group::2). Each block stages
//           its 128 rows of A, its 128 rows of B, A's scales for its rows
//           and B's for all 256. Two accumulators of 256 columns and 48
//           columns of scales do not fit the 512 of tensor memory, so the
//           accumulators share 48 columns: the epilogue drains the shared
//           ones first and then lets the next tile's MMAs start.
//   single  128 x 128 tiles on one SM, for products with few tiles; of very
//           few, a cluster's blocks split K and add their shares through
//           distributed shared memory.
// Long sums with an FP32 result (LONG) come in parts, accumulator by
// accumulator; the epilogue's warps add them up in registers.
//
// Rows past M and N are read as zeros (TMA fill, zero scales) and not stored.
// Waits are bounded as in the other tensor-core kernels.

#include "mx4_tile.h"

#include <cstring>

namespace tgemm {

__device__ int g_mx4_status;

namespace {

using namespace mx4_tile;

constexpr int STAGE_K = MX4_SPAN;
constexpr int OPERAND_BYTES = 128 * SW;       // 128 rows of codes
constexpr int STAGES = 5;
constexpr int EPI_BYTES = 8 * BUF_BYTES;
constexpr int PART_STAGES = SUM_STEPS * 64 / STAGE_K;      // of a long sum

template <int FMT, bool PAIR, bool LONG>
struct Shape {
    static constexpr int TM = PAIR ? 256 : 128;           // rows of a tile
    static constexpr int TN = PAIR ? 256 : 128;           // columns
    // Epilogue: sets of four warps (one to a quarter of tensor memory's lanes)
    // with BUFS buffers a warp. A second set shortens the only tile's way out
    // (1024^3 MXFP4 8.5 -> 7.4 us); between tiles shared memory is the bound,
    // and it costs (8192 x 14336 x 4096 NVFP4 155 -> 158 us). Long sums need two:
    // a thread holds half a row of the tile, for a pair in 128 of its 168
    // registers (14336 x 4096 x 8192 NVFP4: 170 us, in one part 164; with the
    // sums spilled around the epilogue's waits 226).
    static constexpr int SETS = PAIR && !LONG ? 1 : 2, BUFS = 2 / SETS;
    static constexpr int EPI_WARPS = 4 * SETS, THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int SF_TILES = STAGE_K / mx4_block(FMT) / 4;     // scale tiles of 128 rows a stage
    static constexpr int SFA_BYTES = SF_TILES * MX4_TILE_BYTES;
    static constexpr int SFB_BYTES = SFA_BYTES * (TN / 128);
    static constexpr int STAGE_BYTES = 2 * OPERAND_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 256;
    // Tensor memory: accumulators at 0 and ACC1, scales from SF on.
    static constexpr int SF_COLS = SF_TILES * 4 * (1 + TN / 128);
    static constexpr int SF = PAIR ? 464 : 256;
    static constexpr int ACC1 = PAIR ? SF - TN : 128;
    static_assert(SF + SF_COLS <= TMEM_COLS && (!PAIR || TN - ACC1 <= 64), "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Sync {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Sync) <= 256, "barrier block");

struct Params : Tiling {
    int kblocks;
    const float *ga, *gb;
};

template <int FMT, bool PAIR, bool LONG, typename TC>
__global__ void __launch_bounds__(Shape<FMT, PAIR, LONG>::THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmC, const Params p) {
    using S = Shape<FMT, PAIR, LONG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* epi = smem + STAGES * S::STAGE_BYTES;
    Sync* sy = reinterpret_cast<Sync*>(epi + EPI_BYTES);
    // The stages' codes first (1 KB aligned), their scales after them.
    const uint32_t codes0 = smem_u32(smem);
    const uint32_t scales0 = codes0 + STAGES * 2 * OPERAND_BYTES;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const int part = PAIR ? 0 : blockIdx.x % p.split;
    const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x / p.split;
    const int kb0 = PAIR ? 0 : (int)((long)p.kblocks * part / p.split);
    const int kb1 = PAIR ? p.kblocks : (int)((long)p.kblocks * (part + 1) / p.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sy->full[s]), 1);
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->tmem_full[a]), 1);
            mbar_init(smem_u32(&sy->tmem_empty[a]), (PAIR ? 2 : 1) * S::EPI_WARPS);
        }
        mbar_init(smem_u32(&sy->drain), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        prefetch_map(&tmSA);
        prefetch_map(&tmSB);
    }
    if (warp == 1) tmem_alloc<PAIR, TMEM_COLS>(smem_u32(&sy->tmem_base));
    tc_fence_before();
    if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sy->tmem_base;
    pdl_launch_dependents();
    pdl_wait();

    const Wait wait{&sy->abort, p.status, p.wait_limit_ns};
    // The leader's barriers, as cluster addresses.
    const uint32_t full0 = PAIR ? map_to_rank(smem_u32(&sy->full[0]), 0) : smem_u32(&sy->full[0]);
    const uint32_t tmem_empty0 =
        PAIR ? map_to_rank(smem_u32(&sy->tmem_empty[0]), 0) : smem_u32(&sy->tmem_empty[0]);

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        // The whole warp runs the loop (addresses stay uniform values), one
        // elected lane issues.
        {
            uint32_t armed = 0, armed_parity = 0, ph = 0;
            int s = 0;
            bool ok = true, stall = p.debug_stall != 0;        // test hook: the first stage is never filled
            for (int t = unit; ok && t < p.num_tiles; t += p.units) {
                int mb, nb;
                tile_coords(t, p, mb, nb);
                const int row = mb * S::TM + (int)rank * 128;
                const int col = nb * S::TN + (int)rank * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(~0u, mbar_wait<true, PAIR>(smem_u32(&sy->empty[s]), ph ^ 1u, wait));
                    if (!ok) break;
                    if (!stall) {
                    if (elect_one()) {
                    const uint32_t full = full0 + (uint32_t)(s * sizeof(uint64_t));
                    if (leader) mbar_arrive_expect_tx(smem_u32(&sy->full[s]), (PAIR ? 2 : 1) * S::STAGE_BYTES);
                    const uint32_t a = codes0 + s * 2 * OPERAND_BYTES;
                    const uint32_t sf = scales0 + s * (S::SFA_BYTES + S::SFB_BYTES);
                    tma_load_2d<PAIR>(a, &tmA, kb * SW, row, full);
                    tma_load_2d<PAIR>(a + OPERAND_BYTES, &tmB, kb * SW, col, full);
                    tma_load_3d<PAIR>(sf, &tmSA, 0, kb * S::SF_TILES, row / 128, full);
                    tma_load_3d<PAIR>(sf + S::SFA_BYTES, &tmSB, 0, kb * S::SF_TILES, nb * (S::TN / 128), full);
                    }
                    armed |= 1u << s;
                    armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
                    }
                    stall = false;
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (leader) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait<false, PAIR>(smem_u32(&sy->full[s]), (armed_parity >> s) & 1u, wait);
            } else if (*(volatile int*)&sy->abort) {
                // After a timeout this block cannot observe its own copies;
                // give any in flight time to land (a copy takes microseconds).
                const unsigned long long t0 = globaltimer();
                while (globaltimer() - t0 < 2000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        // The whole warp runs the loop, so that addresses and descriptors are
        // uniform values; one elected lane issues.
        if (leader) {
            int it = 0, s = 0;
            uint32_t ph = 0;
            bool ok = true;
            // A tile's sum, or of LONG ones each part in turn: first to last - 1.
            for (int t = unit, first = kb0; ok && t < p.num_tiles; ++it) {
                const int last = LONG ? min(first + PART_STAGES, kb1) : kb1;
                // Pair: the previous sum's shared columns have left tensor
                // memory (and with them all of the sum before it). Single:
                // the sum two before, which used this accumulator.
                if (PAIR ? it >= 1 : it >= 2)
                    if (!__all_sync(~0u, mbar_wait<true, PAIR>(smem_u32(&sy->tmem_empty[PAIR ? 0 : it & 1]),
                                                     (uint32_t)(PAIR ? it - 1 : (it >> 1) - 1) & 1u, wait)))
                        break;
                tc_fence_after();
                const uint32_t d = tmem_base + ((it & 1) ? S::ACC1 : 0);
                const uint32_t sfa = tmem_base + S::SF, sfb = sfa + S::SF_TILES * 4;
                for (int kb = first; kb < last; ++kb) {
                    ok = __all_sync(~0u, mbar_wait<true, PAIR>(smem_u32(&sy->full[s]), ph, wait));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                    const uint32_t sf = scales0 + s * (S::SFA_BYTES + S::SFB_BYTES);
#pragma unroll
                    for (int k = 0; k < S::SF_TILES; ++k) {
                        copy_scale_tile<PAIR>(sfa + k * 4, sf + k * MX4_TILE_BYTES);
#pragma unroll
                        for (int n = 0; n < S::TN / 128; ++n)
                            copy_scale_tile<PAIR>(sfb + (k * (S::TN / 128) + n) * 4,
                                                  sf + S::SFA_BYTES + (n * S::SF_TILES + k) * MX4_TILE_BYTES);
                    }
                    const uint32_t a = codes0 + s * 2 * OPERAND_BYTES;
#pragma unroll
                    for (int k = 0; k < STAGE_K / 64; ++k) {
                        const int tile = FMT == TGEMM_MXFP4 ? k / 2 : k;
                        const uint32_t half = FMT == TGEMM_MXFP4 ? (k & 1) * 2 : 0;
                        mma_mx4<FMT, PAIR>(d, smem_desc(a + k * 32, 16, 1024, 2),
                                           smem_desc(a + OPERAND_BYTES + k * 32, 16, 1024, 2),
                                           mx4_instr<FMT, S::TM, S::TN>(half), sfa + tile * 4,
                                           sfb + tile * 4 * (S::TN / 128), kb != first || k != 0);
                    }
                    tc_commit<PAIR>(smem_u32(&sy->empty[s]));
                    if (kb == last - 1) tc_commit<PAIR>(smem_u32(&sy->tmem_full[it & 1]));
                    }
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
                first = last;
                if (last == kb1) {
                    first = kb0;
                    t += p.units;
                }
            }
            if (elect_one()) tc_commit<PAIR>(smem_u32(&sy->drain));
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                            // tensor-memory lanes 32 q .. 32 q + 31
        const int set = (warp - 2) >> 2;
        uint8_t* bufs = epi + (warp - 2) * S::BUFS * BUF_BYTES;
        const float ga = mx4_g(p.ga), gb = mx4_g(p.gb);
        int it = 0;
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 31) {
                const uint32_t bar = tmem_empty0 + (uint32_t)((PAIR ? 0 : it & 1) * sizeof(uint64_t));
                if constexpr (PAIR) mbar_arrive_cluster(bar); else mbar_arrive(bar);
            }
        };
        if constexpr (LONG) {
            // This set's half of the row, 64 columns a turn. The turn that may
            // hold columns which the other accumulator shares -- a pair's first
            // 64, set 0's, or last, set 1's -- comes first, and then the next
            // part may start.
            constexpr int HALF = S::TN / 2, TURNS = HALF / 64;
            bool ok = true;
            for (int t = unit; ok && t < p.num_tiles; t += p.units) {
                float sum[TURNS][2][32] = {};            // (a first part that is moved instead of added: more registers)
                #pragma unroll 1
                for (int first = kb0; first < kb1; first += PART_STAGES, ++it) {
                    ok = __all_sync(~0u, mbar_wait<true, PAIR, true>(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem_base + ((it & 1) ? S::ACC1 : 0) + ((uint32_t)(q * 32) << 16) + set * HALF;
#pragma unroll
                    for (int i = 0; i < TURNS; ++i) {
                        const uint32_t from = acc + (i ^ (TURNS > 1 ? set : 0)) * 64;
#pragma unroll
                        for (int c = 0; c < 64; c += 16) {
                            uint32_t r[16];
                            tmem_ld16(from + c, r);
                            tmem_wait_ld(r);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[i][c / 32][c % 32 + j] += __uint_as_float(r[j]);
                        }
                        if (i == 0) release();
                    }
                }
                if (!ok) break;
                if (!PAIR && p.split > 1) {
                    // The tile's copies and MMAs are done: its stages hold the share.
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        share_columns(smem, q * 32 + lane, set * HALF + h * 32, reinterpret_cast<uint32_t (&)[32]>(sum[0][h]));
                    break;
                }
                int mb, nb;
                tile_coords(t, p, mb, nb);
                const int row0 = mb * S::TM + (int)rank * 128 + q * 32;
#pragma unroll
                for (int i = 0; i < TURNS; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        store_half<S::BUFS, TC>(p, &tmC, bufs, i, h, row0, min(32, p.M - row0),
                                                nb * S::TN + set * HALF + (i ^ (TURNS > 1 ? set : 0)) * 64, ga, gb,
                                                reinterpret_cast<uint32_t (&)[32]>(sum[i][h]));
            }
        } else
        for (int t = unit; t < p.num_tiles; t += p.units, ++it) {
            int mb, nb;
            tile_coords(t, p, mb, nb);
            const bool ok = mbar_wait<true, PAIR>(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (!PAIR && p.split > 1) {
                // The tile's copies and MMAs are done: its stages hold the share.
                if (set == 0) store_share(smem, tmem_base + ((uint32_t)(q * 32) << 16), q);
                break;
            }
            // Pair: the next tile may start once the shared columns, turn 0,
            // are out; single: once this accumulator is.
            drain_tile<S::TN, S::SETS, true, S::BUFS, TC>(
                p, &tmC, tmem_base + ((it & 1) ? S::ACC1 : 0) + ((uint32_t)(q * 32) << 16), bufs,
                mb * S::TM + (int)rank * 128 + q * 32, nb * S::TN, PAIR && !(it & 1), set,
                PAIR ? 0 : S::TN / 64 - S::SETS + set, ga, gb, release);
        }
        tma_store_wait_all();
    }

    tc_fence_before();
    if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
    tc_fence_after();
    if (!PAIR && p.split > 1) {
        int mb, nb;
        tile_coords(unit, p, mb, nb);
        join_shares<TC>(p, smem, 128, part, mb * S::TM, nb * S::TN, mx4_g(p.ga), mx4_g(p.gb));
    }
    if (warp == 1) tmem_free<PAIR, TMEM_COLS>(tmem_base);
}

// K == 0: acc is 0.
template <typename TC>
__global__ void __launch_bounds__(256) empty_sum_kernel(int M, int N, const Mx4Out out) {
    pdl_launch_dependents();
    pdl_wait();
    const long c = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= N) return;
    for (long r = blockIdx.y; r < M; r += gridDim.y)
        mx4_store(static_cast<TC*>(out.C) + r * out.ldc + c, 0.0f, 1.0f, 1.0f, out, (int)c);
}

template <int FMT, bool PAIR, bool LONG, typename TC>
cudaError_t launch_kernel(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmSA, const CUtensorMap& tmSB,
                          const CUtensorMap& tmC, const Params& p, cudaStream_t s) {
    using S = Shape<FMT, PAIR, LONG>;
    const cudaError_t e = set_smem_limit_once<mx4_gemm_kernel<FMT, PAIR, LONG, TC>>(S::SMEM);
    if (e != cudaSuccess) return e;
    ClusterLaunch cfg((PAIR ? 2 : p.split) * p.units, S::THREADS, S::SMEM, PAIR ? 2 : p.split, s);
    return cudaLaunchKernelEx(&cfg.config, mx4_gemm_kernel<FMT, PAIR, LONG, TC>, tmA, tmB, tmSA, tmSB, tmC, p);
}

template <int FMT, bool PAIR, typename TC>
cudaError_t launch(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, const Mx4Out& out,
                   int num_sms, cudaStream_t s) {
    using S = Shape<FMT, PAIR, false>;
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    CUtensorMap tmA, tmB, tmSA, tmSB, tmC;
    if (!encode_codes(enc, &tmA, A, M, K) || !encode_codes(enc, &tmB, B, N, K) ||
        !encode_scales(enc, &tmSA, A, M, K, FMT, S::SF_TILES, 1) ||
        !encode_scales(enc, &tmSB, B, N, K, FMT, S::SF_TILES, S::TN / 128))
        return cudaErrorInvalidValue;
    memset(&tmC, 0, sizeof(tmC));
    Params p;
    cudaError_t e = make_tiling(p, M, N, S::TM, S::TN, PAIR ? num_sms / 2 : num_sms, out);
    p.kblocks = (int)(((long)K + STAGE_K - 1) / STAGE_K);
    p.ga = A.g; p.gb = B.g;
    p.tma_c = encode_c(enc, &tmC, out, M, N) ? 1 : 0;
    if (!PAIR && p.num_tiles * 2 <= num_sms) {
        // 10 steps: 128 x 2048 x 2048, 6 saved, whole 5.5 us and split 6.3;
        // x 4096, 12 saved, 7.8 and 6.9; 1024 x 1024 x 4096, 8 saved, 8.4 and 9.2.
        unsigned long long fits = 0;
        if (e == cudaSuccess) e = set_smem_limit_once<mx4_gemm_kernel<FMT, PAIR, false, TC>>(S::SMEM);
        if (e == cudaSuccess) e = clusters_that_fit<mx4_gemm_kernel<FMT, PAIR, false, TC>>(S::THREADS, S::SMEM, &fits);
        p.split = split_for(p.num_tiles, p.kblocks, fits, 10);
        p.units = p.num_tiles;
    }
    if (e != cudaSuccess) return e;
    if constexpr (sizeof(TC) == 4)
        if ((p.kblocks + p.split - 1) / p.split > PART_STAGES)
            return launch_kernel<FMT, PAIR, true, TC>(tmA, tmB, tmSA, tmSB, tmC, p, s);
    return launch_kernel<FMT, PAIR, false, TC>(tmA, tmB, tmSA, tmSB, tmC, p, s);
}

template <int FMT, bool PAIR>
cudaError_t launch_type(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, const Mx4Out& out,
                        int num_sms, cudaStream_t s) {
    return out.c_type == TGEMM_TYPE_F32 ? launch<FMT, PAIR, float>(M, N, K, A, B, out, num_sms, s)
                                        : launch<FMT, PAIR, __nv_bfloat16>(M, N, K, A, B, out, num_sms, s);
}

}  // namespace

cudaError_t mx4_status_word(int** word) {
    static std::atomic<int*> known[64];                   // looked up once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*word = known[dev].load(std::memory_order_acquire)) != nullptr) return cudaSuccess;
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_mx4_status);
    *word = static_cast<int*>(p);
    if (e == cudaSuccess && dev < 64) known[dev].store(*word, std::memory_order_release);
    return e;
}

cudaError_t mx4_read_and_clear_status(int* status, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(status, g_mx4_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *status == 0) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_mx4_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e != cudaSuccess ? e : cudaStreamSynchronize(s);
}

cudaError_t mx4_empty_sum(int M, int N, const Mx4Out& out, cudaStream_t s) {
    const dim3 grid((unsigned)(((long)N + 255) / 256), (unsigned)(M < 32768 ? M : 32768));
    return out.c_type == TGEMM_TYPE_F32
               ? launch_pdl(empty_sum_kernel<float>, grid, dim3(256), 0, s, M, N, out)
               : launch_pdl(empty_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, M, N, out);
}

cudaError_t mx4_gemm(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, int fmt,
                     const Mx4Out& out, int num_sms, cudaStream_t s) {
    if (K == 0) return mx4_empty_sum(M, N, out, s);
    if (use_pair(M, N, num_sms))
        return fmt == TGEMM_MXFP4 ? launch_type<TGEMM_MXFP4, true>(M, N, K, A, B, out, num_sms, s)
                                  : launch_type<TGEMM_NVFP4, true>(M, N, K, A, B, out, num_sms, s);
    return fmt == TGEMM_MXFP4 ? launch_type<TGEMM_MXFP4, false>(M, N, K, A, B, out, num_sms, s)
                              : launch_type<TGEMM_NVFP4, false>(M, N, K, A, B, out, num_sms, s);
}

}  // namespace tgemm
