// BF16 rows times a kept 4-bit matrix, C = alpha A W^T + beta C + bias, on the
// tensor cores (tcgen05, kind f16): W is made BF16 on its way through shared
// memory. (C of few tiles goes to mx4_weights_tmem.cu, few rows to
// mx4_weights_rows.cu.)
//
// The form is that of gemm_mx4's kernel for many tiles -- 256 x 256 tiles on SM
// pairs, persistent, two accumulators in tensor memory (which leave no room
// there for W) -- with eight more warps: TMA brings A's rows (64 columns of K,
// one pipeline stage) and, in chunks of 256 columns, W's codes and scales; the
// eight warps, two on each of a chunk's four stages, turn 128 rows x 64 codes
// into the 128-byte-swizzled BF16 that the MMA reads, and arrive on the
// stage's barrier beside A's bytes. A thread takes 32 codes of a row: one
// 16-byte read, one or two scales, four 16-byte writes. 8192 x 14336 x 4096
// MXFP4: 513 us, 640 cycles a stage for 512 of MMAs.

#include "mx4_decode.h"
#include "mx4_tile.h"

#include <cstring>

namespace tgemm {
namespace {

using namespace mx4_tile;
using namespace mx4_decode;

constexpr int STAGE_K = 64;
constexpr int OPERAND_BYTES = 128 * SW;              // 128 rows x 64 BF16
// Codes come in chunks of as many stages as there are groups of decoding
// warps, so that a group meets each chunk once.
constexpr int CHUNK_K = 256, CHUNKS = 2;
constexpr int EPI_WARPS = 4;
constexpr int EPI_BYTES = EPI_WARPS * BUF_BYTES;
constexpr int STAGES = 5;
constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;       // a block's rows of A and of W
constexpr int DECODE_WARPS = 8;
constexpr int GROUPS = 4;                          // the decoding warps' groups, each on its own stages
constexpr int GROUP_WARPS = DECODE_WARPS / GROUPS;
constexpr int CODES_WARP = 2 + EPI_WARPS + DECODE_WARPS;
constexpr int THREADS = 32 * (CODES_WARP + 1);

constexpr int CHUNK_STAGES = CHUNK_K / STAGE_K;
constexpr int ROW = CHUNK_K / 2;                     // bytes of a row of a chunk's codes
constexpr int CODES_BYTES = 128 * ROW;
template <int FMT> constexpr int SF_TILES = CHUNK_K / mx4_block(FMT) / 4;
template <int FMT> constexpr int SF_BYTES = SF_TILES<FMT> * MX4_TILE_BYTES;

struct Sync {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t codes_full[CHUNKS], codes_empty[CHUNKS];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    uint32_t factors[256];
};
constexpr int SYNC_BYTES = 1408;
static_assert(sizeof(Sync) <= SYNC_BYTES, "barrier block");

template <int FMT>
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + CHUNKS * (CODES_BYTES + SF_BYTES<FMT>) + EPI_BYTES + SYNC_BYTES;
static_assert(SMEM<TGEMM_NVFP4> <= 227 * 1024, "shared memory");
// A warp that waits for a slot has seen the slot's last use but one freed only
// if its previous stage was at most as many stages back as there are slots
// (barriers tell phases apart by parity).
static_assert(STAGES >= GROUPS && CHUNK_STAGES == GROUPS && ROW == SW, "slots, chunks and groups");

struct Params : Tiling {
    int kblocks;                // of 64 columns
    // The sum of a tile in `parts` parts (a long one, FP32 C): each is made in
    // the second accumulator and added to the first (8192 x 14336 x 4096 MXFP4
    // with FP32 C: 615 us, in one part 541).
    int parts, part_blocks;
    const float* gb;
};

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

template <int FMT, typename TC>
__global__ void __launch_bounds__(THREADS, 1)
weights_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmC,
               const Params p) {
    constexpr int TM = 256, TN = 256, A_BYTES = OPERAND_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* codes = smem + STAGES * STAGE_BYTES;
    uint8_t* epi = codes + CHUNKS * CODES_BYTES;               // 1 KB aligned, as its swizzle wants
    uint8_t* scales = epi + EPI_BYTES;
    Sync* sy = reinterpret_cast<Sync*>(scales + CHUNKS * SF_BYTES<FMT>);
    const uint32_t stage0 = smem_u32(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int unit = blockIdx.x >> 1;
    const int chunks = (p.kblocks + CHUNK_STAGES - 1) / CHUNK_STAGES;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // A's bytes of both blocks, and the decoding warps' arrivals.
            mbar_init(smem_u32(&sy->full[s]), 1 + 2 * GROUP_WARPS);
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int c = 0; c < CHUNKS; ++c) {
            mbar_init(smem_u32(&sy->codes_full[c]), 1);
            mbar_init(smem_u32(&sy->codes_empty[c]), DECODE_WARPS);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->tmem_full[a]), 1);
            mbar_init(smem_u32(&sy->tmem_empty[a]), 2 * EPI_WARPS);
        }
        mbar_init(smem_u32(&sy->drain), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        prefetch_map(&tmSB);
    }
    if (threadIdx.x < 256) sy->factors[threadIdx.x] = factor<FMT>(threadIdx.x);
    if (warp == 1) tmem_alloc<true, TMEM_COLS>(smem_u32(&sy->tmem_base));
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = sy->tmem_base;
    pdl_launch_dependents();
    pdl_wait();

    const Wait wait{&sy->abort, p.status, p.wait_limit_ns};
    // The leader's barriers, as cluster addresses.
    const uint32_t full0 = map_to_rank(smem_u32(&sy->full[0]), 0);
    const uint32_t tmem_empty0 = map_to_rank(smem_u32(&sy->tmem_empty[0]), 0);

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        uint32_t armed = 0, armed_parity = 0, ph = 0;
        int s = 0;
        bool ok = true, stall = p.debug_stall != 0;        // test hook: the first stage is never filled
        for (int t = unit; ok && t < p.num_tiles; t += p.units) {
            int mb, nb;
            tile_coords(t, p, mb, nb);
            const int row = mb * TM + (int)rank * 128;
            for (int kb = 0; kb < p.kblocks; ++kb) {
                ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->empty[s]), ph ^ 1u, wait));
                if (!ok) break;
                if (!stall) {
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(smem_u32(&sy->full[s]), 2 * A_BYTES);
                        tma_load_2d<true>(stage0 + s * STAGE_BYTES, &tmA, kb * STAGE_K, row,
                                          full0 + (uint32_t)(s * sizeof(uint64_t)));
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
            for (int i = 0; i < STAGES; ++i)
                if (armed & (1u << i))
                    mbar_wait<false, true>(smem_u32(&sy->full[i]), (armed_parity >> i) & 1u, wait);
        } else if (*(volatile int*)&sy->abort) {
            // After a timeout this block cannot observe its own copies; give
            // any in flight time to land (a copy takes microseconds).
            const unsigned long long t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        if (leader) {
            constexpr uint32_t IDESC = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(TN >> 3) << 17 | (uint32_t)(TM >> 4) << 24;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int t = unit + i / p.parts * p.units, part = i % p.parts;
                if (t >= p.num_tiles) break;
                // What this accumulator held before is out.
                const int acc = p.parts > 1 ? 1 : i & 1, turn = p.parts > 1 ? i : i >> 1;
                ok = turn == 0 || __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->tmem_empty[acc]), (uint32_t)(turn - 1) & 1u, wait));
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * TN);
                const int first = part * p.part_blocks, last = min(first + p.part_blocks, p.kblocks) - 1;
                for (int kb = first; kb <= last; ++kb) {
                    ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->full[s]), ph, wait));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t a = stage0 + s * STAGE_BYTES;
#pragma unroll
                        for (int k = 0; k < STAGE_K / 16; ++k)
                            mma_bf16(d, smem_desc(a + k * 32, 16, 1024, 2), smem_desc(a + A_BYTES + k * 32, 16, 1024, 2),
                                     IDESC, kb != first || k != 0);
                        tc_commit<true>(smem_u32(&sy->empty[s]));
                        if (kb == last) tc_commit<true>(smem_u32(&sy->tmem_full[acc]));
                    }
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (elect_one()) tc_commit<true>(smem_u32(&sy->drain));
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else if (warp < 2 + EPI_WARPS) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                            // tensor-memory lanes 32 q .. 32 q + 31
        uint8_t* bufs = epi + (warp - 2) * BUF_BYTES;
        const float gb = mx4_g(p.gb);
        const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
        bool ok = true;
        uint32_t it = 0;
        for (int t = unit; ok && t < p.num_tiles; t += p.units) {
            int mb, nb;
            tile_coords(t, p, mb, nb);
            auto release = [&](int acc) {
                tc_fence_before();
                __syncwarp();
                if (lane == 31) mbar_arrive_cluster(tmem_empty0 + (uint32_t)(acc * sizeof(uint64_t)));
            };
            const int row0 = mb * TM + (int)rank * 128 + q * 32;
            bool stored = false;
            if constexpr (sizeof(TC) == 4) {
                if (p.parts > 1) {
                    for (int part = 0; ok && part < p.parts; ++part, ++it) {
                        ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->tmem_full[1]), it & 1u, wait));
                        if (!ok) break;
                        tc_fence_after();
                        add_sums(lanes, lanes + TN, TN, part == 0);
                        release(1);
                    }
                    if (!ok) break;
                    drain_tile<TN, 1, false, 1, TC>(p, &tmC, lanes, bufs, row0, nb * TN, false, 0, TN / 64 - 1,
                                                    unscale<FMT>(), gb, [] {});
                    stored = true;
                }
            }
            if (!stored) {
                const int acc = (int)(it & 1);
                ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->tmem_full[acc]), it >> 1 & 1u, wait));
                if (!ok) break;
                ++it;
                tc_fence_after();
                drain_tile<TN, 1, false, 1, TC>(p, &tmC, lanes + (uint32_t)(acc * TN), bufs, row0, nb * TN, false, 0,
                                                TN / 64 - 1, unscale<FMT>(), gb, [&] { release(acc); });
            }
        }
        tma_store_wait_all();
    } else if (warp == CODES_WARP) {
        // ---------------------------------------- TMA producer of the codes
        // A warp of its own: it runs as far ahead as there are chunks, A's
        // producer as far as there are slots.
        uint32_t armed = 0, armed_parity = 0, ph = 0;
        int c = 0;
        bool ok = true;
        for (int t = unit; ok && t < p.num_tiles; t += p.units) {
            int mb, nb;
            tile_coords(t, p, mb, nb);
            const int col = nb * TN + (int)rank * 128;
            for (int ch = 0; ch < chunks; ++ch) {
                ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->codes_empty[c]), ph ^ 1u, wait));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = smem_u32(&sy->codes_full[c]);
                    mbar_arrive_expect_tx(bar, CODES_BYTES + SF_BYTES<FMT>);
                    tma_load_2d<false>(smem_u32(codes) + c * CODES_BYTES, &tmB, ch * ROW, col, bar);
                    tma_load_3d<false>(smem_u32(scales) + c * SF_BYTES<FMT>, &tmSB, 0, ch * SF_TILES<FMT>,
                                       col / 128, bar);
                }
                __syncwarp();
                armed |= 1u << c;
                armed_parity = (armed_parity & ~(1u << c)) | (ph << c);
                if (++c == CHUNKS) { c = 0; ph ^= 1u; }
            }
        }
        for (int i = 0; i < CHUNKS; ++i)
            if (armed & (1u << i)) mbar_wait<false>(smem_u32(&sy->codes_full[i]), (armed_parity >> i) & 1u, wait);
    } else {
        // ------------------------------------------------------ decoding
        // Group i takes stages i, i + GROUPS, .. of the block's. A stage's
        // values are made before its slot is free: between a slot's release
        // and its readiness lie only the writes, their fence and the arrival.
        // All groups release each chunk, in a tile's last one those without a
        // stage too.
        const int dw = warp - 2 - EPI_WARPS, group = dw / GROUP_WARPS;
        const int tid = dw % GROUP_WARPS * 32 + lane;
        constexpr int ITEMS = 256 / (32 * GROUP_WARPS);          // runs of 32 codes a thread and stage
        uint32_t cph = 0, sph = 1;                               // parities to wait for
        int c = 0, s = group, next = group;                      // this group's next stage: its slot, its K block
        bool ok = true;
        for (int t = unit; ok && t < p.num_tiles; t += p.units, next -= p.kblocks) {
            for (int ch = 0; ch < chunks; ++ch) {
                ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->codes_full[c]), cph, wait));
                if (!ok) break;
                if (next < min((ch + 1) * CHUNK_STAGES, p.kblocks)) {
                    const int q = next - ch * CHUNK_STAGES;
                    uint4 w[ITEMS];
                    uint32_t b0[ITEMS], b1[ITEMS];
                    bool is_wide = false;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        const int item = i * 32 * GROUP_WARPS + tid, row = item & 127, half = item >> 7;
                        w[i] = *reinterpret_cast<const uint4*>(codes + c * CODES_BYTES + swizzled(row, q * 2 + half));
                        const uint8_t* sc = scales + c * SF_BYTES<FMT> + (row & 31) * 16 + (row >> 5) * 4;
                        if (FMT == TGEMM_MXFP4) {
                            b0[i] = b1[i] = sc[(q >> 1) * MX4_TILE_BYTES + (q & 1) * 2 + half];
                            is_wide |= wide(b0[i]);
                        } else {
                            const uint32_t two = *reinterpret_cast<const uint16_t*>(sc + q * MX4_TILE_BYTES + half * 2);
                            b0[i] = two & 0xFF;
                            b1[i] = two >> 8;
                        }
                    }
                    is_wide = FMT == TGEMM_MXFP4 && __any_sync(~0u, is_wide);
                    uint4 v[ITEMS][4];
                    if (is_wide) {
#pragma unroll
                        for (int i = 0; i < ITEMS; ++i) {
                            // Beside a wide block the others take their scale alone too.
                            const uint32_t f = b0[i] == 255 ? 0x7FC07FC0u : b0[i] == 0 ? 0x00400040u : b0[i] << 7 | b0[i] << 23;
                            decode_run<true>(v[i], w[i], f, f);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < ITEMS; ++i) {
                            const uint32_t f0 = sy->factors[b0[i]];
                            decode_run<false>(v[i], w[i], f0, FMT == TGEMM_MXFP4 ? f0 : sy->factors[b1[i]]);
                        }
                    }
                    ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->empty[s]), sph, wait));
                    if (!ok) break;
                    uint8_t* dst = smem + s * STAGE_BYTES + A_BYTES;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        const int item = i * 32 * GROUP_WARPS + tid, row = item & 127, half = item >> 7;
#pragma unroll
                        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(dst + swizzled(row, half * 4 + j)) = v[i][j];
                    }
                    fence_async_smem();          // the MMA reads through the async proxy
                    __syncwarp();
                    if (lane == 0) {
                        release_smem();
                        mbar_arrive_cluster(full0 + (uint32_t)(s * sizeof(uint64_t)));
                    }
                    next += GROUPS;
                    s += GROUPS;
                    if (s >= STAGES) { s -= STAGES; sph ^= 1u; }
                }
                if (lane == 0) mbar_arrive(smem_u32(&sy->codes_empty[c]));
                if (++c == CHUNKS) { c = 0; cph ^= 1u; }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_free<true, TMEM_COLS>(tmem_base);
}

template <int FMT, typename TC>
cudaError_t launch(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, const Mx4Out& out,
                   int num_sms, cudaStream_t s) {
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    CUtensorMap tmA, tmB, tmSB, tmC;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M}, strides[1] = {(cuuint64_t)lda * 2};
    const cuuint32_t box[2] = {STAGE_K, 128};
    if (!encode(enc, &tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, A, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_codes(enc, &tmB, B, N, K) || !encode_scales(enc, &tmSB, B, N, K, FMT, SF_TILES<FMT>, 1))
        return cudaErrorInvalidValue;
    memset(&tmC, 0, sizeof(tmC));
    Params p;
    cudaError_t e = make_tiling(p, M, N, 256, 256, num_sms / 2, out);
    p.kblocks = (int)(((long)K + STAGE_K - 1) / STAGE_K);
    p.part_blocks = sizeof(TC) == 4 ? SUM_K / STAGE_K : p.kblocks;
    p.parts = (p.kblocks + p.part_blocks - 1) / p.part_blocks;
    p.gb = B.g;
    p.tma_c = encode_c(enc, &tmC, out, M, N) ? 1 : 0;
    if (e == cudaSuccess) e = set_smem_limit_once<weights_kernel<FMT, TC>>(SMEM<FMT>);
    if (e != cudaSuccess) return e;
    ClusterLaunch cfg(2 * p.units, THREADS, SMEM<FMT>, 2, s);
    return cudaLaunchKernelEx(&cfg.config, weights_kernel<FMT, TC>, tmA, tmB, tmSB, tmC, p);
}

template <int FMT>
cudaError_t launch_type(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, const Mx4Out& out,
                        int num_sms, cudaStream_t s) {
    return out.c_type == TGEMM_TYPE_F32 ? launch<FMT, float>(M, N, K, A, lda, B, out, num_sms, s)
                                        : launch<FMT, __nv_bfloat16>(M, N, K, A, lda, B, out, num_sms, s);
}

cudaError_t run(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt, const Mx4Out& out,
                int num_sms, cudaStream_t s) {
    if (use_pair(M, N, num_sms))
        return fmt == TGEMM_MXFP4 ? launch_type<TGEMM_MXFP4>(M, N, K, A, lda, B, out, num_sms, s)
                                  : launch_type<TGEMM_NVFP4>(M, N, K, A, lda, B, out, num_sms, s);
    return mx4_weights_tmem(M, N, K, A, lda, B, fmt, out, s);
}

}  // namespace

cudaError_t mx4_weights(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt,
                        const Mx4Out& out, int num_sms, cudaStream_t s) {
    if (K == 0) return mx4_empty_sum(M, N, out, s);
    // (Its offsets within 32 rows of codes are 32-bit.)
    if (mx4_few_rows(M, N, K) && K < 1 << 27) return mx4_weights_rows(M, N, K, A, lda, B, fmt, out, num_sms, s);
    if (reinterpret_cast<uintptr_t>(A) % 16 == 0 && lda % 8 == 0)
        return run(M, N, K, A, lda, B, fmt, out, num_sms, s);
    // TMA copies rows that start on 16-byte boundaries: others are repacked.
    const long ld = ((long)K + 63) / 64 * 64;
    void* packed = nullptr;
    cudaError_t e = scratch_take(&packed, (size_t)M * ld * 2, s);
    if (e != cudaSuccess) return e;
    e = repack_rows(A, lda, packed, ld, M, K, 2, s);
    if (e == cudaSuccess) e = run(M, N, K, packed, ld, B, fmt, out, num_sms, s);
    const cudaError_t f = cudaFreeAsync(packed, s);
    return e != cudaSuccess ? e : f;
}

}  // namespace tgemm
