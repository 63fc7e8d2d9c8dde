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
// Two forms, both persistent, one block on an SM, six warps (0: TMA, 1: MMA,
// 2-5: epilogue):
//   pair    256 x 256 tiles on an SM pair (cta_group::2). Each block stages
//           its 128 rows of A, its 128 rows of B, A's scales for its rows
//           and B's for all 256. Two accumulators of 256 columns and 48
//           columns of scales do not fit the 512 of tensor memory, so the
//           accumulators share 48 columns: the epilogue drains the shared
//           ones first and then lets the next tile's MMAs start.
//   single  128 x 128 tiles on one SM, for products with few tiles.
//
// Rows past M and N are read as zeros (TMA fill, zero scales) and not stored.
// Waits are bounded as in the other tensor-core kernels.

#include "mx4_ptx.h"

#include <cstring>

namespace tgemm {

__device__ int g_mx4_status;

namespace {

using namespace mx4_ptx;

constexpr int SW = 128;                       // bytes of a staged row: 256 codes
constexpr int STAGE_K = MX4_SPAN;
constexpr int OPERAND_BYTES = 128 * SW;       // 128 rows of codes
constexpr int STAGES = 5;
constexpr int THREADS = 192;
constexpr int EPI_WARPS = 4;
constexpr int BUF_BYTES = 32 * 128;           // 32 rows x 128 bytes of C
constexpr int EPI_BYTES = EPI_WARPS * 2 * BUF_BYTES;
constexpr int TMEM_COLS = 512;
constexpr int GROUP_M = 8;

template <int FMT, bool PAIR>
struct Shape {
    static constexpr int TM = PAIR ? 256 : 128;           // rows of a tile
    static constexpr int TN = PAIR ? 256 : 128;           // columns
    static constexpr int SF_TILES = STAGE_K / mx4_block(FMT) / 4;     // scale tiles of 128 rows a stage
    static constexpr int SFA_BYTES = SF_TILES * MX4_TILE_BYTES;
    static constexpr int SFB_BYTES = SFA_BYTES * (TN / 128);
    static constexpr int STAGE_BYTES = 2 * OPERAND_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 256;
    // Tensor memory: accumulators at 0 and ACC1, scales from SF on.
    static constexpr int SF_COLS = SF_TILES * 4 * (1 + TN / 128);
    static constexpr int SF = PAIR ? 464 : 256;
    static constexpr int ACC1 = PAIR ? SF - TN : 128;
    static constexpr int FREE_FIRST = PAIR ? 64 : TN;     // columns drained before the next tile may start
    static_assert(SF + SF_COLS <= TMEM_COLS && TN - ACC1 <= FREE_FIRST, "tensor memory");
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

struct Params {
    int M, N, kblocks;
    int tiles_m, tiles_n, num_tiles, units;
    const float *ga, *gb;
    Mx4Out out;
    int tma_c;                  // C leaves by TMA stores
    unsigned long long wait_limit_ns;
    int* status;
    int debug_stall;
};

__device__ __forceinline__ void tile_coords(int t, const Params& p, int& mb, int& nb) {
    const int per_group = GROUP_M * p.tiles_n;
    const int first = t / per_group * GROUP_M;
    const int gm = min(p.tiles_m - first, GROUP_M);
    mb = first + t % per_group % gm;
    nb = t % per_group / gm;
}

// Where 16-byte piece j of row r lies in a 128-byte-swizzled buffer.
__device__ __forceinline__ uint32_t swizzled(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// Drains this warp's 32 rows of a tile, 64 columns a turn. `last_first`: the
// last 64 columns, which the next tile's accumulator shares, go first.
// release() is called as soon as FREE_FIRST columns have left tensor memory.
template <typename S, typename TC, typename Release>
__device__ __forceinline__ void drain_tile(const Params& p, const CUtensorMap* tmC, uint32_t tmem,
                                           uint8_t* bufs, int row0, int col0, bool last_first,
                                           float ga, float gb, Release release) {
    constexpr int W = 64;
    constexpr int TURNS = S::TN / W, REL = S::FREE_FIRST / W;
    const int lane = threadIdx.x & 31;
    const Mx4Out& o = p.out;
#pragma unroll 1
    for (int i = 0; i < TURNS; ++i) {
        const int part = last_first ? (i == 0 ? TURNS - 1 : i - 1) : i;
        const int col = col0 + part * W;
        uint32_t r[2][32];
        tmem_ld32(tmem + (uint32_t)(part * W), r[0]);
        tmem_ld32(tmem + (uint32_t)(part * W + 32), r[1]);
        tmem_wait_ld(r[0]);
        tmem_wait_ld(r[1]);
        if (i == REL - 1) release();
        if (p.tma_c) {
            // FP32: two boxes of 32 columns, BF16: one of 64. The previous
            // turn's boxes have to have left the buffers.
            if (lane == 0) tma_store_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float v = __uint_as_float(r[h][j]) * ga * gb * o.alpha;
                    if (o.bias != nullptr && col + h * 32 + j < p.N) v += __ldg(o.bias + col + h * 32 + j);
                    r[h][j] = __float_as_uint(v);
                }
                if constexpr (sizeof(TC) == 4) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(bufs + h * BUF_BYTES + swizzled(lane, j)) =
                            make_uint4(r[h][4 * j], r[h][4 * j + 1], r[h][4 * j + 2], r[h][4 * j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[h][8 * j + 2 * k]),
                                                                           __uint_as_float(r[h][8 * j + 2 * k + 1]));
                            w[k] = *reinterpret_cast<const uint32_t*>(&b);
                        }
                        *reinterpret_cast<uint4*>(bufs + swizzled(lane, h * 4 + j)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.M) {
                if (col < p.N) tma_store_2d(tmC, col, row0, smem_u32(bufs));
                if (sizeof(TC) == 4 && col + 32 < p.N) tma_store_2d(tmC, col + 32, row0, smem_u32(bufs) + BUF_BYTES);
            }
        } else {
            // Any alignment, and beta: 32 x 32 FP32 blocks through shared
            // memory, then whole row segments under the output rule.
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(bufs + h * BUF_BYTES + swizzled(lane, j)) =
                        make_uint4(r[h][4 * j], r[h][4 * j + 1], r[h][4 * j + 2], r[h][4 * j + 3]);
            __syncwarp();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int c = col + h * 32 + lane;
                if (c >= p.N) continue;
                TC* out = static_cast<TC*>(o.C) + c;
#pragma unroll 4
                for (int k = 0; k < 32; ++k)
                    if (row0 + k < p.M)
                        mx4_store(out + (long)(row0 + k) * o.ldc,
                                  *reinterpret_cast<const float*>(bufs + h * BUF_BYTES + swizzled(k, lane >> 2) +
                                                                  (lane & 3) * 4),
                                  ga, gb, o, c);
            }
            __syncwarp();
        }
    }
}

template <int FMT, bool PAIR, typename TC>
__global__ void __launch_bounds__(THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmC, const Params p) {
    using S = Shape<FMT, PAIR>;
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
    const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sy->full[s]), 1);
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->tmem_full[a]), 1);
            mbar_init(smem_u32(&sy->tmem_empty[a]), (PAIR ? 2 : 1) * EPI_WARPS);
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
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->empty[s]), ph ^ 1u, wait));
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
                        mbar_wait<false>(smem_u32(&sy->full[s]), (armed_parity >> s) & 1u, wait);
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
            for (int t = unit; ok && t < p.num_tiles; t += p.units, ++it) {
                // Pair: the previous tile's shared columns have left tensor
                // memory (and with them all of the tile before it). Single:
                // the tile two before, which used this accumulator.
                if (PAIR ? it >= 1 : it >= 2)
                    if (!__all_sync(~0u, mbar_wait<true, PAIR>(smem_u32(&sy->tmem_empty[PAIR ? 0 : it & 1]),
                                                               (uint32_t)(PAIR ? it - 1 : (it >> 1) - 1) & 1u, wait)))
                        break;
                tc_fence_after();
                const uint32_t d = tmem_base + ((it & 1) ? S::ACC1 : 0);
                const uint32_t sfa = tmem_base + S::SF, sfb = sfa + S::SF_TILES * 4;
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->full[s]), ph, wait));
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
                                           sfb + tile * 4 * (S::TN / 128), (kb | k) != 0);
                    }
                    tc_commit<PAIR>(smem_u32(&sy->empty[s]));
                    if (kb == p.kblocks - 1) tc_commit<PAIR>(smem_u32(&sy->tmem_full[it & 1]));
                    }
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (elect_one()) tc_commit<PAIR>(smem_u32(&sy->drain));
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                            // tensor-memory lanes 32 q .. 32 q + 31
        uint8_t* bufs = epi + (warp - 2) * 2 * BUF_BYTES;
        const float ga = mx4_g(p.ga), gb = mx4_g(p.gb);
        int it = 0;
        for (int t = unit; t < p.num_tiles; t += p.units, ++it) {
            int mb, nb;
            tile_coords(t, p, mb, nb);
            const bool ok = mbar_wait(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 31) {
                    const uint32_t bar = tmem_empty0 + (uint32_t)((PAIR ? 0 : it & 1) * sizeof(uint64_t));
                    if constexpr (PAIR) mbar_arrive_cluster(bar); else mbar_arrive(bar);
                }
            };
            drain_tile<S, TC>(p, &tmC, tmem_base + ((it & 1) ? S::ACC1 : 0) + ((uint32_t)(q * 32) << 16), bufs,
                              mb * S::TM + (int)rank * 128 + q * 32, nb * S::TN, PAIR && !(it & 1), ga, gb, release);
        }
        tma_store_wait_all();
    }

    tc_fence_before();
    if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
    tc_fence_after();
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

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(EncodeTiledFn enc, CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
            CUtensorMapSwizzle swizzle) {
    const cuuint32_t ones[3] = {1, 1, 1};
    return enc(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes in boxes of 128 rows x 128 bytes.
bool encode_codes(EncodeTiledFn enc, CUtensorMap* map, const Mx4Operand& m, int rows, int K) {
    const cuuint64_t dims[2] = {(cuuint64_t)mx4_pitch(K), (cuuint64_t)rows}, strides[1] = {(cuuint64_t)mx4_pitch(K)};
    const cuuint32_t box[2] = {SW, 128};
    return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, dims, strides, box,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles: x within a tile (as 128 words), y along K, z along the rows.
bool encode_scales(EncodeTiledFn enc, CUtensorMap* map, const Mx4Operand& m, int rows, int K, int fmt,
                   int tiles_y, int tiles_z) {
    const cuuint64_t tk = (cuuint64_t)mx4_tiles_k(K, fmt);
    const cuuint64_t dims[3] = {128, tk, (cuuint64_t)(rows + 127) / 128};
    const cuuint64_t strides[2] = {MX4_TILE_BYTES, tk * MX4_TILE_BYTES};
    const cuuint32_t box[3] = {128, (cuuint32_t)tiles_y, (cuuint32_t)tiles_z};
    return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, m.scales, dims, strides, box,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

// C in boxes of 32 rows x 128 bytes, when it may leave by TMA: beta = 0, its
// rows on 16-byte boundaries and whole 16-byte pieces long (a box clipped
// inside such a piece also writes the rest of it).
bool encode_c(EncodeTiledFn enc, CUtensorMap* map, const Mx4Out& o, int M, int N) {
    const int esz = o.c_type == TGEMM_TYPE_F32 ? 4 : 2;
    if (o.beta != 0.0f || reinterpret_cast<uintptr_t>(o.C) % 16 != 0 || o.ldc * esz % 16 != 0 || (long)N * esz % 16 != 0)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {(cuuint64_t)o.ldc * esz};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esz), 32};
    return encode(enc, map, esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.C,
                  dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int FMT, bool PAIR, typename TC>
cudaError_t launch(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, const Mx4Out& out,
                   int num_sms, cudaStream_t s) {
    using S = Shape<FMT, PAIR>;
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    CUtensorMap tmA, tmB, tmSA, tmSB, tmC;
    if (!encode_codes(enc, &tmA, A, M, K) || !encode_codes(enc, &tmB, B, N, K) ||
        !encode_scales(enc, &tmSA, A, M, K, FMT, S::SF_TILES, 1) ||
        !encode_scales(enc, &tmSB, B, N, K, FMT, S::SF_TILES, S::TN / 128))
        return cudaErrorInvalidValue;
    memset(&tmC, 0, sizeof(tmC));
    Params p;
    p.M = M; p.N = N;
    p.kblocks = (int)(((long)K + STAGE_K - 1) / STAGE_K);
    p.tiles_m = (int)(((long)M + S::TM - 1) / S::TM);
    p.tiles_n = (int)(((long)N + S::TN - 1) / S::TN);
    if ((long)p.tiles_m * p.tiles_n > 0x3FFFFFFF) return cudaErrorInvalidValue;
    p.num_tiles = p.tiles_m * p.tiles_n;
    const int slots = PAIR ? num_sms / 2 : num_sms;
    p.units = p.num_tiles < slots ? p.num_tiles : slots;
    p.ga = A.g; p.gb = B.g;
    p.out = out;
    p.tma_c = encode_c(enc, &tmC, out, M, N) ? 1 : 0;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    cudaError_t e = mx4_status_word(&p.status);
    if (e == cudaSuccess) e = set_smem_limit_once<mx4_gemm_kernel<FMT, PAIR, TC>>(S::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((PAIR ? 2 : 1) * p.units);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see launch_pdl
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<FMT, PAIR, TC>, tmA, tmB, tmSA, tmSB, tmC, p);
}

template <int FMT, bool PAIR>
cudaError_t launch_type(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, const Mx4Out& out,
                        int num_sms, cudaStream_t s) {
    return out.c_type == TGEMM_TYPE_F32 ? launch<FMT, PAIR, float>(M, N, K, A, B, out, num_sms, s)
                                        : launch<FMT, PAIR, __nv_bfloat16>(M, N, K, A, B, out, num_sms, s);
}

// Pair tiles once they occupy half of the SM pairs.
bool use_pair(int M, int N, int num_sms) {
    return (((long)M + 255) / 256) * (((long)N + 255) / 256) * 4 >= num_sms;
}

}  // namespace

cudaError_t mx4_status_word(int** word) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_mx4_status);
    *word = static_cast<int*>(p);
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
