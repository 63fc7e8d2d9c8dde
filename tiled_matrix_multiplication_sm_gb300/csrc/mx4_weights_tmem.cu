// BF16 rows times a kept 4-bit matrix, C = alpha X W^T + beta C + bias, where
// C has too few tiles for mx4_weights.cu: W is made BF16 on its way into
// tensor memory.
//
// The MMA (tcgen05, kind f16) takes W as its first operand, 128 rows of W from
// tensor memory, and up to 128 rows of X from shared memory as its second, so
// its result is a tile of C transposed: lanes are columns of C, tensor-memory
// columns rows of C. The decoded weights are the bulk of the data; in shared
// memory, written and read by the MMA, they take 32 of the 64 KB that a stage
// of 64 columns of K moves there (of 512 cycles at 128 bytes a cycle), and the
// MMA over padded rows of X has 128 rows' cost.
//
// A block has one tile, or a share of its sum over K. A stage is 128 columns
// of K: with 64, the handshakes of the warp that issues the MMAs take longer
// than the MMAs (64 x 14336 x 4096 MXFP4: 18.3 us, with 128 17.7). TMA brings
// X's rows into a stage's slot, and W's codes and scales into a longer ring;
// four groups of four warps decode every fourth stage each (a thread one row of W:
// four 16-byte reads, four to eight scales, 64 columns of tensor memory
// written; half stages to twice as many groups' turns: 17.7 us, whole ones 16.4).
// Four more warps add up the parts of long sums (SUM_K).

#include "mx4_decode.h"
#include "mx4_tile.h"

#include <cstring>
#include <type_traits>

namespace tgemm {
namespace {

using namespace mx4_tile;
using namespace mx4_decode;

constexpr int TW = 128;                              // rows of W in a tile: lanes of tensor memory
constexpr int STAGE_K = 128;
constexpr int PARTS = 2, PART_K = STAGE_K / PARTS;   // a row of X or of decoded weights in 128 bytes
constexpr int GROUPS = 4;                            // of decoding warps, each on its own stages
constexpr int ROW = STAGE_K / 2;                     // bytes of a row of a stage's codes
constexpr int CODES_BYTES = TW * ROW;
constexpr int SLOTS = 4, CHUNKS = 8;                // rings of X and decoded weights, of codes
constexpr int SUM_COLS = 128, SLOT_COLS = STAGE_K / 2;   // of tensor memory: a sum, a long sum's total, slots of weights
constexpr int PART_STAGES = SUM_K / STAGE_K;
constexpr int DECODE_WARPS = 4 * GROUPS;
constexpr int CODES_WARP = 2 + DECODE_WARPS;
template <typename TC> constexpr bool LONG_SUMS = sizeof(TC) == 4;
template <typename TC> constexpr int THREADS = 32 * (CODES_WARP + 1 + (LONG_SUMS<TC> ? 4 : 0));
constexpr int SMEM_LIMIT = 227 * 1024;
// A group meets all uses of the slots and codes that it meets at all (barriers
// tell phases apart by parity).
static_assert(SLOTS % GROUPS == 0 && CHUNKS % GROUPS == 0, "groups");
static_assert(2 * SUM_COLS + SLOTS * SLOT_COLS <= TMEM_COLS && SLOTS * PARTS * SW >= TW * 4,
              "room for the slots, and for a share in them");

template <int FMT> constexpr int SF_TILES = STAGE_K / mx4_block(FMT) / 4;
template <int FMT> constexpr int SF_BYTES = SF_TILES<FMT> * MX4_TILE_BYTES;

struct Sync {
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t codes_full[CHUNKS], codes_empty[CHUNKS];
    uint64_t done, drain, part_full[2], part_empty[2];
    uint32_t tmem_base;
    int abort;
    uint32_t factors[256];
};
constexpr int SYNC_BYTES = 1408;
static_assert(sizeof(Sync) <= SYNC_BYTES, "barrier block");

// Rows of X in a tile: a multiple of 16, 128 at most, as even as tiles allow.
inline int rows_of(int M) {
    const long tiles = ((long)M + 127) / 128;
    return (int)(((M + tiles - 1) / tiles + 15) / 16 * 16);
}
template <int FMT>
constexpr int smem_bytes(int rows) {
    return 1024 + SLOTS * PARTS * rows * SW + CHUNKS * (CODES_BYTES + SF_BYTES<FMT>) + SYNC_BYTES;
}
static_assert(smem_bytes<TGEMM_NVFP4>(128) <= SMEM_LIMIT, "shared memory");
// A block takes all of an SM's tensor memory and waits for it without a limit:
// of two clusters that shared SMs, each could hold what the other waits for. A
// launch asks for so much shared memory that no SM holds two blocks.
constexpr int ONE_BLOCK = SMEM_LIMIT / 2 + 1024;

struct Params : Tiling {
    int stages;                 // of K
    int rows;                   // of X in a tile
    const float* gb;
};

// Where 16-byte piece j of row r lies in a stage's codes (64-byte swizzle).
__device__ __forceinline__ uint32_t codes_at(int r, int j) { return (uint32_t)(r * ROW + ((j ^ (r >> 1 & 3)) << 4)); }

// D (+)= W X^T over 16 columns of K: W in tensor memory, X in shared memory.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

template <int FMT, typename TC>
__global__ void __launch_bounds__(THREADS<TC>, 1)
weights_tmem_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmS, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int part_bytes = p.rows * SW, slot_bytes = PARTS * part_bytes;      // of X
    uint8_t* codes = smem + SLOTS * slot_bytes;
    uint8_t* scales = codes + CHUNKS * CODES_BYTES;
    Sync* sy = reinterpret_cast<Sync*>(scales + CHUNKS * SF_BYTES<FMT>);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % p.split;
    int mb, nb;
    tile_coords(blockIdx.x / p.split, p, mb, nb);
    // This block's stages of its tile.
    const int k0 = (int)((long)p.stages * part / p.split), k1 = (int)((long)p.stages * (part + 1) / p.split);

    // A long sum's parts alternate between two accumulators where there is room
    // (FP32 C, MXFP4, 14336 x 4096: 64 rows 17.3 us, with one 17.8, in one part
    // 16.4; 128 rows, with one 21.9, in one part 18.4).
    const bool long_sum = LONG_SUMS<TC> && k1 - k0 > PART_STAGES;
    const int accs = p.rows <= SUM_COLS / 2 ? 2 : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(smem_u32(&sy->full[s]), 1 + 4);          // X's bytes, a group's warps
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int c = 0; c < CHUNKS; ++c) {
            mbar_init(smem_u32(&sy->codes_full[c]), 1);
            mbar_init(smem_u32(&sy->codes_empty[c]), 4);
        }
        mbar_init(smem_u32(&sy->done), long_sum ? 4 : 1);
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->part_full[a]), 1);
            mbar_init(smem_u32(&sy->part_empty[a]), 4);
        }
        mbar_init(smem_u32(&sy->drain), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_map(&tmX);
        prefetch_map(&tmW);
        prefetch_map(&tmS);
    }
    if (threadIdx.x < 256) sy->factors[threadIdx.x] = factor<FMT>(threadIdx.x);
    if (warp == 1) tmem_alloc<false, TMEM_COLS>(smem_u32(&sy->tmem_base));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sy->tmem_base, tmem_slots = tmem_base + 2 * SUM_COLS;
    pdl_launch_dependents();
    pdl_wait();

    const Wait wait{&sy->abort, p.status, p.wait_limit_ns};

    if (warp == 0) {
        // ------------------------------------------------- TMA producer of X
        uint32_t armed = 0, armed_parity = 0, ph = 0;
        int s = 0;
        bool stall = p.debug_stall != 0;                   // test hook: the first stage is never filled
        for (int k = k0; k < k1; ++k) {
            if (!__all_sync(~0u, mbar_wait(smem_u32(&sy->empty[s]), ph ^ 1u, wait))) break;
            if (!stall) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(smem_u32(&sy->full[s]), slot_bytes);
#pragma unroll
                    for (int i = 0; i < PARTS; ++i)
                        tma_load_2d<false>(smem_u32(smem) + s * slot_bytes + i * part_bytes, &tmX,
                                           k * STAGE_K + i * PART_K, mb * p.rows, smem_u32(&sy->full[s]));
                }
                armed |= 1u << s;
                armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
            }
            stall = false;
            __syncwarp();
            if (++s == SLOTS) { s = 0; ph ^= 1u; }
        }
        for (int i = 0; i < SLOTS; ++i)
            if (armed & (1u << i)) mbar_wait<false>(smem_u32(&sy->full[i]), (armed_parity >> i) & 1u, wait);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(p.rows >> 3) << 17 | (uint32_t)(TW >> 4) << 24;
        if (elect_one()) {
            int s = 0, in_part = 0, acc = 0, turn = 0;     // of a part: stages done, its accumulator and that one's turn
            uint32_t ph = 0;
            for (int k = k0; k < k1; ++k, ++in_part) {
                if (long_sum && in_part == PART_STAGES) {
                    in_part = 0;
                    if (++acc == accs) { acc = 0; ++turn; }
                }
                if (in_part == 0 && turn > 0 &&
                    !mbar_wait(smem_u32(&sy->part_empty[acc]), (uint32_t)(turn - 1) & 1u, wait)) break;
                if (!mbar_wait(smem_u32(&sy->full[s]), ph, wait)) break;
                tc_fence_after();
                const uint32_t x = smem_u32(smem) + s * slot_bytes, w = tmem_slots + (uint32_t)(s * SLOT_COLS);
#pragma unroll
                for (int j = 0; j < STAGE_K / 16; ++j)
                    mma_bf16(tmem_base + acc * (SUM_COLS / 2), w + j * 8, smem_desc(x + j / 4 * part_bytes + j % 4 * 32, 16, 1024, 2), idesc,
                             in_part != 0 || j != 0);
                tc_commit<false>(smem_u32(&sy->empty[s]));
                if (long_sum && (in_part == PART_STAGES - 1 || k == k1 - 1))
                    tc_commit<false>(smem_u32(&sy->part_full[acc]));
                if (!long_sum && k == k1 - 1) tc_commit<false>(smem_u32(&sy->done));
                if (++s == SLOTS) { s = 0; ph ^= 1u; }
            }
            tc_commit<false>(smem_u32(&sy->drain));
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else if (warp == CODES_WARP) {
        // ---------------------------------------- TMA producer of the codes
        uint32_t armed = 0, armed_parity = 0, ph = 0;
        int c = 0;
        for (int k = k0; k < k1; ++k) {
            if (!__all_sync(~0u, mbar_wait(smem_u32(&sy->codes_empty[c]), ph ^ 1u, wait))) break;
            if (elect_one()) {
                const uint32_t bar = smem_u32(&sy->codes_full[c]);
                mbar_arrive_expect_tx(bar, CODES_BYTES + SF_BYTES<FMT>);
                tma_load_2d<false>(smem_u32(codes) + c * CODES_BYTES, &tmW, k * ROW, nb * TW, bar);
                tma_load_3d<false>(smem_u32(scales) + c * SF_BYTES<FMT>, &tmS, 0, k * SF_TILES<FMT>, nb, bar);
            }
            __syncwarp();
            armed |= 1u << c;
            armed_parity = (armed_parity & ~(1u << c)) | (ph << c);
            if (++c == CHUNKS) { c = 0; ph ^= 1u; }
        }
        for (int i = 0; i < CHUNKS; ++i)
            if (armed & (1u << i)) mbar_wait<false>(smem_u32(&sy->codes_full[i]), (armed_parity >> i) & 1u, wait);
        __syncwarp();
    } else if (warp > CODES_WARP) {
        // -------------------------------------------- parts of long sums
        if (long_sum) {
            const uint32_t sum = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
            for (int k = k0, part = 0; k < k1; k += PART_STAGES, ++part) {
                const int acc = part % accs;
                if (!__all_sync(~0u, mbar_wait(smem_u32(&sy->part_full[acc]), (uint32_t)(part / accs) & 1u, wait))) break;
                tc_fence_after();
                add_sums(sum + SUM_COLS, sum + acc * (SUM_COLS / 2), p.rows, part == 0);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(k + PART_STAGES < k1 ? &sy->part_empty[acc] : &sy->done));
            }
        }
    } else {
        // ------------------------------------------------------ decoding
        // A stage's values are made before its slot is free.
        const int quarter = warp & 3, group = (warp - 2) / 4, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;   // those of tensor memory that this warp reaches
        uint32_t cph = 0, sph = 1;
        int c = group, s = group % SLOTS;
        bool ok = true;
        for (int k = k0 + group; k < k1; k += GROUPS) {
            ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->codes_full[c]), cph, wait));
            if (!ok) break;
            const uint8_t* sc = scales + c * SF_BYTES<FMT> + (row & 31) * 16 + (row >> 5) * 4;
            uint32_t sf[SF_TILES<FMT>];                  // the row's scales
#pragma unroll
            for (int i = 0; i < SF_TILES<FMT>; ++i) sf[i] = *reinterpret_cast<const uint32_t*>(sc + i * MX4_TILE_BYTES);
            const bool is_wide =
                FMT == TGEMM_MXFP4 && __any_sync(~0u, wide(sf[0] & 0xFF) || wide(sf[0] >> 8 & 0xFF) ||
                                                          wide(sf[0] >> 16 & 0xFF) || wide(sf[0] >> 24));
            const uint32_t slot = tmem_slots + lanes + (uint32_t)(s * SLOT_COLS);
            auto decode = [&](auto wide_scales) {
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    uint32_t v[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 w = *reinterpret_cast<const uint4*>(codes + c * CODES_BYTES +
                                                                        codes_at(row, i * 2 + h));
                        uint32_t f0, f1;
                        if (FMT == TGEMM_NVFP4) {
                            const uint32_t b = sf[i % SF_TILES<FMT>] >> h * 16;
                            f0 = sy->factors[b & 0xFF];
                            f1 = sy->factors[b >> 8 & 0xFF];
                        } else {
                            const uint32_t b = sf[0] >> (i * 2 + h) * 8 & 0xFF;
                            // Beside a wide block the others take their scale alone too.
                            f0 = f1 = !decltype(wide_scales)::value ? sy->factors[b] : b == 255 ? 0x7FC07FC0u : b == 0 ? 0x00400040u
                                                                                              : b << 7 | b << 23;
                        }
                        uint4 out[4];
                        decode_run<decltype(wide_scales)::value>(out, w, f0, f1);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[h * 16 + j * 4] = out[j].x;
                            v[h * 16 + j * 4 + 1] = out[j].y;
                            v[h * 16 + j * 4 + 2] = out[j].z;
                            v[h * 16 + j * 4 + 3] = out[j].w;
                        }
                    }
                    if (i == 0) {
                        if (!__all_sync(~0u, mbar_wait(smem_u32(&sy->empty[s]), sph, wait))) return false;
                        tc_fence_after();
                    }
                    tmem_st32(slot + (uint32_t)(i * (PART_K / 2)), v);
                }
                return true;
            };
            ok = is_wide ? decode(std::true_type()) : decode(std::false_type());
            if (!ok) break;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sy->full[s]));
                mbar_arrive(smem_u32(&sy->codes_empty[c]));
            }
            s += GROUPS;
            if (s >= SLOTS) { s -= SLOTS; sph ^= 1u; }
            c += GROUPS;
            if (c >= CHUNKS) { c -= CHUNKS; cph ^= 1u; }
        }
        // ------------------------------------------------------ the sums
        // They go where X's stages were (copies and MMAs are done), a row of C
        // in 512 bytes, in the order that join_shares reads.
        ok = __all_sync(~0u, ok && mbar_wait(smem_u32(&sy->done), 0, wait));
        if (ok) {
            tc_fence_after();
            const int piece = row >> 2;
            uint8_t* at = smem + (row & 3) * 4;
            const uint32_t sum = tmem_base + (long_sum ? SUM_COLS : 0);
#pragma unroll 1
            for (int m = group * 32; m < p.rows; m += 32 * GROUPS) {
                uint32_t r[32];
                tmem_ld32(sum + lanes + (uint32_t)m, r);
                tmem_wait_ld(r);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (m + j < p.rows) *reinterpret_cast<uint32_t*>(at + (m + j) * 512 + ((piece ^ j) << 4)) = r[j];
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    join_shares<TC>(p, smem, p.rows, part, mb * p.rows, nb * TW, unscale<FMT>(), mx4_g(p.gb));
    if (warp == 1) tmem_free<false, TMEM_COLS>(tmem_base);
}

template <int FMT, typename TC>
cudaError_t launch(int M, int N, int K, const void* X, long ldx, const Mx4Operand& W, const Mx4Out& out,
                   cudaStream_t s) {
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    Params p;
    p.rows = rows_of(M);
    CUtensorMap tmX, tmW, tmS;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M}, strides[1] = {(cuuint64_t)ldx * 2};
    const cuuint32_t box[2] = {PART_K, (cuuint32_t)p.rows};
    if (!encode(enc, &tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, X, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_codes(enc, &tmW, W, N, K, ROW) || !encode_scales(enc, &tmS, W, N, K, FMT, SF_TILES<FMT>, 1))
        return cudaErrorInvalidValue;
    cudaError_t e = make_tiling(p, M, N, p.rows, TW, 0x3FFFFFFF, out);
    p.stages = (int)(((long)K + STAGE_K - 1) / STAGE_K);
    p.gb = W.g;
    if (e == cudaSuccess) e = set_smem_limit_once<weights_tmem_kernel<FMT, TC>>(SMEM_LIMIT);
    unsigned long long fits = 0;
    if (e == cudaSuccess) e = clusters_that_fit<weights_tmem_kernel<FMT, TC>>(THREADS<TC>, SMEM_LIMIT, &fits);
    if (e != cudaSuccess) return e;
    p.split = split_for(p.num_tiles, p.stages, fits, 3);
    const int smem = smem_bytes<FMT>(p.rows) > ONE_BLOCK ? smem_bytes<FMT>(p.rows) : ONE_BLOCK;
    ClusterLaunch cfg(p.split * p.num_tiles, THREADS<TC>, smem, p.split, s);
    return cudaLaunchKernelEx(&cfg.config, weights_tmem_kernel<FMT, TC>, tmX, tmW, tmS, p);
}

}  // namespace

cudaError_t mx4_weights_tmem(int M, int N, int K, const void* X, long ldx, const Mx4Operand& W, int fmt,
                             const Mx4Out& out, cudaStream_t s) {
    if (out.c_type == TGEMM_TYPE_F32)
        return fmt == TGEMM_MXFP4 ? launch<TGEMM_MXFP4, float>(M, N, K, X, ldx, W, out, s)
                                  : launch<TGEMM_NVFP4, float>(M, N, K, X, ldx, W, out, s);
    return fmt == TGEMM_MXFP4 ? launch<TGEMM_MXFP4, __nv_bfloat16>(M, N, K, X, ldx, W, out, s)
                              : launch<TGEMM_NVFP4, __nv_bfloat16>(M, N, K, X, ldx, W, out, s);
}

}  // namespace tgemm
