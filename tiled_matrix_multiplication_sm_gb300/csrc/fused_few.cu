// The fused products whose C has few tiles of 256 x 256: few tokens, small
// layers.
//
// One SM a tile, and C transposed: the MMA's 128 rows are columns of C (a
// layer's outputs, a vocabulary's entries), its columns are C's rows (tokens), 16
// to 256 of them. So the weights, which are most of what there is to read,
// fill the MMA whatever the number of tokens, and a lane has a column of C: its
// 32 lanes' loads and stores are segments of rows, of any alignment.
//
// A tile takes `height` columns of C, 16 to 128, so that tiles are about as many as
// SMs (14336 columns: 150 tiles of 96); the MMA's other rows multiply what lies
// behind them in shared memory, and nobody reads them. Where that is not
// enough, a cluster's blocks split K and add their shares through distributed
// shared memory, in the order of their ranks; a sum over a vocabulary, longer than that,
// comes in slices, each to an FP32 matrix of its own.
//
// Eighteen warps: 0 copies (TMA, as many stages as fit), 1 issues the MMAs, the
// others are the epilogue, four sets of four on a quarter of the tokens each. Two accumulators (gated: of two halves each). Long sums that end in
// 32 bits, and logits, come in parts, as in fused_gemm.cu.

#include "fused_column.h"

#include <cstring>

namespace tgemm {
namespace {

using namespace mx4_tile;
using namespace fused_act;
using namespace fused_column;

constexpr int CHUNK_K = 64;                          // columns of K in a swizzled row
constexpr int MAX_STAGES = 24;
constexpr int SETS = FUSED_FEW_SETS, EPI_WARPS = 4 * SETS;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
// The MMA reads 128 rows of the weights whatever the height: the last stage's reach past the ring.
constexpr int GUARD_BYTES = 128 * SW;
constexpr int SYNC_BYTES = 512;
constexpr int SMEM = 227 * 1024;
constexpr int RING_BYTES = FUSED_FEW_RING;
static_assert(1024 + RING_BYTES + GUARD_BYTES + SYNC_BYTES <= SMEM, "shared memory");

// A stage's bytes: chunks of K of `halves` times `height` rows of weights and of `tokens` rows.
constexpr int stage_bytes_of(int height, int tokens, int chunks, int halves) { return chunks * (halves * height + tokens) * SW; }
// What the MMA reads from a stage's start on: of the last half, 128 rows behind its last
// chunk's start, or, MN-major, two boxes of 64, the second behind all of the first's chunks.
constexpr int reach_of(int height, int chunks, int halves, bool w_mn) {
    return (halves - 1) * chunks * height * SW + (w_mn ? 2 * chunks * CHUNK_K * SW : ((chunks - 1) * height + 128) * SW);
}
// As many stages as fit, with what the MMA reads from the last one on.
constexpr int stages_of(int height, int tokens, int chunks, int halves, bool w_mn) {
    const int bytes = stage_bytes_of(height, tokens, chunks, halves);
    int n = RING_BYTES / bytes < MAX_STAGES ? RING_BYTES / bytes : MAX_STAGES;
    while (n > 0 && (n - 1) * bytes + reach_of(height, chunks, halves, w_mn) > RING_BYTES + GUARD_BYTES) --n;
    return n;
}
// Of all shapes that a plan may have: fewest stages.
constexpr int fewest_stages() {
    int fewest = MAX_STAGES;
    for (int halves = 1; halves <= 2; ++halves)
        for (int height = 16; height <= 128; height += 8)
            for (int tokens = 16; tokens <= 256 / halves; tokens += 16)
                for (int chunks = 1; chunks <= 4; chunks *= 2) {
                    if (chunks > 1 && 4 * stage_bytes_of(height, tokens, chunks, halves) > RING_BYTES) continue;
                    for (int mn = 0; mn < 2; ++mn) {
                        if (mn && height % 64 != 0) continue;
                        const int n = stages_of(height, tokens, chunks, halves, mn != 0);
                        fewest = n < fewest ? n : fewest;
                    }
                }
    return fewest;
}
static_assert(fewest_stages() >= 4, "every plan's tiles run four stages deep");

struct Sync {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Sync) <= SYNC_BYTES, "barrier block");

struct Params {
    int M, N, kblocks;
    int height, tokens;                              // of a tile: columns and rows of C
    int tiles_m, num_tiles, units, split;
    int slices;                                      // of a tile's sum: num_tiles counts each
    int chunks, part_blocks;                         // chunks of K a stage, stages a part of a long sum
    int stages, half_bytes, stage_bytes;             // of a stage: one half of the weights, all
    int w_box, x_box;                                // K-major: a stage's chunks in one box
    int acc;                                         // tensor-memory columns of an accumulator's half
    int x_mn, w_mn;
    FusedEpilogue e;
    unsigned long long wait_limit_ns;
    int* status;
    int debug_stall;
};

struct Maps {
    CUtensorMap X, W, W2;
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :: "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// Eight sums of this thread's lane (zeros where there is nothing to sum).
__device__ __forceinline__ void load_sums8(uint32_t taddr, float (&v)[8], int kblocks) {
    tmem_ld8(taddr, v);
    if (kblocks == 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// One thread: `rows` rows of an operand, from `row` on, of `chunks` chunks of K from `chunk` on.
__device__ __forceinline__ void load_stage(const CUtensorMap* map, uint32_t to, int row, int rows, int chunk, int chunks, int mn,
                                           int box, uint32_t full) {
    if (box) {
        tma_load_3d<false>(to, map, 0, row, chunk, full);
    } else if (mn) {
        for (int i = 0; i < rows; i += 64) tma_load_2d<false>(to + i * chunks * SW, map, row + i, chunk * CHUNK_K, full);
    } else {
        for (int c = 0; c < chunks; ++c) tma_load_2d<false>(to + c * rows * SW, map, (chunk + c) * CHUNK_K, row, full);
    }
}

// Of 32 values a lane, value j combined over the 32 lanes, in lane j: each step
// exchanges half of the values that are left with the lane half as far away.
template <typename Op>
__device__ __forceinline__ float across(const float (&from)[32], Op op) {
    const int lane = threadIdx.x & 31;
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = from[j];
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const bool upper = lane & w;
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const float send = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
            v[j] = op(keep, __shfl_xor_sync(~0u, send, w));
        }
    }
    return v[0];
}

// `n` (up to 32) tokens from `row` on, whose sums sums(v) gives, against this warp's vocabulary entries, `c` this lane's
// (`in`: it is one): the maximum and the sum of exp(z - maximum) of each token, as
// entry `block` of what fused_join_ce joins, and the target's logit.
template <typename Sums>
__device__ __forceinline__ void ce_tokens(const Params& p, Sums sums, int row, int n, int c, bool in, long block) {
    const FusedEpilogue& e = p.e;
    const int lane = threadIdx.x & 31;
    float v[32];
    sums(v);
    const bool token = lane < n;
    // Where the target of token `lane` is among the warp's entries: its lane.
    const long long t = token ? e.target[row + lane] - (c - lane) : -1;
    const int at = t >= 0 && t < 32 ? (int)t : -1;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = in ? v[j] * e.alpha : -INFINITY;
    if (__any_sync(~0u, at >= 0))
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (__shfl_sync(~0u, at, j) == lane && in) e.picked[row + j] = v[j];
    __syncwarp();
    const float m = across(v, [](float a, float b) { return fmaxf(a, b); });
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = exp2_fast((v[j] - __shfl_sync(~0u, base, j)) * LOG2E);
    const float s = across(v, [](float a, float b) { return a + b; });
    if (token) e.parts[block * p.M + row + lane] = make_float2(m, s);
}

template <int KIND, bool GATED, bool LONG>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    constexpr bool TWO = KIND == FUSED_ACT && GATED;
    constexpr int HALVES = TWO ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Sync* sy = reinterpret_cast<Sync*>(smem + RING_BYTES + GUARD_BYTES);
    const uint32_t stage0 = smem_u32(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % p.split, unit = blockIdx.x / p.split;
    // A tile's row and column in C, and this block's stages of its sum: its share of
    // the cluster's, or the tile's slice.
    auto tile = [&](int t, int& row, int& col, int& kb0, int& kb1) {
        const int n = p.split > 1 ? p.split : p.slices, i = p.split > 1 ? part : t % p.slices;
        kb0 = (int)((long)p.kblocks * i / n);
        kb1 = (int)((long)p.kblocks * (i + 1) / n);
        t /= p.slices;
        row = t % p.tiles_m * p.tokens;
        col = t / p.tiles_m * p.height;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&sy->full[s]), 1);
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->tmem_full[a]), 1);
            mbar_init(smem_u32(&sy->tmem_empty[a]), EPI_WARPS);
        }
        mbar_init(smem_u32(&sy->drain), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        if (p.kblocks > 0) {
            prefetch_map(&maps.X);
            prefetch_map(&maps.W);
        }
    }
    if (warp == 1) tmem_alloc<false, TMEM_COLS>(smem_u32(&sy->tmem_base));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sy->tmem_base;
    pdl_launch_dependents();
    pdl_wait();

    const Wait wait{&sy->abort, p.status, p.wait_limit_ns};

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        // (One thread has the whole loop: with the warp in step a stage took 750 cycles.)
        if (elect_one()) {
            uint32_t armed = 0, armed_parity = 0, ph = 0, to = stage0;
            int s = 0;
            bool ok = true, stall = p.debug_stall != 0;        // test hook: the first stage is never filled
            for (int t = unit; ok && t < p.num_tiles; t += p.units) {
                int row, col, kb0, kb1;
                tile(t, row, col, kb0, kb1);
                int chunk = kb0 * p.chunks;
                for (int kb = kb0; kb < kb1; ++kb, chunk += p.chunks) {
                    ok = mbar_wait(smem_u32(&sy->empty[s]), ph ^ 1u, wait);
                    if (!ok) break;
                    if (!stall) {
                        const uint32_t full = smem_u32(&sy->full[s]);
                        mbar_arrive_expect_tx(full, p.stage_bytes);
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            load_stage(h == 0 ? &maps.W : &maps.W2, to + h * p.half_bytes, col, p.height, chunk, p.chunks, p.w_mn,
                                       p.w_box, full);
                        load_stage(&maps.X, to + HALVES * p.half_bytes, row, p.tokens, chunk, p.chunks, p.x_mn, p.x_box, full);
                        armed |= 1u << s;
                        armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
                    }
                    stall = false;
                    to += p.stage_bytes;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1u;
                        to = stage0;
                    }
                }
            }
            for (int i = 0; i < p.stages; ++i)
                if (armed & (1u << i)) mbar_wait<false>(smem_u32(&sy->full[i]), (armed_parity >> i) & 1u, wait);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.w_mn << 15 | (uint32_t)p.x_mn << 16 |
                               (uint32_t)(p.tokens >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
        // K-major: 16 columns of K are 32 bytes of a row, chunks lie one after the
        // other. MN-major: 16 rows of 64 columns, the next 64 behind all of the stage's
        // rows. (Addresses in descriptors count 16 bytes; their upper words are the same.)
        const uint32_t w_step = (p.w_mn ? 16 * SW : 32) >> 4, w_chunk = (p.w_mn ? CHUNK_K * SW : p.height * SW) >> 4;
        const uint32_t x_step = (p.x_mn ? 16 * SW : 32) >> 4, x_chunk = (p.x_mn ? CHUNK_K * SW : p.tokens * SW) >> 4;
        const uint64_t w0 = smem_desc(stage0, p.w_mn ? p.chunks * CHUNK_K * SW : 16, 1024, 2);
        const uint64_t x0 = smem_desc(stage0 + HALVES * p.half_bytes, p.x_mn ? p.chunks * CHUNK_K * SW : 16, 1024, 2);
        const uint32_t upper = (uint32_t)(w0 >> 32);
        if (elect_one()) {
            int it = 0, s = 0;
            uint32_t ph = 0, at = 0;                           // (at: the stage, in descriptors' units)
            bool ok = true;
            int row, col, kb0, kb1;
            tile(unit, row, col, kb0, kb1);
            for (int t = unit, first = kb0; ok && t < p.num_tiles; ++it) {
                const int last = LONG ? min(first + p.part_blocks, kb1) : kb1;
                if (it >= 2 && !mbar_wait(smem_u32(&sy->tmem_empty[it & 1]), (uint32_t)((it >> 1) - 1) & 1u, wait)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)((it & 1) * HALVES * p.acc);
                uint32_t more = 0;
                for (int kb = first; kb < last; ++kb) {
                    ok = mbar_wait(smem_u32(&sy->full[s]), ph, wait);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t w = (uint32_t)w0 + at, x = (uint32_t)x0 + at;
#pragma unroll 1
                    for (int c = 0; c < p.chunks; ++c, w += w_chunk, x += x_chunk)
#pragma unroll
                        for (int k = 0; k < CHUNK_K / 16; ++k) {
#pragma unroll
                            for (int h = 0; h < HALVES; ++h)
                                mma_bf16<false>(d + (uint32_t)(h * p.acc),
                                                (uint64_t)upper << 32 | (w + (h ? p.half_bytes >> 4 : 0) + k * w_step),
                                                (uint64_t)upper << 32 | (x + k * x_step), idesc, more);
                            more = 1;
                        }
                    tc_commit<false>(smem_u32(&sy->empty[s]));
                    at += (uint32_t)p.stage_bytes >> 4;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1u;
                        at = 0;
                    }
                }
                if (ok) tc_commit<false>(smem_u32(&sy->tmem_full[it & 1]));
                first = last;
                if (last == kb1) {
                    t += p.units;
                    tile(t, row, col, kb0, kb1);
                    first = kb0;
                }
            }
            tc_commit<false>(smem_u32(&sy->drain));
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                                // tensor-memory lanes 32 q .. 32 q + 31
        const int set = (warp - 2) >> 2;
        // This set's tokens of a tile, in groups of eight (CE: of 32).
        constexpr int GROUP = KIND == FUSED_CE ? 32 : 8;
        const int each = (p.tokens + SETS * GROUP - 1) / (SETS * GROUP) * GROUP;
        const int begin = min(set * each, p.tokens), end = min(begin + each, p.tokens);
        int it = 0;
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 31) mbar_arrive(smem_u32(&sy->tmem_empty[it & 1]));
        };
        if (KIND == FUSED_CE_GRAD && p.e.kept != nullptr)
            keep_rows(p.e, p.M, (long)blockIdx.x * EPI_WARPS + warp - 2, (long)gridDim.x * EPI_WARPS);
        for (int t = unit; t < p.num_tiles; t += p.units, ++it) {
            int row, col, kb0, kb1;
            tile(t, row, col, kb0, kb1);
            const int c = col + q * 32 + lane;
            const bool in = q * 32 + lane < p.height && c < p.N;
            // What the epilogue reads, while the sums are made: bias, and R or Z into L2.
            Column<KIND, GATED> column(p.e, p.N, in ? c : 0, (long)(t % p.slices) * p.M * p.e.ldc);
            if (in) column.ask(row + begin + lane, min(p.M, row + end));
            bool ok = true;
            const uint32_t lanes = (uint32_t)(q * 32) << 16;
            if constexpr (LONG) {
                // (The total aside, in columns of its own, so that the last part's are free at
                // once: no gain.)
                constexpr int MOST = 256 / SETS / 8;
                float sum[MOST][8] = {};
                #pragma unroll 1
                for (int first = kb0; ok && first < kb1; first += p.part_blocks) {
                    ok = __all_sync(~0u, mbar_wait<true, false, true>(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem_base + (uint32_t)((it & 1) * p.acc) + lanes + begin;
                    const bool final = first + p.part_blocks >= kb1;
#pragma unroll
                    for (int i = 0; i < MOST; ++i)
                        if (begin + i * 8 < end) {
                            float v[8];
                            tmem_ld8(acc + i * 8, v);
#pragma unroll
                            for (int j = 0; j < 8; ++j) sum[i][j] += v[j];
                            if (final) tmem_st8(acc + i * 8, sum[i]);
                        }
                    if (!final) {
                        release();
                        ++it;
                    }
                }
                if (ok) tmem_wait_st();
            } else {
                ok = __all_sync(~0u, mbar_wait(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait));
                tc_fence_after();
            }
            if (!ok) break;
            const uint32_t acc = tmem_base + (uint32_t)((it & 1) * HALVES * p.acc) + lanes;
            if (p.split > 1) {
                // The tile's copies and MMAs are done: its stages hold the share,
                // a row of 128 columns a token.
                float* share = reinterpret_cast<float*>(smem) + q * 32 + lane;
#pragma unroll 1
                for (int k = begin; k < end; k += 8) {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        float v[8];
                        load_sums8(acc + h * p.acc + k, v, kb1 - kb0);
#pragma unroll
                        for (int j = 0; j < 8; ++j) share[(h * p.tokens + k + j) * 128] = v[j];
                    }
                }
                break;
            }
            if constexpr (KIND == FUSED_CE) {
                if (q * 32 < p.height)
#pragma unroll 1
                    for (int k = begin; k < end && row + k < p.M; k += 32)
                        ce_tokens(p, [&](float (&v)[32]) { load_sums(acc + k, v, p.kblocks); }, row + k, min(end - k, p.M - row - k), c, in, (long)(col / p.height) * ((p.height + 31) / 32) + q);
            } else {
                column.rows(row, begin, min(end, p.M - row), 8, in, [] {}, [&](int k, float (&x)[8], float (&y)[8]) {
                    load_sums8(acc + k, x, kb1 - kb0);
                    if constexpr (TWO) load_sums8(acc + p.acc + k, y, kb1 - kb0);
                });
                if (in) column.leave((long)(row / p.tokens) * SETS + set);
                __syncwarp();
            }
            release();
        }
    }

    if (p.split > 1) {
        int row, col, kb0, kb1;
        tile(unit, row, col, kb0, kb1);
        const int q = warp & 3, set = (warp - 2) >> 2, c = col + q * 32 + lane;
        // A column's share of token k, from block i.
        auto share = [&](int i, int k) { return map_to_rank(stage0, (uint32_t)i) + (uint32_t)((k * 128 + q * 32 + lane) * 4); };
        if (KIND == FUSED_CE || warp < 2) cluster_sync_all();
        if (KIND == FUSED_CE && warp >= 2 && q * 32 < p.height) {
            // Groups of 32 tokens, in turn to the cluster's blocks and their sets. (Rows
            // past the tile's are other memory of the stages, and not used.)
#pragma unroll 1
            for (int k = (part * SETS + set) * 32; k < p.tokens && row + k < p.M; k += SETS * 32 * p.split)
                ce_tokens(p,
                          [&](float (&v)[32]) {
#pragma unroll
                              for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
                              for (int i = 0; i < p.split; ++i) {
                                  const uint32_t from = share(i, k);
#pragma unroll
                                  for (int j = 0; j < 32; ++j) v[j] += ld_cluster(from + j * 512);
                              }
                          },
                          row + k, min(p.tokens - k, p.M - row - k), c, q * 32 + lane < p.height && c < p.N,
                          (long)(col / p.height) * ((p.height + 31) / 32) + q);
        } else if (KIND != FUSED_CE && warp >= 2) {
            // Groups of eight tokens, in turn to the cluster's blocks and their sets.
            const bool in = q * 32 + lane < p.height && c < p.N;
            Column<KIND, GATED> column(p.e, p.N, in ? c : 0);
            column.rows(row, (part * SETS + set) * 8, min(p.tokens, p.M - row), SETS * 8 * p.split, in,
                        [&] {
                            __syncwarp();
                            cluster_sync_all();
                        },
                        [&](int k, float (&x)[8], float (&y)[8]) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
#pragma unroll 4
                            for (int i = 0; i < p.split; ++i) {
                                const uint32_t from = share(i, k);
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    x[j] += ld_cluster(from + j * 512);
                                    if constexpr (TWO) y[j] += ld_cluster(from + (p.tokens + j) * 512);
                                }
                            }
                        });
            if (in) column.leave(((long)(row / p.tokens) * p.split + part) * SETS + set);
        }
        __syncwarp();
        cluster_sync_all();           // no block leaves while another reads its share
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<false, TMEM_COLS>(tmem_base);
}

template <int KIND, bool GATED, bool LONG>
cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t s) {
    const cudaError_t e = set_smem_limit_once<few_kernel<KIND, GATED, LONG>>(SMEM);
    if (e != cudaSuccess) return e;
    ClusterLaunch cfg(p.split * p.units, THREADS, SMEM, p.split, s);
    return cudaLaunchKernelEx(&cfg.config, few_kernel<KIND, GATED, LONG>, maps, p);
}

// An operand's stages of `chunks` chunks of K: K-major in boxes of `box_rows`
// rows, all of its chunks in one box where K is whole chunks (*whole), else a chunk
// a box; MN-major in boxes of 64 columns.
bool encode_operand(EncodeTiledFn enc, CUtensorMap* map, const void* x, long ld, int rows, int K, bool mn, int box_rows, int chunks,
                    int* whole) {
    const cuuint64_t pitch = (cuuint64_t)ld * 2;
    *whole = !mn && K % CHUNK_K == 0 ? 1 : 0;
    if (*whole) {
        const cuuint64_t dims[3] = {CHUNK_K, (cuuint64_t)rows, (cuuint64_t)(K / CHUNK_K)}, strides[2] = {pitch, SW};
        const cuuint32_t box[3] = {CHUNK_K, (cuuint32_t)box_rows, (cuuint32_t)chunks};
        return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    const cuuint64_t dims[2] = {(cuuint64_t)(mn ? rows : K), (cuuint64_t)(mn ? K : rows)};
    const cuuint32_t box[2] = {64, mn ? (cuuint32_t)(chunks * CHUNK_K) : (cuuint32_t)box_rows};
    return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, dims, &pitch, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

// Clusters of each size that the GPU holds at once, by any of the kernels here
// (they ask for the same threads and shared memory).
cudaError_t fused_few_clusters(unsigned long long* fits) {
    const cudaError_t e = set_smem_limit_once<few_kernel<FUSED_ACT, false, false>>(SMEM);
    return e != cudaSuccess ? e : clusters_that_fit<few_kernel<FUSED_ACT, false, false>>(THREADS, SMEM, fits);
}

cudaError_t fused_few(FusedKind kind, const FusedProduct& m, const FusedEpilogue& e, const FusedPlan& plan, int num_sms,
                      cudaStream_t s) {
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    const bool two = kind == FUSED_ACT && e.gated;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    Params p;
    p.M = m.M;
    p.N = m.N;
    const bool logits = kind == FUSED_CE || kind == FUSED_CE_GRAD;
    p.chunks = logits && plan.chunks > 2 ? 2 : plan.chunks;                // (a part's 128 columns)
    p.part_blocks = fused_parts(kind, true, (m.K - 1) / (plan.split * plan.slices) + 1, CHUNK_K * p.chunks).rest;
    p.kblocks = (int)(((long)m.K + p.chunks * CHUNK_K - 1) / (p.chunks * CHUNK_K));
    p.height = plan.height;
    p.tokens = plan.tokens;
    p.split = plan.split;
    p.tiles_m = (m.M + p.tokens - 1) / p.tokens;
    p.slices = plan.slices;
    const long tiles = (long)p.tiles_m * (((long)m.N + p.height - 1) / p.height) * p.slices;
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;
    p.num_tiles = (int)tiles;
    p.units = p.split > 1 || p.num_tiles < num_sms ? p.num_tiles : num_sms;
    p.half_bytes = p.chunks * p.height * SW;
    p.stage_bytes = stage_bytes_of(p.height, p.tokens, p.chunks, two ? 2 : 1);
    p.stages = stages_of(p.height, p.tokens, p.chunks, two ? 2 : 1, m.b_mn);
    if (p.stages < 1) return cudaErrorInvalidValue;
    p.acc = (p.tokens + 31) / 32 * 32;
    p.x_mn = m.a_mn ? 1 : 0;
    p.w_mn = m.b_mn ? 1 : 0;
    p.e = e;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    const cudaError_t err = mx4_status_word(&p.status);
    if (err != cudaSuccess) return err;
    p.w_box = p.x_box = 0;
    if (m.K > 0 && (!encode_operand(enc, &maps.X, m.A, m.lda, m.M, m.K, m.a_mn, p.tokens, p.chunks, &p.x_box) ||
                    !encode_operand(enc, &maps.W, m.B, m.ldb, m.N, m.K, m.b_mn, p.height, p.chunks, &p.w_box) ||
                    (two && !encode_operand(enc, &maps.W2, m.B2, m.ldb, m.N, m.K, m.b_mn, p.height, p.chunks, &p.w_box))))
        return cudaErrorInvalidValue;
    const bool parts = p.kblocks > p.part_blocks * p.split * p.slices;
    switch (kind) {
        case FUSED_ACT:
            if (two) return launch<FUSED_ACT, true, false>(maps, p, s);
            return parts && e.c_f32 ? launch<FUSED_ACT, false, true>(maps, p, s) : launch<FUSED_ACT, false, false>(maps, p, s);
        case FUSED_GRAD: {
            const bool l = parts && (e.c_f32 || e.sums != nullptr);
            if (e.gated) return l ? launch<FUSED_GRAD, true, true>(maps, p, s) : launch<FUSED_GRAD, true, false>(maps, p, s);
            return l ? launch<FUSED_GRAD, false, true>(maps, p, s) : launch<FUSED_GRAD, false, false>(maps, p, s);
        }
        case FUSED_CE:
            return parts ? launch<FUSED_CE, false, true>(maps, p, s) : launch<FUSED_CE, false, false>(maps, p, s);
        default:
            return parts ? launch<FUSED_CE_GRAD, false, true>(maps, p, s) : launch<FUSED_CE_GRAD, false, false>(maps, p, s);
    }
}

}  // namespace tgemm
