// Products of BF16 matrices with what follows them in their epilogue: bias,
// activation, gating and residual; an activation's gradient and its column sums;
// the maxima and sums of a softmax cross entropy, and its gradient.
//
// The product is the tensor cores' (tcgen05, kind f16, FP32 accumulators): 256 x
// 256 tiles on SM pairs (cta_group::2), persistent, one block on an SM.
// Warp 0 copies (TMA), 1 issues the MMAs, the others are the epilogue, two
// or four sets of four (one to a quarter of tensor memory's lanes), each set on its
// share of the tile's columns. Stages of 64 columns of K, two accumulators, so that a tile's
// epilogue runs beside the next tile's MMAs. Either operand is read as it is
// kept, K-major in boxes of 128 rows x 128 bytes or MN-major in two boxes of 64
// rows of K x 128 bytes, both in the 128-byte swizzle.
//
// Gated products take 128 columns of g (the pair's first block) and the same 128
// of u (its second) for a tile, so that a thread holds both of a row.
//
// Sums of more than a part's columns that end in 32 bits, and logits (LONG), come in parts,
// accumulator by accumulator; the epilogue's warps add them up in registers and
// work from there where they can, so that accumulators are free as soon as they
// are read.
//
// Where tiles are few and sums long, a cluster's two, three or four pairs share a tile's K (one
// tile a cluster). Each pair leaves its sums in its stages' shared memory, a turn of 64
// columns falls to one of them, which adds up all shares, in the pairs' order, through
// distributed shared memory, and goes on from there: 512 x 4096 x 14336 73 -> 45 us.
// (Not for a gated gradient, whose totals in registers leave no room for it, nor for
// what is as wide as a vocabulary.)
//
// A thread has a row of the tile. Where C, R and Z allow TMA, boxes of 32 rows x
// 128 bytes pass between its registers and memory through shared memory; where
// they do not, 32 x 32 blocks of sums go through shared memory to a column a
// lane, and the epilogue works on segments of rows.
//
// Rows past M and columns past N are read as zeros and not stored. Waits are
// bounded as in the other tensor-core kernels.

#include "fused_column.h"

#include <cstring>

namespace tgemm {
namespace {

using namespace mx4_tile;
using namespace fused_act;
using namespace fused_column;
constexpr int TILE = 256;                            // rows of a tile, and columns of an accumulator
constexpr int STAGE_K = 64;
constexpr int OPERAND_BYTES = 128 * SW;              // a block's 128 rows of A, or of B
constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;
constexpr int STAGES = 5;
constexpr int EPI_BYTES = 16 * BUF_BYTES;
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 512;
static_assert(SMEM <= 227 * 1024, "shared memory");
// The epilogue: sets of four warps, each on its share of a tile's columns. Boxes
// and gated sums take two buffers a warp; a column a lane takes one, and more
// warps hide its latencies (3000 x 5001 x 1537 with R and Z: 99 us with two sets).
template <int KIND, bool GATED, bool BOXES>
struct Shape {
    static constexpr bool TWO = KIND == FUSED_ACT && GATED;      // 128 columns of C a tile
    static constexpr int SETS = BOXES || TWO || KIND == FUSED_CE ? 2 : 4, WARPS = 4 * SETS;
    static constexpr int WARP_BYTES = EPI_BYTES / WARPS;
    static constexpr int THREADS = 64 + 32 * WARPS;
};

struct Sync {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t loaded[8];                              // boxes of R or Z
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Sync) <= 512, "barrier block");

struct Params {
    int M, N, kblocks;
    int tiles_n, num_tiles, units, group_m, tiles_m;
    int split;                  // ACT and GRAD (not gated): pairs that share a tile's sum
    FusedParts part;
    int a_mn, b_mn;
    int bias4;                  // bias in pieces of 16 bytes
    FusedEpilogue e;
    unsigned long long wait_limit_ns;
    int* status;
    int debug_stall;
};

struct Maps {
    CUtensorMap A, B, B2;       // B2: gated, u's
    // ACT: C, R, Z, Z's second half. GRAD: C, Z, and the second halves of both.
    CUtensorMap E[4];
};

// ------------------------------------------------- boxes in shared memory
// This thread's row of a box: 32 FP32 or half h of 64 BF16.
__device__ __forceinline__ void put_f32(uint8_t* buf, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(buf + swizzled(lane, j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void put_bf16(uint8_t* buf, int h, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(buf + swizzled(lane, h * 4 + j)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void get_f32(const uint8_t* buf, float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 w = *reinterpret_cast<const float4*>(buf + swizzled(lane, j));
        v[4 * j] = w.x; v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
    }
}
__device__ __forceinline__ void get_bf16(const uint8_t* buf, int h, float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(buf + swizzled(lane, h * 4 + j));
        const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[8 * j + 2 * k] = __uint_as_float(p[k] << 16);
            v[8 * j + 2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
        }
    }
}

// v += bias of columns `at`, .. (of `cols`, from `bias` on).
__device__ __forceinline__ void add_bias(const Params& p, const float* bias, int at, float (&v)[32]) {
    if (bias == nullptr) return;
    if (p.bias4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at + 4 * j < p.N) {
                const float4 b = *reinterpret_cast<const float4*>(bias + at + 4 * j);
                v[4 * j] += b.x; v[4 * j + 1] += b.y; v[4 * j + 2] += b.z; v[4 * j + 3] += b.w;
            }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (at + j < p.N) v[j] += bias[at + j];
    }
}

// Sums over the warp's 32 rows of 32 columns: lane j gets column j's. Each step
// exchanges half of the columns that are left with the lane half as far away.
__device__ __forceinline__ float column_sums(float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const bool upper = lane & w;
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const float send = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
            v[j] = keep + __shfl_xor_sync(~0u, send, w);
        }
    }
    return v[0];
}

// --------------------------------------------- C in segments of its rows
// 32 columns from column `col` on of C of this warp's `rows` rows, from registers
// (a row a lane, by sums(v, v2); v2: gated ACT, u's sums) through `bufs` to a column a
// lane.
template <int KIND, bool GATED, typename Sums>
__device__ __forceinline__ void store_columns(const Params& p, uint8_t* bufs, int row0, int rows, int col, Sums sums) {
    const FusedEpilogue& e = p.e;
    const int lane = threadIdx.x & 31, c = col + lane;
    constexpr bool TWO = KIND == FUSED_ACT && GATED;
    const bool in = c < p.N;
    Column<KIND, GATED> column(e, p.N, in ? c : 0);
    // Where this lane's column lies in the rows of a group of eight.
    uint32_t at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) at[j] = swizzled(j, lane >> 2) + (lane & 3) * 4;
    column.rows(row0, 0, rows, 8, in, [&]() {
        float v[32], v2[32];
        sums(v, v2);
        __syncwarp();
        put_f32(bufs, v);
        if constexpr (TWO) put_f32(bufs + BUF_BYTES, v2);
        __syncwarp();
    }, [&](int k, float (&x)[8], float (&y)[8]) {
        const uint8_t* group = bufs + k * SW;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = *reinterpret_cast<const float*>(group + at[j]);
            if constexpr (TWO) y[j] = *reinterpret_cast<const float*>(group + BUF_BYTES + at[j]);
        }
    });
    if (in) column.leave(row0 / FUSED_SUM_ROWS);
    __syncwarp();
}

// ------------------------------------------------------- C by TMA, in boxes
// One lane: a box from shared memory to C or Z, of columns from c on.
__device__ __forceinline__ void store_box(const Params& p, const CUtensorMap* map, int c, int row0, uint8_t* buf) {
    if (c < p.N) tma_store_2d(map, c, row0, smem_u32(buf));
    tma_store_commit();                                  // counted even when there is none
}

// One lane: the boxes of R or Z that 64 columns from `col` on need, to the two
// buffers as turn_boxes wants them.
template <int KIND, bool GATED>
__device__ __forceinline__ void load_boxes(const Params& p, const Maps* maps, uint8_t* bufs, uint32_t bar, int row0, int col) {
    const FusedEpilogue& e = p.e;
    const uint32_t b0 = smem_u32(bufs), b1 = b0 + BUF_BYTES;
    const bool wide = KIND == FUSED_ACT && e.r_f32, two = (KIND == FUSED_GRAD && GATED) || (wide && col + 32 < p.N);
    mbar_arrive_expect_tx(bar, (two ? 2 : 1) * BUF_BYTES);
    tma_load_2d<false>(!wide && !GATED && e.c_f32 ? b1 : b0, &maps->E[1], col, row0, bar);
    if (two) tma_load_2d<false>(b1, wide ? &maps->E[1] : &maps->E[3], wide ? col + 32 : col, row0, bar);
}

// 64 columns of C from column `col` on. sums(h, v) gives half h's sums; acc2: gated
// ACT, u's in tensor memory. The buffers are free; the boxes that load_boxes asked
// for are in them.
template <int KIND, bool GATED, typename Sums, typename Release>
__device__ __forceinline__ void turn_boxes(const Params& p, const Maps* maps, uint8_t* bufs, Sums sums, uint32_t acc2,
                                           int row0, int rows, int col, int& box, Release release) {
    const FusedEpilogue& e = p.e;
    const int lane = threadIdx.x & 31;
    uint8_t *const b0 = bufs, *const b1 = bufs + BUF_BYTES;
    const bool aux = KIND == FUSED_GRAD || (KIND == FUSED_ACT && (e.R != nullptr || e.Z != nullptr));
    float v[32], w[32];
    auto send = [&](int map, int c, uint8_t* buf) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) store_box(p, &maps->E[map], c, row0, buf);
    };
    auto wait_sent = [&]() {
        if (lane == 0) tma_store_wait_read<0>();
        __syncwarp();
    };
    if constexpr (KIND == FUSED_ACT && GATED) {
        if (e.Z != nullptr) {
            // Both halves of Z leave first, through both buffers.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sums(h, v);
                add_bias(p, e.bias, col + h * 32, v);
                put_bf16(b0, h, v);
                load_sums(acc2 + h * 32, v, p.kblocks);
                add_bias(p, e.bias != nullptr ? e.bias + p.N : nullptr, col + h * 32, v);
                put_bf16(b1, h, v);
            }
            send(2, col, b0);
            send(3, col, b1);
            wait_sent();
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = col + h * 32;
        sums(h, v);
        if constexpr (KIND == FUSED_ACT) {
            add_bias(p, e.bias, c, v);
            if constexpr (GATED) {
                load_sums(acc2 + h * 32, w, p.kblocks);
                add_bias(p, e.bias != nullptr ? e.bias + p.N : nullptr, c, w);
            }
        }
        if (h == 1) release();
        uint8_t* out = b0;                               // of this half's C
        if constexpr (KIND == FUSED_ACT) {
            if constexpr (GATED) {
                apply(e.act, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= w[j];
            }
            if (e.R != nullptr) {
                if (e.r_f32) get_f32(h == 0 ? b0 : b1, w);
                else get_bf16(!GATED && e.c_f32 ? b1 : b0, h, w);
            }
            if constexpr (!GATED) {
                if (e.Z != nullptr) put_bf16(b1, h, v);
                apply(e.act, v);
            }
            if (e.R != nullptr)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = fmaf(e.r_scale, w[j], v[j]);
            if (e.c_f32 && e.Z == nullptr && h == 1) out = b1;
        } else {
            float g[32];
            if constexpr (GATED) {
                get_bf16(b0, h, g);
                get_bf16(b1, h, w);
                gated_grad(e.act, v, g, w);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = g[j];
                put_bf16(b1, h, w);
            } else {
                get_bf16(e.c_f32 ? b1 : b0, h, w);
                times_slope(e.act, v, w);
                if (e.c_f32 && h == 1) out = b1;
            }
        }
        if (!aux) {
            // Boxes through the two buffers in turn.
            out = bufs + (box & 1) * BUF_BYTES;
            if (e.c_f32 || h == 0) {
                if (lane == 0) tma_store_wait_read<1>();
                __syncwarp();
            }
        } else if (KIND == FUSED_ACT && e.c_f32 && e.Z != nullptr && h == 1) {
            wait_sent();
        }
        if (e.c_f32) {
            put_f32(out, v);
            send(0, c, out);
            ++box;
        } else {
            put_bf16(out, h, v);
        }
        if constexpr (KIND == FUSED_GRAD) {
            if (e.sums != nullptr) {
                // (Rows past M may hold a NaN: 0 times an infinity of B's.)
                float* to = e.sums + (long)(row0 / FUSED_SUM_ROWS) * (GATED ? 2L * p.N : p.N) + c + lane;
                if (rows < 32)
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = lane < rows ? v[j] : 0.0f;
                float sum = column_sums(v);
                if (c + lane < p.N) to[0] = sum;
                if constexpr (GATED) {
                    if (rows < 32)
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = lane < rows ? w[j] : 0.0f;
                    sum = column_sums(w);
                    if (c + lane < p.N) to[p.N] = sum;
                }
            }
        }
    }
    if (!e.c_f32) {
        send(0, col, aux ? b0 : bufs + (box & 1) * BUF_BYTES);
        ++box;
        if constexpr (KIND == FUSED_GRAD && GATED) send(2, col, b1);
    }
    if (KIND == FUSED_ACT && !GATED && e.Z != nullptr) send(2, col, b1);
}

// ------------------------------------------------------------ cross entropy
// Past this a row's differences from its maximum are taken before their product with log2(e):
// rounded, that product is off by as much as its bits are apart (128 and more from 2^31 on:
// 2^128 is an infinity), and from 2.36e38 on an infinity itself.
constexpr float FAR = 1024.0f;

// The maximum of this thread's row over its set's columns and the sum of exp(z -
// maximum), taken 32 columns at a time; the target's logit where it is among them.
struct CeRow {
    const Params& p;
    const int row;
    const bool in;
    const long long target;
    float m = -INFINITY, s = 0.0f;

    __device__ __forceinline__ CeRow(const Params& p_, int row_)
        : p(p_), row(row_), in(row_ < p_.M), target(row_ < p_.M ? p_.e.target[row_] - p_.e.first : -1) {}

    // The logits of columns c .. c + 31.
    __device__ __forceinline__ void add(int c, float (&v)[32]) {
        const FusedEpilogue& e = p.e;
        if (e.alpha != 1.0f)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= e.alpha;
        if (c + 32 > p.N)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = c + j < p.N ? v[j] : -INFINITY;
        const long long t = target - c;
        const bool here = t >= 0 && t < 32 && target < p.N;
        if (__any_sync(~0u, here)) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = t == j ? v[j] : z;
            if (here) e.picked[row] = z;
            __syncwarp();
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < 32; ++j) top = fmaxf(top, v[j]);
        // exp(v - top) as 2^(v L - at), at = top L rounded: one multiply-add each. What at is
        // off by, exactly the remainder of that product, goes back into the sum.
        const float base = top == -INFINITY ? 0.0f : top;
        float from = base;
        if (fabsf(base) > FAR) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] -= base;
            from = 0.0f;
        }
        const float at = from * LOG2E, off = fmaf(from, LOG2E, -at);
        s *= exp2_fast((m - base) * LOG2E);
        float q[4] = {};
#pragma unroll
        for (int j = 0; j < 32; ++j) q[j & 3] += exp2_fast(fmaf(v[j], LOG2E, -at));
        s += ((q[0] + q[1]) + (q[2] + q[3])) * exp2_fast(-off);
        m = top;
    }

    __device__ __forceinline__ void leave(int col) const {
        if (in && col < p.N) p.e.parts[(long)(col / FUSED_CE_COLS) * p.M + row] = make_float2(m, s);
    }
};

// 64 columns of the logits' gradient, whose sums sums(h, v) gives for either half, rounded to
// BF16: operands of the two products that follow. (In two BF16 numbers each those products, two
// thirds of the call's, would be twice as long.)
template <typename Sums>
__device__ __forceinline__ void ce_grad_turn(const Params& p, const Maps* maps, uint8_t* bufs, Sums sums, int row0, int col,
                                             int& box, float lse, float scale, long long target, bool kept) {
    const int lane = threadIdx.x & 31;
    uint8_t* buf = bufs + (box++ & 1) * BUF_BYTES;
    if (lane == 0) tma_store_wait_read<1>();
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[32];
        sums(h, v);
        const long long t = target - (col + h * 32);
        const bool any = __any_sync(~0u, t >= 0 && t < 32);
        float own = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = fmaf(v[j], p.e.alpha, -lse);
        if (any)
#pragma unroll
            for (int j = 0; j < 32; ++j) own = t == j ? v[j] : own;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = exp2_fast(v[j] * LOG2E);
        if (any) {
            own = expm1f(own);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = t == j ? own : v[j];
        }
        // (A row left out may hold infinities.)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = kept ? v[j] * scale : 0.0f;
        put_bf16(buf, h, v);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) store_box(p, &maps->E[0], col, row0, buf);
}

// ------------------------------------------------------------------- kernel
__device__ __forceinline__ void tile_at(int t, const Params& p, int& mb, int& nb) {
    const int per_group = p.group_m * p.tiles_n;
    const int first = t / per_group * p.group_m;
    const int gm = min(p.tiles_m - first, p.group_m);
    mb = first + t % per_group % gm;
    nb = t % per_group / gm;
}

// The end of the part that begins at stage `first` of a pair's `stages`.
__device__ __forceinline__ int part_end(const Params& p, int first, int stages) {
    return min(first + (first < 2 * p.part.first ? p.part.first : p.part.rest), stages);
}

// A pair's share of a tile's sums, in its stages' place: of a block, four columns of
// its 128 rows after the other. 32 columns from `col` on of row `row`.
__device__ __forceinline__ uint32_t share_at(int col, int row) { return (uint32_t)(col * 128 + row * 4) * 4; }
__device__ __forceinline__ void leave_share(uint8_t* share, int col, int row, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(share + share_at(col + j, row)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
}
// All pairs' shares of them, added up in the pairs' order.
__device__ __forceinline__ void gather_shares(uint32_t share, int split, uint32_t rank, int col, int row, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < split; ++i) {
        const uint32_t from = map_to_rank(share, 2u * i + rank);
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[j].x), "=f"(x[j].y), "=f"(x[j].z), "=f"(x[j].w) : "r"(from + share_at(col + 4 * j, row)) : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[4 * j] += x[j].x; v[4 * j + 1] += x[j].y; v[4 * j + 2] += x[j].z; v[4 * j + 3] += x[j].w;
        }
    }
}

// BOXES: C, R and Z pass by TMA (fused_boxes).
template <int KIND, bool GATED, bool LONG, bool BOXES>
__global__ void __launch_bounds__(Shape<KIND, GATED, BOXES>::THREADS, 1) fused_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using S = Shape<KIND, GATED, BOXES>;
    constexpr bool TWO = S::TWO;
    constexpr int TC = TWO ? TILE / 2 : TILE;            // columns of C a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* epi = smem + STAGES * STAGE_BYTES;
    Sync* sy = reinterpret_cast<Sync*>(epi + EPI_BYTES);
    const uint32_t stage0 = smem_u32(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The cluster's pair, and the block's place in it.
    constexpr bool SPLITS = KIND == FUSED_ACT || (KIND == FUSED_GRAD && !GATED);
    const uint32_t block = cluster_rank(), rank = block & 1u, pair0 = block - rank;
    const bool leader = rank == 0;
    const int split = SPLITS ? p.split : 1, part = SPLITS ? (int)(block >> 1) : 0;
    const int unit = SPLITS ? blockIdx.x / (2 * split) : blockIdx.x >> 1;
    // This pair's stages of a tile's sum.
    const int kb0 = (int)((long)p.kblocks * part / split), stages = (int)((long)p.kblocks * (part + 1) / split) - kb0;
    bool met = false;                                    // the cluster's pairs, over their shares

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sy->full[s]), 1);
            mbar_init(smem_u32(&sy->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&sy->tmem_full[a]), 1);
            mbar_init(smem_u32(&sy->tmem_empty[a]), 2 * S::WARPS);
        }
        for (int w = 0; w < 8; ++w) mbar_init(smem_u32(&sy->loaded[w]), 1);
        mbar_init(smem_u32(&sy->drain), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        if (p.kblocks > 0) {
            prefetch_map(&maps.A);
            prefetch_map(&maps.B);
        }
    }
    if (warp == 1) tmem_alloc<true, TMEM_COLS>(smem_u32(&sy->tmem_base));
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = sy->tmem_base;
    pdl_launch_dependents();
    pdl_wait();

    const Wait wait{&sy->abort, p.status, p.wait_limit_ns};
    // The leader's barriers, as cluster addresses.
    const uint32_t full0 = map_to_rank(smem_u32(&sy->full[0]), pair0);
    const uint32_t tmem_empty0 = map_to_rank(smem_u32(&sy->tmem_empty[0]), pair0);

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        uint32_t armed = 0, armed_parity = 0, ph = 0;
        int s = 0;
        bool ok = true, stall = p.debug_stall != 0;            // test hook: the first stage is never filled
        const CUtensorMap* mapB = TWO && !leader ? &maps.B2 : &maps.B;
        for (int t = unit; ok && t < p.num_tiles; t += p.units) {
            int mb, nb;
            tile_at(t, p, mb, nb);
            const int row = mb * TILE + (int)rank * 128;
            const int col = nb * TC + (TWO ? 0 : (int)rank * 128);
            for (int kb = kb0; kb < kb0 + stages; ++kb) {
                ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->empty[s]), ph ^ 1u, wait));
                if (!ok) break;
                if (!stall) {
                    if (elect_one()) {
                        const uint32_t full = full0 + (uint32_t)(s * sizeof(uint64_t));
                        if (leader) mbar_arrive_expect_tx(smem_u32(&sy->full[s]), 2 * STAGE_BYTES);
                        const uint32_t a = stage0 + s * STAGE_BYTES, b = a + OPERAND_BYTES;
                        if (p.a_mn) {
                            tma_load_2d<true>(a, &maps.A, row, kb * STAGE_K, full);
                            tma_load_2d<true>(a + OPERAND_BYTES / 2, &maps.A, row + 64, kb * STAGE_K, full);
                        } else {
                            tma_load_2d<true>(a, &maps.A, kb * STAGE_K, row, full);
                        }
                        if (p.b_mn) {
                            tma_load_2d<true>(b, mapB, col, kb * STAGE_K, full);
                            tma_load_2d<true>(b + OPERAND_BYTES / 2, mapB, col + 64, kb * STAGE_K, full);
                        } else {
                            tma_load_2d<true>(b, mapB, kb * STAGE_K, col, full);
                        }
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
                if (armed & (1u << i)) mbar_wait<false, true>(smem_u32(&sy->full[i]), (armed_parity >> i) & 1u, wait);
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
            const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.a_mn << 15 | (uint32_t)p.b_mn << 16 |
                                   (uint32_t)(TILE >> 3) << 17 | (uint32_t)(TILE >> 4) << 24;
            // A step of 16 columns of K: 32 bytes of a K-major row, 16 rows MN-major
            // (whose 64-column halves are half an operand apart).
            const uint32_t a_step = p.a_mn ? 16 * SW : 32, a_lead = p.a_mn ? OPERAND_BYTES / 2 : 16;
            const uint32_t b_step = p.b_mn ? 16 * SW : 32, b_lead = p.b_mn ? OPERAND_BYTES / 2 : 16;
            int it = 0, s = 0;
            uint32_t ph = 0;
            bool ok = true;
            // A tile's sum, or of LONG ones each part in turn: first to last - 1.
            for (int t = unit, first = 0; ok && t < p.num_tiles; ++it) {
                const int last = LONG ? part_end(p, first, stages) : stages;
                if (it >= 2)
                    if (!__all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->tmem_empty[it & 1]), (uint32_t)((it >> 1) - 1) & 1u, wait)))
                        break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(it & 1) * TILE;
                for (int kb = first; kb < last; ++kb) {
                    ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->full[s]), ph, wait));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t a = stage0 + s * STAGE_BYTES, b = a + OPERAND_BYTES;
#pragma unroll
                        for (int k = 0; k < STAGE_K / 16; ++k)
                            mma_bf16<true>(d, smem_desc(a + k * a_step, a_lead, 1024, 2), smem_desc(b + k * b_step, b_lead, 1024, 2),
                                     idesc, kb != first || k != 0);
                        tc_commit<true>(smem_u32(&sy->empty[s]), pair0);
                    }
                    __syncwarp();
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
                if (ok && elect_one()) tc_commit<true>(smem_u32(&sy->tmem_full[it & 1]), pair0);
                __syncwarp();
                first = last;
                if (last == stages) {
                    first = 0;
                    t += p.units;
                }
            }
            if (elect_one()) tc_commit<true>(smem_u32(&sy->drain), pair0);
            mbar_wait<false>(smem_u32(&sy->drain), 0, wait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                                // tensor-memory lanes 32 q .. 32 q + 31
        const int set = (warp - 2) >> 2;
        uint8_t* bufs = epi + (warp - 2) * S::WARP_BYTES;
        const uint32_t loaded = smem_u32(&sy->loaded[(warp - 2) & 7]);
        const bool loads = BOXES && (KIND == FUSED_GRAD || (KIND == FUSED_ACT && p.e.R != nullptr));
        constexpr int SET_COLS = TC / S::SETS, TURNS = SET_COLS / 64, HALVES = TWO ? 2 : 1;
        // A long sum's total stays in registers (HELD), or goes back to where its last
        // part lay (BACK): with a column a lane a warp's registers are few, and a copy of the
        // epilogue for each 32 of them cost more (3000 x 5001 x 1537 in two parts 121 us for 95).
        constexpr bool BACK = LONG && !BOXES && KIND != FUSED_CE, HELD = LONG && !BACK;
        int it = 0, box = 0;
        uint32_t load_ph = 0;
        bool loading = false;                                  // boxes asked for and not waited for
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 31) mbar_arrive_cluster(tmem_empty0 + (uint32_t)((it & 1) * sizeof(uint64_t)));
        };
        if (KIND == FUSED_CE_GRAD && p.e.kept != nullptr)
            keep_rows(p.e, p.M, (long)blockIdx.x * S::WARPS + warp - 2, (long)gridDim.x * S::WARPS);
        for (int t = unit; t < p.num_tiles; t += p.units, ++it) {
            int mb, nb;
            tile_at(t, p, mb, nb);
            const int row0 = mb * TILE + (int)rank * 128 + q * 32, rows = min(32, p.M - row0);
            const int col0 = nb * TC + set * SET_COLS;
            // R or Z of the first turn, while the sums are made. (Gated ACT with
            // Z: the buffers carry Z out first.)
            auto ask = [&](int col) {
                if (lane == 0) {
                    tma_store_wait_read<0>();
                    load_boxes<KIND, GATED>(p, &maps, bufs, loaded, row0, col);
                }
                __syncwarp();
                loading = true;
            };
            // The set's turns that are this pair's: each in turn to one of the cluster's.
            auto owns = [&](int i) { return split == 1 || (set * TURNS + i) % split == part; };
            bool asked = false;
            if constexpr (KIND == FUSED_ACT || KIND == FUSED_GRAD)
                if (loads && rows > 0 && col0 < p.N && owns(0)) {
                    ask(col0);
                    asked = true;
                }
            // A column a lane: on their way to L2 only. (A tile ahead of that: 3 % slower.)
            if constexpr (!BOXES && (KIND == FUSED_ACT || KIND == FUSED_GRAD))
                for (int c = col0; owns(0) && c < min(p.N, col0 + SET_COLS); c += 32) Column<KIND, GATED>(p.e, p.N, c).ask(row0 + lane, row0 + rows);

            const uint32_t lanes = (uint32_t)(q * 32) << 16;
            auto accumulator = [&]() { return tmem_base + (uint32_t)(it & 1) * TILE + lanes + set * SET_COLS; };
            bool ok = true;
            float sum[LONG ? SET_COLS / 32 : 1][32] = {};
            if constexpr (LONG) {
                #pragma unroll 1
                for (int first = 0; first < stages;) {
                    ok = __all_sync(~0u, mbar_wait<true, true, true>(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = accumulator();
                    first = part_end(p, first, stages);
                    const bool final = first == stages;
#pragma unroll
                    for (int i = 0; i < SET_COLS / 32; ++i) {
#pragma unroll
                        for (int c = 0; c < 32; c += 16) {
                            uint32_t r[16];
                            tmem_ld16(acc + i * 32 + c, r);
                            tmem_wait_ld(r);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[i][c + j] += __uint_as_float(r[j]);
                        }
                        if (BACK && final) tmem_st32(acc + i * 32, reinterpret_cast<uint32_t (&)[32]>(sum[i]));
                    }
                    if (!BACK || !final) release();
                    if (!final) ++it;
                }
                if (BACK && ok) tmem_wait_st();
            } else {
                ok = __all_sync(~0u, mbar_wait<true, true>(smem_u32(&sy->tmem_full[it & 1]), (uint32_t)(it >> 1) & 1u, wait));
                tc_fence_after();
            }
            if (!ok) break;
            const uint32_t acc = accumulator();
            if (SPLITS && split > 1) {
                // The tile's copies and MMAs are done: the stages hold the pair's share. What all
                // shares add up to goes where the sums were.
                const int mine = q * 32 + lane;
                if constexpr (HELD) {
#pragma unroll
                    for (int i = 0; i < SET_COLS / 32; ++i) leave_share(smem, set * SET_COLS + i * 32, mine, sum[i]);
                } else {
#pragma unroll 1
                    for (int i = 0; i < SET_COLS / 32 * HALVES; ++i) {
                        const int at = i % HALVES * 128 + i / HALVES * 32;
                        float v[32];
                        load_sums(acc + at, v, stages);
                        leave_share(smem, set * SET_COLS + at, mine, v);
                    }
                }
                __syncwarp();
                cluster_sync_all();
                met = true;
                if constexpr (HELD) {
#pragma unroll
                    for (int i = 0; i < SET_COLS / 32; ++i)
                        if (owns(i / 2)) gather_shares(stage0, split, rank, set * SET_COLS + i * 32, mine, sum[i]);
                } else {
#pragma unroll 1
                    for (int i = 0; i < SET_COLS / 32 * HALVES; ++i) {
                        const int at = i % HALVES * 128 + i / HALVES * 32;
                        float v[32];
                        if (!owns(i / HALVES / 2)) continue;
                        gather_shares(stage0, split, rank, set * SET_COLS + at, mine, v);
                        __syncwarp();
                        tmem_st32(acc + at, reinterpret_cast<uint32_t (&)[32]>(v));
                    }
                    tmem_wait_st();
                }
            }
            // Columns 32 i .. 32 i + 31 of the set's.
            auto sums = [&](int i, float (&v)[32]) {
                if constexpr (HELD) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = sum[i][j];
                } else {
                    load_sums(acc + i * 32, v, p.kblocks);
                }
            };
            if constexpr (KIND == FUSED_CE) {
                CeRow ce(p, row0 + lane);
                if constexpr (HELD) {
#pragma unroll
                    for (int i = 0; i < SET_COLS / 32; ++i) ce.add(col0 + i * 32, sum[i]);
                } else {
#pragma unroll 1
                    for (int i = 0; i < SET_COLS / 32; ++i) {
                        float v[32];
                        sums(i, v);
                        ce.add(col0 + i * 32, v);
                    }
                    release();
                }
                ce.leave(col0);
            } else {
                // Of this thread's row (CE_GRAD).
                long long target = -1;
                float lse = 0.0f, scale = 0.0f;
                if (KIND == FUSED_CE_GRAD && lane < rows) {
                    target = p.e.target[row0 + lane];
                    lse = p.e.lse[row0 + lane];
                    scale = p.e.alpha * p.e.dloss[row0 + lane];
                }
                // 64 columns of the set's; false: a wait ran out.
                auto turn = [&](int i) {
                    const int col = col0 + i * 64;
                    auto done = [&]() {
                        if (!HELD && i == TURNS - 1) release();
                    };
                    if (rows <= 0 || col >= p.N || !owns(i)) {
                        done();
                        return true;
                    }
                    if constexpr (KIND == FUSED_CE_GRAD) {
                        ce_grad_turn(p, &maps, bufs, [&](int h, float (&v)[32]) { sums(i * 2 + h, v); }, row0, col, box, lse,
                                     scale, target - p.e.first, target >= 0 && target < p.e.vocabulary);
                        done();
                    } else if constexpr (BOXES) {
                        if (loads && !asked) ask(col);
                        asked = false;
                        if (loading) {
                            if (!__all_sync(~0u, mbar_wait<true>(loaded, load_ph, wait))) return false;
                            load_ph ^= 1u;
                            loading = false;
                        } else if (KIND == FUSED_ACT && p.e.Z != nullptr) {
                            if (lane == 0) tma_store_wait_read<0>();
                            __syncwarp();
                        }
                        turn_boxes<KIND, GATED>(p, &maps, bufs, [&](int h, float (&v)[32]) { sums(i * 2 + h, v); },
                                                acc + 128 + i * 64, row0, rows, col, box, done);
                    } else {
                        auto half = [&](int h) {
                            store_columns<KIND, GATED>(p, bufs, row0, rows, col + h * 32, [&](float (&v)[32], float (&w)[32]) {
                                sums(i * 2 + h, v);
                                if constexpr (TWO) load_sums(acc + 128 + i * 64 + h * 32, w, p.kblocks);
                                if (h == 1) done();
                            });
                        };
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) half(h);
                    }
                    return true;
                };
                if constexpr (HELD) {
#pragma unroll
                    for (int i = 0; i < TURNS; ++i) ok = ok && turn(i);
                } else {
#pragma unroll 1
                    for (int i = 0; ok && i < TURNS; ++i) ok = turn(i);
                }
                if (!ok) break;
            }
        }
        if (loading) mbar_wait<false>(loaded, load_ph, wait);
        tma_store_wait_all();
    }

    if (SPLITS && split > 1 && !met) {
        __syncwarp();
        cluster_sync_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();                                  // no block leaves while another reads its share
    tc_fence_after();
    if (warp == 1) tmem_free<true, TMEM_COLS>(tmem_base);
}

// ------------------------------------------------------------------- launch
// An operand, K-major (rows x K) in boxes of 64 columns x 128 rows, or MN-major
// (K x rows) in boxes of 64 columns x 64 rows.
bool encode_operand(EncodeTiledFn enc, CUtensorMap* map, const void* x, long ld, int rows, int K, bool mn) {
    const cuuint64_t dims[2] = {(cuuint64_t)(mn ? rows : K), (cuuint64_t)(mn ? K : rows)}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, mn ? 64u : 128u};
    return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// C, R or Z in boxes of 32 rows x 128 bytes.
bool encode_boxes(EncodeTiledFn enc, CUtensorMap* map, const void* x, long ld, int M, int N, bool f32) {
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, 32};
    return encode(enc, map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, dims, strides,
                  box, CU_TENSOR_MAP_SWIZZLE_128B);
}
const void* second_half(const void* x, int N) { return static_cast<const bf16*>(x) + N; }

template <int KIND, bool GATED, bool LONG, bool BOXES>
cudaError_t launch_kernel(const Maps& maps, const Params& p, cudaStream_t s) {
    const cudaError_t e = set_smem_limit_once<fused_kernel<KIND, GATED, LONG, BOXES>>(SMEM);
    if (e != cudaSuccess) return e;
    ClusterLaunch cfg(2 * p.split * p.units, Shape<KIND, GATED, BOXES>::THREADS, SMEM, 2 * p.split, s);
    return cudaLaunchKernelEx(&cfg.config, fused_kernel<KIND, GATED, LONG, BOXES>, maps, p);
}
template <int KIND, bool GATED, bool LONG>
cudaError_t launch(const Maps& maps, const Params& p, bool boxes, cudaStream_t s) {
    return boxes ? launch_kernel<KIND, GATED, LONG, true>(maps, p, s) : launch_kernel<KIND, GATED, LONG, false>(maps, p, s);
}

}  // namespace

cudaError_t fused_gemm(FusedKind kind, const FusedProduct& m, const FusedEpilogue& e, const FusedPlan& plan, int num_sms,
                       cudaStream_t s) {
    if (plan.few) return fused_few(kind, m, e, plan, num_sms, s);
    const auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    const bool two = kind == FUSED_ACT && e.gated;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    Params p;
    p.M = m.M;
    p.N = m.N;
    p.kblocks = (int)(((long)m.K + STAGE_K - 1) / STAGE_K);
    p.split = plan.split;
    p.part = fused_parts(kind, false, (m.K - 1) / p.split + 1, STAGE_K);
    const int cols = two ? TILE / 2 : TILE;
    p.tiles_m = (int)(((long)m.M + TILE - 1) / TILE);
    p.tiles_n = (int)(((long)m.N + cols - 1) / cols);
    if ((long)p.tiles_m * p.tiles_n > 0x3FFFFFFF) return cudaErrorInvalidValue;
    p.num_tiles = p.tiles_m * p.tiles_n;
    p.units = p.split > 1 || p.num_tiles < num_sms / 2 ? p.num_tiles : num_sms / 2;
    p.group_m = p.tiles_m >= 32 ? 16 : 8;
    p.a_mn = m.a_mn ? 1 : 0;
    p.b_mn = m.b_mn ? 1 : 0;
    p.e = e;
    p.bias4 = reinterpret_cast<uintptr_t>(e.bias) % 16 == 0 && m.N % 4 == 0 ? 1 : 0;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    const cudaError_t err = mx4_status_word(&p.status);
    if (err != cudaSuccess) return err;
    if (m.K > 0 && (!encode_operand(enc, &maps.A, m.A, m.lda, m.M, m.K, m.a_mn) ||
                    !encode_operand(enc, &maps.B, m.B, m.ldb, m.N, m.K, m.b_mn) ||
                    (two && !encode_operand(enc, &maps.B2, m.B2, m.ldb, m.N, m.K, m.b_mn))))
        return cudaErrorInvalidValue;
    const bool boxes = plan.boxes;
    if (boxes) {
        // (The logits' gradient is scratch, its rows whole 64 columns long: what lies
        // past N there, from rows past the vocabulary, is read by no product.)
        bool ok = encode_boxes(enc, &maps.E[0], e.C, e.ldc, m.M, kind == FUSED_CE_GRAD ? (m.N + 7) / 8 * 8 : m.N, e.c_f32);
        if (kind == FUSED_ACT) {
            if (e.R != nullptr) ok = ok && encode_boxes(enc, &maps.E[1], e.R, e.ldr, m.M, m.N, e.r_f32);
            if (e.Z != nullptr) ok = ok && encode_boxes(enc, &maps.E[2], e.Z, e.ldz, m.M, m.N, false);
            if (e.Z != nullptr && two) ok = ok && encode_boxes(enc, &maps.E[3], second_half(e.Z, m.N), e.ldz, m.M, m.N, false);
        } else if (kind == FUSED_GRAD) {
            ok = ok && encode_boxes(enc, &maps.E[1], e.Z, e.ldz, m.M, m.N, false);
            if (e.gated)
                ok = ok && encode_boxes(enc, &maps.E[2], second_half(e.C, m.N), e.ldc, m.M, m.N, false) &&
                     encode_boxes(enc, &maps.E[3], second_half(e.Z, m.N), e.ldz, m.M, m.N, false);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    const bool parts = p.kblocks > p.part.first * p.split;
    switch (kind) {
        case FUSED_ACT:
            if (two) return launch<FUSED_ACT, true, false>(maps, p, boxes, s);
            return parts && e.c_f32 ? launch<FUSED_ACT, false, true>(maps, p, boxes, s)
                                    : launch<FUSED_ACT, false, false>(maps, p, boxes, s);
        case FUSED_GRAD: {
            const bool l = parts && (e.c_f32 || e.sums != nullptr);
            if (e.gated) return l ? launch<FUSED_GRAD, true, true>(maps, p, boxes, s) : launch<FUSED_GRAD, true, false>(maps, p, boxes, s);
            return l ? launch<FUSED_GRAD, false, true>(maps, p, boxes, s) : launch<FUSED_GRAD, false, false>(maps, p, boxes, s);
        }
        case FUSED_CE:
            return parts ? launch_kernel<FUSED_CE, false, true, false>(maps, p, s)
                         : launch_kernel<FUSED_CE, false, false, false>(maps, p, s);
        default:
            return parts ? launch_kernel<FUSED_CE_GRAD, false, true, true>(maps, p, s)
                         : launch_kernel<FUSED_CE_GRAD, false, false, true>(maps, p, s);
    }
}

}  // namespace tgemm
