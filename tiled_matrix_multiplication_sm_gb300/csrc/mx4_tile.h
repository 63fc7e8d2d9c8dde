// What the tensor-core kernels of the 4-bit operators share: tiles of C and
// their way out of tensor memory, tensor maps, launches.
#pragma once

#include "mx4_ptx.h"

namespace tgemm {
namespace mx4_tile {

using namespace mx4_ptx;

constexpr int SW = 128;                       // bytes of a staged row (128-byte swizzle)
constexpr int BUF_BYTES = 32 * 128;           // 32 rows x 128 bytes of C
constexpr int TMEM_COLS = 512;

// A product's output in tiles, walked by `units` blocks or pairs of blocks.
struct Tiling {
    int M, N;
    int tiles_m, tiles_n, num_tiles, units;
    int split;                  // blocks of a cluster that share a tile's sum (1: none; then units tiles in all)
    int group_m;                // rows of tiles walked together, so that they share panels of B in L2
    Mx4Out out;
    int tma_c;                  // C leaves by TMA stores
    unsigned long long wait_limit_ns;
    int* status;
    int debug_stall;
};

__device__ __forceinline__ void tile_coords(int t, const Tiling& p, int& mb, int& nb) {
    const int per_group = p.group_m * p.tiles_n;
    const int first = t / per_group * p.group_m;
    const int gm = min(p.tiles_m - first, p.group_m);
    mb = first + t % per_group % gm;
    nb = t % per_group / gm;
}

// Where 16-byte piece j of row r lies in a 128-byte-swizzled buffer.
__device__ __forceinline__ uint32_t swizzled(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// Stores 32 columns of this warp's 32 rows from registers, the accumulator's
// values: half h of turn `turn`, whose 64 columns start at column `col` of C.
template <int BUFS, typename TC>
__device__ __forceinline__ void store_half(const Tiling& p, const CUtensorMap* tmC, uint8_t* bufs, int turn, int h,
                                           int row0, int rows, int col, float ga, float gb, uint32_t (&r)[32]) {
    constexpr int CW = 128 / (int)sizeof(TC);
    const int lane = threadIdx.x & 31;
    const Mx4Out& o = p.out;
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * ga * gb * o.alpha);
    if (p.tma_c) {
        // Boxes of 128-byte rows -- FP32: two of 32 columns, BF16: one of 64 --
        // through BUFS buffers in turn: the last box in this one has to have
        // left it.
        uint8_t* buf = bufs + (sizeof(TC) == 4 ? h : turn) % BUFS * BUF_BYTES;
        if (sizeof(TC) == 4 || h == 0) {
            if (lane == 0) tma_store_wait_read<BUFS - 1>();
            __syncwarp();
        }
        if (o.bias != nullptr)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col + h * 32 + j < p.N)
                    r[j] = __float_as_uint(__uint_as_float(r[j]) + o.bias[col + h * 32 + j]);
        if constexpr (sizeof(TC) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(buf + swizzled(lane, j)) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[8 * j + 2 * k]),
                                                                   __uint_as_float(r[8 * j + 2 * k + 1]));
                    w[k] = *reinterpret_cast<const uint32_t*>(&b);
                }
                *reinterpret_cast<uint4*>(buf + swizzled(lane, h * 4 + j)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (sizeof(TC) == 4 || h == 1) {
            fence_async_smem();
            __syncwarp();
            const int c = col + (sizeof(TC) == 4 ? h * CW : 0);
            if (lane == 0) {
                if (rows > 0 && c < p.N) tma_store_2d(tmC, c, row0, smem_u32(buf));
                tma_store_commit();                       // counted even when there is none
            }
        }
    } else {
        // Any alignment, and beta: 32 x 32 FP32 blocks through shared memory,
        // then whole row segments, a column a lane, eight rows' loads ahead of
        // their stores.
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(bufs + swizzled(lane, j)) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        __syncwarp();
        const int c = col + h * 32 + lane;
        if (c < p.N) {
            TC* out = static_cast<TC*>(o.C) + (long)row0 * o.ldc + c;
            const uint8_t* buf = bufs + (lane & 3) * 4;
            const float bias = o.bias != nullptr ? o.bias[c] : 0.0f;
#pragma unroll 1
            for (int k = 0; k < rows; k += 8) {
                float v[8], old[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = *reinterpret_cast<const float*>(buf + swizzled(k + j, lane >> 2));
                    old[j] = o.beta != 0.0f && k + j < rows ? (float)out[j * o.ldc] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (o.beta != 0.0f) v[j] = fmaf(o.beta, old[j], v[j]);
                    if (o.bias != nullptr) v[j] += bias;
                    if (k + j < rows) out[j * o.ldc] = (TC)v[j];
                }
                out += 8 * o.ldc;
            }
        }
    }
}

// Drains this warp's 32 rows of a tile, 64 columns a turn; of SETS sets of
// epilogue warps, set `set` takes every SETS-th turn. `last_first`: the last
// 64 columns, which the next tile's accumulator shares, are turn 0. release()
// is called as soon as turn `release_turn` has left tensor memory. BOTH: a
// turn's columns are in registers before any is stored (an earlier release for
// 32 registers more).
template <int TN, int SETS, bool BOTH, int BUFS, typename TC, typename Release>
__device__ __forceinline__ void drain_tile(const Tiling& p, const CUtensorMap* tmC, uint32_t tmem,
                                           uint8_t* bufs, int row0, int col0, bool last_first, int set,
                                           int release_turn, float ga, float gb, Release release) {
    constexpr int W = 64;
    constexpr int TURNS = TN / W;
    const int rows = min(32, p.M - row0);
#pragma unroll 1
    for (int i = set; i < TURNS; i += SETS) {
        const int part = last_first ? (i == 0 ? TURNS - 1 : i - 1) : i;
        const int col = col0 + part * W;
        uint32_t held[BOTH ? 2 : 1][32];
        if constexpr (BOTH) {
            tmem_ld32(tmem + (uint32_t)(part * W), held[0]);
            tmem_ld32(tmem + (uint32_t)(part * W + 32), held[1]);
            tmem_wait_ld(held[0]);
            tmem_wait_ld(held[1]);
            if (i == release_turn) release();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t (&r)[32] = held[BOTH ? h : 0];
            if constexpr (!BOTH) {
                tmem_ld32(tmem + (uint32_t)(part * W + h * 32), r);
                tmem_wait_ld(r);
                if (h == 1 && i == release_turn) release();
            }
            store_half<BUFS, TC>(p, tmC, bufs, i / SETS, h, row0, rows, col, ga, gb, r);
        }
    }
}

// Adds `cols` columns of `part` to `total` (`first`: moves them there), both in
// this warp's lanes of tensor memory.
__device__ __forceinline__ void add_sums(uint32_t total, uint32_t part, int cols, bool first) {
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
        uint32_t a[32], b[32];
        tmem_ld32(part + (uint32_t)c, a);
        if (!first) {
            tmem_ld32(total + (uint32_t)c, b);
            tmem_wait_ld(b);
        }
        tmem_wait_ld(a);
        if (!first)
#pragma unroll
            for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) + __uint_as_float(b[j]));
        tmem_st32(total + (uint32_t)c, a);
    }
    tmem_wait_st();
}

// A tile whose sum is split over a cluster: the block's share, FP32, goes to
// `partial` (128 rows of 128 columns, 16-byte pieces permuted by the row so that
// neither side's accesses conflict). 32 columns of a row from registers, and this
// warp's 32 rows from tensor memory.
__device__ __forceinline__ void share_columns(uint8_t* partial, int row, int c, const uint32_t (&r)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(partial + row * 512 + (((c / 4 + j) ^ (row & 31)) << 4)) =
            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}
__device__ __forceinline__ void store_share(uint8_t* partial, uint32_t tmem, int q) {
    const int row = q * 32 + (threadIdx.x & 31);
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + (uint32_t)c, r);
        tmem_wait_ld(r);
        share_columns(partial, row, c, r);
    }
}

// The cluster's shares, of `rows` rows, added in the order of their ranks and
// stored: block `part` takes every split-th row. All threads of all the
// cluster's blocks.
template <typename TC>
__device__ __forceinline__ void join_shares(const Tiling& p, const uint8_t* partial, int rows, int part, int row0,
                                            int col0, float ga, float gb) {
    cluster_sync_all();
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int r = part + p.split * (int)(threadIdx.x >> 5); r < rows && row0 + r < p.M; r += p.split * warps) {
        float v[4] = {};
        for (int i = 0; i < p.split; ++i) {
            const uint32_t base = map_to_rank(smem_u32(partial), (uint32_t)i) + r * 512;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = k * 32 + lane;
                float w;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w)
                             : "r"(base + (((c >> 2) ^ (r & 31)) << 4) + (c & 3) * 4) : "memory");
                v[k] += w;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = col0 + k * 32 + lane;
            if (c < p.N) mx4_store(static_cast<TC*>(p.out.C) + (long)(row0 + r) * p.out.ldc + c, v[k], ga, gb, p.out, c);
        }
    }
    cluster_sync_all();           // no block leaves while another reads its share
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline bool encode(EncodeTiledFn enc, CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                   CUtensorMapSwizzle swizzle) {
    const cuuint32_t ones[3] = {1, 1, 1};
    auto call = [&]() {
        return enc(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // A thread that has made no runtime call yet (a backward pass runs on
        // one) has no current context: the encoder is the driver's.
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = call();
    }
    return r == CUDA_SUCCESS;
}

// Codes in boxes of 128 rows x `width` bytes (128 or 64), swizzled over as many.
inline bool encode_codes(EncodeTiledFn enc, CUtensorMap* map, const Mx4Operand& m, int rows, int K, int width = SW) {
    const cuuint64_t dims[2] = {(cuuint64_t)mx4_pitch(K), (cuuint64_t)rows}, strides[1] = {(cuuint64_t)mx4_pitch(K)};
    const cuuint32_t box[2] = {(cuuint32_t)width, 128};
    return encode(enc, map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, dims, strides, box,
                  width == SW ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Scale tiles: x within a tile (as 128 words), y along K, z along the rows.
inline bool encode_scales(EncodeTiledFn enc, CUtensorMap* map, const Mx4Operand& m, int rows, int K, int fmt,
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
inline bool encode_c(EncodeTiledFn enc, CUtensorMap* map, const Mx4Out& o, int M, int N) {
    const int esz = o.c_type == TGEMM_TYPE_F32 ? 4 : 2;
    if (o.beta != 0.0f || reinterpret_cast<uintptr_t>(o.C) % 16 != 0 || o.ldc * esz % 16 != 0 || (long)N * esz % 16 != 0)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {(cuuint64_t)o.ldc * esz};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esz), 32};
    return encode(enc, map, esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.C,
                  dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

inline cudaError_t make_tiling(Tiling& p, int M, int N, int tile_m, int tile_n, int slots, const Mx4Out& out) {
    p.M = M; p.N = N;
    p.tiles_m = (int)(((long)M + tile_m - 1) / tile_m);
    p.tiles_n = (int)(((long)N + tile_n - 1) / tile_n);
    if ((long)p.tiles_m * p.tiles_n > 0x3FFFFFFF) return cudaErrorInvalidValue;
    p.num_tiles = p.tiles_m * p.tiles_n;
    p.units = p.num_tiles < slots ? p.num_tiles : slots;
    // 8192 x 14336 x 4096 NVFP4: 152 us with 16 and 158 with 8; 4096^3: 40 and 38.
    p.group_m = p.tiles_m >= 32 ? 16 : 8;
    p.split = 1;
    p.out = out;
    p.tma_c = 0;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    return mx4_status_word(&p.status);
}

// Launch attributes: programmatic dependent launch (see launch_pdl) and
// clusters of `cluster` blocks.
struct ClusterLaunch {
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int blocks, int threads, int smem, int cluster, cudaStream_t s) {
        config.gridDim = dim3((unsigned)blocks);
        config.blockDim = dim3((unsigned)threads);
        config.dynamicSmemBytes = (size_t)smem;
        config.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        config.attrs = attr;
        config.numAttrs = cluster > 1 ? 2 : 1;
    }
};

// How many clusters of c blocks the GPU holds at once, in byte c - 1 of *fits
// (2 <= c <= 8), for a kernel of one block per SM. The SMs come in groups that
// a cluster does not cross: 152 hold 36 clusters of 4, 23 of 6 but 15 of 8.
template <auto KERNEL>
cudaError_t clusters_that_fit(int threads, int smem, unsigned long long* fits) {
    static std::atomic<unsigned long long> known[64];      // of each device; byte 0: asked
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *fits = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*fits != 0) return cudaSuccess;
    *fits = 1;
    for (int c = 2; c <= 8; ++c) {
        ClusterLaunch cfg(c, threads, smem, c, nullptr);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg.config);
        if (e != cudaSuccess) return e;
        *fits |= (unsigned long long)(n < 0 ? 0 : n > 255 ? 255 : n) << 8 * (c - 1);
    }
    if (dev < 64) known[dev].store(*fits, std::memory_order_relaxed);
    return cudaSuccess;
}

// How many blocks of a cluster share the sum of one of few 128 x 128 tiles:
// as many as fit for all tiles at once (16 tiles of gemm_w4, 64 x 2048 x 2048
// MXFP4: 8.5 us with 6 blocks each, 15.1 with 8, which run one after another),
// each with two steps of K at least; none if that saves a block fewer than
// `worth` steps, what joining the shares takes.
inline int split_for(long tiles, int steps, unsigned long long fits, int worth) {
    int c = steps / 2 < 8 ? steps / 2 : 8;
    while (c > 1 && (long)(fits >> 8 * (c - 1) & 255) < tiles) --c;
    return c < 2 || steps - (steps + c - 1) / c < worth ? 1 : c;
}

// Pair tiles (256 x 256) once they occupy half of the SM pairs: past that, 128 x
// 128 tiles are more than the SMs (512 x 5120 x 4096: gemm_w4 26 us, in small
// tiles 34; gemm_mx4 10.6 and 13.4). Up to 128 rows half of a pair tile would be
// padding (128 x 14336 x 4096 MXFP4 weights: 27 us, in small tiles 18).
inline bool use_pair(int M, int N, int num_sms) {
    return M > 128 && (((long)M + 255) / 256) * (((long)N + 255) / 256) * 4 >= num_sms;
}

}  // namespace mx4_tile
}  // namespace tgemm
