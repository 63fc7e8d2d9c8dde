// Quantising to 4-bit floating point with block scales, reading back, and the
// import of row-major codes and scales. Formats and layout are described in
// include/tgemm_mx4.h.

#include "mx4_tile.h"

#include <cuda_fp16.h>

namespace tgemm {
namespace {

constexpr float kMinG = 7.888609052210118e-31f;      // 2^-100
constexpr float kMaxG = 1.661534994731145e+35f;      // 2^117

__device__ __forceinline__ uint32_t e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFF;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// E4M3 bytes (not NaN) to FP32 through halves, which hold them exactly.
__device__ __forceinline__ float e4m3_fast(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
    return __half2float(__ushort_as_half((unsigned short)h));
}

// An E4M3 byte as two equal halves; 0x7F gives NaN.
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)((byte & 0x7F) * 0x0101u)));
    return h;
}

// What the scales of a matrix are made with.
struct Scaling {
    float g, six_g, inv, cap;
    float down, g_down;                                  // a power of two, and g times it
    __device__ __forceinline__ explicit Scaling(const float* gp) {
        g = mx4_g(gp);
        if (!(g >= kMinG && g <= kMaxG)) g = 0.0f;       // every scale NaN
        six_g = 6.0f * g;
        inv = __frcp_rn(six_g);
        cap = 896.0f * six_g;                            // quotients from 464 on all give 448
        down = g >= 0x1p60f ? 0x1p-64f : 1.0f;
        g_down = g * down;
    }
};

// The scale byte of a block whose largest |x| is m (an infinity or a NaN if
// the block holds one), and what its values are multiplied with: a number just
// below 1 / d and the rest of 1 / d (0 and 0: every code is 0). A quotient is
// x inv + x rest in one rounding, so that one that is the midpoint of two codes,
// common for BF16 values over scales of 4 bits, comes out exact, where x (1 / d)
// alone would fall to either side. Both terms have x's sign: a quotient past
// FP32's range (under a g far too small for x) is an infinity of that sign,
// which the conversion makes the largest code. (A correction step
// q + (x - q d) (1 / d) makes it NaN.) The rest is 2^-22 of 1 / d, a normal number
// for d up to 2^100: under a large g, x and g are brought down by 2^64 first.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(float m, const Scaling& k, float& inv, float& rest) {
    const bool bad = __float_as_uint(m) >= 0x7F800000u;
    if (FMT == TGEMM_MXFP4) {
        const int e = (int)(__float_as_uint(m) >> 23) - 2;     // biased floor(log2 m), minus 2
        const uint32_t byte = e > 0 ? (uint32_t)e : 0u;
        inv = bad ? 0.0f : __uint_as_float((254u - byte) << 23);       // 2^(127 - byte): exact
        rest = 0.0f;
        return bad ? 0xFFu : byte;
    }
    const float c = fminf(m, k.cap);
    float q = c * k.inv;
    q = fmaf(fmaf(-q, k.six_g, c), k.inv, q);
    const uint32_t byte = e4m3(q);
    const float d = e4m3_fast(byte) * k.g_down;
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));      // within 2^-23 of itself
    y = __uint_as_float(__float_as_uint(y) - 2u);
    const bool none = bad || byte == 0 || k.g == 0.0f;
    inv = none ? 0.0f : y;
    rest = none ? 0.0f : fmaf(-d, y, 1.0f) * y;
    return bad || k.g == 0.0f ? 0x7Fu : byte;
}

// Two values over their divisors.
template <int FMT>
__device__ __forceinline__ float2 divide2(float x0, float x1, uint64_t inv2, uint64_t rest2, uint64_t down2) {
    uint64_t x = pack2(x0, x1);
    if (FMT == TGEMM_NVFP4) x = fma2(x, down2, 0);
    return unpack2(fma2(x, inv2, FMT == TGEMM_NVFP4 ? fma2(x, rest2, 0) : 0));
}

// Eight values to a word of codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(float a, float b, float c, float d, float e, float f, float g, float h) {
    uint32_t r;
    asm("{\n\t.reg .b8 p, q, r, s;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
        "mov.b32 %0, {p, q, r, s};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
    return r;
}

__global__ void __launch_bounds__(32) scale_init_kernel(float* g) {
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x == 0) *g = kMinG;
}

// The smallest power of two with 2688 g >= m, within [kMinG, kMaxG].
__device__ __forceinline__ float power_for(float m) {
    const uint32_t bits = __float_as_uint(__fdiv_rn(m, 2688.0f));
    const uint32_t up = (bits & 0x7F800000u) + ((bits & 0x007FFFFFu) ? 0x00800000u : 0u);
    return fminf(fmaxf(__uint_as_float(up), kMinG), kMaxG);
}

// The larger magnitude of each half (BF16) or of the word (FP32), its sign
// arbitrary. With NAN_WINS it is NaN if either is, without if both are.
template <typename T, bool NAN_WINS = true>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (sizeof(T) == 2) {
        if constexpr (NAN_WINS) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    } else {
        float f;
        if constexpr (NAN_WINS)
            asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        else
            asm("max.xorsign.abs.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        r = __float_as_uint(f);
    }
    return r;
}
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// The largest magnitude that max_abs left in a word, as the bits of an FP32.
template <typename T>
__device__ __forceinline__ uint32_t magnitude(uint32_t m) {
    if constexpr (sizeof(T) == 2) return max(m << 16 & 0x7FFF0000u, m & 0x7FFF0000u);
    else return m & 0x7FFFFFFFu;
}

// Eight loads a thread, all in flight before the first is used; bound by
// reading X. Rows that start on 16-byte boundaries are read in 16-byte pieces
// (`vec`). A block takes a run of 8 x 256 pieces of a row (shift 8), or eight
// times 256 >> shift rows of up to 1 << shift pieces.
template <typename T>
__global__ void __launch_bounds__(256)
tensor_scale_kernel(long rows, long cols, const T* X, long ldx, bool vec, int shift, float* g) {
    constexpr int V = 16 / (int)sizeof(T), LOADS = 8;
    pdl_launch_dependents();
    pdl_wait();
    uint32_t m = 0;
    auto take = [&](uint32_t b) {
        b &= 0x7FFFFFFFu;
        if (b < 0x7F800000u) m = max(m, b);
    };
    const long width = vec ? V : 1, pieces = (cols + width - 1) / width;
    const long parts = shift == 8 ? (pieces + 256 * LOADS - 1) / (256 * LOADS) : 1;      // runs of a row
    const long dr = shift == 8 ? 0 : 256 >> shift, dc = shift == 8 ? 256 : 0;
    const long runs = shift == 8 ? rows * parts : (rows + dr * LOADS - 1) / (dr * LOADS);
    for (long run = blockIdx.x; run < runs; run += gridDim.x) {
        const long r0 = shift == 8 ? run / parts : run * dr * LOADS + (threadIdx.x >> shift);
        const long p0 = shift == 8 ? run % parts * 256 * LOADS + threadIdx.x : threadIdx.x & ((1 << shift) - 1);
        if (vec) {
            uint4 v[LOADS];
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const long r = r0 + j * dr, c = (p0 + j * dc) * V;
                v[j] = r < rows && c + V <= cols ? *reinterpret_cast<const uint4*>(X + r * ldx + c) : make_uint4(0, 0, 0, 0);
            }
            uint32_t all = 0;
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                all = max_abs<T, false>(max_abs<T, false>(max_abs<T, false>(all, v[j].x), max_abs<T, false>(v[j].y, v[j].z)), v[j].w);
            if (magnitude<T>(all) < 0x7F800000u) m = max(m, magnitude<T>(all));
            else                                         // infinities or NaN among them: one by one
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (sizeof(T) == 4) take(w[k]);
                        else {
                            take(w[k] << 16);
                            take(w[k] & 0xFFFF0000u);
                        }
                    }
                }
        } else {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const long r = r0 + j * dr, c = p0 + j * dc;
                if (r < rows && c < cols) take(__float_as_uint((float)X[r * ldx + c]));
            }
        }
        if (vec && cols % V != 0) {                      // the piece that the row's end cuts
            for (int j = 0; j < LOADS; ++j) {
                const long r = r0 + j * dr, c = (p0 + j * dc) * V;
                if (r < rows && c < cols && c + V > cols)
                    for (long k = c; k < cols; ++k) take(__float_as_uint((float)X[r * ldx + k]));
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t most[8];
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 8) {
        m = __reduce_max_sync(0xffu, most[threadIdx.x]);
        // Positive floats order as their bits, and g only grows with |x|: the
        // result does not depend on the order of the blocks.
        if (threadIdx.x == 0) {
            const float p = power_for(__uint_as_float(m));
            if (gridDim.x == 1) *g = p;
            else atomicMax(reinterpret_cast<unsigned*>(g), __float_as_uint(p));
        }
    }
}

// Quantising, tile by tile of 128 x 128 elements of X in shared memory: in it
// both directions read 128 rows of 128 / B blocks, and both write whole scale
// tiles and 64-byte runs of codes, so X is read once even when its transpose
// is wanted too.
//
// A tile lies in panels of 128-byte rows (64 BF16 or 32 FP32 columns) in the
// 128-byte swizzle, as TMA writes them: the 16-byte reads of eight rows along
// the rows, and a row's 128 bytes read across the columns, fall in different
// banks.
constexpr int QT = 128;
constexpr int Q_THREADS = 512;
constexpr int Q_STAGES = 3;       // tiles in flight
constexpr int Q_CODES = 80;       // bytes between staged rows of transposed codes (64 used)
constexpr int Q_OUT = QT * Q_CODES + 2 * 1024;        // transposed codes, scales of both directions

template <typename T> __host__ __device__ constexpr int q_tile() { return QT * QT * (int)sizeof(T); }
template <typename T> __host__ __device__ constexpr int q_panel() { return 128 / (int)sizeof(T); }   // columns

struct QSync {
    uint64_t full[Q_STAGES];
    int abort;
};
template <typename T> __host__ __device__ constexpr int q_smem() { return 1024 + Q_STAGES * q_tile<T>() + Q_OUT + 64; }

// Byte of a tile's element (r, c).
template <typename T>
__device__ __forceinline__ int tile_at(int r, int c) {
    const int panel = c / q_panel<T>(), byte = c % q_panel<T>() * (int)sizeof(T);
    return panel * QT * 128 + r * 128 + ((byte >> 4 ^ (r & 7)) << 4) + (byte & 15);
}

// A block along a row: its values in words of T, in order, to codes and the
// scale byte.
template <typename T, int FMT>
__device__ __forceinline__ uint32_t quantize_row(const uint32_t* w, const Scaling& k, uint32_t* codes) {
    constexpr int B = mx4_block(FMT), WORDS = B * (int)sizeof(T) / 4;
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < WORDS; ++i) m = max_abs<T>(m, w[i]);
    float inv, rest;
    const uint32_t byte = block_scale<FMT>(__uint_as_float(magnitude<T>(m)), k, inv, rest);
    const uint64_t inv2 = pack2(inv, inv), rest2 = pack2(rest, rest), down2 = pack2(k.down, k.down);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
        float2 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2)
                q[j] = divide2<FMT>(low_bf16(w[i * 4 + j]), high_bf16(w[i * 4 + j]), inv2, rest2, down2);
            else
                q[j] = divide2<FMT>(__uint_as_float(w[i * 8 + 2 * j]), __uint_as_float(w[i * 8 + 2 * j + 1]), inv2, rest2, down2);
        }
        codes[i] = e2m1x8(q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y);
    }
    return byte;
}

// Blocks of two neighbouring columns, their values side by side (a word of
// two BF16, or two words of FP32, to a row). Codes of the first column, then
// of the second; the scale bytes in the low and high half.
template <typename T, int FMT>
__device__ __forceinline__ uint32_t quantize_columns(const uint32_t* w, const Scaling& k, uint32_t (&codes)[2][mx4_block(FMT) / 8]) {
    constexpr int B = mx4_block(FMT);
    float most[2];
    if constexpr (sizeof(T) == 2) {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < B; ++i) m = max_abs<T>(m, w[i]);
        most[0] = fabsf(low_bf16(m));
        most[1] = fabsf(high_bf16(m));
    } else {
        uint32_t m[2] = {w[0], w[1]};
#pragma unroll
        for (int i = 1; i < B; ++i) {
            m[0] = max_abs<T>(m[0], w[2 * i]);
            m[1] = max_abs<T>(m[1], w[2 * i + 1]);
        }
        most[0] = fabsf(__uint_as_float(m[0]));
        most[1] = fabsf(__uint_as_float(m[1]));
    }
    float inv[2], rest[2];
    const uint32_t b0 = block_scale<FMT>(most[0], k, inv[0], rest[0]), b1 = block_scale<FMT>(most[1], k, inv[1], rest[1]);
    const uint64_t inv2 = pack2(inv[0], inv[1]), rest2 = pack2(rest[0], rest[1]), down2 = pack2(k.down, k.down);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
        float2 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(T) == 2)
                q[j] = divide2<FMT>(low_bf16(w[i * 8 + j]), high_bf16(w[i * 8 + j]), inv2, rest2, down2);
            else
                q[j] = divide2<FMT>(__uint_as_float(w[i * 16 + 2 * j]), __uint_as_float(w[i * 16 + 2 * j + 1]), inv2, rest2, down2);
        }
        codes[0][i] = e2m1x8(q[0].x, q[1].x, q[2].x, q[3].x, q[4].x, q[5].x, q[6].x, q[7].x);
        codes[1][i] = e2m1x8(q[0].y, q[1].y, q[2].y, q[3].y, q[4].y, q[5].y, q[6].y, q[7].y);
    }
    return b0 | b1 << 16;
}

// Where a tile's scale byte of row r, block b lies in its 128 / B / 4 scale tiles.
__device__ __forceinline__ int tile_scale_at(int r, int b) {
    return (b >> 2) * MX4_TILE_BYTES + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// The tile's scale tiles to their place among those of a row of tiles.
template <int FMT>
__device__ __forceinline__ void write_scales(uint8_t* dst, const uint8_t* staged, int t) {
    constexpr int BYTES = QT / mx4_block(FMT) / 4 * MX4_TILE_BYTES;
    if (t < BYTES / 16) reinterpret_cast<uint4*>(dst)[t] = reinterpret_cast<const uint4*>(staged)[t];
}

// One tile (at row r0, column c0 of X) from shared memory.
template <typename T, int FMT, bool ROWS, bool TRANS>
__device__ __forceinline__ void quantize_tile(int R, int C, long r0, long c0, const uint8_t* tile, uint8_t* staged,
                                              const Scaling& k, uint8_t* codes) {
    constexpr int B = mx4_block(FMT), NB = QT / B, WORDS = B * (int)sizeof(T) / 4;
    uint8_t* sc = staged + QT * Q_CODES;                    // scales, then those of the transpose
    const int t = threadIdx.x, lane = t & 31;
    if (ROWS) {
        const long pitch = mx4_pitch(C);
#pragma unroll 1
        for (int i = t >> 5; i < QT * NB / 32; i += Q_THREADS / 32) {
            const int row = i / (NB / 4) * 8 + (lane & 7), b = i % (NB / 4) * 4 + (lane >> 3);
            uint32_t w[WORDS], out[B / 8];
#pragma unroll
            for (int j = 0; j < WORDS / 4; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(tile + tile_at<T>(row, b * B + j * (16 / (int)sizeof(T))));
                w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
            }
            sc[tile_scale_at(row, b)] = (uint8_t)quantize_row<T, FMT>(w, k, out);
            const long at = c0 / 2 + b * (B / 2);
            if (r0 + row < R && at < pitch) {
                uint8_t* dst = codes + (r0 + row) * pitch + at;
                if constexpr (B == 32) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
                else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
            }
        }
    }
    if (TRANS) {
        // Two columns a thread; lanes on neighbouring columns.
#pragma unroll 1
        for (int i = t; i < QT / 2 * NB; i += Q_THREADS) {
            const int c = i % (QT / 2) * 2, b = i / (QT / 2);
            constexpr int W = (int)sizeof(T) / 2;            // words of a row of two columns
            uint32_t w[B * W], out[2][B / 8];
            const uint8_t* src = tile + c / q_panel<T>() * QT * 128 + b * B * 128;
            const int byte = c % q_panel<T>() * (int)sizeof(T), piece = byte >> 4 << 4, in = byte & 15;
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const uint8_t* at = src + j * 128 + ((piece ^ (j & 7) << 4) | in);      // rows from a multiple of 8 on
                if constexpr (W == 1) {
                    w[j] = *reinterpret_cast<const uint32_t*>(at);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(at);
                    w[2 * j] = u.x;
                    w[2 * j + 1] = u.y;
                }
            }
            const uint32_t bytes = quantize_columns<T, FMT>(w, k, out);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc[1024 + tile_scale_at(c + h, b)] = (uint8_t)(bytes >> 16 * h);
                uint8_t* dst = staged + (c + h) * Q_CODES + b * (B / 2);
                if constexpr (B == 32) *reinterpret_cast<uint4*>(dst) = make_uint4(out[h][0], out[h][1], out[h][2], out[h][3]);
                else *reinterpret_cast<uint2*>(dst) = make_uint2(out[h][0], out[h][1]);
            }
        }
    }
}

// What quantize_tile left in shared memory.
template <int FMT, bool ROWS, bool TRANS>
__device__ __forceinline__ void write_tile(int R, int C, long r0, long c0, const uint8_t* staged, uint8_t* scales,
                                           uint8_t* codes_t, uint8_t* scales_t) {
    constexpr int SCALE_BYTES = QT / mx4_block(FMT) / 4 * MX4_TILE_BYTES;
    const uint8_t* sc = staged + QT * Q_CODES;
    const int t = threadIdx.x;
    if (ROWS && r0 < R)
        write_scales<FMT>(scales + ((r0 / QT) * mx4_tiles_k(C, FMT)) * MX4_TILE_BYTES + (c0 / QT) * SCALE_BYTES, sc, t);
    if (TRANS && c0 < C) {
        write_scales<FMT>(scales_t + ((c0 / QT) * mx4_tiles_k(R, FMT)) * MX4_TILE_BYTES + (r0 / QT) * SCALE_BYTES,
                          sc + 1024, t);
        const long pitch = mx4_pitch(R);
#pragma unroll
        for (int i = t; i < QT * 4; i += Q_THREADS) {
            const int c = i >> 2;
            const long at = r0 / 2 + (i & 3) * 16;
            if (c0 + c < C && at < pitch)
                *reinterpret_cast<uint4*>(codes_t + (c0 + c) * pitch + at) =
                    *reinterpret_cast<const uint4*>(staged + c * Q_CODES + (i & 3) * 16);
        }
    }
}

// Persistent blocks over the tiles (the scales cover spans of 256, so rows and
// columns go on to an even tile), TMA three tiles ahead with zeros outside X.
// Bound by HBM (X in, codes and scales out) in one direction, by instruction
// issue in both.
template <typename T, int FMT, bool ROWS, bool TRANS>
__global__ void __launch_bounds__(Q_THREADS, sizeof(T) == 2 ? 2 : 1)
quantize_kernel(const __grid_constant__ CUtensorMap tmX, int R, int C, const float* gp, uint8_t* codes, uint8_t* scales,
                uint8_t* codes_t, uint8_t* scales_t, unsigned long long wait_limit_ns, int* status) {
    using namespace mx4_ptx;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* staged = smem + Q_STAGES * q_tile<T>();
    QSync* sy = reinterpret_cast<QSync*>(staged + Q_OUT);
    if (threadIdx.x == 0) {
        for (int s = 0; s < Q_STAGES; ++s) mbar_init(smem_u32(&sy->full[s]), 1);
        sy->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_map(&tmX);
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int tiles_c = (int)(((long)C + 255) / 256 * 2);
    const long tiles = ((long)R + 255) / 256 * 2 * tiles_c;
    auto fetch = [&](long i, int s) {
        if (i >= tiles) return;
        const uint32_t bar = smem_u32(&sy->full[s]), dst = smem_u32(smem) + s * q_tile<T>();
        mbar_arrive_expect_tx(bar, q_tile<T>());
        for (int j = 0; j < QT / q_panel<T>(); ++j)
            tma_load_2d<false>(dst + j * QT * 128, &tmX, (int)(i % tiles_c) * QT + j * q_panel<T>(), (int)(i / tiles_c) * QT, bar);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < Q_STAGES; ++s) fetch(blockIdx.x + (long)s * gridDim.x, s);
    const Scaling k(gp);
    const Wait wait{&sy->abort, status, wait_limit_ns};
    int s = 0;
    uint32_t ph = 0;
    for (long i = blockIdx.x; i < tiles; i += gridDim.x) {
        const long r0 = i / tiles_c * QT, c0 = i % tiles_c * QT;
        // A copy that has not landed within the limit ends the block (its other
        // copies are older than that wait).
        if (__syncthreads_or(!mbar_wait<false>(smem_u32(&sy->full[s]), ph, wait))) return;
        quantize_tile<T, FMT, ROWS, TRANS>(R, C, r0, c0, smem + s * q_tile<T>(), staged, k, codes);
        __syncthreads();
        if (threadIdx.x == 0) fetch(i + (long)Q_STAGES * gridDim.x, s);
        write_tile<FMT, ROWS, TRANS>(R, C, r0, c0, staged, scales, codes_t, scales_t);
        if (++s == Q_STAGES) { s = 0; ph ^= 1u; }
    }
}

// The same for rows that do not start on 16-byte boundaries, which TMA cannot
// copy: one tile to a block, element by element.
template <typename T, int FMT, bool ROWS, bool TRANS>
__global__ void __launch_bounds__(Q_THREADS)
quantize_any_kernel(int R, int C, const T* X, long ldx, const float* gp, uint8_t* codes, uint8_t* scales,
                    uint8_t* codes_t, uint8_t* scales_t) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (mx4_ptx::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* staged = smem + q_tile<T>();
    pdl_launch_dependents();
    pdl_wait();
    const Scaling k(gp);
    const int tiles_c = (int)(((long)C + 255) / 256 * 2);
    const long tiles = ((long)R + 255) / 256 * 2 * tiles_c;
    for (long i = blockIdx.x; i < tiles; i += gridDim.x) {
        const long r0 = i / tiles_c * QT, c0 = i % tiles_c * QT;
#pragma unroll 8
        for (int e = threadIdx.x; e < QT * QT; e += Q_THREADS) {
            const int r = e / QT, c = e % QT;
            *reinterpret_cast<T*>(smem + tile_at<T>(r, c)) =
                r0 + r < R && c0 + c < C ? X[(r0 + r) * ldx + c0 + c] : (T)0.0f;
        }
        __syncthreads();
        quantize_tile<T, FMT, ROWS, TRANS>(R, C, r0, c0, smem, staged, k, codes);
        __syncthreads();
        write_tile<FMT, ROWS, TRANS>(R, C, r0, c0, staged, scales, codes_t, scales_t);
        __syncthreads();
    }
}

// Eight codes of each of eight rows a thread, all loads before the first use;
// a warp stores 512 bytes of a row side by side. Bound by writing X.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(int R, int C, const uint8_t* codes, const uint8_t* scales, const float* gp, T* X,
                  long ldx) {
    constexpr int B = mx4_block(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const long c = ((long)blockIdx.x * blockDim.x + threadIdx.x) * 8;
    if (c >= C) return;
    const float g = mx4_g(gp);
    const long pitch = mx4_pitch(C), row_of_tiles = mx4_tiles_k(C, FMT) * MX4_TILE_BYTES;
    const uint8_t* code = codes + c / 2;
    const uint8_t* scale = scales + mx4_scale_at(0, c / B, 0);
    constexpr int ROWS = 8;                                  // consecutive rows a thread
    const long r0 = (long)blockIdx.y * ROWS;
    for (long r = r0; r < R; r += (long)gridDim.y * ROWS) {
        const int n = (int)min((long)ROWS, R - r);
        uint32_t w[ROWS], b[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i < n) {
                w[i] = *reinterpret_cast<const uint32_t*>(code + (r + i) * pitch);
                // Eight rows from a multiple of 8 on lie in one column of a tile.
                b[i] = scale[(r >> 7) * row_of_tiles + ((r & 31) + i) * 16 + ((r & 127) >> 5) * 4];
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i >= n) break;
            float v[8];
            const float s = FMT == TGEMM_MXFP4 ? e8m0_value(b[i]) : 1.0f;
            const uint32_t sh = FMT == TGEMM_MXFP4 ? 0 : e4m3_halves(b[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h;      // two codes as halves; NVFP4 scales multiply exactly in them
                asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(w[i] >> 8 * j));
                __half2 x = *reinterpret_cast<const __half2*>(&h);
                if (FMT == TGEMM_NVFP4) x = __hmul2(x, *reinterpret_cast<const __half2*>(&sh));
                const float2 f = __half22float2(x);
                v[2 * j] = FMT == TGEMM_MXFP4 ? f.x * s : f.x * g;
                v[2 * j + 1] = FMT == TGEMM_MXFP4 ? f.y * s : f.y * g;
            }
            T* dst = X + (r + i) * ldx + c;
            if (c + 8 <= C) {
                if constexpr (sizeof(T) == 4) {
                    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    __nv_bfloat162 o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < C) dst[j] = (T)v[j];
            }
        }
    }
}

// The same for rows of X that do not start on 16-byte boundaries: a column of
// eight rows a thread, so that a warp's stores lie side by side.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_any_kernel(int R, int C, const uint8_t* codes, const uint8_t* scales, const float* gp, T* X, long ldx) {
    constexpr int B = mx4_block(FMT), ROWS = 8;
    pdl_launch_dependents();
    pdl_wait();
    const long c = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C) return;
    const float g = mx4_g(gp);
    const long pitch = mx4_pitch(C), row_of_tiles = mx4_tiles_k(C, FMT) * MX4_TILE_BYTES;
    const uint8_t* code = codes + c / 2;
    const uint8_t* scale = scales + mx4_scale_at(0, c / B, 0);
    for (long r = (long)blockIdx.y * ROWS; r < R; r += (long)gridDim.y * ROWS) {
        uint32_t w[ROWS], b[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (r + i < R) {
                w[i] = code[(r + i) * pitch] >> (c & 1) * 4;
                b[i] = scale[(r >> 7) * row_of_tiles + ((r & 31) + i) * 16 + ((r & 127) >> 5) * 4];
            }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (r + i < R) X[(r + i) * ldx + c] = (T)(e2m1_value(w[i] & 15) * mx4_scale_value<FMT>(b[i]) * g);
    }
}

// A thread moves, of every row that it takes, a byte of codes and a scale byte.
template <int FMT>
__global__ void __launch_bounds__(256)
pack_kernel(int R, int C, const uint8_t* sc, long ldc, const uint8_t* ss, long lds, uint8_t* codes,
            uint8_t* scales) {
    constexpr int B = mx4_block(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const long pitch = mx4_pitch(C), tiles_k = mx4_tiles_k(C, FMT);
    const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
    for (long r = blockIdx.y; r < ((long)R + 127) / 128 * 128; r += gridDim.y) {
        if (i < pitch && r < R) {
            uint32_t v = 2 * i < C ? sc[r * ldc + i] : 0u;
            if (2 * i + 1 >= C) v &= 15u;
            codes[r * pitch + i] = (uint8_t)v;
        }
        if (i < tiles_k * 4)
            scales[mx4_scale_at(r, i, tiles_k)] = r < R && i * B < C ? ss[r * lds + i] : 0;
    }
}

unsigned grid_rows(long rows) { return (unsigned)(rows < 1 ? 1 : rows > 32768 ? 32768 : rows); }

bool rows_on_16(const void* X, long ldx, int esz) {
    return reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx * esz % 16 == 0;
}

template <typename T, int FMT, bool ROWS, bool TRANS>
cudaError_t launch_quantize(int R, int C, const void* X, long ldx, const float* g, uint8_t* codes,
                            uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, int num_sms, cudaStream_t s) {
    const long tiles = ((long)R + 255) / 256 * 2 * (((long)C + 255) / 256 * 2);
    const auto enc = reinterpret_cast<mx4_tile::EncodeTiledFn>(tensor_map_encoder());
    if (!rows_on_16(X, ldx, sizeof(T)) || enc == nullptr) {
        const int smem = 1024 + q_tile<T>() + Q_OUT;
        const cudaError_t e = set_smem_limit_once<quantize_any_kernel<T, FMT, ROWS, TRANS>>(smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(quantize_any_kernel<T, FMT, ROWS, TRANS>, dim3((unsigned)(tiles < 1 << 30 ? tiles : 1 << 30)),
                          dim3(Q_THREADS), smem, s, R, C, static_cast<const T*>(X), ldx, g, codes, scales, codes_t, scales_t);
    }
    CUtensorMap tmX;
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)R}, strides[1] = {(cuuint64_t)ldx * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)q_panel<T>(), QT};
    if (!mx4_tile::encode(enc, &tmX, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          2, X, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    int* status = nullptr;
    cudaError_t e = mx4_status_word(&status);
    if (e == cudaSuccess) e = set_smem_limit_once<quantize_kernel<T, FMT, ROWS, TRANS>>(q_smem<T>());
    if (e != cudaSuccess) return e;
    const long slots = (sizeof(T) == 2 ? 2L : 1L) * num_sms;
    return launch_pdl(quantize_kernel<T, FMT, ROWS, TRANS>, dim3((unsigned)(tiles < slots ? tiles : slots)),
                      dim3(Q_THREADS), q_smem<T>(), s, tmX, R, C, g, codes, scales, codes_t, scales_t, wait_limit_ns(),
                      status);
}

template <typename T, int FMT>
cudaError_t quantize_type(int R, int C, const void* X, long ldx, const float* g, uint8_t* codes,
                          uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, int num_sms, cudaStream_t s) {
    if (codes_t == nullptr)
        return launch_quantize<T, FMT, true, false>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s);
    if (codes == nullptr)
        return launch_quantize<T, FMT, false, true>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s);
    return launch_quantize<T, FMT, true, true>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s);
}

}  // namespace

cudaError_t mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type, float* g,
                             int num_sms, cudaStream_t s) {
    const int esz = x_type == TGEMM_TYPE_F32 ? 4 : 2;
    long r = rows, c = cols;
    if (ldx == cols) {                                   // one long row
        r = 1;
        c = (long)rows * cols;
    }
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (r == 1 || ldx * esz % 16 == 0);
    const long pieces = vec ? (c * esz + 15) / 16 : c;
    int shift = 0;
    while (shift < 8 && (1L << shift) < pieces) ++shift;
    const long runs = shift == 8 ? r * ((pieces + 2047) / 2048) : (r + (2048 >> shift) - 1) / (2048 >> shift);
    // One block, which needs no initial value, takes up to four runs: less
    // than a second launch costs.
    const dim3 grid((unsigned)(runs <= 4 ? 1 : runs < 8L * num_sms ? runs : 8L * num_sms));
    if (runs > 4) {
        const cudaError_t e = launch_pdl(scale_init_kernel, dim3(1), dim3(32), 0, s, g);
        if (e != cudaSuccess) return e;
    }
    return x_type == TGEMM_TYPE_F32
               ? launch_pdl(tensor_scale_kernel<float>, grid, dim3(256), 0, s, r, c, static_cast<const float*>(X), ldx,
                            vec, shift, g)
               : launch_pdl(tensor_scale_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, r, c,
                            static_cast<const __nv_bfloat16*>(X), ldx, vec, shift, g);
}

cudaError_t mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                         const float* g, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                         uint8_t* scales_t, int num_sms, cudaStream_t s) {
    if (x_type == TGEMM_TYPE_F32)
        return fmt == TGEMM_MXFP4
                   ? quantize_type<float, TGEMM_MXFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s)
                   : quantize_type<float, TGEMM_NVFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s);
    return fmt == TGEMM_MXFP4
               ? quantize_type<__nv_bfloat16, TGEMM_MXFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s)
               : quantize_type<__nv_bfloat16, TGEMM_NVFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, num_sms, s);
}

template <typename T>
static cudaError_t dequantize_type(int rows, int cols, const uint8_t* codes, const uint8_t* scales,
                                   int fmt, const float* g, void* X, long ldx, cudaStream_t s) {
    const dim3 grid((unsigned)(((long)cols + 2047) / 2048), grid_rows(((long)rows + 7) / 8));
    const dim3 any((unsigned)(((long)cols + 255) / 256), grid.y);
    auto x = static_cast<T*>(X);
    if (!rows_on_16(X, ldx, sizeof(T)))
        return fmt == TGEMM_MXFP4
                   ? launch_pdl(dequantize_any_kernel<T, TGEMM_MXFP4>, any, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx)
                   : launch_pdl(dequantize_any_kernel<T, TGEMM_NVFP4>, any, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx);
    return fmt == TGEMM_MXFP4
               ? launch_pdl(dequantize_kernel<T, TGEMM_MXFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx)
               : launch_pdl(dequantize_kernel<T, TGEMM_NVFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx);
}

cudaError_t mx4_dequantize(int rows, int cols, const uint8_t* codes, const uint8_t* scales,
                           int fmt, const float* g, void* X, long ldx, int x_type, cudaStream_t s) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    return x_type == TGEMM_TYPE_F32
               ? dequantize_type<float>(rows, cols, codes, scales, fmt, g, X, ldx, s)
               : dequantize_type<__nv_bfloat16>(rows, cols, codes, scales, fmt, g, X, ldx, s);
}

cudaError_t mx4_pack(int rows, int cols, int fmt, const uint8_t* src_codes, long src_ldc,
                     const uint8_t* src_scales, long src_lds, uint8_t* codes, uint8_t* scales,
                     cudaStream_t s) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const long n = mx4_pitch(cols) > mx4_tiles_k(cols, fmt) * 4 ? mx4_pitch(cols)
                                                                : mx4_tiles_k(cols, fmt) * 4;
    const dim3 grid((unsigned)((n + 255) / 256), grid_rows(((long)rows + 127) / 128 * 128));
    return fmt == TGEMM_MXFP4
               ? launch_pdl(pack_kernel<TGEMM_MXFP4>, grid, dim3(256), 0, s, rows, cols, src_codes, src_ldc, src_scales, src_lds, codes, scales)
               : launch_pdl(pack_kernel<TGEMM_NVFP4>, grid, dim3(256), 0, s, rows, cols, src_codes, src_ldc, src_scales, src_lds, codes, scales);
}

}  // namespace tgemm
