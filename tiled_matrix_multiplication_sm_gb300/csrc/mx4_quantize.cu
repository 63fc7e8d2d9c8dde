// Quantising to 4-bit floating point with block scales, reading back, and the
// import of row-major codes and scales. Formats and layout are described in
// include/tgemm_mx4.h.

#include "mx4_internal.h"

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

// The scale byte of a block whose largest |x| has the bits `m`, the divisor d
// of its values and 1 / d (0, 0: every code is 0).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t m, float g, float& d, float& inv) {
    d = inv = 0.0f;
    if (m >= 0x7F800000u) return FMT == TGEMM_MXFP4 ? 0xFF : 0x7F;   // an infinity or a NaN in the block
    if (FMT == TGEMM_MXFP4) {
        const int e = (int)(m >> 23) - 2;         // biased floor(log2 m), minus 2
        const uint32_t byte = e > 0 ? (uint32_t)e : 0u;
        inv = __uint_as_float((254u - byte) << 23);     // exact: 2^(127 - byte)
        return byte;
    }
    if (!(g >= kMinG && g <= kMaxG)) return 0x7F;
    const uint32_t byte = e4m3(__fdiv_rn(__uint_as_float(m), 6.0f * g));
    if (byte != 0) {
        d = e4m3_value(byte) * g;
        inv = __frcp_rn(d);
    }
    return byte;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Two values over d. A power of two (MXFP4) multiplies exactly. An NVFP4
// divisor needs a true quotient, or values that lie on the midpoint of two
// codes (common: BF16 values over scales of 4 bits) would round either way:
// q = x / d from the correctly rounded reciprocal with one correction step,
// q + (x - q d) inv, which rounds correctly (Markstein, 1990).
template <int FMT>
__device__ __forceinline__ void divide2(float& x0, float& x1, uint64_t inv2, uint64_t negd2) {
    const uint64_t x = pack2(x0, x1);
    uint64_t q = fma2(x, inv2, 0);
    if (FMT == TGEMM_NVFP4) q = fma2(fma2(q, negd2, x), inv2, q);
    unpack2(q, x0, x1);
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

// 1 << shift threads to a row (rows that start on 16-byte boundaries in
// 16-byte pieces, `vec`); bound by reading X.
template <typename T>
__global__ void __launch_bounds__(256)
tensor_scale_kernel(int rows, int cols, const T* X, long ldx, bool vec, int shift, float* g) {
    constexpr int V = 16 / (int)sizeof(T);
    pdl_launch_dependents();
    pdl_wait();
    uint32_t m = 0;
    auto take = [&](uint32_t b) {
        b &= 0x7FFFFFFFu;
        if (b < 0x7F800000u) m = max(m, b);
    };
    const int width = vec ? V : 1, step = width << shift;
    const int first = (threadIdx.x & ((1 << shift) - 1)) * width;
    const int per_block = 256 >> shift;
    for (long r = (long)blockIdx.x * per_block + (threadIdx.x >> shift); r < rows; r += (long)gridDim.x * per_block) {
        const T* row = X + r * ldx;
#pragma unroll 8
        for (long c = first; c < cols; c += step) {
            if (vec && c + V <= cols) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + c));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (sizeof(T) == 4) take(w[k]);
                    else {
                        take(w[k] << 16);
                        take(w[k] & 0xFFFF0000u);
                    }
                }
            } else {
                for (int k = 0; k < width; ++k)
                    if (c + k < cols) take(__float_as_uint((float)row[c + k]));
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
        if (threadIdx.x == 0 && m != 0)
            atomicMax(reinterpret_cast<unsigned*>(g), __float_as_uint(power_for(__uint_as_float(m))));
    }
}

// Quantising, one block of threads to a 128 x 128 tile of X staged in shared
// memory: in it both directions read 128 rows of 128 / B blocks, and both
// write whole scale tiles and 64-byte runs of codes, so X is read once even
// when its transpose is wanted too. Bound by HBM (X in, codes and scales out).
constexpr int QT = 128;
constexpr int Q_THREADS = 256;
constexpr int Q_CODES = 80;       // bytes between staged rows of transposed codes (64 used)

template <typename T> __host__ __device__ constexpr int q_pitch() { return QT * (int)sizeof(T) + 16; }   // bytes
template <typename T> __host__ __device__ constexpr int q_smem() { return QT * q_pitch<T>() + QT * Q_CODES + 2 * 1024; }

// Largest |x| of two packed BF16, or of one FP32, as an integer per half.
template <typename T>
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t v) {
    if constexpr (sizeof(T) == 2) return __vmaxu2(m, v & 0x7FFF7FFFu);
    else return max(m, v & 0x7FFFFFFFu);
}

// The codes of B values held as words of T, and the block's scale byte.
template <typename T, int FMT>
__device__ __forceinline__ uint32_t quantize_block(const uint32_t* w, float g, uint32_t* codes) {
    constexpr int B = mx4_block(FMT), WORDS = B * (int)sizeof(T) / 4;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) m = max_abs<T>(m, w[i]);
    if constexpr (sizeof(T) == 2) m = max(m << 16, m & 0xFFFF0000u);
    float d, inv;
    const uint32_t byte = block_scale<FMT>(m, g, d, inv);
    const uint64_t inv2 = pack2(inv, inv), negd2 = pack2(-d, -d);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t v = w[i * 4 + j / 2];
                x[j] = __uint_as_float(v << 16);
                x[j + 1] = __uint_as_float(v & 0xFFFF0000u);
            } else {
                x[j] = __uint_as_float(w[i * 8 + j]);
                x[j + 1] = __uint_as_float(w[i * 8 + j + 1]);
            }
            divide2<FMT>(x[j], x[j + 1], inv2, negd2);
        }
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(codes[i]) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    }
    return byte;
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

template <typename T, int FMT, bool ROWS, bool TRANS>
__global__ void __launch_bounds__(Q_THREADS)
quantize_kernel(int R, int C, const T* X, long ldx, bool vec, const float* gp, uint8_t* codes,
                uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t) {
    constexpr int B = mx4_block(FMT), NB = QT / B, WORDS = B * (int)sizeof(T) / 4;
    constexpr int PITCH = q_pitch<T>(), SCALE_BYTES = NB / 4 * MX4_TILE_BYTES;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* staged = smem + QT * PITCH;                    // transposed codes
    uint8_t* sc = staged + QT * Q_CODES;                    // scales, then those of the transpose
    const int t = threadIdx.x, lane = t & 31;
    const long c0 = (long)blockIdx.x * QT;
    pdl_launch_dependents();
    pdl_wait();
    const float g = mx4_g(gp);
    // The scales cover spans of 256, so the grid goes on to an even tile.
    const long end = ((long)R + 2 * QT - 1) / (2 * QT) * (2 * QT);
    for (long r0 = (long)blockIdx.y * QT; r0 < end; r0 += (long)gridDim.y * QT) {
        // Load, zeros outside.
        if (vec) {
            constexpr int V = 16 / (int)sizeof(T), PER_ROW = QT / V;
#pragma unroll 4
            for (int i = t; i < QT * PER_ROW; i += Q_THREADS) {
                const int r = i / PER_ROW, c = i % PER_ROW * V;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r0 + r < R && c0 + c < C) {
                    const T* src = X + (r0 + r) * ldx + c0 + c;
                    if (c0 + c + V <= C) v = __ldg(reinterpret_cast<const uint4*>(src));
                    else {
                        alignas(16) T part[V];
#pragma unroll
                        for (int k = 0; k < V; ++k) part[k] = c0 + c + k < C ? src[k] : (T)0.0f;
                        v = *reinterpret_cast<const uint4*>(part);
                    }
                }
                *reinterpret_cast<uint4*>(smem + r * PITCH + c * (int)sizeof(T)) = v;
            }
        } else {
#pragma unroll 8
            for (int i = t; i < QT * QT; i += Q_THREADS) {
                const int r = i / QT, c = i % QT;
                *reinterpret_cast<T*>(smem + r * PITCH + c * (int)sizeof(T)) =
                    r0 + r < R && c0 + c < C ? X[(r0 + r) * ldx + c0 + c] : (T)0.0f;
            }
        }
        __syncthreads();
        if (ROWS) {
            const long pitch = mx4_pitch(C);
            // 8 lanes take 8 rows: their 16-byte reads fall in different banks.
#pragma unroll 1
            for (int i = t >> 5; i < QT * NB / 32; i += Q_THREADS / 32) {
                const int row = i / (NB / 4) * 8 + (lane & 7), b = i % (NB / 4) * 4 + (lane >> 3);
                uint32_t w[WORDS], out[B / 8];
#pragma unroll
                for (int k = 0; k < WORDS / 4; ++k) {
                    const uint4 v = *reinterpret_cast<const uint4*>(smem + row * PITCH + b * B * (int)sizeof(T) + k * 16);
                    w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
                }
                sc[tile_scale_at(row, b)] = (uint8_t)quantize_block<T, FMT>(w, g, out);
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
                uint32_t w[2][WORDS], out[B / 8];
                const uint8_t* src = smem + b * B * PITCH + c * (int)sizeof(T);
#pragma unroll
                for (int k = 0; k < WORDS; ++k) {
                    if constexpr (sizeof(T) == 2) {
                        const uint32_t u = *reinterpret_cast<const uint32_t*>(src + 2 * k * PITCH);
                        const uint32_t v = *reinterpret_cast<const uint32_t*>(src + (2 * k + 1) * PITCH);
                        w[0][k] = __byte_perm(u, v, 0x5410);
                        w[1][k] = __byte_perm(u, v, 0x7632);
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(src + k * PITCH);
                        w[0][k] = u.x;
                        w[1][k] = u.y;
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sc[1024 + tile_scale_at(c + h, b)] = (uint8_t)quantize_block<T, FMT>(w[h], g, out);
                    uint8_t* dst = staged + (c + h) * Q_CODES + b * (B / 2);
                    if constexpr (B == 32) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
                    else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
                }
            }
        }
        __syncthreads();
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
        __syncthreads();
    }
}

// Eight codes a thread, several rows in flight; bound by writing X.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(int R, int C, const uint8_t* codes, const uint8_t* scales, const float* gp, T* X,
                  long ldx, bool vec) {
    constexpr int B = mx4_block(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const long c = ((long)blockIdx.x * blockDim.x + threadIdx.x) * 8;
    if (c >= C) return;
    const float g = mx4_g(gp);
    const long pitch = mx4_pitch(C), tiles_k = mx4_tiles_k(C, FMT);
#pragma unroll 4
    for (long r = blockIdx.y; r < R; r += gridDim.y) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + r * pitch + c / 2));
        const float s = mx4_scale_value<FMT>(__ldg(scales + mx4_scale_at(r, c / B, tiles_k)));
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;      // two codes as halves
            asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(w >> 8 * j));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * j] = f.x * s * g;
            v[2 * j + 1] = f.y * s * g;
        }
        T* dst = X + r * ldx + c;
        if (vec && c + 8 <= C) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(b);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < C) dst[j] = (T)v[j];
        }
    }
}

// One thread moves 16 bytes of codes or, in the second part of the grid's
// work, one scale byte.
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
                            uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, cudaStream_t s) {
    const cudaError_t e = set_smem_limit_once<quantize_kernel<T, FMT, ROWS, TRANS>>(q_smem<T>());
    if (e != cudaSuccess) return e;
    const long rows = ((long)R + 255) / 256 * 2;
    const dim3 grid((unsigned)(((long)C + 255) / 256 * 2), (unsigned)(rows < 65535 ? rows : 65535));
    return launch_pdl(quantize_kernel<T, FMT, ROWS, TRANS>, grid, dim3(Q_THREADS), q_smem<T>(), s, R, C,
                      static_cast<const T*>(X), ldx, rows_on_16(X, ldx, sizeof(T)), g, codes, scales, codes_t,
                      scales_t);
}

template <typename T, int FMT>
cudaError_t quantize_type(int R, int C, const void* X, long ldx, const float* g, uint8_t* codes,
                          uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, cudaStream_t s) {
    if (codes_t == nullptr)
        return launch_quantize<T, FMT, true, false>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, s);
    if (codes == nullptr)
        return launch_quantize<T, FMT, false, true>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, s);
    return launch_quantize<T, FMT, true, true>(R, C, X, ldx, g, codes, scales, codes_t, scales_t, s);
}

}  // namespace

cudaError_t mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type, float* g,
                             int num_sms, cudaStream_t s) {
    cudaError_t e = launch_pdl(scale_init_kernel, dim3(1), dim3(32), 0, s, g);
    if (e != cudaSuccess || rows == 0 || cols == 0) return e;
    const int esz = x_type == TGEMM_TYPE_F32 ? 4 : 2;
    const bool vec = rows_on_16(X, ldx, esz);
    const long pieces = vec ? ((long)cols * esz + 15) / 16 : cols;
    int shift = 5;
    while (shift < 8 && (1L << shift) < pieces) ++shift;
    const long blocks = ((long)rows + (256 >> shift) - 1) / (256 >> shift);
    const dim3 grid((unsigned)(blocks < 8L * num_sms ? blocks : 8L * num_sms));
    return x_type == TGEMM_TYPE_F32
               ? launch_pdl(tensor_scale_kernel<float>, grid, dim3(256), 0, s, rows, cols,
                            static_cast<const float*>(X), ldx, vec, shift, g)
               : launch_pdl(tensor_scale_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, rows, cols,
                            static_cast<const __nv_bfloat16*>(X), ldx, vec, shift, g);
}

cudaError_t mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                         const float* g, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                         uint8_t* scales_t, cudaStream_t s) {
    if (x_type == TGEMM_TYPE_F32)
        return fmt == TGEMM_MXFP4
                   ? quantize_type<float, TGEMM_MXFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, s)
                   : quantize_type<float, TGEMM_NVFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, s);
    return fmt == TGEMM_MXFP4
               ? quantize_type<__nv_bfloat16, TGEMM_MXFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, s)
               : quantize_type<__nv_bfloat16, TGEMM_NVFP4>(rows, cols, X, ldx, g, codes, scales, codes_t, scales_t, s);
}

template <typename T>
static cudaError_t dequantize_type(int rows, int cols, const uint8_t* codes, const uint8_t* scales,
                                   int fmt, const float* g, void* X, long ldx, cudaStream_t s) {
    const dim3 grid((unsigned)(((long)cols + 2047) / 2048), grid_rows(((long)rows + 3) / 4));
    const bool vec = rows_on_16(X, ldx, sizeof(T));
    auto x = static_cast<T*>(X);
    return fmt == TGEMM_MXFP4
               ? launch_pdl(dequantize_kernel<T, TGEMM_MXFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx, vec)
               : launch_pdl(dequantize_kernel<T, TGEMM_NVFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, x, ldx, vec);
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
