// Quantising to 4-bit floating point with block scales, reading back, and the
// import of row-major codes and scales. Formats and layout are described in
// include/tgemm_mx4.h.

#include "mx4_internal.h"

namespace tgemm {
namespace {

constexpr float kMinG = 7.888609052210118e-31f;      // 2^-100
constexpr float kMaxG = 1.661534994731145e+35f;      // 2^117

template <typename T>
__device__ __forceinline__ float load_f32(const T* p) { return (float)*p; }

// Two FP32 values to a byte of two E2M1 codes (nearest even, saturating).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFF;
}

// The scale byte of a block whose largest |x| has the bits `m`, and the
// divisor of its values (0: every code is 0).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t m, float g, float& divisor) {
    if (m >= 0x7F800000u) {                       // an infinity or a NaN in the block
        divisor = 0.0f;
        return FMT == TGEMM_MXFP4 ? 0xFF : 0x7F;
    }
    if (FMT == TGEMM_MXFP4) {
        const int e = (int)(m >> 23) - 2;         // biased floor(log2 m), minus 2
        const uint32_t byte = e > 0 ? (uint32_t)e : 0u;
        divisor = e8m0_value(byte);
        return byte;
    }
    if (!(g >= kMinG && g <= kMaxG)) {
        divisor = 0.0f;
        return 0x7F;
    }
    const uint32_t byte = e4m3(__fdiv_rn(__uint_as_float(m), 6.0f * g));
    divisor = e4m3_value(byte) * g;
    return byte;
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

template <typename T>
__global__ void __launch_bounds__(256)
tensor_scale_kernel(int rows, int cols, const T* X, long ldx, float* g) {
    pdl_launch_dependents();
    pdl_wait();
    uint32_t m = 0;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            const uint32_t b = __float_as_uint(load_f32(X + (long)r * ldx + c)) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) m = max(m, b);
        }
    m = __reduce_max_sync(0xffffffffu, m);
    // Positive floats order as their bits, and g only grows with |x|.
    if ((threadIdx.x & 31) == 0 && m != 0)
        atomicMax(reinterpret_cast<unsigned*>(g), __float_as_uint(power_for(__uint_as_float(m))));
}

// One thread quantises one block of a row of the R x C matrix whose element
// (r, c) is X[r * rs + c * cs]; blocks and rows up to the end of the scale
// tiles get scale 0, and codes past C are 0.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
quantize_kernel(int R, int C, const T* X, long rs, long cs, const float* gp, uint8_t* codes,
                uint8_t* scales) {
    constexpr int B = mx4_block(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const long tiles_k = mx4_tiles_k(C, FMT);
    const long nb = tiles_k * 4;
    const long b = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= nb) return;
    const float g = mx4_g(gp);
    for (long r = blockIdx.y; r < ((long)R + 127) / 128 * 128; r += gridDim.y) {
        uint32_t byte = 0;
        if (r < R && b * B < C) {
            const T* x = X + r * rs + b * B * cs;
            const int n = (int)min((long)B, C - b * B);
            uint32_t m = 0;
            for (int i = 0; i < n; ++i)
                m = max(m, __float_as_uint(load_f32(x + i * cs)) & 0x7FFFFFFFu);
            float d;
            byte = block_scale<FMT>(m, g, d);
            uint8_t* out = codes + r * mx4_pitch(C) + b * (B / 2);
            for (int i = 0; i < B && b * B + i < mx4_pitch(C) * 2; i += 2) {
                const float lo = i < n && d != 0.0f ? __fdiv_rn(load_f32(x + i * cs), d) : 0.0f;
                const float hi = i + 1 < n && d != 0.0f ? __fdiv_rn(load_f32(x + (i + 1) * cs), d) : 0.0f;
                out[i / 2] = (uint8_t)e2m1x2(lo, hi);
            }
        } else if (r < R && b * B < mx4_pitch(C) * 2) {
            for (int i = 0; i < B / 2; ++i) codes[r * mx4_pitch(C) + b * (B / 2) + i] = 0;
        }
        scales[mx4_scale_at(r, b, tiles_k)] = (uint8_t)byte;
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_kernel(int R, int C, const uint8_t* codes, const uint8_t* scales, const float* gp, T* X,
                  long ldx) {
    constexpr int B = mx4_block(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const long c = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C) return;
    const float g = mx4_g(gp);
    for (long r = blockIdx.y; r < R; r += gridDim.y) {
        const uint32_t pair = codes[r * mx4_pitch(C) + c / 2];
        const float s = mx4_scale_value<FMT>(scales[mx4_scale_at(r, c / B, mx4_tiles_k(C, FMT))]);
        X[r * ldx + c] = (T)(e2m1_value((c & 1) ? pair >> 4 : pair & 15) * s * g);
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

template <typename T, int FMT>
cudaError_t launch_quantize(int R, int C, const void* X, long rs, long cs, const float* g,
                            uint8_t* codes, uint8_t* scales, cudaStream_t s) {
    const long nb = mx4_tiles_k(C, FMT) * 4;
    if (nb == 0 || R == 0) return cudaSuccess;
    const dim3 grid((unsigned)((nb + 255) / 256), grid_rows(((long)R + 127) / 128 * 128));
    return launch_pdl(quantize_kernel<T, FMT>, grid, dim3(256), 0, s, R, C,
                      static_cast<const T*>(X), rs, cs, g, codes, scales);
}

template <typename T>
cudaError_t quantize_type(int R, int C, const void* X, long rs, long cs, int fmt, const float* g,
                          uint8_t* codes, uint8_t* scales, cudaStream_t s) {
    return fmt == TGEMM_MXFP4 ? launch_quantize<T, TGEMM_MXFP4>(R, C, X, rs, cs, g, codes, scales, s)
                              : launch_quantize<T, TGEMM_NVFP4>(R, C, X, rs, cs, g, codes, scales, s);
}

}  // namespace

cudaError_t mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type, float* g,
                             int num_sms, cudaStream_t s) {
    cudaError_t e = launch_pdl(scale_init_kernel, dim3(1), dim3(32), 0, s, g);
    if (e != cudaSuccess || rows == 0 || cols == 0) return e;
    const dim3 grid((unsigned)min(rows, 8 * num_sms));
    return x_type == TGEMM_TYPE_F32
               ? launch_pdl(tensor_scale_kernel<float>, grid, dim3(256), 0, s, rows, cols,
                            static_cast<const float*>(X), ldx, g)
               : launch_pdl(tensor_scale_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, rows, cols,
                            static_cast<const __nv_bfloat16*>(X), ldx, g);
}

cudaError_t mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                         const float* g, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                         uint8_t* scales_t, cudaStream_t s) {
    auto run = [&](int R, int C, long rs, long cs, uint8_t* c, uint8_t* sc) {
        return x_type == TGEMM_TYPE_F32 ? quantize_type<float>(R, C, X, rs, cs, fmt, g, c, sc, s)
                                        : quantize_type<__nv_bfloat16>(R, C, X, rs, cs, fmt, g, c, sc, s);
    };
    if (codes != nullptr) {
        const cudaError_t e = run(rows, cols, ldx, 1, codes, scales);
        if (e != cudaSuccess) return e;
    }
    return codes_t != nullptr ? run(cols, rows, 1, ldx, codes_t, scales_t) : cudaSuccess;
}

cudaError_t mx4_dequantize(int rows, int cols, const uint8_t* codes, const uint8_t* scales,
                           int fmt, const float* g, void* X, long ldx, int x_type, cudaStream_t s) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const dim3 grid((unsigned)((cols + 255) / 256), grid_rows(rows));
    auto f = static_cast<float*>(X);
    auto h = static_cast<__nv_bfloat16*>(X);
    if (x_type == TGEMM_TYPE_F32)
        return fmt == TGEMM_MXFP4
                   ? launch_pdl(dequantize_kernel<float, TGEMM_MXFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, f, ldx)
                   : launch_pdl(dequantize_kernel<float, TGEMM_NVFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, f, ldx);
    return fmt == TGEMM_MXFP4
               ? launch_pdl(dequantize_kernel<__nv_bfloat16, TGEMM_MXFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, h, ldx)
               : launch_pdl(dequantize_kernel<__nv_bfloat16, TGEMM_NVFP4>, grid, dim3(256), 0, s, rows, cols, codes, scales, g, h, ldx);
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
