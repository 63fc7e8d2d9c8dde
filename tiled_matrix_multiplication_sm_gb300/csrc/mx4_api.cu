// C ABI of the 4-bit operators: argument checks and dispatch. The contract
// of every entry point is in include/tgemm_mx4.h.

#include "mx4_internal.h"

#include <cstdint>

namespace {

using tgemm::Mx4Operand;
using tgemm::Mx4Out;

bool valid_fmt(int fmt) { return fmt == TGEMM_MXFP4 || fmt == TGEMM_NVFP4; }
bool valid_type(int t) { return t == TGEMM_TYPE_F32 || t == TGEMM_TYPE_BF16; }
bool off(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool valid_dim(int n) { return n >= 0 && n <= TGEMM_MX4_MAX_DIM; }
size_t type_bytes(int t) { return t == TGEMM_TYPE_F32 ? 4 : 2; }

// A matrix of `type` elements that is not empty.
int check_matrix(const void* X, long ldx, int cols, int type) {
    if (ldx < cols || X == nullptr || off(X, type_bytes(type))) return TGEMM_ERR_INVALID_ARG;
    return TGEMM_OK;
}

int check_g(const float* g, int fmt) {
    return (g != nullptr && fmt == TGEMM_MXFP4) || off(g, 4) ? TGEMM_ERR_INVALID_ARG : TGEMM_OK;
}

// A 4-bit matrix that is not empty.
int check_mx4(const void* codes, const void* scales) {
    if (codes == nullptr || scales == nullptr) return TGEMM_ERR_INVALID_ARG;
    return off(codes, 16) || off(scales, 16) ? TGEMM_ERR_ALIGNMENT : TGEMM_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? TGEMM_OK : TGEMM_ERR_CUDA; }

// The output of a product and what both products have in common. TGEMM_OK,
// an error, or -1 for an empty output.
int check_product(int M, int N, int K, const float* ga, const Mx4Operand& B, int fmt,
                  const Mx4Out& o) {
    if (!valid_dim(M) || !valid_dim(N) || !valid_dim(K) || !valid_fmt(fmt) || !valid_type(o.c_type) || o.ldc < N)
        return TGEMM_ERR_INVALID_ARG;
    if (check_g(ga, fmt) != TGEMM_OK || check_g(B.g, fmt) != TGEMM_OK || off(o.bias, 4))
        return TGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return -1;
    const int st = check_matrix(o.C, o.ldc, N, o.c_type);
    if (st != TGEMM_OK || K == 0) return st;
    return check_mx4(B.codes, B.scales);
}

Mx4Operand operand(const void* codes, const void* scales, const float* g) {
    return {static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), g};
}

}  // namespace

extern "C" {

long long gemm_mx4_codes_pitch(int cols) {
    return !valid_dim(cols) ? -TGEMM_ERR_INVALID_ARG : tgemm::mx4_pitch(cols);
}

long long gemm_mx4_scales_bytes(int rows, int cols, int fmt) {
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_fmt(fmt)) return -TGEMM_ERR_INVALID_ARG;
    return (long long)tgemm::mx4_scale_bytes(rows, cols, fmt);
}

int gemm_mx4_tensor_scale(int rows, int cols, const void* X, long ldx, int x_type, float* g,
                          cudaStream_t stream) {
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_type(x_type) || g == nullptr || off(g, 4) || ldx < cols)
        return TGEMM_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && check_matrix(X, ldx, cols, x_type) != TGEMM_OK)
        return TGEMM_ERR_INVALID_ARG;
    int sms = 0;
    const int st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_tensor_scale(rows, cols, X, ldx, x_type, g, sms, stream));
}

int gemm_mx4_quantize(int rows, int cols, const void* X, long ldx, int x_type, int fmt,
                      float* g, int flags, void* codes, void* scales, void* codes_t, void* scales_t,
                      cudaStream_t stream) {
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_type(x_type) || !valid_fmt(fmt) || ldx < cols)
        return TGEMM_ERR_INVALID_ARG;
    if (check_g(g, fmt) != TGEMM_OK || (flags & ~TGEMM_MX4_SET_G) != 0 || (flags != 0 && g == nullptr))
        return TGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0)
        return flags != 0 ? gemm_mx4_tensor_scale(rows, cols, X, ldx, x_type, g, stream) : TGEMM_OK;
    if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr) ||
        (codes == nullptr && codes_t == nullptr))
        return TGEMM_ERR_INVALID_ARG;
    int st = check_matrix(X, ldx, cols, x_type);
    if (st == TGEMM_OK && codes != nullptr) st = check_mx4(codes, scales);
    if (st == TGEMM_OK && codes_t != nullptr) st = check_mx4(codes_t, scales_t);
    int sms = 0;
    if (st == TGEMM_OK) st = tgemm::device_sms(&sms);
    if (st == TGEMM_OK && flags != 0) st = done(tgemm::mx4_tensor_scale(rows, cols, X, ldx, x_type, g, sms, stream));
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_quantize(rows, cols, X, ldx, x_type, fmt, g, static_cast<uint8_t*>(codes),
                                    static_cast<uint8_t*>(scales), static_cast<uint8_t*>(codes_t),
                                    static_cast<uint8_t*>(scales_t), sms, stream));
}

int gemm_mx4_dequantize(int rows, int cols, const void* codes, const void* scales, int fmt,
                        const float* g, void* X, long ldx, int x_type, cudaStream_t stream) {
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_type(x_type) || !valid_fmt(fmt) || ldx < cols)
        return TGEMM_ERR_INVALID_ARG;
    if (check_g(g, fmt) != TGEMM_OK) return TGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TGEMM_OK;
    int st = check_matrix(X, ldx, cols, x_type);
    if (st == TGEMM_OK) st = check_mx4(codes, scales);
    int sms = 0;
    if (st == TGEMM_OK) st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_dequantize(rows, cols, static_cast<const uint8_t*>(codes),
                                      static_cast<const uint8_t*>(scales), fmt, g, X, ldx, x_type,
                                      stream));
}

int gemm_mx4_pack(int rows, int cols, int fmt, const void* src_codes, long src_ldc,
                  const void* src_scales, long src_lds, void* codes, void* scales,
                  cudaStream_t stream) {
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_fmt(fmt)) return TGEMM_ERR_INVALID_ARG;
    const int block = tgemm::mx4_block(fmt);
    if (src_ldc < ((long)cols + 1) / 2 || src_lds < ((long)cols + block - 1) / block)
        return TGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TGEMM_OK;
    if (src_codes == nullptr || src_scales == nullptr) return TGEMM_ERR_INVALID_ARG;
    int st = check_mx4(codes, scales);
    int sms = 0;
    if (st == TGEMM_OK) st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_pack(rows, cols, fmt, static_cast<const uint8_t*>(src_codes), src_ldc,
                                static_cast<const uint8_t*>(src_scales), src_lds,
                                static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), stream));
}

int gemm_mx4(int M, int N, int K, const void* a_codes, const void* a_scales, const float* ga,
             const void* b_codes, const void* b_scales, const float* gb, int fmt, void* C,
             long ldc, int c_type, float alpha, float beta, const float* bias,
             cudaStream_t stream) {
    const Mx4Operand A = operand(a_codes, a_scales, ga), B = operand(b_codes, b_scales, gb);
    const Mx4Out out{C, ldc, c_type, alpha, beta, bias};
    int st = check_product(M, N, K, ga, B, fmt, out);
    if (st == -1) return TGEMM_OK;
    if (st == TGEMM_OK && K > 0) st = check_mx4(a_codes, a_scales);
    int sms = 0;
    if (st == TGEMM_OK) st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_gemm(M, N, K, A, B, fmt, out, sms, stream));
}

int gemm_w4(int M, int N, int K, const void* A, long lda, const void* b_codes,
            const void* b_scales, const float* gb, int fmt, void* C, long ldc, int c_type,
            float alpha, float beta, const float* bias, cudaStream_t stream) {
    const Mx4Operand B = operand(b_codes, b_scales, gb);
    const Mx4Out out{C, ldc, c_type, alpha, beta, bias};
    if (lda < K) return TGEMM_ERR_INVALID_ARG;
    int st = check_product(M, N, K, nullptr, B, fmt, out);
    if (st == -1) return TGEMM_OK;
    if (st == TGEMM_OK && K > 0) st = check_matrix(A, lda, K, TGEMM_TYPE_BF16);
    int sms = 0;
    if (st == TGEMM_OK) st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(tgemm::mx4_weights(M, N, K, A, lda, B, fmt, out, sms, stream));
}

}  // extern "C"
