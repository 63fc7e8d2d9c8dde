/*
 * tgemm_fused — products of BF16 matrices with what follows them in a model's
 * layers computed in their epilogue, on one NVIDIA GB300 (sm_103a): activations
 * with bias, gating and residual, their gradient, and the softmax cross entropy
 * of a head over its vocabulary with its gradients.
 *
 * Part of libtgemm.so; a C ABI like tgemm.h, with its status codes, its rules
 * on streams, CUDA graphs, threads and scratch memory (stream-ordered, from the
 * library's pool), and its bounded waits (gemm_device_status). Matrices are
 * row-major with a leading dimension, of BF16 elements where no type is given;
 * TGEMM_TYPE_* are those of tgemm_mx4.h. Any alignment to the element size is
 * taken; rows on 16-byte boundaries are read and written as they are, operands
 * off them are copied to scratch first (with rows on 16-byte boundaries).
 * Sizes are at most TGEMM_FUSED_MAX_DIM. Results must not overlap operands,
 * but for what an entry says.
 *
 * Sums of products are FP32: on the tensor cores, which cut low bits off at
 * every step. Where a result keeps 32 bits long sums are made of parts, added
 * with rounding to nearest, so that it is off by 1e-6 of its norm or less where
 * terms have random signs, 2e-6 where all have one (an FP32 C and db: parts of up to
 * 1152 columns of K; loss and lse: 256; a bias or residual that cancels
 * most of the sums leaves that much of the sums' norm, and a loss far below its
 * logits is off by 4e-7 of them; gemm_ce_grad's results are as exact as its BF16 dz).
 * Sums that end in BF16 are one part, which loses less than their rounding up to K =
 * 65536 (4e-4 of the norm where all terms have one sign, 1.6e-3 at 262144). Values
 * go from the sum to the result in FP32 and are rounded once, to nearest even,
 * where the result is BF16.
 *
 * Activations, act(z):
 *   TGEMM_ACT_NONE       z
 *   TGEMM_ACT_RELU       max(z, 0); its slope at 0 is 0
 *   TGEMM_ACT_GELU       z Phi(z), Phi the normal distribution
 *   TGEMM_ACT_GELU_TANH  z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2
 *   TGEMM_ACT_SILU       z / (1 + exp(-z))
 * Evaluated in FP32 they are off by 2^-20 of themselves and, below zero, by what the
 * roundings of their exponents make (SILU 2^-24 |z| more, GELU 2^-23 z^2 / 2).
 */
#ifndef TGEMM_FUSED_H
#define TGEMM_FUSED_H

#include "tgemm.h"
#include "tgemm_mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest M, N, K, T, V or D: two halves of a gated operand, and tiles' ends, stay in
 * an int. */
#define TGEMM_FUSED_MAX_DIM 1073741312

#define TGEMM_ACT_NONE      0
#define TGEMM_ACT_RELU      1
#define TGEMM_ACT_GELU      2
#define TGEMM_ACT_GELU_TANH 3
#define TGEMM_ACT_SILU      4

/* A flag beside TGEMM_TRANS_A and TGEMM_TRANS_B. */
#define TGEMM_GATED 4

/*
 * gemm_act — a layer's product with its bias, activation and residual:
 *
 *     z = op(A) op(B) + bias,   Z = z,   C = act(z) + R
 *
 * op(A) is M x K and op(B) K x N, stored as in gemm_ex: with TGEMM_TRANS_A A is
 * kept K x M, with TGEMM_TRANS_B B is kept N x K (a weight matrix with a row
 * for each output). C is M x N, c_type TGEMM_TYPE_BF16 or _F32. May be NULL:
 * bias (N floats), R (M x N, r_type BF16 or FP32; it may be C itself, with C's
 * ld and type) and Z (M x N, BF16, written for gemm_act_grad).
 *
 * TGEMM_GATED: op(B) has 2 N columns, and so have bias and Z (M x 2 N); with
 * z = [g, u], C = act(g) u + R. It takes a BF16 C.
 *
 * K == 0 makes sums of 0; M == 0 or N == 0 is a no-op. Returns TGEMM_OK,
 * TGEMM_ERR_INVALID_ARG (a size out of range, a leading dimension below its
 * row's length, a null or misaligned pointer, an unknown act, type or flag, a
 * gated product with an FP32 C), TGEMM_ERR_UNSUPPORTED or TGEMM_ERR_CUDA.
 */
TGEMM_API int gemm_act(int M, int N, int K, const void* A, long lda, const void* B, long ldb, int flags, int act,
                       const float* bias, const void* R, long ldr, int r_type, void* Z, long ldz,
                       void* C, long ldc, int c_type, cudaStream_t stream);

/*
 * gemm_act_grad — the backward pass through the next layer's product and this
 * layer's activation:
 *
 *     d = op(A) op(B),   dZ = d act'(Z),   db[j] = sum over i of dZ[i][j]
 *
 * say A = dY and B the next layer's weights (kept outputs x inputs: no flags).
 * Z is the one that gemm_act wrote, M x N; dZ is M x N, dz_type BF16 or FP32
 * (it may be Z itself if it has Z's ld and BF16); db, NULL or N floats, sums
 * the dZ before their rounding, rows in blocks (32 on SM pairs, 8 to 64 in few
 * tiles; scratch: 4 bytes for each block and column), in the same order for the
 * same call.
 *
 * TGEMM_GATED: Z = [g, u] and dZ are M x 2 N (BF16), db has 2 N entries:
 * dZ = [d u act'(g), d act(g)].
 *
 * Sizes of 0 and errors as gemm_act; with M == 0 db is zeros.
 */
TGEMM_API int gemm_act_grad(int M, int N, int K, const void* A, long lda, const void* B, long ldb, int flags, int act,
                            const void* Z, long ldz, void* dZ, long lddz, int dz_type, float* db,
                            cudaStream_t stream);

/*
 * gemm_ce — softmax cross entropy of T tokens over a vocabulary of V entries,
 * without keeping the logits z = alpha X W^T:
 *
 *     lse[i] = log sum over j of exp z[i][j],   loss[i] = lse[i] - z[i][target[i]]
 *
 * X is T x D, W is V x D; target (T entries of 64 bits), loss and lse (T floats
 * each) are in device memory. A row whose target is not in 0 .. V - 1 is left
 * out: its loss is 0 whatever X holds there. Each 128 columns of the
 * vocabulary or so leave a maximum and a sum for each token (scratch: 8 bytes for
 * each of them; tokens are taken in turns of 256 MB of it).
 *
 * T == 0 is a no-op. Errors as gemm_act, and TGEMM_ERR_INVALID_ARG for an
 * alpha that is not finite.
 */
TGEMM_API int gemm_ce(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha,
                      const long long* target, float* loss, float* lse, cudaStream_t stream);

/*
 * gemm_ce_grad — the gradients of sum over i of dloss[i] loss[i], given gemm_ce's
 * lse (or any other):
 *
 *     dz[i][j] = alpha dloss[i] (exp(z[i][j] - lse[i]) - [j == target[i]])
 *     dX = dz W,   dW = dz^T X + beta dW
 *
 * dz is made from X and W again, in BF16 scratch, for as many columns at a time
 * as 256 MB hold (1024 at least), so that memory does not grow with the
 * vocabulary; over more than one such piece dX is summed in FP32, in scratch or, one
 * of FP32 with rows on 16 bytes and D a multiple of 4, where it is. dX
 * (T x D) and dW (V x D) are BF16 or FP32; either may be NULL. In either type
 * they carry dz's rounding (half a step of BF16, 2^-8 of each at most): up to 2.3e-3
 * of their norm, beside the 1.7e-3 of a BF16 result's own. z is summed as in gemm_ce,
 * and dz of the target is a difference that keeps its digits: of a sure token it is as
 * exact as its lse, off by 2^-23 of lse over 1 - p (p the target's probability). dW is not read
 * when beta == 0. Rows left out (see gemm_ce) get a dX of 0 and add nothing to
 * dW, whatever X, lse and dloss hold there (with a finite W).
 *
 * Sizes of 0 give sums of 0. Errors as gemm_ce, and TGEMM_ERR_INVALID_ARG for a
 * beta that is not finite.
 */
TGEMM_API int gemm_ce_grad(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha,
                           const long long* target, const float* lse, const float* dloss,
                           void* dX, long lddx, int dx_type, void* dW, long lddw, int dw_type, float beta,
                           cudaStream_t stream);

/*
 * gemm_set_fused_kernel — the kernel of these products, for tests and tuning:
 * -1 by a model of their times (the default), 0 always 256 x 256 tiles on SM
 * pairs, 1 always few tiles on one SM each. Process-wide, for calls made
 * after it. Returns TGEMM_OK or TGEMM_ERR_INVALID_ARG.
 */
TGEMM_API int gemm_set_fused_kernel(int mode);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_FUSED_H */
