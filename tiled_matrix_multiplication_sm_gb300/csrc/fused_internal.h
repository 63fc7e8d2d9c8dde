// Internal interface of the products with what follows them in their epilogue.
// The public contract is in include/tgemm_fused.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/tgemm_fused.h"
#include "tgemm_internal.h"

namespace tgemm {

// The operands of a product, op(A) M x K and op(B) K x N, BF16.
struct FusedProduct {
    int M, N, K;
    const void* A;
    long lda;
    bool a_mn;                  // kept K x M
    const void* B;
    long ldb;
    bool b_mn;                  // kept K x N
    const void* B2;             // gated: the second N columns of op(B), kept like B
};

// What the epilogue does with a sum.
enum FusedKind {
    FUSED_ACT,                  // C = act(z) + r_scale R, Z = z (gated: C = act(g) u + r_scale R)
    FUSED_GRAD,                 // C = d act'(Z) (gated: the two halves), sums of its columns
    FUSED_CE,                   // m, the maximum of a block of logits, and the sum of exp(z - m); the target's logit
    FUSED_CE_GRAD,              // C = scale dloss (softmax - one hot)
};

struct FusedEpilogue {
    int act = TGEMM_ACT_NONE;
    bool gated = false;
    void* C = nullptr;
    long ldc = 0;
    bool c_f32 = false;
    const float* bias = nullptr;
    const void* R = nullptr;
    long ldr = 0;
    bool r_f32 = false;
    float r_scale = 1.0f;
    void* Z = nullptr;          // FUSED_ACT: written; FUSED_GRAD: read
    long ldz = 0;
    float* sums = nullptr;      // FUSED_GRAD: [blocks of rows][columns of C]
    // Cross entropy.
    float alpha = 1.0f;
    const long long* target = nullptr;
    long first = 0;             // the vocabulary entry of column 0
    long vocabulary = 0;
    const float* lse = nullptr;
    const float* dloss = nullptr;
    float2* parts = nullptr;    // FUSED_CE: [blocks of columns][M], m and sum of exp(z - m)
    float* picked = nullptr;    // FUSED_CE: M logits of the targets
    // FUSED_CE_GRAD: X's rows (whole 16 bytes, `keep_cols` BF16) to `kept`, those whose
    // target is not in the vocabulary as zeros; NULL: none.
    const void* keep = nullptr;
    long ld_keep = 0;
    void* kept = nullptr;
    long ld_kept = 0;
    int keep_cols = 0;
};

// In fused_gemm.cu: rows of C a partial column sum covers, columns of logits a
// maximum and a sum cover.
constexpr int FUSED_SUM_ROWS = 32;
constexpr int FUSED_CE_COLS = 128;

// In fused_few.cu: sets of epilogue warps, each with its sums of columns; bytes of
// shared memory for stages.
constexpr int FUSED_FEW_SETS = 4;
constexpr int FUSED_FEW_RING = 209 * 1024;

// Long sums come in parts where the result keeps 32 bits, in stages of so many
// columns of K: `first` stages for the first two parts, `rest` for the others.
//
// A part of n stages of 64 loses 6.2e-8 n of its sums' norm where terms have random
// signs, nearly all of it in proportion to each sum, and 1.2e-7 n where all have one;
// parts of n_i, the mean of n_i weighted by n_i: their number does not matter. An FP32
// product in torch loses 0.2e-6 to 0.7e-6 in all. So an FP32 C and column sums come in parts of
// a weighted mean of 13: 0.8e-6, 0.95e-6 once SiLU is taken of it (a column a lane, 3000 x
// 5001 x 1537 with R and Z in two parts 93 us for 76 in one of 1.6e-6; column sums of 65536 rows,
// K = 4096, in parts of a mean of 14.5 1.04e-6). A loss is a small difference of large logits,
// off by what its target's loses: parts of 4, for few tokens of 2 (8192 x 65536 x 4096, us, in
// parts of 7, 5, 4, 3: 2206, 2203, 2213, 2287); and the logits that its gradient makes again
// come in the same ones, or exp(z - lse) - 1 of a sure token is off by far more than lse is.
//
// On pairs the MMAs are two parts ahead of the epilogue at most, and that of a
// gated gradient takes 9 us, the time of 34 stages: the first two parts are
// longer (8192 x 14336 x 4096: 711 us in parts of 13, one part 618; an FP32 C of 4096 x 9728 x
// 4096 with GELU 212 in parts of 13, 207 with longer first ones).
struct FusedParts {
    int first, rest;
};
FusedParts fused_parts(FusedKind kind, bool few, int K, int chunk_k);

// How a product runs: on SM pairs (fused_gemm.cu), or as few tiles (fused_few.cu).
struct FusedPlan {
    bool few;
    bool boxes;                          // pairs: fused_boxes
    int height, tokens, chunks;          // few: columns and rows of C a tile, 64s of K a stage
    int split;                           // blocks (few) or pairs that share a tile's sum
    int slices;                          // few: C comes as so many FP32 matrices of M x N, to be added up (1: as it is)
    long sum_blocks;                     // rows of FusedEpilogue::sums
    long ce_blocks;                      // of FusedEpilogue::parts
};
// Only the sizes and storage of the operands are read, and of the epilogue what
// decides whether its matrices pass by TMA.
cudaError_t fused_plan(FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, int num_sms, FusedPlan* plan);

// The plan of a plain FUSED_ACT product whose sum may come in slices (a long one, of
// a C with few tiles).
cudaError_t fused_plan_slices(const FusedProduct& p, int num_sms, FusedPlan* plan);

// Whether C, R and Z pass by TMA on pairs, in boxes of 32 rows x 128 bytes: bases
// and rows on 16 bytes, whole 16-byte pieces long (a store clipped inside such a
// piece also writes the rest of it), and two boxes of shared memory for all of a
// turn's (an FP32 R takes both and leaves none for Z). The logits' gradient is scratch
// laid out for it.
bool fused_boxes(FusedKind kind, int N, const FusedEpilogue& e);

// Operands on 16-byte boundaries, with rows on them.
cudaError_t fused_gemm(FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, const FusedPlan& plan, int num_sms,
                       cudaStream_t s);
cudaError_t fused_few(FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, const FusedPlan& plan, int num_sms,
                      cudaStream_t s);
cudaError_t fused_few_clusters(unsigned long long* fits);

// ---- what joins the epilogues' shares (fused_join.cu)
// db[c] = the sum of `blocks` rows of sums, `cols` wide.
cudaError_t fused_join_sums(const float* sums, long blocks, long cols, float* db, cudaStream_t s);
// loss and lse of T rows from their `blocks` maxima and sums.
cudaError_t fused_join_ce(const float2* parts, const float* picked, const long long* target, int T, long V, long blocks,
                          float* loss, float* lse, cudaStream_t s);
// out (ld, FP32 or BF16) = the sum of `slices` matrices, rows x cols each, FP32.
cudaError_t fused_join_slices(const float* parts, int slices, int rows, int cols, void* out, long ld, bool f32, cudaStream_t s);
// Copies of up to three BF16 matrices in one launch, to rows of whole 64 columns;
// with `target`, rows whose target is not in 0 .. V - 1 as zeros.
struct CopyJob {
    const void* src;
    long ld_src;
    void* dst;
    long ld_dst;
    int rows, cols;
    const long long* target;
    long V;
    bool wide;                    // set by fused_copy_rows
};
cudaError_t fused_copy_rows(const CopyJob* jobs, int count, cudaStream_t s);

}  // namespace tgemm
