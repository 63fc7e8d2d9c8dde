// C ABI of the products with what follows them in their epilogue: argument
// checks, operands off 16 bytes, pieces of the vocabulary. The contract of
// every entry point is in include/tgemm_fused.h.

#include "fused_internal.h"

#include <cmath>
#include <cstdint>

namespace {

using tgemm::FusedEpilogue;
using tgemm::FusedProduct;

bool off(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool valid_dim(int n) { return n >= 0 && n <= TGEMM_FUSED_MAX_DIM; }
bool valid_type(int t) { return t == TGEMM_TYPE_F32 || t == TGEMM_TYPE_BF16; }
size_t type_bytes(int t) { return t == TGEMM_TYPE_F32 ? 4 : 2; }
// A matrix of `type` elements that is not empty.
bool valid_matrix(const void* x, int type) { return x != nullptr && !off(x, type_bytes(type)); }
int done(cudaError_t e) { return e == cudaSuccess ? TGEMM_OK : TGEMM_ERR_CUDA; }
size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Scratch of one call: parts are asked for first, then taken together.
class Scratch {
public:
    explicit Scratch(cudaStream_t s) : stream_(s) {}
    size_t add(size_t bytes) {
        const size_t at = size_;
        size_ += whole(bytes);
        return at;
    }
    cudaError_t take() { return size_ == 0 ? cudaSuccess : tgemm::scratch_take(&base_, size_, stream_); }
    void* at(size_t offset) const { return static_cast<char*>(base_) + offset; }
    // Gives it back; e, or the first error.
    cudaError_t give(cudaError_t e) {
        if (base_ == nullptr) return e;
        const cudaError_t f = cudaFreeAsync(base_, stream_);
        base_ = nullptr;
        return e != cudaSuccess ? e : f;
    }

private:
    cudaStream_t stream_;
    void* base_ = nullptr;
    size_t size_ = 0;
};

// An operand as TMA reads it: its rows on 16-byte boundaries, else copied to
// scratch with rows on 128 bytes. (Of a single row the leading dimension says nothing.)
struct Operand {
    const void* x;
    long ld;
    int rows, cols;
    size_t at = 0;
    bool copied = false;
    Operand(const void* x_, long ld_, int rows_, int cols_, Scratch& scratch) : x(x_), ld(ld_), rows(rows_), cols(cols_) {
        if (rows == 0 || cols == 0) return;
        if (rows == 1) ld = ((long)cols + 7) / 8 * 8;
        copied = off(x, 16) || ld % 8 != 0;
        if (copied) at = scratch.add((size_t)rows * padded() * 2);
    }
    long padded() const { return ((long)cols + 63) / 64 * 64; }
    // The copy that lays it in its scratch (none: an empty one).
    tgemm::CopyJob lay(const Scratch& scratch) {
        if (!copied) return tgemm::CopyJob{};
        const tgemm::CopyJob job{x, ld, scratch.at(at), padded(), rows, cols, nullptr, 0, false};
        x = job.dst;
        ld = padded();
        return job;
    }
};

// A product's operands, checked; op(B) has `wide` columns, in `halves` halves.
struct Operands {
    int M, N, K, flags, halves;
    const void *A, *B;
    long lda, ldb;
    int status() const {
        const long wide = (long)halves * N;
        if (!valid_dim(M) || !valid_dim(N) || !valid_dim(K) || (flags & ~(TGEMM_TRANS_A | TGEMM_TRANS_B)) != 0)
            return TGEMM_ERR_INVALID_ARG;
        if (lda < ((flags & TGEMM_TRANS_A) ? M : K) || ldb < ((flags & TGEMM_TRANS_B) ? (long)K : wide)) return TGEMM_ERR_INVALID_ARG;
        if (M > 0 && N > 0 && K > 0 && (!valid_matrix(A, TGEMM_TYPE_BF16) || !valid_matrix(B, TGEMM_TYPE_BF16)))
            return TGEMM_ERR_INVALID_ARG;
        return TGEMM_OK;
    }
};

// The product of checked operands that is not empty. db: the column sums of a
// gradient's result, or NULL; e.sums is set here.
cudaError_t run(const Operands& o, tgemm::FusedKind kind, FusedEpilogue& e, float* db, int sms, cudaStream_t s) {
    Scratch scratch(s);
    const bool a_mn = (o.flags & TGEMM_TRANS_A) != 0, b_mn = (o.flags & TGEMM_TRANS_B) == 0;
    FusedProduct p{o.M, o.N, o.K, nullptr, 0, a_mn, nullptr, 0, b_mn, nullptr};
    tgemm::FusedPlan plan;
    cudaError_t err = tgemm::fused_plan(kind, p, e, sms, &plan);
    if (err != cudaSuccess) return err;
    Operand a(o.A, o.lda, o.K == 0 ? 0 : a_mn ? o.K : o.M, a_mn ? o.M : o.K, scratch);
    // Two halves side by side in a row (K x 2 N) start on 16 bytes only where N
    // is a multiple of 8 and are two matrices otherwise.
    const bool apart = o.halves == 2 && b_mn && o.N % 8 != 0;
    const int rows = o.K == 0 ? 0 : b_mn ? o.K : o.halves * o.N, cols = !b_mn ? o.K : apart ? o.N : o.halves * o.N;
    const __nv_bfloat16* second = static_cast<const __nv_bfloat16*>(o.B) + (b_mn ? (long)o.N : (long)o.N * o.ldb);
    Operand b(o.B, o.ldb, rows, cols, scratch), b2(second, o.ldb, apart ? rows : 0, cols, scratch);
    if (apart && b.copied != b2.copied) {
        // One leading dimension serves both.
        Operand& other = b.copied ? b2 : b;
        other.copied = true;
        other.at = scratch.add((size_t)other.rows * other.padded() * 2);
    }
    const long wide = (e.gated ? 2L : 1L) * o.N;
    const size_t sums = scratch.add(db != nullptr ? (size_t)plan.sum_blocks * wide * sizeof(float) : 0);
    err = scratch.take();
    if (err != cudaSuccess) return err;
    const tgemm::CopyJob jobs[3] = {a.lay(scratch), b.lay(scratch), b2.lay(scratch)};
    err = tgemm::fused_copy_rows(jobs, 3, s);
    if (o.halves == 2 && !apart)
        b2.x = static_cast<const __nv_bfloat16*>(b.x) + (b_mn ? (long)o.N : (long)o.N * b.ld);
    if (db != nullptr) e.sums = static_cast<float*>(scratch.at(sums));
    p.A = a.x;
    p.lda = a.ld;
    p.B = b.x;
    p.ldb = b.ld;
    p.B2 = b2.x;
    if (err == cudaSuccess) err = tgemm::fused_gemm(kind, p, e, plan, sms, s);
    if (err == cudaSuccess && db != nullptr) err = tgemm::fused_join_sums(e.sums, plan.sum_blocks, wide, db, s);
    return scratch.give(err);
}

// ------------------------------------------------------------ cross entropy
constexpr size_t PIECE_BYTES = 256u << 20;
constexpr int PIECE_COLS = 1024;             // at least

int check_ce(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha, const long long* target) {
    if (!valid_dim(T) || !valid_dim(V) || !valid_dim(D) || ldx < D || ldw < D || !std::isfinite(alpha) || off(target, 8))
        return TGEMM_ERR_INVALID_ARG;
    if (T > 0 && target == nullptr) return TGEMM_ERR_INVALID_ARG;
    if (T > 0 && V > 0 && D > 0 && (!valid_matrix(X, TGEMM_TYPE_BF16) || !valid_matrix(W, TGEMM_TYPE_BF16)))
        return TGEMM_ERR_INVALID_ARG;
    return TGEMM_OK;
}

cudaError_t ce(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha, const long long* target,
               float* loss, float* lse, int sms, cudaStream_t s) {
    tgemm::FusedPlan plan;
    cudaError_t e = tgemm::fused_plan(tgemm::FUSED_CE, FusedProduct{T, V, D, nullptr, 0, false, nullptr, 0, false, nullptr},
                                      FusedEpilogue(), sms, &plan);
    if (e != cudaSuccess) return e;
    const long blocks = plan.ce_blocks;
    // Tokens a turn: whole tiles, as many as the maxima and sums leave room for.
    long turn = T;
    if (blocks > 0 && (size_t)T * blocks * sizeof(float2) > PIECE_BYTES) {
        turn = (long)(PIECE_BYTES / sizeof(float2) / blocks) / 256 * 256;
        if (turn < 256) turn = 256;
    }
    Scratch scratch(s);
    Operand x(X, ldx, V == 0 || D == 0 ? 0 : T, D, scratch), w(W, ldw, D == 0 ? 0 : V, D, scratch);
    const size_t parts = scratch.add((size_t)turn * blocks * sizeof(float2)), picked = scratch.add((size_t)turn * sizeof(float));
    e = scratch.take();
    if (e != cudaSuccess) return e;
    const tgemm::CopyJob jobs[2] = {x.lay(scratch), w.lay(scratch)};
    e = tgemm::fused_copy_rows(jobs, 2, s);
    for (long t = 0; e == cudaSuccess && t < T; t += turn) {
        const int n = (int)(T - t < turn ? T - t : turn);
        FusedEpilogue ep;
        ep.alpha = alpha;
        ep.target = target + t;
        ep.vocabulary = V;
        ep.parts = static_cast<float2*>(scratch.at(parts));
        ep.picked = static_cast<float*>(scratch.at(picked));
        const FusedProduct p{n, V, D, static_cast<const __nv_bfloat16*>(x.x) + t * x.ld, x.ld, false, w.x, w.ld, false, nullptr};
        if (V > 0) e = tgemm::fused_gemm(tgemm::FUSED_CE, p, ep, plan, sms, s);
        if (e == cudaSuccess) e = tgemm::fused_join_ce(ep.parts, ep.picked, ep.target, n, V, blocks, loss + t, lse + t, s);
    }
    return scratch.give(e);
}

struct Gradient {
    void* x;
    long ld;
    int type;
};

// A product as its plan has it.
cudaError_t product(tgemm::FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, int sms, cudaStream_t s) {
    tgemm::FusedPlan plan;
    const cudaError_t err = tgemm::fused_plan(kind, p, e, sms, &plan);
    return err != cudaSuccess ? err : tgemm::fused_gemm(kind, p, e, plan, sms, s);
}

cudaError_t ce_grad(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha, const long long* target,
                    const float* lse, const float* dloss, const Gradient& dX, const Gradient& dW, float beta, int sms,
                    cudaStream_t s) {
    // Columns a piece: whole tiles.
    long piece = (long)(PIECE_BYTES / 2 / (T > 0 ? T : 1)) / 256 * 256;
    if (piece < PIECE_COLS) piece = PIECE_COLS;
    if (piece > V) piece = V;
    const bool sums = dX.x != nullptr && piece < V;          // dX over several pieces
    // An FP32 dX holds its own sum, where the products before the last can pass it by TMA
    // as they pass scratch (131072 x 2048: 1 GB less of that).
    const bool inside_x = sums && dX.type == TGEMM_TYPE_F32 && !off(dX.x, 16) && dX.ld % 4 == 0 && D % 4 == 0;
    const long ldz = (piece + 63) / 64 * 64, ldk = ((long)D + 63) / 64 * 64;
    Scratch scratch(s);
    // A dW takes X with the rows left out as zeros: copied by the logits' product where
    // that reads X as it is, else before it, and then the logits take it, too.
    const bool keep = dW.x != nullptr && T > 0 && V > 0;
    const bool inside = keep && !off(X, 16) && ldx % 8 == 0 && D % 8 == 0, before = keep && !inside;
    Operand x(X, ldx, V == 0 || before ? 0 : T, D, scratch), w(W, ldw, T == 0 ? 0 : V, D, scratch);
    const size_t z_at = scratch.add((size_t)T * ldz * 2);
    const size_t kept_at = scratch.add(keep ? (size_t)T * ldk * 2 : 0);
    // Few tokens: dX, a sum over all of the vocabulary, in slices.
    tgemm::FusedPlan slice{};
    slice.slices = 1;
    cudaError_t e = cudaSuccess;
    if (dX.x != nullptr && T > 0 && piece == V && V > 0)
        e = tgemm::fused_plan_slices(FusedProduct{T, D, V, nullptr, 0, false, nullptr, 0, true, nullptr}, sms, &slice);
    if (e != cudaSuccess) return e;
    const size_t sum_at = scratch.add(sums && !inside_x ? (size_t)T * ldk * 4 : slice.slices > 1 ? (size_t)slice.slices * T * D * 4 : 0);
    e = scratch.take();
    if (e != cudaSuccess) return e;
    void *const z = scratch.at(z_at), *const kept = scratch.at(kept_at);
    void *const sum = inside_x ? dX.x : scratch.at(sum_at);
    const long ld_sum = inside_x ? dX.ld : ldk;
    const tgemm::CopyJob jobs[3] = {x.lay(scratch), w.lay(scratch), {X, ldx, kept, ldk, before ? T : 0, D, target, V, false}};
    e = tgemm::fused_copy_rows(jobs, 3, s);
    if (before) {
        x.x = kept;
        x.ld = ldk;
    }
    for (long v = 0; e == cudaSuccess && (v < V || v == 0); v += piece > 0 ? piece : 1) {
        const int n = (int)(V - v < piece ? V - v : piece);
        const __nv_bfloat16* wv = static_cast<const __nv_bfloat16*>(w.x) + v * w.ld;
        if (T > 0 && n > 0) {
            FusedEpilogue ep;
            ep.C = z;
            ep.ldc = ldz;
            ep.alpha = alpha;
            ep.target = target;
            ep.first = v;
            ep.vocabulary = V;
            ep.lse = lse;
            ep.dloss = dloss;
            if (inside && v == 0) {
                ep.keep = X;
                ep.ld_keep = ldx;
                ep.kept = kept;
                ep.ld_kept = ldk;
                ep.keep_cols = D;
            }
            const FusedProduct p{T, n, D, x.x, x.ld, false, wv, w.ld, false, nullptr};
            e = product(tgemm::FUSED_CE_GRAD, p, ep, sms, s);
        }
        if (e == cudaSuccess && slice.slices > 1) {
            FusedEpilogue ep;
            ep.C = sum;
            ep.ldc = D;
            ep.c_f32 = true;
            const FusedProduct p{T, D, n, z, ldz, false, wv, w.ld, true, nullptr};
            e = tgemm::fused_gemm(tgemm::FUSED_ACT, p, ep, slice, sms, s);
            if (e == cudaSuccess)
                e = tgemm::fused_join_slices(static_cast<const float*>(sum), slice.slices, T, D, dX.x, dX.ld,
                                             dX.type == TGEMM_TYPE_F32, s);
        } else if (e == cudaSuccess && dX.x != nullptr && T > 0) {
            const bool last = v + piece >= V;
            FusedEpilogue ep;
            ep.C = last ? dX.x : sum;
            ep.ldc = last ? dX.ld : ld_sum;
            ep.c_f32 = !last || dX.type == TGEMM_TYPE_F32;
            if (v > 0) {
                ep.R = sum;
                ep.ldr = ld_sum;
                ep.r_f32 = true;
            }
            const FusedProduct p{T, D, n, z, ldz, false, wv, w.ld, true, nullptr};
            e = product(tgemm::FUSED_ACT, p, ep, sms, s);
        }
        if (e == cudaSuccess && dW.x != nullptr && n > 0) {
            FusedEpilogue ep;
            ep.C = static_cast<char*>(dW.x) + v * dW.ld * (long)type_bytes(dW.type);
            ep.ldc = dW.ld;
            ep.c_f32 = dW.type == TGEMM_TYPE_F32;
            if (beta != 0.0f) {
                ep.R = ep.C;
                ep.ldr = ep.ldc;
                ep.r_f32 = ep.c_f32;
                ep.r_scale = beta;
            }
            const FusedProduct p{n, D, T, z, ldz, true, kept, ldk, true, nullptr};
            e = product(tgemm::FUSED_ACT, p, ep, sms, s);
        }
    }
    return scratch.give(e);
}

}  // namespace

extern "C" {

int gemm_act(int M, int N, int K, const void* A, long lda, const void* B, long ldb, int flags, int act, const float* bias,
             const void* R, long ldr, int r_type, void* Z, long ldz, void* C, long ldc, int c_type, cudaStream_t stream) {
    const bool gated = (flags & TGEMM_GATED) != 0;
    const Operands o{M, N, K, flags & ~TGEMM_GATED, gated ? 2 : 1, A, B, lda, ldb};
    int st = o.status();
    if (st != TGEMM_OK) return st;
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_SILU || !valid_type(c_type) || (gated && c_type != TGEMM_TYPE_BF16) ||
        ldc < N || off(bias, 4))
        return TGEMM_ERR_INVALID_ARG;
    if (R != nullptr && (!valid_type(r_type) || ldr < N || !valid_matrix(R, r_type) || (R == C && (ldr != ldc || r_type != c_type))))
        return TGEMM_ERR_INVALID_ARG;
    if (Z != nullptr && (ldz < (long)o.halves * N || off(Z, 2))) return TGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TGEMM_OK;
    if (!valid_matrix(C, c_type)) return TGEMM_ERR_INVALID_ARG;
    int sms = 0;
    st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    FusedEpilogue e;
    e.act = act;
    e.gated = gated;
    e.C = C;
    e.ldc = ldc;
    e.c_f32 = c_type == TGEMM_TYPE_F32;
    e.bias = bias;
    e.R = R;
    e.ldr = ldr;
    e.r_f32 = r_type == TGEMM_TYPE_F32;
    e.Z = Z;
    e.ldz = ldz;
    return done(run(o, tgemm::FUSED_ACT, e, nullptr, sms, stream));
}

int gemm_act_grad(int M, int N, int K, const void* A, long lda, const void* B, long ldb, int flags, int act, const void* Z,
                  long ldz, void* dZ, long lddz, int dz_type, float* db, cudaStream_t stream) {
    const bool gated = (flags & TGEMM_GATED) != 0;
    const Operands o{M, N, K, flags & ~TGEMM_GATED, 1, A, B, lda, ldb};
    int st = o.status();
    if (st != TGEMM_OK) return st;
    const long wide = (gated ? 2L : 1L) * N;
    if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_SILU || !valid_type(dz_type) || (gated && dz_type != TGEMM_TYPE_BF16) ||
        ldz < wide || lddz < wide || off(db, 4))
        return TGEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!valid_matrix(Z, TGEMM_TYPE_BF16) || !valid_matrix(dZ, dz_type) ||
                           (Z == dZ && (ldz != lddz || dz_type != TGEMM_TYPE_BF16))))
        return TGEMM_ERR_INVALID_ARG;
    if (N == 0 || (M == 0 && db == nullptr)) return TGEMM_OK;
    int sms = 0;
    st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    if (M == 0) return done(tgemm::fused_join_sums(nullptr, 0, wide, db, stream));
    FusedEpilogue e;
    e.act = act;
    e.gated = gated;
    e.C = dZ;
    e.ldc = lddz;
    e.c_f32 = dz_type == TGEMM_TYPE_F32;
    e.Z = const_cast<void*>(Z);
    e.ldz = ldz;
    return done(run(o, tgemm::FUSED_GRAD, e, db, sms, stream));
}

int gemm_ce(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha, const long long* target,
            float* loss, float* lse, cudaStream_t stream) {
    int st = check_ce(T, V, D, X, ldx, W, ldw, alpha, target);
    if (st != TGEMM_OK) return st;
    if (T == 0) return off(loss, 4) || off(lse, 4) ? TGEMM_ERR_INVALID_ARG : TGEMM_OK;
    if (!valid_matrix(loss, TGEMM_TYPE_F32) || !valid_matrix(lse, TGEMM_TYPE_F32)) return TGEMM_ERR_INVALID_ARG;
    int sms = 0;
    st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(ce(T, V, D, X, ldx, W, ldw, alpha, target, loss, lse, sms, stream));
}

int gemm_ce_grad(int T, int V, int D, const void* X, long ldx, const void* W, long ldw, float alpha, const long long* target,
                 const float* lse, const float* dloss, void* dX, long lddx, int dx_type, void* dW, long lddw, int dw_type,
                 float beta, cudaStream_t stream) {
    int st = check_ce(T, V, D, X, ldx, W, ldw, alpha, target);
    if (st != TGEMM_OK) return st;
    if (!std::isfinite(beta) || off(lse, 4) || off(dloss, 4) || (T > 0 && (lse == nullptr || dloss == nullptr)))
        return TGEMM_ERR_INVALID_ARG;
    const Gradient gx{dX, lddx, dx_type}, gw{dW, lddw, dw_type};
    for (const Gradient* g : {&gx, &gw})
        if (g->x != nullptr && (!valid_type(g->type) || g->ld < D || off(g->x, type_bytes(g->type)))) return TGEMM_ERR_INVALID_ARG;
    const bool want_x = dX != nullptr && T > 0, want_w = dW != nullptr && V > 0;
    if (D == 0 || (!want_x && !want_w)) return TGEMM_OK;
    int sms = 0;
    st = tgemm::device_sms(&sms);
    if (st != TGEMM_OK) return st;
    return done(ce_grad(T, V, D, X, ldx, W, ldw, alpha, target, lse, dloss, want_x ? gx : Gradient{nullptr, 0, 0},
                        want_w ? gw : Gradient{nullptr, 0, 0}, beta, sms, stream));
}

}  // extern "C"
