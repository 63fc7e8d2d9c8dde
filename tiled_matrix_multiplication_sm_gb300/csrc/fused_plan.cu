// Which kernel a fused product runs in, how many pairs share a tile's sum, and the
// tiles of few.
//
// By a model of the kernels' times in microseconds, fitted to 1800 measured runs of
// fused_few.cu's tiles (1 to 1024 tokens, 256 x 256 to 65536 x 4096 weights, plain,
// gated, gradients and cross entropy) and 2600 of fused_gemm.cu's. Over 4600 others what
// it picks takes 0.2 % more than the better of both kernels on average, 36 % at most; over
// 2600 of 150 to 2048 tokens that could share sums 1 % more than the best sharing. A few
// of them (us: tokens x columns x K, on pairs, and as few tiles):
//        1 x 14336 x 4096   47.1   22.1        256 x 14336 x 4096   31.9   36.6
//       16 x 4096 x 14336   34.4   23.6        512 x 4096 x 4096    20.0   20.0
//       64 x 4096 x 4096    17.4   11.5        512 x 4096 x 14336   45.0   51.6
//      128 x 14336 x 4096   31.4   26.0       1024 x 4096 x 4096    27.6   31.1
//      256 x 1024 x 1024    10.8    5.8       1024 x 2048 x 8192    28.8   32.3

#include "fused_internal.h"

#include <atomic>
#include <cmath>

namespace tgemm {
namespace {

std::atomic<int> g_forced{-1};               // gemm_set_fused_kernel

long up(long a, long b) { return (a + b - 1) / b; }
double power4(double x) { return (x * x) * (x * x); }

constexpr double HBM = 6.17e6;               // bytes a microsecond, all SMs
constexpr double CHIP = 25.8e6;              // into all SMs, from L2 too
constexpr double SM = 119e3;                 // into one SM
constexpr double MMA_CYCLES = 61, CLOCK = 1950;      // the shortest MMA of 128 rows x 16, cycles a microsecond

struct Tiles {
    int height, tokens, split, chunks;
};

// Stages of as many chunks as leave room for four (a stage's waits and copies take the
// same time whatever it holds: 140 tiles of 32 columns x 16 tokens, K = 14336, 46.6, 29.7,
// 27.4 us with 1, 2, 4 chunks; of 96 x 128, K = 4096, in 7 stages of one 24.7, in 3 of two 26.4).
int chunks_for(long rows, int K) {
    int chunks = rows * 128 * 4 * 4 <= FUSED_FEW_RING ? 4 : rows * 128 * 2 * 4 <= FUSED_FEW_RING ? 2 : 1;
    while (chunks > 1 && K <= 64 * (chunks / 2)) chunks /= 2;
    return chunks;
}

double few_us(int M, long N, int K, int halves, const Tiles& t, int fits) {
    const long tiles = up(M, t.tokens) * up(N, t.height), rows = (long)t.height * halves + t.tokens;
    const double rounds = (double)up(tiles, fits), stages = (double)up(up(K, 64 * t.chunks), t.split), bytes = 2.0 * K * rows;
    const double half = t.tokens / 2.0, mma = 4.0 * t.chunks * halves * (half > MMA_CYCLES ? half : MMA_CYCLES) / CLOCK;
    const double load = (double)rows * 128 * t.chunks / SM;
    const double sm = rounds * stages * (mma > load ? mma : load) + (rounds - 1) * (0.59 + 0.146 / 16 * t.tokens);
    const double hbm = 2.0 * K * ((double)N * halves + M) / HBM, chip = (double)tiles * bytes / CHIP;
    return 2.7 + std::sqrt(std::sqrt(power4(sm) + power4(hbm) + power4(chip))) + 0.325 * (double)up(t.tokens, 16 * t.split) +
           (t.split > 1 ? 1.5 + 0.013 * t.tokens : 0.0);
}

// `split`: pairs that share a tile's sum (what they take longer: leaving and adding up
// the shares).
double pair_us(int M, long N, int K, int halves, int pairs, int split) {
    const double rounds = split > 1 ? 1.0 : (double)up(up(M, 256) * up(N * halves, 256), pairs);
    const double sm = rounds * (double)up(up(K, 64), split) * 0.285, hbm = 2.0 * K * ((double)N * halves + M) / HBM;
    return (split > 1 ? 8.0 + 0.55 * split : 7.5) + std::sqrt(std::sqrt(power4(sm) + power4(hbm)));
}

}  // namespace

FusedParts fused_parts(FusedKind kind, bool few, int K, int chunk_k) {
    const int stages = (int)up(K, chunk_k), scale = chunk_k / 64 > 0 ? chunk_k / 64 : 1;
    auto even = [&](int most) {
        most = most / scale > 0 ? most / scale : 1;
        const int n = stages > 0 ? (int)up(stages, up(stages, most)) : 1;
        return FusedParts{n, n};
    };
    if (kind == FUSED_CE || kind == FUSED_CE_GRAD) return even(few ? 2 : 4);
    // On pairs: the first two parts up to 18, as long as a mean of 13 allows it, the others even.
    constexpr int EVEN = 13;
    if (few || stages <= EVEN) return even(EVEN);
    for (int first = 18; first > EVEN; --first) {
        const int left = stages - 2 * first, second = stages - first;
        if (left < 1) {
            if (second > 0 && first * first + second * second <= EVEN * stages) return {first, second};
            continue;
        }
        for (int most = EVEN; most >= 8; --most) {
            const int parts = (int)up(left, most), rest = (int)up(left, parts);
            const double last = left - rest * (parts - 1), squares = 2.0 * first * first + (double)rest * rest * (parts - 1) + last * last;
            if (squares <= (double)EVEN * stages) return {first, rest};
        }
    }
    return even(EVEN);
}

bool fused_boxes(FusedKind kind, int N, const FusedEpilogue& e) {
    auto fits = [&](const void* x, long ld, bool f32) {
        const int size = f32 ? 4 : 2;
        return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld * size % 16 == 0 && (long)N * size % 16 == 0;
    };
    switch (kind) {
        case FUSED_ACT:
            return fits(e.C, e.ldc, e.c_f32) && (e.R == nullptr || fits(e.R, e.ldr, e.r_f32)) &&
                   (e.Z == nullptr || (fits(e.Z, e.ldz, false) && !(e.R != nullptr && (e.r_f32 || e.gated))));
        case FUSED_GRAD: return fits(e.C, e.ldc, e.c_f32) && fits(e.Z, e.ldz, false);
        case FUSED_CE_GRAD: return true;
        default: return false;
    }
}

namespace {

// fused_plan, with its estimate of the time (0: not made).
cudaError_t make_plan(FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, int num_sms, FusedPlan* plan, double* us) {
    *us = 0.0;
    const int halves = kind == FUSED_ACT && e.gated ? 2 : 1;
    plan->few = false;
    plan->height = plan->tokens = plan->chunks = 0;
    plan->split = plan->slices = 1;
    plan->boxes = fused_boxes(kind, p.N, e);
    plan->sum_blocks = up(p.M, FUSED_SUM_ROWS);
    plan->ce_blocks = up(p.N, FUSED_CE_COLS);
    // Many rows, and two rounds of pair tiles or more: always on pairs. (Few rows of many
    // columns are a stream of weights: 16 x 65536 x 4096 103 us on pairs, 85 as few.)
    const int forced = g_forced.load(std::memory_order_relaxed);
    if (p.M == 0 || p.N == 0 || p.K == 0 ||
        (forced < 0 && p.M > 512 && up(p.M, 256) * up((long)p.N * halves, 256) >= num_sms))
        return cudaSuccess;
    unsigned long long fits = 0;
    const cudaError_t err = fused_few_clusters(&fits);
    if (err != cudaSuccess) return err;
    double best = forced == 1 ? 1e300 : pair_us(p.M, p.N, p.K, halves, num_sms / 2, 1);
    // Pairs that share a tile's sum, in clusters that the GPU holds all at once, two stages
    // each at least (512 x 4096 x 14336 73 us alone, 45 with two pairs a tile).
    const long pair_tiles = up(p.M, 256) * up((long)p.N * halves, 256);
    for (int c = 2; forced != 1 && (kind == FUSED_ACT || (kind == FUSED_GRAD && !e.gated)) && c <= 4 / halves; ++c) {
        if (pair_tiles > (long)(fits >> 8 * (2 * c - 1) & 255) || up(p.K, 64) < 2 * c) continue;
        const double us_c = pair_us(p.M, p.N, p.K, halves, num_sms / 2, c);
        if (us_c < best) {
            best = us_c;
            plan->split = c;
        }
    }
    if (forced == 0) return cudaSuccess;
    const int most = halves == 2 ? 128 : 256, whole = (int)up(p.M, 16) * 16;
    const int tokens[5] = {whole, 32, 64, 128, 256};
    for (int i = 0; i < 5; ++i) {
        int t = tokens[i];
        if (p.a_mn) t = (int)up(t, 64) * 64;                     // MN-major boxes: 64 columns
        if (t > most || (i > 0 && t >= whole)) continue;
        const long tiles_m = up(p.M, t);
        for (int c = 1; c <= 8; ++c) {
            const long units = c == 1 ? num_sms : (long)(fits >> 8 * (c - 1) & 255);
            if (units < 1 || up(p.K, 64) < c) continue;
            // Heights: whole MMAs, and those that fill one or two rounds of units.
            for (int h = 0; h < 5; ++h) {
                long height = h == 0 ? 128 : h == 1 ? 64 : h == 2 ? 32 : 0;
                if (height == 0) {
                    const long across = units * (h - 2) / tiles_m;
                    if (across < 1) continue;
                    height = up(up(p.N, across), 8) * 8;
                    if (height < 16 || height > 128) continue;
                }
                if (p.b_mn) height = up(height, 64) * 64;
                if (c > 1 && tiles_m * up(p.N, height) > units) continue;
                const Tiles tiles{(int)height, t, c, chunks_for(height * halves + t, p.K)};
                const double t_us = few_us(p.M, p.N, p.K, halves, tiles, (int)units);
                if (t_us < best) {
                    best = t_us;
                    plan->few = true;
                    plan->height = tiles.height;
                    plan->tokens = tiles.tokens;
                    plan->split = tiles.split;
                    plan->chunks = tiles.chunks;
                }
            }
        }
    }
    *us = best;
    if (plan->few) {
        plan->sum_blocks = up(p.M, plan->tokens) * plan->split * FUSED_FEW_SETS;
        plan->ce_blocks = up(p.N, plan->height) * up(plan->height, 32);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t fused_plan(FusedKind kind, const FusedProduct& p, const FusedEpilogue& e, int num_sms, FusedPlan* plan) {
    double us;
    return make_plan(kind, p, e, num_sms, plan, &us);
}

cudaError_t fused_plan_slices(const FusedProduct& p, int num_sms, FusedPlan* plan) {
    double best;
    const cudaError_t err = make_plan(FUSED_ACT, p, FusedEpilogue(), num_sms, plan, &best);
    if (err != cudaSuccess || best == 0.0) return err;
    const int whole = (int)up(p.M, 16) * 16, tokens[3] = {64, 128, 256};
    for (int t : tokens) {
        if (!p.a_mn && t > whole) t = whole;
        const int height = p.b_mn && p.N <= 64 ? 64 : 128;
        const long tiles = up(p.M, t) * up(p.N, height);
        const long slices = num_sms / tiles < up(p.K, 1024) ? num_sms / tiles : up(p.K, 1024);
        if (slices < 2) continue;
        const Tiles shape{height, t, 1, chunks_for(height + t, p.K)};
        // A slice's time, and adding them up: a launch, and their bytes twice.
        const double us = few_us(p.M, p.N, (int)up(p.K, slices), 1, shape, (int)tiles) + 4.0 + 8.0 * slices * p.M * p.N / HBM;
        if (us > 0.95 * best) continue;
        best = us;
        plan->few = true;
        plan->height = height;
        plan->tokens = t;
        plan->split = 1;
        plan->slices = (int)slices;
        plan->chunks = shape.chunks;
    }
    return cudaSuccess;
}

}  // namespace tgemm

extern "C" int gemm_set_fused_kernel(int mode) {
    if (mode < -1 || mode > 1) return TGEMM_ERR_INVALID_ARG;
    tgemm::g_forced.store(mode, std::memory_order_relaxed);
    return TGEMM_OK;
}
