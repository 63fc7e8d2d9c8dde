// Which kernel a fused product runs in, and the tiles of few.
//
// By a model of both kernels' times in microseconds, fitted to 1800 measured runs of
// fused_few.cu's tiles (1 to 1024 tokens, 256 x 256 to 65536 x 4096 weights, plain,
// gated, gradients and cross entropy) and of fused_gemm.cu's: what it picks takes
// 1.7 % more than the best of them on average, 27 % at most. A few of them (us: tokens
// x columns x K, on pairs, and as few tiles: best measured):
//        1 x 14336 x 4096   42.9   21.4        256 x 1024 x 1024    12.6    5.7
//       16 x 4096 x 14336   72.2   23.0        256 x 14336 x 4096   32.5   39.6
//       64 x 4096 x 4096    26.5   11.2        512 x 4096 x 4096    27.7   22.0
//      128 x 14336 x 4096   31.9   28.2       1024 x 4096 x 4096    28.5   34.7

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

// Stages of as many chunks as leave room for three (a row's pieces next to each
// other in memory: 16 x 14336 x 4096 29.1, 23.0, 22.4 us with 1, 2, 4 chunks).
int chunks_for(long rows, int K) {
    int chunks = rows * 128 * 4 * 3 <= FUSED_FEW_RING ? 4 : rows * 128 * 2 * 3 <= FUSED_FEW_RING ? 2 : 1;
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

double pair_us(int M, long N, int K, int halves, int pairs) {
    const double rounds = (double)up(up(M, 256) * up(N * halves, 256), pairs);
    const double sm = rounds * (double)up(K, 64) * 0.388, hbm = 2.0 * K * ((double)N * halves + M) / HBM;
    return 5.4 + (sm > hbm ? sm : hbm);
}

}  // namespace

FusedParts fused_parts(FusedKind kind, bool few, int K, int chunk_k) {
    const int stages = (int)up(K, chunk_k), scale = chunk_k / 64 > 0 ? chunk_k / 64 : 1;
    auto even = [&](int most) {
        most = most / scale > 0 ? most / scale : 1;
        const int n = stages > 0 ? (int)up(stages, up(stages, most)) : 1;
        return FusedParts{n, n};
    };
    if (kind == FUSED_CE) return even(few ? 2 : 7);
    if (kind != FUSED_GRAD) return stages * scale <= 26 ? FusedParts{stages, stages} : even(21);
    if (few || stages <= 28) return even(14);
    for (int first = 18; first > 14; --first) {
        const int left = stages - 2 * first;
        if (left < 1) continue;
        for (int most = 14; most >= 8; --most) {
            const int parts = (int)up(left, most), rest = (int)up(left, parts);
            const double squares = 2.0 * first * first + (double)rest * rest * (parts - 1) +
                                   (double)(left - rest * (parts - 1)) * (left - rest * (parts - 1));
            if (squares <= 14.5 * stages) return {first, rest};
        }
    }
    return even(14);
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
    plan->height = plan->tokens = plan->split = plan->chunks = 0;
    plan->slices = 1;
    plan->boxes = fused_boxes(kind, p.N, e);
    plan->sum_blocks = up(p.M, FUSED_SUM_ROWS);
    plan->ce_blocks = up(p.N, FUSED_CE_COLS);
    // Many rows, and two rounds of pair tiles or more: always on pairs. (Few rows of many
    // columns are a stream of weights: 16 x 65536 x 4096 103 us on pairs, 85 as few.)
    const int forced = g_forced.load(std::memory_order_relaxed);
    if (p.M == 0 || p.N == 0 || p.K == 0 || forced == 0 ||
        (forced < 0 && p.M > 512 && up(p.M, 256) * up((long)p.N * halves, 256) >= num_sms))
        return cudaSuccess;
    unsigned long long fits = 0;
    const cudaError_t err = fused_few_clusters(&fits);
    if (err != cudaSuccess) return err;
    double best = forced == 1 ? 1e300 : pair_us(p.M, p.N, p.K, halves, num_sms / 2);
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
