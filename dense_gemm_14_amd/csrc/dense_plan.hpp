// dense_plan.hpp -- host side of the dense layer's products: which kernel runs a
// product, its tiles and splits, and its launches. Shared by the calls that are
// made of such products (dense_ops.hip, loss_ops.hip).
#pragma once

#include <algorithm>
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "checks.hpp"
#include "dense_large.hpp"
#include "dense_small.hpp"
#include "dense_tile.hpp"

namespace gemm355 {
namespace host {

namespace d = gemm355::dense;
using d::DenseArgs;

// ---- products --------------------------------------------------------------

constexpr int kMaxSplits = 16;

// One product C = op(A) op(B)^T of a batch, as the plans see it.
struct Shape {
    int M, N, K;      // of one batch entry; N: columns of C
    int batch;
    bool symmetric;
    bool gated;
    bool row_k;       // both operands
    int max_splits = kMaxSplits;   // of 128 x 128 tiles; more than that only with eight steps each
};

// How a product runs on tiles of one size, in rounds of `grid` workgroups: the
// first `whole` tiles one workgroup each, the K steps of the rest (fewer than a
// round) split over as many workgroups as a round has.
struct TilePlan {
    int side, tiles_m, tiles_n, tiles, grid, whole, splits, steps_per_split;
    size_t workspace_bytes;
    double steps;     // of the busiest workgroup
};
inline TilePlan plan_tiles(const Shape &s, int side, int cus, int min_steps, bool split)
{
    TilePlan t = {};
    t.side = side;
    t.tiles_m = (int)ceil_div(s.M, side);
    t.tiles_n = (int)ceil_div(s.N, s.gated ? side / 2 : side);
    t.tiles = s.symmetric ? t.tiles_m * (t.tiles_m + 1) / 2 : t.tiles_m * t.tiles_n;
    t.grid = std::max(8, cus & ~7);
    const int nk = (int)ceil_div(s.K, d::TILE_BK);
    const int all = t.tiles * s.batch, tail = all % t.grid;
    t.whole = all;
    t.splits = 1;
    t.steps_per_split = nk;
    if (split && tail > 0) {
        const int most = side == d::TILE ? std::max(kMaxSplits, std::min(s.max_splits, nk / 8)) : kMaxSplits;
        int n = std::min({t.grid / tail, most, nk / min_steps});
        // no part shorter than min_steps, the last one included
        while (n > 1 && nk - ceil_div(nk, n) * (n - 1) < min_steps)
            --n;
        if (n > 1) {
            t.splits = n;
            t.steps_per_split = (int)ceil_div(nk, n);
            t.whole = all - tail;
            t.workspace_bytes = size_t(tail) * n * side * side * sizeof(float);
        }
    }
    t.steps = double(t.whole / t.grid) * nk + (all % t.grid != 0 ? t.steps_per_split : 0);
    return t;
}

inline TilePlan plan_tile(const Shape &s, int cus) { return plan_tiles(s, d::TILE, cus, 4, true); }

// The small-tile kernel's tile, in blocks of 16 rows of A and of B, and its
// waves (8, or fewer with more workgroups per compute unit).
struct SmallPlan {
    int mb, nb, waves, tiles_m, tiles_n, tiles;
};

// 64 x 64 tiles, or narrow ones: 32 x 32, and for the few tokens of a forward
// layer 16 or 32 rows against 16 columns (16 gate and 16 up rows of a gated
// layer), so that every compute unit streams weights; with 16 rows, as many
// columns up to 64 as still leave a tile for every unit.
inline SmallPlan plan_small(const Shape &s, bool layer, bool narrow, int cus)
{
    SmallPlan t = {4, 4, 8, 0, 0, 0};
    if (narrow) {
        t.mb = layer && s.M <= 16 ? 1 : 2;
        t.nb = layer && s.M <= 32 && !s.gated ? 1 : 2;
        while (t.mb == 1 && t.nb < 4 && ceil_div(s.N, s.gated ? 16 * t.nb : 32 * t.nb) * s.batch >= cus)
            t.nb *= 2;
    }
    t.tiles_m = (int)ceil_div(s.M, 16 * t.mb);
    t.tiles_n = (int)ceil_div(s.N, s.gated ? 8 * t.nb : 16 * t.nb);
    t.tiles = s.symmetric ? t.tiles_m * (t.tiles_m + 1) / 2 : t.tiles_m * t.tiles_n;
    return t;
}

// Which kernel runs a product: 1 = 256 x 256 tiles, 2 = the same with the last
// round's tiles split, 3 = 128 x 128 tiles, 4 = 64 x 64 tiles, 5 = narrow
// tiles. Set through gemm355_force_layer_kernel (0 = by size).
inline std::atomic<int> g_layer_kernel{0};
enum { KERNEL_WHOLE = 1, KERNEL_SPLIT = 2, KERNEL_TILE = 3, KERNEL_SMALL = 4, KERNEL_NARROW = 5 };

// Estimated microseconds of each kernel, fitted to 1200 products measured on
// MI355X (M from 1, N and K from 64 to 8192, forward layers and both gradient
// products; a typical estimate is 10 % off, and the choice by them costs 2 %
// over the best kernel of every product).
//   small tiles: per K slice of a wave, a wait that the ring's stages share and
//     the traffic, by the tile's width and how many units are busy;
//   128 and 256: per K step, part of it only when every unit is busy; per round
//     the tiles' beginning and end; for a split the second launch and its
//     partials (MB).
constexpr double kStart = 3.4;
inline int small_slots(const SmallPlan &t, int cus) { return cus * (8 / t.waves); }
inline double time_small_tile(const SmallPlan &t, int nk, double fill)
{
    const double width = (t.mb + t.nb) / 8.0, stages = d::small_stages(t.mb, t.nb);
    return 0.8 + double(ceil_div(nk, t.waves)) * (1.08 / stages + 1.27 * width * fill);
}
inline double time_small(const SmallPlan &t, int nk, int batch, int cus)
{
    const double tiles = double(t.tiles) * batch, slots = small_slots(t, cus);
    return kStart + ceil(tiles / slots) * time_small_tile(t, nk, std::min(1.0, tiles / slots));
}
// 64 x 64 tiles with fewer waves, and so more workgroups to a unit, where that is
// estimated faster; two waves or one only for what is more than a round of the
// next larger. Measured, before and after (us): eight waves and four, 1024 x 1152
// x 1024, 288 tiles, 11.8 and 8.7; 64 x 18000 x 512 9.7 and 6.6; a backward pass
// of 170 x 1528 x 1608 15.1 and 9.8. Four waves and fewer: 1310 x 6288 x 168, 2079
// tiles of three slices, 18.6 and 12.6; a gated layer of 877 x 2344 x 72 10.0 and
// 6.8. Eight waves keep long contractions of few tiles, where a wave's share of K
// is what takes the time (1024 x 1024 x 1024: 6.9), and four the short ones: eight
// matrices of 64 x 512 orthogonalised in 53.6, with one wave 57.4.
inline SmallPlan plan_small_waves(const Shape &s, bool layer, bool narrow, int cus)
{
    SmallPlan best = plan_small(s, layer, narrow, cus);
    const int nk = (int)ceil_div(s.K, d::SMALL_BK);
    if (!narrow)
        for (int waves = 4; waves >= 1; waves /= 2) {
            SmallPlan t = best;
            t.waves = 2 * waves;
            if (waves < 4 && int64_t(t.tiles) * s.batch <= small_slots(t, cus))
                break;
            t.waves = waves;
            if (time_small(t, nk, s.batch, cus) < time_small(best, nk, s.batch, cus))
                best = t;
        }
    return best;
}
struct TileTimes {
    double fixed, step, step_full, round, split, split_mb;
};
constexpr TileTimes kTile = {2.2, 0.31, 0.22, 4.3, 5.1, 0.46}, kBig = {4.0, 1.19, 0.42, 6.0, 0.0, 0.0},
                    kBigSplit = {1.6, 1.25, 0.0, 13.4, 1.6, 0.30}, kMid = {4.0, 0.70, 0.25, 5.0, 0.0, 0.0};
inline double time_tiles(const TilePlan &t, int batch, const TileTimes &c)
{
    const int64_t items = t.whole + (int64_t(t.tiles) * batch - t.whole) * t.splits;
    const double fill = std::min(1.0, double(items) / t.grid);
    return c.fixed + t.steps * (c.step + c.step_full * fill) + double(ceil_div(items, t.grid)) * c.round +
           (t.splits > 1 ? c.split + c.split_mb * 1e-6 * double(t.workspace_bytes) : 0.0);
}

// 256 x 256 tiles; for a symmetric product that is not split 192 x 192 ones
// where they are estimated faster. A K step of theirs takes two thirds of the
// larger ones' time for 9/16 of the work, so they serve where the larger leave
// units idle: 4096 x 4096 has 136 of those for 256 units and 253 of these (its
// square 94 -> 66 us, X X^T of 4096 x 8192 169 -> 122). Other products fill a
// round or have their last one split, without the factor of a triangle.
inline TilePlan plan_large(const Shape &s, int cus, bool split)
{
    const TilePlan t = plan_tiles(s, d::BIG, cus, d::BIG_MIN_STEPS, split);
    if (split || !s.symmetric || !s.row_k)
        return t;
    const TilePlan u = plan_tiles(s, d::MID, cus, d::BIG_MIN_STEPS, false);
    return time_tiles(u, s.batch, kMid) < time_tiles(t, s.batch, kBig) ? u : t;
}

struct Choice {
    int kernel;
    double us;
};
inline Choice choose_kernel(const Shape &s, bool layer, int cus)
{
    const int nk = (int)ceil_div(s.K, d::BIG_BK);
    const bool big_ok = nk >= d::BIG_MIN_STEPS;
    const int forced = g_layer_kernel.load(std::memory_order_relaxed);
    if (forced != 0)
        return {forced <= KERNEL_SPLIT && !big_ok ? KERNEL_TILE : forced, 0.0};
    // The symmetric products are FP16, whose 128 x 128 steps take 15 % longer
    // than the BF16 ones of the fit (the 256 x 256 ones do not): 4096 x 4096
    // orthogonalised in 1410 us on 256 x 256 tiles, in 1620 with 128 x 128 ones
    // for the symmetric products.
    Choice best = {KERNEL_TILE, time_tiles(plan_tile(s, cus), s.batch, kTile) * (s.symmetric ? 1.15 : 1.0)};
    auto offer = [&](int kernel, double us) {
        if (us < best.us)
            best = {kernel, us};
    };
    offer(KERNEL_SMALL, time_small(plan_small_waves(s, layer, false, cus), nk, s.batch, cus));
    offer(KERNEL_NARROW, time_small(plan_small(s, layer, true, cus), nk, s.batch, cus));
    if (big_ok) {
        const TilePlan w = plan_large(s, cus, false);
        offer(KERNEL_WHOLE, time_tiles(w, s.batch, w.side == d::MID ? kMid : kBig));
        const TilePlan b = plan_large(s, cus, true);
        if (b.splits > 1)
            offer(KERNEL_SPLIT, time_tiles(b, s.batch, kBigSplit));
    }
    return best;
}

// What a product runs, decided once per call (the kernel's override may change
// at any time): the workspace it was given and what it launches agree.
struct ProductPlan {
    int kernel;
    double us;                // estimated
    TilePlan tiles;           // KERNEL_WHOLE, _SPLIT, _TILE
    SmallPlan small;          // KERNEL_SMALL, _NARROW
    size_t workspace_bytes;
};
inline ProductPlan plan_product(const Shape &s, bool layer, int cus)
{
    const Choice c = choose_kernel(s, layer, cus);
    ProductPlan p = {c.kernel, c.us, {}, {}, 0};
    if (c.kernel >= KERNEL_SMALL)
        p.small = plan_small_waves(s, layer, c.kernel == KERNEL_NARROW, cus);
    else
        p.tiles = c.kernel == KERNEL_TILE ? plan_tile(s, cus) : plan_large(s, cus, c.kernel == KERNEL_SPLIT);
    p.workspace_bytes = p.tiles.workspace_bytes;
    return p;
}

// One instance of the small-tile kernel; its threads are the instance's own.
template <class T, int LA, int LB, int EPI, class TO, int MB, int NB, int WAVES>
int launch_small(unsigned blocks, DenseArgs &p, hipStream_t stream)
{
    return launch_kernel(d::dense_small_kernel<T, LA, LB, EPI, TO, MB, NB, WAVES>, blocks, 64u * WAVES, p, stream);
}

template <class T, int LA, int LB, int EPI, class TO>
int product_small(DenseArgs p, const SmallPlan &t, hipStream_t stream)
{
    p.tiles_m = t.tiles_m;
    p.tiles_n = t.tiles_n;
    p.tiles = p.whole = t.tiles;
    p.splits = 1;
    const unsigned blocks = (unsigned)(ceil_div(int64_t(t.tiles) * p.batch, 8) * 8);
    if constexpr (EPI == d::EPI_LINEAR || EPI == d::EPI_CE || EPI == d::EPI_CE_GRAD) {
        if (t.nb == 1)
            return t.mb == 1 ? launch_small<T, LA, LB, EPI, TO, 1, 1, 8>(blocks, p, stream)
                             : launch_small<T, LA, LB, EPI, TO, 2, 1, 8>(blocks, p, stream);
    }
    if constexpr (EPI == d::EPI_LINEAR || EPI == d::EPI_GATED || EPI == d::EPI_CE || EPI == d::EPI_CE_GRAD) {
        if (t.mb == 1)
            return t.nb == 2 ? launch_small<T, LA, LB, EPI, TO, 1, 2, 8>(blocks, p, stream)
                             : launch_small<T, LA, LB, EPI, TO, 1, 4, 8>(blocks, p, stream);
    }
    if (t.mb == 2)
        return launch_small<T, LA, LB, EPI, TO, 2, 2, 8>(blocks, p, stream);
    switch (t.waves) {
    case 1: return launch_small<T, LA, LB, EPI, TO, 4, 4, 1>(blocks, p, stream);
    case 2: return launch_small<T, LA, LB, EPI, TO, 4, 4, 2>(blocks, p, stream);
    case 4: return launch_small<T, LA, LB, EPI, TO, 4, 4, 4>(blocks, p, stream);
    default: return launch_small<T, LA, LB, EPI, TO, 4, 4, 8>(blocks, p, stream);
    }
}

inline void set_plan(DenseArgs &p, const TilePlan &t)
{
    p.tiles_m = t.tiles_m;
    p.tiles_n = t.tiles_n;
    p.tiles = t.tiles;
    p.grid = t.grid;
    p.whole = t.whole;
    p.splits = t.splits;
    p.steps_per_split = t.steps_per_split;
}

template <class T, int LA, int LB, int EPI, class TO>
int product_tile(DenseArgs p, const TilePlan &t, hipStream_t stream)
{
    set_plan(p, t);
    const int64_t tail = int64_t(t.tiles) * p.batch - t.whole, items = t.whole + tail * t.splits;
    // whole rounds, then the last one's runs for each of the eight XCDs
    const int64_t blocks = items / t.grid * t.grid + ceil_div(items % t.grid, 8) * 8;
    int st = launch_kernel(d::dense_tile_kernel<T, LA, LB, EPI, TO>, (unsigned)blocks, (unsigned)d::TILE_THREADS, p, stream);
    if (st != GEMM355_OK || tail == 0)
        return st;
    if constexpr (EPI == d::EPI_ACC) {
        if (t.splits > kMaxSplits)
            return launch_kernel(d::dense_reduce_many_kernel<EPI, TO>, (unsigned)(tail * 8), 64u * d::REDUCE_MANY_WAVES, p, stream);
    }
    return launch_kernel(d::dense_reduce_kernel<EPI, TO>, (unsigned)ceil_div(tail * 8, d::REDUCE_WAVES),
                         64u * d::REDUCE_WAVES, p, stream);
}

template <class T, int LA, int LB, int EPI, class TO>
int product_large(DenseArgs p, const TilePlan &t, hipStream_t stream)
{
    set_plan(p, t);
    const int64_t tail = int64_t(t.tiles) * p.batch - t.whole;
    // persistent: a workgroup per compute unit at most, each an item per round
    p.grid = (int)std::min<int64_t>(t.grid, ceil_div(t.whole + tail * t.splits, 8) * 8);
    const bool ragged = p.K % d::BIG_BK != 0;
    auto kernel = ragged ? d::dense_large_kernel<T, LA, LB, EPI, TO, true> : d::dense_large_kernel<T, LA, LB, EPI, TO, false>;
    if constexpr (d::epi_symmetric(EPI) && LA == d::ROW_K && LB == d::ROW_K)
        if (t.side == d::MID)
            kernel = ragged ? d::dense_large_kernel<T, LA, LB, EPI, TO, true, 6>
                            : d::dense_large_kernel<T, LA, LB, EPI, TO, false, 6>;
    int st = launch_kernel(kernel, (unsigned)p.grid, (unsigned)d::BIG_THREADS, p, stream);
    if (st == GEMM355_OK && tail > 0)
        st = launch_kernel(d::dense_large_reduce_kernel<EPI, TO>, (unsigned)ceil_div(tail * 16, d::BIG_REDUCE_WAVES),
                           64u * d::BIG_REDUCE_WAVES, p, stream);
    return st;
}

// Launches a product as planned; `ws` has the plan's workspace_bytes.
template <class T, int LA, int LB, int EPI, class TO = T>
int product(DenseArgs p, const ProductPlan &plan, void *ws, hipStream_t stream)
{
    p.supergroup = 8;
    p.ws = static_cast<float *>(ws);
    if (p.lda == 0)      // (the rows side by side)
        p.lda = LA == d::ROW_K ? p.K : p.M;
    if (plan.kernel >= KERNEL_SMALL)
        return product_small<T, LA, LB, EPI, TO>(p, plan.small, stream);
    return plan.kernel == KERNEL_TILE ? product_tile<T, LA, LB, EPI, TO>(p, plan.tiles, stream)
                                      : product_large<T, LA, LB, EPI, TO>(p, plan.tiles, stream);
}

inline DenseArgs args_of(int M, int N, int K, const void *a, const void *b, void *c)
{
    DenseArgs p = {};
    p.M = M;
    p.N = N;
    p.K = K;
    p.a = K > 0 ? a : nullptr;
    p.b = K > 0 ? b : nullptr;
    p.c = c;
    p.batch = 1;
    p.alpha = 1.0f;
    return p;
}

// ---- backward passes in one launch ------------------------------------------

// How a backward pass runs as one launch (kernel 0: not).
struct Together {
    int kernel, waves;
};

// Whether a backward pass runs as one launch of small tiles (KERNEL_SMALL or
// KERNEL_NARROW; 0: its products one by one); pa, pb: the plans of the products
// that are wanted. Together the tiles fill the compute units better and launches
// fall away, the bias gradient's too. Estimate: the tiles' time shared out over
// the units, and no less than the longest tile; it comes out a tenth too short,
// and what separate launches cost is in each one's own estimate already. (Over
// 140 backward passes of up to 4096 tokens: ten vectors of 7336 x 328 weights,
// 115 slices of which one tile of dA takes every eighth, 22 us together, 14 apart;
// 170 x 1528 x 1608 10.5 together, 28 as two products of 128 x 128 tiles.)
constexpr double kTogether = 1.1, kBiasLaunch = 1.0;
inline Together backward_together(const Shape &a, const ProductPlan *pa, const Shape &b, const ProductPlan *pb, int cus)
{
    if (!pa && !pb)   // the bias gradient alone
        return {KERNEL_SMALL, 8};
    if (!pa || !pb) {
        // alone, a product runs as it would anywhere: beside the bias gradient in
        // one launch where that has the planned tiles and waves, else by itself
        const ProductPlan &one = pa ? *pa : *pb;
        const bool has = one.kernel == KERNEL_NARROW || (one.kernel == KERNEL_SMALL && one.small.waves >= 4);
        return has ? Together{one.kernel, one.small.waves} : Together{0, 0};
    }
    const bool small = pa->kernel >= KERNEL_SMALL && pb->kernel >= KERNEL_SMALL, forced = pa->us == 0.0;
    if (forced && !small)
        return {0, 0};
    double best_us = forced ? 1e30 : (pa->us + pb->us) / kTogether + kBiasLaunch;
    Together best = {0, 0};
    for (const Together &how : {Together{KERNEL_SMALL, 8}, Together{KERNEL_SMALL, 4}, Together{KERNEL_NARROW, 8}}) {
        if (forced && how.kernel != pa->kernel)
            continue;
        SmallPlan ta = plan_small(a, false, how.kernel == KERNEL_NARROW, cus), tb = plan_small(b, false, how.kernel == KERNEL_NARROW, cus);
        ta.waves = tb.waves = how.waves;
        const double na = ta.tiles, nb = tb.tiles, slots = small_slots(ta, cus), fill = std::min(1.0, (na + nb) / slots);
        const int ka = (int)ceil_div(a.K, d::SMALL_BK), kb = (int)ceil_div(b.K, d::SMALL_BK);
        const double one_a = time_small_tile(ta, ka, fill), one_b = time_small_tile(tb, kb, fill);
        // a long tile goes on when the others are done
        const double longest = std::max(time_small_tile(ta, ka, std::min(1.0, na / slots)),
                                        time_small_tile(tb, kb, std::min(1.0, nb / slots)));
        // (the last tiles end up to one short tile apart)
        const double us = kStart + std::max(longest, (na * one_a + nb * one_b) / slots + 0.5 * std::min(one_a, one_b));
        if (us < best_us) {
            best_us = us;
            best = how;
        }
    }
    return best;
}

} // namespace host
} // namespace gemm355
