// dense_ops.hip -- host side of the dense layer's fused operators: argument
// checks, plans, workspace layout and launches of the kernels in
// dense_large.hpp, dense_tile.hpp, dense_small.hpp, dense_grad.hpp and
// newton_schulz.hpp. The C ABI is declared in include/gemm355.h. Nothing here
// allocates memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "gemm355.h"
#include "host.hpp"
#include "dense_large.hpp"
#include "dense_small.hpp"
#include "dense_tile.hpp"
#include "dense_grad.hpp"
#include "newton_schulz.hpp"

namespace {

using namespace gemm355::host;
namespace d = gemm355::dense;
using d::DenseArgs;

constexpr size_t kAlign = 256;
size_t align_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// ---- products --------------------------------------------------------------

// One product C = op(A) op(B)^T of a batch, as the plans see it.
struct Shape {
    int M, N, K;      // of one batch entry; N: columns of C
    int batch;
    bool symmetric;
    bool gated;
    bool row_k;       // both operands
};

// How a product runs on tiles of one size, in rounds of `grid` workgroups: the
// first `whole` tiles one workgroup each, the K steps of the rest (fewer than a
// round) split over as many workgroups as a round has.
struct TilePlan {
    int side, tiles_m, tiles_n, tiles, grid, whole, splits, steps_per_split;
    size_t workspace_bytes;
    double steps;     // of the busiest workgroup
};
constexpr int kMaxSplits = 16;

TilePlan plan_tiles(const Shape &s, int side, int cus, int min_steps, bool split)
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
        int n = std::min({t.grid / tail, kMaxSplits, nk / min_steps});
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

TilePlan plan_tile(const Shape &s, int cus) { return plan_tiles(s, d::TILE, cus, 4, true); }

// The small-tile kernel's tile, in blocks of 16 rows of A and of B, and its
// waves (8, or fewer with more workgroups per compute unit).
struct SmallPlan {
    int mb, nb, waves, tiles_m, tiles_n, tiles;
};

// 64 x 64 tiles, or narrow ones: 32 x 32, and for the few tokens of a forward
// layer 16 or 32 rows against 16 columns (16 gate and 16 up rows of a gated
// layer), so that every compute unit streams weights; with 16 rows, as many
// columns up to 64 as still leave a tile for every unit.
SmallPlan plan_small(const Shape &s, bool layer, bool narrow, int cus)
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
std::atomic<int> g_layer_kernel{0};
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
int small_slots(const SmallPlan &t, int cus) { return cus * (8 / t.waves); }
double time_small_tile(const SmallPlan &t, int nk, double fill)
{
    const double width = (t.mb + t.nb) / 8.0, stages = d::small_stages(t.mb, t.nb);
    return 0.8 + double(ceil_div(nk, t.waves)) * (1.08 / stages + 1.27 * width * fill);
}
double time_small(const SmallPlan &t, int nk, int batch, int cus)
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
SmallPlan plan_small_waves(const Shape &s, bool layer, bool narrow, int cus)
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
double time_tiles(const TilePlan &t, int batch, const TileTimes &c)
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
TilePlan plan_large(const Shape &s, int cus, bool split)
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
Choice choose_kernel(const Shape &s, bool layer, int cus)
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
ProductPlan plan_product(const Shape &s, bool layer, int cus)
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
    p.tiles = t.tiles;
    const unsigned blocks = (unsigned)(ceil_div(int64_t(t.tiles) * p.batch, 8) * 8);
    if constexpr (EPI == d::EPI_LINEAR) {
        if (t.nb == 1)
            return t.mb == 1 ? launch_small<T, LA, LB, EPI, TO, 1, 1, 8>(blocks, p, stream)
                             : launch_small<T, LA, LB, EPI, TO, 2, 1, 8>(blocks, p, stream);
    }
    if constexpr (EPI == d::EPI_LINEAR || EPI == d::EPI_GATED) {
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

void set_plan(DenseArgs &p, const TilePlan &t)
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
    if (st == GEMM355_OK && tail > 0)
        st = launch_kernel(d::dense_reduce_kernel<EPI, TO>, (unsigned)ceil_div(tail * 8, d::REDUCE_WAVES),
                           64u * d::REDUCE_WAVES, p, stream);
    return st;
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
    if constexpr (EPI >= d::EPI_STORE_SYM && LA == d::ROW_K && LB == d::ROW_K)
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
    if (plan.kernel >= KERNEL_SMALL)
        return product_small<T, LA, LB, EPI, TO>(p, plan.small, stream);
    return plan.kernel == KERNEL_TILE ? product_tile<T, LA, LB, EPI, TO>(p, plan.tiles, stream)
                                      : product_large<T, LA, LB, EPI, TO>(p, plan.tiles, stream);
}

DenseArgs args_of(int M, int N, int K, const void *a, const void *b, void *c)
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

// ---- argument checks -------------------------------------------------------

// An array of a call: its address, size and required alignment.
struct Array {
    const void *p;
    size_t bytes;
};

// Whether any output overlaps an input, the workspace or another output.
bool any_overlap(const Array *out, int outs, const Array *in, int ins)
{
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return true;
        for (int j = i + 1; j < outs; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return true;
    }
    return false;
}

bool all_aligned(const Array *a, int n)
{
    for (int i = 0; i < n; ++i)
        if (!aligned(a[i].p, 16))
            return false;
    return true;
}

bool act_ok(int act) { return act >= GEMM355_ACT_NONE && act <= GEMM355_ACT_SILU; }

// Extents of a layer with `rows` weight rows and N outputs: every array,
// padded to whole tiles (at least one), below 2^31 bytes.
bool layer_extents_ok(int64_t M, int64_t N, int64_t rows, int64_t K)
{
    M = std::max<int64_t>(M, 1);
    return extent_ok(M, K * 2) && extent_ok(rows, K * 2) && extent_ok(M, rows * 2) && extent_ok(M, N * 2);
}

// ---- forward layers --------------------------------------------------------

template <bool GATED>
int layer_forward(int M, int N, int K, const void *A, const void *B, const void *bias, int act, const void *R, void *Z,
                  void *C, void *workspace, size_t workspace_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0 || !act_ok(act))
        return GEMM355_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return GEMM355_OK;
    if (!C || (K > 0 && (!A || !B)) || (workspace_bytes > 0 && !workspace))
        return GEMM355_ERR_INVALID_ARG;
    const size_t rows = (GATED ? 2 : 1) * size_t(N);
    const size_t c_bytes = size_t(M) * size_t(N) * 2;
    const Array out[] = {{C, c_bytes}, {Z, size_t(M) * rows * 2}, {workspace, workspace_bytes}};
    // C may be R itself: every element is read before it is written, by the same lane
    const Array in[] = {{A, size_t(M) * K * 2}, {B, rows * K * 2}, {bias, rows * 2}, {R == C ? nullptr : R, c_bytes}};
    if (any_overlap(out, 3, in, 4) || overlaps(Z, out[1].bytes, R, c_bytes) ||
        overlaps(workspace, workspace_bytes, R, c_bytes))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 3) || !all_aligned(in, 4) || K % 8 != 0 || N % 8 != 0 ||
        !layer_extents_ok(M, N, GATED ? 2 * int64_t(N) : N, K))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const ProductPlan plan = plan_product({M, N, K, 1, false, GATED}, true, cus);
    if (workspace_bytes < plan.workspace_bytes)
        return GEMM355_ERR_UNSUPPORTED;
    DenseArgs p = args_of(M, N, K, A, B, C);
    p.bias = bias;
    p.act = act;
    p.r = R;
    p.z = Z;
    return product<__bf16, d::ROW_K, d::ROW_K, GATED ? d::EPI_GATED : d::EPI_LINEAR>(
        p, plan, workspace, static_cast<hipStream_t>(stream));
}

template <bool GATED>
int layer_forward_workspace(int M, int N, int K, size_t *bytes)
{
    if (M < 0 || N < 0 || K < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!layer_extents_ok(M, N, GATED ? 2 * int64_t(N) : N, K))
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (M == 0 || N == 0)
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)
        *bytes = plan_product({M, N, K, 1, false, GATED}, true, cus).workspace_bytes;
    return rc;
}

// ---- backward layers -------------------------------------------------------

// Rows of a workgroup of the elementwise pass: enough workgroups for eight per
// compute unit (256 units) where the array has the rows, at most 64 rows.
int grad_rows(int M, int N)
{
    const int64_t col_blocks = ceil_div(N, d::GRAD_COLS);
    const int64_t rows = ceil_div(int64_t(M) * col_blocks, 2048);
    return (int)std::min<int64_t>(64, std::max<int64_t>(d::GRAD_LANES, ceil_div(rows, d::GRAD_LANES) * d::GRAD_LANES));
}

// How a backward pass runs as one launch (kernel 0: not).
struct Together {
    int kernel, waves;
};

template <int BLOCKS, int WAVES>
int launch_small_bwd(unsigned blocks, d::SmallBwdArgs &g, hipStream_t s)
{
    return launch_kernel(d::dense_small_bwd_kernel<BLOCKS, WAVES>, blocks, 64u * WAVES, g, s);
}

// A backward pass whose products are small, in one launch: 32 x 32 tiles, or
// 64 x 64 with eight or four waves (there are no other instances; what plans
// fewer waves runs product by product).
int backward_small(DenseArgs pa, bool wants_a, DenseArgs pb, bool wants_b, const d::BiasArgs &bias, int bias_blocks,
                   const Together &how, int cus, hipStream_t s)
{
    d::SmallBwdArgs g = {};
    auto place = [&](DenseArgs &p, bool wanted) {
        const SmallPlan t = plan_small({p.M, p.N, p.K, 1, false, false}, false, how.kernel == KERNEL_NARROW, cus);
        p.tiles_m = t.tiles_m;
        p.tiles_n = t.tiles_n;
        p.tiles = wanted ? t.tiles : 0;
        p.supergroup = 8;
    };
    place(pa, wants_a);
    place(pb, wants_b);
    g.a = pa;
    g.b = pb;
    g.bias = bias;
    g.bias_blocks = bias_blocks;
    g.first_b = pb.K > pa.K;
    const unsigned blocks = (unsigned)(pa.tiles + pb.tiles + bias_blocks);
    if (how.kernel == KERNEL_NARROW)
        return launch_small_bwd<2, 8>(blocks, g, s);
    return how.waves == 8 ? launch_small_bwd<4, 8>(blocks, g, s) : launch_small_bwd<4, 4>(blocks, g, s);
}

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
Together backward_together(const Shape &a, const ProductPlan *pa, const Shape &b, const ProductPlan *pb, int cus)
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

// A backward call: its two products (dA = dZ B and dB = dZ^T A), whether they
// run as one launch of small tiles, and its workspace: the gradient of the
// pre-activations (unless it is dC itself), the column sums, and the partials
// of whichever product splits more.
struct BackwardPlan {
    ProductPlan a, b;
    Together together;
    size_t sums_at, partials_at, bytes;
};

BackwardPlan plan_backward(int M, int N, int K, bool gated, int act, bool wants_a, bool wants_b, int cus)
{
    const int rows = gated ? 2 * N : N;
    const Shape a = {M, K, rows, 1, false, false}, b = {rows, K, M, 1, false, false};
    BackwardPlan w = {};
    w.sums_at = gated || act != GEMM355_ACT_NONE ? align_up(size_t(M) * rows * 2) : 0;
    w.partials_at = w.sums_at + align_up(size_t(ceil_div(M, grad_rows(M, N))) * rows * sizeof(float));
    if (M > 0 && K > 0)
        w.a = plan_product(a, false, cus);
    if (rows > 0 && K > 0)
        w.b = plan_product(b, false, cus);
    w.together = backward_together(a, wants_a ? &w.a : nullptr, b, wants_b ? &w.b : nullptr, cus);
    w.bytes = w.partials_at + std::max(w.a.workspace_bytes, w.b.workspace_bytes);
    return w;
}

template <bool GATED>
int layer_backward(int M, int N, int K, const void *A, const void *B, const void *Z, int act, const void *dC, void *dA,
                   void *dB, void *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0 || !act_ok(act))
        return GEMM355_ERR_INVALID_ARG;
    const size_t rows = (GATED ? 2 : 1) * size_t(N);
    const bool wants_a = dA && M > 0 && K > 0, wants_b = dB && N > 0 && K > 0, wants_bias = dbias && N > 0;
    if (!wants_a && !wants_b && !wants_bias)
        return GEMM355_OK;
    const bool needs_z = GATED || act != GEMM355_ACT_NONE;
    if (M > 0 && N > 0 && (!dC || (needs_z && !Z) || (wants_a && !B) || (wants_b && !A)))
        return GEMM355_ERR_INVALID_ARG;
    if (workspace_bytes > 0 && !workspace)
        return GEMM355_ERR_INVALID_ARG;
    const size_t a_bytes = size_t(M) * K * 2, b_bytes = rows * K * 2;
    const Array out[] = {{dA, a_bytes}, {dB, b_bytes}, {dbias, rows * 2}, {workspace, workspace_bytes}};
    const Array in[] = {{A, a_bytes}, {B, b_bytes}, {Z, size_t(M) * rows * 2}, {dC, size_t(M) * N * 2}};
    if (any_overlap(out, 4, in, 4))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 4) || !all_aligned(in, 4) || K % 8 != 0 || N % 8 != 0 ||
        !layer_extents_ok(M, N, GATED ? 2 * int64_t(N) : N, K))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const BackwardPlan w = plan_backward(M, N, K, GATED, act, wants_a, wants_b, cus);
    if (workspace_bytes < w.bytes)
        return GEMM355_ERR_UNSUPPORTED;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const void *dz = needs_z ? ws : dC;
    float *sums = reinterpret_cast<float *>(ws + w.sums_at);
    const int per = grad_rows(M, N), blocks = (int)ceil_div(M, per);
    if (needs_z && M > 0 && N > 0) {
        d::GradArgs g = {};
        g.z = static_cast<const uint16_t *>(Z);
        g.dc = static_cast<const uint16_t *>(dC);
        g.dz = reinterpret_cast<uint16_t *>(ws);
        g.sums = wants_bias ? sums : nullptr;
        g.M = M;
        g.N = N;
        g.act = act;
        g.rows = per;
        g.col_blocks = (int)ceil_div(N, d::GRAD_COLS);
        const int st = launch_kernel(d::dense_grad_kernel<GATED>, (unsigned)(int64_t(g.col_blocks) * blocks),
                                     (unsigned)d::GRAD_THREADS, g, s);
        if (st != GEMM355_OK)
            return st;
    }
    d::BiasArgs q = {needs_z ? sums : nullptr, static_cast<const uint16_t *>(dC), static_cast<uint16_t *>(dbias), (int)rows,
                     needs_z ? blocks : M};
    const int bias_blocks = wants_bias ? (int)ceil_div(rows, d::BIAS_COLS) : 0;
    const DenseArgs pa = args_of(M, K, (int)rows, dz, B, dA);          // dA = dZ B
    const DenseArgs pb = args_of((int)rows, K, M, dz, A, dB);          // dB = dZ^T A
    if (w.together.kernel != 0)
        return backward_small(pa, wants_a, pb, wants_b, q, bias_blocks, w.together, cus, s);
    if (wants_bias) {
        const int st = launch_kernel(d::dense_bias_kernel, (unsigned)bias_blocks, (unsigned)d::BIAS_THREADS, q, s);
        if (st != GEMM355_OK)
            return st;
    }
    if (wants_a) {
        const int st = product<__bf16, d::ROW_K, d::COL_K, d::EPI_STORE>(pa, w.a, ws + w.partials_at, s);
        if (st != GEMM355_OK)
            return st;
    }
    return wants_b ? product<__bf16, d::COL_K, d::COL_K, d::EPI_STORE>(pb, w.b, ws + w.partials_at, s) : GEMM355_OK;
}

template <bool GATED>
int layer_backward_workspace(int M, int N, int K, int act, size_t *bytes)
{
    if (M < 0 || N < 0 || K < 0 || !act_ok(act) || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!layer_extents_ok(M, N, GATED ? 2 * int64_t(N) : N, K))
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (N == 0 && (M == 0 || K == 0))   // no output has an element
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)   // (the same whichever outputs are wanted)
        *bytes = plan_backward(M, N, K, GATED, act, true, true, cus).bytes;
    return rc;
}

// ---- Newton-Schulz ---------------------------------------------------------

// With m the smaller and n the larger side, X (rows x cols) stays as it is
// stored: the Gram matrix is X X^T of a wide and X^T X of a tall matrix, and
// the update P X or X P.
constexpr float kPolyScale = 256.0f;   // S and P are held times this
// X is held times this, as large as loses nothing at the top: an element of 16,
// FP16's largest value then, makes a diagonal element of S overflow too.
constexpr float kIterateScale = 4096.0f;

struct OrthoPlan {
    ProductPlan gram, square, update;
    size_t x1_at, s_at, p_at, norm_at, partials_at, bytes;
    int norm_blocks;
};

OrthoPlan plan_ortho(int batch, int rows, int cols, int cus)
{
    const int m = std::min(rows, cols), n = std::max(rows, cols);
    const size_t x = align_up(size_t(batch) * rows * cols * 2), s = align_up(size_t(batch) * m * m * 2);
    OrthoPlan o = {};
    o.gram = plan_product({m, m, n, batch, true, false, rows <= cols}, false, cus);
    o.square = plan_product({m, m, m, batch, true, false, true}, false, cus);
    o.update = plan_product({rows, cols, m, batch, false, false}, false, cus);
    // (a launch has fewer than 2^32 threads, whatever the batch)
    o.norm_blocks = (int)std::min<int64_t>({d::NS_BLOCKS, ceil_div(int64_t(rows) * cols, d::NS_THREADS * 8),
                                            ((int64_t(1) << 32) - 1) / d::NS_THREADS / batch});
    o.x1_at = x;
    o.s_at = 2 * x;
    o.p_at = o.s_at + s;
    o.norm_at = o.p_at + s;
    o.partials_at = o.norm_at + align_up(size_t(batch) * o.norm_blocks * sizeof(double));
    o.bytes = o.partials_at + std::max({o.gram.workspace_bytes, o.square.workspace_bytes, o.update.workspace_bytes});
    return o;
}

template <bool FP32>
int ortho_start(const d::NormArgs &n, int batch, hipStream_t s)
{
    d::NormArgs a = n;
    const unsigned blocks = (unsigned)(int64_t(n.blocks) * batch);
    const int st = launch_kernel(d::ns_norm_kernel<FP32>, blocks, (unsigned)d::NS_THREADS, a, s);
    return st == GEMM355_OK ? launch_kernel(d::ns_scale_kernel<FP32>, blocks, (unsigned)d::NS_THREADS, a, s) : st;
}

// One Newton-Schulz step from x to out (BF16 and unscaled after the last).
template <bool WIDE, class TO>
int ortho_step(const OrthoPlan &o, int batch, int rows, int cols, const void *x, uint8_t *ws, void *out, float a, float b,
               float c, bool last, hipStream_t s)
{
    typedef _Float16 h;
    const int m = WIDE ? rows : cols, n = WIDE ? cols : rows;
    void *S = ws + o.s_at, *P = ws + o.p_at, *partials = ws + o.partials_at;
    DenseArgs p = args_of(m, m, n, x, x, S);
    p.batch = batch;
    p.alpha = kPolyScale / (kIterateScale * kIterateScale);
    int st = WIDE ? product<h, d::ROW_K, d::ROW_K, d::EPI_STORE_SYM>(p, o.gram, partials, s)
                  : product<h, d::COL_K, d::COL_K, d::EPI_STORE_SYM>(p, o.gram, partials, s);
    if (st != GEMM355_OK)
        return st;
    p = args_of(m, m, m, S, S, P);   // P = a I + b S + c S^2
    p.batch = batch;
    p.r = S;
    p.alpha = c / kPolyScale;
    p.beta = b;
    p.gamma = a * kPolyScale;
    st = product<h, d::ROW_K, d::ROW_K, d::EPI_POLY>(p, o.square, partials, s);
    if (st != GEMM355_OK)
        return st;
    p = WIDE ? args_of(rows, cols, m, P, x, out) : args_of(rows, cols, m, x, P, out);
    p.batch = batch;
    p.alpha = (last ? 1.0f / kIterateScale : 1.0f) / kPolyScale;
    // P = P^T: as the right-hand operand its rows are its columns
    return WIDE ? product<h, d::ROW_K, d::COL_K, d::EPI_STORE, TO>(p, o.update, partials, s)
                : product<h, d::ROW_K, d::ROW_K, d::EPI_STORE, TO>(p, o.update, partials, s);
}

// Each matrix as any other operand; the batch's blocks of 16 x 16 (of which no
// tile has fewer) below 2^28, so that counts of tiles stay within 32 bits.
bool ortho_extents_ok(int64_t batch, int64_t rows, int64_t cols)
{
    const int64_t m = std::min(rows, cols);
    return extent_ok(rows, cols * 2) && extent_ok(cols, rows * 2) && extent_ok(m, m * 2) && batch <= 65535 &&
           batch * ceil_div(rows, 16) * ceil_div(cols, 16) <= (int64_t(1) << 28);
}

} // namespace

extern "C" int gemm355_force_layer_kernel(int kernel)
{
    if (kernel < 0 || kernel > KERNEL_NARROW)
        return GEMM355_ERR_INVALID_ARG;
    g_layer_kernel.store(kernel, std::memory_order_relaxed);
    return GEMM355_OK;
}

extern "C" int gemm_bf16_nt_bias_act_res(int M, int N, int K, const void *A, const void *B, const void *bias,
                                         int activation, const void *R, void *Z, void *C, void *workspace,
                                         size_t workspace_bytes, void *stream)
{
    return layer_forward<false>(M, N, K, A, B, bias, activation, R, Z, C, workspace, workspace_bytes, stream);
}

extern "C" int gemm_bf16_nt_bias_act_res_workspace_size(int M, int N, int K, size_t *bytes)
{
    return layer_forward_workspace<false>(M, N, K, bytes);
}

extern "C" int gemm_bf16_nt_bias_act_bwd(int M, int N, int K, const void *A, const void *B, const void *Z,
                                         int activation, const void *dC, void *dA, void *dB, void *dbias,
                                         void *workspace, size_t workspace_bytes, void *stream)
{
    return layer_backward<false>(M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace, workspace_bytes, stream);
}

extern "C" int gemm_bf16_nt_bias_act_bwd_workspace_size(int M, int N, int K, int activation, size_t *bytes)
{
    return layer_backward_workspace<false>(M, N, K, activation, bytes);
}

extern "C" int gemm_bf16_nt_gated(int M, int N, int K, const void *A, const void *B, const void *bias, int activation,
                                  void *Z, void *C, void *workspace, size_t workspace_bytes, void *stream)
{
    return layer_forward<true>(M, N, K, A, B, bias, activation, nullptr, Z, C, workspace, workspace_bytes, stream);
}

extern "C" int gemm_bf16_nt_gated_workspace_size(int M, int N, int K, size_t *bytes)
{
    return layer_forward_workspace<true>(M, N, K, bytes);
}

extern "C" int gemm_bf16_nt_gated_bwd(int M, int N, int K, const void *A, const void *B, const void *Z, int activation,
                                      const void *dC, void *dA, void *dB, void *dbias, void *workspace,
                                      size_t workspace_bytes, void *stream)
{
    return layer_backward<true>(M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace, workspace_bytes, stream);
}

extern "C" int gemm_bf16_nt_gated_bwd_workspace_size(int M, int N, int K, size_t *bytes)
{
    return layer_backward_workspace<true>(M, N, K, GEMM355_ACT_NONE, bytes);
}

extern "C" int gemm355_newton_schulz_workspace_size(int batch, int rows, int cols, size_t *bytes)
{
    if (batch < 0 || rows < 0 || cols < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!ortho_extents_ok(batch, rows, cols))
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (batch == 0 || rows == 0 || cols == 0)
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)
        *bytes = plan_ortho(batch, rows, cols, cus).bytes;
    return rc;
}

extern "C" int gemm355_newton_schulz(int batch, int rows, int cols, int g_type, const void *G, int steps, float a,
                                     float b, float c, float eps, void *O, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    if (batch < 0 || rows < 0 || cols < 0 || (g_type != GEMM355_BF16 && g_type != GEMM355_FP32) || steps < 1 ||
        steps > 64 || !isfinite(a) || !isfinite(b) || !isfinite(c) || !isfinite(eps) || eps < 0.0f)
        return GEMM355_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0)
        return GEMM355_OK;
    if (!G || !O || !workspace)
        return GEMM355_ERR_INVALID_ARG;
    const int64_t elements = int64_t(rows) * cols;
    const Array out[] = {{O, size_t(batch) * elements * 2}, {workspace, workspace_bytes}};
    const Array in[] = {{G, size_t(batch) * elements * (g_type == GEMM355_FP32 ? 4 : 2)}};
    if (any_overlap(out, 2, in, 1))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 2) || !all_aligned(in, 1) || rows % 8 != 0 || cols % 8 != 0 ||
        !ortho_extents_ok(batch, rows, cols))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const OrthoPlan o = plan_ortho(batch, rows, cols, cus);
    if (workspace_bytes < o.bytes)
        return GEMM355_ERR_UNSUPPORTED;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    d::NormArgs n = {};
    n.g = G;
    n.partial = reinterpret_cast<double *>(ws + o.norm_at);
    n.x = reinterpret_cast<uint16_t *>(ws);
    n.elements = elements;
    n.blocks = o.norm_blocks;
    n.scale = kIterateScale;
    n.eps = eps;
    int st = g_type == GEMM355_FP32 ? ortho_start<true>(n, batch, s) : ortho_start<false>(n, batch, s);
    uint8_t *x = ws, *next = ws + o.x1_at;
    for (int i = 0; i < steps && st == GEMM355_OK; ++i) {
        const bool last = i == steps - 1, wide = rows <= cols;
        auto step = wide ? (last ? ortho_step<true, __bf16> : ortho_step<true, _Float16>)
                         : (last ? ortho_step<false, __bf16> : ortho_step<false, _Float16>);
        st = step(o, batch, rows, cols, x, ws, last ? O : next, a, b, c, last, s);
        std::swap(x, next);
    }
    return st;
}
