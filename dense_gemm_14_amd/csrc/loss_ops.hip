// loss_ops.hip -- host side of the softmax cross entropy over a vocabulary and its
// gradient (cross_entropy.hpp): argument checks, plans, workspace layout and
// launches. The C ABI is declared in include/gemm355.h. Nothing here allocates
// memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "gemm355.h"
#include "cross_entropy.hpp"
#include "dense_plan.hpp"

namespace {

using namespace gemm355::host;

constexpr int kPieceUnit = 256;     // columns: whole tiles of every kernel

// Largest number of columns whose `row_bytes` each stay below 2^31 bytes.
int64_t columns_within(int64_t row_bytes)
{
    return ((int64_t(1) << 31) - 1) / std::max<int64_t>(row_bytes, 1) / kPieceUnit * kPieceUnit;
}

// V cut into pieces of at most `most` columns, all but the last of that size.
struct Pieces {
    int count, width, last;
};
Pieces cut(int V, int64_t most)
{
    Pieces p = {};
    if (V == 0)
        return p;
    p.width = (int)std::min<int64_t>(V, most);
    p.count = (int)ceil_div(V, p.width);
    p.last = V - (p.count - 1) * p.width;
    return p;
}

// Columns of a run of EPI_CE by the kernel of its product.
int run_width(const ProductPlan &p)
{
    return p.kernel >= KERNEL_SMALL ? 16 * p.small.nb : p.kernel == KERNEL_TILE ? d::TILE / 2 : d::BIG / 2;
}

bool id_type_ok(int t) { return t == GEMM355_INT32 || t == GEMM355_INT64; }
size_t id_size(int t) { return t == GEMM355_INT64 ? 8 : 4; }

// Whether the forward call moves the kept rows of A together first. Not for few
// tokens, where a row more or less changes nothing in the time of a tile, and not
// where the whole product takes little more than the launch that moves them (1500 x
// 1000, K = 128, nothing left out: 14.3 us with it, 9.9 without).
constexpr int kDirectRows = 64;
bool moves_rows(int M, int V, int K) { return M > kDirectRows && int64_t(M) * V * std::max(K, 64) > int64_t(1) << 33; }

struct ForwardPlan {
    Pieces pieces;
    ProductPlan product[2];      // of a piece, of the last one
    int runs[2];
    size_t rows_at, map_at, target_at, a_at, picked_at, stats_at, partials_at, bytes;
};

ForwardPlan plan_forward(int M, int V, int K, int cus)
{
    ForwardPlan f = {};
    // (blocks of 16 x 16, of which no tile has fewer, below 2^27, so that counts of
    // tiles stay within 32 bits)
    const int64_t counted = (int64_t(1) << 27) / ceil_div(M, 16) * 16 / kPieceUnit * kPieceUnit;
    f.pieces = cut(V, std::min(columns_within(int64_t(K) * 2), counted));
    int64_t runs = 0;
    size_t partials = 0;
    for (int i = 0; i < 2 && f.pieces.count > i; ++i) {
        // (one piece: it is the last)
        const bool last = i == 1 || f.pieces.count == 1;
        const int N = last ? f.pieces.last : f.pieces.width;
        f.product[i] = plan_product({M, N, K, 1, false, false}, true, cus);
        f.runs[i] = (int)ceil_div(N, run_width(f.product[i]));
        runs += int64_t(f.runs[i]) * (last ? 1 : f.pieces.count - 1);
        partials = std::max(partials, f.product[i].workspace_bytes);
    }
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes);
        return here;
    };
    const bool moved = moves_rows(M, V, K);
    f.rows_at = take(moved ? sizeof(int) : 0);
    f.map_at = take(moved ? size_t(M) * 4 : 0);
    f.target_at = take(moved ? size_t(M) * 4 : 0);
    f.a_at = take(moved ? size_t(M) * K * 2 : 0);
    f.picked_at = take(size_t(M) * 4);
    f.stats_at = take(size_t(runs) * M * 8);
    f.partials_at = take(partials);
    f.bytes = at;
    return f;
}

constexpr int64_t kMaxTokens = 1 << 26;

// Tokens, and a piece of at least one unit of the vocabulary, within 32-bit
// offsets.
bool extents_ok(int64_t M, int64_t K)
{
    return M <= kMaxTokens && extent_ok(std::max<int64_t>(M, 1), K * 2) && columns_within(K * 2) >= kPieceUnit;
}

constexpr size_t kMaxLogits = size_t(1) << 46;   // (M V, so that no size runs over)

// Workgroups that move rows, each after a look at all targets: two rows for each of
// a workgroup's waves, or more than four workgroups to a unit would be.
int prep_blocks(int M, int cus) { return (int)std::min<int64_t>(std::max<int64_t>(ceil_div(M, 2 * d::CE_WAVES), 1), 4 * int64_t(cus)); }

// Bytes of a piece's gradient of the logits.
constexpr int64_t kPieceBytes = int64_t(256) << 20;

// dA of few tokens is a few tiles that each sum over a whole piece of the vocabulary:
// more workgroups take a share of it than a layer's products are split over (whole
// gradients with 64 and with 16 at most, us: 5 x 29422 x 72 30.7 and 38.3, 82 x 65635 x
// 472 99 and 114, 200 x 50000 x 264 78 and 87, 1000 x 20000 x 128 70 and 74).
constexpr int kSumSplits = 64;

// The small tiles sum a vocabulary up to here; beyond, where their estimates were not
// fitted and fall short of what they take, 128 x 128 ones, split (whole gradients, small
// and 128, us: 110 x 4699 x 1120 38 and 45, 2 x 7170 x 2424 56 and 58, 64 x 8000 x 1024
// 48 and 45, 43 x 9226 x 480 40 and 38, 16 x 16000 x 4096 144 and 123). Both products in
// one launch, which saves one, somewhat further (so, and apart: 150 x 8000 x 128 28 and
// 32, 150 x 12696 x 88 47 and 33, 300 x 12000 x 64 40 and 32).
constexpr int kSmallSums = 7680, kSmallBoth = 10240;
ProductPlan plan_sum(const Shape &s, int cus)
{
    ProductPlan p = plan_product(s, false, cus);
    if (p.kernel >= KERNEL_SMALL && s.K > kSmallSums && p.us > 0.0) {      // (0: forced)
        p.kernel = KERNEL_TILE;
        p.tiles = plan_tile(s, cus);
        p.workspace_bytes = p.tiles.workspace_bytes;
    }
    return p;
}

struct BackwardPlan {
    Pieces pieces;
    ProductPlan z[2], a[2], b[2];     // of a piece, of the last one
    Together together;                // both products of the only piece
    int min_steps[2];
    int pitch;                        // of dz
    size_t rows_at, scale_at, map_at, target_at, lse_at, weight_at, a_at, dz_at, acc_at, partials_at, bytes;
};

// Rows of dz and of the moved A, for their extents: where the product over them may
// take whole K steps, up to a step for each split more than there are tokens.
int64_t padded_rows(int64_t M)
{
    return M > (d::BIG_MIN_STEPS - 1) * d::BIG_BK ? M + d::BIG_BK * kMaxSplits : ceil_div(M, 256) * 256;
}
// Columns that a piece's dz may have.
int64_t piece_columns(int64_t M) { return columns_within(padded_rows(M) * 2); }
bool backward_extents_ok(int64_t M, int64_t K)
{
    M = std::max<int64_t>(M, 1);
    return extents_ok(M, K) && extent_ok(padded_rows(M), K * 2) && piece_columns(M) >= kPieceUnit;
}

int splits_of(const ProductPlan &p) { return p.kernel >= KERNEL_SMALL ? 1 : p.tiles.splits; }

BackwardPlan plan_backward(int M, int V, int K, bool wants_a, bool wants_b, int cus)
{
    BackwardPlan w = {};
    const int rows = std::max(M, 1);
    const int64_t fit = piece_columns(rows);
    const int64_t want = std::max<int64_t>(8192, kPieceBytes / 2 / rows / kPieceUnit * kPieceUnit);
    // Pieces of sixteen tiles' columns: with a multiple of sixteen tiles of rows
    // (4096 tokens or values of K) a piece's products fill whole rounds of 256 units,
    // and only the last one leaves some idle (4096 x 128000, K = 4096: 31.25 rounds in
    // all, 32 for four equal pieces).
    int64_t most = std::min({want, fit, columns_within(int64_t(K) * 2)});
    if (most >= 16 * kPieceUnit)
        most = most / (16 * kPieceUnit) * (16 * kPieceUnit);
    w.pieces = cut(V, most);
    w.pitch = (int)(ceil_div(w.pieces.width, 8) * 8);
    size_t partials = 0;
    int64_t depth = 0;
    for (int i = 0; i < 2; ++i) {
        const int N = i == 1 ? w.pieces.last : w.pieces.width;
        w.z[i] = plan_product({rows, N, K, 1, false, false}, true, cus);
        w.a[i] = plan_sum({rows, K, N, 1, false, false, false, kSumSplits}, cus);
        w.b[i] = plan_product({N, K, rows, 1, false, false}, false, cus);
        w.min_steps[i] = w.b[i].kernel <= KERNEL_SPLIT ? d::BIG_MIN_STEPS : 0;
        partials = std::max({partials, w.z[i].workspace_bytes, w.a[i].workspace_bytes, w.b[i].workspace_bytes});
        depth = std::max(depth, d::ce_depth(rows, splits_of(w.b[i]), w.min_steps[i]));
    }
    // (one launch takes none of the partials and whole steps that are set aside)
    if (w.pieces.count == 1 && M > 0 && wants_a && wants_b && V <= kSmallBoth)
        w.together = backward_together({M, K, V, 1, false, false}, &w.a[1], {V, K, M, 1, false, false}, &w.b[1], cus);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes);
        return here;
    };
    w.rows_at = take(sizeof(int));
    w.scale_at = take(sizeof(float));
    w.map_at = take(size_t(M) * 4);
    w.target_at = take(size_t(M) * 4);
    w.lse_at = take(size_t(M) * 4);
    w.weight_at = take(size_t(M) * 4);
    w.a_at = take(size_t(depth) * K * 2);
    w.dz_at = take(size_t(depth) * w.pitch * 2);
    w.acc_at = take(w.pieces.count > 1 ? size_t(M) * K * 4 : 0);
    w.partials_at = take(partials);
    w.bytes = at;
    return w;
}

template <int BLOCKS, int WAVES>
int launch_small_loss(unsigned blocks, d::SmallLossArgs &g, hipStream_t s)
{
    return launch_kernel(d::dense_small_loss_kernel<BLOCKS, WAVES>, blocks, 64u * WAVES, g, s);
}

// Both products of the only piece in one launch.
int both_small(DenseArgs pa, DenseArgs pb, const Together &how, int cus, hipStream_t s)
{
    d::SmallLossArgs g = {};
    auto place = [&](DenseArgs &p) {
        const SmallPlan t = plan_small({p.M, p.N, p.K, 1, false, false}, false, how.kernel == KERNEL_NARROW, cus);
        p.tiles_m = t.tiles_m;
        p.tiles_n = t.tiles_n;
        p.tiles = p.whole = t.tiles;
        p.splits = 1;
        p.supergroup = 8;
    };
    place(pa);
    place(pb);
    g.a = pa;
    g.b = pb;
    g.tiles_a = pa.tiles;
    g.tiles_b = pb.tiles;
    g.first_b = pb.K > pa.K;
    const unsigned blocks = (unsigned)(pa.tiles + pb.tiles);
    if (how.kernel == KERNEL_NARROW)
        return launch_small_loss<2, 8>(blocks, g, s);
    return how.waves == 8 ? launch_small_loss<4, 8>(blocks, g, s) : launch_small_loss<4, 4>(blocks, g, s);
}

} // namespace

extern "C" int gemm_bf16_nt_cross_entropy_workspace_size(int M, int V, int K, size_t *bytes)
{
    if (M < 0 || V < 0 || K < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!extents_ok(M, K) || size_t(M) * size_t(V) > kMaxLogits)
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (M == 0)
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)
        *bytes = plan_forward(M, V, K, cus).bytes;
    return rc;
}

extern "C" int gemm_bf16_nt_cross_entropy(int M, int V, int K, const void *A, const void *B, int target_type,
                                          const void *targets, float *loss, float *lse, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    if (M < 0 || V < 0 || K < 0 || !id_type_ok(target_type))
        return GEMM355_ERR_INVALID_ARG;
    if (M == 0)
        return GEMM355_OK;
    if (!targets || !loss || !lse || !workspace || (K > 0 && (!A || (V > 0 && !B))))
        return GEMM355_ERR_INVALID_ARG;
    if (K % 8 != 0 || !extents_ok(M, K) || size_t(M) * size_t(V) > kMaxLogits)
        return GEMM355_ERR_UNSUPPORTED;
    const Array out[] = {{workspace, workspace_bytes}, {loss, size_t(M) * 4}, {lse, size_t(M) * 4}};
    const Array in[] = {{A, size_t(M) * K * 2}, {B, size_t(V) * K * 2}, {targets, size_t(M) * id_size(target_type)}};
    if (any_overlap(out, 3, in, 3))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 1) || !all_aligned(in, 2) || !aligned(targets, id_size(target_type)) || !aligned(loss, 4) ||
        !aligned(lse, 4))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const ForwardPlan f = plan_forward(M, V, K, cus);
    if (workspace_bytes < f.bytes)
        return GEMM355_ERR_UNSUPPORTED;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const bool moved = moves_rows(M, V, K), wide = target_type == GEMM355_INT64;
    if (moved) {
        d::CePrepArgs q = {};
        q.ids = targets;
        q.a = A;
        q.rows = reinterpret_cast<int *>(ws + f.rows_at);
        q.map = reinterpret_cast<int *>(ws + f.map_at);
        q.target = reinterpret_cast<int *>(ws + f.target_at);
        q.ka = ws + f.a_at;
        q.loss0 = loss;
        q.lse0 = lse;
        q.M = M;
        q.V = V;
        q.K = K;
        const int blocks = prep_blocks(M, cus);
        q.chunk = (int)ceil_div(M, blocks);
        q.wide = wide;
        const int st = launch_kernel(d::ce_prep_kernel<false>, (unsigned)blocks, (unsigned)d::CE_THREADS, q, s);
        if (st != GEMM355_OK)
            return st;
    }
    int runs = 0;
    for (int i = 0; i < f.pieces.count; ++i) {
        const bool last = i == f.pieces.count - 1;
        const int which = last && f.pieces.count > 1 ? 1 : 0;
        const int N = last ? f.pieces.last : f.pieces.width;
        DenseArgs p = args_of(M, N, K, moved ? ws + f.a_at : A,
                              static_cast<const uint8_t *>(B) + size_t(i) * f.pieces.width * K * 2, nullptr);
        p.v0 = i * f.pieces.width;
        p.stats = reinterpret_cast<gemm355::f32x2 *>(ws + f.stats_at) + size_t(runs) * M;
        p.picked = reinterpret_cast<float *>(ws + f.picked_at);
        p.stats_rows = M;
        p.vocab = V;
        p.wide = wide;
        if (moved) {
            p.rows = reinterpret_cast<int *>(ws + f.rows_at);
            p.target = reinterpret_cast<int *>(ws + f.target_at);
        } else {
            p.ids = targets;
        }
        runs += f.runs[which];
        const int st = product<__bf16, d::ROW_K, d::ROW_K, d::EPI_CE>(p, f.product[which], ws + f.partials_at, s);
        if (st != GEMM355_OK)
            return st;
    }
    d::CeJoinArgs j = {};
    j.stats = reinterpret_cast<gemm355::f32x2 *>(ws + f.stats_at);
    j.picked = reinterpret_cast<float *>(ws + f.picked_at);
    if (moved) {
        j.rows = reinterpret_cast<int *>(ws + f.rows_at);
        j.map = reinterpret_cast<int *>(ws + f.map_at);
    }
    j.ids = targets;
    j.wide = wide;
    j.loss = loss;
    j.lse = lse;
    j.M = M;
    j.V = V;
    j.stride = M;
    j.runs = runs;
    return M > kDirectRows ? launch_kernel(d::ce_join_kernel<16>, (unsigned)ceil_div(M, 16), (unsigned)d::CE_THREADS, j, s)
                           : launch_kernel(d::ce_join_kernel<1>, (unsigned)M, (unsigned)d::CE_THREADS, j, s);
}

extern "C" int gemm_bf16_nt_cross_entropy_bwd_workspace_size(int M, int V, int K, size_t *bytes)
{
    if (M < 0 || V < 0 || K < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!backward_extents_ok(M, K) || size_t(M) * size_t(V) > kMaxLogits)
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (K == 0 || (M == 0 && V == 0))
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)
        *bytes = plan_backward(M, V, K, false, false, cus).bytes;   // (the same whichever outputs are wanted)
    return rc;
}

extern "C" int gemm_bf16_nt_cross_entropy_bwd(int M, int V, int K, const void *A, const void *B, int target_type,
                                              const void *targets, const float *lse, const float *dloss, void *dA,
                                              void *dB, void *workspace, size_t workspace_bytes, void *stream)
{
    if (M < 0 || V < 0 || K < 0 || !id_type_ok(target_type))
        return GEMM355_ERR_INVALID_ARG;
    const bool wants_a = dA && M > 0 && K > 0, wants_b = dB && V > 0 && K > 0;
    if (!wants_a && !wants_b)
        return GEMM355_OK;
    if ((M > 0 && (!A || !targets || !lse)) || (V > 0 && M > 0 && !B) || !workspace)
        return GEMM355_ERR_INVALID_ARG;
    if (K % 8 != 0 || !backward_extents_ok(M, K) || size_t(M) * size_t(V) > kMaxLogits)
        return GEMM355_ERR_UNSUPPORTED;
    const size_t a_bytes = size_t(M) * K * 2, b_bytes = size_t(V) * K * 2;
    const Array out[] = {{dA, a_bytes}, {dB, b_bytes}, {workspace, workspace_bytes}};
    const Array in[] = {{A, a_bytes}, {B, b_bytes}, {targets, size_t(M) * id_size(target_type)}, {lse, size_t(M) * 4},
                        {dloss, size_t(M) * 4}};
    if (any_overlap(out, 3, in, 5))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 3) || !all_aligned(in, 2) || !aligned(targets, id_size(target_type)) || !aligned(lse, 4) ||
        !aligned(dloss, 4))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const BackwardPlan w = plan_backward(M, V, K, wants_a, wants_b, cus);
    if (workspace_bytes < w.bytes)
        return GEMM355_ERR_UNSUPPORTED;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    d::CePrepArgs q = {};
    q.ids = targets;
    q.a = A;
    q.lse = lse;
    q.dloss = dloss;
    q.rows = reinterpret_cast<int *>(ws + w.rows_at);
    q.scale = reinterpret_cast<float *>(ws + w.scale_at);
    q.map = reinterpret_cast<int *>(ws + w.map_at);
    q.target = reinterpret_cast<int *>(ws + w.target_at);
    q.klse = reinterpret_cast<float *>(ws + w.lse_at);
    q.weight = reinterpret_cast<float *>(ws + w.weight_at);
    q.ka = ws + w.a_at;
    q.da = wants_a ? dA : nullptr;
    q.dz = ws + w.dz_at;
    q.M = M;
    q.V = V;
    q.K = K;
    q.dz_pitch = w.pitch;
    for (int i = 0; i < 2; ++i) {
        q.splits[i] = splits_of(w.b[i]);
        q.min_steps[i] = w.min_steps[i];
    }
    q.wide = target_type == GEMM355_INT64;
    const int blocks = prep_blocks(M, cus);
    q.chunk = (int)ceil_div(M, blocks);
    int st = launch_kernel(d::ce_prep_kernel<true>, (unsigned)blocks, (unsigned)d::CE_THREADS, q, s);
    for (int i = 0; i < w.pieces.count && st == GEMM355_OK; ++i) {
        const int which = i == w.pieces.count - 1 ? 1 : 0;
        const int N = which ? w.pieces.last : w.pieces.width;
        const size_t from = size_t(i) * w.pieces.width * K * 2;
        const uint8_t *b = M > 0 ? static_cast<const uint8_t *>(B) + from : nullptr;
        void *partials = ws + w.partials_at;
        if (M > 0) {
            DenseArgs p = args_of(M, N, K, q.ka, b, q.dz);      // dz
            p.rows = q.rows;
            p.target = q.target;
            p.lse = q.klse;
            p.weight = q.weight;
            p.v0 = i * w.pieces.width;
            p.ldc = w.pitch;
            st = product<__bf16, d::ROW_K, d::ROW_K, d::EPI_CE_GRAD>(p, w.z[which], partials, s);
        }
        // dB = dz^T A, dA += dz B
        const bool one = w.together.kernel != 0;
        DenseArgs pb = args_of(N, K, one ? M : (int)d::ce_depth(std::max(M, 1), q.splits[which], q.min_steps[which]), q.dz,
                               q.ka, wants_b ? static_cast<uint8_t *>(dB) + from : nullptr);
        pb.rows = q.rows;
        pb.rows_in_k = 1;
        pb.min_steps = one ? 0 : q.min_steps[which];
        pb.lda = w.pitch;
        pb.scale = q.scale;
        DenseArgs pa = args_of(M, K, N, q.dz, b, dA);
        pa.rows = q.rows;
        pa.lda = w.pitch;
        pa.scale = q.scale;
        pa.acc = reinterpret_cast<float *>(ws + w.acc_at);
        pa.map = q.map;
        pa.c_rows = M;
        pa.add = i > 0;
        pa.last = which;
        if (one) {
            if (st == GEMM355_OK)
                st = both_small(pa, pb, w.together, cus, s);
            continue;
        }
        if (wants_b && st == GEMM355_OK)
            st = product<__bf16, d::COL_K, d::COL_K, d::EPI_SCALE>(pb, w.b[which], partials, s);
        if (wants_a && st == GEMM355_OK)
            st = product<__bf16, d::ROW_K, d::COL_K, d::EPI_ACC>(pa, w.a[which], partials, s);
    }
    return st;
}
