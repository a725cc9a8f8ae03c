// model_ops.hip -- host side of the calls around a network's layers that pass
// over rows: embedding, layer norm and their gradients (embedding.hpp,
// layer_norm.hpp). Argument checks, workspace layout and launches. The C ABI is
// declared in include/gemm355.h. Nothing here allocates memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "gemm355.h"
#include "checks.hpp"
#include "embedding.hpp"
#include "layer_norm.hpp"

namespace {

using namespace gemm355::host;
namespace r = gemm355::rows;
using gemm355::Int;

bool type_ok(int t) { return t == GEMM355_BF16 || t == GEMM355_FP32; }
bool id_type_ok(int t) { return t == GEMM355_INT32 || t == GEMM355_INT64; }
size_t size_of(int type) { return type == GEMM355_FP32 ? 4 : 2; }
size_t id_size(int type) { return type == GEMM355_INT64 ? 8 : 4; }

// Elements of an array; arrays beyond this are refused, so that no product of
// sizes runs over.
constexpr int64_t kMaxElements = int64_t(1) << 40;
bool elements_ok(int64_t rows, int64_t cols) { return rows * cols <= kMaxElements; }

// f(T{}) for a type of the C ABI.
template <class F>
int with_type(int type, F &&f)
{
    return type == GEMM355_FP32 ? f(float{}) : f(__bf16{});
}

int ceil_log2(int64_t n)
{
    int l = 0;
    while ((int64_t(1) << l) < n)
        ++l;
    return l;
}

// ---- embedding -------------------------------------------------------------

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

template <int PER>
int launch_embed(r::EmbedArgs &p, int e_type, int y_type, int64_t blocks, hipStream_t s)
{
    return with_type(e_type, [&](auto e) {
        return with_type(y_type, [&](auto y) {
            return launch_kernel(r::embed_kernel<decltype(e), decltype(y), PER>, (unsigned)std::min(blocks, kMaxBlocks),
                                 (unsigned)r::EMBED_THREADS, p, s);
        });
    });
}

// ---- embedding's gradient ----------------------------------------------------

constexpr int kMaxVocab = 1 << 30;     // (a launch has fewer than 2^32 threads)

struct EmbedBwdPlan {
    bool few;                   // tokens, in one launch
    int range, groups;          // ids per workgroup (few: of all; else: of the order), workgroups
    int block, blocks, pieces;
    int shift, buckets, chunks; // many tokens (chunks > 0): ids per bucket 1 << shift
    size_t sorted_at, partial_at, counts_at, total_at, bucket_start_at, bucketed_at, bytes;
};

// Tokens from which on they are dealt out to buckets first, and the ids that those
// hold. Measured, BF16, every workgroup reading all ids and so (us): 32768 of 128000 x
// 1024 81 and 98, 65536 of 128000 x 1024 120 and 125, 131072 of 256000 x 1024 227 and
// 191, 262144 of 50000 x 512 205 and 131, 1048576 of 1048576 x 64 2020 and 181.
constexpr int kBucketTokens = 3 << 15;
constexpr int64_t kBucketVocab = int64_t(r::MAX_BUCKETS) * r::ORDER_MAX_RANGE;

EmbedBwdPlan plan_embed_bwd(int tokens, int vocab, int cols, int cus)
{
    EmbedBwdPlan e = {};
    e.pieces = (int)ceil_div(cols, 512);
    e.few = tokens <= r::FEW_TOKENS;
    if (e.few) {
        // four workgroups for every unit, or as many as there are ids
        e.range = (int)std::min<int64_t>(r::FEW_RANGE, ceil_div(int64_t(vocab) * e.pieces, 4 * int64_t(cus)));
        e.groups = (int)ceil_div(vocab, e.range);
        return e;
    }
    e.range = (int)std::min<int64_t>(r::ORDER_MAX_RANGE, ceil_div(vocab, cus));
    e.groups = (int)ceil_div(vocab, e.range);
    // blocks of up to 32 tokens, fewer where that leaves fewer waves than run
    // at a time
    e.block = r::SUMS_BLOCK;
    while (e.block > 4 && ceil_div(tokens, e.block) * e.pieces < 16 * int64_t(cus))
        e.block /= 2;
    e.blocks = (int)ceil_div(tokens, e.block);
    e.sorted_at = align_up((size_t(vocab) + 1) * sizeof(int));
    e.partial_at = e.sorted_at + align_up(size_t(tokens) * 8);
    e.bytes = e.partial_at + size_t(e.blocks) * 2 * cols * sizeof(float);
    if (tokens >= kBucketTokens && vocab <= kBucketVocab) {
        e.shift = ceil_log2(ceil_div(vocab, r::MAX_BUCKETS));
        e.range = 1 << e.shift;
        e.groups = e.buckets = (int)ceil_div(vocab, e.range);
        e.chunks = (int)ceil_div(tokens, r::CHUNK);
        // (read for the last time before the first partial row is written)
        e.counts_at = e.partial_at;
        e.total_at = e.counts_at + align_up(size_t(e.chunks) * e.buckets * sizeof(int));
        e.bucket_start_at = e.total_at + align_up(size_t(e.buckets) * sizeof(int));
        e.bucketed_at = e.bucket_start_at + align_up((size_t(e.buckets) + 1) * sizeof(int));
        e.bytes = std::max(e.bytes, e.bucketed_at + size_t(tokens) * 8);
    }
    return e;
}

// ---- layer norm --------------------------------------------------------------

// f(Int<lanes>{}, Int<1>{}) with the lanes, a wave's at most, that hold rows of up
// to 512 columns.
template <class F>
int with_lanes(int cols, F &&f)
{
    if (cols <= 64)
        return f(Int<8>{}, Int<1>{});
    if (cols <= 128)
        return f(Int<16>{}, Int<1>{});
    if (cols <= 256)
        return f(Int<32>{}, Int<1>{});
    return f(Int<64>{}, Int<1>{});
}

// The kernel that holds rows of `cols` columns: f(Int<lanes>{}, Int<eights of
// columns per lane>{}), or f(Int<0>{}, Int<0>{}) for wider rows, which are read
// again. A wave holds up to 4096 columns where there are rows for every wave of
// the card, four waves otherwise.
template <class F>
int with_rows(int cols, bool many, F &&f)
{
    const int64_t per_wave = ceil_div(cols, 512), per_four = ceil_div(cols, 2048);
    if (per_wave <= 1)
        return with_lanes(cols, f);
    if (many) {
        if (per_wave <= 2)
            return f(Int<64>{}, Int<2>{});
        if (per_wave <= 4)
            return f(Int<64>{}, Int<4>{});
        if (per_wave <= 8)
            return f(Int<64>{}, Int<8>{});
    }
    if (per_four <= 1)
        return f(Int<256>{}, Int<1>{});
    if (per_four <= 2)
        return f(Int<256>{}, Int<2>{});
    if (per_four <= 4)
        return f(Int<256>{}, Int<4>{});
    if (per_four <= 8)
        return f(Int<256>{}, Int<8>{});
    return f(Int<0>{}, Int<0>{});
}

// Whether the gradients of few or very wide rows take one launch: its workgroups
// for dgamma and dbeta each pass over all rows of their columns, 5 ns a row, the
// other form pays for a second launch and for workgroups' sums. Measured, one launch
// and two (us): 301 x 1000 5.0 and 8.1, 301 x 4096 5.1 and 11.9, 600 x 1000 6.7 and
// 9.1, 1200 x 512 9.2 and 7.7, 1200 x 2048 FP32 13.9 and 17.8, 2000 x 2048 FP32 21.5
// and 19.6, 4000 x 8192 FP32 146 and 96, 2000 x 16384 77 and 76.
bool norm_direct(int rows, int cols, bool fp32) { return rows <= 800 || cols > (fp32 ? 8192 : 16384); }

// Lanes that hold a row where there are many, and the workgroups that walk them: none
// where one launch does it, whose rows may be wider than a workgroup's lanes hold. A
// lane holds eight columns of FP32 rows and of short ones, sixteen of others.
int norm_bwd_lanes(int cols, bool fp32)
{
    const int64_t lanes = ceil_div(cols, fp32 || cols <= 512 ? 8 : 16);
    return std::max(8, 1 << ceil_log2(lanes));
}
int norm_bwd_blocks(int rows, int cols, bool fp32, int cus)
{
    if (norm_direct(rows, cols, fp32))
        return 0;
    return (int)std::min<int64_t>(cus, ceil_div(rows, r::NORM_BWD_THREADS / norm_bwd_lanes(cols, fp32)));
}
template <class X, class F>
int with_bwd_rows(int cols, F &&f)
{
    constexpr bool FP32 = sizeof(X) == 4;
    typedef Int<FP32 ? 1 : 2> Vpt;
    if (cols <= 512)
        return with_lanes(cols, f);
    switch (norm_bwd_lanes(cols, FP32)) {
    case 64: return f(Int<64>{}, Vpt{});
    case 128: return f(Int<128>{}, Vpt{});
    case 256: return f(Int<256>{}, Vpt{});
    case 512: return f(Int<512>{}, Vpt{});
    default: return f(Int<1024>{}, Vpt{});
    }
}

} // namespace

extern "C" int gemm355_embedding(int tokens, int vocab, int cols, int id_type, const void *ids, int e_type, const void *E,
                                 float scale, int y_type, void *Y, void *stream)
{
    if (tokens < 0 || vocab < 0 || cols < 0 || !id_type_ok(id_type) || !type_ok(e_type) || !type_ok(y_type) ||
        !isfinite(scale))
        return GEMM355_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0)
        return GEMM355_OK;
    if (!ids || !Y || (vocab > 0 && !E))
        return GEMM355_ERR_INVALID_ARG;
    if (cols % 8 != 0 || !elements_ok(tokens, cols) || !elements_ok(vocab, cols))
        return GEMM355_ERR_UNSUPPORTED;
    const Array out[] = {{Y, size_t(tokens) * cols * size_of(y_type)}};
    const Array in[] = {{E, size_t(vocab) * cols * size_of(e_type)}, {ids, size_t(tokens) * id_size(id_type)}};
    if (any_overlap(out, 1, in, 2))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 1) || !all_aligned(in, 1) || !aligned(ids, id_size(id_type)))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    r::EmbedArgs p = {};
    p.ids = ids;
    p.e = E;
    p.y = Y;
    p.tokens = tokens;
    p.vocab = vocab;
    p.cols = cols;
    p.scale = scale;
    p.wide = id_type == GEMM355_INT64;
    const int units = cols / r::embed_width(y_type == GEMM355_FP32);
    p.lanes_log2 = std::min(6, ceil_log2(units));
    p.pieces = (int)ceil_div(units, int64_t(1) << p.lanes_log2);
    const int64_t groups = r::EMBED_THREADS >> p.lanes_log2;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // four tokens per lane where that leaves eight workgroups for every unit
    const int64_t four = ceil_div(tokens, groups * 4) * p.pieces;
    if (four >= 8 * int64_t(cus)) {
        p.items = four;
        return launch_embed<4>(p, e_type, y_type, p.items, s);
    }
    p.items = ceil_div(tokens, groups) * p.pieces;
    return launch_embed<1>(p, e_type, y_type, p.items, s);
}

extern "C" int gemm355_embedding_bwd_workspace_size(int tokens, int vocab, int cols, size_t *bytes)
{
    if (tokens < 0 || vocab < 0 || cols < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!elements_ok(tokens, cols) || !elements_ok(vocab, cols) || vocab > kMaxVocab)
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (vocab == 0 || cols == 0)
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)
        *bytes = plan_embed_bwd(tokens, vocab, cols, cus).bytes;
    return rc;
}

extern "C" int gemm355_embedding_bwd(int tokens, int vocab, int cols, int id_type, const void *ids, int y_type,
                                     const void *dY, float scale, int e_type, const void *R, void *dE, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    if (tokens < 0 || vocab < 0 || cols < 0 || !id_type_ok(id_type) || !type_ok(e_type) || !type_ok(y_type) ||
        !isfinite(scale))
        return GEMM355_ERR_INVALID_ARG;
    if (vocab == 0 || cols == 0)
        return GEMM355_OK;
    if (!dE || (workspace_bytes > 0 && !workspace) || (tokens > 0 && (!ids || !dY)))
        return GEMM355_ERR_INVALID_ARG;
    if (cols % 8 != 0 || !elements_ok(tokens, cols) || !elements_ok(vocab, cols) || vocab > kMaxVocab)
        return GEMM355_ERR_UNSUPPORTED;
    const size_t e_bytes = size_t(vocab) * cols * size_of(e_type);
    const Array out[] = {{dE, e_bytes}, {workspace, workspace_bytes}};
    // dE may be R itself: every element is read before it is written, by the same lane
    const Array in[] = {{dY, size_t(tokens) * cols * size_of(y_type)}, {R == dE ? nullptr : R, e_bytes},
                        {ids, size_t(tokens) * id_size(id_type)}};
    if (any_overlap(out, 2, in, 3))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 2) || !all_aligned(in, 2) || !aligned(ids, id_size(id_type)))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    const EmbedBwdPlan e = plan_embed_bwd(tokens, vocab, cols, cus);
    if (workspace_bytes < e.bytes)
        return GEMM355_ERR_UNSUPPORTED;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    r::EmbedBwdArgs p = {};
    p.ids = ids;
    p.dy = dY;
    p.r = R;
    p.de = dE;
    p.start = reinterpret_cast<int *>(ws);
    p.sorted = reinterpret_cast<int2 *>(ws + e.sorted_at);
    p.partial = reinterpret_cast<float *>(ws + e.partial_at);
    p.tokens = tokens;
    p.vocab = vocab;
    p.cols = cols;
    p.range = e.range;
    p.block = e.block;
    p.blocks = e.blocks;
    p.pieces = e.pieces;
    p.scale = scale;
    p.wide = id_type == GEMM355_INT64;
    p.counts = reinterpret_cast<int *>(ws + e.counts_at);
    p.total = reinterpret_cast<int *>(ws + e.total_at);
    p.bucket_start = e.shift > 0 ? reinterpret_cast<int *>(ws + e.bucket_start_at) : p.start;
    p.bucketed = e.shift > 0 ? reinterpret_cast<int2 *>(ws + e.bucketed_at) : p.sorted;
    p.shift = e.shift;
    p.buckets = e.buckets;
    p.chunks = e.chunks;
    if (e.few)
        return with_type(e_type, [&](auto te) {
            return with_type(y_type, [&](auto ty) {
                return launch_kernel(r::embed_few_kernel<decltype(te), decltype(ty)>, (unsigned)(int64_t(e.groups) * e.pieces),
                                     (unsigned)r::EMBED_THREADS, p, s);
            });
        });
    constexpr int per = r::EMBED_THREADS / 64;
    const int64_t sum_groups = std::min<int64_t>(ceil_div(int64_t(e.blocks) * e.pieces, per), 16 * int64_t(cus));
    // Rows without a token are filled beside the ordering, and those with one as well,
    // where at most a quarter have one; else beside the sums.
    const bool early = vocab / 4 >= tokens;
    const bool fills = R != dE;
    const int64_t early_groups =
        fills && early ? std::min<int64_t>(ceil_div(int64_t(vocab) * cols, 32 * r::FILL_THREADS), cus) : 0;
    const int64_t late_groups =
        fills && !early ? std::min<int64_t>(ceil_div(ceil_div(vocab, r::FILL_ROWS) * e.pieces, per), 8 * int64_t(cus)) : 0;
    p.order_groups = e.groups;
    p.sum_waves = (int)(sum_groups * per);
    return with_type(e_type, [&](auto te) {
        return with_type(y_type, [&](auto ty) {
            typedef decltype(te) TE;
            int st = GEMM355_OK;
            if (e.chunks > 0) {
                st = launch_kernel(r::embed_count_kernel<TE>, (unsigned)(e.chunks + early_groups), (unsigned)r::ORDER_THREADS, p, s);
                if (st == GEMM355_OK)
                    st = launch_kernel(r::embed_scan_kernel, (unsigned)ceil_div(e.buckets, 64), (unsigned)r::ORDER_THREADS, p, s);
                if (st == GEMM355_OK)
                    st = launch_kernel(r::embed_place_kernel, (unsigned)e.chunks, (unsigned)r::ORDER_THREADS, p, s);
                if (st == GEMM355_OK && e.shift > 0)
                    st = launch_kernel(r::embed_order_kernel<TE, true>, (unsigned)e.groups, (unsigned)r::ORDER_THREADS, p, s);
            } else {
                st = launch_kernel(r::embed_order_kernel<TE, false>, (unsigned)(e.groups + early_groups),
                                   (unsigned)r::ORDER_THREADS, p, s);
            }
            if (st != GEMM355_OK)
                return st;
            st = launch_kernel(r::embed_sums_kernel<TE, decltype(ty)>, (unsigned)(sum_groups + late_groups),
                               (unsigned)r::EMBED_THREADS, p, s);
            if (st != GEMM355_OK)
                return st;
            return launch_kernel(r::embed_join_kernel<TE>,
                                 (unsigned)std::min<int64_t>(ceil_div(e.blocks, r::JOIN_BLOCKS) * e.pieces, 16 * int64_t(cus)),
                                 (unsigned)r::JOIN_THREADS, p, s);
        });
    });
}

extern "C" int gemm355_layer_norm(int rows, int cols, int x_type, const void *X, int w_type, const void *gamma,
                                  const void *beta, float eps, void *Y, float *mean, float *rstd, void *stream)
{
    if (rows < 0 || cols < 0 || !type_ok(x_type) || !type_ok(w_type) || !isfinite(eps) || eps < 0.0f)
        return GEMM355_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0)
        return GEMM355_OK;
    if (!X || !Y)
        return GEMM355_ERR_INVALID_ARG;
    if (cols % 8 != 0 || !elements_ok(rows, cols))
        return GEMM355_ERR_UNSUPPORTED;
    const size_t n = size_t(rows) * cols, w = size_t(cols) * size_of(w_type);
    const Array out[] = {{Y, n * 2}, {mean, size_t(rows) * 4}, {rstd, size_t(rows) * 4}};
    const Array in[] = {{X, n * size_of(x_type)}, {gamma, w}, {beta, w}};
    if (any_overlap(out, 3, in, 3))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 1) || !all_aligned(in, 3) || !aligned(mean, 4) || !aligned(rstd, 4))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    r::NormArgs p = {X, gamma, beta, Y, mean, rstd, rows, cols, eps};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return with_type(x_type, [&](auto tx) {
        return with_type(w_type, [&](auto tw) {
            return with_rows(cols, rows >= 4 * cus, [&](auto lanes_c, auto vpt_c) {
                constexpr int LANES = decltype(lanes_c)::value, VPT = decltype(vpt_c)::value;
                if constexpr (LANES == 0) {
                    return launch_kernel(r::norm_wide_kernel<decltype(tx), decltype(tw)>,
                                         (unsigned)std::min<int64_t>(rows, 2 * int64_t(cus)),
                                         (unsigned)r::NORM_WIDE_THREADS, p, s);
                } else {
                    return launch_kernel(r::norm_kernel<decltype(tx), decltype(tw), LANES, VPT>,
                                         (unsigned)std::min<int64_t>(ceil_div(int64_t(rows) * LANES, r::NORM_THREADS), 8 * int64_t(cus)),
                                         (unsigned)r::NORM_THREADS, p, s);
                }
            });
        });
    });
}

extern "C" int gemm355_layer_norm_bwd_workspace_size(int rows, int cols, size_t *bytes)
{
    if (rows < 0 || cols < 0 || !bytes)
        return GEMM355_ERR_INVALID_ARG;
    if (!elements_ok(rows, cols))
        return GEMM355_ERR_UNSUPPORTED;
    *bytes = 0;
    if (rows == 0 || cols == 0 || norm_direct(rows, cols, false))
        return GEMM355_OK;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc == GEMM355_OK)   // (of the type that takes more)
        *bytes = size_t(std::max(norm_bwd_blocks(rows, cols, false, cus), norm_bwd_blocks(rows, cols, true, cus))) * 2 * cols *
                 sizeof(float);
    return rc;
}

extern "C" int gemm355_layer_norm_bwd(int rows, int cols, int x_type, const void *X, int w_type, const void *gamma,
                                      const float *mean, const float *rstd, const void *dY, const void *R, void *dX,
                                      void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes, void *stream)
{
    if (rows < 0 || cols < 0 || !type_ok(x_type) || !type_ok(w_type))
        return GEMM355_ERR_INVALID_ARG;
    const bool wants_columns = dgamma || dbeta, wants_x = dX && rows > 0;
    if (cols == 0 || (!wants_x && !wants_columns))
        return GEMM355_OK;
    if (rows > 0 && (!X || !mean || !rstd || !dY))
        return GEMM355_ERR_INVALID_ARG;
    if (workspace_bytes > 0 && !workspace)
        return GEMM355_ERR_INVALID_ARG;
    if (cols % 8 != 0 || !elements_ok(rows, cols))
        return GEMM355_ERR_UNSUPPORTED;
    const size_t n = size_t(rows) * cols, w = size_t(cols) * size_of(w_type);
    const Array out[] = {{dX, n * size_of(x_type)}, {dgamma, w}, {dbeta, w}, {workspace, workspace_bytes}};
    // dX may be R itself: every element is read before it is written, by the same lane
    const Array in[] = {{X, n * size_of(x_type)}, {dY, n * 2}, {gamma, w}, {dX == R ? nullptr : R, n * size_of(x_type)},
                        {mean, size_t(rows) * 4}, {rstd, size_t(rows) * 4}};
    if (any_overlap(out, 4, in, 6))
        return GEMM355_ERR_INVALID_ARG;
    if (!all_aligned(out, 4) || !all_aligned(in, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return GEMM355_ERR_UNSUPPORTED;
    int cus = 0;
    const int rc = compute_units(&cus);
    if (rc != GEMM355_OK)
        return rc;
    r::NormBwdArgs p = {X, gamma, mean, rstd, dY, R, wants_x ? dX : nullptr, dgamma, dbeta, static_cast<float *>(workspace),
                        rows, cols, 0, wants_columns};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool fp32 = x_type == GEMM355_FP32;
    if (norm_direct(rows, cols, fp32)) {      // (no rows: the column blocks write zeros)
        const unsigned columns = wants_columns ? (unsigned)std::min<int64_t>(ceil_div(cols, 64), kMaxBlocks) : 0u;
        return with_type(x_type, [&](auto tx) {
            return with_type(w_type, [&](auto tw) {
                auto go = [&](auto vpt_c) {
                    constexpr int VPT = decltype(vpt_c)::value;
                    p.blocks = wants_x ? (int)std::min<int64_t>(rows, (VPT ? 8 : 2) * int64_t(cus)) : 0;
                    return launch_kernel(r::norm_bwd_direct_kernel<decltype(tx), decltype(tw), VPT>,
                                         (unsigned)p.blocks + columns, (unsigned)r::norm_direct_threads<VPT>(), p, s);
                };
                return cols <= 2048 ? go(Int<1>{}) : cols <= 4096 ? go(Int<2>{}) : cols <= 8192 ? go(Int<4>{}) : go(Int<0>{});
            });
        });
    }
    p.blocks = norm_bwd_blocks(rows, cols, fp32, cus);
    if (workspace_bytes < size_t(p.blocks) * 2 * cols * sizeof(float))
        return GEMM355_ERR_UNSUPPORTED;
    return with_type(x_type, [&](auto tx) {
        return with_type(w_type, [&](auto tw) {
            typedef decltype(tw) TW;
            const int st = with_bwd_rows<decltype(tx)>(cols, [&](auto lanes_c, auto vpt_c) {
                return launch_kernel(r::norm_bwd_kernel<decltype(tx), TW, decltype(lanes_c)::value, decltype(vpt_c)::value>,
                                     (unsigned)p.blocks, (unsigned)r::NORM_BWD_THREADS, p, s);
            });
            if (st != GEMM355_OK || !wants_columns)
                return st;
            return launch_kernel(r::norm_sums_kernel<TW>, (unsigned)ceil_div(2 * int64_t(cols), r::NORM_SUM_COLS),
                                 (unsigned)r::NORM_SUM_THREADS, p, s);
        });
    });
}
