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
#include "dense_plan.hpp"
#include "dense_grad.hpp"
#include "newton_schulz.hpp"

namespace {

using namespace gemm355::host;
// ---- argument checks -------------------------------------------------------

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
        const int st = launch_kernel(d::dense_bias_kernel<d::BIAS_THREADS>, (unsigned)bias_blocks, (unsigned)d::BIAS_THREADS, q, s);
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
