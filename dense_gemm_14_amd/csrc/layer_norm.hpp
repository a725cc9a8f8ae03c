// layer_norm.hpp -- layer norm and its gradients.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd gamma + beta
//   with u = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum g / n - u sum (g u) / n) + r
//   dgamma = sum over rows of dy u,  dbeta = sum over rows of dy
//
// Bound by memory, so one pass over it: a row is held in registers between its sums
// and its results, by one wave (up to 4096 columns, where there are rows for every
// wave of the card) or four (up to 16384), by 8, 16 or 32 lanes up to 64, 128 or 256
// columns (heads: 262144 x 128 BF16 22.5 us, 64.5 with a wave for each row; gradients
// 36 and 105); wider rows are read again, by then from the caches (1024 x 32768 BF16 in 34
// to 39 us, gradients 77 to 83). Measured, BF16: 8192 x 4096 in 24.2 us, 5.5 TB/s (29.2
// with so many arrays in turn that the last-level cache holds none), its gradients with a
// residual's in 57.5, 4.7 TB/s, of which 8 the second launch; FP32 rows and weights 43
// and 92; one row of 4096 2.4 us on the card, 4.9 with its call.
// The variance is that of the differences from the mean, not of the squares, so no
// large mean cancels in it; four waves join their means and sums of squared
// differences m2 by
//   m2 = m2a + m2b + (mean_a - mean_b)^2 n_a n_b / (n_a + n_b).
// All statistics and sums are FP32; a result is rounded once, as it is stored.
#pragma once

#include "vector8.hpp"

namespace gemm355 {
namespace rows {

constexpr int NORM_THREADS = 256;
constexpr int NORM_WIDE_THREADS = 1024;

struct NormArgs {
    const void *x;
    const void *gamma, *beta;   // or NULL: ones, zeros
    void *y;                    // BF16
    float *mean, *rstd;         // or NULL
    int rows, cols;
    float eps;
};

// The statistics of part of a row; of no values where n is 0, which joins as if it had
// the other's mean: the square of a distance to 0 may be beyond FP32. (Means that are a
// distance without end apart are added: infinite, or NaN, as the sum of the row is.)
struct Moments {
    float n, mean, m2;
};
__device__ inline Moments join(const Moments &a, const Moments &b)
{
    const float n = a.n + b.n, d = b.n > 0.0f ? b.mean - a.mean : 0.0f, part = n > 0.0f ? b.n / n : 0.0f;
    return Moments{n, fabsf(d) < __builtin_inff() ? a.mean + d * part : a.mean + b.mean, a.m2 + b.m2 + d * d * a.n * part};
}

// A row in the registers of LANES lanes, of which there are 8, 16 or 32 (a wave
// then has several rows), a wave's or several waves': lane `i` of them holds the
// eight columns 8 (i + LANES v), v < VPT.
template <int LANES>
__device__ inline int norm_col(int i, int v)
{
    return 8 * (i + LANES * v);
}
// Sum over a row's lanes of this wave, the same in each of them. (Fewer than 64:
// each step adds what the lanes at the other end of a pair, four, eight and sixteen hold.)
template <int LANES>
__device__ inline float lanes_sum(float x)
{
    if constexpr (LANES >= 64)
        return wave_sum(x);
    x += dpp_or_zero<0xB1, 0xF>(x);    // lanes 1 0 3 2 of four
    x += dpp_or_zero<0x4E, 0xF>(x);    // 2 3 0 1
    x += dpp_or_zero<0x141, 0xF>(x);   // eight, mirrored
    if constexpr (LANES > 8)
        x += dpp_or_zero<0x140, 0xF>(x);   // sixteen, mirrored
    if constexpr (LANES > 16)
        x += __shfl_xor(x, 16);
    return x;
}

template <class X, class W, int LANES, int VPT>
__global__ __launch_bounds__(NORM_THREADS) void norm_kernel(NormArgs p)
{
    constexpr int GROUPS = NORM_THREADS / LANES, WAVES = (LANES + 63) / 64;   // rows at a time; waves of one
    __shared__ Moments part[2][4];
    const int group = (int)threadIdx.x / LANES, lane = (int)threadIdx.x % LANES;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const float n = (float)p.cols;
    Raw8<W> gamma[VPT], beta[VPT];
    float own = 0.0f;     // columns of this wave
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = norm_col<LANES>(lane, v);
        gamma[v].fill(1.0f);
        beta[v].fill(0.0f);
        if (c < p.cols && p.gamma)
            gamma[v].load(p.gamma, c);
        if (c < p.cols && p.beta)
            beta[v].load(p.beta, c);
        own += (float)min(8 * min(LANES, 64), max(0, p.cols - norm_col<LANES>(lane & ~63, v)));
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * GROUPS + group; row - group < p.rows; row += (int64_t)gridDim.x * GROUPS) {
        const size_t base = (size_t)row * (size_t)p.cols;
        const bool in = row < p.rows;
        Raw8<X> x[VPT];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = norm_col<LANES>(lane, v);
            x[v].fill(0.0f);
            if (in && c < p.cols)
                x[v].load(p.x, base + c);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += x[v].get(e);
        Moments m = {own, own > 0.0f ? lanes_sum<LANES>(s) / own : 0.0f, 0.0f};
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (norm_col<LANES>(lane, v) < p.cols)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = x[v].get(e) - m.mean;
                    s += d * d;
                }
        m.m2 = lanes_sum<LANES>(s);
        if constexpr (WAVES > 1) {
            // (two sets in turn: a wave may be a row ahead of one that still reads)
            if ((threadIdx.x & 63) == 0)
                part[turn][wave] = m;
            __syncthreads();
            m = join(join(part[turn][0], part[turn][1]), join(part[turn][2], part[turn][3]));
            turn ^= 1;
        }
        const float rstd = 1.0f / sqrtf(m.m2 / n + p.eps);
        if (!in)
            continue;
        if (lane == 0) {
            if (p.mean)
                p.mean[row] = m.mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = norm_col<LANES>(lane, v);
            if (c < p.cols) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = (x[v].get(e) - m.mean) * rstd * gamma[v].get(e) + beta[v].get(e);
                Raw8<__bf16> out;
                out.set(y);
                out.store(p.y, base + c);
            }
        }
    }
}

// Sum over a workgroup of sixteen waves, the same in every thread.
__device__ inline float wide_sum(float x, float *part)
{
    x = wave_sum(x);
    __syncthreads();   // (the last sum's readers are done)
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < NORM_WIDE_THREADS / 64; ++i)
        x += part[i];
    return x;
}

// Rows of any width, a workgroup each, read three times.
template <class X, class W>
__global__ __launch_bounds__(NORM_WIDE_THREADS) void norm_wide_kernel(NormArgs p)
{
    __shared__ float part[NORM_WIDE_THREADS / 64];
    const float n = (float)p.cols;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const size_t base = (size_t)row * (size_t)p.cols;
        auto each = [&](auto &&f) {
            for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8 * NORM_WIDE_THREADS) {
                Raw8<X> x;
                x.load(p.x, base + c);
                f(c, x);
            }
        };
        float s = 0.0f;
        each([&](int64_t, const Raw8<X> &x) {
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t += x.get(e);
            s += t;
        });
        const float mean = wide_sum(s, part) / n;
        s = 0.0f;
        each([&](int64_t, const Raw8<X> &x) {
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = x.get(e) - mean;
                t += d * d;
            }
            s += t;
        });
        const float rstd = 1.0f / sqrtf(wide_sum(s, part) / n + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
        each([&](int64_t c, const Raw8<X> &x) {
            Raw8<W> gamma, beta;
            gamma.fill(1.0f);
            beta.fill(0.0f);
            if (p.gamma)
                gamma.load(p.gamma, c);
            if (p.beta)
                beta.load(p.beta, c);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = (x.get(e) - mean) * rstd * gamma.get(e) + beta.get(e);
            Raw8<__bf16> out;
            out.set(y);
            out.store(p.y, base + c);
        });
    }
}

// ---- gradients -----------------------------------------------------------------

struct NormBwdArgs {
    const void *x;
    const void *gamma;              // or NULL: ones
    const float *mean, *rstd;
    const void *dy;                 // BF16
    const void *r;                  // or NULL: zeros; may be dx itself
    void *dx;                       // or NULL
    void *dgamma, *dbeta;           // or NULL
    float *sums;                    // norm_bwd_kernel: [blocks][2][cols] column sums
    int rows, cols;
    int blocks;                     // norm_bwd_kernel: workgroups; norm_bwd_direct_kernel: those of dX
    bool wants_columns;             // dgamma or dbeta
};

// One row of dX by the LANES lanes that hold it, and (COLUMNS) its terms added
// to their columns' sums; exchange(a, b) joins the two sums of the lanes.
template <class X, class W, int LANES, int VPT, bool COLUMNS, class Exchange>
__device__ inline void norm_bwd_row(const NormBwdArgs &p, int64_t row, bool in, int lane, Raw8<W> (&gamma)[VPT],
                                    float (&dg)[COLUMNS ? VPT : 1][8], float (&db)[COLUMNS ? VPT : 1][8],
                                    Exchange &&exchange)
{
    const size_t base = (size_t)row * (size_t)p.cols;
    Raw8<X> x[VPT];
    Raw8<__bf16> dy[VPT];
    float mean = 0.0f, rstd = 0.0f;
    if (in) {
        mean = p.mean[row];
        rstd = p.rstd[row];
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = norm_col<LANES>(lane, v);
        x[v].fill(0.0f);
        dy[v].fill(0.0f);
        if (in && c < p.cols) {
            x[v].load(p.x, base + c);
            dy[v].load(p.dy, base + c);
        }
    }
    float sg = 0.0f, su = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        // (columns past the last have no part in it: dy is 0 there, but the mean's
        // distance from 0 may be beyond FP32)
        if (norm_col<LANES>(lane, v) < p.cols) {
            float tg = 0.0f, tu = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = dy[v].get(e), u = (x[v].get(e) - mean) * rstd, g = d * gamma[v].get(e);
                if constexpr (COLUMNS) {
                    dg[v][e] += d * u;
                    db[v][e] += d;
                }
                tg += g;
                tu += g * u;
            }
            sg += tg;
            su += tu;
        }
        // unpacked again below: kept, the values would take the registers of
        // a row more
        x[v].hold();
        dy[v].hold();
        gamma[v].hold();
    }
    if (!p.dx)
        return;
    exchange(sg, su);
    if (!in)
        return;
    sg /= (float)p.cols;
    su /= (float)p.cols;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = norm_col<LANES>(lane, v);
        if (c < p.cols) {
            Raw8<X> r;
            r.fill(0.0f);
            if (p.r)
                r.load(p.r, base + c);
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = (x[v].get(e) - mean) * rstd;
                dx[e] = rstd * (dy[v].get(e) * gamma[v].get(e) - sg - u * su) + r.get(e);
            }
            Raw8<X> out;
            out.set(dx);
            out.store(p.dx, base + c);
        }
    }
}

template <class W, int LANES, int VPT>
__device__ inline void norm_gamma(const NormBwdArgs &p, int lane, Raw8<W> (&gamma)[VPT])
{
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        gamma[v].fill(1.0f);
        if (norm_col<LANES>(lane, v) < p.cols && p.gamma)
            gamma[v].load(p.gamma, norm_col<LANES>(lane, v));
    }
}

// Joins the sums of the lanes that hold a row (two sets in turn, as above).
template <int LANES>
__device__ inline void norm_exchange(float &a, float &b, f32x2 *part, int &turn, int wave)
{
    constexpr int WAVES = LANES / 64;
    a = lanes_sum<LANES>(a);
    b = lanes_sum<LANES>(b);
    if constexpr (WAVES > 1) {
        f32x2 *mine = part + (wave / WAVES * 2 + turn) * WAVES;
        if ((threadIdx.x & 63) == 0)
            mine[wave % WAVES] = f32x2{a, b};
        __syncthreads();
        f32x2 t = mine[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            t += mine[w];
        a = t[0];
        b = t[1];
        turn ^= 1;
    }
}

// Many rows: a workgroup walks rows (sixteen waves: 128 rows of up to
// 64 columns down to one at a time), its lanes keep the sums of their columns, the workgroup's rows are joined
// through LDS and leave one row of column sums each for dgamma and dbeta. One
// workgroup per unit, so that those rows are few; sixteen waves, each with so few
// columns that 128 registers hold them, so that loads are always in flight (8192 x
// 4096: 57.5 us; with eight waves and up to 256 registers 67).
constexpr int NORM_BWD_THREADS = 1024;
template <class X, class W, int LANES, int VPT>
__global__ __launch_bounds__(NORM_BWD_THREADS) void norm_bwd_kernel(NormBwdArgs p)
{
    constexpr int GROUPS = NORM_BWD_THREADS / LANES;
    __shared__ f32x2 part[2 * NORM_BWD_THREADS / 64];
    __shared__ float join[GROUPS][LANES * 16];
    const int group = (int)threadIdx.x / LANES, lane = (int)threadIdx.x % LANES;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    Raw8<W> gamma[VPT];
    norm_gamma<W, LANES, VPT>(p, lane, gamma);
    float dg[VPT][8] = {}, db[VPT][8] = {};
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * GROUPS + group; row - group < p.rows; row += (int64_t)p.blocks * GROUPS)
        norm_bwd_row<X, W, LANES, VPT, true>(p, row, row < p.rows, lane, gamma, dg, db,
                                             [&](float &a, float &b) { norm_exchange<LANES>(a, b, part, turn, wave); });
    if (!p.wants_columns)
        return;
    float *out = p.sums + (size_t)blockIdx.x * 2 * (size_t)p.cols;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        __syncthreads();
        // [which][element][lane]: neighbouring lanes, neighbouring banks
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            join[group][e * LANES + lane] = dg[v][e];
            join[group][(8 + e) * LANES + lane] = db[v][e];
        }
        __syncthreads();
        for (int i = (int)threadIdx.x; i < 16 * LANES; i += NORM_BWD_THREADS) {
            float t = 0.0f;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
                t += join[g][i];
            const int which = i / (8 * LANES), e = i / LANES & 7, l = i % LANES;
            const int c = norm_col<LANES>(l, v) + e;
            if (c < p.cols)
                out[(size_t)which * p.cols + c] = t;
        }
    }
}

// Adds the workgroups' column sums in order: 32 columns per workgroup.
constexpr int NORM_SUM_THREADS = 1024, NORM_SUM_COLS = 32, NORM_SUM_LANES = NORM_SUM_THREADS / NORM_SUM_COLS;
template <class W>
__global__ __launch_bounds__(NORM_SUM_THREADS) void norm_sums_kernel(NormBwdArgs p)
{
    __shared__ float part[NORM_SUM_LANES][NORM_SUM_COLS];
    const int tx = threadIdx.x % NORM_SUM_COLS, ty = threadIdx.x / NORM_SUM_COLS;
    const int64_t c = (int64_t)blockIdx.x * NORM_SUM_COLS + tx, cols = 2 * (int64_t)p.cols;
    float t = 0.0f;
    if (c < cols)
#pragma unroll 4
        for (int b = ty; b < p.blocks; b += NORM_SUM_LANES)
            t += p.sums[(size_t)b * (size_t)cols + (size_t)c];
    part[ty][tx] = t;
    __syncthreads();
    if (ty == 0 && c < cols) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < NORM_SUM_LANES; ++i)
            t += part[i][tx];
        const bool second = c >= p.cols;
        void *out = second ? p.dbeta : p.dgamma;
        const size_t at = (size_t)(second ? c - p.cols : c);
        if (out) {
            if constexpr (sizeof(W) == 2)
                static_cast<uint16_t *>(out)[at] = (uint16_t)pack_bf16(t, 0.0f);
            else
                static_cast<float *>(out)[at] = t;
        }
    }
}

// Few rows or very wide ones: dX as above (VPT > 0: held by four waves; 0: read
// twice by sixteen), and beside it, in the same launch, workgroups that pass
// over 64 columns of every row for dgamma and dbeta. X and dY are read a second
// time there, but no sums go through memory and no second launch waits.
template <int VPT>
constexpr int norm_direct_threads() { return VPT ? 256 : NORM_WIDE_THREADS; }

template <class X, class W, int THREADS>
__device__ inline void norm_columns(const NormBwdArgs &p, int64_t block, float (*part)[2][65])
{
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int64_t c = block * 64 + 8 * tx;
    float dg[8] = {}, db[8] = {};
    if (c < p.cols)
#pragma unroll 4
        for (int row = ty; row < p.rows; row += THREADS / 8) {
            Raw8<X> x;
            Raw8<__bf16> dy;
            x.load(p.x, (size_t)row * (size_t)p.cols + (size_t)c);
            dy.load(p.dy, (size_t)row * (size_t)p.cols + (size_t)c);
            const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dg[e] += dy.get(e) * ((x.get(e) - mean) * rstd);
                db[e] += dy.get(e);
            }
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        part[ty][0][8 * tx + e] = dg[e];
        part[ty][1][8 * tx + e] = db[e];
    }
    __syncthreads();
    const int i = threadIdx.x & 63, which = (threadIdx.x >> 6) & 1;
    void *out = which ? p.dbeta : p.dgamma;
    const int64_t col = block * 64 + i;
    if (threadIdx.x < 128 && col < p.cols && out) {
        float t = 0.0f;
        for (int r = 0; r < THREADS / 8; ++r)
            t += part[r][which][i];
        if constexpr (sizeof(W) == 2)
            static_cast<uint16_t *>(out)[col] = (uint16_t)pack_bf16(t, 0.0f);
        else
            static_cast<float *>(out)[col] = t;
    }
}

template <class X, class W, int VPT>
__global__ __launch_bounds__(norm_direct_threads<VPT>()) void norm_bwd_direct_kernel(NormBwdArgs p)
{
    constexpr int THREADS = norm_direct_threads<VPT>();
    __shared__ float part[THREADS / 8][2][65];
    if ((int)blockIdx.x >= p.blocks) {
        for (int64_t block = (int64_t)blockIdx.x - p.blocks; block * 64 < p.cols; block += (int64_t)gridDim.x - p.blocks) {
            norm_columns<X, W, THREADS>(p, block, part);
            __syncthreads();
        }
        return;
    }
    if constexpr (VPT > 0) {
        const int lane = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        Raw8<W> gamma[VPT];
        norm_gamma<W, 256, VPT>(p, lane, gamma);
        f32x2 *xch = reinterpret_cast<f32x2 *>(part);
        int turn = 0;
        float none[1][8];
        for (int64_t row = blockIdx.x; row < p.rows; row += p.blocks)
            norm_bwd_row<X, W, 256, VPT, false>(p, row, true, lane, gamma, none, none,
                                              [&](float &a, float &b) { norm_exchange<256>(a, b, xch, turn, wave); });
    } else {
        float *sums = &part[0][0][0];
        for (int64_t row = blockIdx.x; row < p.rows; row += p.blocks) {
            const size_t base = (size_t)row * (size_t)p.cols;
            const float mean = p.mean[row], rstd = p.rstd[row], n = (float)p.cols;
            auto each = [&](auto &&f) {
                for (int64_t c = 8 * (int64_t)threadIdx.x; c < p.cols; c += 8 * THREADS) {
                    Raw8<X> x;
                    Raw8<__bf16> dy;
                    Raw8<W> gamma;
                    gamma.fill(1.0f);
                    x.load(p.x, base + c);
                    dy.load(p.dy, base + c);
                    if (p.gamma)
                        gamma.load(p.gamma, c);
                    float u[8], g[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u[e] = (x.get(e) - mean) * rstd;
                        g[e] = dy.get(e) * gamma.get(e);
                    }
                    f(c, u, g);
                }
            };
            float sg = 0.0f, su = 0.0f;
            each([&](int64_t, const float (&u)[8], const float (&g)[8]) {
                float tg = 0.0f, tu = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    tg += g[e];
                    tu += g[e] * u[e];
                }
                sg += tg;
                su += tu;
            });
            sg = wide_sum(sg, sums) / n;
            su = wide_sum(su, sums) / n;
            each([&](int64_t c, const float (&u)[8], const float (&g)[8]) {
                Raw8<X> r;
                r.fill(0.0f);
                if (p.r)
                    r.load(p.r, base + c);
                float dx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dx[e] = rstd * (g[e] - sg - u[e] * su) + r.get(e);
                Raw8<X> out;
                out.set(dx);
                out.store(p.dx, base + c);
            });
        }
    }
}

} // namespace rows
} // namespace gemm355
