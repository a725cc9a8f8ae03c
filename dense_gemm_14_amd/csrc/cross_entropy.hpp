// cross_entropy.hpp -- softmax cross entropy over a vocabulary, and its gradient,
// without keeping the logits z = A B^T (M tokens, V rows of the vocabulary).
//
//   lse[m] = log sum exp z[m][v],  loss[m] = lse[m] - z[m][target[m]]
//   dz[m][v] = (exp(z[m][v] - lse[m]) - [v = target[m]]) dloss[m]
//   dA = dz B,  dB = dz^T A
//
// Forward: one product whose epilogue leaves, for each row and run of 64 or 128
// columns, the sum of the exponentials under a base near the largest z, and the
// target's z (dense_loss.hpp); a second kernel joins the runs. 8 bytes for every
// 128 logits go through memory.
// Backward: for a piece of the vocabulary at a time z again, with dz as its
// epilogue's result, and both products of that piece; dA's sums are kept in FP32
// between the pieces. A piece's dz, in BF16, is what the workspace has to hold.
//
// Rows that are left out (padding, prompts) cost nothing in the backward pass and in a
// forward one of more than 2^33 multiplications: the kept rows are moved together
// beforehand, and the products take their number from device memory. (Smaller forward
// products take all rows, which is less than the launch that moves them.) That also
// keeps whatever the other rows hold, infinities included, out of dB.
//
// Measured on several cards: forward of 8192 x 128000, K = 4096 in 5.98 to 6.32 ms, 1437
// to 1360 TFLOP/s (a library product of these sizes 5.85 to 6.06), bounded by the matrix
// cores at the power limit; one token 169 us, 6.2 TB/s, bounded by memory. Backward of
// 4096 x 128000, K = 4096 in 9.06 to 9.48 ms, 1422 to 1359 TFLOP/s: in a piece of 32768
// columns z and dz, dB and dA in 786, 790 and 742 us under the profiler.
//
// dz enters the products in BF16. The rows' weights dloss are taken relative to
// the largest, and that one multiplies the FP32 results: with equal weights, a
// mean's, dz is rounded as if there were none (2^-8 of a weight at most, the same
// for every element, would otherwise be in both gradients).
#pragma once

#include "dense_loss.hpp"

namespace gemm355 {
namespace dense {

constexpr int CE_THREADS = 256, CE_WAVES = CE_THREADS / 64;

struct CePrepArgs {
    const void *ids;          // the targets
    const void *a;
    const float *lse, *dloss; // backward (dloss may be NULL: ones)
    int *rows;                // number of kept rows
    int *map, *target;        // of each kept row: where it was, its target
    float *klse, *weight;     // backward: its lse, its weight relative to *scale and loss_excess(lse)
    float *scale;             // backward
    void *ka;                 // the kept rows of A, zeros behind them
    float *loss0, *lse0;      // forward: zeros for rows that are left out
    void *da;                 // backward: zeros for their gradient, or NULL
    void *dz;                 // backward: zeros behind the kept rows
    int M, V, K;
    int chunk;                // rows per workgroup
    int dz_pitch;
    int splits[2], min_steps[2];   // backward: of the products over the rows
    bool wide;
};

// Rows of dz and A that a product over them reads: whole K steps for a kernel
// that needs some (min_steps > 0), else those that there are.
__host__ __device__ inline int64_t ce_depth(int64_t rows, int splits, int min_steps)
{
    if (min_steps == 0)
        return rows;
    const int64_t steps = ((rows + 63) / 64 + splits - 1) / splits;
    return 64 * splits * (steps > min_steps ? steps : min_steps);
}

template <bool BWD>
__global__ __launch_bounds__(CE_THREADS) void ce_prep_kernel(CePrepArgs p)
{
    __shared__ int part[3][CE_WAVES], place[CE_THREADS];
    __shared__ float top[CE_WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t r0 = (int64_t)blockIdx.x * p.chunk, r1 = min((int64_t)p.M, r0 + p.chunk);

    // every workgroup looks at all targets, and so waits for no other
    int before = 0, kept = 0;
    float largest = 0.0f;
    constexpr int AHEAD = 4;
    for (int64_t m0 = tid; m0 < p.M; m0 += AHEAD * CE_THREADS) {
        int id[AHEAD];
        float w[AHEAD] = {};
        rows::ids_at<AHEAD>(p.ids, p.wide, m0, CE_THREADS, p.M, p.V, id);
        if (BWD && p.dloss)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                w[k] = p.dloss[min(m0 + k * CE_THREADS, (int64_t)p.M - 1)];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            before += id[k] >= 0 && m0 + k * CE_THREADS < r0;
            kept += id[k] >= 0;
            largest = id[k] >= 0 && fabsf(w[k]) < __builtin_inff() ? fmaxf(largest, fabsf(w[k])) : largest;
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        before += __shfl_xor(before, d);
        kept += __shfl_xor(kept, d);
        if constexpr (BWD)
            largest = fmaxf(largest, __shfl_xor(largest, d));
    }
    if (lane == 0) {
        part[0][wave] = before;
        part[1][wave] = kept;
        top[wave] = largest;
    }
    __syncthreads();
    before = kept = 0;
    largest = 0.0f;
#pragma unroll
    for (int w = 0; w < CE_WAVES; ++w) {
        before += part[0][w];
        kept += part[1][w];
        largest = fmaxf(largest, top[w]);
    }
    const float scale = BWD && p.dloss && largest > 0.0f ? largest : 1.0f;
    if (blockIdx.x == 0 && tid == 0) {
        *p.rows = kept;
        if constexpr (BWD)
            *p.scale = scale;
    }

    const uint16_t *a = static_cast<const uint16_t *>(p.a);
    uint16_t *ka = static_cast<uint16_t *>(p.ka);
    for (int64_t first = r0; first < r1; first += CE_THREADS) {
        const int64_t m = first + tid;
        const int target = m < r1 ? rows::id_at(p.ids, p.wide, (size_t)m, p.V) : -1;
        const unsigned long long in = __ballot(target >= 0);
        if (lane == 0)
            part[2][wave] = __popcll(in);
        __syncthreads();
        int at = before + __popcll(in & ((1ull << lane) - 1));
#pragma unroll
        for (int w = 0; w < CE_WAVES; ++w) {
            at += w < wave ? part[2][w] : 0;
            before += part[2][w];
        }
        place[tid] = target >= 0 ? at : -1;
        if (target >= 0) {
            p.map[at] = (int)m;
            p.target[at] = target;
            if constexpr (BWD) {
                const float lse = p.lse[m], w = p.dloss ? p.dloss[m] / scale : 1.0f;
                p.klse[at] = lse;
                p.weight[at] = w / loss_excess(lse);
            }
        } else if (!BWD && m < r1) {
            p.loss0[m] = 0.0f;
            p.lse0[m] = 0.0f;
        }
        __syncthreads();
        for (int i = wave; i < CE_THREADS && first + i < r1; i += CE_WAVES) {
            const int to = __builtin_amdgcn_readfirstlane(place[i]);
            if (to >= 0) {
                const uint16_t *from = a + (size_t)(first + i) * (size_t)p.K;
#pragma unroll 8
                for (int c = 8 * lane; c < p.K; c += 512)
                    *reinterpret_cast<u32x4 *>(ka + (size_t)to * (size_t)p.K + (size_t)c) = *reinterpret_cast<const u32x4 *>(from + c);
            } else if (BWD && p.da) {
                for (int c = 8 * lane; c < p.K; c += 512)
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.da) + (size_t)(first + i) * (size_t)p.K + (size_t)c) = u32x4{};
            }
        }
    }
    if constexpr (BWD) {
        // zeros behind the kept rows, up to the last step of the products over them
        const int64_t depth = max(ce_depth(kept, p.splits[0], p.min_steps[0]), ce_depth(kept, p.splits[1], p.min_steps[1]));
        for (int64_t row = kept + (int64_t)blockIdx.x * CE_WAVES + wave; row < depth; row += (int64_t)gridDim.x * CE_WAVES) {
            for (int c = 8 * lane; c < p.K; c += 512)
                *reinterpret_cast<u32x4 *>(ka + (size_t)row * (size_t)p.K + (size_t)c) = u32x4{};
            for (int c = 8 * lane; c < p.dz_pitch; c += 512)
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.dz) + (size_t)row * (size_t)p.dz_pitch + (size_t)c) = u32x4{};
        }
    }
}

// Joins the runs of ROWS rows: as many lanes side by side, the others share out
// the runs.
struct CeJoinArgs {
    const f32x2 *stats;      // [run][stride]: as loss_stat has them
    const float *picked;
    const int *rows, *map;   // or NULL: M rows, in place, whose targets say which are left out
    const void *ids;
    float *loss, *lse;
    int M, V, stride, runs;
    bool wide;
};

struct CeSum {
    float base, sum;         // a sum of powers of two under a base that is a whole number, -inf and 0 if there is none;
                             // from LOSS_FAR on the largest logit and minus the number of those that are the same
    float rest;              // what was not finite
};
__device__ inline CeSum ce_join_near(const CeSum &a, const CeSum &b)
{
    const float base = fmaxf(a.base, b.base), ref = __builtin_isinf(base) ? 0.0f : base;
    return CeSum{base, a.sum * __builtin_amdgcn_exp2f(a.base - ref) + b.sum * __builtin_amdgcn_exp2f(b.base - ref), a.rest + b.rest};
}
// Where one is from LOSS_FAR on: logits that large outweigh all that are smaller, and
// nothing where there is any that is larger (e^-64 and less). (0 times the sums: NaN stays.)
__device__ inline CeSum ce_join_far(const CeSum &a, const CeSum &b)
{
    const float ka = a.sum < 0.0f || __builtin_isinf(a.base) ? a.base : 0.0f;
    const float kb = b.sum < 0.0f || __builtin_isinf(b.base) ? b.base : 0.0f;
    return CeSum{ka >= kb ? a.base : b.base, (ka >= kb ? a.sum : 0.0f) + (kb >= ka ? b.sum : 0.0f),
                 a.rest + b.rest + 0.0f * (a.sum + b.sum)};
}
__device__ inline CeSum ce_join(const CeSum &a, const CeSum &b)
{
    return a.sum < 0.0f || b.sum < 0.0f ? ce_join_far(a, b) : ce_join_near(a, b);
}
// join(ce_join) where some lane of the wave is `far`, else join(ce_join_near): one
// branch for several joins.
template <class F>
__device__ inline void with_join(bool far, F &&join)
{
    if (__ballot(far) != 0)
        join([](const CeSum &a, const CeSum &b) { return ce_join(a, b); });
    else
        join([](const CeSum &a, const CeSum &b) { return ce_join_near(a, b); });
}

template <int ROWS>
__global__ __launch_bounds__(CE_THREADS) void ce_join_kernel(CeJoinArgs p)
{
    constexpr int LANES = CE_THREADS / ROWS, AHEAD = 8;
    __shared__ CeSum part[CE_WAVES][ROWS];
    const int tx = threadIdx.x % ROWS, ty = threadIdx.x / ROWS;
    const int M = p.rows ? __builtin_amdgcn_readfirstlane(*p.rows) : p.M;
    const int m = (int)blockIdx.x * ROWS + tx;
    CeSum s = {-__builtin_inff(), 0.0f, 0.0f};
    if (m < M)
        for (int i0 = ty; i0 < p.runs; i0 += AHEAD * LANES) {
            f32x2 t[AHEAD];
            float base = -__builtin_inff();
            bool far = s.sum < 0.0f;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                t[k] = p.stats[(size_t)min(i0 + k * LANES, p.runs - 1) * (size_t)p.stride + (size_t)m];
                base = fmaxf(base, t[k][0]);
                far |= t[k][1] < 0.0f;
            }
            if (far) {      // one by one
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
                    if (i0 + k * LANES < p.runs)
                        s = ce_join(s, __builtin_isinf(t[k][0]) ? CeSum{t[k][0], 0.0f, t[k][1]} : CeSum{t[k][0], t[k][1], 0.0f});
                continue;
            }
            CeSum x = {base, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i0 + k * LANES < p.runs) {
                    const bool finite = !__builtin_isinf(t[k][0]);
                    x.sum += finite ? t[k][1] * __builtin_amdgcn_exp2f(t[k][0] - base) : 0.0f;
                    x.rest += finite ? 0.0f : t[k][1];
                }
            s = ce_join_near(s, x);
        }
    // the lanes of a row within a wave, then the waves
    with_join(s.sum < 0.0f, [&](auto join) {
#pragma unroll
        for (int d = ROWS; d < 64; d *= 2)
            s = join(s, CeSum{__shfl_xor(s.base, d), __shfl_xor(s.sum, d), __shfl_xor(s.rest, d)});
    });
    if ((threadIdx.x & 63) < ROWS)
        part[threadIdx.x >> 6][tx] = s;
    __syncthreads();
    bool far = false;
#pragma unroll
    for (int w = 0; w < CE_WAVES; ++w)
        far |= part[w][tx].sum < 0.0f;
    with_join(far, [&](auto join) {
#pragma unroll
        for (int w = 0; w < CE_WAVES; ++w)
            s = w == 0 ? part[0][tx] : join(s, part[w][tx]);
    });
    if (ty == 0 && m < M) {
        // in 64 bits: rounded to 32 it would be the largest error of all. Divided by the
        // log2(e) that the logits were multiplied by, not multiplied by log(2): rounded, that
        // is 2^-26 off.
        const double base = __builtin_isinf(s.base) ? 0.0 : s.sum < 0.0f ? (double)s.base : (double)s.base * (1.0 / (double)LOG2E);
        const float rest = logf(fabsf(s.sum) + s.rest);
        const int row = p.map ? p.map[m] : m;
        const bool out = !p.map && rows::id_at(p.ids, p.wide, (size_t)m, p.V) < 0;
        p.lse[row] = out ? 0.0f : (float)(base + rest);
        p.loss[row] = out ? 0.0f : (float)(base - p.picked[m] + rest);
    }
}

} // namespace dense
} // namespace gemm355
