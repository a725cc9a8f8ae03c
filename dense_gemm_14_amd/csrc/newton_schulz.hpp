// newton_schulz.hpp -- the start of a Newton-Schulz orthogonalisation: each
// matrix of a batch divided by its Frobenius norm, into scaled FP16.
//
// The sum of squares is taken in FP64, so no gradient is too small or too
// large for it, in two passes (a partial sum per workgroup, added in order by
// every workgroup of the second pass): the result does not depend on timing.
//
// FP16, not BF16, carries the iterates: both have the same matrix rate, the
// singular values stay below about 1.3, and three more bits keep five steps'
// rounding at 1.5e-3 of the result where BF16 iterates lose 1e-2. X is held
// times 2^12: that puts the elements, about |G| / (|G| + eps) / sqrt(rows cols)
// at the start, into FP16's normal range also where eps outweighs the norm (down
// to a share of 2^-26 sqrt(rows cols) of it; with a scale of sqrt(min(rows,
// cols)) a share of 1e-4 of 256 x 1032 lost 6e-3 and of 1e-5 6e-2), and X reaches
// FP16's largest value no earlier than X X^T does.
//
// Bound by memory: 4096 x 8192 of FP32 are read in 28 us (4.8 TB/s, what a copy
// reaches) and read again and written in 30, of 1970 to 2110 for all five steps.
#pragma once

#include "dense_common.hpp"

namespace gemm355 {
namespace dense {

constexpr int NS_THREADS = 256;
constexpr int NS_BLOCKS = 1024;  // workgroups (partial sums) per matrix at most

struct NormArgs {
    const void *g;       // batch matrices of `elements` each
    double *partial;     // [batch][blocks]
    uint16_t *x;         // FP16 out
    int64_t elements;    // per matrix, a multiple of 8
    int blocks;          // workgroups per matrix
    double scale, eps;   // x = g scale / (norm + eps)
};

template <bool FP32>
__device__ inline void load8(const void *g, int64_t at, float (&x)[8])
{
    if constexpr (FP32) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(g) + at);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    } else {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(g) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

// Sum over the workgroup, in a fixed order.
__device__ inline double block_sum(double v)
{
    __shared__ double part[NS_THREADS / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

template <bool FP32>
__global__ __launch_bounds__(NS_THREADS) void ns_norm_kernel(NormArgs p)
{
    const int b = (int)blockIdx.x / p.blocks, k = (int)blockIdx.x % p.blocks;
    double s = 0.0;
    for (int64_t at = ((int64_t)k * NS_THREADS + threadIdx.x) * 8; at < p.elements; at += (int64_t)p.blocks * NS_THREADS * 8) {
        float x[8];
        load8<FP32>(p.g, (int64_t)b * p.elements + at, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s += (double)x[e] * (double)x[e];
    }
    s = block_sum(s);
    if (threadIdx.x == 0)
        p.partial[(size_t)b * p.blocks + k] = s;
}

template <bool FP32>
__global__ __launch_bounds__(NS_THREADS) void ns_scale_kernel(NormArgs p)
{
    const int b = (int)blockIdx.x / p.blocks, k = (int)blockIdx.x % p.blocks;
    double mine = 0.0;
    for (int i = threadIdx.x; i < p.blocks; i += NS_THREADS)
        mine += p.partial[(size_t)b * p.blocks + i];
    const double norm2 = block_sum(mine);
    const double below = sqrt(norm2) + p.eps;
    const double f = below > 0.0 ? p.scale / below : 0.0;   // a zero matrix stays zero
    for (int64_t at = ((int64_t)k * NS_THREADS + threadIdx.x) * 8; at < p.elements; at += (int64_t)p.blocks * NS_THREADS * 8) {
        float x[8];
        load8<FP32>(p.g, (int64_t)b * p.elements + at, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = (float)((double)x[e] * f);
        *reinterpret_cast<u32x4 *>(p.x + (size_t)b * (size_t)p.elements + (size_t)at) =
            u32x4{pack2<_Float16>(x[0], x[1]), pack2<_Float16>(x[2], x[3]), pack2<_Float16>(x[4], x[5]),
                  pack2<_Float16>(x[6], x[7])};
    }
}

} // namespace dense
} // namespace gemm355
