// dense_grad.hpp -- the elementwise part of the dense layers' gradients: the
// gradient of the pre-activations and the column sums that the bias gets.
//
//   linear  dZ = dC act'(Z)
//   gated   dZ_gate = dC Z_up act'(Z_gate),  dZ_up = dC act(Z_gate)
//   dbias[n] = sum over rows of dZ[m][n], from the FP32 values before they are
//              rounded to BF16
//
// One pass over the data, bound by memory: 16 bytes per lane and access, 32
// lanes side by side (512 contiguous bytes of a row), 8 rows at a time. A
// workgroup walks a block of rows and leaves one row of FP32 column sums; a
// second kernel adds those rows in order, so the sums do not depend on timing.
// Measured: 4096 x 8192 in 40 to 45 us, 4.5 to 5.0 TB/s, gated (4096 x 16384
// pre-activations) in 63 us, 5.3 TB/s; a copy reaches 4.8. It is a pass of its own
// because both products read dZ, a tile of it as often as there are tiles beside
// it: recomputing it there would read Z and dC as often and take the activation's
// instructions between the matrix ones.
#pragma once

#include "dense_common.hpp"

namespace gemm355 {
namespace dense {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_COLS = 256;    // columns per workgroup
constexpr int GRAD_LANES = 8;     // rows side by side

struct GradArgs {
    const uint16_t *z;    // M x N (gated: M x 2 N) BF16
    const uint16_t *dc;   // M x N
    uint16_t *dz;         // M x N (gated: M x 2 N)
    float *sums;          // [row blocks][N or 2 N], or NULL
    int M, N;
    int act;
    int rows;             // rows per workgroup
    int col_blocks;
};

__device__ inline void unpack8(u32x4 w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ inline u32x4 pack8(const float (&x)[8])
{
    return u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

// Adds the 8 row lanes' sums of 256 columns and writes them out.
__device__ inline void column_sums(float (*part)[GRAD_COLS], const float (&s)[8], int tx, int ty, float *out, int col0,
                                   int cols)
{
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e)
        part[ty][8 * tx + e] = s[e];
    __syncthreads();
    const int c = threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < GRAD_LANES; ++r)
        t += part[r][c];
    if (col0 + c < cols)
        out[col0 + c] = t;
}

template <bool GATED>
__global__ __launch_bounds__(GRAD_THREADS) void dense_grad_kernel(GradArgs p)
{
    __shared__ float part[GRAD_LANES][GRAD_COLS];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int cb = (int)blockIdx.x % p.col_blocks, rb = (int)blockIdx.x / p.col_blocks;
    const int n = cb * GRAD_COLS + 8 * tx;
    const int m_end = min(p.M, (rb + 1) * p.rows);
    const size_t width = GATED ? 2 * (size_t)p.N : (size_t)p.N;
    float sg[8] = {}, su[8] = {};
    if (n < p.N)
        with_act(p.act, [&](auto act_c) {
            constexpr int ACT = decltype(act_c)::value;
            for (int m = rb * p.rows + ty; m < m_end; m += GRAD_LANES) {
                float d[8], g[8], u[8];
                unpack8(*reinterpret_cast<const u32x4 *>(p.dc + (size_t)m * p.N + n), d);
                unpack8(*reinterpret_cast<const u32x4 *>(p.z + (size_t)m * width + n), g);
                if constexpr (GATED) {
                    unpack8(*reinterpret_cast<const u32x4 *>(p.z + (size_t)m * width + p.N + n), u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float value;
                        const float slope = act_slope<ACT>(g[e], &value);
                        g[e] = d[e] * u[e] * slope;
                        u[e] = d[e] * value;
                        sg[e] += g[e];
                        su[e] += u[e];
                    }
                    *reinterpret_cast<u32x4 *>(p.dz + (size_t)m * width + n) = pack8(g);
                    *reinterpret_cast<u32x4 *>(p.dz + (size_t)m * width + p.N + n) = pack8(u);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float value;
                        d[e] *= act_slope<ACT>(g[e], &value);
                        sg[e] += d[e];
                    }
                    *reinterpret_cast<u32x4 *>(p.dz + (size_t)m * width + n) = pack8(d);
                }
            }
        });
    if (p.sums) {
        float *out = p.sums + (size_t)rb * width;
        column_sums(part, sg, tx, ty, out, cb * GRAD_COLS, p.N);
        if constexpr (GATED)
            column_sums(part, su, tx, ty, out + p.N, cb * GRAD_COLS, p.N);
    }
}

// The bias gradient of 64 columns by THREADS threads: from the workgroups'
// column sums, or, where nothing else has to pass over dC (the identity), from dC
// itself. `part`: THREADS / 8 x 65 floats of LDS. From dC it takes cols / 64
// workgroups whatever the rows, and so grows with them where the columns are few:
// 4096 x 4096 in 9 us, 8192 x 1024 in 11, 65536 x 64 in 114 (alone, with the
// launch).
struct BiasArgs {
    const float *sums;     // [blocks][cols], or NULL
    const uint16_t *dc;    // else: blocks x cols BF16
    uint16_t *dbias;
    int cols, blocks;
};
constexpr int BIAS_COLS = 64, BIAS_THREADS = 512, BIAS_PITCH = 65;
template <int THREADS>
__device__ inline void bias_block(const BiasArgs &p, int block, float *part)
{
    const int c0 = block * BIAS_COLS;
    int lanes;
    if (p.sums) {
        const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, c = c0 + tx;
        float t = 0.0f;
        if (c < p.cols)
#pragma unroll 4
            for (int r = ty; r < p.blocks; r += THREADS / 64)
                t += p.sums[(size_t)r * p.cols + c];
        part[ty * BIAS_PITCH + tx] = t;
        lanes = THREADS / 64;
    } else {
        const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, c = c0 + 8 * tx;
        float s[8] = {};
        if (c < p.cols)
#pragma unroll 4
            for (int r = ty; r < p.blocks; r += THREADS / 8) {
                float x[8];
                unpack8(*reinterpret_cast<const u32x4 *>(p.dc + (size_t)r * p.cols + c), x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] += x[e];
            }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[ty * BIAS_PITCH + 8 * tx + e] = s[e];
        lanes = THREADS / 8;
    }
    __syncthreads();
    const int tx = threadIdx.x;
    if (tx < BIAS_COLS && c0 + tx < p.cols) {
        float t = 0.0f;
        for (int r = 0; r < lanes; ++r)
            t += part[r * BIAS_PITCH + tx];
        p.dbias[c0 + tx] = (uint16_t)pack_bf16(t, 0.0f);
    }
}

__global__ __launch_bounds__(BIAS_THREADS) void dense_bias_kernel(BiasArgs p)
{
    __shared__ float part[BIAS_THREADS / 8 * BIAS_PITCH];
    bias_block<BIAS_THREADS>(p, (int)blockIdx.x, part);
}

} // namespace dense
} // namespace gemm355
