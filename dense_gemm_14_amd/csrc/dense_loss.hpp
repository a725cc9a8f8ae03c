// dense_loss.hpp -- epilogues of the products around the softmax cross entropy
// over a vocabulary (cross_entropy.hpp has the other kernels and the whole):
//
//   EPI_CE       z = A B^T of a tile. Nothing of it is stored but, for each row
//                and run of columns, the sum of 2^(z log2(e) - base) with its base
//                (see loss_base for large z), and the target's z where the run holds it.
//   EPI_CE_GRAD  z again, C = round((exp(z - lse) - [column = target]) weight),
//                zeros in the columns between N and the next multiple of 8
//   EPI_ACC      sums over pieces of the contraction: FP32 sums, added to those
//                of the pieces before, rounded to C by the last piece
//
// Work per element: an exponential, at a quarter of the vector rate, and three or
// four plain instructions (maximum, multiply-add, sum; or multiply-add, factor,
// conversion), 4 % of a tile's time at K = 4096; a compare with the target only in
// the runs that hold one. Measured, forward of 8192 x 128000 with K = 4096: 6.0 ms,
// a library product of these sizes 5.9; 6.06 with an epilogue that stores one value
// a row, so what is left of it hides behind the power limit.
#pragma once

#include "dense_common.hpp"
#include "vector8.hpp"

namespace gemm355 {
namespace dense {

constexpr float LOG2E = 1.4426950408889634f;

// Variants of a tile's epilogue. EPI_CE, EPI_CE_GRAD: LOSS_EDGE, the run has
// columns past N. EPI_ACC: LOSS_ADD, there is a piece before; LOSS_LAST, there is
// none after. Copies of the code, not branches in each row: with those the
// compiler moved accumulators about in the main loop (8192 x 128000, K = 4096:
// 6250 us instead of 6020).
enum { LOSS_EDGE = 1, LOSS_ADD = 1, LOSS_LAST = 2 };

template <int EPI, class F>
__device__ inline void with_loss(const DenseArgs &p, int col, int width, F &&f)
{
    if constexpr (EPI == EPI_ACC) {
        if (p.add)
            p.last ? f(Int<LOSS_ADD | LOSS_LAST>{}) : f(Int<LOSS_ADD>{});
        else
            p.last ? f(Int<LOSS_LAST>{}) : f(Int<0>{});
    } else {
        col + width > p.N ? f(Int<LOSS_EDGE>{}) : f(Int<0>{});
    }
}

// What an epilogue needs to know of row m: EPI_CE the target's column, EPI_CE_GRAD
// that and the row's lse and weight, EPI_ACC (last piece) the row of C.
struct LossRow {
    int at;
    float lse, weight;
};
// Column of row m's target; below 0 for a row that is left out.
__device__ inline int loss_target(const DenseArgs &p, int m)
{
    return (p.target ? p.target[m] : rows::id_at(p.ids, p.wide, (size_t)m, p.vocab)) - p.v0;
}
template <int EPI, int MODE>
__device__ inline LossRow loss_row_of(const DenseArgs &p, int m)
{
    LossRow r = {-1, 0.0f, 0.0f};
    if (m < p.M) {
        if constexpr (EPI == EPI_ACC) {
            if constexpr (MODE & LOSS_LAST)
                r.at = p.map ? p.map[m] : m;
        } else {
            r.at = loss_target(p, m);
            if constexpr (EPI == EPI_CE_GRAD) {
                r.lse = p.lse[m];
                r.weight = p.weight[m];
            }
        }
    }
    return r;
}

// Largest and sum over the four lanes that hold a row (l16, 16 + l16, ...): a swap
// of a value with itself leaves each lane both halves' values.
struct Two {
    float a, b;
};
__device__ inline Two swap_halves(float x)
{
    const unsigned w = __builtin_bit_cast(unsigned, x);
    const auto s = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const unsigned a = s[0], b = s[1];
    return Two{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ inline Two swap_rows(float x)
{
    const unsigned w = __builtin_bit_cast(unsigned, x);
    const auto s = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    const unsigned a = s[0], b = s[1];
    return Two{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ inline float row_max(float x)
{
    const Two h = swap_halves(x), r = swap_rows(fmaxf(h.a, h.b));
    return fmaxf(r.a, r.b);
}
__device__ inline float row_add(float x)
{
    const Two h = swap_halves(x), r = swap_rows(h.a + h.b);
    return r.a + r.b;
}

// Exponentials are powers of two: exp(z) = 2^(z log2(e)). What their arguments are
// taken from is a whole number near the largest argument (0 where that is
// infinite: all -inf then give a sum of 0, and +inf one of +inf; NaN is in the sum
// in any case), so that an argument is one multiply-add with one rounding of its
// small result, and joining two sums multiplies by a power of two, exactly.
// A large base is rounded, by half a step, at most 64 below 1.5 2^30; the arguments
// are taken from it as it is, so the sum has that difference as a factor.
// From LOSS_FAR on (a mask's -1e30, say) the difference would be more than a power of
// two holds, and from 2.4e38 on the product overflows. But FP32 values that are not the
// same lie 64 and more apart there, and so do those nearer to 0: beside the largest
// logit no other weighs, to any base. Its run's arguments are z - top: a factor and a
// base of their own for the row's multiply-adds, and nothing more for each element (330 x
// 81578, K = 328: 62.8 us with it, 62.0 without; differences taken first instead, in a
// branch a row, 63.6, in a copy of the code for such rows 85, as it spilt).
constexpr float LOSS_FAR = 1073741824.0f;      // 2^30
__device__ inline bool loss_far(float x) { return fabsf(x) >= LOSS_FAR; }
__device__ inline float loss_factor(float x) { return loss_far(x) ? 1.0f : LOG2E; }
__device__ inline float loss_base(float top, float factor) { return __builtin_isinf(top) ? 0.0f : __builtin_rintf(top * factor); }
__device__ inline float loss_exp(float z, float factor, float base) { return __builtin_amdgcn_exp2f(__builtin_fmaf(z, factor, -base)); }
// {base, sum} as it is stored: base -inf where no value was finite, the sum then 0,
// +inf or NaN; from LOSS_FAR on {top, -sum}.
__device__ inline f32x2 loss_stat(float top, float base, float sum)
{
    return __builtin_isinf(top) ? f32x2{-__builtin_inff(), sum} : f32x2{base, loss_far(top) ? -sum : sum};
}
// What the rounding of a row's base, lse log2(e), multiplies its exponentials by. Below
// LOSS_EXACT, where all rows are that a network has learnt from, less than 2^-14 of
// them, the lse's own rounding; from LOSS_FAR on there is none.
constexpr float LOSS_EXACT = 1024.0f;
__device__ inline float loss_excess(float lse)
{
    const bool none = !(fabsf(lse) >= LOSS_EXACT && fabsf(lse) < LOSS_FAR);
    return none ? 1.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(lse, LOG2E, -(lse * LOG2E)));
}

// What a row of blocks reads besides its sums (EPI_ACC: the pieces' before).
template <int EPI, int MODE, int BJ>
__device__ inline void load_acc_row(const DenseArgs &p, int m, int col, int lane, f32x4 (&add)[BJ])
{
    if constexpr (EPI == EPI_ACC && (MODE & LOSS_ADD))
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            const int n = col + 16 * j + 4 * (lane >> 4);
            add[j] = m < p.M && n < p.N ? *reinterpret_cast<const f32x4 *>(p.acc + (size_t)m * (size_t)p.N + (size_t)n) : f32x4{};
        }
}

// The epilogue of one row of blocks: x[0 .. BJ - 1], BJ blocks side by side at
// column `col`, this lane's row m.
template <int EPI, int MODE, int BJ>
__device__ inline void loss_row(const DenseArgs &p, const __amdgpu_buffer_rsrc_t &rc, f32x4 (&x)[BJ], int m, int col,
                                int lane, const LossRow &row, const f32x4 (&add)[BJ])
{
    const int n0 = col + 4 * (lane >> 4);
    // (a real branch, for what one run in a hundred needs: the statement in it
    // keeps the compiler from computing both sides and choosing)
    const bool hit = __ballot(row.at >= col && row.at < col + 16 * BJ) != 0;
    const int d = row.at - n0;
    if constexpr (EPI == EPI_CE) {
        if constexpr (MODE & LOSS_EDGE) {
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[j][e] = n0 + 16 * j + e < p.N ? x[j][e] : -__builtin_inff();
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fmaxf(top, x[j][e]);
        top = row_max(top);
        const float factor = loss_factor(top), base = loss_base(top, factor);
        if (hit) {
            float picked = 0.0f;
            asm volatile("");
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    picked = d == 16 * j + e ? x[j][e] : picked;
            if (d >= 0 && d < 16 * BJ && (d & 12) == 0)
                p.picked[m] = picked;
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            float t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = loss_exp(x[j][e], factor, base);
            sum += (t[0] + t[1]) + (t[2] + t[3]);
        }
        sum = row_add(sum);
        if (lane < 16 && m < p.M && col < p.N)
            p.stats[(size_t)(col / (16 * BJ)) * (size_t)p.stats_rows + (size_t)m] = loss_stat(top, base, sum);
    }
    if constexpr (EPI == EPI_CE_GRAD) {
        const float factor = loss_factor(row.lse), base = row.lse * factor;
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[j][e] = loss_exp(x[j][e], factor, base);
        if (hit) {
            asm volatile("");
            const float one = loss_excess(row.lse);      // (the weight has it divided out)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[j][e] -= d == 16 * j + e ? one : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[j][e] *= row.weight;
        if constexpr (MODE & LOSS_EDGE) {
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[j][e] = n0 + 16 * j + e < p.N ? x[j][e] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < BJ; j += 2)
            store16(pack_pair<__bf16>(x[j], x[j + 1]), rc, pair_offset(p, m, col + 16 * j, p.ldc, 0, lane));
    }
    if constexpr (EPI == EPI_ACC) {
#pragma unroll
        for (int j = 0; j < BJ; ++j)
            if constexpr (MODE & LOSS_ADD)
                x[j] += add[j];
        if constexpr (MODE & LOSS_LAST) {
#pragma unroll
            for (int j = 0; j < BJ; j += 2) {
                const u32x4 w = pack_pair<__bf16>(x[j] * p.alpha, x[j + 1] * p.alpha);
                const int n = col + 16 * j + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
                store16(w, rc, m < p.M && n < p.N ? (int)(((unsigned)row.at * (unsigned)p.N + (unsigned)n) * 2u) : OOB);
            }
        } else {
#pragma unroll
            for (int j = 0; j < BJ; ++j)
                if (m < p.M && n0 + 16 * j < p.N)
                    *reinterpret_cast<f32x4 *>(p.acc + (size_t)m * (size_t)p.N + (size_t)(n0 + 16 * j)) = x[j];
        }
    }
}

// Where the epilogue stores 16-bit values.
template <int EPI>
__device__ inline __amdgpu_buffer_rsrc_t loss_rsrc(const DenseArgs &p)
{
    const unsigned bytes = EPI == EPI_CE_GRAD ? (unsigned)p.M * (unsigned)p.ldc * 2u
                           : EPI == EPI_ACC   ? (unsigned)p.c_rows * (unsigned)p.N * 2u : 0u;
    return make_rsrc(p.c, bytes);
}

// Rows of blocks m0 + 16 i, i < R, of a wave's tile, BJ blocks wide at `col`;
// hold(i) before row i's sums are used.
template <int EPI, int R, int BJ, class Hold>
__device__ inline void loss_rows(const DenseArgs &p, f32x4 (&x)[R][BJ], int m0, int col, int lane, Hold &&hold)
{
    const __amdgpu_buffer_rsrc_t rc = loss_rsrc<EPI>(p);
    with_loss<EPI>(p, col, 16 * BJ, [&](auto mode_c) {
        constexpr int MODE = decltype(mode_c)::value;
        constexpr int AHEAD = EPI == EPI_ACC && (MODE & LOSS_ADD) ? (R < 2 ? R : 2) : 1;
        LossRow row[R];
        f32x4 add[AHEAD][BJ];
#pragma unroll
        for (int i = 0; i < R; ++i)
            row[i] = loss_row_of<EPI, MODE>(p, m0 + 16 * i + (lane & 15));
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            load_acc_row<EPI, MODE>(p, m0 + 16 * i + (lane & 15), col, lane, add[i]);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            hold(i);
            loss_row<EPI, MODE>(p, rc, x[i], m0 + 16 * i + (lane & 15), col, lane, row[i], add[i % AHEAD]);
            if (i + AHEAD < R)
                load_acc_row<EPI, MODE>(p, m0 + 16 * (i + AHEAD) + (lane & 15), col, lane, add[i % AHEAD]);
        }
    });
}

// The same for eight consecutive columns n .. n + 7 of row m, one of the RUNS
// neighbouring lanes that hold a tile's row (small tiles). All of them call it, in
// or out of C. What it reads besides its sums is asked for beforehand.
struct LossEight {
    LossRow row;
    f32x4 add[2];
};
template <int EPI>
__device__ inline LossEight loss_eight_of(const DenseArgs &p, int m, int n)
{
    LossEight r = {loss_row_of<EPI, LOSS_LAST>(p, m), {}};
    if constexpr (EPI == EPI_ACC)
        if (p.add && m < p.M && n < p.N) {
            const f32x4 *acc = reinterpret_cast<const f32x4 *>(p.acc + (size_t)m * (size_t)p.N + (size_t)n);
            r.add[0] = acc[0];
            r.add[1] = acc[1];
        }
    return r;
}
template <int EPI, int RUNS>
__device__ inline void loss_eight(const DenseArgs &p, float (&x)[8], int m, int n, int part, const LossEight &r)
{
    const bool in = m < p.M && n < p.N;
    const int d = r.row.at - n;
    if constexpr (EPI == EPI_CE) {
        float top = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = in && n + e < p.N ? x[e] : -__builtin_inff();
            top = fmaxf(top, x[e]);
        }
#pragma unroll
        for (int d = 1; d < RUNS; d *= 2)
            top = fmaxf(top, __shfl_xor(top, d));
        const float factor = loss_factor(top), base = loss_base(top, factor);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += loss_exp(x[e], factor, base);
#pragma unroll
        for (int d = 1; d < RUNS; d *= 2)
            sum += __shfl_xor(sum, d);
        if (!in)
            return;
        if (((int)threadIdx.x & (RUNS - 1)) == 0)
            p.stats[(size_t)part * (size_t)p.stats_rows + (size_t)m] = loss_stat(top, base, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (d == e && n + e < p.N)
                p.picked[m] = x[e];
    } else {
        if (!in)
            return;
        if constexpr (EPI == EPI_CE_GRAD) {
            const float factor = loss_factor(r.row.lse), base = r.row.lse * factor, one = loss_excess(r.row.lse);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = n + e < p.N ? (loss_exp(x[e], factor, base) - (d == e ? one : 0.0f)) * r.row.weight : 0.0f;
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.c) + (size_t)m * (size_t)p.ldc + (size_t)n) =
                u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
        }
        if constexpr (EPI == EPI_ACC) {
            if (p.add)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] += r.add[0][e];
                    x[4 + e] += r.add[1][e];
                }
            if (p.last) {
                const float scale = p.alpha;
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.c) + (size_t)r.row.at * (size_t)p.N + (size_t)n) =
                    u32x4{pack_bf16(x[0] * scale, x[1] * scale), pack_bf16(x[2] * scale, x[3] * scale),
                          pack_bf16(x[4] * scale, x[5] * scale), pack_bf16(x[6] * scale, x[7] * scale)};
            } else {
                f32x4 *acc = reinterpret_cast<f32x4 *>(p.acc + (size_t)m * (size_t)p.N + (size_t)n);
                acc[0] = f32x4{x[0], x[1], x[2], x[3]};
                acc[1] = f32x4{x[4], x[5], x[6], x[7]};
            }
        }
    }
}

} // namespace dense
} // namespace gemm355
