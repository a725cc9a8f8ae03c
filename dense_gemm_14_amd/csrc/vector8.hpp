// vector8.hpp -- eight consecutive values of a BF16 or FP32 array, as the
// kernels that pass over rows (embedding, layer norm) load and store them, ids
// of either integer type, and sums over a wave.
#pragma once

#include "common.hpp"

namespace gemm355 {
namespace rows {

// Eight values as they lie in memory: 16 bytes of BF16, 32 of FP32.
template <class T> struct Raw8;
template <> struct Raw8<__bf16> {
    u32x4 w;
    __device__ inline void load(const void *p, size_t at)
    {
        w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
    }
    // Past the L2 (a wave's 1 KiB is whole lines, and nothing here reads it again):
    // norms of 8192 x 4096, several sets of arrays in turn, in 29.2 us instead of 31.0,
    // their gradients in 57.6 instead of 58.5.
    __device__ inline void store(void *p, size_t at) const
    {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at));
    }
    __device__ inline float get(int e) const { return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]); }
    __device__ inline void set(const float (&x)[8])
    {
        w = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
    __device__ inline void fill(float v) { w = u32x4{} + pack_bf16(v, v); }
    // Keeps the compiler from carrying the unpacked values past this point.
    __device__ inline void hold() { asm volatile("" : "+v"(w)); }
};
template <> struct Raw8<float> {
    f32x4 lo, hi;
    __device__ inline void load(const void *p, size_t at)
    {
        lo = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at);
        hi = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at + 4);
    }
    // (through the L2, which joins the two halves of a line: a table's gradient of 32000 x
    // 4096 from 16384 tokens in 285 us, past it in 337)
    __device__ inline void store(void *p, size_t at) const
    {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at) = lo;
        *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at + 4) = hi;
    }
    __device__ inline float get(int e) const { return e < 4 ? lo[e] : hi[e - 4]; }
    __device__ inline void set(const float (&x)[8])
    {
        lo = f32x4{x[0], x[1], x[2], x[3]};
        hi = f32x4{x[4], x[5], x[6], x[7]};
    }
    __device__ inline void fill(float v) { lo = hi = f32x4{v, v, v, v}; }
    __device__ inline void hold() { asm volatile("" : "+v"(lo), "+v"(hi)); }
};

// Four values, 8 bytes of BF16 or 16 of FP32, each read or written once; a wave's are
// whole lines, and go past the L2 (16384 x 4096 rows looked up in 67 us, through it 72).
template <class T> struct Raw4;
template <> struct Raw4<__bf16> {
    u32x2 w;
    __device__ inline void load(const void *p, size_t at)
    {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(p) + at));
    }
    __device__ inline void store(void *p, size_t at) const
    {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + at));
    }
    __device__ inline float get(int e) const { return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]); }
    __device__ inline void set(const float (&x)[4]) { w = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}; }
};
template <> struct Raw4<float> {
    f32x4 v;
    __device__ inline void load(const void *p, size_t at)
    {
        v = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at));
    }
    __device__ inline void store(void *p, size_t at) const
    {
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at));
    }
    __device__ inline float get(int e) const { return v[e]; }
    __device__ inline void set(const float (&x)[4]) { v = f32x4{x[0], x[1], x[2], x[3]}; }
};
template <class T, int N> struct RawOf { typedef Raw8<T> type; };
template <class T> struct RawOf<T, 4> { typedef Raw4<T> type; };

// Id `i` of an array of 32- or 64-bit ids; -1 for one outside 0 .. count - 1.
__device__ inline int id_at(const void *ids, bool wide, size_t i, int count)
{
    const long long v = wide ? static_cast<const long long *>(ids)[i] : static_cast<const int *>(ids)[i];
    return v >= 0 && v < count ? (int)v : -1;
}

// Ids first, first + step, ... below last, N at once; -1 from there on. (The choice of
// type stands outside the loads, which would else wait for each other.)
template <int N>
__device__ inline void ids_at(const void *ids, bool wide, int64_t first, int64_t step, int64_t last, int count, int (&id)[N])
{
    long long v[N];
    if (wide) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] = first + k * step < last ? static_cast<const long long *>(ids)[first + k * step] : -1;
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] = first + k * step < last ? static_cast<const int *>(ids)[first + k * step] : -1;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        id[k] = v[k] >= 0 && v[k] < count ? (int)v[k] : -1;
}

// One step of a sum over lanes: x of the lane that CTRL names, 0 where there is
// none or ROWS (a mask of the wave's four rows of 16 lanes) leaves it out.
template <int CTRL, int ROWS>
__device__ inline float dpp_or_zero(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
}
// Sum over the wave's 64 lanes, the same in every lane: prefix sums inside the
// rows of 16 lanes, then of the rows; the order is fixed.
__device__ inline float wave_sum(float x)
{
    x += dpp_or_zero<0x111, 0xF>(x);   // one lane to the left
    x += dpp_or_zero<0x112, 0xF>(x);   // two
    x += dpp_or_zero<0x114, 0xF>(x);   // four
    x += dpp_or_zero<0x118, 0xF>(x);   // eight
    x += dpp_or_zero<0x142, 0xA>(x);   // the last lane of the row before, into rows 1 and 3
    x += dpp_or_zero<0x143, 0xC>(x);   // lane 31, into rows 2 and 3
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

} // namespace rows
} // namespace gemm355
