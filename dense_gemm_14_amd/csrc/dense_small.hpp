// dense_small.hpp -- small output tiles for the dense layer's operators where
// latency counts: few tokens, small layers. One launch, nothing in a workspace.
//
//   * A workgroup owns 16 MB rows x 16 NB columns (of B rows) of the output; its
//     WAVES waves share out K: wave w takes the K slices (64 elements) w, w +
//     WAVES, ... and computes the whole tile for them, so no LDS byte is read twice
//     and the waves never wait for each other until they add their sums. Eight
//     waves fill a compute unit; where there are more tiles than units, 64 x 64
//     tiles also run with four, two or one, as many more workgroups to a unit, so
//     that the last tiles do not wait for a unit of their own and short
//     contractions leave no wave idle.
//   * A wave copies its slices through the memory pipeline into its own LDS
//     ring (SMALL_STAGES stages of 2 KiB per block and slice): it waits for a
//     stage, reads the whole slice into registers, refills the stage at once and
//     then multiplies, so close to 128 KiB per compute unit are in flight all the
//     time -- several times HBM's latency times a compute unit's share of its
//     rate, which is what bounds these sizes.
//   * The waves' partial tiles meet in LDS (rows padded by 16 bytes: sixteen rows'
//     16-byte writes fall into 64 different banks), are added in wave order, and
//     each thread finishes eight consecutive columns of a row.
//   * Tiles: 64 x 64; 32 x 32 where those leave compute units idle; for few tokens
//     16 or 32 rows against 16 columns of weights (16 + 16 of a gated layer), so
//     that every compute unit has weights to stream.
//
// Measured (BF16, operands in cache, one launch behind the other, which alone
// takes 2.6 us): 1 x 1024 x 1024 3.5 us; 1 x 4096 x 4096 5.2, and 7.4 with the
// weights in HBM, 4.5 TB/s; 64 x 512 x 512 3.7; 333 x 1032 x 2056 8.9; 1024^3
// 6.8. Both products of a backward pass of 301 tokens, 1384 gated columns and K =
// 512 in one launch: 13 us. Bounded by latency: the launch, then the memory's
// once per slice that a wave takes.
#pragma once

#include "dense_common.hpp"
#include "dense_grad.hpp"

namespace gemm355 {
namespace dense {

constexpr int SMALL_BK = 64;
constexpr int small_stage(int mb, int nb) { return (mb + nb) * 2048; }
constexpr int small_stages(int mb, int nb) { return 20480 / small_stage(mb, nb); }
// floats per row of a partial tile
constexpr int small_pitch(int nb) { return 16 * nb + 4; }
constexpr int small_lds(int mb, int nb, int waves)
{
    return waves * (small_stages(mb, nb) * small_stage(mb, nb) > 16 * mb * small_pitch(nb) * 4
                              ? small_stages(mb, nb) * small_stage(mb, nb) : 16 * mb * small_pitch(nb) * 4);
}

// One operand of a tile of 16 RB rows, as one wave copies and reads it.
// GATED: the unit's first 8 RB rows are gate rows, the others the up rows of
// the same outputs.
// COL_K units: 64 K rows of 32 RB bytes; 32-byte segment s of K row k at
// s ^ key(k), so that the K rows 0..3 and 8..11 that half a transposing read
// touches fall into different bank groups (RB = 1: no choice, two-way).
template <class T, int LAYOUT, bool GATED, int RB>
struct SmallOperand {
    typedef typename Frag<T>::type frag_t;
    static constexpr int COPIES = 2 * RB;
    i32x4 rsrc;
    unsigned off[COPIES];
    int chunk_k[LAYOUT == ROW_K ? 2 : COPIES];
    unsigned step;
    unsigned lds;       // this wave's ring
    unsigned read_at[2];

    static __device__ inline int key(int k)
    {
        return RB == 4 ? ((k >> 1) & 1) | ((k >> 2) & 2) : RB == 2 ? (k >> 3) & 1 : 0;
    }

    __device__ inline void init(const void *base, int rows, int row0, int K, int gate_rows, unsigned ring, int lane)
    {
        const int l16 = lane & 15, grp = lane >> 4;
        const unsigned extent = (unsigned)(GATED ? 2 * gate_rows : rows) * (unsigned)K * 2u;
        rsrc = rsrc_words(static_cast<const uint8_t *>(base) - COPY_SHIFT, base ? extent + COPY_SHIFT : 0u);
        lds = ring;
#pragma unroll
        for (int t = 0; t < COPIES; ++t) {
            if constexpr (LAYOUT == ROW_K) {
                const int r = 8 * t + (lane >> 3);
                const int c = swizzle_row(r, lane & 7);
                const int row = row0 + (GATED ? (t < RB ? 0 : gate_rows - 8 * RB) : 0) + r;
                off[t] = ((unsigned)row * (unsigned)K + 8u * (unsigned)c) * 2u + COPY_SHIFT - 1024u * (t & 1);
                chunk_k[t & 1] = 8 * c;   // the same for every second copy; rows past the operand: past its range
            } else {
                const int k = t * (32 / RB) + lane / (2 * RB), pos = lane % (2 * RB);
                const int col = row0 + 16 * ((pos >> 1) ^ key(k)) + 8 * (pos & 1);
                off[t] = ((unsigned)k * (unsigned)rows + (unsigned)col) * 2u + COPY_SHIFT - 1024u * (t & 1);
                chunk_k[t] = col < rows ? 0 : NEVER;   // K rows past the operand lie past its range
            }
        }
        if constexpr (LAYOUT == ROW_K) {
            step = SMALL_BK * 2u;
            read_at[0] = (unsigned)(l16 * 128 + (swizzle_row(l16, grp) << 4));
            read_at[1] = (unsigned)(l16 * 128 + (swizzle_row(l16, 4 + grp) << 4));
        } else {
            step = (unsigned)SMALL_BK * (unsigned)rows * 2u;
            read_at[0] = (unsigned)((8 * grp + (l16 >> 2)) * 32 * RB + (l16 & 3) * 8);
            read_at[1] = (unsigned)(key(8 * grp + (l16 >> 2)) << 5);
        }
    }

    // K slice `ks` into the unit at byte `slot` of the ring; zeros when !in.
    __device__ inline void copy(int ks, bool in, unsigned slot, int K) const
    {
#pragma unroll
        for (int t = 0; t < COPIES; t += 2) {
            unsigned v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                v[u] = in && ks * SMALL_BK + chunk_k[LAYOUT == ROW_K ? u : t + u] < K ? off[t + u] + (unsigned)ks * step : OFF_NONE;
            copy_two(rsrc, __builtin_amdgcn_readfirstlane(lds + slot + 1024u * t), v[0], v[1]);
        }
    }

    // Fragment of block `blk`, K half h of the slice.
    __device__ inline frag_t read(unsigned slot, int blk, int h) const
    {
        if constexpr (LAYOUT == ROW_K) {
            return *(__attribute__((address_space(3))) const frag_t *)(uintptr_t)(lds + slot + read_at[h] + (unsigned)(blk * 2048));
        } else {
            const unsigned at = lds + slot + read_at[0] + (read_at[1] ^ (unsigned)(blk << 5)) + (unsigned)(h * 1024 * RB);
            const s16x4 lo = read_tr(at), hi = read_tr(at + 128 * RB);
            return __builtin_bit_cast(frag_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    }
};

// ---- epilogue of eight consecutive columns -----------------------------------

template <class T>
__device__ inline u32x4 pack_eight(const float (&x)[8])
{
    return u32x4{pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7])};
}
template <class T>
__device__ inline void unpack_eight(u32x4 w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 v = unpack2<T>(w[i]);
        x[2 * i] = v[0];
        x[2 * i + 1] = v[1];
    }
}
__device__ inline u32x4 *at16(const void *p, size_t element)
{
    return reinterpret_cast<u32x4 *>(const_cast<uint8_t *>(static_cast<const uint8_t *>(p)) + element * 2);
}

// C[m][n .. n + 7] from the sums x (EPI_GATED: the gate's, u the up's). Leaves
// the values before rounding in x.
template <int EPI, class TO>
__device__ inline void finish8(const DenseArgs &p, float (&x)[8], float (&u)[8], int m, int n)
{
    const size_t at = (size_t)m * p.N + n;
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_GATED) {
        float b[8];
        u32x4 res;
        if (EPI == EPI_LINEAR && p.r)
            res = *at16(p.r, at);
        if (p.bias) {
            unpack_eight<TO>(*at16(p.bias, n), b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] += b[e];
            if constexpr (EPI == EPI_GATED) {
                unpack_eight<TO>(*at16(p.bias, (size_t)p.N + n), b);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[e] += b[e];
            }
        }
        if (p.z) {
            if constexpr (EPI == EPI_GATED) {
                *at16(p.z, (size_t)m * 2 * p.N + n) = pack_eight<TO>(x);
                *at16(p.z, (size_t)m * 2 * p.N + p.N + n) = pack_eight<TO>(u);
            } else {
                *at16(p.z, at) = pack_eight<TO>(x);
            }
        }
        with_act(p.act, [&](auto act_c) {
            constexpr int ACT = decltype(act_c)::value;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = EPI == EPI_GATED ? act_value<ACT>(x[e]) * u[e] : act_value<ACT>(x[e]);
        });
        if (EPI == EPI_LINEAR && p.r) {
            unpack_eight<TO>(res, b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] += b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] *= p.alpha;
        if constexpr (EPI == EPI_POLY) {
            float r[8];
            unpack_eight<TO>(*at16(p.r, at), r);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] += p.beta * r[e] + (m == n + e ? p.gamma : 0.0f);
        }
    }
    *at16(p.c, at) = pack_eight<TO>(x);
}

// ---- one tile ------------------------------------------------------------------

constexpr int small_columns(int epi, int nb) { return epi == EPI_GATED ? 8 * nb : 16 * nb; }

template <class T, int LA, int LB, int EPI, class TO, int MB, int NB, int WAVES>
__device__ inline void small_tile(DenseArgs &p, int b, int tm, int tn, uint8_t *lds)
{
    typedef typename Frag<T>::type frag_t;
    constexpr int STAGE = small_stage(MB, NB), STAGES = small_stages(MB, NB), PITCH = small_pitch(NB);
    constexpr int SLICE_COPIES = 2 * (MB + NB);
    static_assert(SLICE_COPIES * (STAGES - 1) <= 63, "vmcnt counts at most 63 outstanding operations");
    if (p.batch > 1)
        enter_batch(p, b);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const unsigned ring = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + (unsigned)(wave * STAGES * STAGE);
    SmallOperand<T, LA, false, MB> oa;
    SmallOperand<T, LB, EPI == EPI_GATED, NB> ob;
    oa.init(p.a, p.M, tm * 16 * MB, p.K, 0, ring, lane);
    ob.init(p.b, p.N, tn * small_columns(EPI, NB), p.K, p.N, ring + 2048 * MB, lane);

    const int nk = (p.K + SMALL_BK - 1) / SMALL_BK;
    auto copies = [&](int s, unsigned slot) {
        const int ks = wave + WAVES * s;
        oa.copy(ks, ks < nk, slot, p.K);
        ob.copy(ks, ks < nk, slot, p.K);
    };
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = f32x4{};
    const int slices = wave < nk ? (nk - wave + WAVES - 1) / WAVES : 0;
    if (slices > 0) {
        for (int s = 0; s < STAGES; ++s)
            copies(s, (unsigned)(s * STAGE));
        unsigned slot = 0;
        for (int s = 0; s < slices; ++s) {
            wait_copies_le<SLICE_COPIES * (STAGES - 1)>();
            frag_t fa[MB][2], fb[NB][2];
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fa[i][h] = oa.read(slot, i, h);
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fb[j][h] = ob.read(slot, j, h);
            wait_reads();
            SCHED_FENCE();
            copies(s + STAGES, slot);   // (zeros past the last slice, never read)
            SCHED_FENCE();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = Frag<T>::mma(fb[j][h], fa[i][h], acc[i][j]);
            slot = slot + STAGE == STAGES * STAGE ? 0u : slot + STAGE;
        }
        wait_all_copies();   // none may still write the LDS that the sums use
    }
    // Lane (l16, grp) of block (i, j) holds row 16 i + l16, columns 16 j +
    // 4 grp .. + 3 of the tile.
    __syncthreads();
    float *sums = reinterpret_cast<float *>(lds);
    constexpr int PART = 16 * MB * PITCH;
    {
        float *mine = sums + wave * PART + (lane & 15) * PITCH + 4 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                *reinterpret_cast<f32x4 *>(mine + 16 * i * PITCH + 16 * j) = acc[i][j];
    }
    __syncthreads();

    constexpr int COLS = small_columns(EPI, NB);
    constexpr int RUNS = COLS / 8;   // of eight columns per row
    auto eight = [&](int r, int c, float (&x)[8]) {
        const float *at = sums + r * PITCH + c;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(at + w * PART), hi = *reinterpret_cast<const f32x4 *>(at + w * PART + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] += lo[e];
                x[4 + e] += hi[e];
            }
        }
    };
    for (int q = threadIdx.x; q < 16 * MB * RUNS; q += 64 * WAVES) {
        const int r = q / RUNS, c = 8 * (q % RUNS);
        const int m = tm * 16 * MB + r, n = tn * COLS + c;
        if (m < p.M && n < p.N) {
            float x[8], u[8];
            eight(r, c, x);
            if constexpr (EPI == EPI_GATED)
                eight(r, COLS + c, u);
            finish8<EPI, TO>(p, x, u, m, n);
            if constexpr (EPI >= EPI_STORE_SYM)
                if (tm != tn) {   // for the mirror image, one element at a time
                    const u32x4 w = pack_eight<TO>(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        static_cast<uint16_t *>(p.c)[(size_t)(n + e) * p.N + m] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
                }
        }
    }
}

// Workgroup -> item of `items`: each XCD takes a run of consecutive items.
__device__ inline int small_item(int items)
{
    const int run = (items + 7) / 8;
    const int item = ((int)blockIdx.x & 7) * run + ((int)blockIdx.x >> 3);
    return ((int)blockIdx.x >> 3) < run && item < items ? item : -1;
}

template <class T, int LA, int LB, int EPI, class TO, int MB, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void dense_small_kernel(DenseArgs p)
{
    static_assert(small_lds(MB, NB, WAVES) * (8 / WAVES) <= 163840, "8 / WAVES workgroups share a compute unit's LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[small_lds(MB, NB, WAVES)];
    fetch_args(p);
    const int item = small_item(p.tiles * p.batch);
    if (item < 0)
        return;
    const int b = p.batch > 1 ? item / p.tiles : 0;
    int tm = 0, tn = item - b * p.tiles;
    if (p.tiles_m > 1)   // (few tokens: no divisions)
        dense_tile<EPI>(p, item - b * p.tiles, tm, tn);
    small_tile<T, LA, LB, EPI, TO, MB, NB, WAVES>(p, b, tm, tn, lds);
}

// Both products of a small backward pass and its bias gradient in one launch:
// dA = dZ B, dB = dZ^T A and the bias blocks. They are independent, and one by
// one they leave most compute units idle. Items are taken in the order of the
// workgroups, the longer product's first (first_b: dB's), so that the short ones
// fill in behind; dealing each XCD a run of items, as one product's tiles are,
// would give one of them all the long ones (24.6 us instead of 13 at M = 301,
// N = 1384, K = 512, gated).
struct SmallBwdArgs {
    DenseArgs a, b;
    BiasArgs bias;
    int bias_blocks;
    int first_b;
};

template <int BLOCKS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void dense_small_bwd_kernel(SmallBwdArgs p)
{
    constexpr int LDS = small_lds(BLOCKS, BLOCKS, WAVES);
    static_assert(8 * WAVES * BIAS_PITCH * 4 <= LDS, "the bias blocks share the launch and its LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
    const int ahead = p.first_b ? p.b.tiles : 0;
    const int item = (int)blockIdx.x - ahead;
    int tm, tn;
    if (item >= 0 && item < p.a.tiles) {
        dense_tile<EPI_STORE>(p.a, item, tm, tn);
        small_tile<__bf16, ROW_K, COL_K, EPI_STORE, __bf16, BLOCKS, BLOCKS, WAVES>(p.a, 0, tm, tn, lds);
    } else if (item < p.a.tiles + p.b.tiles - ahead) {
        dense_tile<EPI_STORE>(p.b, item < 0 ? item + ahead : item - p.a.tiles, tm, tn);
        small_tile<__bf16, COL_K, COL_K, EPI_STORE, __bf16, BLOCKS, BLOCKS, WAVES>(p.b, 0, tm, tn, lds);
    } else {
        bias_block<64 * WAVES>(p.bias, item - (p.a.tiles + p.b.tiles - ahead), reinterpret_cast<float *>(lds));
    }
}

} // namespace dense
} // namespace gemm355
