// dense_wide.hpp -- 256 x 128 output tiles for the dense layer's operators,
// between the 128 x 128 tiles (dense_tile.hpp) and the 256 x 256 ones
// (dense_large.hpp): any pair of operand layouts, every epilogue, batches, and
// a last round whose tiles are split along K.
//
// What it is for: a 128 x 128 step moves 32 KiB into LDS for 2 MFLOP, and at
// 0.5 us a step its workgroups draw 17 TB/s from the L2s, which is what bounds
// them (matrix cores busy 43 %, no LDS bank conflicts). 256 x 128 moves 48 KiB
// for twice the work, and leaves twice as many workgroups as 256 x 256.
//
//   * 8 waves in 4 x 2, two per SIMD; a wave owns 64 x 64 (4 x 4 blocks, 64
//     accumulation registers) for the whole of K, so its sums stay in registers
//     until the epilogue.
//   * K advances 32 per step: one matrix instruction per block and step. A ring
//     of six stages of 24 KiB holds five steps in flight.
//   * LDS places. ROW_K: rows of 64 bytes; chunk c (16 bytes) of row r at
//     c ^ ((r >> 2) & 3), so that the 16 rows a fragment read touches at one
//     chunk fall into 16 different bank groups. COL_K: K rows of 512 (A) or 256
//     bytes (B), segments as in the other kernels.
//   * Step s: wait for this wave's copies of step s + 1, one barrier, then the 16
//     matrix instructions of step s; between them the reads of step s + 1 and the
//     copies of step s + 5, into the stage that every wave left before the last
//     barrier. The copies are spread out because a compute unit takes one in 16
//     cycles: issued together before the barrier, those of all waves kept the
//     matrix cores waiting for as long as they worked.
//   * A symmetric result: row tm of tiles has 2 tm + 2 tiles; the last two
//     straddle the diagonal and hold both halves of it, the others are stored a
//     second time, mirrored.
#pragma once

#include "dense_tile.hpp"

namespace gemm355 {
namespace dense {

constexpr int WIDE_M = 256, WIDE_N = 128;
constexpr int WIDE_BK = 32;
constexpr int WIDE_THREADS = 512;
constexpr int WIDE_STAGES = 6;
constexpr int WIDE_A = WIDE_M * WIDE_BK * 2, WIDE_B = WIDE_N * WIDE_BK * 2;   // bytes of a unit
constexpr int WIDE_COPIES = 3;                                              // per wave and step
constexpr int WIDE_FLOATS = WIDE_M * WIDE_N;

static_assert(WIDE_STAGES * (WIDE_A + WIDE_B) <= 163840, "LDS ring exceeds the 160 KiB of a gfx950 workgroup");
static_assert(WIDE_COPIES * (WIDE_STAGES - 1) <= 63, "vmcnt counts at most 63 outstanding operations");

// One operand (ROWS = 256: A, 128: B) of a tile.
template <class T, int LAYOUT, bool GATED, int ROWS>
struct WideOperand {
    typedef typename Frag<T>::type frag_t;
    static constexpr int COPIES = ROWS / 128;   // per wave
    i32x4 rsrc;
    unsigned off[COPIES];
    int chunk_k[COPIES];
    unsigned step, copy_lds, read_lds, flip;

    // `part`: the wave's 64 rows of the unit.
    __device__ inline void init(const void *base, int rows, int row0, int K, int gate_rows, unsigned lds, int wave,
                                int lane, int part)
    {
        const int l16 = lane & 15, grp = lane >> 4;
        const unsigned extent = (unsigned)(GATED ? 2 * gate_rows : rows) * (unsigned)K * 2u;
        rsrc = rsrc_words(base, base ? extent : 0u);
        copy_lds = lds + (unsigned)(1024 * COPIES * wave);
#pragma unroll
        for (int t = 0; t < COPIES; ++t) {
            const int block = COPIES * wave + t;   // 1 KiB block of the unit
            if constexpr (LAYOUT == ROW_K) {
                const int r = 16 * block + (lane >> 2), c = (lane & 3) ^ ((r >> 2) & 3);
                const int row = GATED ? ((r & 32) ? gate_rows : 0) + row0 + 32 * (r >> 6) + (r & 31) : row0 + r;
                off[t] = ((unsigned)row * (unsigned)K + 8u * (unsigned)c) * 2u;
                chunk_k[t] = 8 * c;   // rows past the operand lie past its range
            } else {
                const int k = block * (512 / ROWS) + lane / (ROWS / 8), pos = lane % (ROWS / 8);
                const int col = row0 + 8 * ((((pos >> 1) ^ key_col(k)) << 1) | (pos & 1));
                off[t] = ((unsigned)k * (unsigned)rows + (unsigned)col) * 2u;
                chunk_k[t] = col < rows ? 0 : NEVER;   // K rows past the operand lie past its range
            }
        }
        if constexpr (LAYOUT == ROW_K) {
            step = WIDE_BK * 2u;
            read_lds = lds + (unsigned)((64 * part + l16) * 64 + ((grp ^ ((l16 >> 2) & 3)) << 4));
            flip = 0;
        } else {
            step = (unsigned)WIDE_BK * (unsigned)rows * 2u;
            read_lds = lds + (unsigned)((8 * grp + (l16 >> 2)) * ROWS * 2 + (l16 & 3) * 8);
            flip = (unsigned)(((4 * part) ^ ((l16 >> 2) | ((grp & 1) << 2))) << 5);
        }
    }

    // This wave's copy t of K step `ks` into the unit at byte `slot` of the
    // ring; zeros when !in.
    __device__ inline void copy(int t, int ks, bool in, unsigned slot, int K) const
    {
        const unsigned v = in && ks * WIDE_BK + chunk_k[t] < K ? off[t] + (unsigned)ks * step : OFF_NONE;
        copy_one(rsrc, __builtin_amdgcn_readfirstlane(copy_lds + slot + 1024u * t), v);
    }

    __device__ inline frag_t read(unsigned slot, int blk) const
    {
        if constexpr (LAYOUT == ROW_K) {
            return *(__attribute__((address_space(3))) const frag_t *)(uintptr_t)(read_lds + slot + (unsigned)(blk * 16 * 64));
        } else {
            const unsigned at = read_lds + slot + (flip ^ (unsigned)(blk << 5));
            const s16x4 lo = read_tr(at), hi = read_tr(at + 8 * ROWS);
            return __builtin_bit_cast(frag_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    }
};

constexpr int wide_columns(int epi) { return epi == EPI_GATED ? WIDE_N / 2 : WIDE_N; }

template <int EPI>
__device__ inline void wide_tile(const DenseArgs &p, int pos, int &tm, int &tn)
{
    if constexpr (EPI >= EPI_STORE_SYM) {
        // tm (tm + 1) tiles come before row tm
        int t = (int)((__builtin_sqrtf(4.0f * (float)pos + 1.0f) - 1.0f) * 0.5f);
        while (t * (t + 1) > pos)
            --t;
        while ((t + 1) * (t + 2) <= pos)
            ++t;
        tm = t;
        tn = pos - t * (t + 1);
    } else {
        supergroup_tile(pos, p.tiles_m, p.tiles_n, p.supergroup, tm, tn);
    }
}

// Epilogue of block rows i0 and i0 + 1 of wave (wm, wn) of a tile.
template <int EPI, class TO>
__device__ inline void wide_store(const DenseArgs &p, f32x4 (&x0)[4], f32x4 (&x1)[4], int tm, int tn, int wm, int wn,
                                  int i0, int lane)
{
    const Views v = make_views<EPI>(p);
    const int m0 = tm * WIDE_M + 64 * wm + 16 * i0;
    const int col = tn * wide_columns(EPI) + wide_columns(EPI) / 2 * wn;
    u32x2 bias[4];
    u32x4 res[2][2];
    load_bias_row<EPI>(p, v, col, lane, bias);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        load_res_row<EPI, 4>(p, v, m0 + 16 * i + (lane & 15), col, lane, res[i]);
    store_row<EPI, TO>(p, v, x0, m0 + (lane & 15), col, lane, bias, res[0]);
    store_row<EPI, TO>(p, v, x1, m0 + 16 + (lane & 15), col, lane, bias, res[1]);
    if constexpr (EPI >= EPI_STORE_SYM)
        if (tn < 2 * tm)
            store_mirrored(p, v, x0, x1, m0, col, lane);
}

template <class T, int LA, int LB, int EPI, class TO>
__global__ __attribute__((amdgpu_flat_work_group_size(WIDE_THREADS, WIDE_THREADS), amdgpu_waves_per_eu(2, 2)))
void dense_wide_kernel(DenseArgs p)
{
    typedef typename Frag<T>::type frag_t;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[WIDE_STAGES * (WIDE_A + WIDE_B)];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 3, wn = wave >> 2;   // the wave's 64 rows and 64 columns (of B rows)

    const int item = tile_item(p);
    if (item < 0)
        return;
    const WorkItem w = work_item(p, item);
    const bool parts = w.tile >= p.whole && p.splits > 1;
    const int b = w.tile / p.tiles;
    int tm, tn;
    wide_tile<EPI>(p, w.tile - b * p.tiles, tm, tn);
    if (p.batch > 1)
        enter_batch(p, b);

    const unsigned lds_base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    WideOperand<T, LA, false, WIDE_M> oa;
    WideOperand<T, LB, EPI == EPI_GATED, WIDE_N> ob;
    oa.init(p.a, p.M, tm * WIDE_M, p.K, 0, lds_base, wave, lane, wm);
    ob.init(p.b, p.N, tn * wide_columns(EPI), p.K, p.N, lds_base + WIDE_STAGES * WIDE_A, wave, lane, wn);

    const int nk = (p.K + WIDE_BK - 1) / WIDE_BK;
    const int first = parts ? w.split * p.steps_per_split : 0;
    const int steps = parts ? max(0, min(p.steps_per_split, nk - first)) : nk;

    // stage counters: of the step to be copied and of the step to be read
    int copy_at = 0, read_at = 0;
    auto after = [](int stage) { return stage + 1 == WIDE_STAGES ? 0 : stage + 1; };
    // Copy c of this wave's three (two of A, one of B) for step s.
    auto copy = [&](int c, int s) {
        if (c < 2)
            oa.copy(c, first + s, s < steps, (unsigned)(copy_at * WIDE_A), p.K);
        else
            ob.copy(0, first + s, s < steps, (unsigned)(copy_at * WIDE_B), p.K);
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{};
    frag_t fa[2][4], fb[2][4];

    if (steps > 0) {
        for (int s = 0; s < WIDE_STAGES - 1; ++s, copy_at = after(copy_at))
            for (int c = 0; c < WIDE_COPIES; ++c)
                copy(c, s);
        wait_copies_le<WIDE_COPIES * (WIDE_STAGES - 2)>();
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[0][i] = oa.read(0, i);
            fb[0][i] = ob.read(0, i);
        }
        read_at = 1;
        auto step = [&](int s, auto buf_c) {
            constexpr int buf = decltype(buf_c)::value;
            wait_reads();
            wait_copies_le<WIDE_COPIES * (WIDE_STAGES - 3)>();
            lds_barrier();
            SCHED_FENCE();
            const unsigned ra = (unsigned)(read_at * WIDE_A), rb = (unsigned)(read_at * WIDE_B);
            read_at = after(read_at);
            static_for<16>([&](auto tc) {
                constexpr int t = decltype(tc)::value;
                constexpr int i = t >> 2, j = t & 3;
                acc[i][j] = Frag<T>::mma(fb[buf][j], fa[buf][i], acc[i][j]);
                // (past the last step: stale LDS, never used)
                if constexpr (t < 8) {
                    if constexpr (t & 1)
                        fb[buf ^ 1][t >> 1] = ob.read(rb, t >> 1);
                    else
                        fa[buf ^ 1][t >> 1] = oa.read(ra, t >> 1);
                }
                if constexpr (t % 5 == 4)
                    copy(t / 5, s + WIDE_STAGES - 1);
                SCHED_VALU_ONLY();
            });
            copy_at = after(copy_at);
        };
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            step(s, Int<0>{});
            step(s + 1, Int<1>{});
        }
        if (s < steps)
            step(s, Int<0>{});
        wait_reads();
        wait_all_copies();   // no copy may still be writing LDS when the workgroup ends
    }

    if (parts) {
        // partial tile, in register order: [wave][i][j][lane]
        f32x4 *ws = reinterpret_cast<f32x4 *>(p.ws) + (size_t)(item - p.whole) * (WIDE_FLOATS / 4) + wave * 16 * 64 + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ws[(i * 4 + j) * 64] = acc[i][j];
    } else {
        wide_store<EPI, TO>(p, acc[0], acc[1], tm, tn, wm, wn, 0, lane);
        wide_store<EPI, TO>(p, acc[2], acc[3], tm, tn, wm, wn, 2, lane);
    }
}

// Adds the splits' partials in order and runs the epilogue: one wave per two
// rows of blocks (32 rows x 64 columns) of a tile.
template <int EPI, class TO>
__global__ __launch_bounds__(64 * REDUCE_WAVES) void dense_wide_reduce_kernel(DenseArgs p)
{
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * REDUCE_WAVES + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tail = p.tiles * p.batch - p.whole, q = unit >> 4;
    if (q >= tail)
        return;
    const int b = (p.whole + q) / p.tiles;
    const int wave = (unit >> 1) & 7, i0 = 2 * (unit & 1);
    int tm, tn;
    wide_tile<EPI>(p, p.whole + q - b * p.tiles, tm, tn);
    const f32x4 *ws = reinterpret_cast<const f32x4 *>(p.ws) + (size_t)q * (WIDE_FLOATS / 4) + (wave * 16 + i0 * 4) * 64 + lane;
    f32x4 x[2][4] = {};
#pragma unroll 4
    for (int z = 0; z < p.splits; ++z) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][j] += ws[(i * 4 + j) * 64];
        ws += (size_t)tail * (WIDE_FLOATS / 4);
    }
    if (p.batch > 1)
        enter_batch(p, b);
    wide_store<EPI, TO>(p, x[0], x[1], tm, tn, wave & 3, wave >> 2, i0, lane);
}

} // namespace dense
} // namespace gemm355
