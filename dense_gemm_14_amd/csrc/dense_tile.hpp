// dense_tile.hpp -- 128 x 128 output tiles for the dense layer's operators:
// any pair of operand layouts, BF16 or FP16 elements, every epilogue, and K
// split over several workgroups when there are few tiles.
//
//   * 8 waves. Waves 0..3 and 4..7 each tile the output 2 x 2 (a wave: 64 x 64
//     = 4 x 4 blocks of the 16 x 16 x 32 matrix instruction, 64 accumulation
//     registers) and take one half (32) of every step's 64 K elements each, so
//     a step reads each LDS byte as often as four waves would and two waves
//     per SIMD cover each other's waits. The halves are added at the end
//     through LDS.
//   * A step's unit is 16 KiB per operand, copied by the memory pipeline
//     straight into a ring of four LDS stages (three steps in flight, 96 KiB
//     per workgroup: a compute unit's share of HBM's latency times its rate).
//     ROW_K: 128 rows of 128 bytes; chunk c (16 bytes) of row r at position
//     c ^ ((r >> 1) & 7). COL_K: 64 K rows of 256 bytes; 32-byte segment s of
//     K row k at s ^ key(k), key = k % 4 + 4 ((k >> 3) & 1): the eight K rows
//     that half of a transposing read touches (0..3 and 8..11 of a group of
//     sixteen) fall into eight different bank groups.
//   * Step s: issue the copies of step s + 3 into the slot that every wave
//     left before the last barrier, wait for this wave's copies of step s + 1,
//     one barrier, then the 16 matrix instructions of step s with the reads of
//     step s + 1 between them.
//   * Split K: tiles that do not fill a round of workgroups are split over all
//     of them. Their partials go to the workspace in the order of the registers
//     (16 bytes per lane and block), and a second kernel adds them in split
//     order and runs the same epilogue: results do not depend on timing.
//
// For the sizes between the small tiles' and the 256 x 256 ones', where those
// would leave most units idle. Measured (BF16): 4096^3 in 144 us as a layer and
// 165 as a weight gradient, 950 and 830 TFLOP/s, the matrix cores busy 43 % of
// the time. What bounds it is the barrier of each step: 16 instructions per
// wave stand between two of them, against about 300 cycles of waiting; a variant
// without the copies, for measurement only, took 109 us. Tried instead: 256 x 128
// tiles (5 % faster on 4096^3 alone), two workgroups of four waves per unit (137
// to 188 us), copies or reads spread over the step (no change).
#pragma once

#include "dense_common.hpp"

namespace gemm355 {
namespace dense {

constexpr int TILE = 128;
constexpr int TILE_BK = 64;
constexpr int TILE_THREADS = 512;
constexpr int TILE_STAGES = 4;
constexpr int TILE_UNIT = TILE * TILE_BK * 2;            // 16 KiB
constexpr int TILE_LDS = TILE_STAGES * 2 * TILE_UNIT;    // 128 KiB
constexpr int TILE_FLOATS = TILE * TILE;
constexpr int TILE_COPIES = 4;                           // per wave and step: two of each operand

static_assert(TILE_LDS <= 163840, "LDS ring exceeds the 160 KiB of a gfx950 workgroup");
static_assert(TILE_COPIES * (TILE_STAGES - 1) <= 63, "vmcnt counts at most 63 outstanding operations");

// One operand of a 128-row tile: where this lane copies from, and where it
// reads its fragments.
// GATED: LDS row r of the unit holds weight row (r & 32 ? gate_rows : 0) +
// row0 + 32 (r / 64) + r % 32: a wave's first two block columns are gate
// columns, its last two the up columns of the same outputs.
template <class T, int LAYOUT, bool GATED>
struct TileOperand {
    typedef typename Frag<T>::type frag_t;
    i32x4 rsrc;
    unsigned off[2];     // buffer offsets of this lane's two copies at K step 0
    int chunk_k[2];      // ROW_K: K of their chunk within a step; NEVER: outside the operand
    unsigned step;       // bytes per K step
    unsigned copy_lds;   // this wave's 2 KiB of a unit
    unsigned read_lds;   // this lane's place of the wave's first block
    unsigned flip;       // COL_K: segment of block 0, to be flipped by the block's number

    __device__ inline void init(const void *base, int rows, int row0, int K, int gate_rows, unsigned lds, int wave,
                                int lane, int half, int k_half)
    {
        const int l16 = lane & 15, grp = lane >> 4;
        const unsigned extent = (unsigned)(GATED ? 2 * gate_rows : rows) * (unsigned)K * 2u;
        rsrc = rsrc_words(static_cast<const uint8_t *>(base) - COPY_SHIFT, base ? extent + COPY_SHIFT : 0u);
        copy_lds = lds + (unsigned)(2048 * wave);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int block = 2 * wave + t;   // 1 KiB block of the unit
            if constexpr (LAYOUT == ROW_K) {
                const int r = 8 * block + (lane >> 3);
                const int c = swizzle_row(r, lane & 7);
                const int row = GATED ? ((r & 32) ? gate_rows : 0) + row0 + 32 * (r >> 6) + (r & 31) : row0 + r;
                off[t] = ((unsigned)row * (unsigned)K + 8u * (unsigned)c) * 2u + COPY_SHIFT - 1024u * t;
                chunk_k[t] = 8 * c;   // rows past the operand lie past its range
            } else {
                const int k = 4 * block + (lane >> 4), pos = lane & 15;
                const int col = row0 + 8 * ((((pos >> 1) ^ key_col(k)) << 1) | (pos & 1));
                off[t] = ((unsigned)k * (unsigned)rows + (unsigned)col) * 2u + COPY_SHIFT - 1024u * t;
                chunk_k[t] = col < rows ? 0 : NEVER;   // K rows past the operand lie past its range
            }
        }
        if constexpr (LAYOUT == ROW_K) {
            step = TILE_BK * 2u;
            read_lds = lds + (unsigned)((64 * half + l16) * 128 + (swizzle_row(l16, 4 * k_half + grp) << 4));
            flip = 0;
        } else {
            step = (unsigned)TILE_BK * (unsigned)rows * 2u;
            read_lds = lds + (unsigned)((32 * k_half + 8 * grp + (l16 >> 2)) * 256 + (l16 & 3) * 8);
            flip = (unsigned)(((4 * half) ^ ((l16 >> 2) | ((grp & 1) << 2))) << 5);
        }
    }

    // This wave's copies of K step `ks` into the unit at byte `slot` of the
    // ring; nothing but zeros when !in.
    __device__ inline void copy(int ks, bool in, unsigned slot, int K) const
    {
        unsigned v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            v[t] = in && ks * TILE_BK + chunk_k[t] < K ? off[t] + (unsigned)ks * step : OFF_NONE;
        copy_two(rsrc, __builtin_amdgcn_readfirstlane(copy_lds + slot), v[0], v[1]);
    }

    // Fragment of block `blk` (16 rows) of this wave's half of the K step.
    __device__ inline frag_t read(unsigned slot, int blk) const
    {
        if constexpr (LAYOUT == ROW_K) {
            return *(__attribute__((address_space(3))) const frag_t *)(uintptr_t)(read_lds + slot + (unsigned)(blk * 16 * 128));
        } else {
            const unsigned at = read_lds + slot + (flip ^ (unsigned)(blk << 5));
            const s16x4 lo = read_tr(at), hi = read_tr(at + 1024);
            return __builtin_bit_cast(frag_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    }
};

// Columns of C per tile.
constexpr int tile_columns(int epi) { return epi == EPI_GATED ? TILE / 2 : TILE; }

// Workgroup -> work item, or -1. Workgroups go to the eight XCDs in turn; in
// every round each XCD takes a run of consecutive items, so the tiles its L2
// serves at one time share operand strips.
__device__ inline int tile_item(const DenseArgs &p)
{
    const int round = (int)blockIdx.x / p.grid, i = (int)blockIdx.x - round * p.grid;
    const int count = min(p.grid, work_items(p) - round * p.grid), run = (count + 7) / 8;
    const int at = (i & 7) * run + (i >> 3);
    return (i >> 3) < run && at < count ? round * p.grid + at : -1;
}

// Epilogue of block rows i0 and i0 + 1 of wave (wm, wn) of a tile.
template <int EPI, class TO>
__device__ inline void tile_store(const DenseArgs &p, f32x4 (&x)[2][4], int tm, int tn, int wm, int wn, int i0, int lane)
{
    const Views v = make_views<EPI>(p);
    const int m0 = tm * TILE + 64 * wm + 16 * i0;
    const int col = tn * tile_columns(EPI) + tile_columns(EPI) / 2 * wn;
    with_epilogue<EPI>(p, [&](auto act_c, auto extra_c) {
        constexpr int ACT = decltype(act_c)::value, EXTRA = decltype(extra_c)::value;
        u32x2 bias[4];
        u32x4 res[2][2];
        load_bias_row<EPI, EXTRA>(p, v, col, lane, bias);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_res_row<EPI, EXTRA, 4>(p, v, m0 + 16 * i + (lane & 15), col, lane, res[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            PackedRow<EPI, 4> row;
            finish_row<EPI, TO, ACT, EXTRA>(p, x[i], m0 + 16 * i + (lane & 15), col, lane, bias, res[i], row);
            store_row<EXTRA>(p, v, row, m0 + 16 * i + (lane & 15), col, lane);
        }
    });
    if constexpr (EPI >= EPI_STORE_SYM)
        if (tm != tn)
            store_mirrored(p, v, x[0], x[1], m0, col, lane);
}

template <class T, int LA, int LB, int EPI, class TO>
__global__ __attribute__((amdgpu_flat_work_group_size(TILE_THREADS, TILE_THREADS), amdgpu_waves_per_eu(2, 2)))
void dense_tile_kernel(DenseArgs p)
{
    typedef typename Frag<T>::type frag_t;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[TILE_LDS];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kh = wave >> 2;        // half of each step's K
    const int wm = wave & 1;         // 64-row half of the tile
    const int wn = (wave >> 1) & 1;  // 64-column half

    fetch_args(p);
    const int item = tile_item(p);
    if (item < 0)
        return;
    const WorkItem w = work_item(p, item);
    const bool parts = w.tile >= p.whole && p.splits > 1;
    const int b = p.batch > 1 ? w.tile / p.tiles : 0;
    int tm, tn;
    dense_tile<EPI>(p, w.tile - b * p.tiles, tm, tn);
    if (p.batch > 1)
        enter_batch(p, b);

    const unsigned lds_base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    TileOperand<T, LA, false> oa;
    TileOperand<T, LB, EPI == EPI_GATED> ob;
    oa.init(p.a, p.M, tm * TILE, p.K, 0, lds_base, wave, lane, wm, kh);
    ob.init(p.b, p.N, tn * tile_columns(EPI), p.K, p.N, lds_base + TILE_STAGES * TILE_UNIT, wave, lane, wn, kh);

    const int nk = (p.K + TILE_BK - 1) / TILE_BK;
    const int first = parts ? w.split * p.steps_per_split : 0;
    const int steps = parts ? max(0, min(p.steps_per_split, nk - first)) : nk;

    auto copies = [&](int s) {
        const unsigned slot = (unsigned)(s % TILE_STAGES) * TILE_UNIT;
        oa.copy(first + s, s < steps, slot, p.K);
        ob.copy(first + s, s < steps, slot, p.K);
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{};
    frag_t fa[2][4], fb[2][4];

    if (steps > 0) {
        for (int s = 0; s < TILE_STAGES - 1; ++s)
            copies(s);
        wait_copies_le<TILE_COPIES * (TILE_STAGES - 2)>();
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[0][i] = oa.read(0, i);
            fb[0][i] = ob.read(0, i);
        }
        auto step = [&](int s, auto buf_c) {
            constexpr int buf = decltype(buf_c)::value;
            copies(s + TILE_STAGES - 1);
            wait_reads();
            wait_copies_le<TILE_COPIES * (TILE_STAGES - 2)>();
            lds_barrier();
            SCHED_FENCE();
            const unsigned next = (unsigned)((s + 1) % TILE_STAGES) * TILE_UNIT;
            static_for<16>([&](auto tc) {
                constexpr int t = decltype(tc)::value;
                constexpr int i = t >> 2, j = t & 3;
                acc[i][j] = Frag<T>::mma(fb[buf][j], fa[buf][i], acc[i][j]);
                // (past the last step: stale LDS, never used)
                if constexpr (t < 8) {
                    if constexpr (t & 1)
                        fb[buf ^ 1][t >> 1] = ob.read(next, t >> 1);
                    else
                        fa[buf ^ 1][t >> 1] = oa.read(next, t >> 1);
                }
                SCHED_VALU_ONLY();
            });
        };
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            step(s, Int<0>{});
            step(s + 1, Int<1>{});
        }
        if (s < steps)
            step(s, Int<0>{});
        wait_reads();
        wait_all_copies();   // no copy may still write the LDS that the exchange uses
    }

    // Add the two K halves: waves kh = 0 finish block rows 0, 1 and kh = 1
    // rows 2, 3; each hands the other two to its partner. 1 KiB per block.
    lds_barrier();
    const int pair = wave & 3;
    f32x4 *xch = reinterpret_cast<f32x4 *>(lds);
    auto slot_of = [&](int owner, int i, int j) { return ((owner * 4 + pair) * 8 + (i & 1) * 4 + j) * 64 + lane; };
    f32x4 out[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xch[slot_of(kh ^ 1, i, j)] = kh ? acc[i][j] : acc[2 + i][j];
            out[i][j] = kh ? acc[2 + i][j] : acc[i][j];
        }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            out[i][j] += xch[slot_of(kh, i, j)];

    if (parts) {
        // partial tile, in register order: block row u = 2 kh + i of wave
        // (wm, wn) is the run [pair][u][j][lane]
        f32x4 *ws = reinterpret_cast<f32x4 *>(p.ws) + (size_t)(item - p.whole) * (TILE_FLOATS / 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ws[((pair * 4 + 2 * kh + i) * 4 + j) * 64 + lane] = out[i][j];
    } else {
        tile_store<EPI, TO>(p, out, tm, tn, wm, wn, 2 * kh, lane);
    }
}

// Adds the splits' partials in order and runs the epilogue: one wave per two
// rows of blocks (32 rows x 64 columns) of a tile.
constexpr int REDUCE_WAVES = 4;
template <int EPI, class TO>
__global__ __launch_bounds__(64 * REDUCE_WAVES) void dense_reduce_kernel(DenseArgs p)
{
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * REDUCE_WAVES + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tail = p.tiles * p.batch - p.whole, q = unit >> 3;
    if (q >= tail)
        return;
    const int b = (p.whole + q) / p.tiles;
    const int pair = (unit >> 1) & 3, i0 = 2 * (unit & 1);
    int tm, tn;
    dense_tile<EPI>(p, p.whole + q - b * p.tiles, tm, tn);
    const f32x4 *ws = reinterpret_cast<const f32x4 *>(p.ws) + (size_t)q * (TILE_FLOATS / 4) + ((pair * 4 + i0) * 4) * 64 + lane;
    f32x4 x[2][4] = {};
#pragma unroll 4
    for (int z = 0; z < p.splits; ++z) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][j] += ws[(i * 4 + j) * 64];
        ws += (size_t)tail * (TILE_FLOATS / 4);
    }
    if (p.batch > 1)
        enter_batch(p, b);
    tile_store<EPI, TO>(p, x, tm, tn, pair & 1, pair >> 1, i0, lane);
}

} // namespace dense
} // namespace gemm355
