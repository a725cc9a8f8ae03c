// dense_large.hpp -- 256 x 256 output tiles for the dense layer's operators
// on large problems: any pair of operand layouts, BF16 or FP16, every epilogue,
// batches, and a last round whose tiles are split along K.
//
// The main loop is the chained one of gemm_bf16.hpp: four waves of 128 x 128
// (8 x 8 blocks, 256 accumulation registers), one ring of five 32 KiB LDS units
// fed by the memory pipeline, both K halves of a block back to back on the same
// accumulators, one barrier per step of K = 64, and copies, ring and fragment
// reads carried across a workgroup's tiles. What differs:
//   * Layouts. A COL_K unit is 64 K rows of 512 bytes; 32-byte segment s of K
//     row k sits at s ^ key_col(k), so that the eight K rows half a transposing
//     read touches fall into eight different bank groups. A fragment is two
//     such reads per K half (8 bytes each) instead of one of 16 bytes.
//   * Work items. Tiles that do not fill the last round of workgroups may have
//     their K steps split over all of them. The parts leave FP32 partials in the
//     workspace, in the order of the registers, and a second kernel adds a
//     tile's parts in K order and runs its epilogue: results do not depend on
//     timing. (Cutting the tail's steps into equal runs that cross tile borders
//     balances better, but its workgroups read a strip's K range at different
//     times: a step then took 2.2 us instead of 1.45, the L2s' hits lost.)
//   * Tiles of 192 x 192 (six blocks to a wave's side) for symmetric products,
//     where those leave fewer units idle.
//   * Epilogues: those of dense_common.hpp, each variant (activation, with or
//     without bias, residual or Z) a copy of the code without branches: with
//     them the accumulators spilled (394 us instead of 362 below).
//
// Measured (BF16; cards and runs differ by 6 %): layer of 8192 x 4096 with K =
// 8192 362 to 371 us, 1520 to 1480 TFLOP/s, and 382 to 406 with a residual read;
// gated layer of 8192 x 8192 with K = 4096 768 us, 1430, and 788 to 843 with its
// pre-activations stored; input and weight gradients of 4096 x 8192 x 4096 181 to
// 186 and 186 to 193 us, 1520 to 1420. Bounded by the matrix cores at the clock
// that the power limit leaves (1544 TFLOP/s for a large library product).
// 192 x 192: the LDS reads and writes of a step take as many cycles as its
// matrix instructions; a ring of six units, three steps ahead, gained nothing.
#pragma once

#include "dense_common.hpp"
#include "dense_loss.hpp"

namespace gemm355 {
namespace dense {

constexpr int BIG = 256;                      // output tile rows, and columns of B rows
constexpr int BIG_BK = 64;
constexpr int BIG_THREADS = 256;
constexpr int BIG_SLOTS = 5;
constexpr int BIG_FLOATS = BIG * BIG;
constexpr int BIG_MIN_STEPS = 4;              // fewest steps of a work item
// A wave's blocks per side, 8 or 6, give tiles of 256 or 192 rows; its 1 KiB
// copies per unit are as many.
constexpr int MID = 192;
constexpr int big_unit(int blocks) { return 32 * blocks * BIG_BK * 2; }
// Buffer resources and bases start BIG_SHIFT bytes early: copy j of a unit
// carries the instruction offset 1024 (j % 4), which moves the LDS destination
// and the global address alike, and the lane's offset stays non-negative.
constexpr int BIG_SHIFT = 3 * 1024;

static_assert(BIG_SLOTS * big_unit(8) <= 163840, "LDS ring exceeds the 160 KiB of a gfx950 workgroup");

// Columns of C per tile.
constexpr int big_columns(int epi, int side = BIG) { return epi == EPI_GATED ? side / 2 : side; }

__device__ inline void big_set_m0(unsigned lds_addr) { asm volatile("s_mov_b32 m0, %0" ::"s"(lds_addr) : "m0"); }
template <int O>
__device__ inline void big_copy(unsigned long long base, unsigned v)
{
    asm volatile("global_load_lds_dwordx4 %0, %1 offset:%2" ::"v"(v), "s"(base), "n"(O) : "memory");
}
template <int O>
__device__ inline void big_copy_buffer(const i32x4 &rsrc, unsigned v)
{
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen offset:%2 lds" ::"v"(v), "s"(rsrc), "n"(O) : "memory");
}

// Lane index recomputed where it is used (volatile, so that it is not kept in
// a register through the whole loop).
__device__ inline int fresh_lane()
{
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

// Keeps a row of accumulators in its accumulation registers up to this point:
// without it the compiler moves all 64 blocks out before the epilogue starts,
// which spills.
template <int BJ>
__device__ inline void hold_row(f32x4 (&x)[BJ])
{
#pragma unroll
    for (int j = 0; j < BJ; ++j)
        asm volatile("" : "+a"(x[j]));
}

// Block pairs of a step, as in gemm_bf16.hpp: the first half walks the upper
// half of the block rows column by column, the second half the lower one; a
// fragment is read after the last pair that uses its registers and at least
// eight pairs before its first use.
template <int BLOCKS>
struct BigOrder {
    static constexpr int HALF = BLOCKS * BLOCKS / 2, ROWS = BLOCKS / 2;
    static constexpr int row(int q) { return (q < HALF ? 0 : ROWS) + q % ROWS; }
    static constexpr int col(int q) { return q % HALF / ROWS; }
    static constexpr int a_read_at(int i)
    {
        return BLOCKS == 8 ? (i < 4 ? 34 + 4 * i : 8 + 6 * (i - 4)) : i < 3 ? 19 + 3 * i : 5 + 3 * (i - 3);
    }
    static constexpr int b_read_at(int j) { return BLOCKS == 8 ? 36 + 4 * j : 21 + 3 * j; }   // but for the last j
    static constexpr int LAST_B_READ = 2;
    static constexpr int a_copy_at(int c) { return BLOCKS * c + 2; }
    static constexpr int b_copy_at(int c, bool last) { return HALF + (last ? 2 : BLOCKS) * c; }
};

// TAIL: K is not a multiple of 64. The copies then go through the buffer form,
// whose range check fills what lies past K with zeros (ROW_K: by an offset past
// the range for the chunks past K; COL_K: those K rows lie past the operand).
template <class T, int LA, int LB, int EPI, class TO, bool TAIL, int BLOCKS = 8>
__global__ __attribute__((amdgpu_flat_work_group_size(BIG_THREADS, BIG_THREADS), amdgpu_waves_per_eu(1, 1)))
void dense_large_kernel(DenseArgs p)
{
    typedef typename Frag<T>::type frag_t;
    static_assert(BLOCKS == 8 || (BLOCKS == 6 && LA == ROW_K && LB == ROW_K && EPI != EPI_GATED));
    typedef BigOrder<BLOCKS> order;
    constexpr int SIDE = 32 * BLOCKS, UNIT = big_unit(BLOCKS), COPIES = BLOCKS, COLS = big_columns(EPI, SIDE);
    __shared__ __attribute__((aligned(1024))) uint8_t lds[BIG_SLOTS * UNIT];

    take_rows<EPI>(p, SIDE);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1;   // half of the tile's rows (A rows)
    const int wn = wave >> 1;  // half of its B rows
    const int l16 = lane & 15, grp = lane >> 4;
    const int nk = (p.K + BIG_BK - 1) / BIG_BK;

    const unsigned lds_base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    const unsigned a_step = LA == ROW_K ? BIG_BK * 2u : (unsigned)BIG_BK * (unsigned)pitch_a<EPI, LA>(p) * 2u;
    const unsigned b_step = LB == ROW_K ? BIG_BK * 2u : (unsigned)BIG_BK * (unsigned)p.N * 2u;
    const unsigned a_bytes = (unsigned)(LA == ROW_K ? p.M : p.K) * (unsigned)pitch_a<EPI, LA>(p) * 2u;
    const unsigned b_bytes = (unsigned)p.N * (unsigned)p.K * 2u * (EPI == EPI_GATED ? 2u : 1u);

    // The workgroup's items: one per round.
    struct Item {
        int at;              // its number; -1: none
        int tile, first, steps;
    };
    const int place = schedule_position(blockIdx.x, 0, p.grid), items = work_items(p);
    auto item_at = [&](int at) {
        if (at >= items)
            return Item{-1, 0, 0, 0};
        const WorkItem w = work_item(p, at);
        const int first = w.split * p.steps_per_split;
        return w.tile < p.whole ? Item{at, w.tile, 0, nk} : Item{at, w.tile, first, min(p.steps_per_split, nk - first)};
    };
    Item item = item_at(place);
    if (item.at < 0)
        return;
    Item next = item_at(place + p.grid);

    // Where the copies read: the operands' addresses (of the batch entry) and
    // this lane's offsets. Two steps before an item ends they move to the next
    // item's tile; after the last one they stay, so the copies issued for a
    // successor that is not there read valid memory and are never used. Rows
    // past M or N (ROW_K) are clamped to the last one, columns past them
    // (COL_K) to the last eight: they only feed outputs that are not stored.
    unsigned long long ga, gb;
    unsigned voff[2][COPIES];
    auto place_rows = [&](auto layout_c, unsigned (&o)[COPIES], int row0, int rows, int pitch, bool gated) {
        constexpr int L = decltype(layout_c)::value;
        const int ln = fresh_lane();
#pragma unroll
        for (int j = 0; j < COPIES; ++j) {
            const int block = COPIES * wave + j;   // 1 KiB block of the unit
            if constexpr (L == ROW_K) {
                const int r = 8 * block + (ln >> 3);
                const int c = swizzle_row(r, ln & 7);
                // gated: a wave's first four block columns are gate columns,
                // its last four the up columns of the same outputs
                const int row = gated ? ((r & 64) ? rows : 0) + min(row0 + 64 * (r >> 7) + (r & 63), rows - 1)
                                      : min(row0 + r, rows - 1);
                o[j] = ((unsigned)row * (unsigned)pitch + 8u * (unsigned)c) * 2u + BIG_SHIFT - 1024u * (j & 3);
            } else {
                const int k = 2 * block + (ln >> 5), pos = ln & 31;
                const int c = (((pos >> 1) ^ key_col(k)) << 1) | (pos & 1);
                const int col = min(row0 + 8 * c, epi_sized(EPI) ? (rows - 1) & ~7 : rows - 8);
                o[j] = ((unsigned)k * (unsigned)pitch + (unsigned)col) * 2u + BIG_SHIFT - 1024u * (j & 3);
            }
        }
    };
    auto place_copies = [&](int tile) {
        const int b = tile / p.tiles;
        int tm, tn;
        dense_tile<EPI>(p, tile - b * p.tiles, tm, tn);
        ga = reinterpret_cast<unsigned long long>(p.a) + (unsigned long long)b * a_bytes - BIG_SHIFT;
        gb = reinterpret_cast<unsigned long long>(p.b) + (unsigned long long)b * b_bytes - BIG_SHIFT;
        place_rows(Int<LA>{}, voff[0], tm * SIDE, p.M, pitch_a<EPI, LA>(p), false);
        place_rows(Int<LB>{}, voff[1], tn * COLS, p.N, LB == ROW_K ? p.K : p.N, EPI == EPI_GATED);
    };
    place_copies(item.tile);
    // ROW_K, per block parity: this lane's chunk of the last K step lies below K
    bool tail_ok[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        tail_ok[j] = (nk - 1) * BIG_BK + 8 * swizzle_row(8 * (COPIES * wave + j) + (lane >> 3), lane & 7) < p.K;

    // Per-step bases, hidden from the optimiser at every step so that addresses
    // are formed where they are used instead of living in registers.
    unsigned copy_base[2] = {lds_base + (unsigned)(COPIES * wave * 1024),
                             lds_base + (unsigned)(COPIES * wave * 1024 + 4096)};
    // ROW_K: lane (l16, grp) reads row l16 of a block, chunk grp (first K half)
    // or 4 + grp. COL_K: rd[0] is the lane's place in segment 0 of the wave's
    // half, rd[1] the flip of the segment number (shifted to bytes).
    unsigned ra[2], rb[2];
    auto read_base = [&](auto layout_c, unsigned (&o)[2], int half) {
        if constexpr (decltype(layout_c)::value == ROW_K) {
            o[0] = lds_base + (unsigned)((half * 16 * BLOCKS + l16) * 128 + (swizzle_row(l16, grp) << 4));
            o[1] = lds_base + (unsigned)((half * 16 * BLOCKS + l16) * 128 + (swizzle_row(l16, 4 + grp) << 4));
        } else {
            o[0] = lds_base + (unsigned)((8 * grp + (l16 >> 2)) * 512 + half * 256 + (l16 & 3) * 8);
            o[1] = (unsigned)(((l16 >> 2) | ((grp & 1) << 2)) << 5);
        }
    };
    read_base(Int<LA>{}, ra, wm);
    read_base(Int<LB>{}, rb, wn);

    // ring[x]: LDS offset of the slot of unit 2 s + x during step s; the next
    // step sees the slots rotated by two units.
    unsigned ring[BIG_SLOTS];
#pragma unroll
    for (int x = 0; x < BIG_SLOTS; ++x)
        ring[x] = (unsigned)(x * UNIT);
    auto rotate = [&]() {
        const unsigned r0 = ring[0], r1 = ring[1];
        ring[0] = ring[2];
        ring[1] = ring[3];
        ring[2] = ring[4];
        ring[3] = r0;
        ring[4] = r1;
    };

    f32x4 acc[BLOCKS][BLOCKS];
    frag_t fa[2][BLOCKS], fb[2][BLOCKS];
    typedef __attribute__((address_space(3))) const frag_t *lds_frag;
    auto read_half = [&](auto layout_c, const unsigned (&rd)[2], unsigned slot, int blk, int h) {
        if constexpr (decltype(layout_c)::value == ROW_K) {
            return *(lds_frag)(uintptr_t)(rd[h] + slot + (unsigned)(blk * 16 * 128));
        } else {
            const unsigned at = (rd[1] ^ (unsigned)(blk << 5)) + (rd[0] + slot) + (unsigned)(h * 32 * 512);
            const s16x4 lo = read_tr(at);
            SCHED_FENCE();
            const s16x4 hi = read_tr(at + 4 * 512);
            return __builtin_bit_cast(frag_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    };
    auto read_a = [&](unsigned slot, int i) {
        fa[0][i] = read_half(Int<LA>{}, ra, slot, i, 0);
        SCHED_FENCE();
        fa[1][i] = read_half(Int<LA>{}, ra, slot, i, 1);
    };
    auto read_b = [&](unsigned slot, int j) {
        fb[0][j] = read_half(Int<LB>{}, rb, slot, j, 0);
        SCHED_FENCE();
        fb[1][j] = read_half(Int<LB>{}, rb, slot, j, 1);
    };

    // Copy j of operand op's unit at K step ks into the slot whose base is in m0.
    auto copy = [&](int op, auto j_c, unsigned ks_off, bool tail) {
        constexpr int j = decltype(j_c)::value;
        const bool row_k = op ? LB == ROW_K : LA == ROW_K;
        unsigned v = voff[op][j];
        if constexpr (TAIL) {
            v = row_k && tail && !tail_ok[j & 1] ? OFF_NONE : v + ks_off;
            const unsigned long long base = op ? gb : ga;
            const i32x4 rsrc = {(int)(unsigned)base, (int)(unsigned)(base >> 32), (int)((op ? b_bytes : a_bytes) + BIG_SHIFT),
                                (int)RSRC_WORD3};
            big_copy_buffer<1024 * (j & 3)>(rsrc, v);
        } else {
            big_copy<1024 * (j & 3)>((op ? gb : ga) + ks_off, v);
        }
    };
    auto mma2 = [&](int q) {
        const int i = order::row(q), j = order::col(q);
        asm volatile("" ::"v"(fb[1][j]), "v"(fa[1][i]));
        SCHED_FENCE();
        acc[i][j] = Frag<T>::mma(fb[0][j], fa[0][i], acc[i][j]);
        SCHED_FENCE();
        acc[i][j] = Frag<T>::mma(fb[1][j], fa[1][i], acc[i][j]);
        SCHED_FENCE();
    };
    // Block pair q with copies 2 c and 2 c + 1 issued inside it, one after
    // each of its two instructions.
    auto mma2_copies = [&](int q, int op, auto c_c, unsigned slot, unsigned ks_off, bool tail) {
        constexpr int c = decltype(c_c)::value;
        const int i = order::row(q), j = order::col(q);
        asm volatile("" ::"v"(fb[1][j]), "v"(fa[1][i]));
        big_set_m0(copy_base[c >> 1] + slot);
        SCHED_FENCE();
        acc[i][j] = Frag<T>::mma(fb[0][j], fa[0][i], acc[i][j]);
        SCHED_FENCE();
        copy(op, Int<2 * c>{}, ks_off, tail);
        SCHED_FENCE();
        acc[i][j] = Frag<T>::mma(fb[1][j], fa[1][i], acc[i][j]);
        SCHED_FENCE();
        copy(op, Int<2 * c + 1>{}, ks_off, tail);
        SCHED_FENCE();
    };

    // Prologue: the first two steps' units, then the fragments that every later
    // item finds read by its predecessor's last step.
#pragma unroll
    for (int u = 0; u < BIG_SLOTS - 1; ++u) {
        const int ks = item.first + (u >> 1);
        const unsigned off = (unsigned)ks * (u & 1 ? b_step : a_step);
        static_for<COPIES / 2>([&](auto c_c) {
            constexpr int c = decltype(c_c)::value;
            big_set_m0(copy_base[c >> 1] + (unsigned)(u * UNIT));
            asm volatile("s_nop 0");
            copy(u & 1, Int<2 * c>{}, off, ks == nk - 1);
            copy(u & 1, Int<2 * c + 1>{}, off, ks == nk - 1);
        });
    }
    // The fragments of an item's first step that are not read within it. The
    // last step of the item before reads them too; where the epilogue needs the
    // registers (REREAD) they are read again behind it.
    constexpr bool REREAD = EPI == EPI_LINEAR || EPI == EPI_POLY || epi_loss(EPI);
    auto read_first = [&]() {
#pragma unroll
        for (int j = 0; j < BLOCKS - 1; ++j) {
            if (j < BLOCKS / 2) {
                read_a(ring[0], j);
                SCHED_FENCE();
            }
            read_b(ring[1], j);
            SCHED_FENCE();
        }
    };
    wait_all_copies();
    lds_barrier();
    read_first();

    // K step that step s of the current item copies for: two steps ahead, the
    // next item's first two in the last two.
    auto step = [&](int ks, auto first_c, auto last_c) {
        constexpr bool first = decltype(first_c)::value;
        constexpr bool last = decltype(last_c)::value;
        asm volatile("" : "+v"(ra[0]), "+v"(ra[1]), "+v"(rb[0]), "+v"(rb[1]), "+s"(copy_base[0]), "+s"(copy_base[1]));
        const bool tail = TAIL && ks == nk - 1;
        const unsigned a_off = (unsigned)ks * a_step, b_off = (unsigned)ks * b_step;
        static_for<order::HALF>([&](auto qc) {
            constexpr int q = decltype(qc)::value;
            constexpr int a0 = order::a_copy_at(0), d = order::a_copy_at(1) - a0;
            if constexpr (q >= a0 && (q - a0) % d == 0 && q <= order::a_copy_at(COPIES / 2 - 1))
                mma2_copies(q, 0, Int<(q - a0) / d>{}, ring[4], a_off, tail);
            else
                mma2(q);
            if constexpr (q == order::LAST_B_READ)
                read_b(ring[1], BLOCKS - 1);
#pragma unroll
            for (int i = BLOCKS / 2; i < BLOCKS; ++i)
                if (q == order::a_read_at(i))
                    read_a(ring[0], i);
            SCHED_VALU_ONLY();
        });
        wait_reads();
        if constexpr (!first)
            wait_copies_le<COPIES>();
        lds_barrier();
        SCHED_FENCE();
        static_for<order::HALF>([&](auto qc) {
            constexpr int q = order::HALF + decltype(qc)::value;
            constexpr int b0 = order::b_copy_at(0, last), d = order::b_copy_at(1, last) - b0;
            if constexpr (q >= b0 && (q - b0) % d == 0 && q <= order::b_copy_at(COPIES / 2 - 1, last))
                mma2_copies(q, 1, Int<(q - b0) / d>{}, ring[0], b_off, tail);
            else
                mma2(q);
#pragma unroll
            for (int i = 0; i < BLOCKS / 2; ++i)
                if (q == order::a_read_at(i))
                    read_a(ring[2], i);
#pragma unroll
            for (int j = 0; j < BLOCKS - 1; ++j)
                if (q == order::b_read_at(j))
                    read_b(ring[3], j);
            SCHED_VALU_ONLY();
        });
        SCHED_FENCE();
        rotate();
    };

    for (;;) {
        // accumulators written to zero in place (see gemm_bf16.hpp)
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                float zero;
                asm volatile("v_mov_b32 %0, 0" : "=v"(zero));
                acc[i][j] = f32x4{zero, zero, zero, zero};
            }
        // every item has at least BIG_MIN_STEPS steps
        step(item.first + 2, Int<1>{}, Int<0>{});
        for (int s = 1; s < item.steps - 2; ++s)
            step(item.first + s + 2, Int<0>{}, Int<0>{});
        const bool more = next.at >= 0;
        const int after = more ? next.first : item.first;
        place_copies(more ? next.tile : item.tile);
#pragma clang loop unroll(disable)
        for (int s = 0; s < 2; ++s)
            step(after + s, Int<0>{}, Int<1>{});
        // the next item's first two steps have landed (its first step waits
        // for no copies), its first fragments are read
        wait_all_copies();

        const int ln = fresh_lane();
        if (BLOCKS == 8 && item.steps < nk) {
            f32x4 *ws = reinterpret_cast<f32x4 *>(p.ws) + (size_t)(item.at - p.whole) * (BIG_FLOATS / 4) + wave * 64 * 64 + ln;
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i) {
                hold_row(acc[i]);
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    ws[(i * 8 + j) * 64] = acc[i][j];
            }
        } else {
            DenseArgs q = p;
            const int b = item.tile / p.tiles;
            int tm, tn;
            dense_tile<EPI>(p, item.tile - b * p.tiles, tm, tn);
            if (p.batch > 1)
                enter_batch(q, b);
            const int m0 = tm * SIDE + SIDE / 2 * wm;
            const int col = tn * COLS + COLS / 2 * wn;
            if constexpr (epi_loss(EPI))
                loss_rows<EPI>(q, acc, m0, col, ln, [&](int i) { hold_row(acc[i]); });
            else {
            const Views v = make_views<EPI>(q);
            with_epilogue<EPI>(q, [&](auto act_c, auto extra_c) {
                constexpr int ACT = decltype(act_c)::value, EXTRA = decltype(extra_c)::value;
                u32x2 bias[BLOCKS];
                load_bias_row<EPI, EXTRA>(q, v, col, ln, bias);
                // residual rows are asked for AHEAD rows before their use, and
                // before the stores of the row at hand
                constexpr int AHEAD = 3;
                u32x4 res[AHEAD][BLOCKS / 2];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    load_res_row<EPI, EXTRA, BLOCKS>(q, v, m0 + 16 * i + (ln & 15), col, ln, res[i]);
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    hold_row(acc[i]);
                    PackedRow<EPI, BLOCKS> row;
                    finish_row<EPI, TO, ACT, EXTRA>(q, acc[i], m0 + 16 * i + (ln & 15), col, ln, bias, res[i % AHEAD], row);
                    if (i + AHEAD < BLOCKS)
                        load_res_row<EPI, EXTRA, BLOCKS>(q, v, m0 + 16 * (i + AHEAD) + (ln & 15), col, ln, res[i % AHEAD]);
                    store_row<EXTRA>(q, v, row, m0 + 16 * i + (ln & 15), col, ln);
                    if constexpr (epi_symmetric(EPI))
                        if ((i & 1) && tm != tn)
                            store_mirrored(q, v, acc[i - 1], acc[i], m0 + 16 * (i - 1), col, ln);
                }
            });
            }
        }
        if constexpr (REREAD)
            read_first();
        if (!more)
            break;
        item = next;
        next = item_at(item.at + p.grid);
    }

    wait_reads();
    wait_all_copies();   // no copy may still be writing LDS when the workgroup ends
}

// Adds the parts of the split tiles in K order and runs the epilogue: one wave
// per two rows of blocks (32 rows x 128 columns of B rows) of a tile.
constexpr int BIG_REDUCE_WAVES = 4;
template <int EPI, class TO>
__global__ __launch_bounds__(64 * BIG_REDUCE_WAVES) void dense_large_reduce_kernel(DenseArgs p)
{
    take_rows<EPI>(p, BIG);
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * BIG_REDUCE_WAVES + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tail = p.tiles * p.batch - p.whole, t = unit >> 4;
    if (t >= tail)
        return;
    const int wave = (unit >> 2) & 3, i0 = 2 * (unit & 3);
    f32x4 x[2][8] = {};
    const f32x4 *ws = reinterpret_cast<const f32x4 *>(p.ws) + (size_t)t * (BIG_FLOATS / 4) + (wave * 64 + i0 * 8) * 64 + lane;
#pragma unroll 2
    for (int z = 0; z < p.splits; ++z) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] += ws[(i * 8 + j) * 64];
        ws += (size_t)tail * (BIG_FLOATS / 4);
    }
    const int tile = p.whole + t;
    const int b = tile / p.tiles;
    int tm, tn;
    dense_tile<EPI>(p, tile - b * p.tiles, tm, tn);
    DenseArgs q = p;
    if (p.batch > 1)
        enter_batch(q, b);
    const int m0 = tm * BIG + 128 * (wave & 1) + 16 * i0;
    const int col = tn * big_columns(EPI) + big_columns(EPI) / 2 * (wave >> 1);
    if constexpr (epi_loss(EPI)) {
        loss_rows<EPI>(q, x, m0, col, lane, [](int) {});
        return;
    } else {
    const Views v = make_views<EPI>(q);
    with_epilogue<EPI>(q, [&](auto act_c, auto extra_c) {
        constexpr int ACT = decltype(act_c)::value, EXTRA = decltype(extra_c)::value;
        u32x2 bias[8];
        u32x4 res[2][4];
        load_bias_row<EPI, EXTRA>(q, v, col, lane, bias);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_res_row<EPI, EXTRA, 8>(q, v, m0 + 16 * i + (lane & 15), col, lane, res[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            PackedRow<EPI, 8> row;
            finish_row<EPI, TO, ACT, EXTRA>(q, x[i], m0 + 16 * i + (lane & 15), col, lane, bias, res[i], row);
            store_row<EXTRA>(q, v, row, m0 + 16 * i + (lane & 15), col, lane);
        }
    });
    if constexpr (epi_symmetric(EPI))
        if (tm != tn)
            store_mirrored(q, v, x[0], x[1], m0, col, lane);
    }
}

} // namespace dense
} // namespace gemm355
