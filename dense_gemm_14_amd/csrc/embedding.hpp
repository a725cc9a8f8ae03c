// embedding.hpp -- embedding lookup with scaling, and its gradient.
//
//   Y[t] = scale E[id(t)],  zeros where id(t) lies outside 0 .. vocab - 1
//   dE[v] = R[v] + scale sum over t with id(t) = v of dY[t]
//
// The lookup is a copy: a group of lanes takes a token's columns, eight to a
// lane, several tokens in flight.
//
// The gradient adds the rows of dY that share an id. No atomics: their order
// would change the sums from call to call. Three launches:
//   * order: the tokens sorted by id, tokens of one id in their own order. Each
//     workgroup owns a range of ids, reads all ids (from the L2s: 8 bytes a
//     token against the 8 KiB of its row of dY) and so knows by itself how many
//     come before its range: no workgroup waits for another, and no pass over
//     digits is needed. Its sixteen waves each count, then place, a run of tokens.
//   * sums: the sorted tokens are cut into blocks of a few. A wave takes a block
//     and 512 columns and adds the rows of every id whose tokens begin in its
//     block, to their end; an id with many tokens is instead cut at the blocks'
//     borders, so that a frequent one does not keep a single wave busy, each
//     block leaving an FP32 partial row. Other waves of the launch write the rows
//     that no token has.
//   * joins: the partial rows of the ids that were cut, added in order.
#pragma once

#include "vector8.hpp"

namespace gemm355 {
namespace rows {

constexpr int EMBED_THREADS = 256;

struct EmbedArgs {
    const void *ids;
    const void *e;
    void *y;
    int64_t items;       // groups of `per` tokens times pieces of a row
    int tokens, vocab, cols;
    int lanes_log2;      // lanes side by side in a row: 1 << lanes_log2, of 8 columns each
    int pieces;          // of that many columns in a row
    float scale;
    bool wide;           // 64-bit ids
};

// PER tokens by one group of lanes.
template <class TE, class TY, int PER>
__global__ __launch_bounds__(EMBED_THREADS) void embed_kernel(EmbedArgs p)
{
    const int groups = EMBED_THREADS >> p.lanes_log2;
    const int group = (int)threadIdx.x >> p.lanes_log2, lane = (int)threadIdx.x & ((1 << p.lanes_log2) - 1);
    for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
        const int64_t block = item / p.pieces;
        const int c = 8 * (lane + ((int)(item - block * p.pieces) << p.lanes_log2));
        if (c >= p.cols)
            continue;
        const int64_t t0 = block * groups * PER + group;
        Raw8<TE> row[PER];
        bool in[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t t = t0 + (int64_t)i * groups;
            const int id = t < p.tokens ? id_at(p.ids, p.wide, (size_t)t, p.vocab) : -1;
            in[i] = id >= 0;
            if (in[i])
                row[i].load(p.e, (size_t)id * (size_t)p.cols + (size_t)c);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t t = t0 + (int64_t)i * groups;
            if (t >= p.tokens)
                break;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = in[i] ? p.scale * row[i].get(e) : 0.0f;
            Raw8<TY> out;
            out.set(x);
            out.store(p.y, (size_t)t * (size_t)p.cols + (size_t)c);
        }
    }
}

// ---- gradient ------------------------------------------------------------------

struct EmbedBwdArgs {
    const void *ids;
    const void *dy;
    const void *r;         // or NULL: zeros; may be de itself
    void *de;
    int *start;            // [vocab + 1]: first place of each id among the sorted tokens
    int2 *sorted;          // [tokens]: {id, token}
    float *partial;        // [blocks][2][cols]: of ids that were cut; 0: begun in an earlier block, 1: beginning here
    int tokens, vocab, cols;
    int range;             // ids per workgroup of the order
    int block;             // tokens per block
    int blocks;            // of the sorted tokens (as many as all tokens would need)
    int pieces;            // of 512 columns in a row
    int sum_waves;         // workgroups' waves that add; the rest of the launch fills
    float scale;
    bool wide;
};

constexpr int ORDER_THREADS = 1024, ORDER_WAVES = ORDER_THREADS / 64;
constexpr int ORDER_MAX_RANGE = 512;

__global__ __launch_bounds__(ORDER_THREADS) void embed_order_kernel(EmbedBwdArgs p)
{
    // [id of the range][wave]: first its tokens, then where the next one goes
    __shared__ int count[ORDER_MAX_RANGE * ORDER_WAVES];
    __shared__ int before[ORDER_WAVES], total[ORDER_WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int v0 = (int)blockIdx.x * p.range, range = min(p.range, p.vocab - v0);
    for (int i = threadIdx.x; i < range * ORDER_WAVES; i += ORDER_THREADS)
        count[i] = 0;
    __syncthreads();

    // this wave's run of tokens, whole groups of 64
    const int64_t run = ((int64_t)p.tokens + ORDER_THREADS - 1) / ORDER_THREADS * 64;
    const int64_t first = wave * run, last = min((int64_t)p.tokens, first + run);
    int less = 0;
#pragma unroll 4
    for (int64_t t = first + lane; t < last; t += 64) {
        const int id = id_at(p.ids, p.wide, (size_t)t, p.vocab);
        less += id >= 0 && id < v0;
        if (id >= v0 && id < v0 + range)
            atomicAdd(&count[(id - v0) * ORDER_WAVES + wave], 1);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        less += __shfl_xor(less, d);
    if (lane == 0)
        before[wave] = less;
    __syncthreads();

    // prefix sums over the range's ids and, within an id, over the waves
    int base = 0;
#pragma unroll
    for (int w = 0; w < ORDER_WAVES; ++w)
        base += before[w];
    for (int i0 = 0; i0 < range; i0 += ORDER_THREADS) {
        const int i = i0 + (int)threadIdx.x;
        int mine = 0;
        if (i < range)
#pragma unroll
            for (int w = 0; w < ORDER_WAVES; ++w)
                mine += count[i * ORDER_WAVES + w];
        int upto = mine;     // of the lanes up to this one
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(upto, d);
            upto += lane >= d ? x : 0;
        }
        if (lane == 63)
            total[wave] = upto;
        __syncthreads();
        int at = base + upto - mine;
#pragma unroll
        for (int w = 0; w < ORDER_WAVES; ++w) {
            at += w < wave ? total[w] : 0;
            base += total[w];
        }
        if (i < range) {
            p.start[v0 + i] = at;
#pragma unroll
            for (int w = 0; w < ORDER_WAVES; ++w) {
                const int n = count[i * ORDER_WAVES + w];
                count[i * ORDER_WAVES + w] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0 && v0 + range == p.vocab)
        p.start[p.vocab] = base;

    // place: tokens of one id in their own order
    for (int64_t t0 = first; t0 < last; t0 += 64) {
        const int64_t t = t0 + lane;
        const int id = t < last ? id_at(p.ids, p.wide, (size_t)t, p.vocab) : -1;
        const int i = id >= v0 && id < v0 + range ? id - v0 : -1;
        for (unsigned long long left = __ballot(i >= 0); left != 0;) {
            const int lead = __builtin_ctzll(left);
            const int which = __builtin_amdgcn_readlane(i, lead);
            const unsigned long long same = __ballot(i == which);
            const int at = count[which * ORDER_WAVES + wave];
            if (i == which)
                p.sorted[at + __popcll(same & ((1ull << lane) - 1))] = make_int2(id, (int)t);
            if (lane == lead)
                count[which * ORDER_WAVES + wave] = at + __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next turn reads what this lane wrote
            left &= ~same;
        }
    }
}

// Adds the rows of the sorted tokens a .. b - 1 of one id.
template <class TY>
__device__ inline void embed_add(const EmbedBwdArgs &p, int a, int b, int c, float (&x)[8])
{
    constexpr int AHEAD = 4;
    if (c >= p.cols)
        return;
    int i = a;
    for (; i + AHEAD <= b; i += AHEAD) {
        Raw8<TY> row[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            row[k].load(p.dy, (size_t)p.sorted[i + k].y * (size_t)p.cols + (size_t)c);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] += row[k].get(e);
    }
    for (; i < b; ++i) {
        Raw8<TY> row;
        row.load(p.dy, (size_t)p.sorted[i].y * (size_t)p.cols + (size_t)c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] += row.get(e);
    }
}

// dE[v] from the sum of its rows of dY.
template <class TE>
__device__ inline void embed_finish(const EmbedBwdArgs &p, int v, int c, float (&x)[8])
{
    if (c >= p.cols)
        return;
    const size_t at = (size_t)v * (size_t)p.cols + (size_t)c;
    Raw8<TE> r;
    r.fill(0.0f);
    if (p.r)
        r.load(p.r, at);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = p.scale * x[e] + r.get(e);
    r.set(x);
    r.store(p.de, at);
}

__device__ inline void embed_partial(const EmbedBwdArgs &p, int block, int which, int c, const float (&x)[8])
{
    if (c >= p.cols)
        return;
    Raw8<float> out;
    out.set(x);
    out.store(p.partial, ((size_t)block * 2 + (size_t)which) * (size_t)p.cols + (size_t)c);
}

// An id with more tokens than a block's is cut.
template <class TE, class TY>
__global__ __launch_bounds__(EMBED_THREADS) void embed_sums_kernel(EmbedBwdArgs p)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int at = (int)blockIdx.x * (EMBED_THREADS / 64) + wave, waves = (int)gridDim.x * (EMBED_THREADS / 64);
    if (at >= p.sum_waves) {
        // rows without a token
        if (p.r == p.de)
            return;
        const int64_t items = (int64_t)p.vocab * p.pieces;
        for (int64_t item = at - p.sum_waves; item < items; item += waves - p.sum_waves) {
            const int v = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)v * p.pieces) + 8 * lane;
            if (p.start[v] != p.start[v + 1])
                continue;
            float x[8] = {};
            embed_finish<TE>(p, v, c, x);
        }
        return;
    }
    const int kept = p.start[p.vocab];
    const int64_t items = (int64_t)p.blocks * p.pieces;
    for (int64_t item = at; item < items; item += p.sum_waves) {
        const int b = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)b * p.pieces) + 8 * lane;
        const int64_t begin = (int64_t)b * p.block;
        if (begin >= kept)
            break;
        const int end = (int)min((int64_t)kept, begin + p.block);
        int i = (int)begin;
        const int v0 = p.sorted[i].x;
        if (p.start[v0] < i) {      // begun in an earlier block
            const int stop = p.start[v0 + 1];
            if (stop - p.start[v0] > p.block) {
                float x[8] = {};
                embed_add<TY>(p, i, min(stop, end), c, x);
                embed_partial(p, b, 0, c, x);
            }
            i = stop;
        }
        while (i < end) {
            const int v = p.sorted[i].x, stop = p.start[v + 1];
            float x[8] = {};
            if (stop - i > p.block) {
                embed_add<TY>(p, i, end, c, x);
                embed_partial(p, b, 1, c, x);
            } else {
                embed_add<TY>(p, i, stop, c, x);
                embed_finish<TE>(p, v, c, x);
            }
            i = stop;
        }
    }
}

// Joins the partial rows of the id that was cut and begins in a block: 512
// columns by a workgroup, whose waves each add a run of the blocks.
constexpr int JOIN_THREADS = 512;
template <class TE>
__global__ __launch_bounds__(JOIN_THREADS) void embed_join_kernel(EmbedBwdArgs p)
{
    constexpr int WAVES = JOIN_THREADS / 64;
    __shared__ float part[WAVES][8][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kept = p.start[p.vocab];
    const int64_t items = (int64_t)p.blocks * p.pieces;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int b = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)b * p.pieces) + 8 * lane;
        const int64_t next = ((int64_t)b + 1) * p.block;
        if (next >= kept)
            break;
        const int v = p.sorted[next - 1].x, begin = p.start[v], stop = p.start[v + 1];
        if (stop - begin <= p.block || begin < next - p.block)
            continue;        // not cut, or begun before
        // block b's part, then those of blocks b + 1 .. last
        const int last = (stop - 1) / p.block, parts = last - b + 1, per = (parts + WAVES - 1) / WAVES;
        float x[8] = {};
        if (c < p.cols)
#pragma unroll 4
            for (int k = wave * per; k < min(parts, (wave + 1) * per); ++k) {
                Raw8<float> row;
                row.load(p.partial, ((size_t)(b + k) * 2 + (k == 0 ? 1 : 0)) * (size_t)p.cols + (size_t)c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] += row.get(e);
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[wave][e][lane] = x[e];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] += part[w][e][lane];
            embed_finish<TE>(p, v, c, x);
        }
    }
}

} // namespace rows
} // namespace gemm355
