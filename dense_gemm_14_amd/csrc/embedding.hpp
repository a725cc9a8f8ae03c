// embedding.hpp -- embedding lookup with scaling, and its gradient.
//
//   Y[t] = scale E[id(t)],  zeros where id(t) lies outside 0 .. vocab - 1
//   dE[v] = R[v] + scale sum over t with id(t) = v of dY[t]
//
// The lookup is a copy: a group of lanes takes a token's columns, several tokens in
// flight. 16384 rows of 4096, BF16 to FP32: 67 us, 4.8 TB/s.
//
// The gradient adds the rows of dY that share an id. No atomics: their order
// would change the sums from call to call. Three launches:
//   * order: the tokens sorted by id, tokens of one id in their own order. Each
//     workgroup owns a range of ids, reads all ids (from the L2s: 8 bytes a
//     token against the 8 KiB of its row of dY) and so knows by itself how many
//     come before its range: no workgroup waits for another, and no pass over
//     digits is needed. Its sixteen waves each count, then place, a run of tokens.
//     (From about 100000 tokens on they are dealt out to buckets of ids first, for up to
//     2^20 ids. More tokens of larger tables are ordered as here, in a time that grows with
//     both: 1000000 of 1048577 ids x 64 2140 us.)
//   * sums: the sorted tokens are cut into blocks of a few. A wave takes a block
//     and 512 columns and adds the rows of every id whose tokens begin in its
//     block, to their end; an id with many tokens is instead cut at the blocks'
//     borders, so that a frequent one does not keep a single wave busy, each
//     block leaving an FP32 partial row. Other waves of the launch write the rows
//     that no token has.
//   * joins: the partial rows of the ids that were cut, added in order.
// Bound by memory, mostly by the writing of the table's gradient: 16384 tokens, 128000
// x 4096 BF16 in 219 us (180 of it rows without tokens, at 5.8 TB/s; 33 the sums, at
// 5.9; 5 the joins; 234 with three sets of arrays in turn).
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
    int lanes_log2;      // lanes side by side in a row: 1 << lanes_log2, of embed_width columns each
    int pieces;          // of that many columns in a row
    float scale;
    bool wide;           // 64-bit ids
};

// Columns of a lane: eight BF16 values, or four where FP32 ones are written, so that
// a wave's store is whole lines either way.
constexpr int embed_width(bool fp32) { return fp32 ? 4 : 8; }

// PER tokens by one group of lanes.
template <class TE, class TY, int PER>
__global__ __launch_bounds__(EMBED_THREADS) void embed_kernel(EmbedArgs p)
{
    constexpr int W = embed_width(sizeof(TY) == 4);
    const int groups = EMBED_THREADS >> p.lanes_log2;
    const int group = (int)threadIdx.x >> p.lanes_log2, lane = (int)threadIdx.x & ((1 << p.lanes_log2) - 1);
    for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
        const int64_t block = item / p.pieces;
        const int c = W * (lane + ((int)(item - block * p.pieces) << p.lanes_log2));
        if (c >= p.cols)
            continue;
        const int64_t t0 = block * groups * PER + group;
        typename RawOf<TE, W>::type row[PER];
        int id[PER];
        ids_at<PER>(p.ids, p.wide, t0, groups, p.tokens, p.vocab, id);
        if (p.vocab > 0)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                row[i].load(p.e, (size_t)max(id[i], 0) * (size_t)p.cols + (size_t)c);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t t = t0 + (int64_t)i * groups;
            if (t >= p.tokens)
                break;
            float x[W];
#pragma unroll
            for (int e = 0; e < W; ++e)
                x[e] = id[i] >= 0 ? p.scale * row[i].get(e) : 0.0f;
            typename RawOf<TY, W>::type out;
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
    int order_groups;      // workgroups of the order
    int block;             // tokens per block
    int blocks;            // of the sorted tokens (as many as all tokens would need)
    int pieces;            // of 512 columns in a row
    int sum_waves;         // workgroups' waves that add; the rest of the launch fills
    float scale;
    bool wide;
    // many tokens, ordered by bucket (id >> shift) first
    int *counts;           // [chunks][buckets] tokens of a chunk; then of the chunks before
    int *total;            // [buckets]
    int *bucket_start;     // [buckets + 1]; where a bucket is one id, `start`
    int2 *bucketed;        // [tokens] {id, token} by bucket; where a bucket is one id, `sorted`
    int shift, buckets, chunks;
};

// This lane's eight columns at c of the rows v0 + i, i in `rows`, that no token
// has: R or zeros, several rows at a time.
template <class TE>
__device__ inline void embed_fill(const EmbedBwdArgs &p, int v0, unsigned long long rows, int c)
{
    constexpr int AHEAD = 8;
    if (p.r == p.de)
        return;
    const int cc = min(c, p.cols - 8);
    while (rows != 0) {
        Raw8<TE> r[AHEAD];
        size_t at[AHEAD];
        const int n = min(AHEAD, __popcll(rows));
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            // (past the last row: that one again)
            at[k] = k < n ? (size_t)(v0 + __builtin_ctzll(rows)) * (size_t)p.cols : at[k > 0 ? k - 1 : 0];
            rows = k < n ? rows & (rows - 1) : rows;
            r[k].fill(0.0f);
        }
        if (p.r)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                r[k].load(p.r, at[k] + (size_t)cc);
        if (c < p.cols)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k < n)
                    r[k].store(p.de, at[k] + (size_t)c);
    }
}

constexpr int FILL_ROWS = 16;

// All rows, R or zeros, by threads that go through memory side by side. Few of them,
// four waves a unit: 1 GiB of zeros takes 162 us so, with eight times as many 190 to
// 240, their stores spread over too many of the memory's pages at a time.
constexpr int FILL_THREADS = 256;
template <class TE>
__device__ inline void embed_fill_all(const EmbedBwdArgs &p, int64_t thread, int64_t threads)
{
    constexpr int AHEAD = 4;
    const int64_t n = (int64_t)p.vocab * p.cols, step = 8 * threads;
    if (!p.r) {      // 16 bytes of either type
        u32x4 *out = static_cast<u32x4 *>(p.de);
        for (int64_t i = thread; i < n / (16 / (int)sizeof(TE)); i += threads)
            __builtin_nontemporal_store(u32x4{}, out + i);
        return;
    }
    for (int64_t i = 8 * thread; i < n; i += AHEAD * step) {
        Raw8<TE> r[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            r[k].load(p.r, (size_t)min(i + k * step, n - 8));
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i + k * step < n)
                r[k].store(p.de, (size_t)(i + k * step));
    }
}

constexpr int ORDER_THREADS = 1024, ORDER_WAVES = ORDER_THREADS / 64;
constexpr int ORDER_MAX_RANGE = 512, ORDER_AHEAD = 8;

// The workgroups past a launch's first `first` fill all rows; whether this is one.
template <class TE>
__device__ inline bool embed_fills(const EmbedBwdArgs &p, int first)
{
    if ((int)blockIdx.x < first)
        return false;
    if (threadIdx.x < FILL_THREADS)
        embed_fill_all<TE>(p, ((int64_t)blockIdx.x - first) * FILL_THREADS + threadIdx.x,
                           ((int64_t)gridDim.x - first) * FILL_THREADS);
    return true;
}

// Workgroups from p.order_groups on fill every row, for the sums to write those
// again that have tokens: where those are few, the ordering then costs no time of
// its own (16384 tokens of 128000 ids: 250 us, 219 so). BUCKETED: a workgroup's range
// is a bucket, whose tokens are listed already, and none fills.
template <class TE, bool BUCKETED>
__global__ __launch_bounds__(ORDER_THREADS) void embed_order_kernel(EmbedBwdArgs p)
{
    // [wave][id of the range]: first its tokens, then where the next one goes
    __shared__ int count[ORDER_WAVES][ORDER_MAX_RANGE];
    __shared__ int before[ORDER_WAVES], total[ORDER_WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (!BUCKETED && embed_fills<TE>(p, p.order_groups))
        return;
    const int v0 = (int)blockIdx.x * p.range, range = min(p.range, p.vocab - v0);
    for (int i = threadIdx.x; i < ORDER_MAX_RANGE * ORDER_WAVES; i += ORDER_THREADS)
        (&count[0][0])[i] = 0;
    __syncthreads();

    // this wave's run of tokens, whole groups of 64
    const int64_t from = BUCKETED ? p.bucket_start[blockIdx.x] : 0, to = BUCKETED ? p.bucket_start[blockIdx.x + 1] : p.tokens;
    const int64_t run = (to - from + ORDER_THREADS - 1) / ORDER_THREADS * 64;
    const int64_t first = from + wave * run, last = min(to, first + run);
    // (loads of eight groups at a time: one after the other they took the time)
    auto each_group = [&](auto &&f) {
        for (int64_t t0 = first; t0 < last; t0 += 64 * ORDER_AHEAD) {
            int id[ORDER_AHEAD], token[ORDER_AHEAD];
            if constexpr (BUCKETED) {
#pragma unroll
                for (int k = 0; k < ORDER_AHEAD; ++k) {
                    const int64_t i = t0 + 64 * k + lane;
                    const int2 x = i < last ? p.bucketed[i] : make_int2(-1, 0);
                    id[k] = x.x;
                    token[k] = x.y;
                }
            } else {
                ids_at<ORDER_AHEAD>(p.ids, p.wide, t0 + lane, 64, last, p.vocab, id);
#pragma unroll
                for (int k = 0; k < ORDER_AHEAD; ++k)
                    token[k] = (int)(t0 + 64 * k) + lane;
            }
#pragma unroll
            for (int k = 0; k < ORDER_AHEAD; ++k)
                f(token[k], id[k]);
        }
    };
    int less = 0;
    each_group([&](int, int id) {
        less += id >= 0 && id < v0;
        if (id >= v0 && id < v0 + range)
            atomicAdd(&count[wave][id - v0], 1);
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        less += __shfl_xor(less, d);
    if (lane == 0)
        before[wave] = less;
    __syncthreads();

    // prefix sums over the range's ids and, within an id, over the waves
    int base = BUCKETED ? (int)from : 0;
    if constexpr (!BUCKETED)
#pragma unroll
        for (int w = 0; w < ORDER_WAVES; ++w)
            base += before[w];
    for (int i0 = 0; i0 < range; i0 += ORDER_THREADS) {
        const int i = i0 + (int)threadIdx.x;
        int mine = 0;
        if (i < range)
#pragma unroll
            for (int w = 0; w < ORDER_WAVES; ++w)
                mine += count[w][i];
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
                const int n = count[w][i];
                count[w][i] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0 && v0 + range == p.vocab)
        p.start[p.vocab] = base;

    // place: tokens of one id in their own order
    each_group([&](int t, int id) {
        const int i = id >= v0 && id < v0 + range ? id - v0 : -1;
        for (unsigned long long left = __ballot(i >= 0); left != 0;) {
            const int lead = __builtin_ctzll(left);
            const int which = __builtin_amdgcn_readlane(i, lead);
            const unsigned long long same = __ballot(i == which);
            const int at = count[wave][which];
            if (i == which)
                p.sorted[at + __popcll(same & ((1ull << lane) - 1))] = make_int2(id, t);
            if (lane == lead)
                count[wave][which] = at + __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next turn reads what this lane wrote
            left &= ~same;
        }
    });
}

// Many tokens: with all ids read by every workgroup, the order would take longer than
// the rows (1048576 tokens of as many ids x 64: 2020 us, 181 so). They are then dealt out to buckets of neighbouring ids, in their own order,
// which takes three launches that read them twice in all: the tokens of each chunk
// and bucket counted, the counts added up over the chunks, the tokens placed. Buckets
// of one id are then in order, others are ordered as above, each by a workgroup.
constexpr int CHUNK = 4096, CHUNK_AHEAD = CHUNK / ORDER_THREADS, BUCKETS_LOG2 = 11, MAX_BUCKETS = 1 << BUCKETS_LOG2;

// This wave's tokens of chunk blockIdx.x, 64 for each k.
__device__ inline int64_t chunk_first(int wave, int lane) { return (int64_t)blockIdx.x * CHUNK + wave * (CHUNK / ORDER_WAVES) + lane; }

template <class TE>
__global__ __launch_bounds__(ORDER_THREADS) void embed_count_kernel(EmbedBwdArgs p)
{
    __shared__ int count[MAX_BUCKETS];
    if (embed_fills<TE>(p, p.chunks))
        return;
    int id[CHUNK_AHEAD];
    ids_at<CHUNK_AHEAD>(p.ids, p.wide, (int64_t)blockIdx.x * CHUNK + threadIdx.x, ORDER_THREADS, p.tokens, p.vocab, id);
    for (int b = threadIdx.x; b < p.buckets; b += ORDER_THREADS)
        count[b] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < CHUNK_AHEAD; ++k)
        if (id[k] >= 0)
            atomicAdd(&count[id[k] >> p.shift], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < p.buckets; b += ORDER_THREADS)
        p.counts[(size_t)blockIdx.x * (size_t)p.buckets + (size_t)b] = count[b];
}

// 64 buckets a workgroup; its waves take sixteen chunks each at a time.
__global__ __launch_bounds__(ORDER_THREADS) void embed_scan_kernel(EmbedBwdArgs p)
{
    constexpr int AHEAD = 16;
    __shared__ int part[ORDER_WAVES][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int b = (int)blockIdx.x * 64 + lane;
    int base = 0;
    for (int64_t c0 = 0; c0 < p.chunks; c0 += AHEAD * ORDER_WAVES) {
        const int64_t c = c0 + AHEAD * wave;
        int n[AHEAD], sum = 0;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            n[k] = b < p.buckets && c + k < p.chunks ? p.counts[(size_t)(c + k) * (size_t)p.buckets + (size_t)b] : 0;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            sum += n[k];
        part[wave][lane] = sum;
        __syncthreads();
        int at = base;
#pragma unroll
        for (int w = 0; w < ORDER_WAVES; ++w) {
            at += w < wave ? part[w][lane] : 0;
            base += part[w][lane];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (b < p.buckets && c + k < p.chunks)
                p.counts[(size_t)(c + k) * (size_t)p.buckets + (size_t)b] = at;
            at += n[k];
        }
        __syncthreads();
    }
    if (wave == 0 && b < p.buckets)
        p.total[b] = base;
}

__global__ __launch_bounds__(ORDER_THREADS) void embed_place_kernel(EmbedBwdArgs p)
{
    constexpr int PER = MAX_BUCKETS / ORDER_THREADS;
    // [wave][bucket]: first its tokens, then where the next one goes
    __shared__ int count[ORDER_WAVES][MAX_BUCKETS];
    __shared__ int total[ORDER_WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int id[CHUNK_AHEAD];
    ids_at<CHUNK_AHEAD>(p.ids, p.wide, chunk_first(wave, lane), 64, p.tokens, p.vocab, id);
    // this thread's buckets: their tokens, and those of the chunks before
    int all[PER], earlier[PER], mine = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int b = PER * tid + k;
        all[k] = b < p.buckets ? p.total[b] : 0;
        earlier[k] = b < p.buckets ? p.counts[(size_t)blockIdx.x * (size_t)p.buckets + (size_t)b] : 0;
        mine += all[k];
    }
    for (int i = tid; i < MAX_BUCKETS * ORDER_WAVES; i += ORDER_THREADS)
        (&count[0][0])[i] = 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int x = __shfl_up(upto, d);
        upto += lane >= d ? x : 0;
    }
    if (lane == 63)
        total[wave] = upto;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < CHUNK_AHEAD; ++k)
        if (id[k] >= 0)
            atomicAdd(&count[wave][id[k] >> p.shift], 1);
    int at = upto - mine, kept = 0;
#pragma unroll
    for (int w = 0; w < ORDER_WAVES; ++w) {
        at += w < wave ? total[w] : 0;
        kept += total[w];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int b = PER * tid + k;
        if (blockIdx.x == 0 && b < p.buckets)
            p.bucket_start[b] = at;
        int next = at + earlier[k];
#pragma unroll
        for (int w = 0; w < ORDER_WAVES; ++w) {
            const int n = count[w][b];
            count[w][b] = next;
            next += n;
        }
        at += all[k];
    }
    if (blockIdx.x == 0 && tid == 0)
        p.bucket_start[p.buckets] = kept;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < CHUNK_AHEAD; ++k) {
        // the lanes whose tokens share a bucket, a bit of its number at a time
        const int b = max(id[k], 0) >> p.shift;
        unsigned long long same = __ballot(id[k] >= 0);
#pragma unroll
        for (int i = 0; i < BUCKETS_LOG2; ++i) {
            const bool bit = b >> i & 1;
            const unsigned long long with = __ballot(bit);
            same &= bit ? with : ~with;
        }
        if (id[k] >= 0) {
            const int next = count[wave][b], rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
            p.bucketed[next + rank] = make_int2(id[k], (int)chunk_first(wave, lane) + 64 * k);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // all have read it
            if (rank == n - 1)
                count[wave][b] = next + n;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // the next turn reads what these lanes wrote
    }
}

// x += the rows of dY of the tokens token(0) .. token(n - 1), asked for in that
// order; after(i) once row i is in. (Rows past the last are the last again: a load
// under a condition would wait for the one before.)
template <class TY, class Token, class After>
__device__ inline void embed_add(const EmbedBwdArgs &p, int n, int c, float (&x)[8], Token &&token, After &&after)
{
    constexpr int AHEAD = 8;
    const int cc = min(c, p.cols - 8);
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        Raw8<TY> row[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            row[k].load(p.dy, (size_t)token(min(i0 + k, n - 1)) * (size_t)p.cols + (size_t)cc);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i0 + k < n) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] += row[k].get(e);
                after(i0 + k);
            }
    }
}

// dE[v] from the sum of its rows of dY.
template <class TE>
__device__ inline void embed_finish(const EmbedBwdArgs &p, int v, int c, const float (&x)[8])
{
    if (c >= p.cols)
        return;
    const size_t at = (size_t)v * (size_t)p.cols + (size_t)c;
    Raw8<TE> r;
    r.fill(0.0f);
    if (p.r)
        r.load(p.r, at);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        y[e] = p.scale * x[e] + r.get(e);
    r.set(y);
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

// An id with more tokens than a block's (at most 32) is cut.
constexpr int SUMS_BLOCK = 32;
template <class TE, class TY>
__global__ __launch_bounds__(EMBED_THREADS) void embed_sums_kernel(EmbedBwdArgs p)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int at = (int)blockIdx.x * (EMBED_THREADS / 64) + wave, waves = (int)gridDim.x * (EMBED_THREADS / 64);
    if (at >= p.sum_waves) {
        // rows without a token
        const int64_t items = (((int64_t)p.vocab + FILL_ROWS - 1) / FILL_ROWS) * p.pieces;
        for (int64_t item = at - p.sum_waves; item < items; item += waves - p.sum_waves) {
            const int group = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)group * p.pieces) + 8 * lane;
            const int v0 = group * FILL_ROWS, v = min(v0 + lane, p.vocab), next = p.start[min(v + 1, p.vocab)];
            embed_fill<TE>(p, v0, __ballot(lane < FILL_ROWS && v < p.vocab && p.start[v] == next), c);
        }
        return;
    }
    const int kept = p.start[p.vocab];
    const int64_t items = (int64_t)p.blocks * p.pieces;
    for (int64_t item = at; item < items; item += p.sum_waves) {
        const int b = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)b * p.pieces) + 8 * lane;
        if ((int64_t)b * p.block >= kept)
            break;
        const int begin = b * p.block, n = min(kept - begin, p.block);
        // lane l: sorted token begin + l, two blocks' worth: an id that is not cut
        // ends within them
        int2 mine = make_int2(-1, 0);
        if (lane < kept - begin)
            mine = p.sorted[begin + lane];
        auto id_of = [&](int i) { return __builtin_amdgcn_readlane(mine.x, i); };
        auto token_of = [&](int i) { return __builtin_amdgcn_readlane(mine.y, i); };
        const int v0 = id_of(0), v1 = id_of(n - 1);
        const int start0 = p.start[v0], stop0 = p.start[v0 + 1], start1 = p.start[v1], stop1 = p.start[v1 + 1];
        int i = 0, end = stop1 - begin;          // of the ids that are added up here
        if (start0 < begin) {                    // begun in an earlier block
            const int stop = min(stop0 - begin, n);
            if (stop0 - start0 > p.block) {
                float x[8] = {};
                embed_add<TY>(p, stop, c, x, token_of, [](int) {});
                embed_partial(p, b, 0, c, x);
            }
            i = stop0 - begin;
        }
        if (i >= n)
            continue;
        if (stop1 - start1 > p.block) {          // goes on into the next blocks
            end = start1 - begin;
            float x[8] = {};
            embed_add<TY>(p, n - end, c, x, [&](int k) { return token_of(end + k); }, [](int) {});
            embed_partial(p, b, 1, c, x);
        }
        float x[8] = {};
        embed_add<TY>(p, end - i, c, x, [&](int k) { return token_of(i + k); },
                      [&](int k) {
                          const int v = id_of(i + k);
                          if (i + k + 1 == end || id_of(i + k + 1) != v) {
                              embed_finish<TE>(p, v, c, x);
#pragma unroll
                              for (int e = 0; e < 8; ++e)
                                  x[e] = 0.0f;
                          }
                      });
    }
}

// Joins the partial rows of the ids that were cut: a workgroup takes 512 columns
// of the ids that begin in JOIN_BLOCKS blocks, one after the other, its waves each
// a run of an id's blocks.
constexpr int JOIN_THREADS = 512, JOIN_BLOCKS = 8;
template <class TE>
__global__ __launch_bounds__(JOIN_THREADS) void embed_join_kernel(EmbedBwdArgs p)
{
    constexpr int WAVES = JOIN_THREADS / 64;
    __shared__ float part[WAVES][8][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kept = p.start[p.vocab];
    const int64_t items = (((int64_t)p.blocks + JOIN_BLOCKS - 1) / JOIN_BLOCKS) * p.pieces;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int group = (int)(item / p.pieces), c = 512 * (int)(item - (int64_t)group * p.pieces) + 8 * lane;
        const int b0 = group * JOIN_BLOCKS;
        // lane l < JOIN_BLOCKS: whether an id is cut that begins in block b0 + l
        const int64_t next = ((int64_t)b0 + lane + 1) * p.block;
        int v = 0, begin = 0, stop = 0;
        if (lane < JOIN_BLOCKS && next < kept) {
            v = p.sorted[next - 1].x;
            begin = p.start[v];
            stop = p.start[v + 1];
        }
        const bool cut = stop - begin > p.block && begin >= next - p.block;
        for (unsigned long long left = __ballot(cut); left != 0; left &= left - 1) {
            const int l = __builtin_ctzll(left), b = b0 + l;
            // block b's part, then those of blocks b + 1 .. last
            const int last = (__builtin_amdgcn_readlane(stop, l) - 1) / p.block, parts = last - b + 1;
            const int per = (parts + WAVES - 1) / WAVES;
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
                embed_finish<TE>(p, __builtin_amdgcn_readlane(v, l), c, x);
            }
        }
    }
}

// ---- few tokens ----------------------------------------------------------------
//
// Up to 1024 tokens take one launch: a workgroup owns a range of ids and 512
// columns, lists the tokens of its ids, and writes its rows, with and without
// tokens. An id with more than a few tokens is added up by its four waves. 777 tokens,
// 32001 x 1000 in 27 us with the gradient it is added to in another array (the three
// launches 34, and two gaps).
constexpr int FEW_TOKENS = 1024, FEW_RANGE = 512, FEW_CUT = 16;

template <class TE, class TY>
__global__ __launch_bounds__(EMBED_THREADS) void embed_few_kernel(EmbedBwdArgs p)
{
    constexpr int WAVES = EMBED_THREADS / 64, GROUPS = FEW_TOKENS / EMBED_THREADS;
    __shared__ int token[FEW_TOKENS], which[FEW_TOKENS], count[FEW_RANGE], before[GROUPS][WAVES];
    __shared__ float part[WAVES][8][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int owner = (int)blockIdx.x / p.pieces, c = 512 * ((int)blockIdx.x - owner * p.pieces) + 8 * lane;
    const int v0 = owner * p.range, range = min(p.range, p.vocab - v0);

    // the tokens of the range's ids, in order
    int id[GROUPS];
    unsigned long long in[GROUPS];
    ids_at<GROUPS>(p.ids, p.wide, tid, EMBED_THREADS, p.tokens, p.vocab, id);
    for (int i = tid; i < range; i += EMBED_THREADS)
        count[i] = 0;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
        id[k] -= v0;
        in[k] = __ballot(id[k] >= 0 && id[k] < range);
        if (lane == 0)
            before[k][wave] = __popcll(in[k]);
    }
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k)
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            if (w == wave && (in[k] >> lane & 1)) {
                const int place = at + __popcll(in[k] & ((1ull << lane) - 1));
                token[place] = k * EMBED_THREADS + tid;
                which[place] = id[k];
                atomicAdd(&count[id[k]], 1);
            }
            at += before[k][w];
        }
    const int listed = at;
    __syncthreads();

    // x += the tokens of id v0 + i that are among its from-th to its to-th
    auto add = [&](int i, int from, int to, float (&x)[8]) {
        int seen = 0;
        for (int l0 = 0; l0 < listed && seen < to; l0 += 64) {
            const int l = l0 + lane;
            unsigned long long of_id = __ballot(l < listed && which[min(l, FEW_TOKENS - 1)] == i);
            const int n = __popcll(of_id);
            const int skip = min(n, max(0, from - seen));
            for (int k = 0; k < skip; ++k)
                of_id &= of_id - 1;
            const int take = min(n, to - seen) - skip, mine = token[min(l, FEW_TOKENS - 1)];
            unsigned long long rest = of_id;
            // (the matches one after the other, as their rows are asked for)
            int asked = 0, t = 0;
            embed_add<TY>(p, max(take, 0), c, x, [&](int k) {
                if (asked <= k) {
                    t = __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest));
                    rest &= rest - 1;
                    ++asked;
                }
                return t;
            }, [](int) {});
            seen += n;
        }
    };
    for (int i0 = 64 * wave; i0 < range; i0 += 64 * WAVES) {
        const int n = i0 + lane < range ? count[i0 + lane] : -1;
        embed_fill<TE>(p, v0 + i0, __ballot(n == 0), c);
        for (unsigned long long left = __ballot(n > 0 && n <= FEW_CUT); left != 0; left &= left - 1) {
            const int l = __builtin_ctzll(left);
            float x[8] = {};
            add(i0 + l, 0, __builtin_amdgcn_readlane(n, l), x);
            embed_finish<TE>(p, v0 + i0 + l, c, x);
        }
    }
    if (listed <= FEW_CUT)
        return;
    for (int i0 = 0; i0 < range; i0 += 64) {
        const int n = i0 + lane < range ? count[i0 + lane] : -1;
        for (unsigned long long left = __ballot(n > FEW_CUT); left != 0; left &= left - 1) {
            const int l = __builtin_ctzll(left), all = __builtin_amdgcn_readlane(n, l), per = (all + WAVES - 1) / WAVES;
            float x[8] = {};
            add(i0 + l, wave * per, min(all, (wave + 1) * per), x);
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
                embed_finish<TE>(p, v0 + i0 + l, c, x);
            }
        }
    }
}

} // namespace rows
} // namespace gemm355
