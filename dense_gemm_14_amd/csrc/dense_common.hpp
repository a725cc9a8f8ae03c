// dense_common.hpp -- pieces shared by the kernels of the dense layer's fused
// operators (linear and gated layers, their gradients, Newton-Schulz): operand
// layouts, LDS-DMA copies, activations with their derivatives, and epilogues.
//
// The products are C = op(A) op(B)^T with the contraction over K:
//   ROW_K  the operand is stored (rows x K), K contiguous: a fragment's eight
//          K elements are 16 consecutive bytes;
//   COL_K  it is stored (K x rows), rows contiguous, as the weights of an
//          input gradient (dZ B) and both operands of a weight gradient
//          (dZ^T A) are. gfx950's transposing LDS read (ds_read_b64_tr_b16)
//          gathers a fragment's K elements, so no operand is transposed in
//          memory first.
#pragma once

#include "common.hpp"

namespace gemm355 {
namespace dense {

enum Layout { ROW_K = 0, COL_K = 1 };
enum Epilogue {
    EPI_STORE = 0,   // C = round(alpha acc)
    EPI_LINEAR = 1,  // z = acc + bias, Z = round(z) if wanted, C = round(act(z) + R)
    EPI_GATED = 2,   // gate and up sums of one column: C = round(act(zg) zu), Z = round of both if wanted
    EPI_STORE_SYM = 3,   // EPI_STORE of a symmetric product: tiles on and below the diagonal, FP16,
                         // those below it stored a second time, mirrored
    EPI_POLY = 4         // C = round(alpha acc + beta R + gamma [row == column]), symmetric likewise
};
// Activations (the values of gemm355_activation).
enum { A_NONE = 0, A_RELU = 1, A_GELU = 2, A_SILU = 3 };

struct DenseArgs {
    const void *a, *b;
    void *c;
    const void *r;       // residual (EPI_LINEAR: BF16, may be NULL or c itself), second term (EPI_POLY: FP16)
    void *z;             // EPI_LINEAR, EPI_GATED: pre-activations, or NULL
    const void *bias;    // EPI_LINEAR: N, EPI_GATED: 2 N BF16 values, or NULL
    float *ws;           // split K: FP32 partial tiles
    int M, N, K;         // C is M x N (EPI_GATED: B has 2 N rows)
    int tiles_m, tiles_n, tiles;   // tiles: per batch entry (symmetric: on and below the diagonal)
    int whole;           // tiles (over the batch) that one workgroup each runs whole; the K steps of
    int splits, steps_per_split;   // the tiles after them are split
    int supergroup;
    int act;
    int batch;
    int grid;            // workgroups of a round
    float alpha, beta, gamma;
};

// Asks for all arguments at the kernel's start, at once: left to the compiler
// they are fetched in three dependent steps, which a product of a few
// microseconds notices.
__device__ inline void fetch_args(const DenseArgs &p)
{
    asm volatile("" ::"s"(p.a), "s"(p.b), "s"(p.c), "s"(p.r), "s"(p.z), "s"(p.bias), "s"(p.M), "s"(p.N), "s"(p.K),
                 "s"(p.tiles_m), "s"(p.tiles_n), "s"(p.tiles), "s"(p.whole), "s"(p.splits), "s"(p.supergroup), "s"(p.act),
                 "s"(p.batch), "s"(p.grid));
}

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <class T> struct Frag;
template <> struct Frag<__bf16> {
    typedef bf16x8 type;
    static __device__ inline f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Frag<_Float16> {
    typedef f16x8 type;
    static __device__ inline f32x4 mma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// Four elements of a transposed fragment. The 16 lanes of a group hand in the
// addresses of four K rows (lane j: row j / 4, 8-byte piece j % 4 of its 32
// bytes); lane j receives column j of those four rows.
__device__ inline s16x4 read_tr(unsigned lds_addr)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)lds_addr);
}

__device__ inline i32x4 rsrc_words(const void *p, unsigned bytes)
{
    const unsigned long long a = reinterpret_cast<unsigned long long>(p);
    return i32x4{(int)(unsigned)a, (int)(unsigned)(a >> 32), (int)bytes, (int)RSRC_WORD3};
}

__device__ inline void wait_all_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
template <int N>
__device__ inline void wait_copies_le() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ inline void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ---- global -> LDS copies ----------------------------------------------------

// Buffer offset past every range (extents are below 2^31), after any
// instruction offset too.
constexpr unsigned OFF_NONE = 0xFFFF0000u;
constexpr int NEVER = 1 << 30;   // K offset past every K
// The resources start COPY_SHIFT bytes early, so that a lane's offset less the
// second copy's instruction offset (1024) is never negative.
constexpr int COPY_SHIFT = 1024;

// Two 1 KiB global -> LDS copies: lane i's 16 bytes at buffer offset v0 (v1 +
// 1024) land at lds_addr (+ 1024) + 16 i. Inline assembly, so that the compiler
// does not order every later LDS read after the LDS writes in flight; the
// kernel orders them with vmcnt waits and barriers. The s_nop: an LDS-DMA
// instruction must not directly follow a scalar write of m0.
__device__ inline void copy_two(const i32x4 &rsrc, unsigned lds_addr, unsigned v0, unsigned v1)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t"
                 "buffer_load_dwordx4 %1, %3, 0 offen offset:0 lds\n\t"
                 "buffer_load_dwordx4 %2, %3, 0 offen offset:1024 lds"
                 :
                 : "s"(lds_addr), "v"(v0), "v"(v1), "s"(rsrc)
                 : "memory", "m0");
}

// LDS places of the 16-byte chunks of a 128-byte ROW_K row, and of the 32-byte
// segments of a COL_K K row of 256 bytes or more.
__device__ inline int swizzle_row(int r, int c) { return c ^ ((r >> 1) & 7); }
__device__ inline int key_col(int k) { return (k & 3) | ((k >> 1) & 4); }

// ---- activations -----------------------------------------------------------
//
// Both gated-linear activations are z sigma(w(z)): w = z for SiLU and
// w = 2 sqrt(2/pi) (z + 0.044715 z^3) for the tanh GELU, sigma the logistic
// function, evaluated with the hardware's exponential and reciprocal (about
// one part in 10^6, far below the 16-bit roundings that follow). Their
// derivative is sigma + z sigma (1 - sigma) w'.
constexpr float GELU_C0 = 1.5957691216f;   // 2 sqrt(2/pi)
constexpr float GELU_C1 = 0.0713548163f;   // 2 sqrt(2/pi) 0.044715

template <int ACT>
__device__ inline float act_value(float z)
{
    if constexpr (ACT == A_RELU)
        return z > 0.0f ? z : 0.0f;
    if constexpr (ACT == A_GELU)
        return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z * (GELU_C0 + GELU_C1 * z * z)));
    if constexpr (ACT == A_SILU)
        return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    return z;
}

// act(z) in *value and act'(z) as the result.
template <int ACT>
__device__ inline float act_slope(float z, float *value)
{
    if constexpr (ACT == A_RELU) {
        *value = z > 0.0f ? z : 0.0f;
        return z > 0.0f ? 1.0f : 0.0f;
    }
    if constexpr (ACT == A_GELU) {
        // past |z| = 12 sigma is 0 or 1 in FP32 and the slope with it; the
        // clamp keeps z^3 finite there
        const float y = fminf(fmaxf(z, -12.0f), 12.0f);
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-y * (GELU_C0 + GELU_C1 * y * y)));
        *value = z * s;
        return s + y * s * (1.0f - s) * (GELU_C0 + 3.0f * GELU_C1 * y * y);
    }
    if constexpr (ACT == A_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
        *value = z * s;
        return s + z * s * (1.0f - s);
    }
    *value = z;
    return 1.0f;
}

// f(Int<ACT>{}) for the activation chosen at run time (uniform).
template <class F>
__device__ inline void with_act(int act, F &&f)
{
    switch (act) {
    case A_RELU: f(Int<A_RELU>{}); break;
    case A_GELU: f(Int<A_GELU>{}); break;
    case A_SILU: f(Int<A_SILU>{}); break;
    default: f(Int<A_NONE>{}); break;
    }
}

// ---- tile order ------------------------------------------------------------

// Tile p of a symmetric result: rows of tiles, the diagonal last.
__device__ inline void triangle_tile(int p, int &tm, int &tn)
{
    int t = (int)((__builtin_sqrtf(8.0f * (float)p + 1.0f) - 1.0f) * 0.5f);
    while (t * (t + 1) / 2 > p)   // the square root is off by one at most
        --t;
    while ((t + 1) * (t + 2) / 2 <= p)
        ++t;
    tm = t;
    tn = p - t * (t + 1) / 2;
}

template <int EPI>
__device__ inline void dense_tile(const DenseArgs &p, int pos, int &tm, int &tn)
{
    if constexpr (EPI >= EPI_STORE_SYM)
        triangle_tile(pos, tm, tn);
    else
        supergroup_tile(pos, p.tiles_m, p.tiles_n, p.supergroup, tm, tn);
}

// A work item: a tile of a batch entry and, for the tiles whose K is split
// (those from `whole` on), its part. Items come in rounds of p.grid; the tail's
// are ordered split by split, so that the workgroups of one round that share
// operand strips also read the same K range of them at the same time.
struct WorkItem {
    int tile, split;
};
__device__ inline int work_items(const DenseArgs &p)
{
    return p.whole + (p.tiles * p.batch - p.whole) * p.splits;
}
__device__ inline WorkItem work_item(const DenseArgs &p, int item)
{
    if (item < p.whole)
        return WorkItem{item, 0};
    const int tail = p.tiles * p.batch - p.whole, q = item - p.whole;
    return WorkItem{p.whole + q % tail, q / tail};
}

// The arguments of batch entry `b`: every array advanced by its own size.
__device__ inline void enter_batch(DenseArgs &p, int b)
{
    const size_t i = (size_t)b;
    p.a = static_cast<const uint8_t *>(p.a) + i * (size_t)p.M * (size_t)p.K * 2;
    p.b = static_cast<const uint8_t *>(p.b) + i * (size_t)p.N * (size_t)p.K * 2;
    p.c = static_cast<uint8_t *>(p.c) + i * (size_t)p.M * (size_t)p.N * 2;
    if (p.r)
        p.r = static_cast<const uint8_t *>(p.r) + i * (size_t)p.M * (size_t)p.N * 2;
}

// ---- epilogues -------------------------------------------------------------
//
// The matrix instruction is fed B rows as its first operand and A rows as its
// second, so lane (l16, grp) of a 16 x 16 block holds C[m][n .. n + 3],
// m = row + l16, n = column + 4 grp. v_permlane16_swap of two neighbouring
// blocks x, y (columns c .. c + 15 and c + 16 .. c + 31) leaves each lane with
// eight consecutive columns, c + 16 (grp & 1) + 8 (grp >> 1): one 16-byte
// access. The swap is its own inverse, so 16 bytes loaded at that place turn
// back into the two blocks' four columns each.

template <class T> __device__ inline unsigned pack2(float lo, float hi);
template <> __device__ inline unsigned pack2<__bf16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <> __device__ inline unsigned pack2<_Float16>(float lo, float hi)
{
    f32x2 v = {lo, hi};
    return __builtin_bit_cast(unsigned, __builtin_convertvector(v, f16x2));   // round to nearest even
}
template <class T> __device__ inline f32x2 unpack2(unsigned w);
template <> __device__ inline f32x2 unpack2<__bf16>(unsigned w) { return f32x2{bf16_lo(w), bf16_hi(w)}; }
template <> __device__ inline f32x2 unpack2<_Float16>(unsigned w)
{
    return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);
}

template <class T>
__device__ inline u32x4 pack_pair(f32x4 x, f32x4 y)
{
    const auto s0 = __builtin_amdgcn_permlane16_swap(pack2<T>(x[0], x[1]), pack2<T>(y[0], y[1]), false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(pack2<T>(x[2], x[3]), pack2<T>(y[2], y[3]), false, false);
    return u32x4{s0[0], s1[0], s0[1], s1[1]};
}

template <class T>
__device__ inline void unpack_pair(u32x4 w, f32x4 &x, f32x4 &y)
{
    const auto s0 = __builtin_amdgcn_permlane16_swap(w[0], w[2], false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(w[1], w[3], false, false);
    const f32x2 x0 = unpack2<T>(s0[0]), x1 = unpack2<T>(s1[0]), y0 = unpack2<T>(s0[1]), y1 = unpack2<T>(s1[1]);
    x = f32x4{x0[0], x0[1], x1[0], x1[1]};
    y = f32x4{y0[0], y0[1], y1[0], y1[1]};
}

__device__ inline f32x4 add_bias(f32x4 x, u32x2 w)
{
    return f32x4{x[0] + bf16_lo(w[0]), x[1] + bf16_hi(w[0]), x[2] + bf16_lo(w[1]), x[3] + bf16_hi(w[1])};
}

template <int ACT>
__device__ inline f32x4 act4(f32x4 x)
{
    return f32x4{act_value<ACT>(x[0]), act_value<ACT>(x[1]), act_value<ACT>(x[2]), act_value<ACT>(x[3])};
}

// The epilogue's view of the arrays (each resource ends at its array's last
// byte; a NULL array's range is empty, so its loads give zeros and its stores
// do nothing).
struct Views {
    __amdgpu_buffer_rsrc_t c, r, z, bias;
};

template <int EPI>
__device__ inline Views make_views(const DenseArgs &p)
{
    constexpr unsigned W = EPI == EPI_GATED ? 2 : 1;
    const unsigned mn = (unsigned)p.M * (unsigned)p.N * 2u;
    return Views{make_rsrc(p.c, mn), make_rsrc(p.r, p.r ? mn : 0u), make_rsrc(p.z, p.z ? W * mn : 0u),
                 make_rsrc(p.bias, p.bias ? W * (unsigned)p.N * 2u : 0u)};
}

// Offset in bytes of this lane's eight columns of the block pair at column
// `col` in row m of an array `width` columns wide; OOB outside C.
__device__ inline int pair_offset(const DenseArgs &p, int m, int col, int width, int shift, int lane)
{
    const int grp = lane >> 4;
    const int n = col + 16 * (grp & 1) + 8 * (grp >> 1);
    return m < p.M && n < p.N ? (int)(((unsigned)m * (unsigned)width + (unsigned)(n + shift)) * 2u) : OOB;
}

// The epilogue's variant: f(Int<activation>{}, Int<EXTRA>{}), EXTRA: there is a
// bias, a residual or Z. Chosen once per tile, so that the rows' code has no
// branches (with them, 256 x 256 tiles spilled, and the reloads waited for the
// stores before them: 12 us a tile, of 90).
template <int EPI, class F>
__device__ inline void with_epilogue(const DenseArgs &p, F &&f)
{
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_GATED) {
        with_act(p.act, [&](auto act_c) {
            if (p.bias || p.z || p.r)
                f(act_c, Int<1>{});
            else
                f(act_c, Int<0>{});
        });
    } else {
        f(Int<A_NONE>{}, Int<EPI == EPI_POLY>{});
    }
}

// What a row of BJ blocks at column `col` reads besides its sums: the bias of
// each block's columns (the same for every row; zeros without one) ...
template <int EPI, int EXTRA, int BJ>
__device__ inline void load_bias_row(const DenseArgs &p, const Views &v, int col, int lane, u32x2 (&bias)[BJ])
{
    if constexpr (EXTRA && (EPI == EPI_LINEAR || EPI == EPI_GATED)) {
        constexpr int H = EPI == EPI_GATED ? BJ / 2 : BJ;
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            // EPI_GATED: the up columns' bias starts at N
            const int n = col + 16 * (j % H) + 4 * (lane >> 4);
            const int off = n < p.N ? (n + (j < H ? 0 : p.N)) * 2 : OOB;
            bias[j] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(v.bias, off, 0, 0));
        }
    }
}

// ... and the row's residual (EPI_LINEAR) or second term (EPI_POLY); zeros
// without one.
template <int EPI, int EXTRA, int BJ>
__device__ inline void load_res_row(const DenseArgs &p, const Views &v, int m, int col, int lane, u32x4 (&res)[BJ / 2])
{
    if constexpr (EXTRA && (EPI == EPI_LINEAR || EPI == EPI_POLY))
#pragma unroll
        for (int j = 0; j < BJ / 2; ++j)
            res[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   v.r, pair_offset(p, m, col + 32 * j, p.N, 0, lane), 0, 0));
}

__device__ inline void store16(u32x4 w, const __amdgpu_buffer_rsrc_t &r, int off)
{
    __builtin_amdgcn_raw_buffer_store_b128(w, r, off, 0, 0);
}

// A finished row of blocks, packed as it is stored: pairs of blocks of C, and
// of Z (EPI_GATED: the gate's pairs, then the up's).
template <int EPI, int BJ>
struct PackedRow {
    static constexpr int C = EPI == EPI_GATED ? BJ / 4 : BJ / 2;
    u32x4 c[C], z[BJ / 2];
};

// The epilogue's arithmetic for one row of blocks of a wave's tile: x[0 .. BJ
// - 1], BJ blocks side by side at column `col` (EPI_GATED: BJ / 2 gate blocks
// at `col`, then the up blocks of the same columns), this lane's row m. Leaves
// the values before rounding in x. Apart from the stores, so that a caller can
// ask for a later row's residual in between: memory operations complete in
// order, and a load asked for after a store is not there before it.
template <int EPI, class TO, int ACT, int EXTRA, int BJ>
__device__ inline void finish_row(const DenseArgs &p, f32x4 (&x)[BJ], int m, int col, int lane, const u32x2 (&bias)[BJ],
                                  const u32x4 (&res)[BJ / 2], PackedRow<EPI, BJ> &out)
{
    static_assert(BJ % (EPI == EPI_GATED ? 4 : 2) == 0, "blocks are stored in pairs");
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_GATED) {
        if constexpr (EXTRA) {
#pragma unroll
            for (int j = 0; j < BJ; ++j)
                x[j] = add_bias(x[j], bias[j]);
#pragma unroll
            for (int j = 0; j < BJ; j += 2)
                out.z[j / 2] = pack_pair<TO>(x[j], x[j + 1]);
        }
        constexpr int H = EPI == EPI_GATED ? BJ / 2 : BJ;
#pragma unroll
        for (int j = 0; j < H; ++j)
            x[j] = EPI == EPI_GATED ? act4<ACT>(x[j]) * x[(H + j) % BJ] : act4<ACT>(x[j]);
        if constexpr (EXTRA && EPI == EPI_LINEAR)
#pragma unroll
            for (int j = 0; j < BJ; j += 2) {
                f32x4 r0, r1;
                unpack_pair<TO>(res[j / 2], r0, r1);
                x[j] += r0;
                x[j + 1] += r1;
            }
    } else {
#pragma unroll
        for (int j = 0; j < BJ; j += 2) {
            x[j] *= p.alpha;
            x[j + 1] *= p.alpha;
            if constexpr (EPI == EPI_POLY) {
                f32x4 r0, r1;
                unpack_pair<TO>(res[j / 2], r0, r1);
                const int n = col + 16 * j + 4 * (lane >> 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[j][e] += p.beta * r0[e] + (m == n + e ? p.gamma : 0.0f);
                    x[j + 1][e] += p.beta * r1[e] + (m == n + 16 + e ? p.gamma : 0.0f);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < PackedRow<EPI, BJ>::C; ++j)
        out.c[j] = pack_pair<TO>(x[2 * j], x[2 * j + 1]);
}

template <int EXTRA, int EPI, int BJ>
__device__ inline void store_row(const DenseArgs &p, const Views &v, const PackedRow<EPI, BJ> &row, int m, int col, int lane)
{
    if constexpr (EXTRA && (EPI == EPI_LINEAR || EPI == EPI_GATED))
        if (p.z)
#pragma unroll
            for (int j = 0; j < BJ / 2; ++j) {
                constexpr int H = EPI == EPI_GATED ? BJ / 4 : BJ / 2;   // pairs of one half
                store16(row.z[j], v.z,
                        pair_offset(p, m, col + 32 * (j % H), EPI == EPI_GATED ? 2 * p.N : p.N, j < H ? 0 : p.N, lane));
            }
#pragma unroll
    for (int j = 0; j < PackedRow<EPI, BJ>::C; ++j)
        store16(row.c[j], v.c, pair_offset(p, m, col + 32 * j, p.N, 0, lane));
}

// The mirror image of two rows of FP16 blocks (m0 and m0 + 16 their first
// rows) of a symmetric result: C[n][m] = C[m][n]. A block in the layout above
// is also the 16 x 16 x 16 instruction's operand layout (lane (l16, grp): row
// l16, K 4 grp .. + 3), so a product with the identity returns it transposed,
// every value exact, and the stores are 16 bytes wide again.
template <int BJ>
__device__ inline void store_mirrored(const DenseArgs &p, const Views &v, const f32x4 (&y0)[BJ], const f32x4 (&y1)[BJ],
                                      int m0, int col, int lane)
{
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    const int l16 = lane & 15, grp = lane >> 4;
    f16x4 eye;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        eye[e] = l16 == 4 * grp + e ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
        const f32x4 t0 = __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_convertvector(y0[j], f16x4), eye, f32x4{}, 0, 0, 0);
        const f32x4 t1 = __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_convertvector(y1[j], f16x4), eye, f32x4{}, 0, 0, 0);
        const int n = col + 16 * j + l16, m = m0 + 16 * (grp & 1) + 8 * (grp >> 1);
        store16(pack_pair<_Float16>(t0, t1), v.c,
                n < p.N && m < p.M ? (int)(((unsigned)n * (unsigned)p.N + (unsigned)m) * 2u) : OOB);
    }
}

} // namespace dense
} // namespace gemm355
