// attend_rows.cuh -- attention of few rows (single tokens, drafts) over the 8-bit
// paged cache, and (from Rows4 on, where it differs) over that of 4 bits.
//
// For the rows r of one (sequence, key/value head) -- G query heads a token --
// and the tokens j they see:
//     s_rj = (q_r . c_j) * (scale log2(e) ks_page / f_r)      q_r: fp16, times the power of two f_r
//     p_rj = 2^(s_rj - m_r),  l_r = sum_j p_rj,  out_r = sum_j p_rj vs_page c'_j / l_r
// with the running maximum m_r of a warp's tokens.  The first product runs over the
// bytes as they stand, fp16 subnormals (c + 128) 2^-24, from a start of -128 2^-24
// sum(q_r).  The second takes the codes themselves, exact in fp16: a start of that
// kind would round away what tokens far from the maximum add.  What enters the
// second product is w_rj = 2^15 p_rj vs_page 2^-d_r in fp16, with the running maximum
// d_r of s_rj - m_r + log2(vs_page): relative to the row's largest contribution,
// however far apart the scales are, it keeps 11 bits down to 2^-29 and comes to
// nothing below 2^-40.  (Relative to m_r: beside a large score the logarithm's bits
// would be rounded away.)
//
// Bound by reading the cache: 48 x 8000 tokens of 8 heads of 128, 32 query heads,
// take 125 us, 6.3 TB/s of the codes; 1 x 131072 tokens 54 us (5.0 TB/s), of which
// some 12 us are a call's beginning and end (a launch, the lengths, pages, codes,
// the join of the parts): 1 x 700 tokens take 13 us.  Rows beyond 16 of a sequence
// and head read the tokens again, out of L2 (16 sequences of up to 4100 tokens, up to
// 40 rows each: 34 us).
//
// q is rounded to fp16's 11 bits where it comes as fp32: each of its values moves by no
// more than 2^-11 of itself, where a key's code is off by up to 2^-8 of its page's largest.
//
// The work -- for every sequence, head and tile of up to 8 * NT rows the tokens in
// steps of 128 -- is one line of steps that the CTAs, as many as are resident at
// once, cut into equal shares, whatever the lengths.  A CTA takes its share item by
// item; an item (one tile's tokens) that several CTAs share is joined by the last of
// them to arrive, in their order.
// A warp takes 32 tokens at a time, in the fragments of mma.sync m16n8k16: a
// lane's 16 bytes of a key are four k steps of a B fragment (the rows of q are
// loaded in the same order), and 16 bytes of the values of four tokens are eight
// A fragments of the transposed values, whose token pairs are put together by the
// byte permutes that widen the codes anyway.  Each warp has a ring of its own in
// shared memory, which its first lane fills by TMA a pair of tiles at a time, and
// no barrier with the other warps.  The pool is seen as rows of 128 bytes (two
// tokens of 64, half a token of 256) that the copies swizzle (16-byte chunk c of
// row r at c ^ (r & 7)); with the order of a tile's tokens chosen for it (order()
// below) the fragments' reads meet no bank conflicts.  The maxima, sums and outputs
// of the warps are joined in shared memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv.h"
#include "qmm_kernel.cuh"

namespace tfq {
namespace attend {

constexpr int WARPS = 4, THREADS = WARPS * 32;
// Tiles of 16 tokens that a warp takes at a time (dim 256: one, or its ring would leave one CTA an SM), and a CTA's tokens.
TFQ_HD constexpr int tiles_of(int d) { return d == 256 ? 1 : 2; }
TFQ_HD constexpr int step_of(int d) { return 16 * tiles_of(d) * WARPS; }
constexpr int CHUNK_TOKENS = 4096;       // tokens whose pages and scales a CTA keeps at a time
constexpr int MAX_PAGES = CHUNK_TOKENS / 16;
constexpr int MAX_PARTS = 768;           // CTAs of a launch, at most
// An item's beginning and end, in steps (4 bits).  48 x 8000 tokens of 8 heads of 128: 63 us so, 70 with 0, 64 with 5.
TFQ_HD constexpr int item_rows(int d) { return d == 256 ? 6 : 3; }
constexpr int NO_TOKEN = 1 << 30;        // past every chunk
constexpr float W_EXP = 15.f;            // exponent offset of w in fp16
// ... by the cache's bits: of 4, w is p times the scale of a code, at most a 15th of what d stands for.
TFQ_HD constexpr float w_exp(int f) { return f == 4 ? 18.f : W_EXP; }

struct Params {
    CUtensorMap tm_k, tm_v;  // the pools as rows of 128 bytes; a box is a pair of tiles, or one of 16-token pages
    tf_kv kv;                // (the 4-bit cache: pools and sizes, no scales)
    const uint32_t *k_affine, *v_affine;     // of the 4-bit cache: a bf16 scale and, above it, a bf16 bias
    tf_kv_batch b;
    const void *q;
    uint16_t *out;
    long long q_stride, out_stride;
    float *part;            // [2 grid][8 NT][dim] outputs, then [2 grid][8 NT][4] row sums (see RowSum)
    int *count;             // [grid] arrivals at the item that a CTA began to share, zero between launches
    int *status;
    float scale;
    int group, window, causal, q_f32;
    int block_log2;         // of kv.block
    int item_steps;         // what an item's beginning and end count for on the line (rows kernel)
    int stall;              // test hook: every CTA's first keys are withheld (rows kernel: every warp's first copies)
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Two biased codes (c + 128) in bytes 0, 1 (or 2, 3) of w as fp16 subnormals, (c + 128) 2^-24.
__device__ __forceinline__ uint32_t lo2_tiny(uint32_t w) { return prmt(w, 0u, 0x4140u); }
__device__ __forceinline__ uint32_t hi2_tiny(uint32_t w) { return prmt(w, 0u, 0x4342u); }
constexpr float TINY = 1.f / 16777216.f;         // 2^-24
// The codes themselves: 1024 + 128 + c, minus 1152 (exact).
__device__ __forceinline__ uint32_t half2_of(uint32_t w, uint32_t sel) {
    const uint32_t u = prmt(w, 0x64646464u, sel);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t lo2(uint32_t w) { return half2_of(w, 0x4140u); }
__device__ __forceinline__ uint32_t hi2(uint32_t w) { return half2_of(w, 0x4342u); }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Consecutive bytes (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// What has been summed of a row: maxima m of s and d of s - m + log2(vs), sum l of p.
struct __align__(16) RowSum {
    float m, d, l, unused;
};
// A maximum to subtract: 0 where there is none (what is below it is then -inf, not NaN).
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// p's d relative to a base that is no smaller than p.m (-inf: no token, or only values of scale 0).
__device__ __forceinline__ float d_at(const RowSum &p, float base) { return p.d + (p.m - base); }
// a's maxima, joined with p's.
__device__ __forceinline__ void join_maxima(RowSum &a, const RowSum &p) {
    const float m = fmaxf(a.m, p.m), base = base_of(m);
    a.d = fmaxf(d_at(a, base), d_at(p, base));
    a.m = m;
}
// Factors of a part's l and outputs in a join of the maxima of `a`: 0 for a part that
// saw no token or only values of scale 0; NaN scores (l NaN) stay NaN.
__device__ __forceinline__ float l_factor(const RowSum &p, const RowSum &a) { return exp2_fast(p.m - base_of(a.m)); }
__device__ __forceinline__ float o_factor(const RowSum &p, const RowSum &a) { return exp2_fast(d_at(p, base_of(a.m)) - base_of(a.d)); }
// Factor of the joined outputs: to the maximum of s, and by the sum.  In two, of which the second is 1 or, where d is so far
// down that the factor could leave fp32's normal numbers and its bits, 2^-64.
struct OutFactor {
    float f, g;
    __device__ __forceinline__ float of(float x) const { return x * f * g; }
};
template <int F = 8>
__device__ __forceinline__ OutFactor out_factor(const RowSum &a) {
    const bool low = a.d < -64.f;
    return {a.l == 0.f ? 0.f : exp2f((low ? a.d + 64.f : a.d) - w_exp(F)) / a.l, low ? 0x1p-64f : 1.f};
}

// Stages of a warp's ring, and CTAs an SM by the shared memory that the rings and the registers that outputs and q
// take.  48 sequences of up to 8000 tokens, 8 heads of 128: 79 us so, 81 with one tile a stage and four stages, 83
// with three stages and two CTAs; one of 131072 tokens 52, 54 and 50.
// 4 bits: as many CTAs as keep the step's registers: 48 x 8000 tokens of 8 heads of 128, 16 rows each: 153 us with two, 178
// with three, whose step keeps 400 bytes in local memory; 16 x 8000 of one head of 64, 16 rows: 19 us with three, 25 with
// four.  One row of each, 8 heads of 128: 63 us with three and three stages, 65 with four and two.
TFQ_HD constexpr int stages(int f, int d) { return f == 4 ? (d == 256 ? 5 : d == 128 ? 3 : 4) : d == 256 ? 3 : 2; }
TFQ_HD constexpr int ctas(int f, int d, int nt) {
    return f == 4 ? (d == 64 ? 5 - nt : d == 128 ? 4 - nt : 2) : d == 64 ? (nt == 1 ? 5 : 4) : d == 128 ? 3 : 2;
}
TFQ_HD constexpr int tile_bytes(int f, int d) { return 4 * f * d; }     // 16 tokens of keys and of values
TFQ_HD constexpr int affine_bytes(int f, int d) { return f == 4 ? 2 * d : 0; }   // ... and their scales and biases
TFQ_HD constexpr int out_pitch(int d) { return d + 4; }            // floats between joined rows
// Shared memory: the rings; after the tokens are done, every warp's outputs, then the parts' factors.
TFQ_HD constexpr int smem_bytes(int f, int d, int nt) {
    const int ring = WARPS * stages(f, d) * tiles_of(d) * (tile_bytes(f, d) + affine_bytes(f, d)), outs = WARPS * 8 * nt * out_pitch(d) * 4;
    const int join = MAX_PARTS * 8 * nt * 4, most = outs > join ? outs : join;
    return ring > most ? ring : most;
}

// Token of a tile (in eights) that column n of the scores stands for.  A quarter
// of a warp reads 16 bytes a lane of the keys of tokens order(2 a), order(2 a + 1),
// and of the values of the four tokens order(2 a) (or the four order(2 a + 1)).
template <int D>
__device__ __forceinline__ int order(int n) {
    const int a = n >> 1;
    if (D == 64) return (a + (a & 2)) ^ (n & 1 ? 3 : 0);
    if (D == 128) return n ^ (n & 1 ? 4 : 0);
    return n & 1 ? (a ^ 2) + 4 : a;
}
// Offset of a byte of a tile under the copies' swizzle.
__device__ __forceinline__ int swizzled(int byte) { return byte ^ ((byte >> 3) & 0x70); }

// Steps of one sequence: for every head and tile of its rows the tokens from
// `base` on, in steps of STEP.
struct SeqWork {
    SeqRows q;
    int base, steps, tiles;
};
template <int D, int R>
__device__ __forceinline__ SeqWork seq_work(const Params &P, int s) {
    SeqWork w;
    w.q = seq_rows(P.b, s);
    const int plan = max(0, min(w.q.end, P.b.max_len));
    if (!w.q.ok) {
        // Rows that lie within the matrices get zeros (no token is seen; the line, and with it the other
        // sequences' bits, stay as they are).
        w.q.end = 0;
        if (!w.q.placed) w.q.n = 0;
    }
    w.tiles = (w.q.n * P.group + R - 1) / R;
    w.base = P.window ? max(0, plan - w.q.n - P.window + 1) & ~31 : 0;
    w.steps = max(1, (plan - w.base + step_of(D) - 1) / step_of(D));
    return w;
}

// Row factor f of a magnitude: the power of two that brings it into [1, 4).
__device__ __forceinline__ float row_factor(float amax) {
    const uint32_t e = __float_as_uint(amax) >> 23;
    if (e == 0 || e == 255) return 1.f;
    return __uint_as_float((e >= 253 ? 1u : 254u - e) << 23);
}

// Two fp32 numbers at a time.
typedef unsigned long long F2;
__device__ __forceinline__ F2 two(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 of_two(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// As mma_f16, for the compiler to move.
__device__ __forceinline__ void mma_f16_free(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Products that begin at 0.
__device__ __forceinline__ void mma_f16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of a warp's 8 x 8 numbers of 16 bits (lane 4 r + c holds row r's 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Four 8 x 8 matrices of 16-bit units out of shared memory (lane 8 i + r gives matrix i's row r, 16 bytes): lane 4 r + c
// gets row r's units 2 c, 2 c + 1 of each; TRANS: unit r of rows 2 c, 2 c + 1.
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&x)[4], const uint8_t *row) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(smem_u32(row)));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(smem_u32(row)));
}
// The larger magnitudes of two pairs of bf16 numbers (signs mean nothing then; NaN is passed over).
__device__ __forceinline__ uint32_t larger_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What a warp of the rows kernel holds of a tile of 8 NT rows, over the 4-bit cache, and how it takes 16 or 32 tokens.
//
//     s_rj = f_r sum_g (scale_jg (q_rg . c_jg) + bias_jg sum(q_rg))        g: groups of 64 dimensions
//     p_rj = 2^(s_rj - m_r),  l_r = sum_j p_rj,  out_rg = sum_j p_rj (scale_jg c'_jg + bias_jg) / l_r
// Codes are bits 0 to 3 or 4 to 7 of a half word, as fp16 subnormals c 2^-24 and c 2^-20: one mask makes two of them
// (the 2^4 goes into q for the first product and into the output for the second).
// First product: the tokens are its 16 rows and the rows of q its 8 columns, so that no part of it is idle with up to 8
// rows; a lane gets the scores of two tokens a tile and two rows, two numbers to an instruction.  The sums with the
// biases are a product of bf16: the cache's pairs (scale, bias) as they lie with (0, a third of sum(q)'s bits).
// Second product: w_rj scale_jg in fp16 (w as over 8 bits: 2^18 p 2^-d, d the running maximum of s - m + log2(15 scale
// or bias)), transposed in the warp, with the codes transposed by the loads (four of a token at a time); the biases' part in fp32.
// (A logarithm for two tokens of a tile, 8 apart: d counts the larger of their scores with the larger of their values.)
// The rounding to fp16's 11 bits (tf32 has no more) is what outputs are off by before their own to bf16: with values that are
// differences of codes and biases by 0.6e-3 of their size, where that one is off by 1.7e-3.
// The maxima m and d are joined over the warp's lanes only where a lane finds one passed by more than SLACK4.
//
// 48 x 8000 tokens of 8 heads of 128, 32 query heads, 63 us; 1 x 131000 tokens 41 us, 5.5 TB/s of the cache while its tokens
// run (27 us), after a beginning of 6 us and before a join of up to 8.  With the rows of q as the first product's 16 rows,
// maxima joined at every step and the biases' sums in fp32: 84 and 53 us; with the codes by plain loads, put together by byte
// permutes: 71 and 44.  (The next tokens' scores beside these tokens' exponentials, and shifts as products: no faster.)
constexpr float SLACK4 = 1.f;            // in powers of two (w stays below fp16's largest: 2^18 / 15 times 2^SLACK4)
// d of a row that has seen a token falls no lower, so that 2^(18 - d), and a p of up to 2^SLACK4 times it, are fp32 numbers.
// (d itself is held there, not the factor: outputs and joins count on the two being one number.  Values of 2^-126, the smallest
// that bf16 holds in full, are then 2^-4 in fp16.)
constexpr float LEAST4 = w_exp(4) - 126.f;
template <int D, int NT>
struct Rows4 {
    static constexpr int KV = D / 64, MT = D / 16, TILES = tiles_of(D), NB = KV == 4 ? 2 : 1;
    static constexpr bool Q_REGS = D < 256 || NT == 1;
    static constexpr int TOK = D / 2;
    static constexpr int SECOND = 16 * TOK == 512 ? 64 : 0;   // what the swizzle adds in a second tile that begins in the middle of 1024 bytes

    uint2 q[NT][Q_REGS ? 4 * KV : 1];    // k steps 2 c, 2 c + 1 of row lr (+ 8): d = 32 c + 8 lc + {0, 1 | 2, 3}, + 4, as stored
    uint32_t qb[NT][NB][2];              // of sum(q): (0, a part), by the lane's place among the pairs
    F2 rowf[NT], mm[NT], f[NT], l[NT];   // of rows 2 lc, 2 lc + 1 (+ 8): factor of a score, base of m, 2^18 2^-d, sum
    F2 ob[NT][KV];                       // sums of w times the biases, this lane's tokens
    float m[NT][2], d[NT][2];
    float o[MT][NT][4];

    template <typename Q>
    static __device__ __forceinline__ uint2 q_at(const Q &sq, int r, int lc, int i) {
        return *reinterpret_cast<const uint2 *>(&sq[r][32 * (i >> 1) + 8 * lc + 4 * (i & 1)]);
    }
    template <typename Q, typename S>
    __device__ __forceinline__ void begin(const Q &sq, const float2 *s_row, const S &s_qs, int lr, int lc, int rows) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            if constexpr (Q_REGS) {
#pragma unroll
                for (int i = 0; i < 4 * KV; ++i) q[u][i] = q_at(sq, lr + 8 * u, lc, i);
            }
            // Parts of 8 bits each of the sum of group lc % KV.
            const float x = s_qs[lr + 8 * u][lc & (KV - 1)];
            auto top = [](float y) { return __float_as_uint(y) & 0xFFFF0000u; };
            const uint32_t p0 = top(x), p1 = top(x - __uint_as_float(p0)), p2 = top(x - __uint_as_float(p0) - __uint_as_float(p1));
            const int k = lc / KV;
            auto part = [&](int i) { return i == 0 ? p0 : i == 1 ? p1 : i == 2 ? p2 : 0u; };
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) qb[u][b][e] = part(k + (2 * b + e) * (4 / KV));
            rowf[u] = two(s_row[min(2 * lc + 8 * u, rows - 1)].x, s_row[min(2 * lc + 1 + 8 * u, rows - 1)].x);
            mm[u] = f[u] = l[u] = 0;
#pragma unroll
            for (int v = 0; v < KV; ++v) ob[u][v] = 0;
            m[u][0] = m[u][1] = d[u][0] = d[u][1] = -INFINITY;
#pragma unroll
            for (int p = 0; p < MT; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[p][u][e] = 0.f;
        }
    }

    // Tokens t + 16 h + 8 nb + ..: their keys' codes in `tiles` and their values' in `values` (rows of matrices: at `at`),
    // scales and biases in k_pairs and v_pairs.
    // full: every row sees every token.  Else seen(i) is whether token t + i is there and any row sees it, and
    // sees(r, i) whether row r does.
    template <typename Q, typename Seen, typename Sees>
    __device__ __forceinline__ void step(const uint8_t *tiles, const uint8_t *values, const uint32_t *k_pairs, const uint32_t *v_pairs,
                                         const int (&at)[KV], const Q &sq, int lr, int lc, bool full, Seen seen, Sees sees) {
        // Scores: tokens t + 8 nb + lr of rows 2 lc, 2 lc + 1 (+ 8).
        uint32_t pair[2 * TILES][KV];
        auto load_pairs = [&](const uint32_t *src) {
#pragma unroll
            for (int nb = 0; nb < 2 * TILES; ++nb) {
                const uint32_t *at = src + (8 * nb + lr) * KV;
                if constexpr (KV == 1) pair[nb][0] = *at;
                if constexpr (KV == 2) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(at);
                    pair[nb][0] = x.x, pair[nb][1] = x.y;
                }
                if constexpr (KV == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(at);
                    pair[nb][0] = x.x, pair[nb][1] = x.y, pair[nb][2] = x.z, pair[nb][3] = x.w;
                }
            }
        };
        load_pairs(k_pairs);
        F2 sc[2 * TILES][NT];
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
            uint32_t a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t(&x)[KV] = pair[2 * h + e];
                if constexpr (KV == 1) a[e] = x[0];
                if constexpr (KV == 2) a[e] = lc & 1 ? x[1] : x[0];
                if constexpr (KV == 4) a[e] = lc & 2 ? (lc & 1 ? x[3] : x[2]) : (lc & 1 ? x[1] : x[0]);
            }
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                float c[4];
                mma_bf16_0(c, a[0], a[1], KV == 1 ? 0u : a[0], KV == 1 ? 0u : a[1], qb[u][0][0], qb[u][0][1]);
                if constexpr (NB == 2) mma_bf16(c, a[0], a[1], a[0], a[1], qb[u][NB - 1][0], qb[u][NB - 1][1]);
                sc[2 * h][u] = two(c[0], c[1]);
                sc[2 * h + 1][u] = two(c[2], c[3]);
            }
        }
#pragma unroll
        for (int v = 0; v < KV; ++v) {
            float raw[TILES][NT][4];
            uint32_t x[TILES][4];                // tokens 0 .. 7 and 8 .. 15 of the first 32 dimensions, and of the others
#pragma unroll
            for (int h = 0; h < TILES; ++h) load_matrices<false>(x[h], tiles + h * 16 * TOK + (at[v] ^ h * SECOND));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < TILES; ++h) {
                    const uint32_t w0 = x[h][2 * (i >> 1)] >> (8 * (i & 1)), w1 = x[h][2 * (i >> 1) + 1] >> (8 * (i & 1));
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
                        const uint2 b = Q_REGS ? q[u][Q_REGS ? 4 * v + i : 0] : q_at(sq, lr + 8 * u, lc, 4 * v + i);
                        if (i == 0)
                            mma_f16_0(raw[h][u], w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u, b.x, b.y);
                        else
                            mma_f16_free(raw[h][u], w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u, b.x, b.y);
                    }
                }
#pragma unroll
            for (int nb = 0; nb < 2 * TILES; ++nb) {
                const float s = __uint_as_float(pair[nb][v] << 16);
#pragma unroll
                for (int u = 0; u < NT; ++u)
                    sc[nb][u] = fma2(two(raw[nb >> 1][u][2 * (nb & 1)], raw[nb >> 1][u][2 * (nb & 1) + 1]), two(s, s), sc[nb][u]);
            }
        }
        load_pairs(v_pairs);
#pragma unroll
        for (int nb = 0; nb < 2 * TILES; ++nb)
#pragma unroll
            for (int u = 0; u < NT; ++u) sc[nb][u] = mul2(sc[nb][u], rowf[u]);     // (rounded here: the largest less the maximum is 0)
        if (!full) {
#pragma unroll
            for (int nb = 0; nb < 2 * TILES; ++nb) {
                const int i = 8 * nb + lr;
                // (Where no row sees a token its values' pairs are 0: whatever stands there, infinities and NaN too, meets
                // weights of 0.)
                if (!seen(i))
#pragma unroll
                    for (int v = 0; v < KV; ++v) pair[nb][v] = 0;
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const float2 x = of_two(sc[nb][u]);
                    sc[nb][u] = two(seen(i) && sees(2 * lc + 8 * u, i) ? x.x : -INFINITY, seen(i) && sees(2 * lc + 1 + 8 * u, i) ? x.y : -INFINITY);
                }
            }
        }
        // Of this lane's tokens of each tile: the logarithm of what no value passes by more than a factor of 2, and the
        // largest scores.
        float vs[TILES], top[TILES][NT][2];
        bool grew = false;
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
            uint32_t most = 0;
#pragma unroll
            for (int v = 0; v < KV; ++v) most = larger_bf16x2(most, larger_bf16x2(pair[2 * h][v], pair[2 * h + 1][v]));
            vs[h] = log2_fast(fmaxf(fabsf(__uint_as_float(most << 16)) * 15.f, fabsf(__uint_as_float(most & 0xFFFF0000u))));
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const float2 x = of_two(sc[2 * h][u]), y = of_two(sc[2 * h + 1][u]), b = of_two(mm[u]);
                const float t0 = top[h][u][0] = fmaxf(x.x, y.x), t1 = top[h][u][1] = fmaxf(x.y, y.y);
                grew |= t0 > m[u][0] + SLACK4 || t1 > m[u][1] + SLACK4 || (t0 - b.x) + vs[h] > d[u][0] + SLACK4 || (t1 - b.y) + vs[h] > d[u][1] + SLACK4;
            }
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                float base[2], scale[2], fac[2], fl[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mt = m[u][e], dt = -INFINITY;
#pragma unroll
                    for (int h = 0; h < TILES; ++h) mt = fmaxf(mt, top[h][u][e]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, x));
                    base[e] = base_of(mt);
#pragma unroll
                    for (int h = 0; h < TILES; ++h) dt = fmaxf(dt, (top[h][u][e] - base[e]) + vs[h]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) dt = fmaxf(dt, __shfl_xor_sync(~0u, dt, x));
                    const float d0 = d[u][e] + (m[u][e] - base[e]);
                    fl[e] = m[u][e] == -INFINITY ? 1.f : exp2_fast(m[u][e] - mt);
                    m[u][e] = mt;
                    d[u][e] = mt == -INFINITY ? -INFINITY : fmaxf(fmaxf(d0, dt), LEAST4);
                    fac[e] = exp2_fast(d0 - base_of(d[u][e]));
                    scale[e] = mt == -INFINITY ? 0.f : exp2_fast(w_exp(4) - d[u][e]);
                }
                mm[u] = two(base[0], base[1]);
                f[u] = two(scale[0], scale[1]);
                l[u] = mul2(l[u], two(fl[0], fl[1]));
                const F2 a = two(fac[0], fac[1]);
#pragma unroll
                for (int v = 0; v < KV; ++v) ob[u][v] = mul2(ob[u][v], a);
#pragma unroll
                for (int p = 0; p < MT; ++p) {
                    const float2 x = of_two(mul2(two(o[p][u][0], o[p][u][1]), a)), y = of_two(mul2(two(o[p][u][2], o[p][u][3]), a));
                    o[p][u][0] = x.x, o[p][u][1] = x.y, o[p][u][2] = y.x, o[p][u][3] = y.y;
                }
            }
        }
        uint32_t pb[KV][NT][2 * TILES];
#pragma unroll
        for (int nb = 0; nb < 2 * TILES; ++nb) {
            F2 w[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const float2 x = of_two(sc[nb][u]), b = of_two(mm[u]);
                const F2 p = two(exp2_fast(x.x - b.x), exp2_fast(x.y - b.y));
                l[u] = add2(l[u], p);
                w[u] = mul2(p, f[u]);
            }
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                const float s = __uint_as_float(pair[nb][v] << 16), b = __uint_as_float(pair[nb][v] & 0xFFFF0000u);
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const float2 x = of_two(mul2(w[u], two(s, s)));
                    pb[v][u][nb] = transposed(pack_half(x.x, x.y));
                    ob[u][v] = fma2(w[u], two(b, b), ob[u][v]);
                }
            }
        }
        // Transposed values: tokens 2 lc, 2 lc + 1 (+ 8) of a tile, d = 32 c + 4 lr + ...
#pragma unroll
        for (int h = 0; h < TILES; ++h)
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                uint32_t x[4];
                load_matrices<true>(x, values + h * 16 * TOK + (at[v] ^ h * SECOND));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = x[2 * (i >> 1)] >> (8 * (i & 1)), b = x[2 * (i >> 1) + 1] >> (8 * (i & 1));
#pragma unroll
                    for (int u = 0; u < NT; ++u)
                        mma_f16_free(o[4 * v + i][u], a & 0x000F000Fu, a & 0x00F000F0u, b & 0x000F000Fu, b & 0x00F000F0u, pb[v][u][2 * h], pb[v][u][2 * h + 1]);
                }
            }
    }

    // The sums over the lanes' tokens: row sums by store(row, sum), the values of a row's dimensions dim, dim + 1 by put.
    template <typename Store, typename Put>
    __device__ __forceinline__ void end(int lr, int lc, Store store, Put put) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            float2 b[KV], s = of_two(l[u]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) s.x += __shfl_xor_sync(~0u, s.x, x), s.y += __shfl_xor_sync(~0u, s.y, x);
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                b[v] = of_two(ob[u][v]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) b[v].x += __shfl_xor_sync(~0u, b[v].x, x), b[v].y += __shfl_xor_sync(~0u, b[v].y, x);
            }
            if (lr == 0) {
                store(2 * lc + 8 * u, RowSum{m[u][0], d[u][0], s.x, 0.f});
                store(2 * lc + 1 + 8 * u, RowSum{m[u][1], d[u][1], s.y, 0.f});
            }
            // (the odd dimensions' codes stood 2^4 higher)
#pragma unroll
            for (int p = 0; p < MT; ++p)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = e ? b[p / 4].y : b[p / 4].x;
                    put(2 * lc + e + 8 * u, p / 2 * 32 + 4 * lr + 2 * (p % 2), make_float2(fmaf(o[p][u][e], 1.f / TINY, x), fmaf(o[p][u][2 + e], 0.0625f / TINY, x)));
                }
        }
    }
};

// F: bits of a code (8 or 4).
template <int F, int D, int NT>
__global__ void __launch_bounds__(THREADS, ctas(F, D, NT)) rows_kernel(const __grid_constant__ Params P) {
    constexpr int R = 8 * NT;                    // rows of a tile
    constexpr int KV = D / 64;                   // vectors of a key a lane: its 16 of each 64 values
    constexpr int MT = D / 16;                   // m tiles of the transposed values
    constexpr int VB = D >= 128 ? 16 : 8;   // values of a token that a lane takes at once
    constexpr int NV = D / (8 * VB);             // ... and how often
    constexpr int NST = stages(F, D), TILES = tiles_of(D), TP = 16 * TILES, STEP = step_of(D);
    constexpr int TOK = D * F / 8;               // bytes of a token
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ uint64_t bars[WARPS][NST];
    __shared__ int s_abort;
    __shared__ __align__(16) __half sq[R][D + 8];
    __shared__ float2 s_row[R];
    __shared__ RowSum s_sum[WARPS][R], s_join[R];    // of each warp, and of all of them
    __shared__ float s_wfac[WARPS][R];               // factors of the warps' outputs in the join
    __shared__ float s_ks[F == 8 ? MAX_PAGES : 1], s_vs[F == 8 ? MAX_PAGES : 1];
    __shared__ float s_qs[F == 4 ? R : 1][KV];       // sums of a row's 64s of q
    __shared__ int2 s_see[F == 4 ? R : 1];           // tokens that a row sees
    __shared__ int s_page[MAX_PAGES];
    __shared__ long long s_warp[WARPS], s_first;
    __shared__ int s_seq;
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = lane >> 2, lc = lane & 3;
    const int H = P.kv.kv_heads, G = P.group, BL = P.block_log2, BM = P.kv.block - 1, item = F == 4 ? P.item_steps : 0;

    if constexpr (F == 4) {
        // The rows of q and of the table, a line of 128 bytes a thread where there are no more, on their way to L2 while the
        // lengths are read.
        const int es = P.q_f32 ? 4 : 2, q_lines = H * G * D * es / 128 + 1, t_lines = ((((P.b.max_len - 1) >> BL) + 1) >> 5) + 1;
        const long long nq = (long long)P.b.rows * q_lines, nt = (long long)P.b.n_seqs * t_lines, all = (long long)gridDim.x * THREADS;
        const long long i = (long long)blockIdx.x * THREADS + tid;
        if (nq + nt <= all && i < nq + nt) {
            const long long j = i < nq ? i : i - nq, row = i < nq ? j / q_lines : j / t_lines, line = i < nq ? j - row * q_lines : j - row * t_lines;
            const char *at = i < nq ? static_cast<const char *>(P.q) + row * P.q_stride * es + min(line * 128, (long long)H * G * D * es - 1)
                                    : reinterpret_cast<const char *>(P.b.table + row * P.b.table_stride + min(line * 32, (long long)((P.b.max_len - 1) >> BL)));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    }

    // This CTA's share: steps [u0, u1) of the line, whose first sequence is s_seq, at s_first of the line.
    const int per = (P.b.n_seqs + THREADS - 1) / THREADS;
    const int s0 = tid * per, s1 = min(P.b.n_seqs, s0 + per);
    long long mine_sum = 0;
    for (int s = s0; s < s1; ++s) {
        const SeqWork w = seq_work<D, R>(P, s);
        if (!w.q.ok && blockIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        mine_sum += (long long)H * w.tiles * (w.steps + item);
    }
    long long incl = mine_sum;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    if (tid == 0) {
        for (int i = 0; i < WARPS * NST; ++i) mbar_init(&bars[0][i], 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp) incl += s_warp[i];
        total += s_warp[i];
    }
    const int C = (int)min((long long)gridDim.x, total);       // CTAs that get a share
    if ((int)blockIdx.x >= C) return;
    const long long u0 = total * blockIdx.x / C, u1 = total * (blockIdx.x + 1) / C;
    auto cta_of = [&](long long u) { return (int)(((u + 1) * C - 1) / total); };
    if (incl - mine_sum <= u0 && u0 < incl) {
        long long at = incl - mine_sum;
        int s = s0;
        for (;; ++s) {
            const SeqWork w = seq_work<D, R>(P, s);
            const long long n = (long long)H * w.tiles * (w.steps + item);
            if (u0 < at + n) break;
            at += n;
        }
        s_seq = s;
        s_first = at;
    }
    __syncthreads();

    // A warp's ring: stages of a pair of tiles' keys, then their values.  (4 bits: after all rings, in the same way,
    // scales and biases.)
    constexpr int STAGE = TILES * tile_bytes(F, D), AFFINE = TILES * affine_bytes(F, D);
    uint8_t *mine = ring + warp * NST * STAGE;
    uint8_t *const mine_affine = ring + WARPS * NST * STAGE + warp * NST * AFFINE;
    uint64_t *bar = bars[warp];
    volatile int *abort = &s_abort;
    const bool single = TILES == 2 && BL == 4;   // pages of one tile only: a stage's tiles come from two
    uint32_t fit = 0, it = 0;                    // pairs fetched and taken, over all items
    // Offsets of this lane's reads in a stage: keys of token order(lr) (+ 8, + 16, + 24), values of four tokens of a tile.
    // (4 bits: rows of matrices, 16 bytes of a token; natural order, whose eight tokens meet eight chunks under the swizzle.)
    int k_at[KV][2], v_at[NV][4], at4[KV];
    const int tok[2] = {order<D>(2 * lc), order<D>(2 * lc + 1)};
#pragma unroll
    for (int v = 0; v < KV; ++v) {
        at4[v] = swizzled((lane & 15) * TOK + 32 * v + 16 * (lane >> 4));
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) k_at[v][nb] = swizzled((order<D>(lr) + 8 * nb) * D + 64 * v + 16 * lc);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) v_at[v][k] = swizzled((tok[k & 1] + 8 * (k >> 1)) * D + v * 8 * VB + VB * lr) + STAGE / 2;

    int seq = s_seq;
    long long seq_at = s_first;                  // the sequence's first step on the line
    SeqWork sw = seq_work<D, R>(P, seq);
    for (long long line = u0; line < u1;) {
        while (line >= seq_at + (long long)H * sw.tiles * (sw.steps + item)) {
            seq_at += (long long)H * sw.tiles * (sw.steps + item);
            sw = seq_work<D, R>(P, ++seq);
        }
        // The item: a head and a tile of the sequence's rows; this CTA's steps of it.
        const int index = (int)((line - seq_at) / (sw.steps + item)), h = index / sw.tiles, tile = index - h * sw.tiles;
        const long long item_at = seq_at + (long long)index * (sw.steps + item) + item;      // (its first step)
        const int step0 = (int)max(0LL, line - item_at), step1 = (int)min((long long)sw.steps, u1 - item_at);
        if (step0 >= step1) break;               // (the share ends in the item's beginning)
        const int r0 = tile * R, rows = min(R, sw.q.n * G - r0);
        const int end = sw.q.end, first = end - sw.q.n;              // (position of the sequence's first row)
        const int i0 = r0 / G, i1 = (r0 + rows - 1) / G;             // first and last of the tile's tokens
        const int to = P.causal ? min(end, first + i1 + 1) : end;    // tokens that any of the rows sees
        const int t_begin = sw.base + step0 * STEP, t_end = min(sw.base + step1 * STEP, to);
        uint16_t *out = P.out + (long long)sw.q.row0 * P.out_stride;
        auto out_at = [&](int r) {               // first value of the tile's row r
            const int gr = r0 + r, i = gr / G;
            return out + (long long)i * P.out_stride + ((long long)h * G + gr - i * G) * D;
        };

        // The rows of q, in fp16 times a power of two each.
        float qx[R / WARPS][D / 32];
#pragma unroll
        for (int k = 0; k < R / WARPS; ++k) {
            const int r = warp + k * WARPS, gr = r0 + r, i = gr / G;
            const long long at = (long long)(sw.q.row0 + i) * P.q_stride + ((long long)h * G + gr - i * G) * D + lane;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                qx[k][e] = 0.f;
                if (r < rows)
                    qx[k][e] = P.q_f32 ? static_cast<const float *>(P.q)[at + e * 32]
                                       : __uint_as_float((uint32_t) static_cast<const uint16_t *>(P.q)[at + e * 32] << 16);
            }
        }
        // Tokens [c0, c1): their pages, the first stages under way, and their scales (of the values' the logarithm).
        const int any_from = P.window ? max(0, first + i0 - P.window + 1) : 0, from = any_from & ~31;   // (the first token that any of them sees)
        int c0 = max(t_begin, from), c1 = c0, pg0 = 0, npages = 0, ft = 0;
        auto fetch = [&](int t) {                // (the warp's first lane)
            if (t >= c1) return;
            const uint32_t stage = fit++ % NST;
            if (P.stall && fit == 1) return;
            const int p0 = s_page[(t >> BL) - pg0], p1 = single && t + 16 < c1 ? s_page[(t >> BL) + 1 - pg0] : -1;
            mbar_arrive_tx(&bar[stage], (uint32_t)((p0 >= 0 ? (single ? 1 : TILES) : 0) + (p1 >= 0 ? 1 : 0)) * (tile_bytes(F, D) + affine_bytes(F, D)));
            uint8_t *dst = mine + stage * STAGE;
            auto copy = [&](int page, int at, int tile) {
                const long long token = (((long long)page * H + h) << BL) + (at & BM);
                const int row = (int)((token * TOK) >> 7);
                uint8_t *to = dst + tile * 16 * TOK;
                tma_2d(to, &P.tm_k, 0, row, &bar[stage]);
                tma_2d(to + STAGE / 2, &P.tm_v, 0, row, &bar[stage]);
                if constexpr (F == 4) {
                    uint8_t *pairs = mine_affine + stage * AFFINE + tile * D;
                    const uint32_t bytes = (single ? 1 : TILES) * D;
                    bulk_copy(pairs, P.k_affine + token * KV, bytes, &bar[stage]);
                    bulk_copy(pairs + AFFINE / 2, P.v_affine + token * KV, bytes, &bar[stage]);
                }
            };
            if (p0 >= 0) copy(p0, t, 0);
            if (p1 >= 0) copy(p1, t + 16, 1);
        };
        bool holes = false;                      // any of the chunk's pages is none
        auto open_chunk = [&]() {
            c1 = min(c0 + CHUNK_TOKENS, t_end);
            pg0 = c0 >> BL;
            npages = ((c1 - 1) >> BL) - pg0 + 1;
            bool hole = false;
            for (int i = tid; i < npages; i += THREADS) {
                int page = P.b.table[seq * P.b.table_stride + pg0 + i];
                if (page < 0 || page >= P.kv.n_blocks) {
                    atomicOr(P.status, STATUS_BOUNDS);
                    page = -1;
                }
                s_page[i] = page;
                hole |= page < 0;
            }
            holes = __syncthreads_or(hole);
            ft = *abort ? NO_TOKEN : c0 + TP * warp;
            for (int i = 0; i < NST - 1; ++i, ft += STEP)
                if (lane == 0) fetch(ft);
            if constexpr (F == 8) {
                for (int i = tid; i < npages; i += THREADS) {
                    const long long ph = (long long)s_page[i] * H + h;
                    s_ks[i] = s_page[i] < 0 ? 0.f : P.kv.k_scale[ph];
                    s_vs[i] = s_page[i] < 0 ? -INFINITY : log2f(P.kv.v_scale[ph]);
                }
            }
        };
        if (c0 < t_end) open_chunk();            // (the loads of q are on their way meanwhile)
#pragma unroll
        for (int k = 0; k < R / WARPS; ++k) {
            const int r = warp + k * WARPS;
            float m = 0.f, sum[F == 8 ? 1 : KV] = {};
#pragma unroll
            for (int e = 0; e < D / 32; ++e) m = fmaxf(m, fabsf(qx[k][e]));
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            const float f = row_factor(m);
            // (4 bits: times 2^8, and of odd dimensions 2^4, whose codes stand 2^4 higher; the eight of a word in the
            // order in which its codes come.)
            constexpr float Q = F == 4 ? 256.f : 1.f;
            const int at4 = (lane & ~7) | (lane & 3) << 1 | (lane >> 2 & 1);
            const float odd = lane & 1 ? 0.0625f : 1.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const __half x = F == 4 ? __float2half_rn(qx[k][e] * f * (Q * odd)) : __float2half_rn(qx[k][e] * f);
                sq[r][e * 32 + (F == 4 ? at4 : lane)] = x;
                sum[F == 4 ? e / 2 : 0] += F == 4 ? __half2float(x) * (1.f / odd) : __half2float(x);
            }
#pragma unroll
            for (int g = 0; g < (F == 8 ? 1 : KV); ++g)
                for (int o = 16; o > 0; o >>= 1) sum[g] += __shfl_xor_sync(~0u, sum[g], o);
            if (lane == 0) {
                s_row[r] = make_float2(P.scale * 1.44269504088896340736f / f * (1.f / (Q * TINY)), sum[0] * (-128.f * TINY));
#pragma unroll
                for (int g = 0; F == 4 && g < KV; ++g) s_qs[r][g] = sum[g] * TINY;
                if constexpr (F == 4) {
                    const int pos = first + (r0 + min(r, rows - 1)) / G;
                    s_see[r] = make_int2(P.window ? pos - P.window + 1 : 0, P.causal ? min(end, pos + 1) : end);
                }
            }
        }
        __syncthreads();

        // A fragments of q: k step (v, i) holds d = 64 v + 16 lc + 4 i + {0, 1 | 2, 3}.  (dim 256: read again for every tile.)
        constexpr bool Q_REGS = D < 256;
        uint2 qa[NT][Q_REGS ? KV : 1][4];
        auto q_at = [&](int u, int v, int i) { return *reinterpret_cast<const uint2 *>(&sq[lr + 8 * u][64 * v + 16 * lc + 4 * i]); };
        if constexpr (F == 8 && Q_REGS) {
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int v = 0; v < KV; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) qa[u][v][i] = q_at(u, v, i);
        }
        float rowf[NT], off[NT];                     // factor of a score; its start, -128 sum(q) 2^-24
        int see_from[NT], see_to[NT];                // tokens that rows lr (+ 8) see
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int r = min(lr + 8 * u, rows - 1);   // (rows past the tile's end are computed, never stored)
            rowf[u] = s_row[r].x;
            off[u] = s_row[r].y;
            const int pos = first + (r0 + r) / G;
            see_to[u] = P.causal ? min(end, pos + 1) : end;
            see_from[u] = P.window ? pos - P.window + 1 : 0;
        }
        int all_from = 0, all_to = end;            // tokens that every row of the tile sees
        if (P.causal) {
            all_to = min(end, first + i0 + 1);
            if (P.window) all_from = first + i1 - P.window + 1;
        }

        float o[MT][NT][4];
        float m[NT], d[NT], l[NT];
        Rows4<D, NT> rows4;                          // (4 bits: all of these, and q)
        if constexpr (F == 4) rows4.begin(sq, s_row, s_qs, lr, lc, rows);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            m[u] = d[u] = -INFINITY;
            l[u] = 0.f;
#pragma unroll
            for (int p = 0; p < MT; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[p][u][e] = 0.f;
        }
        for (bool opened = true; c0 < t_end; c0 = c1, opened = false) {
            if (!opened) {
                open_chunk();
                __syncthreads();
            }
            auto next_stage = [&]() {                // the codes of the tokens whose turn it is, and a fetch in place of the last ones
                if (lane == 0) fetch(ft);
                ft += STEP;
                if (!mbar_try(&bar[it % NST], (it / NST) & 1)) {
                    if (!*abort) mbar_wait(&bar[it % NST], (it / NST) & 1, abort, P.status);
                    if (*abort) ft = NO_TOKEN;       // (a wait ran out: nothing more is fetched, the stages may be on their way)
                }
                return mine + (it % NST) * STAGE;
            };
            if constexpr (F == 4) {
                for (int t = c0 + TP * warp; t < c1; t += STEP, ++it) {
                    const uint8_t *tiles = next_stage();
                    const uint32_t *const pairs = reinterpret_cast<const uint32_t *>(mine_affine + (it % NST) * AFFINE);
                    const bool full = t >= all_from && t + TP <= all_to && !holes;
                    // (a tile of no page is not seen)
                    auto there = [&](int h) { return s_page[min(((t + 16 * h) >> BL) - pg0, npages - 1)] >= 0 && !(h == 1 && single && t + 16 >= c1); };
                    rows4.step(
                        tiles, tiles + STAGE / 2, pairs, pairs + AFFINE / 8, at4, sq, lr, lc, full,
                        [&](int i) { return there(i < 16 ? 0 : 1) && t + i >= any_from && t + i < to; },
                        [&](int r, int i) { return t + i >= s_see[r].x && t + i < s_see[r].y; });
                    __syncwarp();                    // (every lane has read the stage that is filled next)
                }
            } else for (int t = c0 + TP * warp; t < c1; t += STEP, ++it) {
                const uint8_t *tiles = next_stage();
                // Tiles t and t + 16: their pages (a tile of no page is not seen).
                int pi[TILES];
                bool on[TILES];
#pragma unroll
                for (int h = 0; h < TILES; ++h) {
                    pi[h] = min(((t + 16 * h) >> BL) - pg0, npages - 1);
                    on[h] = s_page[pi[h]] >= 0 && !(h == 1 && single && t + 16 >= c1);
                }
                const bool full = t >= all_from && t + TP <= all_to && on[0] && on[TILES - 1];
                // Scores of the tiles' tokens: n tile 2 h + nb holds tokens t + 16 h + 8 nb + ...
                float sc[2 * TILES][4];
#pragma unroll
                for (int nb = 0; nb < 2 * TILES; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nb][e] = e >> 1 < NT ? off[NT > 1 ? e >> 1 : 0] : 0.f;
#pragma unroll
                for (int v = 0; v < KV; ++v) {
                    uint32_t kw[2 * TILES][4];
#pragma unroll
                    for (int nb = 0; nb < 2 * TILES; ++nb) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(tiles + (nb >> 1) * 16 * D + k_at[v][nb & 1]);
                        kw[nb][0] = x.x ^ 0x80808080u, kw[nb][1] = x.y ^ 0x80808080u;
                        kw[nb][2] = x.z ^ 0x80808080u, kw[nb][3] = x.w ^ 0x80808080u;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 qa0 = Q_REGS ? qa[0][Q_REGS ? v : 0][i] : q_at(0, v, i);
                        uint2 qa1 = make_uint2(0u, 0u);
                        if constexpr (NT > 1) qa1 = Q_REGS ? qa[NT - 1][Q_REGS ? v : 0][i] : q_at(NT - 1, v, i);
#pragma unroll
                        for (int nb = 0; nb < 2 * TILES; ++nb) mma_f16(sc[nb], qa0.x, qa1.x, qa0.y, qa1.y, lo2_tiny(kw[nb][i]), hi2_tiny(kw[nb][i]));
                    }
                }
                // Rows lr and lr + 8: tokens t + 8 nb + tok[e] in sc[nb][2 u + e].
                float ks[TILES], vs[TILES];
#pragma unroll
                for (int h = 0; h < TILES; ++h) ks[h] = s_ks[pi[h]], vs[h] = s_vs[pi[h]];
                uint32_t pb[NT][2 * TILES];
                bool grew = false;
                float mt[NT], mm[NT], dt[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u)
#pragma unroll
                    for (int h = 0; h < TILES; ++h) {
                        const float f = rowf[u] * ks[h];
#pragma unroll
                        for (int nb = 2 * h; nb < 2 * h + 2; ++nb) {
                            // (rounded here, so that the largest less the maximum is 0)
                            sc[nb][2 * u] = __fmul_rn(sc[nb][2 * u], f);
                            sc[nb][2 * u + 1] = __fmul_rn(sc[nb][2 * u + 1], f);
                        }
                    }
                if (!full) {
#pragma unroll
                    for (int u = 0; u < NT; ++u)
#pragma unroll
                        for (int nb = 0; nb < 2 * TILES; ++nb)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int j = t + 8 * nb + tok[e];
                                if (!(on[nb >> 1] && j >= see_from[u] && j < see_to[u])) sc[nb][2 * u + e] = -INFINITY;
                            }
                }
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    float top[TILES];
#pragma unroll
                    for (int h = 0; h < TILES; ++h)
                        top[h] = fmaxf(fmaxf(sc[2 * h][2 * u], sc[2 * h][2 * u + 1]), fmaxf(sc[2 * h + 1][2 * u], sc[2 * h + 1][2 * u + 1]));
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1)
#pragma unroll
                        for (int h = 0; h < TILES; ++h) top[h] = fmaxf(top[h], __shfl_xor_sync(~0u, top[h], o));
                    mt[u] = m[u];
#pragma unroll
                    for (int h = 0; h < TILES; ++h) mt[u] = fmaxf(mt[u], top[h]);
                    mm[u] = base_of(mt[u]);
                    dt[u] = -INFINITY;
#pragma unroll
                    for (int h = 0; h < TILES; ++h) dt[u] = fmaxf(dt[u], (top[h] - mm[u]) + vs[h]);
                    grew |= mt[u] > m[u] || dt[u] > d[u];
                }
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
                        if (m[u] != -INFINITY) l[u] *= exp2_fast(m[u] - mt[u]);
                        const float d0 = d[u] + (m[u] - mm[u]);
                        m[u] = mt[u];
                        d[u] = fmaxf(d0, dt[u]);
                        const float a = exp2_fast(d0 - base_of(d[u]));
                        // Accumulators hold rows 2 lc + {0, 1} (+ 8 u): their factors sit in lanes 4 (2 lc + e).
                        const float a0 = __shfl_sync(~0u, a, 8 * lc), a1 = __shfl_sync(~0u, a, 8 * lc + 4);
#pragma unroll
                        for (int p = 0; p < MT; ++p) {
                            o[p][u][0] *= a0;
                            o[p][u][1] *= a1;
                            o[p][u][2] *= a0;
                            o[p][u][3] *= a1;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < NT; ++u) {
#pragma unroll
                    for (int h = 0; h < TILES; ++h) {
                        // (The largest that fp32 holds: tokens of p below 2^-112 count for less than they are.)
                        const float f = d[u] == -INFINITY ? 0.f : exp2_fast(fminf(vs[h] + (W_EXP - d[u]), 127.f));
#pragma unroll
                        for (int nb = 2 * h; nb < 2 * h + 2; ++nb) {
                            const float p0 = exp2_fast(sc[nb][2 * u] - mm[u]), p1 = exp2_fast(sc[nb][2 * u + 1] - mm[u]);
                            l[u] += p0 + p1;
                            pb[u][nb] = pack_half(p0 * f, p1 * f);
                        }
                    }
                }
                // Transposed values: tokens tok[0], tok[1] (+ 8) of d = 16 lr + .. (dim 64: 8 lr + ..).
#pragma unroll
                for (int h = 0; h < TILES; ++h) {
                    if (!on[h]) continue;                // (its codes were not fetched)
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        uint32_t a[4][VB / 4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint8_t *src = tiles + h * 16 * D + v_at[v][k];
                            if constexpr (VB == 16) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                                a[k][0] = x.x ^ 0x80808080u, a[k][1] = x.y ^ 0x80808080u;
                                a[k][2] = x.z ^ 0x80808080u, a[k][3] = x.w ^ 0x80808080u;
                            } else {
                                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                                a[k][0] = x.x ^ 0x80808080u, a[k][1] = x.y ^ 0x80808080u;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < VB / 4; ++i) {
                            // Bytes (token, token + 1) of d + 0, d + 1 and of d + 2, d + 3.
                            const uint32_t x0 = prmt(a[0][i], a[1][i], 0x5140u), x1 = prmt(a[0][i], a[1][i], 0x7362u);
                            const uint32_t y0 = prmt(a[2][i], a[3][i], 0x5140u), y1 = prmt(a[2][i], a[3][i], 0x7362u);
                            const int p = v * VB / 2 + 2 * i;
                            const uint32_t f0 = lo2(x0), f1 = hi2(x0), f2 = lo2(y0), f3 = hi2(y0);
                            const uint32_t g0 = lo2(x1), g1 = hi2(x1), g2 = lo2(y1), g3 = hi2(y1);
#pragma unroll
                            for (int u = 0; u < NT; ++u) {
                                mma_f16(o[p][u], f0, f1, f2, f3, pb[u][2 * h], pb[u][2 * h + 1]);
                                mma_f16(o[p + 1][u], g0, g1, g2, g3, pb[u][2 * h], pb[u][2 * h + 1]);
                            }
                        }
                    }
                }
                __syncwarp();                        // (every lane has read the stage that is filled next)
            }
            __syncthreads();                         // (and every warp this chunk's pages)
        }

        // Join the warps: row sums, and the outputs (in the rings' place) in warp order.
        auto out_of = [&](int wi, int r) { return reinterpret_cast<float *>(ring) + (wi * R + r) * out_pitch(D); };
        if constexpr (F == 4) {
            rows4.end(lr, lc, [&](int r, const RowSum &x) { s_sum[warp][r] = x; },
                      [&](int r, int d, float2 x) { *reinterpret_cast<float2 *>(out_of(warp, r) + d) = x; });
        } else {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                l[u] += __shfl_xor_sync(~0u, l[u], 1);
                l[u] += __shfl_xor_sync(~0u, l[u], 2);
                if (lc == 0) s_sum[warp][lr + 8 * u] = RowSum{m[u], d[u], l[u], 0.f};
            }
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float *dst = out_of(warp, 2 * lc + e + 8 * u);
#pragma unroll
                    for (int p = 0; p < MT; ++p)
                        *reinterpret_cast<float2 *>(dst + p / (VB / 2) * 8 * VB + VB * lr + 2 * (p % (VB / 2))) = make_float2(o[p][u][e], o[p][u][2 + e]);
                }
        }
        __syncthreads();
        if (tid < R) {
            RowSum a = s_sum[0][tid];
            for (int k = 1; k < WARPS; ++k) join_maxima(a, s_sum[k][tid]);
            a.l = 0.f;
            for (int k = 0; k < WARPS; ++k) {
                a.l += s_sum[k][tid].l * l_factor(s_sum[k][tid], a);
                s_wfac[k][tid] = o_factor(s_sum[k][tid], a);
            }
            s_join[tid] = a;
        }
        __syncthreads();
        auto joined4 = [&](int r, int d) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < WARPS; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(out_of(k, r) + d);
                const float f = s_wfac[k][r];
                y.x = fmaf(x.x, f, y.x), y.y = fmaf(x.y, f, y.y), y.z = fmaf(x.z, f, y.z), y.w = fmaf(x.w, f, y.w);
            }
            return y;
        };
        // Four values of an output row (aligned to 2 bytes only).
        auto store4 = [&](int r, int d, float4 x, const OutFactor &f) {
            uint16_t *dst = out_at(r) + d;
            dst[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f.of(x.x)));
            dst[1] = __bfloat16_as_ushort(__float2bfloat16_rn(f.of(x.y)));
            dst[2] = __bfloat16_as_ushort(__float2bfloat16_rn(f.of(x.z)));
            dst[3] = __bfloat16_as_ushort(__float2bfloat16_rn(f.of(x.w)));
        };
        // The CTAs that share the item, in order.
        const int c_first = cta_of(item_at), parts = cta_of(item_at + sw.steps - 1) - c_first + 1;
        if (parts == 1) {
            for (int v = 4 * tid; v < rows * D; v += 4 * THREADS)
                store4(v / D, v % D, joined4(v / D, v % D), out_factor<F>(s_join[v / D]));
        } else {
            // A CTA's first item's part is in its slot 0, that of a later one (its last) in slot 1.
            const int slot0 = 2 * c_first + (item_at - item > total * c_first / C ? 1 : 0), k_mine = (int)blockIdx.x - c_first;
            auto slot = [&](int k) { return k == 0 ? slot0 : 2 * (c_first + k); };
            float4 *sums = reinterpret_cast<float4 *>(P.part + 2LL * gridDim.x * R * D);
            float *part = P.part + (long long)slot(k_mine) * R * D;
            for (int v = 4 * tid; v < rows * D; v += 4 * THREADS)
                *reinterpret_cast<float4 *>(part + v) = joined4(v / D, v % D);
            if (tid < rows) sums[slot(k_mine) * R + tid] = make_float4(s_join[tid].m, s_join[tid].d, s_join[tid].l, 0.f);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(P.count + c_first, 1) == parts - 1;
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (tid == 0) P.count[c_first] = 0;
                // The row sums of all parts (in s_join) and the parts' factors, a warp a row.
                float(*s_fac)[R] = reinterpret_cast<float(*)[R]>(ring);      // (the outputs in the ring have been read)
                // (a lane's first parts' of all the warp's rows in one round of loads)
                constexpr int ROWS = R / WARPS, AT = 2;
                auto sum_of = [&](int r, int k) {
                    const float4 x = __ldcg(sums + slot(k) * R + r);
                    return RowSum{x.x, x.y, x.z, 0.f};
                };
                RowSum own[ROWS][AT];
#pragma unroll
                for (int j = 0; j < ROWS; ++j)
#pragma unroll
                    for (int i = 0; i < AT; ++i) own[j][i] = sum_of(min(warp + j * WARPS, rows - 1), min(lane + 32 * i, parts - 1));
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    const int r = warp + j * WARPS;
                    if (r >= rows) break;
                    RowSum a = own[j][0];
#pragma unroll
                    for (int i = 1; i < AT; ++i) join_maxima(a, own[j][i]);
                    for (int k = lane + 32 * AT; k < parts; k += 32) join_maxima(a, sum_of(r, k));
                    for (int o = 16; o > 0; o >>= 1) {
                        const float m = __shfl_xor_sync(~0u, a.m, o), d = __shfl_xor_sync(~0u, a.d, o);
                        join_maxima(a, RowSum{m, d, 0.f, 0.f});
                    }
                    a.l = 0.f;
                    auto take = [&](int k, const RowSum &x) {
                        a.l += x.l * l_factor(x, a);
                        s_fac[k][r] = o_factor(x, a);
                    };
#pragma unroll
                    for (int i = 0; i < AT; ++i)
                        if (lane + 32 * i < parts) take(lane + 32 * i, own[j][i]);
                    for (int k = lane + 32 * AT; k < parts; k += 32) take(k, sum_of(r, k));
                    for (int o = 16; o > 0; o >>= 1) a.l += __shfl_xor_sync(~0u, a.l, o);
                    if (lane == 0) s_join[r] = a;
                }
                __syncthreads();
                // The outputs, in the parts' order, JOIN parts of AT_ONCE vectors a thread at a time.
                constexpr int JOIN = F == 4 ? 16 : 8, AT_ONCE = F == 4 && D == 256 ? 2 : 1;
                for (int v0 = 4 * tid; v0 < rows * D; v0 += 4 * THREADS * AT_ONCE) {
                    float4 y[AT_ONCE];
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k0 = 0; k0 < parts; k0 += JOIN) {
                        float4 x[AT_ONCE][JOIN];
#pragma unroll
                        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                            for (int k = 0; k < JOIN; ++k)
                                x[i][k] = __ldcg(reinterpret_cast<const float4 *>(P.part + (long long)slot(min(k0 + k, parts - 1)) * R * D + min(v0 + 4 * THREADS * i, rows * D - 4)));
#pragma unroll
                        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
                            for (int k = 0; k < JOIN; ++k) {
                                const float f = k0 + k < parts ? s_fac[min(k0 + k, parts - 1)][min(v0 + 4 * THREADS * i, rows * D - 4) / D] : 0.f;
                                y[i].x = fmaf(x[i][k].x, f, y[i].x), y[i].y = fmaf(x[i][k].y, f, y[i].y);
                                y[i].z = fmaf(x[i][k].z, f, y[i].z), y[i].w = fmaf(x[i][k].w, f, y[i].w);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) {
                        const int v = v0 + 4 * THREADS * i;
                        if (v < rows * D) store4(v / D, v % D, y[i], out_factor<F>(s_join[v / D]));
                    }
                }
            }
        }
        // The ring goes back from plain stores to copies.
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        line = item_at + step1;
    }
    if (*abort && lane == 0) {
        // A wait ran out (the items were gone through all the same, so that every part has arrived and the counters
        // are zero again): no copy may be in flight when the CTA ends.
        for (uint32_t j = fit > NST ? fit - NST : 0; j < fit; ++j)
            if (!(P.stall && j == 0)) mbar_wait(&bar[j % NST], (j / NST) & 1, abort, P.status, false);
    }
}

}  // namespace attend
}  // namespace tfq
