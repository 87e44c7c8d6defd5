// attend_rows.cuh -- attention of few rows (single tokens, drafts) over the
// 8-bit paged cache.
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
constexpr int NO_TOKEN = 1 << 30;        // past every chunk
constexpr float W_EXP = 15.f;            // exponent offset of w in fp16

struct Params {
    CUtensorMap tm_k, tm_v;  // the pools as rows of 128 bytes; a box is a pair of tiles, or one of 16-token pages
    tf_kv kv;
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
// Factor of the joined outputs: to the maximum of s, and by the sum.
__device__ __forceinline__ float out_factor(const RowSum &a) { return a.l == 0.f ? 0.f : exp2f(a.d - W_EXP) / a.l; }

// Stages of a warp's ring, and CTAs an SM by the shared memory that the rings and the registers that outputs and q
// take.  48 sequences of up to 8000 tokens, 8 heads of 128: 79 us so, 81 with one tile a stage and four stages, 83
// with three stages and two CTAs; one of 131072 tokens 52, 54 and 50.
TFQ_HD constexpr int stages(int d) { return d == 256 ? 3 : 2; }
TFQ_HD constexpr int ctas(int d, int nt) { return d == 64 ? (nt == 1 ? 5 : 4) : d == 128 ? 3 : 2; }
TFQ_HD constexpr int tile_bytes(int d) { return 32 * d; }          // 16 tokens of keys and of values
TFQ_HD constexpr int out_pitch(int d) { return d + 4; }            // floats between joined rows
// Shared memory: the rings; after the tokens are done, every warp's outputs, then the parts' factors.
TFQ_HD constexpr int smem_bytes(int d, int nt) {
    const int ring = WARPS * stages(d) * tiles_of(d) * tile_bytes(d), outs = WARPS * 8 * nt * out_pitch(d) * 4;
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

template <int D, int NT>
__global__ void __launch_bounds__(THREADS, ctas(D, NT)) rows_kernel(const __grid_constant__ Params P) {
    constexpr int R = 8 * NT;                    // rows of a tile
    constexpr int KV = D / 64;                   // 16-byte vectors of a key a lane (a quad covers 64 bytes)
    constexpr int MT = D / 16;                   // m tiles of the transposed values
    constexpr int VB = D >= 128 ? 16 : 8;        // bytes that a lane takes of a token's values at once
    constexpr int NV = D / (8 * VB);             // ... and how often
    constexpr int NST = stages(D), TILES = tiles_of(D), TP = 16 * TILES, STEP = step_of(D);
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ uint64_t bars[WARPS][NST];
    __shared__ int s_abort;
    __shared__ __align__(16) __half sq[R][D + 8];
    __shared__ float2 s_row[R];
    __shared__ RowSum s_sum[WARPS][R], s_join[R];    // of each warp, and of all of them
    __shared__ float s_wfac[WARPS][R];               // factors of the warps' outputs in the join
    __shared__ float s_ks[MAX_PAGES], s_vs[MAX_PAGES];
    __shared__ int s_page[MAX_PAGES];
    __shared__ long long s_warp[WARPS], s_first;
    __shared__ int s_seq;
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = lane >> 2, lc = lane & 3;
    const int H = P.kv.kv_heads, G = P.group, BL = P.block_log2, BM = P.kv.block - 1;

    // This CTA's share: steps [u0, u1) of the line, whose first sequence is s_seq, at s_first of the line.
    const int per = (P.b.n_seqs + THREADS - 1) / THREADS;
    const int s0 = tid * per, s1 = min(P.b.n_seqs, s0 + per);
    long long mine_sum = 0;
    for (int s = s0; s < s1; ++s) {
        const SeqWork w = seq_work<D, R>(P, s);
        if (!w.q.ok && blockIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        mine_sum += (long long)H * w.tiles * w.steps;
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
            const long long n = (long long)H * w.tiles * w.steps;
            if (u0 < at + n) break;
            at += n;
        }
        s_seq = s;
        s_first = at;
    }
    __syncthreads();

    // A warp's ring: stages of a pair of tiles' keys, then their values.
    constexpr int STAGE = TILES * tile_bytes(D);
    uint8_t *mine = ring + warp * NST * STAGE;
    uint64_t *bar = bars[warp];
    volatile int *abort = &s_abort;
    const bool single = TILES == 2 && BL == 4;   // pages of one tile only: a stage's tiles come from two
    uint32_t fit = 0, it = 0;                    // pairs fetched and taken, over all items
    // Offsets of this lane's reads in a stage: keys of token order(lr) (+ 8, + 16, + 24), values of four tokens of a tile.
    int k_at[KV][2], v_at[NV][4];
    const int tok[2] = {order<D>(2 * lc), order<D>(2 * lc + 1)};
#pragma unroll
    for (int v = 0; v < KV; ++v)
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) k_at[v][nb] = swizzled((order<D>(lr) + 8 * nb) * D + 64 * v + 16 * lc);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) v_at[v][k] = swizzled((tok[k & 1] + 8 * (k >> 1)) * D + v * 8 * VB + VB * lr) + STAGE / 2;

    int seq = s_seq;
    long long seq_at = s_first;                  // the sequence's first step on the line
    SeqWork sw = seq_work<D, R>(P, seq);
    for (long long line = u0; line < u1;) {
        while (line >= seq_at + (long long)H * sw.tiles * sw.steps) {
            seq_at += (long long)H * sw.tiles * sw.steps;
            sw = seq_work<D, R>(P, ++seq);
        }
        // The item: a head and a tile of the sequence's rows; this CTA's steps of it.
        const int index = (int)((line - seq_at) / sw.steps), h = index / sw.tiles, tile = index - h * sw.tiles;
        const long long item_at = seq_at + (long long)index * sw.steps;
        const int step0 = (int)(line - item_at), step1 = (int)min((long long)sw.steps, u1 - item_at);
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
        const int from = P.window ? max(0, first + i0 - P.window + 1) & ~31 : 0;
        int c0 = max(t_begin, from), c1 = c0, pg0 = 0, npages = 0, ft = 0;
        auto fetch = [&](int t) {                // (the warp's first lane)
            if (t >= c1) return;
            const uint32_t stage = fit++ % NST;
            if (P.stall && fit == 1) return;
            const int p0 = s_page[(t >> BL) - pg0], p1 = single && t + 16 < c1 ? s_page[(t >> BL) + 1 - pg0] : -1;
            mbar_arrive_tx(&bar[stage], (uint32_t)((p0 >= 0 ? (single ? 1 : TILES) : 0) + (p1 >= 0 ? 1 : 0)) * tile_bytes(D));
            uint8_t *dst = mine + stage * STAGE;
            auto copy = [&](int page, int at, uint8_t *to) {
                const int row = (int)((((((long long)page * H + h) << BL) + (at & BM)) * D) >> 7);
                tma_2d(to, &P.tm_k, 0, row, &bar[stage]);
                tma_2d(to + STAGE / 2, &P.tm_v, 0, row, &bar[stage]);
            };
            if (p0 >= 0) copy(p0, t, dst);
            if (p1 >= 0) copy(p1, t + 16, dst + 16 * D);
        };
        auto open_chunk = [&]() {
            c1 = min(c0 + CHUNK_TOKENS, t_end);
            pg0 = c0 >> BL;
            npages = ((c1 - 1) >> BL) - pg0 + 1;
            for (int i = tid; i < npages; i += THREADS) {
                int page = P.b.table[seq * P.b.table_stride + pg0 + i];
                if (page < 0 || page >= P.kv.n_blocks) {
                    atomicOr(P.status, STATUS_BOUNDS);
                    page = -1;
                }
                s_page[i] = page;
            }
            __syncthreads();
            ft = *abort ? NO_TOKEN : c0 + TP * warp;
            for (int i = 0; i < NST - 1; ++i, ft += STEP)
                if (lane == 0) fetch(ft);
            for (int i = tid; i < npages; i += THREADS) {
                const long long ph = (long long)s_page[i] * H + h;
                s_ks[i] = s_page[i] < 0 ? 0.f : P.kv.k_scale[ph];
                s_vs[i] = s_page[i] < 0 ? -INFINITY : log2f(P.kv.v_scale[ph]);
            }
        };
        if (c0 < t_end) open_chunk();            // (the loads of q are on their way meanwhile)
#pragma unroll
        for (int k = 0; k < R / WARPS; ++k) {
            const int r = warp + k * WARPS;
            float m = 0.f, sum = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) m = fmaxf(m, fabsf(qx[k][e]));
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            const float f = row_factor(m);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const __half x = __float2half_rn(qx[k][e] * f);
                sq[r][e * 32 + lane] = x;
                sum += __half2float(x);
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (lane == 0) s_row[r] = make_float2(P.scale * 1.44269504088896340736f / f * (1.f / TINY), sum * (-128.f * TINY));
        }
        __syncthreads();

        // A fragments of q: k step (v, i) holds d = 64 v + 16 lc + 4 i + {0, 1 | 2, 3}.  (dim 256: read again for every tile.)
        constexpr bool Q_REGS = D < 256;
        uint2 qa[NT][Q_REGS ? KV : 1][4];
        auto q_at = [&](int u, int v, int i) { return *reinterpret_cast<const uint2 *>(&sq[lr + 8 * u][64 * v + 16 * lc + 4 * i]); };
        if constexpr (Q_REGS) {
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
            for (int t = c0 + TP * warp; t < c1; t += STEP, ++it) {
                if (lane == 0) fetch(ft);
                ft += STEP;
                if (!mbar_try(&bar[it % NST], (it / NST) & 1)) {
                    if (!*abort) mbar_wait(&bar[it % NST], (it / NST) & 1, abort, P.status);
                    if (*abort) ft = NO_TOKEN;       // (a wait ran out: nothing more is fetched, the stages may be on their way)
                }
                const uint8_t *tiles = mine + (it % NST) * STAGE;
                // Tiles t and t + 16: their pages (a tile of no page is not seen).
                int pi[TILES];
                bool on[TILES];
#pragma unroll
                for (int h = 0; h < TILES; ++h) {
                    pi[h] = min(((t + 16 * h) >> BL) - pg0, npages - 1);
                    on[h] = s_page[pi[h]] >= 0 && !(h == 1 && single && t + 16 >= c1);
                }
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
                const bool full = t >= all_from && t + TP <= all_to && on[0] && on[TILES - 1];
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
                        const float f = d[u] == -INFINITY ? 0.f : exp2_fast(fminf(vs[h] + (W_EXP - d[u]), 115.f));
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
                for (int p = 0; p < MT; ++p) {
                    const int d = p / (VB / 2) * 8 * VB + VB * lr + 2 * (p % (VB / 2));
                    *reinterpret_cast<float2 *>(dst + d) = make_float2(o[p][u][e], o[p][u][2 + e]);
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
        auto store4 = [&](int r, int d, float4 x, float f) {
            uint16_t *dst = out_at(r) + d;
            dst[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x.x * f));
            dst[1] = __bfloat16_as_ushort(__float2bfloat16_rn(x.y * f));
            dst[2] = __bfloat16_as_ushort(__float2bfloat16_rn(x.z * f));
            dst[3] = __bfloat16_as_ushort(__float2bfloat16_rn(x.w * f));
        };
        // The CTAs that share the item, in order.
        const int c_first = cta_of(item_at), parts = cta_of(item_at + sw.steps - 1) - c_first + 1;
        if (parts == 1) {
            for (int v = 4 * tid; v < rows * D; v += 4 * THREADS)
                store4(v / D, v % D, joined4(v / D, v % D), out_factor(s_join[v / D]));
        } else {
            // A CTA's first item's part is in its slot 0, that of a later one (its last) in slot 1.
            const int slot0 = 2 * c_first + (item_at > total * c_first / C ? 1 : 0), k_mine = (int)blockIdx.x - c_first;
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
                for (int r = warp; r < rows; r += WARPS) {
                    auto sum_of = [&](int k) {
                        const float4 x = __ldcg(sums + slot(k) * R + r);
                        return RowSum{x.x, x.y, x.z, 0.f};
                    };
                    const RowSum own = sum_of(min(lane, parts - 1));
                    RowSum a = own;
                    for (int k = lane + 32; k < parts; k += 32) join_maxima(a, sum_of(k));
                    for (int o = 16; o > 0; o >>= 1) {
                        const float m = __shfl_xor_sync(~0u, a.m, o), d = __shfl_xor_sync(~0u, a.d, o);
                        join_maxima(a, RowSum{m, d, 0.f, 0.f});
                    }
                    a.l = 0.f;
                    for (int k = lane; k < parts; k += 32) {
                        const RowSum x = k < 32 ? own : sum_of(k);
                        a.l += x.l * l_factor(x, a);
                        s_fac[k][r] = o_factor(x, a);
                    }
                    for (int o = 16; o > 0; o >>= 1) a.l += __shfl_xor_sync(~0u, a.l, o);
                    if (lane == 0) s_join[r] = a;
                }
                __syncthreads();
                // The outputs, in the parts' order, eight loads at a time.
                for (int v = 4 * tid; v < rows * D; v += 4 * THREADS) {
                    const int r = v / D;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k0 = 0; k0 < parts; k0 += 8) {
                        float4 x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            x[k] = __ldcg(reinterpret_cast<const float4 *>(P.part + (long long)slot(min(k0 + k, parts - 1)) * R * D + v));
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float f = k0 + k < parts ? s_fac[min(k0 + k, parts - 1)][r] : 0.f;
                            y.x = fmaf(x[k].x, f, y.x), y.y = fmaf(x[k].y, f, y.y);
                            y.z = fmaf(x[k].z, f, y.z), y.w = fmaf(x[k].w, f, y.w);
                        }
                    }
                    store4(r, v % D, y, out_factor(s_join[r]));
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
