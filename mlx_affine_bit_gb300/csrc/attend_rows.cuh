// attend_rows.cuh -- attention of few rows (single tokens, drafts) over the
// 8-bit paged cache.
//
// For the rows r of one (sequence, key/value head) -- G query heads a token --
// and the tokens j they see:
//     s_rj = (q_r . c_j) * (scale log2(e) ks_page / f_r)      q_r: fp16, times the power of two f_r
//     p_rj = 2^(s_rj - m_r),  l_r = sum_j p_rj,  out_r = sum_j p_rj vs_page c'_j / l_r
// with the running maximum m_r of a warp's tokens.  Codes are exact in fp16.  What
// enters the second product is w_rj = 2^15 p_rj vs_page 2^(m_r - n_r) in fp16, with
// the running maximum n_r of s_rj + log2(vs_page): relative to the row's largest
// contribution, however far apart the scales are, it keeps 11 bits down to 2^-29
// and comes to nothing below 2^-40.
//
// Bound by reading the cache.  A CTA takes up to 8 * NT rows and one piece of the
// tokens; a warp takes 16 tokens at a time straight from global memory into the
// fragments of mma.sync m16n8k16: a lane's 16 bytes of a key are four k steps of
// a B fragment (the rows of q are loaded in the same order), and 16 bytes of the
// values of four tokens are eight A fragments of the transposed values, whose
// token pairs are put together by the byte permutes that widen the codes anyway.
// The maxima, sums and outputs of the warps are joined in shared memory, those of
// the pieces by the last CTA to arrive, in piece order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv.h"

namespace tfq {
namespace attend {

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int STEP = 16 * WARPS;         // tokens a CTA takes at a time
constexpr int MAX_PIECE = 4096;          // tokens of one piece
constexpr int MAX_PAGES = MAX_PIECE / 16 + 1;
constexpr float W_EXP = 15.f;            // exponent offset of w in fp16

struct Params {
    tf_kv kv;
    tf_kv_batch b;
    const void *q;
    uint16_t *out;
    long long q_stride, out_stride;
    float *part;            // [grid][8 NT][dim] sums, then [grid][8 NT][3] maxima m and n, sums of p
    int *count;             // [items] arrivals, zero between launches
    int *status;
    float scale;
    int group, window, causal, q_f32;
    int tiles, piece, nsplit;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Two biased codes (c + 128) in bytes 0, 1 (or 2, 3) of w as fp16: 1024 + 128 + c, minus 1152 (exact).
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

// What has been summed of a row: maxima m of s and n of s + log2(vs), sum l of p.
struct RowSum {
    float m, n, l;
};
// Factors of a part's l and outputs in a join of maxima m and n: 0 for a part that
// saw no token (l = 0) or only values of scale 0; NaN scores (l NaN) stay NaN.
__device__ __forceinline__ float l_factor(const RowSum &p, float m) { return p.l == 0.f ? 0.f : exp2_fast(p.m - m); }
__device__ __forceinline__ float o_factor(const RowSum &p, float n) { return p.n == -INFINITY ? 0.f : exp2_fast(p.n - n); }
// Factor of the joined outputs: to the maximum of s, and by the sum.
__device__ __forceinline__ float out_factor(const RowSum &a) {
    return a.l == 0.f ? 0.f : exp2f(a.n - a.m - W_EXP) / a.l;
}

// The rows and tokens of one CTA.
struct Work {
    int s, h, tile, split;       // sequence, key/value head, tile of rows, piece
    int row0, n, end;            // the sequence's rows and tokens
    int r0, rows;                // group rows r0 .. r0 + rows - 1 (row r: token r / G, head r % G)
    int from, to, pieces;        // tokens that any of them sees, and the pieces that holds
};

// Row factor f of a magnitude: the power of two that brings it into [1, 4).
__device__ __forceinline__ float row_factor(float amax) {
    const uint32_t e = __float_as_uint(amax) >> 23;
    if (e == 0 || e == 255) return 1.f;
    return __uint_as_float((e >= 253 ? 1u : 254u - e) << 23);
}

template <int D, int NT>
__global__ void __launch_bounds__(THREADS) rows_kernel(const Params P) {
    constexpr int R = 8 * NT;                    // rows of a tile
    constexpr int KV = D / 64;                   // 16-byte vectors of a key a lane (a quad covers 64 bytes)
    constexpr int MT = D / 16;                   // m tiles of the transposed values
    __shared__ __align__(16) __half sq[R][D];
    __shared__ float s_row[R];
    __shared__ RowSum s_sum[WARPS][R];
    __shared__ float s_ks[MAX_PAGES], s_vs[MAX_PAGES];
    __shared__ int s_page[MAX_PAGES];
    __shared__ __align__(16) float so[R][D + 4];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = lane >> 2, lc = lane & 3;
    const int H = P.kv.kv_heads, B = P.kv.block, G = P.group;

    Work w;
    unsigned id = blockIdx.x;
    w.split = id % P.nsplit;
    id /= P.nsplit;
    const unsigned item = id;
    w.tile = id % P.tiles;
    id /= P.tiles;
    w.h = id % H;
    w.s = id / H;
    const SeqRows q = seq_rows(P.b, w.s);
    w.row0 = q.row0;
    w.n = q.n;
    w.end = q.end;
    if (!q.ok) {
        if (tid == 0) atomicOr(P.status, STATUS_BOUNDS);
        // Rows that lie within the matrices get zeros.
        if (w.row0 < 0 || w.n < 0 || w.n > P.b.max_rows || w.row0 + w.n > P.b.rows) return;
        w.end = 0;
    }
    w.r0 = w.tile * R;
    w.rows = min(R, w.n * G - w.r0);
    if (w.rows <= 0) return;
    // Tokens that the tile's rows may see.
    const int i0 = w.r0 / G, i1 = (w.r0 + w.rows - 1) / G;       // first and last of its tokens
    w.from = 0;
    w.to = w.end;
    if (P.causal) {
        w.to = min(w.end, w.end - w.n + i1 + 1);
        if (P.window) w.from = max(0, w.end - w.n + i0 - P.window + 1);
    }
    const int base = w.from / 16 * 16;
    w.pieces = w.to > w.from ? (w.to - base + P.piece - 1) / P.piece : 0;
    uint16_t *out = P.out + (long long)w.row0 * P.out_stride;
    auto out_at = [&](int r) {                  // first value of the tile's row r
        const int gr = w.r0 + r, i = gr / G;
        return out + (long long)i * P.out_stride + ((long long)w.h * G + gr - i * G) * D;
    };
    if (w.pieces == 0) {
        if (w.split == 0)
            for (int v = tid; v < w.rows * D; v += THREADS) out_at(v / D)[v % D] = 0;
        return;
    }
    if (w.split >= w.pieces) return;
    const int t0 = base + w.split * P.piece, t1 = min(t0 + P.piece, w.to);   // tokens of the piece

    // Pages and scales of the piece (of the values' the logarithm).
    const int pg0 = t0 / B, npages = (t1 - 1) / B - pg0 + 1;
    for (int i = tid; i < npages; i += THREADS) {
        int page = P.b.table[w.s * P.b.table_stride + pg0 + i];
        if (page < 0 || page >= P.kv.n_blocks) {
            atomicOr(P.status, STATUS_BOUNDS);
            page = -1;
        }
        s_page[i] = page;
        const long long ph = (long long)page * H + w.h;
        s_ks[i] = page < 0 ? 0.f : P.kv.k_scale[ph];
        s_vs[i] = page < 0 ? -INFINITY : log2f(P.kv.v_scale[ph]);
    }
    // The rows of q in fp16, times a power of two each.
    for (int r = warp; r < R; r += WARPS) {
        float x[D / 32], m = 0.f;
        const int gr = w.r0 + r, i = gr / G;
        const long long at = (long long)(w.row0 + i) * P.q_stride + ((long long)w.h * G + gr - i * G) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            x[e] = 0.f;
            if (r < w.rows)
                x[e] = P.q_f32 ? static_cast<const float *>(P.q)[at + e * 32 + lane]
                               : __uint_as_float((uint32_t) static_cast<const uint16_t *>(P.q)[at + e * 32 + lane] << 16);
            m = fmaxf(m, fabsf(x[e]));
        }
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const float f = row_factor(m);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) sq[r][e * 32 + lane] = __float2half_rn(x[e] * f);
        if (lane == 0) s_row[r] = P.scale * 1.44269504088896340736f / f;
    }
    __syncthreads();

    // A fragments of q: k step (v, i) holds d = 64 v + 16 lc + 4 i + {0, 1 | 2, 3}.
    uint2 qa[NT][KV][4];
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int v = 0; v < KV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qa[u][v][i] = *reinterpret_cast<const uint2 *>(&sq[lr + 8 * u][64 * v + 16 * lc + 4 * i]);
    float rowf[NT];
    int see_from[NT], see_to[NT];                // tokens that rows lr (+ 8) see
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        const int r = min(lr + 8 * u, w.rows - 1);   // (rows past the tile's end are computed, never stored)
        rowf[u] = s_row[r];
        const int pos = w.end - w.n + (w.r0 + r) / G;
        see_to[u] = P.causal ? min(w.end, pos + 1) : w.end;
        see_from[u] = P.window ? pos - P.window + 1 : 0;
    }
    int all_from = 0, all_to = w.end;            // tokens that every row of the tile sees
    if (P.causal) {
        all_to = min(w.end, w.end - w.n + i0 + 1);
        if (P.window) all_from = w.end - w.n + i1 - P.window + 1;
    }

    float o[MT][NT][4];
    float m[NT], n[NT], l[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        m[u] = n[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int p = 0; p < MT; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[p][u][e] = 0.f;
    }
    for (int t = t0 + 16 * warp; t < t1; t += STEP) {
        const int pi = t / B - pg0, page = s_page[pi];
        if (page < 0) continue;
        const long long at = (((long long)page * H + w.h) * B + t % B) * D;
        const int8_t *kp = P.kv.k + at, *vp = P.kv.v + at;
        // Scores of 16 tokens: two n tiles of 8.
        float sc[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nb][e] = 0.f;
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                const uint4 kk = *reinterpret_cast<const uint4 *>(kp + (8 * nb + lr) * D + 64 * v + 16 * lc);
                const uint32_t kw[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = kw[i] ^ 0x80808080u;
                    mma_f16(sc[nb], qa[0][v][i].x, NT > 1 ? qa[NT - 1][v][i].x : 0u, qa[0][v][i].y,
                            NT > 1 ? qa[NT - 1][v][i].y : 0u, lo2(x), hi2(x));
                }
            }
        }
        // Rows lr and lr + 8: tokens t + 8 nb + 2 lc + {0, 1} in sc[nb][2 u + {0, 1}].
        const bool full = t >= all_from && t + 16 <= all_to;
        const float ks = s_ks[pi], vs = s_vs[pi];
        uint32_t pb[NT][2];
        bool grew = false;
        float mt[NT], nt[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const float f = rowf[u] * ks;
            float top = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = sc[nb][2 * u + e];
                    x *= f;
                    const int j = t + 8 * nb + 2 * lc + e;
                    if (!full && !(j >= see_from[u] && j < see_to[u])) x = -INFINITY;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            mt[u] = fmaxf(m[u], top);
            nt[u] = fmaxf(n[u], top + vs);
            grew |= mt[u] > m[u] || nt[u] > n[u];
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                if (m[u] != -INFINITY) l[u] *= exp2_fast(m[u] - mt[u]);
                const float a = n[u] == -INFINITY ? 0.f : exp2_fast(n[u] - nt[u]);
                m[u] = mt[u];
                n[u] = nt[u];
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
            const float mm = m[u] == -INFINITY ? 0.f : m[u];
            const float f = n[u] == -INFINITY ? 0.f : exp2_fast(fminf(mm + vs - n[u] + W_EXP, 115.f));
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const float p0 = exp2_fast(sc[nb][2 * u] - mm), p1 = exp2_fast(sc[nb][2 * u + 1] - mm);
                l[u] += p0 + p1;
                pb[u][nb] = pack_half(p0 * f, p1 * f);
            }
        }
        // Transposed values: tokens 2 lc, 2 lc + 1 (+ 8) of d = 16 lr + .. (D = 64: 8 lr + ..).
        constexpr int VB = D >= 128 ? 16 : 8;        // bytes a lane takes of a token at once
#pragma unroll
        for (int v = 0; v < D / (8 * VB); ++v) {
            uint32_t a[4][VB / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int8_t *src = vp + (2 * lc + (k & 1) + 8 * (k >> 1)) * D + v * 8 * VB + VB * lr;
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
                    mma_f16(o[p][u], f0, f1, f2, f3, pb[u][0], pb[u][1]);
                    mma_f16(o[p + 1][u], g0, g1, g2, g3, pb[u][0], pb[u][1]);
                }
            }
        }
    }

    // Join the warps: row sums, then the outputs in warp order.
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        l[u] += __shfl_xor_sync(~0u, l[u], 1);
        l[u] += __shfl_xor_sync(~0u, l[u], 2);
        if (lc == 0) s_sum[warp][lr + 8 * u] = RowSum{m[u], n[u], l[u]};
    }
    __syncthreads();
    auto joined = [&](int r) {
        RowSum a = s_sum[0][r];
        for (int k = 1; k < WARPS; ++k) a.m = fmaxf(a.m, s_sum[k][r].m), a.n = fmaxf(a.n, s_sum[k][r].n);
        a.l = 0.f;
        for (int k = 0; k < WARPS; ++k) a.l += s_sum[k][r].l * l_factor(s_sum[k][r], a.m);
        return a;
    };
    constexpr int VB = D >= 128 ? 16 : 8;
    for (int wi = 0; wi < WARPS; ++wi) {
        if (warp == wi) {
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * lc + e + 8 * u;
                    const float a = o_factor(s_sum[wi][r], joined(r).n);
#pragma unroll
                    for (int p = 0; p < MT; ++p) {
                        const int d = p / (VB / 2) * 8 * VB + VB * lr + 2 * (p % (VB / 2));
                        float *dst = &so[r][d];
                        if (wi == 0) {
                            dst[0] = o[p][u][e] * a;
                            dst[1] = o[p][u][2 + e] * a;
                        } else {
                            dst[0] += o[p][u][e] * a;
                            dst[1] += o[p][u][2 + e] * a;
                        }
                    }
                }
        }
        __syncthreads();
    }
    auto store = [&](int r, int d, float x) {
        out_at(r)[d] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    };
    if (w.pieces == 1) {
        for (int v = tid; v < w.rows * D; v += THREADS) store(v / D, v % D, so[v / D][v % D] * out_factor(joined(v / D)));
        return;
    }
    // A part: its outputs and row sums.
    const long long first = (long long)item * P.nsplit;
    RowSum *sums = reinterpret_cast<RowSum *>(P.part + (long long)gridDim.x * R * D) + first * R;
    float *part = P.part + first * R * D;
    for (int v = tid; v < w.rows * D; v += THREADS) part[w.split * R * D + v] = so[v / D][v % D];
    if (tid < w.rows) sums[w.split * R + tid] = joined(tid);
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(P.count + item, 1) == w.pieces - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (tid == 0) P.count[item] = 0;
    auto sum_of = [&](int k, int r) {
        const float *x = &sums[k * R + r].m;
        return RowSum{__ldcg(x), __ldcg(x + 1), __ldcg(x + 2)};
    };
    for (int v = tid; v < w.rows * D; v += THREADS) {
        const int r = v / D;
        RowSum a{-INFINITY, -INFINITY, 0.f};
        for (int k = 0; k < w.pieces; ++k) {
            const RowSum x = sum_of(k, r);
            a.m = fmaxf(a.m, x.m);
            a.n = fmaxf(a.n, x.n);
        }
        float acc = 0.f;
        for (int k = 0; k < w.pieces; ++k) {
            const RowSum x = sum_of(k, r);
            a.l += x.l * l_factor(x, a.m);
            acc += __ldcg(part + (long long)k * R * D + v) * o_factor(x, a.n);
        }
        store(r, v % D, acc * out_factor(a));
    }
}

}  // namespace attend
}  // namespace tfq
