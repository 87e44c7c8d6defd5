// rope.cu -- tf_rope: rotary positions (tfserve.h).
//
//     a' = f (a cos - b sin),   b' = f (b cos + a sin),   angle = 2 pi frac(p t / 2^64)
// p t is a 64-bit product modulo 2^64, so that the angle is exact to 2^-32 of a turn
// at any position; cosine and sine come of at most an eighth of a turn either way,
// and the quarter turns are put on by signs.
//
// Bound by memory: 4000 rows of 40 heads of 128, fp32 to bf16, are 123 MB.  A CTA
// takes a few rows: their cosines and sines once, into shared memory, for all heads;
// then a thread a place in the row, for four of the CTA's rows at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv.h"

using namespace tfq;

namespace {

constexpr int THREADS = 256, MAX_PAIRS = 512, MAX_ROWS = 8;

struct RopeParams {
    const uint64_t *turns;
    const int32_t *positions;
    const void *x;
    void *out;
    long long x_stride, out_stride;
    int rows, heads, dim, rot;
    int per_head;           // items of a head: of N pairs of the turned part, of 2 N values of the rest
    float factor;
    bool back, copy;        // turn the other way; the rest is copied (else it stands there already)
    int rows_cta = 1;       // rows of a CTA
    uint32_t by_items = 0, by_head = 0;      // reciprocals of a row's items and a head's
};

// N values: fp32, or bf16; in as few accesses as N and their size allow where VEC.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load(const T *p, float (&v)[N]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sizeof(T) == 4 ? (float)p[i] : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
    } else {
        constexpr int W = N * (int)sizeof(T) / 4;
        uint32_t w[W];
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 a = reinterpret_cast<const uint4 *>(p)[i / 4];
                w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
            }
        } else {
            static_assert(W == 2, "8 or 16 bytes at a time");
            const uint2 a = *reinterpret_cast<const uint2 *>(p);
            w[0] = a.x, w[1] = a.y;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __uint_as_float(sizeof(T) == 4 ? w[i] : i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
}
template <typename T, int N, bool VEC>
__device__ __forceinline__ void store(T *p, const float (&v)[N]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = (T)v[i];
    } else {
        constexpr int W = N * (int)sizeof(T) / 4;
        uint32_t w[W];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        }
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int i = 0; i < W; i += 4) reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        } else {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        }
    }
}

// n / d by ceil(2^32 / d), which is too large by less than 1: exact where n d < 2^32.  (0: a division.)
__device__ __forceinline__ int over(int n, uint32_t reciprocal, int d) { return reciprocal ? (int)__umulhi((uint32_t)n, reciprocal) : n / d; }

// N pairs an item; a CTA has P.rows_cta rows, and where there are few of those a part of their items (blockIdx.y).
template <typename TI, typename TO, int N, bool PAIRS, int AT, bool WIDE>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeParams P) {
    constexpr bool VEC = N > 1;
    extern __shared__ float2 s_turn[];                  // [rows_cta][rot / 2] cosine, sine
    __shared__ int s_pos[MAX_ROWS];
    const int tid = threadIdx.x, half = P.rot / 2;
    const long long r0 = (long long)blockIdx.x * P.rows_cta;
    for (int i = tid; i < P.rows_cta * half; i += THREADS) {
        const int k = i / half, j = i - k * half;
        const int pos = r0 + k < P.rows ? P.positions[r0 + k] : -1;
        if (j == 0) s_pos[k] = pos;
        const uint32_t angle = (uint32_t)(((unsigned long long)(unsigned)pos * P.turns[j]) >> 32);
        const uint32_t quarter = (angle + (1u << 29)) >> 30;
        float s, c;
        sincospif((float)(int)(angle - (quarter << 30)) * (1.f / 2147483648.f), &s, &c);
        if (quarter & 1) {
            const float t = c;
            c = -s, s = t;
        }
        if (quarter & 2) c = -c, s = -s;
        s_turn[i] = make_float2(P.factor * c, P.back ? -P.factor * s : P.factor * s);
    }
    __syncthreads();
    const int turned = half / N, items = P.heads * P.per_head, all = WIDE ? items : items * P.rows_cta;
    // A thread takes AT items at a time.  WIDE: one place of the row, in AT rows.  Else items go over the row and then over
    // the CTA's rows.
    for (int n = blockIdx.y * THREADS + tid; n < all; n += gridDim.y * THREADS * (WIDE ? 1 : AT)) {
        int row[AT], at[AT], second[AT];                // row -1: nothing to do; second: from the item's first values to its others
        int turn[AT];                                   // place of its first turn, -1: of the rest
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int m = WIDE ? n : n + i * THREADS, k = WIDE ? i : over(m, P.by_items, items), item = WIDE ? n : m - k * items;
            const int h = over(item, P.by_head, P.per_head), e = item - h * P.per_head;
            const bool rest = e >= turned;
            // The item's first and second values: pairs as they lie, or 2 N values of the rest.
            at[i] = h * P.dim + (rest ? P.rot + (e - turned) * 2 * N : PAIRS ? e * 2 * N : e * N);
            second[i] = rest || PAIRS ? N : half;
            turn[i] = rest ? -1 : k * half + e * N;
            row[i] = (WIDE || m < all) && s_pos[k] >= 0 && !(rest && !P.copy) ? k : -1;
        }
        float a[AT][N], b[AT][N];
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            if (row[i] < 0) continue;
            const TI *x = static_cast<const TI *>(P.x) + (r0 + row[i]) * P.x_stride + at[i];
            load<TI, N, VEC>(x, a[i]);
            load<TI, N, VEC>(x + second[i], b[i]);
        }
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            if (row[i] < 0) continue;
            if (turn[i] >= 0) {
                const float2 *t = s_turn + turn[i];
                if (PAIRS) {
                    float y[2 * N];
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float u = 2 * j < N ? a[i][(2 * j) % N] : b[i][(2 * j) % N], v = 2 * j + 1 < N ? a[i][(2 * j + 1) % N] : b[i][(2 * j + 1) % N];
                        const float2 z = t[j];
                        y[2 * j] = u * z.x - v * z.y;
                        y[2 * j + 1] = v * z.x + u * z.y;
                    }
#pragma unroll
                    for (int j = 0; j < N; ++j) a[i][j] = y[j], b[i][j] = y[N + j];
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float2 z = t[j];
                        const float u = a[i][j], v = b[i][j];
                        a[i][j] = u * z.x - v * z.y;
                        b[i][j] = v * z.x + u * z.y;
                    }
                }
            }
            TO *out = static_cast<TO *>(P.out) + (r0 + row[i]) * P.out_stride + at[i];
            store<TO, N, VEC>(out, a[i]);
            store<TO, N, VEC>(out + second[i], b[i]);
        }
    }
}

template <typename TI, typename TO, int N, bool PAIRS>
cudaError_t launch(RopeParams &P, int nsm, cudaStream_t st) {
    const int items = P.heads * P.per_head;
    // Four rows a CTA where that leaves some CTAs an SM, else one, and a row over as many CTAs as SMs are idle.  Rows of few
    // items: eight, and an item at a time.  (16000 rows of 16 heads of 64, bf16: 11 us, two or four items at a time 12 and 16 us,
    // four rows a CTA 31 us; 4000 rows of 40 heads of 128, fp32 to bf16: 20 us, and 24 us with the items over all rows.)
    const int half = P.rot / 2, most = (items + THREADS - 1) / THREADS;
    auto reciprocal = [](long long n, int d) { return n * d < (1LL << 32) ? (uint32_t)((0xFFFFFFFFull + d) / d) : 0u; };     // (of 1: 0, too)
    P.by_head = reciprocal(items, P.per_head);
    if ((long long)P.rows < 8LL * nsm) {
        const int cols = P.rows >= nsm ? 1 : (nsm + P.rows - 1) / P.rows;
        rope_kernel<TI, TO, N, PAIRS, 1, true><<<dim3(P.rows, cols < most ? cols : most), THREADS, half * sizeof(float2), st>>>(P);
        return cudaGetLastError();
    }
    int n = 4;
    while (n < MAX_ROWS && n * items < 2 * THREADS && (long long)P.rows >= 8LL * nsm * n) n *= 2;
    P.rows_cta = n;
    P.by_items = reciprocal((long long)items * n, items);
    const unsigned ctas = (unsigned)((P.rows + (long long)n - 1) / n);
    if (n == 4)
        rope_kernel<TI, TO, N, PAIRS, 4, true><<<ctas, THREADS, n * half * sizeof(float2), st>>>(P);
    else
        rope_kernel<TI, TO, N, PAIRS, 1, false><<<ctas, THREADS, n * half * sizeof(float2), st>>>(P);
    return cudaGetLastError();
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename TI, typename TO>
cudaError_t choose(RopeParams &P, bool pairs, int nsm, cudaStream_t st) {
    // N pairs at once where every access is then aligned: 16 bytes of fp32, 16 of bf16 where both are.
    constexpr int N = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
    const bool vec = P.rot % (2 * N) == 0 && P.dim % (2 * N) == 0 && aligned(P.x, N * sizeof(TI)) && aligned(P.out, N * sizeof(TO)) &&
                     P.x_stride % N == 0 && P.out_stride % N == 0;
    if (vec) {
        P.per_head = P.dim / (2 * N);
        return pairs ? launch<TI, TO, N, true>(P, nsm, st) : launch<TI, TO, N, false>(P, nsm, st);
    }
    P.per_head = P.dim / 2;
    return pairs ? launch<TI, TO, 1, true>(P, nsm, st) : launch<TI, TO, 1, false>(P, nsm, st);
}

}  // namespace

extern "C" int tf_rope(const uint64_t *turns, int rot, float factor, const int32_t *positions, int rows, const void *x,
                       int64_t x_stride, void *out, int64_t out_stride, int heads, int dim, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~(TF_IN_F32 | TF_OUT_BF16 | TF_ROPE_PAIRS | TF_ROPE_BACK)) return fail_message(TF_EINVAL_FLAGS, "unknown flags of tf_rope");
    const bool in32 = flags & TF_IN_F32, out16 = flags & TF_OUT_BF16;
    const int xs = in32 ? 4 : 2, os = out16 ? 2 : 4;
    if (!turns || !positions || !x || !out || !aligned(turns, 8) || !aligned(positions, 4) || !aligned(x, xs) || !aligned(out, os))
        return fail_message(TF_EINVAL_PTR, "NULL turns, positions, x or out, or not aligned to their type");
    if (rows < 1) return fail_message(TF_EINVAL_ROWS, "rows must be at least 1");
    if (heads < 1 || heads > 65536 || dim < 2 || dim > 2 * MAX_PAIRS || dim % 2 || rot < 2 || rot > dim || rot % 2)
        return fail_message(TF_EINVAL_SIZE, "heads must be in [1, 65536], dim even in [2, 1024], rot even in [2, dim]");
    const long long width = (long long)heads * dim;
    if (x_stride < width || out_stride < width) return fail_message(TF_EINVAL_STRIDE, "x_stride or out_stride below heads * dim");
    // The same rows in place, or other columns of the same rows; no other overlap.
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), oa = reinterpret_cast<uintptr_t>(out);
    const uintptr_t xe = xa + ((uintptr_t)(rows - 1) * x_stride + width) * xs, oe = oa + ((uintptr_t)(rows - 1) * out_stride + width) * os;
    const bool same = xa == oa && xs == os && (x_stride == out_stride || rows == 1);
    if (!same && xa < oe && oa < xe) {
        const uintptr_t step = (uintptr_t)x_stride * xs, lo = xa < oa ? xa : oa, by = (xa < oa ? oa : xa) - lo;
        const uintptr_t w_lo = width * (xa < oa ? xs : os), w_hi = width * (xa < oa ? os : xs);
        if (step != (uintptr_t)out_stride * os || by % step < w_lo || by % step + w_hi > step)
            return fail_message(TF_EINVAL_PTR, "out overlaps x, and is neither x itself nor other columns of its rows");
    }
    int nsm = 0, *status = nullptr;
    const int rc = device_info(&nsm, &status);
    if (rc) return rc;
    RopeParams P{turns, positions, x, out, x_stride, out_stride, rows, heads, dim, rot, 0, factor, (flags & TF_ROPE_BACK) != 0, !same};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool pairs = flags & TF_ROPE_PAIRS;
    cudaError_t e;
    if (in32)
        e = out16 ? choose<float, __nv_bfloat16>(P, pairs, nsm, st) : choose<float, float>(P, pairs, nsm, st);
    else
        e = out16 ? choose<__nv_bfloat16, __nv_bfloat16>(P, pairs, nsm, st) : choose<__nv_bfloat16, float>(P, pairs, nsm, st);
    return e == cudaSuccess ? TF_OK : cuda_error(e, "rope launch");
}
