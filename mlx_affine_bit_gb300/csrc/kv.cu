// kv.cu -- tf_kv_append and tf_kv_read: the 8-bit paged cache of tfdecode.h,
// quantized as it is written, and read back.
//
// A page (block tokens x dim of one head) has scale = amax * (1 / 127) and codes
// rint(x / scale).  Both kernels stream: append reads each new row once, holds a
// page's new values in registers between the maximum and the rounding, and
// writes codes; read turns codes into a row's values, 16 bytes of it a thread.
// Memory and, closely, instructions bound long calls, latency the short ones (a
// launch, the lengths, the page table, the rows, a barrier, the stores, one after
// another).  Measured, 8 heads of 128: append of 40000 bf16 tokens 67 us (3.7 TB/s
// of the 246 MB that it reads and writes; 121 us with each code rounded, clamped
// and tested by itself), read of them 51 us (4.8 TB/s); 4000 fp32 tokens 9.0 and
// 9.2 us; a token for each of 48 sequences, most of whose begun pages are quantized
// again, 5.9 and 2.8 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <string>

#include "kv.h"

using namespace tfq;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ----------------------------------------------------------------- append --

struct AppendParams {
    tf_kv kv;
    tf_kv_batch b;
    const void *src[2];
    long long stride[2];
    int nb;                 // pages that a sequence's new tokens may touch
    int block_log2, dim_log2;
    int *status;
};

// Eight values as they came: fp32 in eight words, bf16 in four.
template <typename T>
struct Raw8 {
    static constexpr int WORDS = sizeof(T) == 4 ? 8 : 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p, bool vec) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 a = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        } else if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ void store(T *p) const {      // (16-byte aligned)
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ float value(int i) const {
        return __uint_as_float(sizeof(T) == 4 ? w[i] : i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    // The largest magnitude; infinities and NaN left out (see the header).  Magnitudes are ordered as their bits.
    __device__ __forceinline__ float amax() const {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) top = sizeof(T) == 4 ? max(top, w[i] & 0x7FFFFFFFu) : __vmaxu2(top, w[i] & 0x7FFF7FFFu);
        if (sizeof(T) == 2) top = max(top >> 16, top & 0xFFFFu) << 16;
        if (top < 0x7F800000u) return __uint_as_float(top);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = fabsf(value(i));
            m = fmaxf(m, a <= FLT_MAX ? a : 0.f);
        }
        return m;
    }
};

// x / scale rounded to the nearest, even in the middle.
__device__ __forceinline__ int divided(float x, float scale) {
    // NaN converts to 0; an infinity saturates and is clamped.
    return scale == 0.f ? 0 : max(-127, min(127, __float2int_rn(rintf(__fdiv_rn(x, scale)))));
}
__device__ __forceinline__ float max_nan(float a, float b) {     // NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Codes of four values, and whether the division has to decide.  x * (1 / scale) is within 1.5 * 2^-23 of the
// rounded x / scale, relatively (2.3e-5 of a code at most), and rounds to the same code unless it lies that near to
// the middle of two; nor does it count for infinities and NaN (whose distance is NaN) and where 1 / scale
// overflows.  A sum with 1.5 * 2^23 rounds to the code and holds it in its low byte.
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, float scale, float inv, bool &open) {
    const float x[4] = {x0, x1, x2, x3};
    uint32_t t[4];
    float far = scale < 1e-30f ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = __fmul_rn(x[i], inv), r = __fadd_rn(q, 12582912.f);
        far = max_nan(far, fabsf(__fsub_rn(q, __fsub_rn(r, 12582912.f))));
        t[i] = __float_as_uint(r);
    }
    open = !(far <= 0.49997f);
    return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
}

constexpr int VPT = 4;      // 8-value vectors a thread: block * dim / 32 threads cover a page

// One CTA a (sequence, page, head, keys or values).  Its new tokens are read
// into registers once; if they change the scale of a page that was already
// begun, the page's earlier tokens are quantized again from the open ring.
// The last two pages' originals go into the ring.  Its halves alternate with the
// pages: a long call may put a last page where the begun page's earlier tokens
// still are, and then the begun page's CTA writes that page's originals, after
// it has read its own.
template <typename T>
__global__ void __launch_bounds__(1024) kv_append_kernel(const AppendParams P) {
    const tf_kv &kv = P.kv;
    const int H = kv.kv_heads, BL = P.block_log2, DL = P.dim_log2, B = 1 << BL, D = 1 << DL;
    const int side = blockIdx.y & 1, h = blockIdx.y >> 1;
    const int s = P.nb == 1 ? blockIdx.x : blockIdx.x / P.nb, j = blockIdx.x - s * P.nb;

    const SeqRows q = seq_rows(P.b, s);
    const int slot = P.b.slots ? P.b.slots[s] : s;
    const int first = q.end - q.n;
    const int pg = (first >> BL) + j;               // page of the sequence
    if (q.ok && q.n == 0) return;
    if (!q.ok || first < 0 || slot < 0 || slot >= kv.n_slots) {
        if (threadIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        return;
    }
    const int base = pg << BL;                      // the page's first token
    if (base >= q.end) return;
    const int page = P.b.table[s * P.b.table_stride + pg];
    const int lo = max(first, base) - base, hi = min(q.end, base + B) - base;   // new tokens of the page
    const int pg0 = first >> BL, last = (q.end - 1) >> BL;
    const bool begun = (first & (B - 1)) != 0;
    // The last two pages; one whose half of the ring the begun page occupies is left to that page's CTA.
    const bool keep = pg >= last - 1 && !(begun && pg > pg0 && ((pg - pg0) & 1) == 0);
    const T *src = static_cast<const T *>(P.src[side]);
    const bool vec = ((reinterpret_cast<uintptr_t>(src) | (P.stride[side] * sizeof(T))) & 15) == 0;
    T *ring = static_cast<T *>(side ? kv.open_v : kv.open_k) + ((((long long)slot * H + h) * 2 << BL) + (base & (2 * B - 1))) * D;
    float *ring_max = kv.open_max + ((((long long)slot * 2 + side) * H + h) * 2 << BL) + (base & (2 * B - 1));

    const int VL = DL - 3, vd = 1 << VL;            // vectors a token: 8, 16 or 32 lanes of one warp
    const int nt = blockDim.x, tid = threadIdx.x;
    // This thread's vectors: at d of tokens t0 + i * dt.
    const int d = (tid & (vd - 1)) * 8, t0 = tid >> VL, dt = B / VPT;
    Raw8<T> x[VPT];
    float amax = 0.f;
    const T *rows = src + (long long)(q.row0 + base + t0 - first) * P.stride[side] + (h << DL) + d;
    // The new rows (and the begun page's earlier magnitudes), while the page is looked up.
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int t = t0 + i * dt;
        if (t >= lo && t < hi) x[i].load(rows + i * (dt * P.stride[side]), vec);
    }
    for (int t = tid; t < lo; t += nt) amax = fmaxf(amax, ring_max[t]);
    if (page < 0 || page >= kv.n_blocks) {
        if (tid == 0) atomicOr(P.status, STATUS_BOUNDS);
        return;
    }
    int8_t *codes = (side ? kv.v : kv.k) + (((long long)page * H + h) << (BL + DL));
    float *scales = (side ? kv.v_scale : kv.k_scale) + (long long)page * H + h;
    const float old_scale = lo > 0 ? *scales : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int t = t0 + i * dt;
        const bool mine = t >= lo && t < hi;
        float m = mine ? x[i].amax() : 0.f;
        amax = fmaxf(amax, m);
        if (keep) {
            for (int o = 1; o < vd; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            if (mine) x[i].store(ring + (t << DL) + d);
            if (mine && d == 0) ring_max[t] = m;
        }
    }
    __shared__ uint32_t part[32];
    // (Magnitudes are ordered as their bits.)
    uint32_t top = __reduce_max_sync(~0u, __float_as_uint(amax));
    if ((tid & 31) == 0) part[tid >> 5] = top;
    __syncthreads();
    top = (tid & 31) < nt / 32 ? part[tid & 31] : 0u;
    amax = __uint_as_float(__reduce_max_sync(~0u, top));
    const float scale = __fmul_rn(amax, 1.f / 127.f);
    // (A long call, which takes these originals out of the ring, does so in any case.)
    const int other = (last - pg) & 1 ? last - 1 : last;      // the last page in this half of the ring
    const bool leaves = pg == pg0 && begun && other > pg;
    const bool again = lo > 0 && (scale != old_scale || leaves);
    if (tid == 0) *scales = scale;
    const float inv = __fdiv_rn(1.f, scale);
    uint32_t open = 0;                               // bit 2 i + (0, 1): four values whose codes the division decides
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int t = t0 + i * dt;
        if (t < lo && again) x[i].load(ring + (t << DL) + d, true);
        if (t < hi && (t >= lo || again)) {
            bool a, b;
            const uint32_t c0 = codes4(x[i].value(0), x[i].value(1), x[i].value(2), x[i].value(3), scale, inv, a);
            const uint32_t c1 = codes4(x[i].value(4), x[i].value(5), x[i].value(6), x[i].value(7), scale, inv, b);
            *reinterpret_cast<uint2 *>(codes + (t << DL) + d) = make_uint2(c0, c1);
            open |= ((uint32_t)a | (uint32_t)b << 1) << (2 * i);
        }
    }
    // The few that are left open (one value in some sixteen thousand) are read again, and divided.
    for (; open; open &= open - 1) {
        const int g = __ffs(open) - 1, t = t0 + (g >> 1) * dt, at = d + 4 * (g & 1);
        const T *p = t < lo ? ring + (t << DL) + at : rows + (g >> 1) * (dt * P.stride[side]) + 4 * (g & 1);
        for (int e = 0; e < 4; ++e) codes[(t << DL) + at + e] = (int8_t)divided((float)p[e], scale);
    }
    if (leaves) {
        __syncthreads();
        const int first_t = other << BL, n = min(q.end - first_t, B);
        for (int i = 0; i < VPT; ++i) {
            const int t = t0 + i * dt;
            float m = 0.f;
            if (t < n) {
                Raw8<T> y;
                y.load(src + (long long)(q.row0 + first_t + t - first) * P.stride[side] + (h << DL) + d, vec);
                m = y.amax();
                y.store(ring + (t << DL) + d);
            }
            for (int o = 1; o < vd; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            if (t < n && d == 0) ring_max[t] = m;
        }
    }
}

// ------------------------------------------------------------------- read --

struct ReadParams {
    tf_kv kv;
    tf_kv_batch b;
    void *out[2];
    long long stride[2];
    int tiles;              // tiles of READ_TOKENS tokens that a sequence may have
    int block_log2, dim_log2;
    int row_log2;           // threads a row: its 16-byte vectors, rounded up to a power of two (256 at most)
    int *status;
};
constexpr int READ_TOKENS = 16, READ_THREADS = 256;

// One CTA a (sequence, 16 of its rows, keys or values): a thread turns the codes of 16 bytes of output into
// values of a row (a warp's stores are then of whole lines), for up to eight rows at a time.
template <typename T>
__global__ void __launch_bounds__(READ_THREADS) kv_read_kernel(const ReadParams P) {
    constexpr int VEC = 16 / sizeof(T), AT = 8;
    const tf_kv &kv = P.kv;
    const int H = kv.kv_heads, BL = P.block_log2, DL = P.dim_log2, BM = kv.block - 1;
    const int side = blockIdx.y;
    const int s = P.tiles == 1 ? blockIdx.x : blockIdx.x / P.tiles, tile = blockIdx.x - s * P.tiles;
    if (!P.out[side]) return;
    const SeqRows q = seq_rows(P.b, s);
    if (!q.ok || q.end < q.n) {
        if (threadIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        return;
    }
    const int t0 = tile * READ_TOKENS, nt = min(READ_TOKENS, q.n - t0);
    if (nt <= 0) return;
    const int VL = DL - (VEC == 4 ? 2 : 3), per = H << VL;      // vectors a head, a row
    T *out = static_cast<T *>(P.out[side]);
    const bool vec = ((reinterpret_cast<uintptr_t>(out) | (P.stride[side] * sizeof(T))) & 15) == 0;
    const int step = READ_THREADS >> P.row_log2;    // rows at a time
    const int32_t *table = P.b.table + s * P.b.table_stride;
    const int8_t *pool = side ? kv.v : kv.k;
    const float *scales = side ? kv.v_scale : kv.k_scale;
    for (int c = threadIdx.x & ((1 << P.row_log2) - 1); c < per; c += 1 << P.row_log2) {
        const int h = c >> VL, d = (c & ((1 << VL) - 1)) * VEC;
        for (int tb = threadIdx.x >> P.row_log2; tb < nt; tb += AT * step) {
            uint2 w[AT];
            float scale[AT];
            int page[AT];
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int t = tb + k * step, pos = q.end - q.n + t0 + t;
                page[k] = t < nt ? table[pos >> BL] : 0;
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int t = tb + k * step, pos = q.end - q.n + t0 + t;
                if (page[k] < 0 || page[k] >= kv.n_blocks) {
                    atomicOr(P.status, STATUS_BOUNDS);
                    page[k] = -1;
                } else if (t < nt) {
                    const long long ph = (long long)page[k] * H + h;
                    const int8_t *src = pool + (((ph << BL) + (pos & BM)) << DL) + d;
                    if (VEC == 4)
                        w[k].x = *reinterpret_cast<const uint32_t *>(src);
                    else
                        w[k] = *reinterpret_cast<const uint2 *>(src);
                    scale[k] = scales[ph];
                }
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int t = tb + k * step;
                if (t >= nt || page[k] < 0) continue;
                T *dst = out + (long long)(q.row0 + t0 + t) * P.stride[side] + (h << DL) + d;
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] = scale[k] * (float)(int8_t)((i < 4 ? w[k].x : w[k].y) >> (8 * (i & 3)));
                uint4 o;
                if constexpr (VEC == 4) {
                    o = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
                } else {
                    uint32_t b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
                    o = make_uint4(b[0], b[1], b[2], b[3]);
                }
                if (vec) {
                    *reinterpret_cast<uint4 *>(dst) = o;
                } else {
                    const T *e = reinterpret_cast<const T *>(&o);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) dst[i] = e[i];
                }
            }
        }
    }
}

}  // namespace

int tfq::check_kv(const tf_kv *kv) {
    if (!kv) return fail_message(TF_EINVAL_PTR, "NULL cache");
    if (!kv->k || !kv->v || !kv->k_scale || !kv->v_scale) return fail_message(TF_EINVAL_PTR, "NULL cache pointer");
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
        return fail_message(TF_EINVAL_PTR, "k and v must be 16-byte aligned, scales 4-byte aligned");
    if (kv->block != 16 && kv->block != 32 && kv->block != 64 && kv->block != 128)
        return fail_message(TF_EINVAL_SIZE, "block must be 16, 32, 64 or 128");
    if (kv->dim != 64 && kv->dim != 128 && kv->dim != 256)
        return fail_message(TF_EINVAL_SIZE, "dim must be 64, 128 or 256");
    if (kv->kv_heads < 1 || kv->kv_heads > 1024) return fail_message(TF_EINVAL_SIZE, "kv_heads must be in [1, 1024]");
    if (kv->n_blocks < 1) return fail_message(TF_EINVAL_SIZE, "n_blocks must be at least 1");
    return TF_OK;
}

int tfq::check_batch(const tf_kv *kv, const tf_kv_batch *b) {
    if (!b) return fail_message(TF_EINVAL_PTR, "NULL batch");
    if (!b->kv_len || !b->table) return fail_message(TF_EINVAL_PTR, "NULL kv_len or table");
    if (!aligned(b->kv_len, 4) || !aligned(b->table, 4) || !aligned(b->row_start, 4) || !aligned(b->slots, 4))
        return fail_message(TF_EINVAL_PTR, "kv_len, table, row_start and slots must be 4-byte aligned");
    if (b->n_seqs < 1 || b->n_seqs > 65536) return fail_message(TF_EINVAL_SIZE, "n_seqs must be in [1, 65536]");
    if (b->rows < 1 || b->max_rows < 1 || b->max_rows > b->rows)
        return fail_message(TF_EINVAL_ROWS, "rows must be at least 1, and max_rows in [1, rows]");
    if (!b->row_start && (long long)b->n_seqs * b->max_rows != b->rows)
        return fail_message(TF_EINVAL_ROWS, "without row_start, rows must be n_seqs * max_rows");
    if (b->max_len < 1 || b->max_len > (1 << 20)) return fail_message(TF_EINVAL_SIZE, "max_len must be in [1, 2^20]");
    if (b->table_stride < (b->max_len + kv->block - 1) / kv->block)
        return fail_message(TF_EINVAL_STRIDE, "table_stride holds fewer pages than max_len needs");
    return TF_OK;
}

extern "C" int tf_kv_append(const tf_kv *kv, const tf_kv_batch *batch, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, void *stream) {
    fail_message(TF_OK, "");
    int rc = check_kv(kv);
    if (!rc) rc = check_batch(kv, batch);
    if (rc) return rc;
    if (kv->f32 != 0 && kv->f32 != 1) return fail_message(TF_EINVAL_FLAGS, "f32 must be 0 or 1");
    if (!kv->open_k || !kv->open_v || !kv->open_max || !aligned(kv->open_k, 16) || !aligned(kv->open_v, 16) ||
        !aligned(kv->open_max, 4))
        return fail_message(TF_EINVAL_PTR, "open_k and open_v must be 16-byte aligned, open_max 4-byte aligned");
    if (kv->n_slots < 1) return fail_message(TF_EINVAL_SIZE, "n_slots must be at least 1");
    if (!batch->slots && batch->n_seqs > kv->n_slots)
        return fail_message(TF_EINVAL_SIZE, "without slots, n_seqs must not exceed n_slots");
    const int es = kv->f32 ? 4 : 2;
    if (!k || !v || !aligned(k, es) || !aligned(v, es))
        return fail_message(TF_EINVAL_PTR, "NULL k or v, or not aligned to their type");
    const int width = kv->kv_heads * kv->dim;
    if (k_stride < width || v_stride < width)
        return fail_message(TF_EINVAL_STRIDE, "k_stride or v_stride below kv_heads * dim");
    int nsm = 0, *status = nullptr;
    rc = device_info(&nsm, &status);
    if (rc) return rc;
    AppendParams P{*kv, *batch, {k, v}, {k_stride, v_stride}, (batch->max_rows + kv->block - 2) / kv->block + 1,
                   __builtin_ctz(kv->block), __builtin_ctz(kv->dim), status};
    const long long pages = (long long)P.nb * batch->n_seqs;
    if (pages > 0x7FFFFFFF) return fail_message(TF_EINVAL_SIZE, "too many pages in one call");
    const int threads = kv->block * kv->dim / (8 * VPT);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)pages, 2u * kv->kv_heads);
    if (kv->f32)
        kv_append_kernel<float><<<grid, threads, 0, st>>>(P);
    else
        kv_append_kernel<__nv_bfloat16><<<grid, threads, 0, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_append launch");
}

extern "C" int tf_kv_read(const tf_kv *kv, const tf_kv_batch *batch, void *k_out, int64_t k_stride, void *v_out,
                          int64_t v_stride, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~TF_OUT_BF16) return fail_message(TF_EINVAL_FLAGS, "tf_kv_read takes TF_OUT_BF16 only");
    int rc = check_kv(kv);
    if (!rc) rc = check_batch(kv, batch);
    if (rc) return rc;
    const int es = flags & TF_OUT_BF16 ? 2 : 4;
    if ((!k_out && !v_out) || !aligned(k_out, es) || !aligned(v_out, es))
        return fail_message(TF_EINVAL_PTR, "no output, or an output not aligned to its type");
    const int width = kv->kv_heads * kv->dim;
    if ((k_out && k_stride < width) || (v_out && v_stride < width))
        return fail_message(TF_EINVAL_STRIDE, "k_stride or v_stride below kv_heads * dim");
    int nsm = 0, *status = nullptr;
    rc = device_info(&nsm, &status);
    if (rc) return rc;
    ReadParams P{*kv, *batch, {k_out, v_out}, {k_stride, v_stride}, (batch->max_rows + READ_TOKENS - 1) / READ_TOKENS,
                 __builtin_ctz(kv->block), __builtin_ctz(kv->dim), 0, status};
    while (P.row_log2 < 8 && (1 << P.row_log2) < width / (16 / es)) ++P.row_log2;
    const long long tiles = (long long)P.tiles * batch->n_seqs;
    if (tiles > 0x7FFFFFFF) return fail_message(TF_EINVAL_SIZE, "too many rows in one call");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)tiles, 2);
    if (flags & TF_OUT_BF16)
        kv_read_kernel<__nv_bfloat16><<<grid, READ_THREADS, 0, st>>>(P);
    else
        kv_read_kernel<float><<<grid, READ_THREADS, 0, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_read launch");
}
