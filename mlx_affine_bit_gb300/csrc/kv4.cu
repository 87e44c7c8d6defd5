// kv4.cu -- tf_kv4_append and tf_kv4_read: the 4-bit paged cache of tfserve.h, quantized
// as it is written, and read back.
//
// Of every 64 values of a token's head: bias = the bf16 number at or below the smallest,
// scale = the bf16 number at or above (largest - bias) / 15, codes rint((x - bias) / scale),
// all as if computed exactly: where fp32 is not sure to decide alike, the exact difference
// (as two fp32 numbers) is compared with the exact border.
//
// Eight lanes hold a group, eight values each: 16 or 32 bytes in, one word of codes out.
// 4000 rows of 8 heads of 128, fp32: written 11 us, 37 MB (with every value's checks for infinities and NaN before the
// group's instead of beside it, divisions of 64 bits for its place and an exact reciprocal: 15 us; two or four vectors a
// thread at a time: no faster), read back 9.4 us.  A few rows take 3 us each, a chain of latencies: a launch, the slot
// beside the row, three shuffles, the stores; lengths, pages, codes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv.h"

using namespace tfq;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int THREADS = 256;
constexpr float MOST = 85070591730234615865843651857942052864.f;     // 2^126

// Eight values of a row.
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        if (vec) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i];
        }
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(h);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)h[i] << 16);
        }
    }
}

// The bf16 number at or below x (finite), at or above x (finite, not negative); as fp32.
__device__ __forceinline__ float bf16_below(float x) {
    const int b = __float_as_int(x), cut = b & (int)0xFFFF0000;
    return __int_as_float(b < 0 && cut != b ? cut + 0x10000 : cut) + 0.f;      // (-0 as 0)
}
__device__ __forceinline__ float bf16_above(float x) {
    return __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u);
}
// a - b as fp32 and what that rounding left out, exactly.
__device__ __forceinline__ float minus(float a, float b, float &left) {
    const float d = __fsub_rn(a, b), z = __fsub_rn(d, a);
    left = __fsub_rn(__fsub_rn(a, __fsub_rn(d, z)), __fadd_rn(b, z));
    return d;
}
// The scale of values from bias to hi: the quotient, a little low, gives the number of 8 bits that is wanted or
// the one before it, and 15 of them (exact) are compared with the exact difference.
__device__ __forceinline__ float scale_of(float bias, float hi) {
    float left;
    const float d = minus(hi, bias, left);
    const float s = bf16_above(__fmul_rn(d, (1.f - 0x1p-21f) / 15.f)), reach = __fmul_rn(15.f, s);
    return reach < d || (reach == d && left > 0.f) ? __uint_as_float(__float_as_uint(s) + 0x10000u) : s;
}

struct AppendParams {
    tf_kv4 kv;
    const long long *slots;
    const void *src[2];
    long long stride[2];
    long long items;        // rows' keys and values: 2 rows
    int items_cta;          // of a CTA, whose vectors of eight values go over them one after another
    uint32_t by_row;        // 2^32 over a row's vectors, rounded up: exact for a CTA's (0: one item only)
    int block_log2, dim_log2;
    int *status;
};

// Eight values of a group whose smallest and largest (whole numbers only) its eight lanes share: scale, bias, codes.
// plain: no value is NaN, infinite or past 2^126, so that none lies outside of [lo, hi].
__device__ __forceinline__ uint32_t codes_of(float (&x)[8], float lo, float hi, bool plain, float &scale, float &bias) {
    bias = bf16_below(lo);
    float b = bias, sc;
    if (hi - bias < 1e-25f) {
        // (So small numbers are scaled up first, out of the reach of subnormals: values are below 1e-17 then.  Or they are all one
        // bf16 number of any size, which stays as it is: differences of 0, and codes of 0.)
        const float m = hi > bias ? 18446744073709551616.f : 1.f;    // 2^64
        scale = hi > bias ? fmaxf(bf16_above(__fmul_rn(scale_of(bias * m, hi * m), 0x1p-64f)), 0x1p-133f) : 0.f;
        b = bias * m, sc = scale * m;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= m;
    } else {
        sc = scale = scale_of(bias, hi);
    }
    // x - bias over scale, rounded by a sum with 1.5 * 2^23: within 4e-6 of the true quotient (2^-24 of the difference,
    // 2^-23 of the reciprocal and 2^-24 of their product, of up to 15).
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sc));
    if (sc == 0.f) inv = 0.f;
    float q[8], far = 0.f;
    // The sums' low bits are the codes; what their high bits, 0x4B400000 each, add to the word is taken off first.
    uint32_t word = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = __fmul_rn(__fsub_rn(x[i], b), inv);
        if (!plain) q[i] = fminf(fmaxf(q[i], 0.f), 15.f);
        const float r = __fadd_rn(q[i], 12582912.f);
        far = fmaxf(far, fabsf(__fsub_rn(q[i], __fsub_rn(r, 12582912.f))));
        word += __float_as_uint(r) * (1u << (4 * i));
    }
    if (far > 0.49999f) {
        // Nearly the middle of two codes for some value: there the middle (exact) is compared with the exact difference.
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float left;
            const float r = rintf(q[i]), low = floorf(q[i]), d = minus(x[i], b, left), mid = __fmul_rn(low + 0.5f, sc);
            const bool up = d > mid || (d == mid && (left > 0.f || (left == 0.f && ((int)low & 1))));
            const int code = fabsf(q[i] - r) > 0.49999f ? (int)low + up : (int)r;
            word |= (uint32_t)code << (4 * i);
        }
    }
    return word;
}

// A vector of eight values a thread; items are a row's keys or its values.
template <typename T>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(const AppendParams P) {
    const tf_kv4 &kv = P.kv;
    const int H = kv.kv_heads, BL = P.block_log2, DL = P.dim_log2;
    const int per = H << (DL - 3);               // vectors of an item (a multiple of 8: a group's lanes stay together)
    const long long item0 = (long long)blockIdx.x * P.items_cta;
    const int all = (int)min((long long)P.items_cta, P.items - item0) * per;
    const int n = blockIdx.y * THREADS + threadIdx.x, in = P.by_row ? (int)__umulhi((uint32_t)n, P.by_row) : 0;
    const long long item = item0 + in, row = item >> 1;
    const int side = (int)(item & 1), c = n - in * per;
    float x[8] = {};
    long long slot = -1;
    if (n < all) {
        slot = P.slots[row];
        const T *src = static_cast<const T *>(side ? P.src[1] : P.src[0]);
        const long long stride = side ? P.stride[1] : P.stride[0];
        const bool vec = ((reinterpret_cast<uintptr_t>(src) | (stride * sizeof(T))) & 15) == 0;
        load8<T>(src + row * stride + 8 * c, vec, x);
    }
    float lo = x[0], hi = x[0], zero = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        zero = fmaf(x[i], 0.f, zero);            // (NaN of an infinity or a NaN)
    }
    const bool plain = zero == 0.f && lo >= -MOST && hi <= MOST;
    if (!plain) {
        lo = INFINITY, hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = x[i];
            const bool whole = fabsf(y) < INFINITY;
            x[i] = y == y ? fminf(fmaxf(y, -MOST), MOST) : 0.f;
            lo = fminf(lo, whole ? x[i] : INFINITY);
            hi = fmaxf(hi, whole ? x[i] : -INFINITY);
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
    }
    if (lo == INFINITY) lo = hi = 0.f;           // no finite value
    float scale, bias;
    const uint32_t word = codes_of(x, lo, hi, plain, scale, bias);
    if (slot < 0 || slot >= (long long)kv.n_blocks << BL) {
        if (slot != -1) atomicOr(P.status, STATUS_BOUNDS);
        return;
    }
    const int h = c >> (DL - 3), d = c & ((1 << (DL - 3)) - 1);
    const long long at = ((((slot >> BL) * H + h) << BL) + (slot & (kv.block - 1)));
    reinterpret_cast<uint32_t *>(side ? kv.v : kv.k)[(at << (DL - 3)) + d] = word;
    if ((d & 7) == 0)
        reinterpret_cast<uint32_t *>(side ? kv.v_affine : kv.k_affine)[(at << (DL - 6)) + (d >> 3)] =
            (__float_as_uint(scale) >> 16) | (__float_as_uint(bias) & 0xFFFF0000u);
}

struct ReadParams {
    tf_kv4 kv;
    tf_kv_batch b;
    void *out[2];
    long long stride[2];
    int tiles;              // tiles of READ_ROWS rows that a sequence may have
    int block_log2, dim_log2;
    int *status;
};
constexpr int READ_ROWS = 4;

// One CTA a (sequence, READ_ROWS of its rows, keys or values); a thread a word of codes, eight values of a row, of all those rows at once.
template <typename T>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(const ReadParams P) {
    const tf_kv4 &kv = P.kv;
    const int H = kv.kv_heads, BL = P.block_log2, DL = P.dim_log2, side = blockIdx.y;
    const int s = P.tiles == 1 ? blockIdx.x : blockIdx.x / P.tiles, tile = blockIdx.x - s * P.tiles;
    T *out = static_cast<T *>(P.out[side]);
    if (!out) return;
    const SeqRows q = seq_rows(P.b, s);
    if (!q.ok || q.end < q.n) {
        if (threadIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        return;
    }
    const int t0 = tile * READ_ROWS, nt = min(READ_ROWS, q.n - t0), first = q.end - q.n + t0;
    if (nt <= 0) return;
    __shared__ long long s_at[READ_ROWS];       // of each row: (page * heads << BL) + its place in the page, -1: no page
    if (threadIdx.x < nt) {
        const int pos = first + threadIdx.x, page = P.b.table[s * P.b.table_stride + (pos >> BL)];
        const bool there = page >= 0 && page < kv.n_blocks;
        if (!there) atomicOr(P.status, STATUS_BOUNDS);
        s_at[threadIdx.x] = there ? (((long long)page * H) << BL) + (pos & (kv.block - 1)) : -1;
    }
    __syncthreads();
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(side ? kv.v : kv.k);
    const uint32_t *affine = reinterpret_cast<const uint32_t *>(side ? kv.v_affine : kv.k_affine);
    const bool vec = ((reinterpret_cast<uintptr_t>(out) | (P.stride[side] * sizeof(T))) & 15) == 0;
    const int per = H << (DL - 3), groups = THREADS / min(per, THREADS);      // rows at a time of short rows
    const int mine = threadIdx.x / min(per, THREADS);
    if (mine >= groups) return;
    for (int c = threadIdx.x - mine * min(per, THREADS); c < per; c += THREADS) {
        const int h = c >> (DL - 3), d = c & ((1 << (DL - 3)) - 1);
        uint32_t w[READ_ROWS], a[READ_ROWS];
#pragma unroll
        for (int k = 0; k < READ_ROWS; ++k) {
            const int t = mine + k * groups;
            if (t >= nt || s_at[t] < 0) continue;
            const long long at = s_at[t] + ((long long)h << BL);
            w[k] = codes[(at << (DL - 3)) + d];
            a[k] = affine[(at << (DL - 6)) + (d >> 3)];
        }
#pragma unroll
        for (int k = 0; k < READ_ROWS; ++k) {
            const int t = mine + k * groups;
            if (t >= nt || s_at[t] < 0) continue;
            T *dst = out + (long long)(q.row0 + t0 + t) * P.stride[side] + 8 * c;
            const float scale = __uint_as_float(a[k] << 16), bias = __uint_as_float(a[k] & 0xFFFF0000u);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmaf((float)((w[k] >> (4 * i)) & 15u), scale, bias);
            if constexpr (sizeof(T) == 4) {
                if (vec) {
                    reinterpret_cast<float4 *>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
                    reinterpret_cast<float4 *>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = y[i];
                }
            } else {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
                if (vec) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(b[0], b[1], b[2], b[3]);
                } else {
                    uint16_t *e = reinterpret_cast<uint16_t *>(dst);
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[i] = (uint16_t)(b[i / 2] >> (16 * (i & 1)));
                }
            }
        }
    }
}

}  // namespace

int tfq::check_kv4(const tf_kv4 *kv) {
    if (!kv) return fail_message(TF_EINVAL_PTR, "NULL cache");
    if (!kv->k || !kv->v || !kv->k_affine || !kv->v_affine) return fail_message(TF_EINVAL_PTR, "NULL cache pointer");
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->k_affine, 16) || !aligned(kv->v_affine, 16))
        return fail_message(TF_EINVAL_PTR, "k, v, k_affine and v_affine must be 16-byte aligned");
    if (kv->block != 16 && kv->block != 32 && kv->block != 64 && kv->block != 128)
        return fail_message(TF_EINVAL_SIZE, "block must be 16, 32, 64 or 128");
    if (kv->dim != 64 && kv->dim != 128 && kv->dim != 256)
        return fail_message(TF_EINVAL_SIZE, "dim must be 64, 128 or 256");
    if (kv->kv_heads < 1 || kv->kv_heads > 1024) return fail_message(TF_EINVAL_SIZE, "kv_heads must be in [1, 1024]");
    if (kv->n_blocks < 1) return fail_message(TF_EINVAL_SIZE, "n_blocks must be at least 1");
    return TF_OK;
}

extern "C" int tf_kv4_append(const tf_kv4 *kv, const int64_t *slots, int rows, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~TF_IN_F32) return fail_message(TF_EINVAL_FLAGS, "tf_kv4_append takes TF_IN_F32 only");
    int rc = check_kv4(kv);
    if (rc) return rc;
    const bool f32 = flags & TF_IN_F32;
    const int es = f32 ? 4 : 2;
    if (!slots || !aligned(slots, 8)) return fail_message(TF_EINVAL_PTR, "NULL slots, or not 8-byte aligned");
    if (!k || !v || !aligned(k, es) || !aligned(v, es))
        return fail_message(TF_EINVAL_PTR, "NULL k or v, or not aligned to their type");
    if (rows < 1) return fail_message(TF_EINVAL_ROWS, "rows must be at least 1");
    const int width = kv->kv_heads * kv->dim;
    if (k_stride < width || v_stride < width)
        return fail_message(TF_EINVAL_STRIDE, "k_stride or v_stride below kv_heads * dim");
    int nsm = 0, *status = nullptr;
    rc = device_info(&nsm, &status);
    if (rc) return rc;
    // A CTA has as many items as give its threads a vector each, or a part of one (blockIdx.y).
    const int per = width / 8, items = per >= THREADS ? 1 : THREADS / per;
    const AppendParams P{*kv, reinterpret_cast<const long long *>(slots), {k, v}, {k_stride, v_stride}, 2LL * rows, items,
                         items == 1 ? 0u : (uint32_t)((0x100000000ull + per - 1) / per), __builtin_ctz(kv->block), __builtin_ctz(kv->dim), status};
    const long long ctas = (2LL * rows + items - 1) / items;
    if (ctas > 0x7FFFFFFF) return fail_message(TF_EINVAL_ROWS, "too many rows in one call");
    const dim3 grid((unsigned)ctas, (unsigned)((per * items + THREADS - 1) / THREADS));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (f32)
        kv4_append_kernel<float><<<grid, THREADS, 0, st>>>(P);
    else
        kv4_append_kernel<__nv_bfloat16><<<grid, THREADS, 0, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv4_append launch");
}

extern "C" int tf_kv4_read(const tf_kv4 *kv, const tf_kv_batch *batch, void *k_out, int64_t k_stride, void *v_out,
                           int64_t v_stride, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~TF_OUT_BF16) return fail_message(TF_EINVAL_FLAGS, "tf_kv4_read takes TF_OUT_BF16 only");
    int rc = check_kv4(kv);
    if (!rc) rc = check_batch(kv->block, batch);
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
    const ReadParams P{*kv, *batch, {k_out, v_out}, {k_stride, v_stride}, (batch->max_rows + READ_ROWS - 1) / READ_ROWS,
                       __builtin_ctz(kv->block), __builtin_ctz(kv->dim), status};
    const long long tiles = (long long)P.tiles * batch->n_seqs;
    if (tiles > 0x7FFFFFFF) return fail_message(TF_EINVAL_SIZE, "too many rows in one call");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)tiles, 2);
    if (flags & TF_OUT_BF16)
        kv4_read_kernel<__nv_bfloat16><<<grid, THREADS, 0, st>>>(P);
    else
        kv4_read_kernel<float><<<grid, THREADS, 0, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv4_read launch");
}
