// sample.cu -- tf_sample (tfdecode.h): one token per row of logits.
//
// A token's weight is the whole number w = round(exp((x - max) / T) * 2^31), so
// sums of weights are exact whatever their order.  top-k, top-p and min-p all
// keep a prefix of the ranking by (logit, then index): the cut of such a prefix
// is found by counting tokens and weights in bins, of z = (x - max) / T first
// and then of the bits of x within the bin that holds the cut, until the bin is
// one token or one value; equal values are cut by index.  The token is then the
// first, in index order, at which the running sum exceeds u times the whole.
//
// One cluster of CTAs a row: each keeps its slice of the row in shared memory (a
// row's logits leave global memory once), counts its own bins, and the CTAs add
// up and search a share of the bins each over distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "kv.h"

namespace cg = cooperative_groups;
using namespace tfq;

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int BINS = 1024;                       // bins of one counting step (at most THREADS)
constexpr int MAX_CLUSTER = 8;
constexpr float WEIGHT_ONE = 2147483648.f;       // weight of the largest logit: 2^31
// exp(z) * 2^31 rounds to 0 below z = -22.2: BINS / 23 bins a unit of z cover the rest.
constexpr float BINS_PER_Z = BINS / 23.f;
constexpr int MAX_SLICE_BYTES = 200 * 1024;      // of a row in one CTA's shared memory

struct Params {
    const void *logits;
    long long stride;
    int rows, vocab, slice;
    const float *u, *temperature, *top_p, *min_p;
    const int *top_k;
    int *tokens;
    float *probs;
};

// Order-preserving bits of a float (no NaN, no -0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// The bin that holds a cut, and what lies above it.
struct Found {
    int bin;                     // -1: the whole distribution lies above
    unsigned count, above;       // tokens in the bin, tokens above it
    u64 mass, mass_above;        // weights in the bin, above it
};

// A prefix of the ranking: bins of z above z_bin whole, in it the keys >= key,
// of the key itself the tokens up to index `last`.
struct Cut {
    int z_bin;
    uint32_t key;
    int last;
};

struct Shared {
    float warp_max[WARPS];
    int warp_at[WARPS];
    u64 warp_sum[WARPS];
    float max;                   // of this CTA's slice
    int at;                      // its index
    unsigned n_part;             // this CTA's share of the bins: tokens, weights
    u64 part;
    Found found[2];              // of alternate searches: a CTA may be one search ahead of another's readers
    int tie_last;
    unsigned n1[BINS], n2[BINS];
    u64 w1[BINS], w2[BINS];
};

template <bool BF16, bool RESIDENT>
struct Row {
    const void *p;               // this CTA's slice in global memory
    const float *s;              // and in shared memory (RESIDENT)
    __device__ __forceinline__ static float clean(float x) { return x != x ? -INFINITY : x + 0.f; }   // NaN, -0
    __device__ __forceinline__ float global(int i) const {
        return clean(BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16)
                          : static_cast<const float *>(p)[i]);
    }
    __device__ __forceinline__ float operator[](int i) const { return RESIDENT ? s[i] : global(i); }
};

template <bool BF16, bool RESIDENT>
__global__ void __launch_bounds__(THREADS) sample_kernel(const Params P) {
    extern __shared__ __align__(16) float values[];
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
    const int row = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = c * P.slice, len = max(0, min(P.slice, P.vocab - first));
    const long long at0 = (long long)row * P.stride + first;
    const Row<BF16, RESIDENT> x{BF16 ? (const void *)(static_cast<const uint16_t *>(P.logits) + at0)
                                     : (const void *)(static_cast<const float *>(P.logits) + at0),
                                values};
    // A warp's part of the slice: indexes [i0, i1), lane by lane.
    const int per = ((P.slice + WARPS - 1) / WARPS + 31) / 32 * 32;
    const int i0 = min(len, warp * per), i1 = min(len, i0 + per);
    auto each = [&](auto f) {
        for (int i = i0 + lane; i < i1; i += 32) f(x[i], i);
    };

    // The slice, and the first of its largest logits.
    float top = -INFINITY;
    int top_at = 0x7FFFFFFF;
    for (int i = i0 + lane; i < i1; i += 32) {
        const float v = x.global(i);
        if (RESIDENT) values[i] = v;
        if (v > top) top = v, top_at = first + i;
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(~0u, top, o);
        const int i = __shfl_xor_sync(~0u, top_at, o);
        if (v > top || (v == top && i < top_at)) top = v, top_at = i;
    }
    if (lane == 0) S.warp_max[warp] = top, S.warp_at[warp] = top_at;
    __syncthreads();
    if (warp == 0) {
        top = S.warp_max[lane];
        top_at = S.warp_at[lane];
        for (int o = 16; o > 0; o >>= 1) {
            const float v = __shfl_xor_sync(~0u, top, o);
            const int i = __shfl_xor_sync(~0u, top_at, o);
            if (v > top || (v == top && i < top_at)) top = v, top_at = i;
        }
        if (lane == 0) S.max = top, S.at = top_at;
    }
    for (int b = tid; b < BINS; b += THREADS) S.n1[b] = 0, S.w1[b] = 0;
    cluster.sync();
    top = -INFINITY;
    for (int k = 0; k < C; ++k) {
        const Shared *o = cluster.map_shared_rank(&S, k);
        if (o->max > top) top = o->max, top_at = o->at;
    }
    float T = P.temperature ? P.temperature[row] : 1.f;
    if (top == -INFINITY || !(T > 0.f)) {
        if (c == 0 && tid == 0) {
            P.tokens[row] = top == -INFINITY ? -1 : top_at;
            if (P.probs) P.probs[row] = top == -INFINITY ? 0.f : 1.f;
        }
        cluster.sync();          // the others may still read this CTA's maximum
        return;
    }
    T = fminf(T, FLT_MAX);
    const float inv = __fdiv_rn(1.f, T);
    auto z_of = [&](float v) { return v == top ? 0.f : __fmul_rn(__fsub_rn(v, top), inv); };
    auto weight = [&](float v) {
        return v == -INFINITY ? 0u : __float2uint_rn(__fmul_rn(expf(z_of(v)), WEIGHT_ONE));
    };
    auto z_bin = [&](float v) { return min(BINS - 1, (int)(z_of(v) * -BINS_PER_Z)); };

    const float p = P.top_p ? P.top_p[row] : 1.f;
    const int k = P.top_k ? P.top_k[row] : 0;
    const float mp = P.min_p ? fminf(P.min_p[row], 1.f) : 0.f;
    const double least = (double)mp * 2147483648.0;

    // Bins of this CTA's share: thread i < BINS / C holds bin c * BINS / C + i.
    const int share = BINS / C;
    int searches = 0;
    // Adds up the cluster's bins; the exclusive prefix over all bins, and the bin's own.
    struct Bin {
        unsigned n, n_before;
        u64 w, w_before;
    };
    auto gather = [&](unsigned (Shared::*n)[BINS], u64 (Shared::*w)[BINS]) {
        cluster.sync();
        Bin b{0, 0, 0, 0};
        if (tid < share)
            for (int r = 0; r < C; ++r) {
                Shared *o = cluster.map_shared_rank(&S, r);
                b.n += (o->*n)[c * share + tid];
                b.w += (o->*w)[c * share + tid];
            }
        unsigned ni = b.n;
        u64 wi = b.w;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned a = __shfl_up_sync(~0u, ni, o);
            const u64 d = __shfl_up_sync(~0u, wi, o);
            if (lane >= o) ni += a, wi += d;
        }
        if (lane == 31) S.warp_at[warp] = (int)ni, S.warp_sum[warp] = wi;
        __syncthreads();
        for (int q = 0; q < warp; ++q) ni += (unsigned)S.warp_at[q], wi += S.warp_sum[q];
        if (tid == share - 1) S.n_part = ni, S.part = wi;
        if (tid == 0) S.found[searches & 1].bin = -1;
        cluster.sync();
        for (int r = 0; r < c; ++r) {
            const Shared *o = cluster.map_shared_rank(&S, r);
            ni += o->n_part, wi += o->part;
        }
        b.n_before = ni - b.n;
        b.w_before = wi - b.w;
        return b;
    };
    // The bin that the target falls into (by tokens: the want-th; by weight: the
    // first whose running sum reaches goal), known to every CTA.
    auto search = [&](const Bin &b, unsigned above, u64 mass_above, bool by_mass, unsigned want, double goal) {
        bool hit = false;
        if (tid < share) {
            if (by_mass)
                hit = (double)(mass_above + b.w_before) < goal && (double)(mass_above + b.w_before + b.w) >= goal;
            else
                hit = above + b.n_before < want && above + b.n_before + b.n >= want;
        }
        if (hit) {
            const Found f{c * share + tid, b.n, above + b.n_before, b.w, mass_above + b.w_before};
            for (int r = 0; r < C; ++r) cluster.map_shared_rank(&S, r)->found[searches & 1] = f;
        }
        cluster.sync();
        return S.found[searches++ & 1];
    };
    // Index of the tie-th (from 1) of the tokens equal to `key`.
    auto tie_index = [&](uint32_t key, unsigned tie) {
        unsigned mine = 0;
        each([&](float v, int) { mine += key_of(v) == key; });
        mine = __reduce_add_sync(~0u, mine);
        if (lane == 0) S.warp_at[warp] = (int)mine;
        __syncthreads();
        unsigned before = 0, all = 0;
        for (int q = 0; q < WARPS; ++q) {
            if (q == warp) before = all;
            all += (unsigned)S.warp_at[q];
        }
        if (tid == 0) S.n_part = all;
        cluster.sync();
        for (int r = 0; r < c; ++r) before += cluster.map_shared_rank(&S, r)->n_part;
        if (before < tie && before + mine >= tie) {
            for (int i = i0; i < i1; i += 32) {
                const bool is = i + lane < i1 && key_of(x[i + lane]) == key;
                const unsigned mask = __ballot_sync(~0u, is);
                if (before + __popc(mask) >= tie) {
                    if (is && before + __popc(mask & ((2u << lane) - 1)) == tie)
                        for (int r = 0; r < C; ++r) cluster.map_shared_rank(&S, r)->tie_last = first + i + lane;
                    break;
                }
                before += __popc(mask);
            }
        }
        cluster.sync();
        return S.tie_last;
    };

    Cut cut{BINS, 0, 0x7FFFFFFF};
    const bool by_k = k > 0 && k < P.vocab, by_p = p < 1.f;
    if (by_k || by_p) {
        each([&](float v, int) {
            const unsigned w = weight(v);
            if (w) {
                const int b = z_bin(v);
                atomicAdd(&S.n1[b], 1u);
                atomicAdd(&S.w1[b], (u64)w);
            }
        });
        const Bin b1 = gather(&Shared::n1, &Shared::w1);
        u64 whole = 0;           // weight of the tokens kept so far
        for (int r = 0; r < C; ++r) whole += cluster.map_shared_rank(&S, r)->part;
        for (int pass = 0; pass < 2; ++pass) {
            const bool by_mass = pass == 1;
            if (!(by_mass ? by_p : by_k)) continue;
            // A goal of at least half a weight keeps the first token.
            const double goal = by_mass ? fmax((double)p * (double)whole, 0.5) : 0.0;
            Found f = search(b1, 0, 0, by_mass, (unsigned)k, goal);
            if (f.bin < 0) continue;
            // Keys that bin can hold, a little more at both ends.
            cut.z_bin = f.bin;
            cut.last = 0x7FFFFFFF;
            const double lo = (f.bin + 1) * (1 + 1e-5) / BINS_PER_Z * (double)T, hi = f.bin * (1 - 1e-5) / BINS_PER_Z * (double)T;
            uint32_t k_lo = f.bin == BINS - 1 ? 0u : key_of(__double2float_rd((double)top - lo) + 0.f);
            uint32_t k_hi = key_of(__double2float_ru((double)top - hi) + 0.f);
            while (f.count > 1 && k_lo < k_hi && !(!by_mass && f.above + f.count == (unsigned)k)) {
                int shift = 0;
                while (((k_hi - k_lo) >> shift) >= (uint32_t)BINS) ++shift;
                __syncthreads();
                for (int b = tid; b < BINS; b += THREADS) S.n2[b] = 0, S.w2[b] = 0;
                __syncthreads();
                each([&](float v, int) {
                    const uint32_t key = key_of(v);
                    if (key >= k_lo && key <= k_hi && v != -INFINITY && z_bin(v) == f.bin) {
                        const unsigned w = weight(v);
                        if (w) {
                            const uint32_t b = (k_hi - key) >> shift;
                            atomicAdd(&S.n2[b], 1u);
                            atomicAdd(&S.w2[b], (u64)w);
                        }
                    }
                });
                const Bin b2 = gather(&Shared::n2, &Shared::w2);
                const int zb = f.bin;
                const Found g = search(b2, f.above, f.mass_above, by_mass, (unsigned)k, goal);
                if (g.bin < 0) break;
                f = g;
                const uint32_t hi2 = k_hi - ((uint32_t)f.bin << shift);
                const u64 room = (u64)(hi2 - k_lo) + 1, span = (u64)1 << shift;
                k_lo = room > span ? hi2 - (uint32_t)(span - 1) : k_lo;
                k_hi = hi2;
                f.bin = zb;
            }
            cut.key = k_lo;
            whole = f.mass_above + f.mass;
            if (k_lo == k_hi && f.count > 1) {
                // Equal tokens: those that the target needs, by index.
                const u64 w = f.mass / f.count;
                unsigned need;
                if (by_mass) {
                    need = 1;
                    const double est = (goal - (double)f.mass_above) / (double)w;
                    if (est > 2.0) need = (unsigned)fmin(est, (double)f.count) - 1;
                    while (need < f.count && (double)(f.mass_above + w * need) < goal) ++need;
                    while (need > 1 && (double)(f.mass_above + w * (need - 1)) >= goal) --need;
                } else {
                    need = (unsigned)k - f.above;
                }
                if (need < f.count) {
                    cut.last = tie_index(k_lo, need);
                    whole = f.mass_above + w * need;
                }
            }
        }
    }
    auto kept = [&](float v, int i) {
        const unsigned w = weight(v);
        if (w == 0 || (double)w < least) return 0u;
        const int b = z_bin(v);
        if (b > cut.z_bin) return 0u;
        if (b < cut.z_bin) return w;
        const uint32_t key = key_of(v);
        return key > cut.key || (key == cut.key && first + i <= cut.last) ? w : 0u;
    };

    // Kept weights by warp, by CTA, of the row; then the token.
    u64 mine = 0;
    each([&](float v, int i) { mine += kept(v, i); });
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
    __syncthreads();
    if (lane == 0) S.warp_sum[warp] = mine;
    __syncthreads();
    u64 before = 0, all = 0;
    for (int q = 0; q < WARPS; ++q) {
        if (q == warp) before = all;
        all += S.warp_sum[q];
    }
    if (tid == 0) S.part = all;
    cluster.sync();
    u64 total = 0;
    for (int r = 0; r < C; ++r) {
        const u64 o = cluster.map_shared_rank(&S, r)->part;
        if (r < c) before += o;
        total += o;
    }
    const double goal = fmax(0.0, fmin((double)P.u[row] * (double)total, (double)total - 0.5));
    if ((double)before <= goal && (double)(before + mine) > goal) {
        for (int i = i0; i < i1; i += 32) {
            const unsigned w = i + lane < i1 ? kept(x[i + lane], i + lane) : 0u;
            u64 run = w;
            for (int o = 1; o < 32; o <<= 1) {
                const u64 a = __shfl_up_sync(~0u, run, o);
                if (lane >= o) run += a;
            }
            run += before;
            const unsigned mask = __ballot_sync(~0u, (double)run > goal);
            if (mask) {
                if (lane == __ffs(mask) - 1) {
                    P.tokens[row] = first + i + lane;
                    if (P.probs) P.probs[row] = (float)((double)w / (double)total);
                }
                break;
            }
            before = __shfl_sync(~0u, run, 31);
        }
    }
    cluster.sync();              // the others may still read this CTA's sum
}

template <bool BF16, bool RESIDENT>
cudaError_t launch(const Params &P, int cluster, int smem, cudaStream_t st) {
    auto k = sample_kernel<BF16, RESIDENT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SLICE_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(P.rows * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)cluster;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k, P);
    return e != cudaSuccess ? e : cudaGetLastError();
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" int tf_sample(const void *logits, int rows, int vocab, int64_t stride, const float *u,
                         const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                         int32_t *tokens, float *probs, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~TF_IN_BF16) return fail_message(TF_EINVAL_FLAGS, "tf_sample takes TF_IN_BF16 only");
    if (rows < 1 || rows > (1 << 20)) return fail_message(TF_EINVAL_ROWS, "rows must be in [1, 2^20]");
    if (vocab < 1 || vocab > (1 << 20)) return fail_message(TF_EINVAL_SIZE, "vocab must be in [1, 2^20]");
    if (stride < vocab) return fail_message(TF_EINVAL_STRIDE, "stride below vocab is refused");
    const int es = flags & TF_IN_BF16 ? 2 : 4;
    if (!logits || !u || !tokens || !aligned(logits, es) || !aligned(u, 4) || !aligned(temperature, 4) ||
        !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(probs, 4))
        return fail_message(TF_EINVAL_PTR, "NULL logits, u or tokens, or a pointer not aligned to its type");
    int nsm = 0, *status = nullptr;
    const int rc = device_info(&nsm, &status);
    if (rc) return rc;
    // CTAs a row: as few as hold it in shared memory, more while SMs are idle and slices long.
    int cluster = 1;
    while (cluster < MAX_CLUSTER && ((long long)vocab * 4 > (long long)cluster * MAX_SLICE_BYTES ||
                                     ((long long)rows * cluster * 2 <= nsm && vocab / cluster > 4096)))
        cluster *= 2;
    const int slice = ((vocab + cluster - 1) / cluster + 7) / 8 * 8;
    const bool resident = (long long)slice * 4 <= MAX_SLICE_BYTES;
    const Params P{logits, stride, rows, vocab, slice, u, temperature, top_p, min_p, top_k, tokens, probs};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int smem = resident ? slice * 4 : 0;
    cudaError_t e;
    if (flags & TF_IN_BF16)
        e = resident ? launch<true, true>(P, cluster, smem, st) : launch<true, false>(P, cluster, smem, st);
    else
        e = resident ? launch<false, true>(P, cluster, smem, st) : launch<false, false>(P, cluster, smem, st);
    return e == cudaSuccess ? TF_OK : cuda_error(e, "sample launch");
}
