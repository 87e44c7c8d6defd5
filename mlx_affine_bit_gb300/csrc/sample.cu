// sample.cu -- tf_sample (tfdecode.h): one token per row of logits.
//
// A token's weight is the whole number w = round(exp((x - max) / T) * 2^31), so
// sums of weights are exact whatever their order.  top-k, top-p and min-p all
// keep a prefix of the ranking by (logit, then index), and the token is the
// first, in index order, at which the running sum exceeds u times the whole.
//
// One cluster of CTAs a row, a slice of the row each, in shared memory where it
// fits (the logits then leave global memory once).  The cut of a prefix is found
// by counting tokens (and adding up weights) in bins: of z = (x - max) / T first,
// each CTA its own slice, all of them added up by every CTA over distributed shared
// memory.  The tokens down to the bin that holds the cut are mostly few: they move,
// in index order, to the first CTA, which cuts them by bins of the bits of x and
// draws, alone.  Where they are many (more than MAX_LIST) the cluster goes on
// together in the same way on its slices.
//
// One row of 248320 fp32 logits takes 17 us, bound by the chain of barriers and of
// reads of the other CTAs' shared memory (four of the cluster, some twenty of the
// first CTA alone); 48 rows 59 us (0.8 TB/s: some 55 instructions for 32 logits in
// three passes over the slice, and barriers, not the read of 48 MB); 300 rows of
// 32003 bf16 logits 34 to 41 us where no row's top-p leaves more than MAX_LIST tokens
// (ten of twelve random inputs), 47 and 62 us where one does: all rows run at once,
// and the slowest is the call's time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "kv.h"

namespace cg = cooperative_groups;
using namespace tfq;

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 512;                        // bins of one counting step (at most THREADS)
constexpr int MAX_CLUSTER = 16;
constexpr float WEIGHT_ONE = 2147483648.f;       // weight of the largest logit: 2^31
// exp(z) * 2^31 rounds to 0 below z = -22.18: BINS / 23 bins a unit of z cover the rest, bin b the nearest to b.
constexpr float BINS_PER_Z = BINS / 23.f, Z_END = -22.25f;
static_assert(BINS == THREADS, "a thread a bin");
// Tokens that one CTA finishes alone.  300 rows of 32003, top-p 0.8, of one input whose rows leave up to some 4000: 34 us;
// 48 with 2048 (the cluster goes on with its whole slices), 60 with 1024.  Inputs with longer lists pay the same way
// with 4096: 62 us with a list of 5738.  The list is 32 KB of the CTA's shared memory.
constexpr int MAX_LIST = 4096;
// Of a row in one CTA's shared memory, for two CTAs an SM beside the list (300 x 32003 bf16: 33 us, 69 with the logits
// read from global memory in each pass; 48 x 248320 fp32: 62 and 73).
constexpr int MAX_SLICE_BYTES = 66 * 1024;

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

__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k); }

// The scaled distribution of a row.
struct Scale {
    float top, inv;              // largest logit, 1 / temperature
    // 0 for the largest (also where it is inf, or 1 / temperature is).
    __device__ __forceinline__ float z(float v) const { return fminf(__fmul_rn(__fsub_rn(v, top), inv), 0.f); }
    __device__ __forceinline__ unsigned weight_of(float z) const { return __float2uint_rn(__fmul_rn(expf(z), WEIGHT_ONE)); }
    __device__ __forceinline__ int bin_of(float z) const {       // for z from Z_END on
        return __float_as_int(fmaf(z, -BINS_PER_Z, 8388608.f)) - 0x4B000000;
    }
    __device__ __forceinline__ unsigned weight(float v) const { return weight_of(z(v)); }
    // BINS for what has no weight.
    __device__ __forceinline__ int bin(float v) const {
        const float x = z(v);
        return x < Z_END ? BINS : bin_of(x);
    }
};

// Tokens and weights of a bin, and of all bins before it.
struct Bin {
    unsigned n, n_before;
    u64 w, w_before;
};
// The bin that holds a cut, and what lies above it.
struct Found {
    int bin;                     // -1: the whole distribution lies above
    unsigned count, above;       // tokens in the bin, tokens above it
    u64 mass, mass_above;        // weights in the bin, above it
};
// A target: the want-th token, or the first at which the running weight reaches goal.
struct Target {
    bool by_mass;
    unsigned want;
    u64 goal;
    __device__ __forceinline__ bool in(unsigned n, unsigned bin_n, u64 w, u64 bin_w) const {
        return by_mass ? w < goal && w + bin_w >= goal : n < want && n + bin_n >= want;
    }
};
// A prefix of the ranking: bins of z above z_bin whole, in it the keys above key,
// of the key itself the tokens up to index `last`.
struct Cut {
    int z_bin;
    uint32_t key;
    int last;
};

struct Shared {
    uint32_t warp_max[WARPS];
    int warp_at[WARPS];
    u64 warp_sum[WARPS];
    uint32_t max;                // key of the largest logit of this CTA's slice
    unsigned n_part;             // this CTA's tokens and weight of a kind that the ranks add up
    u64 part;
    Found found;
    int tie_last;
    // Tokens by bin, and their weights in 16-bit halves (a slice holds at most 2^16 tokens); of alternate
    // countings, so that a CTA may be one ahead of another's reading.
    unsigned n[2][BINS], lo[2][BINS], hi[2][BINS];
    float list_x[MAX_LIST];      // this CTA's tokens of the set that one CTA finishes, in index order; the first CTA's grows to all of them
    int list_i[MAX_LIST];
};

// f * whole in double precision (f in [0, 1), whole < 2^52), rounded to a whole number down, or up.  By whole numbers:
// the SM has few units for doubles, and every thread can have it at once.
__device__ __forceinline__ u64 product(float f, u64 whole, bool up) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const u64 m = e ? (b & 0x7FFFFFu) | 0x800000u : b;       // f = m 2^(max(e, 1) - 150)
    const u64 hi = __umul64hi(m, whole), lo = m * whole;
    const int length = hi ? 128 - __clzll(hi) : 64 - __clzll(lo), over = max(0, length - 53);
    u64 q = lo;
    if (over) {                                              // to 53 bits: the nearest, even in the middle
        q = hi << (64 - over) | lo >> over;
        const u64 rest = lo & ((1ull << over) - 1), half = 1ull << (over - 1);
        q += rest > half || (rest == half && (q & 1));
    }
    const int down = 150 - (int)max(e, 1u) - over;
    if (down <= 0) return q << -down;
    if (down >= 64) return up && q;
    return (q >> down) + (up && (q & ((1ull << down) - 1)));
}

// The CTAs that work together: the row's cluster, or one CTA.
template <bool CLUSTER>
struct Group {
    cg::cluster_group g;
    int size, rank;
    __device__ __forceinline__ void sync() const {
        if (CLUSTER)
            g.sync();
        else
            __syncthreads();
    }
    // The two halves of sync().
    __device__ __forceinline__ void arrive() const { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
    __device__ __forceinline__ void wait() const { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
    __device__ __forceinline__ Shared *of(Shared &S, int r) const { return CLUSTER ? g.map_shared_rank(&S, r) : &S; }
};

// Sums of the ranks' n_part and part: over all of them, and over those before this one.
struct Parts {
    unsigned n, n_before;
    u64 w, w_before;
};
template <bool CLUSTER>
__device__ __forceinline__ Parts parts_of(Shared &S, const Group<CLUSTER> &G) {
    const int lane = threadIdx.x & 31;
    Parts p{0, 0, 0, 0};
    if (lane < G.size) {
        const Shared *o = G.of(S, lane);
        p.n = o->n_part, p.w = o->part;
        if (lane < G.rank) p.n_before = p.n, p.w_before = p.w;
    }
    if (CLUSTER)
        for (int o = MAX_CLUSTER / 2; o > 0; o >>= 1) {
            p.n += __shfl_xor_sync(~0u, p.n, o);
            p.w += __shfl_xor_sync(~0u, p.w, o);
            p.n_before += __shfl_xor_sync(~0u, p.n_before, o);
            p.w_before += __shfl_xor_sync(~0u, p.w_before, o);
        }
    p.n = __shfl_sync(~0u, p.n, 0);
    p.w = __shfl_sync(~0u, p.w, 0);
    p.n_before = __shfl_sync(~0u, p.n_before, 0);
    p.w_before = __shfl_sync(~0u, p.w_before, 0);
    return p;
}
// What lies in the warps before this one, and in all, of one number a warp (left in S.warp_sum by lane 0).
__device__ __forceinline__ u64 warps_of(Shared &S, u64 mine, u64 &all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) S.warp_sum[warp] = mine;
    __syncthreads();
    u64 x = S.warp_sum[lane % WARPS], before = lane % WARPS < warp ? x : 0;
    for (int o = WARPS / 2; o > 0; o >>= 1) {
        x += __shfl_xor_sync(~0u, x, o);
        before += __shfl_xor_sync(~0u, before, o);
    }
    all = x;
    return before;
}

// Counts tokens (and adds up weights, where `weighted`) that each(add) gives as add(bin, weight), over the group; thread t holds
// bin t with what lies before it.  The sums of all bins go to `all`.
template <bool CLUSTER, class Each>
__device__ __forceinline__ Bin count_bins(Shared &S, const Group<CLUSTER> &G, int &counting, bool weighted, Bin &all, Each each) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, now = counting++ & 1;
    S.n[now][tid] = 0;
    if (weighted) S.lo[now][tid] = S.hi[now][tid] = 0;
    __syncthreads();
    each([&](int b, unsigned w) {
        atomicAdd(&S.n[now][b], 1u);
        if (weighted) {
            atomicAdd(&S.lo[now][b], w & 0xFFFFu);
            if (w >> 16) atomicAdd(&S.hi[now][b], w >> 16);
        }
    });
    G.sync();
    Bin b{0, 0, 0, 0};
#pragma unroll 8
    for (int r = 0; r < (CLUSTER ? G.size : 1); ++r) b.n += G.of(S, r)->n[now][tid];
    if (weighted) {
        u64 lo = 0, hi = 0;
#pragma unroll 4
        for (int r = 0; r < (CLUSTER ? G.size : 1); ++r) lo += G.of(S, r)->lo[now][tid], hi += G.of(S, r)->hi[now][tid];
        b.w = lo + (hi << 16);
    }
    unsigned ni = b.n;
    u64 wi = b.w;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned a = __shfl_up_sync(~0u, ni, o);
        if (lane >= o) ni += a;
    }
    if (weighted)
        for (int o = 1; o < 32; o <<= 1) {
            const u64 d = __shfl_up_sync(~0u, wi, o);
            if (lane >= o) wi += d;
        }
    if (lane == 31) S.warp_at[warp] = (int)ni, S.warp_sum[warp] = wi;
    if (tid == 0) S.found.bin = -1;
    __syncthreads();
    unsigned na = lane < WARPS ? (unsigned)S.warp_at[lane] : 0, nb = lane < warp ? na : 0;
    u64 wa = lane < WARPS ? S.warp_sum[lane] : 0, wb = lane < warp ? wa : 0;
    na = __reduce_add_sync(~0u, na);
    nb = __reduce_add_sync(~0u, nb);
    if (weighted)
        for (int o = WARPS / 2; o > 0; o >>= 1) {                // (the other lanes hold none)
            wa += __shfl_xor_sync(~0u, wa, o);
            wb += __shfl_xor_sync(~0u, wb, o);
        }
    wa = __shfl_sync(~0u, wa, 0);
    wb = __shfl_sync(~0u, wb, 0);
    b.n_before = nb + ni - b.n;
    b.w_before = wb + wi - b.w;
    all = Bin{na, 0, wa, 0};
    return b;
}
// The bin that the target falls into, with `above` and `mass_above` before all bins.  (After a counting, or
// where one has been found before and there is one.)
__device__ __forceinline__ Found find_bin(Shared &S, const Bin &b, unsigned above, u64 mass_above, const Target &t) {
    __syncthreads();                             // (every thread has read the last one)
    if (t.in(above + b.n_before, b.n, mass_above + b.w_before, b.w))
        S.found = Found{(int)threadIdx.x, b.n, above + b.n_before, b.w, mass_above + b.w_before};
    __syncthreads();
    return S.found;
}

// Cuts the group's tokens, in bins of z down to `f.bin`, at the target, which lies in that bin; returns the weight kept
// (where `weighted`).
// each(g) calls g(logit, index) for this thread's tokens; in_order(g) does so warp by warp in index order,
// 32 tokens at a time (index -1 past the end).
template <bool CLUSTER, class Each, class InOrder>
__device__ __forceinline__ u64 refine(Shared &S, const Group<CLUSTER> &G, int &counting, const Scale &sc, float T, Found f,
                                      const Target &t, bool weighted, Cut &cut, Each each, InOrder in_order) {
    // Keys that the bin can hold, a little more at both ends.
    cut.z_bin = f.bin;
    cut.last = 0x7FFFFFFF;
    uint32_t k_lo = key_of(__fsub_rd(sc.top, (f.bin + 0.501f) * (1.00001f / BINS_PER_Z) * T) + 0.f);
    uint32_t k_hi = key_of(__fsub_ru(sc.top, fmaxf(f.bin - 0.501f, 0.f) * (0.99999f / BINS_PER_Z) * T) + 0.f);
    while (f.count > 1 && k_lo < k_hi && (t.by_mass || f.above + f.count != t.want)) {
        int shift = 0;
        while (((k_hi - k_lo) >> shift) >= (uint32_t)BINS) ++shift;
        Bin all;
        const Bin b = count_bins(S, G, counting, weighted, all, [&](auto add) {
            each([&](float v, int) {
                const uint32_t key = key_of(v);
                if (key >= k_lo && key <= k_hi && sc.bin(v) == cut.z_bin) add((int)((k_hi - key) >> shift), weighted ? sc.weight(v) : 0u);
            });
        });
        const Found g = find_bin(S, b, f.above, f.mass_above, t);
        if (g.bin < 0) break;
        f = g;
        const uint32_t hi2 = k_hi - ((uint32_t)f.bin << shift);
        const u64 room = (u64)(hi2 - k_lo) + 1, span = (u64)1 << shift;
        k_lo = room > span ? hi2 - (uint32_t)(span - 1) : k_lo;
        k_hi = hi2;
    }
    cut.key = k_lo;
    if (k_lo != k_hi || f.count < 2) return f.mass_above + f.mass;
    // Equal tokens: those that the target needs, by index.
    const u64 w = f.mass / f.count;              // (a bin that a weight is reached in has some)
    const unsigned need = t.by_mass ? (unsigned)((t.goal - f.mass_above + w - 1) / w) : t.want - f.above;
    if (need >= f.count) return f.mass_above + f.mass;
    const int lane = threadIdx.x & 31;
    unsigned mine = 0;
    each([&](float v, int) { mine += key_of(v) == k_lo; });
    mine = __reduce_add_sync(~0u, mine);
    u64 all;
    unsigned before = (unsigned)warps_of(S, mine, all);
    if (threadIdx.x == 0) S.n_part = (unsigned)all;
    G.sync();
    before += parts_of(S, G).n_before;
    if (before < need && before + mine >= need)
        in_order([&](float v, int i) {
            const bool is = i >= 0 && key_of(v) == k_lo;
            const unsigned mask = __ballot_sync(~0u, is);
            if (is && before + __popc(mask & ((2u << lane) - 1)) == need)
                for (int r = 0; r < G.size; ++r) G.of(S, r)->tie_last = i;
            before += __popc(mask);
            return before >= need;
        });
    G.sync();
    cut.last = S.tie_last;
    return f.mass_above + w * need;
}

// Draws among the group's tokens above the cut and of weight `least` at least.
template <bool CLUSTER, class Each, class InOrder>
__device__ __forceinline__ void draw(Shared &S, const Group<CLUSTER> &G, const Scale &sc, const Cut &cut, unsigned least, float u,
                                     int *token, float *prob, Each each, InOrder in_order) {
    const int lane = threadIdx.x & 31;
    auto kept = [&](float v, int i) {
        const float z = sc.z(v);
        if (z < Z_END) return 0u;
        const int b = sc.bin_of(z);
        if (b > cut.z_bin) return 0u;
        if (b == cut.z_bin) {
            const uint32_t key = key_of(v);
            if (key < cut.key || (key == cut.key && i > cut.last)) return 0u;
        }
        const unsigned w = sc.weight_of(z);
        return w < least ? 0u : w;
    };
    u64 mine = 0;
    each([&](float v, int i) { mine += kept(v, i); });
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
    u64 all, before = warps_of(S, mine, all);
    if (threadIdx.x == 0) S.part = all;
    G.sync();
    const Parts parts = parts_of(S, G);
    const u64 total = parts.w;
    before += parts.w_before;
    // The running sum exceeds u * total where it exceeds its whole part (u from 1 on: the last token).
    const u64 goal = u < 1.f ? min(product(fmaxf(u, 0.f), total, false), total - 1) : total - 1;
    if (before <= goal && before + mine > goal)
        in_order([&](float v, int i) {
            const unsigned w = i >= 0 ? kept(v, i) : 0u;
            u64 run = w;
            for (int o = 1; o < 32; o <<= 1) {
                const u64 a = __shfl_up_sync(~0u, run, o);
                if (lane >= o) run += a;
            }
            run += before;
            const unsigned mask = __ballot_sync(~0u, run > goal);
            if (mask && lane == __ffs(mask) - 1) {
                *token = i;
                if (prob) *prob = (float)((double)w / (double)total);
            }
            before = __shfl_sync(~0u, run, 31);
            return mask != 0;
        });
}

template <bool BF16, bool RESIDENT>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const Params P) {
    extern __shared__ __align__(16) uint8_t slice[];
    __shared__ Shared S;
    const Group<true> G{cg::this_cluster(), (int)cg::this_cluster().num_blocks(), (int)cg::this_cluster().block_rank()};
    const int row = blockIdx.x / G.size;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = G.rank * P.slice, len = max(0, min(P.slice, P.vocab - first));
    const long long at0 = (long long)row * P.stride + first;
    const uint16_t *g16 = static_cast<const uint16_t *>(P.logits) + (BF16 ? at0 : 0);
    const float *g32 = static_cast<const float *>(P.logits) + (BF16 ? 0 : at0);
    auto value = [](float x) { return x != x ? -INFINITY : x + 0.f; };                  // NaN is -inf, -0 is 0
    auto of16 = [&](uint32_t h) { return value(__uint_as_float(h << 16)); };
    // (A resident slice holds the values so.)
    auto at = [&](int i) {
        if (RESIDENT) return BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(slice)[i] << 16) : reinterpret_cast<const float *>(slice)[i];
        return BF16 ? of16(g16[i]) : value(g32[i]);
    };
    // A warp's part of the slice: indexes [i0, i1), four by four and lane by lane.
    const int per = ((P.slice + WARPS - 1) / WARPS + 127) / 128 * 128;
    static_assert((1 << 20) / MAX_CLUSTER / WARPS <= 32 * 128 && MAX_SLICE_BYTES / 2 / WARPS <= 32 * 128, "32 times 128 tokens a warp at most");
    const int i0 = min(len, warp * per), i1 = min(len, i0 + per);
    // f of this thread's tokens, done(c) after those of the c-th 128.
    auto each_done = [&](auto f, auto done) {
        int i = i0 + 4 * lane;
        if (RESIDENT) {
#pragma unroll 2
            for (; i + 3 < i1; i += 128) {
                if (BF16) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(slice) + i);
                    f(__uint_as_float(x.x << 16), first + i), f(__uint_as_float(x.x & 0xFFFF0000u), first + i + 1);
                    f(__uint_as_float(x.y << 16), first + i + 2), f(__uint_as_float(x.y & 0xFFFF0000u), first + i + 3);
                } else {
                    const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(slice) + i);
                    f(x.x, first + i), f(x.y, first + i + 1), f(x.z, first + i + 2), f(x.w, first + i + 3);
                }
                done((i - i0) >> 7);
            }
        } else {
            for (; i + 3 < i1; i += 128) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = at(i + e);
#pragma unroll
                for (int e = 0; e < 4; ++e) f(x[e], first + i + e);
                done((i - i0) >> 7);
            }
        }
        for (int e = 0; e < 4 && i + e < i1; ++e) f(at(i + e), first + i + e);
        if (i < i1) done((i - i0) >> 7);
    };
    auto each = [&](auto f) { each_done(f, [](int) {}); };
    auto in_order = [&](auto f) {
        for (int i = i0; i < i1; i += 32) {
            const bool is = i + lane < i1;
            if (f(is ? at(i + lane) : -INFINITY, is ? first + i + lane : -1)) break;
        }
    };

    // The row's parameters (on their way while the logits are).
    const float temperature = P.temperature ? P.temperature[row] : 1.f, T = fminf(temperature, FLT_MAX);
    const float p = P.top_p ? P.top_p[row] : 1.f, u = P.u[row], min_p = P.min_p ? P.min_p[row] : 0.f;
    const int top_k = P.top_k ? P.top_k[row] : 0;

    // The slice, and its largest logit.
    float top = -INFINITY;
    if (RESIDENT) {
        // 16 bytes at a time from the first aligned token on.
        constexpr int VEC = BF16 ? 8 : 4;
        const int es = BF16 ? 2 : 4;
        const uintptr_t base = BF16 ? reinterpret_cast<uintptr_t>(g16) : reinterpret_cast<uintptr_t>(g32);
        const int head = min(len, (int)(((16 - base % 16) % 16) / es)), vecs = (len - head) / VEC;
        auto keep16 = [](float x) { return __float_as_uint(x) >> 16; };
        auto one = [&](int i) {
            const float x = BF16 ? of16(g16[i]) : value(g32[i]);
            if (BF16)
                reinterpret_cast<uint16_t *>(slice)[i] = (uint16_t)keep16(x);
            else
                reinterpret_cast<float *>(slice)[i] = x;
            top = fmaxf(top, x);
        };
        if (tid < head) one(tid);
        for (int i = head + vecs * VEC + tid; i < len; i += THREADS) one(i);
        // (A row whose first token is not aligned goes to shared memory word by word.)
#pragma unroll 4
        for (int v = tid; v < vecs; v += THREADS) {
            const int i = head + v * VEC;
            if (BF16) {
                const uint4 x = *reinterpret_cast<const uint4 *>(g16 + i);
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = of16(w[e] & 0xFFFFu), b = of16(w[e] >> 16);
                    top = fmaxf(top, fmaxf(a, b));
                    w[e] = keep16(a) | (__float_as_uint(b) & 0xFFFF0000u);
                    if (head) {
                        reinterpret_cast<uint16_t *>(slice)[i + 2 * e] = (uint16_t)w[e];
                        reinterpret_cast<uint16_t *>(slice)[i + 2 * e + 1] = (uint16_t)(w[e] >> 16);
                    }
                }
                if (head == 0) *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(slice) + i) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                float4 x = *reinterpret_cast<const float4 *>(g32 + i);
                x = make_float4(value(x.x), value(x.y), value(x.z), value(x.w));
                float *dst = reinterpret_cast<float *>(slice) + i;
                if (head == 0)
                    *reinterpret_cast<float4 *>(dst) = x;
                else
                    dst[0] = x.x, dst[1] = x.y, dst[2] = x.z, dst[3] = x.w;
                top = fmaxf(top, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
            }
        }
    } else {
        each([&](float v, int) { top = fmaxf(top, v); });
    }
    uint32_t top_key = __reduce_max_sync(~0u, key_of(top));
    if (lane == 0) S.warp_max[warp] = top_key;
    __syncthreads();
    if (warp == 0) {
        top_key = __reduce_max_sync(~0u, lane < WARPS ? S.warp_max[lane] : 0u);
        if (lane == 0) S.max = top_key;
    }
    G.sync();
    top = of_key(__reduce_max_sync(~0u, lane < G.size ? G.of(S, lane)->max : 0u));
    if (top == -INFINITY) {
        if (G.rank == 0 && tid == 0) {
            P.tokens[row] = -1;
            if (P.probs) P.probs[row] = 0.f;
        }
        G.sync();                // (the others may still read this CTA's maximum)
        return;
    }
    const bool greedy = !(temperature > 0.f);    // (NaN too, which T is not)
    const Scale sc{top, greedy ? 1.f : __fdiv_rn(1.f, T)};
    // The least whole weight of at least min_p times the largest (a power of two times min_p is exact).
    const unsigned least = min_p > 0.f && !greedy ? max(1u, __float2uint_ru(fminf(min_p, 1.f) * WEIGHT_ONE)) : 1u;
    const int k = greedy ? 1 : top_k;            // (the first of the largest: the one token that top-k 1 keeps)
    const bool by_k = k > 0 && k < P.vocab, by_p = p < 1.f && !greedy;
    const float Tk = greedy ? 1.f : T;
    float *prob = P.probs ? P.probs + row : nullptr;
    // The goal of top-p over a weight: the least whole number that reaches it, at least 1 (the first token).
    auto goal_of = [&](u64 whole) { return max(1ull, product(fmaxf(p, 0.f), whole, true)); };

    Cut cut{BINS - 1, 0, 0x7FFFFFFF};
    int counting = 0;
    if (by_k || by_p) {
        const bool mass = by_p && !by_k;         // (top-p after top-k is cut among the tokens that top-k leaves)
        Bin all_bins;
        const Bin b = count_bins(S, G, counting, mass, all_bins, [&](auto add) {
            each([&](float v, int) {
                const float z = sc.z(v);
                if (z >= Z_END) add(sc.bin_of(z), mass ? sc.weight_of(z) : 0u);
            });
        });
        u64 whole = all_bins.w;
        Found f = find_bin(S, b, 0, 0, Target{mass, (unsigned)k, mass ? goal_of(whole) : 0});
        // Tokens in bins down to the cut's: the set that it cuts.
        const int z_bin = f.bin < 0 ? BINS - 1 : f.bin;
        const unsigned set = f.bin < 0 ? all_bins.n : f.above + f.count;
        if (set <= MAX_LIST) {
            // Each CTA lists its own, in index order, and the first takes them all.
            const float last_bin = 8388608.f + z_bin;
            auto in_set = [&](float v) {
                const float z = sc.z(v);
                return z >= Z_END && fmaf(z, -BINS_PER_Z, 8388608.f) <= last_bin;      // bin_of(z) <= z_bin
            };
            unsigned mine = 0, chunks = 0;       // chunks: which 128 of the warp's tokens (32 at most) hold some
            unsigned mine_before = 0;
            each_done([&](float v, int) { mine += in_set(v); },
                      [&](int c) { chunks |= (unsigned)(mine != mine_before) << c, mine_before = mine; });
            mine = __reduce_add_sync(~0u, mine);
            chunks = __reduce_or_sync(~0u, chunks);
            u64 all;
            unsigned before = (unsigned)warps_of(S, mine, all);
            if (tid == 0) S.n_part = (unsigned)all;
            for (; chunks; chunks &= chunks - 1)
                for (int i = i0 + (__ffs(chunks) - 1) * 128, end = min(i1, i + 128); i < end; i += 32) {
                    const float v = i + lane < end ? at(i + lane) : -INFINITY;
                    const bool is = in_set(v);
                    const unsigned mask = __ballot_sync(~0u, is), slot = before + __popc(mask & ((1u << lane) - 1));
                    if (is && slot < MAX_LIST) S.list_x[slot] = v, S.list_i[slot] = first + i + lane;
                    before += __popc(mask);
                }
            G.sync();
            if (G.rank != 0) {
                G.sync();        // (the first CTA has read the list)
                return;
            }
            // A warp takes a rank's list.
            const unsigned count = lane < G.size ? G.of(S, lane)->n_part : 0;
            const unsigned n_all = __reduce_add_sync(~0u, count), skip = __reduce_add_sync(~0u, lane < warp ? count : 0);
            if (warp > 0 && warp < G.size) {
                const Shared *o = G.of(S, warp);
                const unsigned m = __shfl_sync(~0u, count, warp);
                for (unsigned i = lane; i < m && skip + i < MAX_LIST; i += 32) S.list_x[skip + i] = o->list_x[i], S.list_i[skip + i] = o->list_i[i];
            }
            G.arrive();
            __syncthreads();
            // From here on the first CTA alone.
            const unsigned n = min(n_all, (unsigned)MAX_LIST);
            const Group<false> one{G.g, 1, 0};
            const int per_warp = ((int)n + THREADS - 1) / THREADS * 32, l0 = min((int)n, warp * per_warp), l1 = min((int)n, l0 + per_warp);
            auto each_listed = [&](auto fn) {
                for (int i = l0 + lane; i < l1; i += 32) fn(S.list_x[i], S.list_i[i]);
            };
            auto listed_in_order = [&](auto fn) {
                for (int i = l0; i < l1; i += 32) {
                    const bool is = i + lane < l1;
                    if (fn(is ? S.list_x[i + lane] : -INFINITY, is ? S.list_i[i + lane] : -1)) break;
                }
            };
            auto whole_listed = [&]() {          // weight of the list's tokens
                u64 w = 0;
                each_listed([&](float v, int) { w += sc.weight(v); });
                for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
                u64 all;
                warps_of(S, w, all);
                return all;
            };
            if (!mass) whole = f.bin >= 0 ? refine(S, one, counting, sc, Tk, f, Target{false, (unsigned)k, 0}, false, cut, each_listed, listed_in_order)
                                          : whole_listed();
            if (!mass && f.bin >= 0 && by_p) {
                // (counted without weights: the weight that top-k keeps)
                u64 w = 0;
                each_listed([&](float v, int i) {
                    const int zb = sc.bin(v);
                    const uint32_t key = key_of(v);
                    if (zb < cut.z_bin || (zb == cut.z_bin && (key > cut.key || (key == cut.key && i <= cut.last)))) w += sc.weight(v);
                });
                for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
                warps_of(S, w, whole);
            }
            if (by_p) {
                const Target t{true, 0, goal_of(whole)};
                if (!mass) {
                    Bin all_listed;
                    const Bin lb = count_bins(S, one, counting, true, all_listed, [&](auto add) {
                        each_listed([&](float v, int) { add(sc.bin(v), sc.weight(v)); });
                    });
                    f = find_bin(S, lb, 0, 0, t);
                }
                if (f.bin >= 0) refine(S, one, counting, sc, Tk, f, t, true, cut, each_listed, listed_in_order);
            }
            draw(S, one, sc, cut, least, u, P.tokens + row, prob, each_listed, listed_in_order);
            G.wait();
            return;
        }
        // Too many tokens for one CTA: the cluster goes on, with weights.
        const Bin wb = mass ? b : count_bins(S, G, counting, true, all_bins, [&](auto add) {
            each([&](float v, int) {
                const float z = sc.z(v);
                if (z >= Z_END) add(sc.bin_of(z), sc.weight_of(z));
            });
        });
        if (!mass) {
            whole = all_bins.w;
            f = find_bin(S, wb, 0, 0, Target{false, (unsigned)k, 0});
            if (f.bin >= 0) whole = refine(S, G, counting, sc, Tk, f, Target{false, (unsigned)k, 0}, true, cut, each, in_order);
            if (by_p) {
                const Target t{true, 0, goal_of(whole)};
                f = find_bin(S, wb, 0, 0, t);
                if (f.bin >= 0) refine(S, G, counting, sc, Tk, f, t, true, cut, each, in_order);
            }
        } else if (f.bin >= 0) {
            refine(S, G, counting, sc, Tk, f, Target{true, 0, goal_of(whole)}, true, cut, each, in_order);
        }
    }
    draw(S, G, sc, cut, least, u, P.tokens + row, prob, each, in_order);
    G.sync();                    // (the others may still read this CTA's sum)
}

template <bool BF16, bool RESIDENT>
cudaError_t launch(const Params &P, int cluster, int smem, cudaStream_t st) {
    auto k = sample_kernel<BF16, RESIDENT>;
    static unsigned attr_set = 0;   // one bit per device: limits raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned bit = 1u << (dev & 31);
    if (!(__atomic_load_n(&attr_set, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SLICE_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_set, bit, __ATOMIC_RELEASE);
    }
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
    // CTAs a row: as few as hold it in shared memory, more while SMs are idle and slices long: over 4096 logits (1 and 8
    // rows of 32003 bf16: 14 and 17 us; over 8192: 15 and 18, over 2048: 15 and 23; one row of 248320 fp32 with 16 CTAs
    // 18 us, with 8 30).
    int cluster = 1;
    while (cluster < MAX_CLUSTER && ((long long)vocab * es > (long long)cluster * MAX_SLICE_BYTES ||
                                     ((long long)rows * cluster <= nsm && vocab / cluster > 4096)))
        cluster *= 2;
    const int slice = ((vocab + cluster - 1) / cluster + 7) / 8 * 8;
    const bool resident = (long long)slice * es <= MAX_SLICE_BYTES;
    const Params P{logits, stride, rows, vocab, slice, u, temperature, top_p, min_p, top_k, tokens, probs};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int smem = resident ? slice * es : 0;
    cudaError_t e;
    if (flags & TF_IN_BF16)
        e = resident ? launch<true, true>(P, cluster, smem, st) : launch<true, false>(P, cluster, smem, st);
    else
        e = resident ? launch<false, true>(P, cluster, smem, st) : launch<false, false>(P, cluster, smem, st);
    return e == cudaSuccess ? TF_OK : cuda_error(e, "sample launch");
}
