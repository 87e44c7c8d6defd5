// attend_prompt.cuh -- attention of many rows (prompts, chunks of prompts) over the
// 8-bit or 4-bit paged cache, on the fifth-generation tensor cores.  (Over 4 bits keys and
// values are widened to scale c + bias, over the largest of 16 tokens: `widened`, `over_unit`.)
//
// For the rows r of one (sequence, key/value head) -- G query heads a token -- and
// the tokens j they see, with q_r in fp16 times a power of two:
//     s_rj = (q_r . c_j) * (scale log2(e) ks_page / f_r)
//     p_rj = 2^(s_rj - m_r),  l_r = sum_j p_rj,  out_r = sum_j p_rj vs_page c'_j / l_r
// The first product runs over the keys' bytes as fp16 subnormals (c + 128) 2^-24
// (its offset, 128 2^-24 sum(q_r), goes into the exponent's constant), the second
// over the codes, exact in fp16, and w_rj = 2^15 p_rj vs_page 2^(m_r - n_r) in fp16,
// n_r the running maximum of s_rj + log2(vs_page): 11 bits down to 2^-29 of the
// row's largest contribution, nothing below 2^-40.  The exponent of w is one fused
// product and sum on what the tensor cores leave; where its terms could be so large
// (FAR) that their rounding showed, a pass of its own turns them into scores less a
// common base first.
//
// Bound by the tensor cores and, closely, by the instructions around them: per row
// and token one exponential and about four others, per token and dimension of the
// cache about two to widen a code.  Over 8 bits, causal, 32 query heads of 128 over 8:
// 4000 tokens of a prompt 196 to 200 us (669 to 656 TFLOP/s), 8000 643 us (815 TFLOP/s);
// 16 heads of 256: 4000 tokens 193 us; 16 heads of 64: 87 us; three chunks of up to 509
// tokens, 16 heads of 256, window 4096: 86 us (scores past FAR: 4000 tokens of 32 heads
// 318 us, the chunks 129).  Over 4 bits: 203, 657, 214 and 89 us, the chunks with fp32 q
// 120.  A step of two tiles (256 rows, 128 tokens, dim 128) takes
// 2.7 us, 1.7 us of them the products: one with N = 128 takes 94 to 107 clocks for
// 16 of K, measured alone, which is 60 to 68 % of the peak.  An item's beginning and
// end (the rows of q, the first scores, the outputs) cost 6 us, the launch's plan 4.
//
// A CTA (one an SM) works on two tiles of 128 rows (dim 256: one, tensor memory holds
// no more) by steps of 128 tokens, so that one widening serves 256 rows and one
// tile's softmax runs beside the other's products:
//     8 warps    (dim 256: 4) softmax, a row a thread: S out of tensor memory, the
//                running maxima, w back into tensor memory as the second product's
//                A operand; the rows of q; the outputs
//     4 warps    (dim 256: 8) keys and values from global memory through registers
//                into shared memory as fp16 (K-major and MN-major, 128-byte swizzle)
//     1 thread   a tile: its products
// The work -- for every tile pair and head the steps of the tokens it sees -- is one
// line that the CTAs cut into equal shares; an item (one pair and head) that several
// CTAs share is joined by the last of them to arrive, in their order.  Every wait is
// bounded.
#pragma once
#include "attend_rows.cuh"
#include "prompt_kernel.cuh"

namespace tfq {
namespace attend {

constexpr int P_THREADS = 512;
// Registers a thread after the split, by warpgroup: with the 512 threads' 128 at launch as their sum's limit.
template <int D>
struct PRegs {
    static constexpr int SOFT = D == 256 ? 232 : 168, CONV = 104, REST = 72;
    static_assert((D == 256 ? SOFT + 2 * CONV : 2 * SOFT + CONV) + REST <= 4 * 128, "registers of the launch");
};
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int KEYS = 128;                        // tokens of a step
TFQ_HD constexpr int p_tiles(int d) { return d == 256 ? 1 : 2; }
// Softmax warps (a row a thread) and widening warps; then four whose first lane issues a tile's products.
TFQ_HD constexpr int p_soft(int d) { return 4 * p_tiles(d); }
TFQ_HD constexpr int p_conv(int d) { return 12 - p_soft(d); }
TFQ_HD constexpr int p_slots(int d) { return d == 256 ? 2 : 4; }          // fp16 tiles of keys or values in flight
TFQ_HD constexpr int p_tile_bytes(int d) { return KEYS * d * 2; }         // one of them, and 128 rows of q
TFQ_HD constexpr int p_smem(int d) { return 1024 + (p_tiles(d) + p_slots(d)) * p_tile_bytes(d); }
constexpr uint32_t PAGES_THERE = 0x8000;         // (the sign of a key scale)
constexpr int SCALES = 4;                        // steps whose scales are kept
constexpr float SLACK = 0.9f;                    // growth of a maximum that is let be, in powers of two (w stays in fp16's range)
// Bound (in powers of two) of the terms of an exponent that are summed as they stand: below it their sums, of up to
// 2^13, round by 2^-11 at most.  The check of a step comes before the wait for its scores (after it: 4 us of 204 for 4000
// tokens of 32 heads of 128).
constexpr float FAR = 4096.f;
constexpr int ITEM_STEPS = 3;                    // an item's beginning and end on the line, in steps (2 to 6: 3 is fastest)
constexpr int MAX_SHARE = 8;                     // CTAs an item, on average: one of them joins their parts

// One tile pair's tokens: [from, to) in steps.
struct TileWork {
    int from, to, steps;
};
struct PSeq {
    SeqRows q;
    int tiles;               // tile pairs of the sequence's rows
    int plan;                // tokens that its place on the line is for
};
template <int R>
__device__ __forceinline__ PSeq p_seq(const Params &P, int s) {
    PSeq w;
    w.q = seq_rows(P.b, s);
    w.plan = max(0, min(w.q.end, P.b.max_len));
    if (!w.q.ok) {
        // Rows that lie within the matrices get zeros (no token is seen; the line, and with it the other
        // sequences' bits, stay as they are).
        w.q.end = 0;
        if (!w.q.placed) w.q.n = 0;
    }
    w.tiles = (w.q.n * P.group + R - 1) / R;
    return w;
}
template <int R>
__device__ __forceinline__ TileWork p_tile(const Params &P, const PSeq &w, int tile) {
    const int first = w.plan - w.q.n, r0 = tile * R, r1 = min(r0 + R, w.q.n * P.group) - 1;
    TileWork t{0, w.plan, 0};
    if (P.causal) {
        t.to = max(0, min(w.plan, first + r1 / P.group + 1));
        if (P.window) t.from = max(0, first + r0 / P.group - P.window + 1) & ~31;
    }
    t.steps = max(1, (t.to - t.from + KEYS - 1) / KEYS);
    if (!w.q.ok) t.to = 0;
    return t;
}

// A CTA's place on the line: sequence, tile pair and head, and its steps of that
// item.  An item takes ITEM_STEPS (its beginning and end) and its steps of the line;
// a CTA whose share ends in the former has none of the latter.
template <int R>
struct Walk {
    int seq, tile, h, step0, step1;
    PSeq s;
    TileWork t;
    long long item_at, begin, end;           // the item's first step; the CTA's share
    __device__ __forceinline__ void span() {
        step0 = (int)max(0LL, begin - item_at);
        step1 = (int)min((long long)t.steps, end - item_at);
    }
    // The first item with steps of this CTA (from the one that holds its share's beginning), false if there is none.
    __device__ __forceinline__ bool first(const Params &P, int seq_, int tile_, int h_, long long at, long long begin_, long long end_) {
        seq = seq_, tile = tile_, h = h_, begin = begin_, end = end_;
        s = p_seq<R>(P, seq);
        t = p_tile<R>(P, s, tile);
        item_at = at + ITEM_STEPS;
        span();
        return step0 < step1;                // (a share that begins in an item's first part and ends there: no other has a part of it)
    }
    __device__ __forceinline__ bool next(const Params &P) {
        const long long at = item_at + t.steps;
        if (at + ITEM_STEPS >= end) return false;
        if (++h == P.kv.kv_heads) {
            h = 0;
            if (++tile == s.tiles) {
                tile = 0;
                do s = p_seq<R>(P, ++seq);
                while (s.tiles == 0);
            }
            t = p_tile<R>(P, s, tile);
        }
        item_at = at + ITEM_STEPS;
        span();
        return true;
    }
};

struct PromptHdr {
    uint64_t kv_full[4], kv_empty[4], s_full[2], s_free, p_full[2], pv_done[2], q_full[2], o_free[2], scales[4], joined[2], turn[2], done;
    uint32_t tmem;
    int abort, last, seq, tile, h;
    long long item_at, total, arrived, sums[P_THREADS / 32];     // (arrived: the last shared item of which a part was counted)
    float2 scale[SCALES][8];                 // key scale, log2 of the value scale, of each 16 tokens (-1: no page)
    // A number a widening warp: the largest key scale of its tokens' pages (the upper half of its bits, rounded up, at least
    // 1; 0 if there is no page), and PAGES_THERE if all of them are there.
    __align__(16) uint16_t top_ks[SCALES][8];
};
static_assert(sizeof(PromptHdr) <= 1024, "header");

// Descriptors with the 128-byte swizzle: rows of 128 bytes in groups of eight, 1024 bytes apart; blocks of 64 values
// (of the dimension) 128 rows apart.  K-major: the rows are the product's rows; MN-major: they are its K.
// (Shared addresses end below 2^18: an offset moves the low word only.)
__device__ __forceinline__ uint32_t sw128_lo(uint32_t addr) { return ((addr >> 4) & 0x3FFF) | ((uint32_t)(KEYS * 128 >> 4) << 16); }
constexpr uint32_t SW128_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ constexpr uint32_t f16_idesc(int n, bool b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t id) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(id), "n"(SW128_HI), "n"((int)ACC)
        : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t id) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(id), "n"(SW128_HI), "n"((int)ACC)
        : "memory");
}
// mbar_wait in few instructions (the kernel has many waits).
__device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity, volatile int *abort, int *status) {
    if (mbar_try(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    while (!mbar_try(bar, parity) && !*abort)
        if (global_ns() - t0 > WAIT_LIMIT_NS) {
            *abort = 1;
            atomicOr(status, STATUS_WAIT);
        }
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Completes the loads issued so far; names the registers, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Pairs of fp32 values at once, each rounded as by itself.
__device__ __forceinline__ void mul2(uint32_t &a, uint32_t &b, float f) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+r"(a), "+r"(b)
        : "r"(__float_as_uint(f)));
}
__device__ __forceinline__ void fma2(uint32_t &a, uint32_t &b, float f, float k) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+r"(a), "+r"(b)
        : "r"(__float_as_uint(f)), "r"(__float_as_uint(k)));
}
__device__ __forceinline__ void add2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Place in a 16-byte chunk of the fp16 tiles of eight dimensions' e-th: with 4-bit codes, the order in which a word's come
// out in pairs (d, d + 4), the same for q and keys, and undone where outputs are stored.
TFQ_HD constexpr int chunk_place(int f, int e) { return f == 4 ? (e & 3) * 2 + (e >> 2) : e; }
// Eight codes of a word as fp16 times a scale plus a bias, in that order: codes stand as the subnormals c 2^-20, scales come
// 2^20 larger than biases; one rounding.  (With the codes made whole numbers by a difference first: 13 instructions, now 11.)
__device__ __forceinline__ uint4 widened(uint32_t w, __half2 scale, __half2 bias) {
    auto value = [&](uint32_t bits) {
        const uint32_t code = bits & 0x00F000F0u;
        const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&code), scale, bias);
        return *reinterpret_cast<const uint32_t *>(&y);
    };
    return make_uint4(value(w << 4), value(w), value(w >> 4), value(w >> 8));
}

// F: bits of a code (8 or 4).
template <int F, int D>
__global__ void __launch_bounds__(P_THREADS, 1) prompt_kernel(const __grid_constant__ Params P) {
    constexpr int NT = p_tiles(D), R = 128 * NT, SLOTS = p_slots(D), TB = p_tile_bytes(D);
    constexpr int P_SOFT = p_soft(D), P_CONV = p_conv(D);
    extern __shared__ __align__(1024) uint8_t smem[];
    PromptHdr &B = *reinterpret_cast<PromptHdr *>(smem);
    uint8_t *const q_s = smem + 1024, *const kv_s = q_s + NT * TB;
    volatile int *abort = &B.abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = P.kv.kv_heads, G = P.group, BL = P.block_log2, BM = P.kv.block - 1;

    // Tensor memory: per tile S (128 columns; w over it, dim 256 beside it twice) and the outputs (D columns).
    constexpr uint32_t S_COL = 0, O_COL = NT * 128, W_COL = O_COL + D;   // (W_COL: dim 256 only, 2 x 64)
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&B.kv_full[i], P_CONV);
            mbar_init(&B.kv_empty[i], NT);
        }
        for (int i = 0; i < NT; ++i) {
            mbar_init(&B.s_full[i], 1);
            mbar_init(&B.p_full[i], 4);
            mbar_init(&B.pv_done[i], 1);
            mbar_init(&B.q_full[i], 4);
            mbar_init(&B.o_free[i], 4);
        }
        for (int i = 0; i < SCALES; ++i) mbar_init(&B.scales[i], P_CONV);
        for (int i = 0; i < 2; ++i) mbar_init(&B.joined[i], 4 * NT);
        mbar_init(&B.turn[0], 1);
        mbar_init(&B.turn[1], 1);
        mbar_init(&B.s_free, 4);
        mbar_init(&B.done, NT);
        B.abort = 0;
        B.arrived = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // The line's length and this CTA's share: first the tile pairs of all sequences, thread by thread over the
    // sequences, then their steps, thread by thread over the tile pairs.
    long long *const flat = reinterpret_cast<long long *>(q_s), *const steps_at = flat + P_THREADS;   // (q's place, before q)
    auto scan = [&](long long mine, long long *out) {        // exclusive, into out[tid]; returns the sum
        long long x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) B.sums[warp] = x;
        __syncthreads();
        const long long own = lane < P_THREADS / 32 ? B.sums[lane] : 0;
        long long y = own;
        for (int o = 1; o < P_THREADS / 32; o <<= 1) {
            const long long z = __shfl_up_sync(~0u, y, o);
            if (lane >= o) y += z;
        }
        const long long all = __shfl_sync(~0u, y, P_THREADS / 32 - 1);
        x += __shfl_sync(~0u, y - own, warp);
        out[tid] = x - mine;
        __syncthreads();
        return all;
    };
    const int per = (P.b.n_seqs + P_THREADS - 1) / P_THREADS;
    long long pairs = 0;
    for (int s = tid * per; s < min(P.b.n_seqs, (tid + 1) * per); ++s) {
        const PSeq w = p_seq<R>(P, s);
        if (!w.q.ok && blockIdx.x == 0) atomicOr(P.status, STATUS_BOUNDS);
        pairs += w.tiles;
    }
    const long long n_pairs = scan(pairs, flat);
    // Tile pair f of the line: its sequence and place there.
    auto pair_at = [&](long long f, int &s, int &tile, PSeq &w) {
        int lo = 0, hi = P_THREADS - 1;                      // the last thread whose sequences begin at or before f
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (flat[mid] <= f) lo = mid; else hi = mid - 1;
        }
        long long at = flat[lo];
        for (s = lo * per;; ++s) {
            w = p_seq<R>(P, s);
            if (f < at + w.tiles) break;
            at += w.tiles;
        }
        tile = (int)(f - at);
    };
    const long long per_f = (n_pairs + P_THREADS - 1) / P_THREADS, f0 = min(n_pairs, tid * per_f), f1 = min(n_pairs, f0 + per_f);
    long long steps = 0;
    if (f0 < f1) {
        int s, tile;
        PSeq w;
        pair_at(f0, s, tile, w);
        for (long long f = f0; f < f1; ++f) {
            while (tile == w.tiles) w = p_seq<R>(P, ++s), tile = 0;
            steps += p_tile<R>(P, w, tile++).steps + ITEM_STEPS;
        }
    }
    const long long total = H * scan(steps, steps_at);
    const int C = (int)min((long long)gridDim.x, min(total, n_pairs * H * MAX_SHARE));     // CTAs that get a share
    bool idle = (int)blockIdx.x >= C;
    const long long u0 = idle ? 0 : total * blockIdx.x / C, u1 = idle ? 0 : total * (blockIdx.x + 1) / C;
    if (!idle && f0 < f1 && H * steps_at[tid] <= u0 && u0 < H * (steps_at[tid] + steps)) {
        int s, tile;
        PSeq w;
        pair_at(f0, s, tile, w);
        long long at = H * steps_at[tid];
        for (;;) {
            while (tile == w.tiles) w = p_seq<R>(P, ++s), tile = 0;
            const int n = p_tile<R>(P, w, tile).steps + ITEM_STEPS;
            if (u0 < at + (long long)H * n) {
                B.seq = s;
                B.tile = tile;
                B.h = (int)((u0 - at) / n);
                B.item_at = at + (long long)B.h * n;
                break;
            }
            at += (long long)H * n;
            ++tile;
        }
    }
    // (Taken as late as it can be: a CTA waits for it for some microseconds, which pass beside the plan so.  4000 tokens of 32
    // heads of 128 over 4 bits: 204 us, and 211 with it at the beginning.)
    if (warp == 0) {
        __syncwarp();                            // (all lanes take it together, and one of them may have searched the share)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = B.tmem;
    Walk<R> w;
    if (!idle) idle = !w.first(P, B.seq, B.tile, B.h, B.item_at, u0, u1);
    __syncthreads();                             // (q's place is free)

    if (idle) {
    } else if (warp >= P_SOFT + P_CONV) {
        regs_down<PRegs<D>::REST>();
        if (warp < P_SOFT + P_CONV + NT && lane == 0) {
            const int t = warp - (P_SOFT + P_CONV);
            const uint32_t id_s = f16_idesc(KEYS, false), id_o = f16_idesc(D, true);
            const uint32_t q_d = sw128_lo(smem_u32(q_s + t * TB)), kv_d = sw128_lo(smem_u32(kv_s));
            const uint32_t s_at = tmem + S_COL + t * 128, o_at = tmem + O_COL + t * D;
            uint32_t st = 0, item = 0;           // steps and items so far
            auto scores = [&](uint32_t step) {   // S = q . keys
                const uint32_t kt = 2 * step, slot = kt % SLOTS;
                wait_for(&B.kv_full[slot], (kt / SLOTS) & 1, abort, P.status);
                // (w lies over S: the product that read it is done.)
                if (NT > 1 && step > 0) wait_for(&B.pv_done[t], (step - 1) & 1, abort, P.status);
                fence_after();
                const uint32_t k_d = kv_d + ((slot * TB) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = ((k >> 2) * (KEYS * 128) + (k & 3) * 32) >> 4;
                    if (k == 0)
                        mma_ss<false>(s_at, q_d + o, k_d + o, id_s);
                    else
                        mma_ss<true>(s_at, q_d + o, k_d + o, id_s);
                }
                prompt::mma_commit(&B.s_full[t]);
                prompt::mma_commit(&B.kv_empty[slot]);
            };
            do {
                wait_for(&B.q_full[t], item & 1, abort, P.status);
                scores(st);
                for (int i = w.step0; i < w.step1 && !*abort; ++i, ++st) {
                    const uint32_t vt = 2 * st + 1, slot = vt % SLOTS;
                    const bool more = i + 1 < w.step1;
                    if (NT == 1 && more) {
                        wait_for(&B.s_free, st & 1, abort, P.status);
                        scores(st + 1);
                    }
                    wait_for(&B.p_full[t], st & 1, abort, P.status);
                    // (The tiles' products take turns: one's run beside the other's softmax.)
                    if (NT > 1) wait_for(&B.turn[t], (st & 1) ^ (t == 0), abort, P.status);
                    wait_for(&B.kv_full[slot], (vt / SLOTS) & 1, abort, P.status);
                    if (i == w.step0) wait_for(&B.o_free[t], (item & 1) ^ 1, abort, P.status);
                    fence_after();
                    // O (+)= w . values
                    const uint32_t w_at = NT > 1 ? s_at : tmem + W_COL + (st & 1) * 64;
                    const uint32_t v_d = kv_d + ((slot * TB) >> 4);
                    if (i == w.step0)
                        mma_ts<false>(o_at, w_at, v_d, id_o);
                    else
                        mma_ts<true>(o_at, w_at, v_d, id_o);
#pragma unroll
                    for (int k = 1; k < KEYS / 16; ++k) mma_ts<true>(o_at, w_at + k * 8, v_d + ((k * 2048) >> 4), id_o);
                    prompt::mma_commit(&B.pv_done[t]);
                    prompt::mma_commit(&B.kv_empty[slot]);
                    if (NT > 1 && more) scores(st + 1);
                    if (NT > 1) mbar_arrive(&B.turn[t ^ 1]);
                }
                ++item;
            } while (w.next(P) && !*abort);
            prompt::mma_commit(&B.done);
            mbar_wait(&B.done, 0, abort, P.status, false);
        }
    } else if (warp >= P_SOFT) {
        regs_down<PRegs<D>::CONV>();
        // Widening: warp v takes tokens TW v .. TW v + TW - 1 of every step, a lane 16 bytes of a token at a time.
        constexpr int TW = KEYS / P_CONV, NP = TW / 16;      // (and as many times 16 tokens, of a page each)
        constexpr int TOK = D * F / 8, LPT = TOK / 16, LOADS = TW * LPT / 32;   // bytes and lanes a token, loads a lane
        // The eight lanes of a 16-byte store meet eight different chunks under the swizzle.  8 bits, two chunks a lane: its
        // low two bits are its place in 64 bytes, the next the token's parity.  4 bits, four chunks a lane: the low bit
        // is its half of a row of 128 bytes, the next two the token's.
        const int v = warp - P_SOFT;
        const int sub = F == 4 ? (lane & 1) | (LPT > 2 ? (lane >> 2) & (LPT - 2) : 0) : (lane & 3) | (LPT > 4 ? (lane >> 1) & (LPT - 4) : 0);
        const int tok = F == 4 ? (LPT == 2 ? lane >> 1 : LPT == 4 ? (lane >> 1 & 3) | (lane >> 2 & 4) : lane >> 1 & 3)
                               : ((lane >> 2) & 1) | (LPT == 4 ? (lane >> 2) & 6 : LPT == 8 ? (lane >> 3) & 2 : 0);
        uint32_t st = 0;
        do {
            const long long seq_table = w.seq * P.b.table_stride;
            uint4 kr[LOADS], vr[LOADS];
            int pages = -1;                      // lane NP s + e: page of the e-th 16 tokens of step (base + s), and its scales
            float2 scale = make_float2(-1.f, -INFINITY);
            auto look_up = [&](int step) {
                const int t = w.t.from + (step + lane / NP) * KEYS + TW * v + 16 * (lane % NP);
                pages = -1;
                scale = make_float2(-1.f, -INFINITY);
                if (t < w.t.to) {
                    const int page = P.b.table[seq_table + (t >> BL)];
                    if (page < 0 || page >= P.kv.n_blocks) {
                        atomicOr(P.status, STATUS_BOUNDS);
                    } else {
                        pages = page;
                        const long long ph = (long long)page * H + w.h;
                        if constexpr (F == 8)
                            scale = make_float2(P.kv.k_scale[ph], log2f(P.kv.v_scale[ph]));
                        else
                            scale = make_float2(1.f, 0.f);
                    }
                }
            };
            int base = w.step0;                  // first step looked up
            struct {
                int p0, p1;                      // pages of a step's first and last 16 tokens of this warp
                float2 scale;                    // lane e: scales of the e-th 16
            } k_of;                              // of the step whose keys are on their way
            auto find = [&](int step) {
                if (step - base == 32 / NP) look_up(base = step);
                const int at = NP * (step - base);
                k_of.p0 = __shfl_sync(~0u, pages, at);
                k_of.p1 = __shfl_sync(~0u, pages, at + NP - 1);
                k_of.scale = make_float2(__shfl_sync(~0u, scale.x, at + lane % NP), __shfl_sync(~0u, scale.y, at + lane % NP));
            };
            auto load = [&](const int8_t *pool, int step, int p0, int p1, uint4 (&r)[LOADS]) {
                const int t0 = w.t.from + step * KEYS + TW * v;
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const int tk = j * (32 / LPT) + tok, page = j < LOADS / NP ? p0 : p1;
                    r[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (page >= 0)
                        r[j] = *reinterpret_cast<const uint4 *>(pool + (((((long long)page * H + w.h) << BL) + ((t0 + tk) & BM)) * TOK) + 16 * sub);
                }
            };
            // 4 bits: scales and biases of a step's keys and values, (0, 0) of tokens that no row of the pair sees (whatever
            // may stand there); those of the values whose turn is next, as fp16 over their unit.
            uint32_t ka[F == 4 ? LOADS : 1], va[F == 4 ? LOADS : 1], v_now[F == 4 ? LOADS : 1];
            const int seen_from = P.window ? max(0, w.s.plan - w.s.q.n + w.tile * R / G - P.window + 1) : 0;
            auto load_affine = [&](int step, int p0, int p1) {
                if constexpr (F == 4) {
                    const int t0 = w.t.from + step * KEYS + TW * v;
#pragma unroll
                    for (int j = 0; j < LOADS; ++j) {
                        const int tk = j * (32 / LPT) + tok, page = j < LOADS / NP ? p0 : p1;
                        ka[j] = va[j] = 0;
                        if (page >= 0 && t0 + tk >= seen_from && t0 + tk < w.t.to) {
                            const long long at = ((((long long)page * H + w.h) << BL) + ((t0 + tk) & BM)) * (D / 64) + (sub >> 1);
                            ka[j] = P.k_affine[at];
                            va[j] = P.v_affine[at];
                        }
                    }
                }
            };
            // Units of the 16 tokens of loads j0 ..: the power of two above every value; scales and biases become fp16 over it,
            // such that widened values are a quarter of what they are over it (scales: at most 2 / 15 of it, times 2^18).
            // Returns its exponent, biased (0: only zeros).
            auto over_unit = [&](uint32_t (&a)[F == 4 ? LOADS : 1], int j0) {
                float most = 0.f;
#pragma unroll
                for (int j = j0; j < j0 + LOADS / NP; ++j) {
                    const float sc = __uint_as_float(a[j] << 16), bias = __uint_as_float(a[j] & 0xFFFF0000u);
                    most = fmaxf(most, fmaxf(fabsf(bias), fabsf(fmaf(15.f, sc, bias))));
                }
                const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(most)), unit = top == 0 ? 0 : min((top >> 23) + 1, 253u);
                const float inv = __uint_as_float((254u - unit) << 23);
#pragma unroll
                for (int j = j0; j < j0 + LOADS / NP; ++j)
                    a[j] = pack_half(__uint_as_float(a[j] << 16) * inv * 262144.f, __uint_as_float(a[j] & 0xFFFF0000u) * inv * 0.25f);
                return unit;
            };
            // Where this lane's 16 values of token tk go: two 16-byte chunks, 2 sub and 2 sub + 1 of the row of blocks of eight.
            auto store = [&](uint8_t *tile, const uint4 (&r)[LOADS], const bool tiny, const uint32_t (&affine)[F == 4 ? LOADS : 1]) {
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const int tk = TW * v + j * (32 / LPT) + tok;
                    if constexpr (F == 4) {
                        uint8_t *row4 = tile + (sub >> 1) * (KEYS * 128) + tk * 128;
                        const __half2 a = *reinterpret_cast<const __half2 *>(&affine[j]), sc = __low2half2(a), bias = __high2half2(a);
                        const uint32_t x4[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(row4 + (((4 * (sub & 1) + i) ^ (tk & 7)) << 4)) = widened(x4[i], sc, bias);
                        continue;
                    }
                    uint8_t *row = tile + (sub >> 2) * (KEYS * 128) + tk * 128;
                    const uint32_t x[4] = {r[j].x ^ 0x80808080u, r[j].y ^ 0x80808080u, r[j].z ^ 0x80808080u, r[j].w ^ 0x80808080u};
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[2 * i] = tiny ? lo2_tiny(x[i]) : lo2(x[i]);
                        y[2 * i + 1] = tiny ? hi2_tiny(x[i]) : hi2(x[i]);
                    }
                    const int c = (sub & 3) * 2;
                    *reinterpret_cast<uint4 *>(row + ((c ^ (tk & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4 *>(row + (((c + 1) ^ (tk & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            };
            auto publish = [&](uint32_t kt) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && !(P.stall && kt == 0)) mbar_arrive(&B.kv_full[kt % SLOTS]);
            };
            auto put_keys = [&](uint32_t step) {
                const uint32_t kt = 2 * step;
                if constexpr (F == 4) {
                    uint32_t k_unit[NP], v_unit[NP];
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        k_unit[e] = over_unit(ka, e * (LOADS / NP));
                        v_unit[e] = over_unit(va, e * (LOADS / NP));
                    }
                    // (Keys of zeros only: scores of 0 with any unit.)
                    const uint32_t ku = lane % NP == 0 ? k_unit[0] : k_unit[NP - 1], vu = lane % NP == 0 ? v_unit[0] : v_unit[NP - 1];
                    if (k_of.scale.x >= 0.f)
                        k_of.scale = make_float2(ku == 0 ? 1.f : __uint_as_float(ku << 23), vu == 0 ? -INFINITY : (float)((int)vu - 125));      // (four units: values stand as quarters)
#pragma unroll
                    for (int j = 0; j < LOADS; ++j) v_now[j] = va[j];
                }
                wait_for(&B.kv_empty[kt % SLOTS], ((kt / SLOTS) & 1) ^ 1, abort, P.status);
                store(kv_s + (kt % SLOTS) * TB, kr, true, ka);
                if (lane < NP) B.scale[step % SCALES][NP * v + lane] = k_of.scale;
                const bool there = __all_sync(~0u, k_of.scale.x >= 0.f);
                const float top_ks = NP > 1 ? fmaxf(k_of.scale.x, __shfl_xor_sync(~0u, k_of.scale.x, 1)) : k_of.scale.x;
                if (lane == 0)
                    B.top_ks[step % SCALES][v] = (there ? PAGES_THERE : 0u) | (top_ks < 0.f ? 0u : max(1u, (__float_as_uint(top_ks) + 0xFFFFu) >> 16));
                publish(kt);
                if (lane == 0) mbar_arrive(&B.scales[step % SCALES]);
            };
            look_up(w.step0);
            find(w.step0);
            load(P.kv.k, w.step0, k_of.p0, k_of.p1, kr);
            load_affine(w.step0, k_of.p0, k_of.p1);
            load(P.kv.v, w.step0, k_of.p0, k_of.p1, vr);
            // The slots are filled in the order in which the products free them.  One tile: a step's keys go before the
            // values of the step before it (99 -> 95 us for three chunks of up to 509 tokens, 16 heads of 256, window
            // 4096); two: after them.
            constexpr int AHEAD = NT == 1;
            if (AHEAD) {
                put_keys(st);
                if (w.step0 + 1 < w.step1) {
                    find(w.step0 + 1);
                    load(P.kv.k, w.step0 + 1, k_of.p0, k_of.p1, kr);
                    load_affine(w.step0 + 1, k_of.p0, k_of.p1);
                }
            }
            for (int i = w.step0; i < w.step1 && !*abort; ++i, ++st) {
                int p0 = k_of.p0, p1 = k_of.p1;              // (of step i + AHEAD)
                uint32_t v_affine[F == 4 ? LOADS : 1];       // (of step i)
                if (F == 4 && AHEAD)
#pragma unroll
                    for (int j = 0; j < (F == 4 ? LOADS : 1); ++j) v_affine[j] = v_now[j];
                if (i + AHEAD < w.step1) put_keys(st + AHEAD);
                if (F == 4 && !AHEAD)
#pragma unroll
                    for (int j = 0; j < (F == 4 ? LOADS : 1); ++j) v_affine[j] = v_now[j];
                if (i + AHEAD + 1 < w.step1) {
                    find(i + AHEAD + 1);
                    load(P.kv.k, i + AHEAD + 1, k_of.p0, k_of.p1, kr);
                    load_affine(i + AHEAD + 1, k_of.p0, k_of.p1);
                    if (!AHEAD) p0 = k_of.p0, p1 = k_of.p1;
                }
                const uint32_t vt = 2 * st + 1;
                wait_for(&B.kv_empty[vt % SLOTS], ((vt / SLOTS) & 1) ^ 1, abort, P.status);
                store(kv_s + (vt % SLOTS) * TB, vr, false, v_affine);
                publish(vt);
                if (i + 1 < w.step1) load(P.kv.v, i + 1, p0, p1, vr);
            }
        } while (w.next(P) && !*abort);
    } else {
        regs_up<PRegs<D>::SOFT>();
        // Softmax: thread `row` of tile t.
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + S_COL + t * 128, o_at = tmem + lanes + O_COL + t * D;
        const bool q16 = ((reinterpret_cast<uintptr_t>(P.q) | (uintptr_t)(P.q_stride * (P.q_f32 ? 4 : 2))) & 15) == 0;
        const bool out16 = ((reinterpret_cast<uintptr_t>(P.out) | (uintptr_t)(P.out_stride * 2)) & 15) == 0;
        uint32_t st = 0, item = 0, joins = 0;
        RowSum sum{-INFINITY, -INFINITY, 0.f, 0.f};
        // What the epilogue of an item needs after the walk has gone on.
        struct Done {
            uint16_t *out;       // null: not a row of the matrix
            long long item_at;
            int steps;
        } last{nullptr, 0, 0};
        auto epilogue = [&]() {
            wait_for(&B.pv_done[t], (st - 1) & 1, abort, P.status);
            fence_after();
            auto store = [&](int d, const float (&y)[32]) {          // 32 values of the row
                if (!last.out) return;
                uint32_t h[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(h[e])
                        : "f"(y[(2 * e & ~7) + chunk_place(F, 2 * e + 1 & 7)]), "f"(y[(2 * e & ~7) + chunk_place(F, 2 * e & 7)]));
                if (out16) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        reinterpret_cast<uint4 *>(last.out + d)[e] = make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        last.out[d + 2 * e] = (uint16_t)h[e];
                        last.out[d + 2 * e + 1] = (uint16_t)(h[e] >> 16);
                    }
                }
            };
            auto cta_of = [&](long long u) { return (int)(((u + 1) * C - 1) / total); };
            const int c_first = cta_of(last.item_at), parts = cta_of(last.item_at + last.steps - 1) - c_first + 1;
            const int k_mine = (int)blockIdx.x - c_first;
            auto slot = [&](int k) { return 2 * (c_first + k) + (k == 0); };     // (of a CTA's first item, which it goes on with; of its last, which it begins)
            // A part: [tile][D / 4][128 rows] of four outputs, after all parts [tile][128 rows] row sums.
            float4 *const parts4 = reinterpret_cast<float4 *>(P.part);
            float4 *const sums4 = parts4 + 2LL * gridDim.x * R * (D / 4);
            const OutFactor f = out_factor(sum);
            float4 *mine = parts4 + ((long long)slot(k_mine) * NT + t) * (D / 4) * 128 + row;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                uint32_t x[32];
                tmem_ld32(o_at + d, x);
                tmem_wait32(x);
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(x[e]);
                if (parts == 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        mul2(x[e], x[e + 1], f.f);
                        mul2(x[e], x[e + 1], f.g);
                        y[e] = sum.l == 0.f ? 0.f : __uint_as_float(x[e]);
                        y[e + 1] = sum.l == 0.f ? 0.f : __uint_as_float(x[e + 1]);
                    }
                    store(d, y);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) mine[(d / 4 + e) * 128] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.o_free[t]);
            if (parts == 1) return;
            sums4[((long long)slot(k_mine) * NT + t) * 128 + row] = make_float4(sum.m, sum.d, sum.l, 0.f);
            __threadfence();
            // (Bounded barriers of the softmax warps.)
            auto meet = [&](int i) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.joined[i]);
                wait_for(&B.joined[i], joins & 1, abort, P.status);
            };
            meet(0);
            if (tid == 0) {
                B.last = atomicAdd(P.count + c_first, 1) == parts - 1;
                B.arrived = last.item_at;
            }
            meet(1);
            ++joins;
            if (!B.last) return;
            __threadfence();
            if (tid == 0) P.count[c_first] = 0;
            auto sum_of = [&](int k) {
                const float4 x = __ldcg(sums4 + ((long long)slot(k) * NT + t) * 128 + row);
                return RowSum{x.x, x.y, x.z, 0.f};
            };
            // (The first parts' sums in one round of loads: mostly there are no more.)
            constexpr int AHEAD = 4;
            RowSum a{-INFINITY, -INFINITY, 0.f, 0.f}, first[AHEAD];
            float g[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) first[k] = sum_of(min(k, parts - 1));
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) join_maxima(a, first[k]);
#pragma unroll 1
            for (int k = AHEAD; k < parts; ++k) join_maxima(a, sum_of(k));
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                g[k] = o_factor(first[k], a) * out_factor(a).g;
                if (k < parts) a.l += first[k].l * l_factor(first[k], a);
            }
#pragma unroll 1
            for (int k = AHEAD; k < parts; ++k) {
                const RowSum x = sum_of(k);
                a.l += x.l * l_factor(x, a);
            }
            const float fa = out_factor(a).f;            // (its second factor is in the parts')
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = 0.f;
#pragma unroll 1
                for (int k = 0; k < parts; ++k) {
                    float f = 0.f;
                    if (k < AHEAD) {
#pragma unroll
                        for (int e = 0; e < AHEAD; ++e) f = k == e ? g[e] : f;
                    } else {
                        f = o_factor(sum_of(k), a) * out_factor(a).g;
                    }
                    const float4 *src = parts4 + ((long long)slot(k) * NT + t) * (D / 4) * 128 + (d / 4) * 128 + row;
                    float4 x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __ldcg(src + e * 128);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // (a part that saw nothing of this row holds no numbers)
                        y[4 * e] = f == 0.f ? y[4 * e] : fmaf(x[e].x, f, y[4 * e]);
                        y[4 * e + 1] = f == 0.f ? y[4 * e + 1] : fmaf(x[e].y, f, y[4 * e + 1]);
                        y[4 * e + 2] = f == 0.f ? y[4 * e + 2] : fmaf(x[e].z, f, y[4 * e + 2]);
                        y[4 * e + 3] = f == 0.f ? y[4 * e + 3] : fmaf(x[e].w, f, y[4 * e + 3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = a.l == 0.f ? 0.f : y[e] * fa;
                store(d, y);
            }
        };
        do {
            // This thread's row of q.
            const int n_rows = w.s.q.n * G, gr = w.tile * R + t * 128 + row;
            const bool real = gr < n_rows;
            const int gc = min(gr, n_rows - 1), i_tok = gc / G, head = w.h * G + gc - i_tok * G;
            const long long q_at = (long long)(w.s.q.row0 + i_tok) * P.q_stride + (long long)head * D;
            float amax = 0.f, sum_q = 0.f, sum_abs = 0.f, fq, sq;
            uint8_t *const q_row = q_s + t * TB + row * 128;
            auto put8 = [&](int d, const float (&x)[8]) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = F == 4 ? pack_half(x[e] * sq, x[e + 4] * sq) : pack_half(x[2 * e] * sq, x[2 * e + 1] * sq);
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                    sum_q += y.x + y.y;
                    sum_abs += fabsf(y.x) + fabsf(y.y);
                }
                *reinterpret_cast<uint4 *>(q_row + (d >> 6) * (KEYS * 128) + ((((d >> 3) & 7) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            };
            auto factors = [&]() {
                fq = row_factor(amax);
                sq = P.scale < 0.f ? -fq : fq;
            };
            if (F == 4 && P.q_f32 && q16) {
                // Whole rows at a time, LR lanes a row; AT of them on their way at once.  (Each thread its own row: three chunks of
                // up to 509 tokens, 16 heads of 256, 161 us, now 126; of bf16 rows the copies below are as fast.)
                constexpr int LR = D / 8, RPI = 32 / LR, AT = 4;
#pragma unroll 1
                for (int j0 = 0; j0 < LR; j0 += AT) {
                    float x[AT][8];
                    const int c = lane % LR;
                    long long src[AT];
#pragma unroll
                    for (int j = 0; j < AT; ++j) src[j] = __shfl_sync(~0u, q_at, (j0 + j) * RPI + lane / LR) + 8 * c;
#pragma unroll
                    for (int j = 0; j < AT; ++j) {
                        const float4 *at = reinterpret_cast<const float4 *>(static_cast<const float *>(P.q) + src[j]), a = at[0], b = at[1];
                        x[j][0] = a.x, x[j][1] = a.y, x[j][2] = a.z, x[j][3] = a.w, x[j][4] = b.x, x[j][5] = b.y, x[j][6] = b.z, x[j][7] = b.w;
                    }
#pragma unroll
                    for (int j = 0; j < AT; ++j) {
                        const int r = (j0 + j) * RPI + lane / LR;
                        float top = 0.f, sum = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[j][e]));
#pragma unroll
                        for (int o = 1; o < LR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                        const float f = P.scale < 0.f ? -row_factor(top) : row_factor(top);
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            h[e] = pack_half(x[j][e] * f, x[j][e + 4] * f);
                            sum += fabsf(x[j][e] * f) + fabsf(x[j][e + 4] * f);
                        }
#pragma unroll
                        for (int o = 1; o < LR; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
                        *reinterpret_cast<uint4 *>(q_s + t * TB + ((warp & 3) * 32 + r) * 128 + (c >> 3) * (KEYS * 128) + (((c & 7) ^ (r & 7)) << 4)) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                        // (to the thread of the row)
                        const float row_top = __shfl_sync(~0u, top, lane % RPI * LR), row_sum = __shfl_sync(~0u, sum, lane % RPI * LR);
                        if (lane / RPI == j0 + j) amax = row_top, sum_abs = row_sum;
                    }
                }
                factors();
            } else if (!P.q_f32 && q16) {
                // The warp's 32 rows as they are to their places, LR lanes a row; then each thread its own row there.
                constexpr int LR = D / 8, RPI = 32 / LR, CU = 2, QU = D == 256 ? 2 : 16;   // (measured: fewer are faster at dim 256, more at 128)
#pragma unroll CU
                for (int j = 0; j < LR; ++j) {
                    const int r = j * RPI + lane / LR, c = lane % LR;
                    const uint16_t *src = static_cast<const uint16_t *>(P.q) + __shfl_sync(~0u, q_at, r) + 8 * c;
                    const uint32_t dst = smem_u32(q_s + t * TB + ((warp & 3) * 32 + r) * 128 + (c >> 3) * (KEYS * 128) + (((c & 7) ^ (r & 7)) << 4));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                auto at = [&](int d) { return *reinterpret_cast<const uint4 *>(q_row + (d >> 6) * (KEYS * 128) + ((((d >> 3) & 7) ^ (row & 7)) << 4)); };
                uint32_t top = 0;                // magnitudes of bf16 are ordered as their bits
#pragma unroll QU
                for (int d = 0; d < D; d += 8) {
                    const uint4 r = at(d);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu)));
                }
                amax = __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16);
                factors();
#pragma unroll QU
                for (int d = 0; d < D; d += 8) {
                    const uint4 r = at(d);
                    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(u[e] << 16), x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                    put8(d, x);
                }
            } else {
                auto q8 = [&](int d, float (&x)[8]) {
                    if (P.q_f32) {
                        const float *src = static_cast<const float *>(P.q) + q_at + d;
                        if (q16) {
                            const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
                            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = src[e];
                        }
                    } else {
                        const uint16_t *src = static_cast<const uint16_t *>(P.q) + q_at + d;
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((uint32_t)src[e] << 16);
                    }
                };
#pragma unroll 8
                for (int d = 0; d < D; d += 8) {
                    float x[8];
                    q8(d, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
                }
                factors();
#pragma unroll 8
                for (int d = 0; d < D; d += 8) {
                    float x[8];
                    q8(d, x);
                    put8(d, x);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.q_full[t]);
            if (item > 0) epilogue();
            last.out = real ? P.out + (long long)(w.s.q.row0 + i_tok) * P.out_stride + (long long)head * D : nullptr;
            last.item_at = w.item_at;
            last.steps = w.t.steps;
            ++item;

            // Factor of a score in tensor memory, and the offset that comes off it first; tokens that the row sees.
            constexpr float CODE = F == 8 ? TINY : 0.25f, TOP = F == 8 ? 128.f * TINY : 0.25f;   // of a key in shared memory: its unit, a bound
            const float rowf = fabsf(P.scale) * 1.44269504088896340736f / fq * (1.f / CODE), off = F == 8 ? sum_q * (-128.f * TINY) : 0.f;
            const int first = w.s.q.end - w.s.q.n, pos = first + i_tok;
            const int see_to = P.causal ? min(w.s.q.end, pos + 1) : w.s.q.end, see_from = P.window ? pos - P.window + 1 : 0;
            const int g0 = min(w.tile * R + t * 128, n_rows - 1), g1 = min(w.tile * R + t * 128 + 127, n_rows - 1);
            const int all_to = P.causal ? min(w.s.q.end, first + g0 / G + 1) : w.s.q.end;
            const int all_from = P.window ? first + g1 / G - P.window + 1 : 0;
            sum = RowSum{-INFINITY, -INFINITY, 0.f, 0.f};
            float n = -INFINITY;                 // the maximum of s + log2(vs)
            // Where the terms of an exponent could pass FAR, which is with a key scale above far_ks (of the warp's rows, twice
            // in its upper half), the warp's scores, m and n are relative to `base` from there on.
            float base = 0.f;
            uint32_t far_ks = __reduce_min_sync(~0u, __float_as_uint(FAR / (sum_abs * TOP * rowf)) >> 16) * 0x10001u;
            for (int i = w.step0; i < w.step1 && !*abort; ++i, ++st) {
                const int t0 = w.t.from + i * KEYS;
                wait_for(&B.scales[st % SCALES], (st / SCALES) & 1, abort, P.status);
                constexpr uint32_t THERE = PAGES_THERE * 0x10001u;
                uint32_t top_ks, there;          // of pairs of the widening warps' numbers
                if (P_CONV > 4) {
                    const uint4 k = *reinterpret_cast<const uint4 *>(B.top_ks[st % SCALES]);
                    top_ks = __vmaxu2(__vmaxu2(k.x & ~THERE, k.y & ~THERE), __vmaxu2(k.z & ~THERE, k.w & ~THERE));
                    there = k.x & k.y & k.z & k.w & THERE;
                } else {
                    const uint2 k = *reinterpret_cast<const uint2 *>(B.top_ks[st % SCALES]);
                    top_ks = __vmaxu2(k.x & ~THERE, k.y & ~THERE);
                    there = k.x & k.y & THERE;
                }
                const bool far = __vmaxu2(top_ks, far_ks) != far_ks;
                const bool masked = t0 < all_from || t0 + KEYS > all_to || there != THERE || far;
                wait_for(&B.s_full[t], st & 1, abort, P.status);
                fence_after();
                const float2 *const sc = B.scale[st % SCALES];
                // f(c, x) on the columns 32 c ..  One tile: all of them are taken into registers at once, so that the
                // next step's scores can follow.  Two: they are read again each time, in a loop (unrolled, a step's
                // code would not stay in the instruction caches).
                uint32_t all[NT == 1 ? 4 : 1][32];
                if constexpr (NT == 1) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, all[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_wait32(all[c]);
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B.s_free);
                }
                auto columns = [&](auto f) {
                    if constexpr (NT == 1) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) f(c, all[c]);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(s_at + 32 * c, x);
                            tmem_wait32(x);
                            f(c, x);
                        }
                    }
                };
                // Factor of a score (`least`: never 0, so that -inf stays -inf; a page of zeros has scores of 0 all the same).
                float row_f = rowf, least = 1e-30f, off_s = off;
                auto factor = [&](float ks) { return fmaxf(row_f * ks, least); };
                if (masked) {
                    // Tokens that the row does not see, first.
                    columns([&](int c, uint32_t (&x)[32]) {
                        const int from = see_from - t0 - 32 * c, to = see_to - t0 - 32 * c;
                        const bool p0 = sc[2 * c].x >= 0.f, p1 = sc[2 * c + 1].x >= 0.f;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e < from || e >= to || !(e < 16 ? p0 : p1)) x[e] = __float_as_uint(-INFINITY);
                        if (NT > 1) tmem_st32(s_at + 32 * c, x);
                    });
                    if (NT > 1) tmem_wait_st();
                    if (far) {
                        // The scores as fp32 numbers less the largest so far, which is the new base; m and n move with it.
                        float top = base + sum.m;
                        columns([&](int c, uint32_t (&x)[32]) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float y = -INFINITY;
#pragma unroll
                                for (int e = 16 * h; e < 16 * h + 16; ++e) y = fmaxf(y, __uint_as_float(x[e]));
                                top = fmaxf(top, __fmul_rn(y + off, factor(sc[2 * c + h].x)));
                            }
                        });
                        const float to = base_of(top), by = base - to;
                        columns([&](int c, uint32_t (&x)[32]) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[e]) + off, factor(sc[2 * c + e / 16].x)), to));
                            if (NT > 1) tmem_st32(s_at + 32 * c, x);
                        });
                        if (NT > 1) tmem_wait_st();
                        sum.l *= exp2_fast(sum.m + by);
                        n += by;
                        sum.m = top == -INFINITY ? -INFINITY : 0.f;
                        base = to;
                        far_ks = 0;                          // (and so in the steps that follow)
                        row_f = off_s = 0.f, least = 1.f;    // (a factor of 1, and no offset)
                    }
                }
                // The maxima of s and of s + log2(vs), by groups of 16 tokens.
                float mt = sum.m, nt = n;
                columns([&](int c, uint32_t (&x)[32]) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 z = sc[2 * c + h];
                        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            top[0] = max3(top[0], __uint_as_float(x[16 * h + e]), __uint_as_float(x[16 * h + e + 1]));
                            top[1] = max3(top[1], __uint_as_float(x[16 * h + e + 2]), __uint_as_float(x[16 * h + e + 3]));
                        }
                        const float m = (fmaxf(top[0], top[1]) + off_s) * factor(z.x);
                        mt = fmaxf(mt, m);
                        nt = fmaxf(nt, m + z.y);
                    }
                });
                // Maxima that have grown by less than SLACK stay as they are: w then reaches 2^(15 + SLACK), below fp16's end.
                mt = mt > sum.m + SLACK ? mt : sum.m;
                nt = nt > n + SLACK ? nt : n;
                const float mm = mt == -INFINITY ? 0.f : mt, nn = nt == -INFINITY ? INFINITY : nt;
                if (mt != sum.m && sum.l != 0.f) sum.l *= exp2_fast(sum.m - mt);
                const bool grew = nt > n;
                const float shrink = n == -INFINITY ? 0.f : exp2_fast(n - nt);
                sum.m = mt;
                n = nt;
                constexpr int AT = NT == 1 ? 1 : 2;          // 32 columns each at once (more measured no faster)
                auto rescale = [&]() {           // the outputs so far, to the new maximum
                    if (i > w.step0 && __any_sync(~0u, grew)) {
#pragma unroll 1
                        for (int d = 0; d < D; d += 32 * AT) {
                            uint32_t x[AT][32];
#pragma unroll
                            for (int c = 0; c < AT; ++c) tmem_ld32(o_at + d + 32 * c, x[c]);
#pragma unroll
                            for (int c = 0; c < AT; ++c) {
                                tmem_wait32(x[c]);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) mul2(x[c][e], x[c][e + 1], shrink);
                                tmem_st32(o_at + d + 32 * c, x[c]);
                            }
                        }
                    }
                };
                if (NT > 1) rescale();           // (every earlier product is done: this step's scores were issued after them)
                // The weights w, over S (dim 256: beside it).
                const uint32_t w_at = NT > 1 ? s_at : tmem + lanes + W_COL + (st & 1) * 64;
                columns([&](int c, uint32_t (&x)[32]) {
                    uint32_t y[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // w = 2^(s - m + e), p = w 2^-e with the page's e; below 2^-45 w is 0 in fp16 whatever it is.  (Past 2^300 no
                        // output is left; w itself is 2^(15 + SLACK) at most with any e.)
                        const float2 z = sc[2 * c + h];
                        const float e0 = fminf(fmaxf(mm + z.y - nn + W_EXP, -45.f), 300.f), f = factor(z.x), k = off_s * f - mm + e0;
                        float l0 = 0.f, l1 = 0.f;
#pragma unroll
                        for (int e = 16 * h; e < 16 * h + 16; e += 2) {
                            fma2(x[e], x[e + 1], f, k);
                            const float a = exp2_fast(__uint_as_float(x[e])), b = exp2_fast(__uint_as_float(x[e + 1]));
                            add2(l0, l1, a, b);
                            y[e / 2] = pack_half(a, b);
                        }
                        sum.l = fmaf(l0 + l1, exp2_fast(-e0), sum.l);
                    }
                    tmem_st16(w_at + 16 * c, y);
                });
                if (NT == 1 && i > w.step0) {
                    // (The last step's product runs beside the exponentials.)
                    wait_for(&B.pv_done[0], (st - 1) & 1, abort, P.status);
                    fence_after();
                    rescale();
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.p_full[t]);
            }
            sum.d = n - base_of(sum.m);
            sum.m += base;
        } while (w.next(P) && !*abort);
        epilogue();
        if (tid == 0 && *abort) {
            // A wait ran out, and the walk stopped.  If the last item of this CTA's share, which the CTAs after it may
            // share, is among those left, its part is counted all the same: the counter comes back to zero, and the
            // launches that follow join when their own parts are there.
            Walk<R> z;
            z.first(P, B.seq, B.tile, B.h, B.item_at, total * blockIdx.x / C, total * (blockIdx.x + 1) / C);
            bool later = false;
            while (z.next(P)) later = true;
            const int parts = (int)(((z.item_at + z.t.steps) * C - 1) / total) - (int)blockIdx.x + 1;
            if (later && parts > 1 && B.arrived != z.item_at && atomicAdd(P.count + blockIdx.x, 1) == parts - 1) P.count[blockIdx.x] = 0;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace attend
}  // namespace tfq
