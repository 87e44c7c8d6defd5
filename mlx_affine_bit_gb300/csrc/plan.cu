// plan.cu -- tf_kv_plan: the pages and places of a step's tokens (tfserve.h).
//
// With had_s and has_s the pages of sequence s before and after its change, three
// running sums over the sequences (rows, pages given back, pages taken) say where
// everything goes: with n pages on the stack and B given back, the k-th page given
// back is put at n + B - 1 - k, and the k-th taken comes from there.  A row's
// sequence is the last whose rows begin at or before it.
//
// Bound by a chain of latencies: a launch, the lengths, two barriers of the sums,
// the stack, the table, the rows (48 sequences of a token 3.2 us a call in a graph).  One CTA does
// the sums and the pages, and the rows too where they are few; more rows are filled
// by a second kernel, a thread a row (64,000 rows of 256 sequences: 16 us in one CTA,
// 9 in two launches; at 4096 rows both take the same).
#include <cuda_runtime.h>

#include <climits>

#include "kv.h"

using namespace tfq;

namespace {

constexpr int MAX_SEQS = 4096, MAX_THREADS = 1024, ROWS_HERE = 4096;
constexpr int AT = 4;                    // pages that a thread looks at at once, and keeps

struct PlanParams {
    tf_kv_pages p;
    const int32_t *change;
    int rows, max_rows, max_len;
    int32_t *row_start, *positions;
    long long *slots;
    int32_t *info;
    int *status;
    int block_log2;
};

// The last of n sums (starts[0] = 0, never falling) that is at or before x.
__device__ __forceinline__ int last_at(const int *starts, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Row r: its token's place in its sequence and in the cache, -1 behind the last row.
__device__ __forceinline__ void place_row(const PlanParams &P, const int *starts, int r) {
    int pos = -1;
    long long slot = -1;
    if (r < starts[P.p.n_seqs]) {
        const int s = last_at(starts, P.p.n_seqs, r);
        pos = P.p.kv_len[s] - (starts[s + 1] - r);
        slot = ((long long)P.p.table[s * P.p.table_stride + (pos >> P.block_log2)] << P.block_log2) + (pos & (P.p.block - 1));
    }
    if (P.positions) P.positions[r] = pos;
    if (P.slots) P.slots[r] = slot;
}

__global__ void __launch_bounds__(MAX_THREADS) plan_kernel(const PlanParams P, bool rows_here) {
    __shared__ int s_more[MAX_SEQS + 1], s_gone[MAX_SEQS + 1];   // pages taken and given back before each sequence; then rows
    __shared__ long long s_sum[3][MAX_THREADS / 32];
    __shared__ int s_longest[2][MAX_THREADS / 32];
    const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, n = P.p.n_seqs, BL = P.block_log2;
    const long long room = min((long long)P.max_len, (long long)P.p.max_pages << BL);

    // The sums over this thread's sequences, and over those of the threads before it.
    const int per = (n + nt - 1) / nt, s0 = min(n, tid * per), s1 = min(n, s0 + per);
    const int n_free = *P.p.n_free;
    bool bad = n_free < 0 || n_free > P.p.n_blocks;
    long long sum[3] = {0, 0, 0};                // rows, pages taken, pages given back
    int longest = 0, stands = 0;
    for (int s = s0; s < s1; ++s) {
        const long long len = P.p.kv_len[s], by = P.change[s], end = len + by;
        stands = max(stands, (int)len);
        if (len < 0 || len > (long long)P.p.max_pages << BL || end < 0 || end > room || by > P.max_rows) {
            bad = true;
            continue;
        }
        const long long pages = ((end + P.p.block - 1) >> BL) - ((len + P.p.block - 1) >> BL);
        longest = max(longest, (int)end);
        sum[0] += max(0LL, by);
        sum[1] += max(0LL, pages);
        sum[2] += max(0LL, -pages);
    }
    long long at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        long long x = sum[i];
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        at[i] = x - sum[i];
        if (lane == 31) s_sum[i][warp] = x;
    }
    longest = __reduce_max_sync(~0u, longest);
    stands = __reduce_max_sync(~0u, stands);
    if (lane == 0) s_longest[0][warp] = longest, s_longest[1][warp] = stands;
    bad = __syncthreads_or(bad);
    // (The warps' sums, in every warp again: a loop over 32 of them takes 2 us.)
    const bool there = lane < nt / 32;
    longest = __reduce_max_sync(~0u, there ? s_longest[0][lane] : 0);
    stands = __reduce_max_sync(~0u, there ? s_longest[1][lane] : 0);
    long long all[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const long long own = there ? s_sum[i][lane] : 0;
        long long x = own;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        all[i] = __shfl_sync(~0u, x, 31);
        at[i] += __shfl_sync(~0u, x - own, warp);
    }
    bad = bad || all[0] > ((P.positions || P.slots) ? P.rows : INT_MAX) || n_free + all[2] > P.p.n_blocks;
    // (From here on every sum fits 32 bits: no more pages are given back than the pool has, and of pages taken no
    // more are looked at than there are.)
    const long long few = bad ? 0 : max(0LL, all[1] - (n_free + all[2]));
    const int gone = (int)all[2], more = bad || few ? 0 : (int)all[1], top = bad ? 0 : n_free + gone;
    if (!bad) {
        long long m = at[1], g = at[2];
        for (int s = s0; s < s1; ++s) {
            const int len = P.p.kv_len[s], end = len + P.change[s];
            const int pages = ((end + P.p.block - 1) >> BL) - ((len + P.p.block - 1) >> BL);
            s_more[s] = (int)min((long long)INT_MAX, m);
            s_gone[s] = (int)g;
            m += max(0, pages);
            g += max(0, -pages);
        }
    }
    __syncthreads();
    auto had = [&](int s) { return (P.p.kv_len[s] + P.p.block - 1) >> BL; };
    auto has = [&](int s) { return (P.p.kv_len[s] + P.change[s] + P.p.block - 1) >> BL; };
    // The k-th page given back: its entry of the table.  It goes to the stack's place top - 1 - k, and from there, if as
    // many are taken, to the k-th place that needs one.
    auto left = [&](int k) {
        const int s = last_at(s_gone, n, k);
        return P.p.table + s * P.p.table_stride + has(s) + (k - s_gone[s]);
    };
    auto page_at = [&](int k) { return k < gone ? *left(k) : P.p.free_pages[top - 1 - k]; };
    auto move = [&](int k, int page) {
        if (k < gone) {
            P.p.free_pages[top - 1 - k] = page;
            *left(k) = -1;
        }
        if (k < more) {
            const int s = last_at(s_more, n, k);
            P.p.table[s * P.p.table_stride + had(s) + (k - s_more[s])] = page;
        }
    };
    // Every number is looked at before any is changed.  (No thread reads what another one changes: sequences give pages
    // back or take some, and those that are taken from under the ones given back lie below them on the stack.)
    const int moved = bad || few ? 0 : max(gone, more);
    int page[AT];
    bool wrong = false;
#pragma unroll
    for (int i = 0; i < AT; ++i) page[i] = tid + i * nt < moved ? page_at(tid + i * nt) : 0;
#pragma unroll
    for (int i = 0; i < AT; ++i) wrong |= page[i] < 0 || page[i] >= P.p.n_blocks;
    for (int k = tid + AT * nt; k < moved; k += nt) {
        const int x = page_at(k);
        wrong |= x < 0 || x >= P.p.n_blocks;
    }
    bad = __syncthreads_or(wrong) || bad;
    const bool go = !bad && !few;
    if (go) {
#pragma unroll
        for (int i = 0; i < AT; ++i)
            if (tid + i * nt < moved) move(tid + i * nt, page[i]);
        for (int k = tid + AT * nt; k < moved; k += nt) move(k, page_at(k));
    }
    __syncthreads();                             // (the lengths have been read)
    int *const starts = s_gone;
    int row = (int)at[0];
    for (int s = s0; s < s1; ++s) {
        const int by = go ? P.change[s] : 0;
        starts[s] = P.row_start[s] = go ? row : 0;
        row += max(0, by);
        if (go && by) P.p.kv_len[s] += by;
    }
    if (tid == 0) {
        starts[n] = P.row_start[n] = go ? (int)all[0] : 0;
        if (go) *P.p.n_free = top - more;
        P.info[0] = bad ? 2 : few ? 1 : 0;
        P.info[1] = bad ? 0 : (int)min((long long)INT_MAX, few);
        P.info[2] = starts[n];
        P.info[3] = go ? longest : stands;
        if (bad) atomicOr(P.status, STATUS_BOUNDS);
    }
    if (rows_here) {
        __syncthreads();
        for (int r = tid; r < P.rows; r += nt) place_row(P, starts, r);
    }
}

__global__ void __launch_bounds__(256) rows_kernel(const PlanParams P) {
    __shared__ int starts[MAX_SEQS + 1];
    for (int s = threadIdx.x; s <= P.p.n_seqs; s += 256) starts[s] = P.row_start[s];
    __syncthreads();
    for (long long r = blockIdx.x * 256LL + threadIdx.x; r < P.rows; r += gridDim.x * 256LL) place_row(P, starts, (int)r);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" int tf_kv_plan(const tf_kv_pages *pages, const int32_t *change, int rows, int max_rows, int max_len,
                          int32_t *row_start, int32_t *positions, int64_t *slots, int32_t *info, void *stream) {
    fail_message(TF_OK, "");
    if (!pages) return fail_message(TF_EINVAL_PTR, "NULL pages");
    const void *words[] = {pages->table, pages->kv_len, pages->free_pages, pages->n_free, change, row_start, info};
    for (const void *p : words)
        if (!p || !aligned(p, 4))
            return fail_message(TF_EINVAL_PTR, "table, kv_len, free_pages, n_free, change, row_start and info must be given, 4-byte aligned");
    if (!aligned(positions, 4) || !aligned(slots, 8))
        return fail_message(TF_EINVAL_PTR, "positions must be 4-byte aligned, slots 8-byte aligned");
    if (pages->n_seqs < 1 || pages->n_seqs > MAX_SEQS) return fail_message(TF_EINVAL_SIZE, "n_seqs must be in [1, 4096]");
    if (pages->block != 16 && pages->block != 32 && pages->block != 64 && pages->block != 128)
        return fail_message(TF_EINVAL_SIZE, "block must be 16, 32, 64 or 128");
    if (pages->n_blocks < 1) return fail_message(TF_EINVAL_SIZE, "n_blocks must be at least 1");
    if (pages->max_pages < 1 || (long long)pages->max_pages * pages->block > (1 << 20))
        return fail_message(TF_EINVAL_SIZE, "max_pages must be at least 1, and hold 2^20 tokens at most");
    if (pages->table_stride < pages->max_pages) return fail_message(TF_EINVAL_STRIDE, "table_stride below max_pages");
    if (rows < 0 || max_rows < 1 || (rows == 0) != (!positions && !slots))
        return fail_message(TF_EINVAL_ROWS, "max_rows must be at least 1, and rows positive where there are positions or slots, else 0");
    if (max_len < 1 || max_len > (1 << 20)) return fail_message(TF_EINVAL_SIZE, "max_len must be in [1, 2^20]");
    int nsm = 0, *status = nullptr;
    const int rc = device_info(&nsm, &status);
    if (rc) return rc;
    const PlanParams P{*pages, change, rows, max_rows, max_len, row_start, positions, reinterpret_cast<long long *>(slots), info, status,
                       __builtin_ctz(pages->block)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool here = rows <= ROWS_HERE;
    const int threads = pages->n_seqs <= 256 && (rows <= 512 || !here) && max_rows <= 64 ? 256 : MAX_THREADS;
    plan_kernel<<<1, threads, 0, st>>>(P, here);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && !here) {
        rows_kernel<<<(unsigned)((rows + 255LL) / 256 < 4LL * nsm ? (rows + 255LL) / 256 : 4LL * nsm), 256, 0, st>>>(P);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_plan launch");
}
