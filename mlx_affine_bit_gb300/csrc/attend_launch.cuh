// attend_launch.cuh -- the host side of an attention call over either cache: checks, the
// choice of the kernel, the launch.  F: bits of a code, 8 (tfdecode.h) or 4 (tfserve.h).
#pragma once
#include <cuda_runtime.h>

#include <algorithm>

#include "attend_prompt.cuh"
#include "attend_rows.cuh"
#include "kv.h"

namespace tfq {
namespace attend {

// The parts and arrival counters of the calls on a stream; allocated on its first call (attend.cu).
struct Workspace {
    float *part = nullptr;
    int *count = nullptr;
};
int workspace(cudaStream_t st, int nsm, Workspace *out);

// CTAs of a rows kernel that an SM holds at once (looked up once a device, with its shared-memory limit raised).
template <int F, int D, int NT>
cudaError_t resident(int *out) {
    static int n[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int v = __atomic_load_n(&n[dev], __ATOMIC_ACQUIRE);
    if (!v) {
        auto k = rows_kernel<F, D, NT>;
        constexpr int smem = smem_bytes(F, D, NT);
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, k, THREADS, smem);
        if (e != cudaSuccess) return e;
        if (v < 1) return cudaErrorLaunchOutOfResources;
        __atomic_store_n(&n[dev], v, __ATOMIC_RELEASE);
    }
    *out = v;
    return cudaSuccess;
}

// The launch: as many CTAs as are resident at once, or one a step where there are fewer.
template <int F, int D, int NT>
int launch_rows(Params &P, long long steps, int nsm, cudaStream_t st) {
    int per_sm = 0;
    cudaError_t e = resident<F, D, NT>(&per_sm);
    if (e != cudaSuccess) return cuda_error(e, "kv_attend set-up");
    const long long grid = std::min({steps, (long long)nsm * per_sm, (long long)MAX_PARTS});
    Workspace w;
    const int rc = workspace(st, nsm, &w);
    if (rc) return rc;
    P.part = w.part;
    P.count = w.count;
    P.item_steps = steps > grid ? item_rows(D) : 0;
    rows_kernel<F, D, NT><<<(unsigned)grid, THREADS, smem_bytes(F, D, NT), st>>>(P);
    e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_attend launch");
}

// The same for the prompt kernel: one CTA an SM.
template <int F, int D>
int launch_prompt(Params &P, long long steps, int nsm, cudaStream_t st) {
    constexpr int smem = p_smem(D);
    static unsigned attr_set = 0;   // one bit per device: shared-memory limit raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    const unsigned bit = 1u << (dev & 31);
    if (!(__atomic_load_n(&attr_set, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(prompt_kernel<F, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_error(e, "kv_attend set-up");
        __atomic_fetch_or(&attr_set, bit, __ATOMIC_RELEASE);
    }
    const long long grid = std::min({steps, (long long)nsm, (long long)MAX_PARTS});
    Workspace w;
    const int rc = workspace(st, nsm, &w);
    if (rc) return rc;
    P.part = w.part;
    P.count = w.count;
    prompt_kernel<F, D><<<(unsigned)grid, P_THREADS, smem, st>>>(P);
    e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_attend launch");
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int check_flags(int flags) {
    if (flags & ~(TF_IN_F32 | TF_KV_CAUSAL | TF_KV_BY_ROWS | TF_KV_BY_TILES))
        return fail_message(TF_EINVAL_FLAGS, "unknown attention flags");
    if ((flags & TF_KV_BY_ROWS) && (flags & TF_KV_BY_TILES))
        return fail_message(TF_EINVAL_FLAGS, "TF_KV_BY_ROWS and TF_KV_BY_TILES exclude each other");
    return TF_OK;
}

// A call whose flags and cache (in P, which this fills) have been checked.
template <int F>
int call(Params &P, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads, void *out, int64_t out_stride, float scale,
         int window, int flags, void *stream) {
    const tf_kv *const kv = &P.kv;
    int rc = check_batch(kv->block, batch);
    if (rc) return rc;
    if (heads < 1 || heads % kv->kv_heads != 0)
        return fail_message(TF_EINVAL_SIZE, "heads must be a multiple of kv_heads");
    if (heads / kv->kv_heads > 1024) return fail_message(TF_EINVAL_SIZE, "more than 1024 query heads a key/value head");
    if (window < 0 || (window > 0 && !(flags & TF_KV_CAUSAL)))
        return fail_message(TF_EINVAL_SIZE, "window must be 0, or positive with TF_KV_CAUSAL");
    if (!q || !out || !aligned(q, flags & TF_IN_F32 ? 4 : 2) || !aligned(out, 2))
        return fail_message(TF_EINVAL_PTR, "NULL q or out, or not aligned to their type");
    const long long width = (long long)heads * kv->dim;
    if (q_stride < width || out_stride < width)
        return fail_message(TF_EINVAL_STRIDE, "q_stride or out_stride below heads * dim");
    int nsm = 0, *status = nullptr;
    rc = device_info(&nsm, &status);
    if (rc) return rc;

    const int token_bytes = kv->dim * F / 8;
    const long long pool_rows = (long long)kv->n_blocks * kv->kv_heads * kv->block * token_bytes / 128;
    if (pool_rows > 0x7FFFFFFF) return fail_message(TF_EINVAL_SIZE, "a pool of more than 2^38 bytes");
    const int box_rows = std::min(kv->block, 16 * tiles_of(kv->dim)) * token_bytes / 128;
    rc = tensor_map_rows128(&P.tm_k, kv->k, pool_rows, box_rows);
    if (!rc) rc = tensor_map_rows128(&P.tm_v, kv->v, pool_rows, box_rows);
    if (rc) return rc;
    P.b = *batch;
    P.q = q;
    P.q_stride = q_stride;
    P.out = static_cast<uint16_t *>(out);
    P.out_stride = out_stride;
    P.status = status;
    P.group = heads / kv->kv_heads;
    P.scale = scale;
    // (A window that holds every token is none; the kernels' positions less a window then stay within 32 bits.)
    P.window = window = window < batch->max_len ? window : 0;
    P.block_log2 = __builtin_ctz(kv->block);
    P.causal = (flags & TF_KV_CAUSAL) != 0;
    P.q_f32 = (flags & TF_IN_F32) != 0;
    P.stall = take_stall();
    const long long max_group_rows = (long long)batch->max_rows * P.group;
    if (max_group_rows > (1 << 30)) return fail_message(TF_EINVAL_SIZE, "too many rows of one sequence");
    long long span = batch->max_len;
    if (window > 0) span = std::min(span, (long long)window + batch->max_rows + 32);
    // Rows or prompt kernel: the one that is expected to take less time, by what they measured over 17 to 400
    // rows of 1 to 16 sequences of 4000 and 60000 tokens.  The rows kernel takes 16 rows at a time (some 6.5 ns
    // for 128 tokens of dim 128 with all SMs at work, on top of 12 us), the prompt kernel 256 (dim 256: 128;
    // some 2.9 us for 128 tokens on one SM, on top of 45 us).  64 rows of 16 x 4000 tokens, dim 128: 109
    // against 107 us; 128 rows 197 against 107; 128 rows of 1 x 4000 tokens 32 against 42.
    // The host knows the largest number of rows and the largest length of a sequence only, and takes them for all:
    // a chunk of 500 rows beside 47 single tokens over 4000 to 4500 tokens goes to the prompt kernel as a whole and takes
    // 328 us (by rows 270), where a call for the chunk and one for the others take 67 and 72 (4 bits: 324, 286, 67 and 58).
    bool prompt = (flags & TF_KV_BY_TILES) != 0;
    if (max_group_rows > 16 && !(flags & (TF_KV_BY_ROWS | TF_KV_BY_TILES))) {
        const double blocks = (double)batch->n_seqs * kv->kv_heads * (double)((span + 127) / 128);
        const int pair = 128 * p_tiles(kv->dim);
        const double pairs = (double)((max_group_rows + pair - 1) / pair), items = (double)batch->n_seqs * kv->kv_heads * pairs;
        const double ctas = std::min((double)nsm, items * MAX_SHARE);
        // 4 bits: the same, over 17 to 512 rows of 1, 4 and 16 sequences of 1000, 4000 and 60000 tokens; times by the dimension.
        // 128 rows of 16 x 4000 tokens, 8 heads of 128: 207 against 110 us; of 1 x 60000: 172 against 190; 64 rows of 16 x
        // 4000, 2 heads of 256: 77 against 57, of 1 x 60000: 75 against 181; 128 rows of 4 x 1000, 16 heads of 64: 36 and 29.
        const int at = kv->dim / 128;
        constexpr double ROWS_STEP[] = {3.9, 5.8, 12.3}, TILES_CALL[] = {26e3, 30e3, 38e3}, TILES_STEP[] = {2300.0, 2900.0, 2600.0};
        const double row_tiles = (double)((max_group_rows + 15) / 16);
        const double t_rows = F == 4 ? 18e3 + ROWS_STEP[at] * blocks * row_tiles : 12e3 + 6.5 * blocks * row_tiles * kv->dim / 128;
        const double t_prompt = F == 4 ? TILES_CALL[at] + TILES_STEP[at] * blocks * pairs / ctas : 45e3 + 2900.0 * blocks * pairs / ctas;
        prompt = t_prompt < t_rows;
    }
    // Rows kernel: tiles of 8 rows where no sequence has more a head (4 rows of 48 x 4000 tokens, 8 heads of 128: 71 us,
    // 77 in a tile of 16; 8 rows of 16 x 4000, 2 heads of 256: 28 and 33), else of 16.
    const int nt = max_group_rows <= 8 ? 1 : 2, tile_rows = prompt ? 128 * p_tiles(kv->dim) : 8 * nt;
    const long long tiles = (max_group_rows + tile_rows - 1) / tile_rows;
    const int step = prompt ? KEYS : step_of(kv->dim);
    const long long most = std::max(1LL, (1LL << 40) / (batch->n_seqs * (long long)kv->kv_heads));
    const long long steps = batch->n_seqs * (long long)kv->kv_heads * std::min(most, tiles * ((span + step - 1) / step));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (prompt) {
        switch (kv->dim) {
            case 64: return launch_prompt<F, 64>(P, steps, nsm, st);
            case 128: return launch_prompt<F, 128>(P, steps, nsm, st);
            default: return launch_prompt<F, 256>(P, steps, nsm, st);
        }
    }
    switch (kv->dim) {
        case 64: return nt == 1 ? launch_rows<F, 64, 1>(P, steps, nsm, st) : launch_rows<F, 64, 2>(P, steps, nsm, st);
        case 128: return nt == 1 ? launch_rows<F, 128, 1>(P, steps, nsm, st) : launch_rows<F, 128, 2>(P, steps, nsm, st);
        default: return nt == 1 ? launch_rows<F, 256, 1>(P, steps, nsm, st) : launch_rows<F, 256, 2>(P, steps, nsm, st);
    }
}

}  // namespace attend
}  // namespace tfq
