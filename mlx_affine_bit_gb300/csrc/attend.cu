// attend.cu -- tf_kv_attend: attention over the 8-bit paged cache (tfdecode.h).
// Host side: checks, the choice of the kernel, the per-(device, stream) workspace
// for the sums of tokens that several CTAs share; the kernels are in
// attend_rows.cuh and attend_prompt.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include "attend_prompt.cuh"
#include "attend_rows.cuh"
#include "kv.h"

using namespace tfq;

namespace {

// Parts of split sequences and their arrival counters (zero between launches), one pair for each (device, stream).
// Allocated once, for the largest launch of either kernel: captured graphs keep these addresses.
struct Ws {
    float *part = nullptr;
    int *count = nullptr;
};
std::mutex g_mu;
std::map<std::pair<int, cudaStream_t>, Ws> g_ws;

// Floats that a launch of `ctas` CTAs on tiles of `rows` rows needs: two parts a CTA, each of outputs and row sums.
constexpr size_t part_floats(size_t ctas, int rows, int d) { return ctas * 2 * rows * (d + 4); }
size_t most_floats(int nsm) {
    size_t most = 0;
    for (int d : {64, 128, 256})
        most = std::max({most, part_floats(attend::MAX_PARTS, 16, d), part_floats(std::min(nsm, attend::MAX_PARTS), 128 * attend::p_tiles(d), d)});
    return most;
}

int workspace(cudaStream_t st, int nsm, Ws *out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lk(g_mu);
    Ws &w = g_ws[{dev, st}];
    if (!w.count) {
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        e = cudaStreamIsCapturing(st, &capture);
        if (e != cudaSuccess) return cuda_error(e, "cudaStreamIsCapturing");
        if (capture != cudaStreamCaptureStatusNone)
            return fail_message(TF_ECUDA, "the first attention call on a stream allocates its workspace and must precede a capture");
        if (!w.part) {
            e = cudaMalloc(&w.part, most_floats(nsm) * sizeof(float));
            if (e != cudaSuccess) return cuda_error(e, "cudaMalloc(attention parts)");
        }
        int *count = nullptr;
        e = cudaMalloc(&count, attend::MAX_PARTS * sizeof(int));
        if (e != cudaSuccess) return cuda_error(e, "cudaMalloc(attention counters)");
        e = cudaMemsetAsync(count, 0, attend::MAX_PARTS * sizeof(int), st);
        if (e != cudaSuccess) {
            cudaFree(count);
            return cuda_error(e, "cudaMemsetAsync(attention counters)");
        }
        w.count = count;
    }
    *out = w;
    return TF_OK;
}

// CTAs of a rows kernel that an SM holds at once (looked up once a device, with its shared-memory limit raised).
template <int D, int NT>
cudaError_t resident(int *out) {
    static int n[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int v = __atomic_load_n(&n[dev], __ATOMIC_ACQUIRE);
    if (!v) {
        auto k = attend::rows_kernel<D, NT>;
        constexpr int smem = attend::smem_bytes(D, NT);
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, k, attend::THREADS, smem);
        if (e != cudaSuccess) return e;
        if (v < 1) return cudaErrorLaunchOutOfResources;
        __atomic_store_n(&n[dev], v, __ATOMIC_RELEASE);
    }
    *out = v;
    return cudaSuccess;
}

// The launch: as many CTAs as are resident at once, or one a step where there are fewer.
template <int D, int NT>
int launch_rows(attend::Params &P, long long steps, int nsm, cudaStream_t st) {
    int per_sm = 0;
    cudaError_t e = resident<D, NT>(&per_sm);
    if (e != cudaSuccess) return cuda_error(e, "kv_attend set-up");
    const long long grid = std::min({steps, (long long)nsm * per_sm, (long long)attend::MAX_PARTS});
    Ws w;
    const int rc = workspace(st, nsm, &w);
    if (rc) return rc;
    P.part = w.part;
    P.count = w.count;
    attend::rows_kernel<D, NT><<<(unsigned)grid, attend::THREADS, attend::smem_bytes(D, NT), st>>>(P);
    e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_attend launch");
}

// The same for the prompt kernel: one CTA an SM.
template <int D>
int launch_prompt(attend::Params &P, long long steps, int nsm, cudaStream_t st) {
    constexpr int smem = attend::p_smem(D);
    static unsigned attr_set = 0;   // one bit per device: shared-memory limit raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    const unsigned bit = 1u << (dev & 31);
    if (!(__atomic_load_n(&attr_set, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(attend::prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_error(e, "kv_attend set-up");
        __atomic_fetch_or(&attr_set, bit, __ATOMIC_RELEASE);
    }
    const long long grid = std::min({steps, (long long)nsm, (long long)attend::MAX_PARTS});
    Ws w;
    const int rc = workspace(st, nsm, &w);
    if (rc) return rc;
    P.part = w.part;
    P.count = w.count;
    attend::prompt_kernel<D><<<(unsigned)grid, attend::P_THREADS, smem, st>>>(P);
    e = cudaGetLastError();
    return e == cudaSuccess ? TF_OK : cuda_error(e, "kv_attend launch");
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" int tf_kv_attend(const tf_kv *kv, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads,
                            void *out, int64_t out_stride, float scale, int window, int flags, void *stream) {
    fail_message(TF_OK, "");
    if (flags & ~(TF_IN_F32 | TF_KV_CAUSAL | TF_KV_BY_ROWS | TF_KV_BY_TILES))
        return fail_message(TF_EINVAL_FLAGS, "unknown attention flags");
    if ((flags & TF_KV_BY_ROWS) && (flags & TF_KV_BY_TILES))
        return fail_message(TF_EINVAL_FLAGS, "TF_KV_BY_ROWS and TF_KV_BY_TILES exclude each other");
    int rc = check_kv(kv);
    if (!rc) rc = check_batch(kv, batch);
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

    const long long pool_rows = (long long)kv->n_blocks * kv->kv_heads * kv->block * kv->dim / 128;
    if (pool_rows > 0x7FFFFFFF) return fail_message(TF_EINVAL_SIZE, "a pool of more than 2^38 bytes");
    attend::Params P{};
    const int box_rows = std::min(kv->block, 16 * attend::tiles_of(kv->dim)) * kv->dim / 128;
    rc = tensor_map_rows128(&P.tm_k, kv->k, pool_rows, box_rows);
    if (!rc) rc = tensor_map_rows128(&P.tm_v, kv->v, pool_rows, box_rows);
    if (rc) return rc;
    P.kv = *kv;
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
    // 334 us (by rows 272), where a call for the chunk and one for the others take 70 and 74.
    bool prompt = (flags & TF_KV_BY_TILES) != 0;
    if (max_group_rows > 16 && !(flags & (TF_KV_BY_ROWS | TF_KV_BY_TILES))) {
        const double blocks = (double)batch->n_seqs * kv->kv_heads * (double)((span + 127) / 128);
        const int pair = 128 * attend::p_tiles(kv->dim);
        const double pairs = (double)((max_group_rows + pair - 1) / pair), items = (double)batch->n_seqs * kv->kv_heads * pairs;
        const double ctas = std::min((double)nsm, items * attend::MAX_SHARE);
        const double t_rows = 12e3 + 6.5 * blocks * (double)((max_group_rows + 15) / 16) * kv->dim / 128;
        const double t_prompt = 45e3 + 2900.0 * blocks * pairs / ctas;
        prompt = t_prompt < t_rows;
    }
    // Rows kernel: tiles of 8 rows where no sequence has more a head (4 rows of 48 x 4000 tokens, 8 heads of 128: 71 us,
    // 77 in a tile of 16; 8 rows of 16 x 4000, 2 heads of 256: 28 and 33), else of 16.
    const int nt = max_group_rows <= 8 ? 1 : 2, tile_rows = prompt ? 128 * attend::p_tiles(kv->dim) : 8 * nt;
    const long long tiles = (max_group_rows + tile_rows - 1) / tile_rows;
    const int step = prompt ? attend::KEYS : attend::step_of(kv->dim);
    const long long most = std::max(1LL, (1LL << 40) / (batch->n_seqs * (long long)kv->kv_heads));
    const long long steps = batch->n_seqs * (long long)kv->kv_heads * std::min(most, tiles * ((span + step - 1) / step));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (prompt) {
        switch (kv->dim) {
            case 64: return launch_prompt<64>(P, steps, nsm, st);
            case 128: return launch_prompt<128>(P, steps, nsm, st);
            default: return launch_prompt<256>(P, steps, nsm, st);
        }
    }
    switch (kv->dim) {
        case 64: return nt == 1 ? launch_rows<64, 1>(P, steps, nsm, st) : launch_rows<64, 2>(P, steps, nsm, st);
        case 128: return nt == 1 ? launch_rows<128, 1>(P, steps, nsm, st) : launch_rows<128, 2>(P, steps, nsm, st);
        default: return nt == 1 ? launch_rows<256, 1>(P, steps, nsm, st) : launch_rows<256, 2>(P, steps, nsm, st);
    }
}
