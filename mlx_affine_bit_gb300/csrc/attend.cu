// attend.cu -- tf_kv_attend: attention over the 8-bit paged cache (tfdecode.h), and
// the per-(device, stream) workspace of both caches' attention, for the sums of
// tokens that several CTAs share.  The host side of a call is in attend_launch.cuh,
// the kernels are in attend_rows.cuh and attend_prompt.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include "attend_launch.cuh"

using namespace tfq;

namespace {

// Parts of split sequences and their arrival counters (zero between launches), one pair for each (device, stream).
// Allocated once, for the largest launch of either kernel: captured graphs keep these addresses.
using Ws = attend::Workspace;
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

}  // namespace

int tfq::attend::workspace(cudaStream_t st, int nsm, Ws *out) {
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

extern "C" int tf_kv_attend(const tf_kv *kv, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads,
                            void *out, int64_t out_stride, float scale, int window, int flags, void *stream) {
    fail_message(TF_OK, "");
    int rc = attend::check_flags(flags);
    if (!rc) rc = check_kv(kv);
    if (rc) return rc;
    attend::Params P{};
    P.kv = *kv;
    return attend::call<8>(P, batch, q, q_stride, heads, out, out_stride, scale, window, flags, stream);
}
