// attend4.cu -- tf_kv4_attend: attention over the 4-bit paged cache (tfserve.h).  The
// host side of a call is in attend_launch.cuh, the kernels, shared with the 8-bit
// cache's, in attend_rows.cuh and attend_prompt.cuh.
#include "attend_launch.cuh"

using namespace tfq;

extern "C" int tf_kv4_attend(const tf_kv4 *kv, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads,
                             void *out, int64_t out_stride, float scale, int window, int flags, void *stream) {
    fail_message(TF_OK, "");
    int rc = attend::check_flags(flags);
    if (!rc) rc = check_kv4(kv);
    if (rc) return rc;
    attend::Params P{};
    P.kv.k = reinterpret_cast<int8_t *>(kv->k);
    P.kv.v = reinterpret_cast<int8_t *>(kv->v);
    P.kv.n_blocks = kv->n_blocks;
    P.kv.kv_heads = kv->kv_heads;
    P.kv.block = kv->block;
    P.kv.dim = kv->dim;
    P.k_affine = reinterpret_cast<const uint32_t *>(kv->k_affine);
    P.v_affine = reinterpret_cast<const uint32_t *>(kv->v_affine);
    return attend::call<4>(P, batch, q, q_stride, heads, out, out_stride, scale, window, flags, stream);
}
