// kv.h -- what the cache, attention and sampling units share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tfdecode.h"
#include "internal.h"

namespace tfq {

// Host checks of the structs (kv.cu): TF_OK or a status with the message recorded.
int check_kv(const tf_kv *kv);
int check_batch(const tf_kv *kv, const tf_kv_batch *b);

// A sequence's rows and tokens: rows row0 .. row0 + n - 1 are its tokens end - n .. end - 1.
struct SeqRows {
    int row0, n, end;
    bool ok;
};
// Reads sequence s of the batch and checks it against the extents the batch declares.
__device__ __forceinline__ SeqRows seq_rows(const tf_kv_batch &b, int s) {
    SeqRows r;
    const int next = b.row_start ? b.row_start[s + 1] : (s + 1) * b.max_rows;
    r.row0 = b.row_start ? b.row_start[s] : s * b.max_rows;
    r.n = next - r.row0;
    r.end = b.kv_len[s];
    r.ok = r.row0 >= 0 && r.n >= 0 && r.n <= b.max_rows && next <= b.rows && r.end >= 0 && r.end <= b.max_len;
    return r;
}

}  // namespace tfq
