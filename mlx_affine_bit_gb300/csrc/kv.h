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
    bool placed;            // the rows lie within the row matrices, and are no more than max_rows
    bool ok;                // and its length is one that the batch declares
};
// Reads sequence s of the batch and checks it against the extents the batch declares.  (Any numbers may stand
// there: the starts are compared before their difference is taken, which could wrap around.)
__host__ __device__ __forceinline__ SeqRows seq_rows(const tf_kv_batch &b, int s) {
    SeqRows r;
    const int next = b.row_start ? b.row_start[s + 1] : (s + 1) * b.max_rows;
    r.row0 = b.row_start ? b.row_start[s] : s * b.max_rows;
    r.n = (int)((unsigned)next - (unsigned)r.row0);
    r.end = b.kv_len[s];
    r.placed = r.row0 >= 0 && next >= r.row0 && r.n <= b.max_rows && next <= b.rows;
    r.ok = r.placed && r.end >= 0 && r.end <= b.max_len;
    return r;
}

}  // namespace tfq
