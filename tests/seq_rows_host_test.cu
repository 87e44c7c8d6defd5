// Host check of how the kernels of tfdecode.h take a sequence's numbers out of device
// memory (mlx_affine_bit_gb300/csrc/kv.h, seq_rows): whatever stands there, rows that it
// calls its own lie within the row matrices.  Host code only; nothing touches a GPU.
#include "../mlx_affine_bit_gb300/csrc/kv.h"

#include <climits>
#include <cstdio>

using namespace tfq;

int main() {
    const int32_t values[] = {INT_MIN, INT_MIN + 1, INT_MIN + 7, -1000, -2, -1, 0, 1, 2, 5, 9, 10, 11, 1000, INT_MAX - 7, INT_MAX - 1, INT_MAX};
    int bad = 0, good = 0;
    for (int rows : {1, 10, INT_MAX})
        for (int max_rows : {1, 5, 10})
            for (int32_t a : values)
                for (int32_t b : values)
                    for (int32_t len : values) {
                        if (max_rows > rows) continue;
                        const int32_t start[2] = {a, b};
                        tf_kv_batch batch{};
                        batch.n_seqs = 1;
                        batch.rows = rows;
                        batch.max_rows = max_rows;
                        batch.max_len = 9;
                        batch.row_start = start;
                        batch.kv_len = &len;
                        const SeqRows r = seq_rows(batch, 0);
                        const long long n = (long long)b - a;
                        const bool placed = a >= 0 && n >= 0 && n <= max_rows && b <= rows;
                        const bool ok = placed && len >= 0 && len <= batch.max_len;
                        if (r.ok != ok || r.placed != placed || (placed && (r.row0 != a || r.n != n || (ok && r.end != len)))) {
                            if (bad++ < 10) printf("rows %d max %d: %d .. %d len %d -> ok %d, row0 %d n %d\n", rows, max_rows, a, b, len, r.ok, r.row0, r.n);
                        }
                        good += ok;
                    }
    // Without row_start: max_rows each.
    int32_t lens[3] = {4, -1, 10};
    tf_kv_batch batch{};
    batch.n_seqs = 3, batch.rows = 6, batch.max_rows = 2, batch.max_len = 9, batch.kv_len = lens;
    for (int s = 0; s < 3; ++s) {
        const SeqRows r = seq_rows(batch, s);
        bad += r.row0 != 2 * s || r.n != 2 || !r.placed || r.ok != (s == 0);
    }
    printf(bad ? "FAIL %d\n" : "PASS %d\n", bad ? bad : good);
    return bad ? 1 : 0;
}
