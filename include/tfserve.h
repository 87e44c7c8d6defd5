/*
 * tfserve.h -- C ABI of what serving many growing sequences adds to tfdecode.h:
 * the pages and places of a step's tokens, made on the device; rotary positions;
 * a paged key/value cache of 4 bits, and attention over it.  Same library
 * (libtfqmm), status codes, memory and stream rules as tfqmm.h: every pointer in
 * the structs and arguments is DEVICE memory owned by the caller (the structs
 * themselves are host memory, read during the call), calls are asynchronous on
 * `stream`, and nothing throws.  Everything that a step needs to know is read by
 * the kernels, so that a whole step can be one CUDA graph.
 *
 * Numbers that live in device memory cannot be checked on the host.  The kernels
 * check them, skip what does not fit, and tf_device_status returns TF_EBOUNDS.
 */
#ifndef TFSERVE_H
#define TFSERVE_H

#include "tfdecode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The pages of growing sequences.  Sequence s holds kv_len[s] tokens in the first
 * ceil(kv_len[s] / block) pages of its row of the table; the pages that no sequence
 * holds are the first n_free[0] of free_pages, a stack whose top is the last of them.
 */
typedef struct tf_kv_pages {
    int32_t *table;           /* [n_seqs][table_stride]; -1 beyond a sequence's pages */
    int64_t table_stride;
    int32_t *kv_len;          /* [n_seqs] */
    int32_t *free_pages;      /* [n_blocks] */
    int32_t *n_free;          /* [1] */
    int n_seqs;               /* 1..4096 */
    int n_blocks;             /* pages of the pool */
    int max_pages;            /* pages that a row of the table has room for; at most table_stride */
    int block;                /* tokens of a page: 16, 32, 64 or 128 */
} tf_kv_pages;

/*
 * tf_kv_plan -- one step of the pages: sequence s gets change[s] tokens (a prompt's,
 * a single one, drafts), or gives -change[s] of its last ones back (rejected
 * drafts; -kv_len[s] ends the sequence).
 *   First the pages that are given back go onto the stack, then the new ones are
 *   taken from its top, both sequence by sequence and in the order of a row (the
 *   pages given back as a whole in reverse, so that a step and the step of its
 *   negated changes leave the stack, the table and the lengths as they were).
 *   max_rows, max_len  the largest change, and length after it, that the step may have
 *   row_start [n_seqs + 1]: where each sequence's new tokens begin among the rows of
 *            the step (sequence by sequence; one that gives tokens back has none)
 *   positions [rows], slots [rows], either or both NULL: of each row its token's place in
 *            the sequence, and in the cache (page * block + the place in the page); -1
 *            for the rows behind the last token.  rows 0: neither.
 *   info     [4]: 0; how many pages there were too few; rows; the longest length.
 * A step that cannot be made is not made at all: lengths, table and stack stay as
 * they were, row_start is all 0 (a batch of no rows), positions and slots are -1, and
 *   info[0] = 1   there are too few free pages: info[1] more would do
 *   info[0] = 2   a length or change out of range, more than `rows` rows (where there are positions
 *                 or slots), or a page number outside the pool on the stack or among the pages given
 *                 back; tf_device_status returns TF_EBOUNDS.
 * (info[2] is then 0 and info[3] the longest length that stands.)
 */
int tf_kv_plan(const tf_kv_pages *pages, const int32_t *change, int rows, int max_rows, int max_len, int32_t *row_start,
               int32_t *positions, int64_t *slots, int32_t *info, void *stream);

/*
 * tf_rope -- rotary positions.  Of each of a row's `heads` heads of dim values, the
 * first `rot` are pairs (a, b) that turn by an angle of the row's position p:
 *     a' = a cos - b sin,   b' = b cos + a sin,   angle of pair i = 2 pi (p turns[i] / 2^64)
 * and the rest is copied.  Pair i is (i, i + rot / 2), or (2 i, 2 i + 1) with
 * TF_ROPE_PAIRS.  TF_ROPE_BACK turns the other way: the gradient of a turn, and its
 * inverse (times factor^2).
 *   turns    [rot / 2]: what a position turns pair i by, in 2^-64 of a full turn.
 *            Products with positions are taken modulo a turn in whole numbers, so
 *            that far positions are as exact as near ones.
 *   factor   multiplies cosines and sines (1 for none).
 *   positions [rows] int32; a row of a negative one is left as it is in `out`.
 *   x, out   rows of heads * dim values, strides in elements.  x is bf16, or fp32 with
 *            TF_IN_F32; out is fp32, or bf16 with TF_OUT_BF16 (rounded once).  out may
 *            be x itself (same type, pointer and stride), or other columns of the same
 *            rows; any other overlap is refused.
 *   dim      even, up to 1024; rot even, 2..dim.
 * Queries and keys that are columns of one product turn in one call, as heads + kv_heads heads.
 */
#define TF_ROPE_PAIRS 256
#define TF_ROPE_BACK 512
int tf_rope(const uint64_t *turns, int rot, float factor, const int32_t *positions, int rows, const void *x, int64_t x_stride,
            void *out, int64_t out_stride, int heads, int dim, int flags, void *stream);

/*
 * The 4-bit cache.  A pool of pages holds `block` consecutive tokens of one sequence
 * each; every 64 values of a token's head are 4-bit codes with a scale and a bias,
 * as the matrices of tfqmm.h have them:
 *
 *     value = scale * code + bias
 *     bias  = the largest bf16 number that is not above the smallest of the 64 values
 *     scale = the smallest bf16 number of which 15 reach from bias to the largest
 *     code  = (x - bias) / scale rounded to the nearest, even in the middle (scale 0: code 0)
 *
 * decided as if computed exactly, so that no value is off by more than half a scale.
 * Values are held within +-2^126; infinities are left out of smallest and largest and
 * held as code 15 or 0, NaN as 0, so that a bad value does not spoil the others (no
 * finite value: scale and bias 0).  A token's content depends on that token only.
 */
typedef struct tf_kv4 {
    uint8_t *k, *v;                 /* [n_blocks][kv_heads][block][dim / 2], 16-byte aligned; value 2 i in the low half of byte i */
    uint16_t *k_affine, *v_affine;  /* [n_blocks][kv_heads][block][dim / 64][2] bf16: scale, bias; 16-byte aligned */
    int n_blocks;
    int kv_heads;                   /* 1..1024 */
    int block;                      /* 16, 32, 64 or 128 */
    int dim;                        /* 64, 128 or 256 */
} tf_kv4;

/*
 * tf_kv4_append -- quantizes rows of keys and values into the slots that tf_kv_plan gave them.
 *   slots    [rows] int64, page * block + the place in the page; a row of -1 is left
 *            out, one of any other slot outside the pool too, and reported.  No slot twice.
 *   k, v     rows of kv_heads * dim values, bf16 or fp32 (TF_IN_F32), strides in elements.
 */
int tf_kv4_append(const tf_kv4 *kv, const int64_t *slots, int rows, const void *k, int64_t k_stride, const void *v,
                  int64_t v_stride, int flags, void *stream);

/*
 * tf_kv4_read -- reads the batch's rows (each sequence's last tokens) back, as
 * tf_kv_read does: fp32 (scale * code + bias, rounded once) or, with TF_OUT_BF16, that
 * rounded to bf16.  Either output may be NULL.
 */
int tf_kv4_read(const tf_kv4 *kv, const tf_kv_batch *batch, void *k_out, int64_t k_stride, void *v_out, int64_t v_stride,
                int flags, void *stream);

/*
 * tf_kv4_attend -- attention of the batch's rows over the 4-bit cache: arguments, flags,
 * masks, workspace and streams are those of tf_kv_attend.
 * Precision: scores, maxima, sums and accumulators are fp32.  q enters the tensor
 * cores as fp16 after an exact power-of-two scaling of its row (fp32 values are
 * rounded to 11 bits).  By rows codes are exact, and each p times a value's scale is
 * rounded to fp16.  By tiles (many rows) each p is, and keys and values themselves,
 * relative to the largest of 16 tokens (11 bits, down to 2^-14 of it).  Fp16 stands for
 * 11 bits down to 2^-28 of the largest p of 16 tokens times the largest value among them,
 * whichever 16 of the row's tokens these are; what is below 2^-39 of that may be left
 * out, and a token whose p is below 2^-112 of the row's largest.  out is rounded once to bf16.
 */
int tf_kv4_attend(const tf_kv4 *kv, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads, void *out,
                  int64_t out_stride, float scale, int window, int flags, void *stream);

#ifdef __cplusplus
}
#endif
#endif
