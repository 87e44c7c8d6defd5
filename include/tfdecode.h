/*
 * tfdecode.h -- C ABI of the parts of a decode step that lie between the
 * quantized products of tfqmm.h: an 8-bit paged key/value cache, attention over
 * it, and the sampling of a token from the language-model head's logits.  Same
 * library (libtfqmm), status codes, memory and stream rules as tfqmm.h: every
 * pointer in the structs and arguments is DEVICE memory owned by the caller
 * (the structs themselves are host memory, read during the call), calls are
 * asynchronous on `stream`, and nothing throws.
 *
 * Numbers that live in device memory (lengths, row starts, page tables, slots)
 * cannot be checked on the host.  The kernels check them: a sequence whose
 * numbers do not fit the buffers that the structs declare, or a page outside the
 * pool, is skipped (attention: its tokens are not seen; a sequence skipped as a
 * whole gets zeros where its rows are known) and tf_device_status returns
 * TF_EBOUNDS.
 */
#ifndef TFDECODE_H
#define TFDECODE_H

#include "tfqmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The cache.  A pool of pages holds `block` consecutive tokens of one sequence
 * each, keys and values as 8-bit codes with one scale per page and head:
 *
 *     value[t][d] = scale * code[t][d],   scale = max |x[t][d]| * (1/127) over the page's tokens,
 *     code = x / scale rounded to nearest even   (fp32 product, division and rounding; scale 0: code 0)
 *
 * Infinities are left out of the maximum and held as +-127 (0 in a page of scale
 * 0), NaN as 0, so that a bad token does not spoil the others of its page.  A page's content depends on
 * its tokens only, not on how the calls that wrote them cut the sequence: the
 * originals of the two pages that a sequence reached last stay in an open ring,
 * and a page whose scale changes is quantized again from there.  A sequence may
 * therefore be rewound (rejected drafts) and written anew, with the same result
 * as if the rejected tokens had never been there, while the ring has the
 * originals of the page that is gone on with:
 *     - to no more than `block` tokens before the longest length that the sequence
 *       has had, however often it was rewound meanwhile (rejected tokens, too,
 *       take their places in the ring);
 *     - or to the first token of any page, which needs no originals.  The sequence
 *       then counts as begun there: its longest length is that from there on.
 * A call that goes on elsewhere is not detected: it quantizes the page's earlier
 * tokens from what stands in their places.
 */
typedef struct tf_kv {
    int8_t *k, *v;            /* [n_blocks][kv_heads][block][dim], 16-byte aligned */
    float *k_scale, *v_scale; /* [n_blocks][kv_heads] */
    void *open_k, *open_v;    /* [n_slots][kv_heads][2*block][dim] bf16 (fp32 if f32), 16-byte aligned; token
                                 position p of the sequence in a slot is at p % (2*block).  Only tf_kv_append
                                 uses these three; the other calls take NULL */
    float *open_max;          /* [n_slots][2 (k, v)][kv_heads][2*block]: max |x| of each of those tokens */
    int n_blocks, n_slots;
    int kv_heads;             /* 1..1024 */
    int block;                /* 16, 32, 64 or 128 */
    int dim;                  /* 64, 128 or 256 */
    int f32;                  /* 1: tf_kv_append's rows and the open ring are fp32; 0: bf16 */
} tf_kv;

/*
 * The rows of one call: sequence s has rows row_start[s] .. row_start[s+1]-1,
 * which stand for its last tokens: kv_len[s] counts the sequence's tokens in the
 * cache, these included.
 */
typedef struct tf_kv_batch {
    int n_seqs;
    int rows;                 /* rows of the row matrices (no row index reaches it) */
    int max_rows;             /* at least every sequence's number of rows */
    int max_len;              /* at least every kv_len; at most table_stride * block, and 2^20 */
    const int32_t *row_start; /* [n_seqs + 1], or NULL: max_rows rows each (rows = n_seqs * max_rows) */
    const int32_t *kv_len;    /* [n_seqs] */
    const int32_t *table;     /* [n_seqs][table_stride]: page of each `block` tokens */
    int64_t table_stride;
    const int32_t *slots;     /* [n_seqs] slot of each sequence's open ring, or NULL: s (tf_kv_append only) */
} tf_kv_batch;

/*
 * tf_kv_append -- quantizes new tokens into the cache.
 *   k, v     rows of kv_heads * dim values (bf16, or fp32 if kv->f32), k_stride
 *            and v_stride elements apart (at least kv_heads * dim): columns of a
 *            strided product are read in place.
 * Pages that the table gives to several sequences must not be written.
 */
int tf_kv_append(const tf_kv *kv, const tf_kv_batch *batch, const void *k, int64_t k_stride, const void *v,
                 int64_t v_stride, void *stream);

/*
 * tf_kv_read -- reads the batch's rows (each sequence's last tokens) back:
 * k_out, v_out get rows of kv_heads * dim values, fp32 (code * scale, rounded
 * once) or, with TF_OUT_BF16, bf16 (that fp32 value rounded to nearest even).
 * Either output may be NULL.
 */
int tf_kv_read(const tf_kv *kv, const tf_kv_batch *batch, void *k_out, int64_t k_stride, void *v_out,
               int64_t v_stride, int flags, void *stream);

/*
 * tf_kv_attend -- attention of the batch's rows over the cache.
 *   q        rows of heads * dim values (bf16, or fp32 with TF_IN_F32), q_stride
 *            elements apart; heads is a multiple of kv_heads, and query head h
 *            reads key/value head h / (heads / kv_heads).
 *   out      rows of heads * dim bf16, out_stride elements apart (the x of the
 *            next product):
 *                out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q . k_j)
 *            over the tokens j that the row sees; a row that sees none gets 0.
 *   flags    TF_IN_F32; TF_KV_CAUSAL: a row sees the tokens up to its own
 *            position (its place among the sequence's last tokens), otherwise
 *            all kv_len.
 *            TF_KV_BY_ROWS, TF_KV_BY_TILES: the kernel for few rows (16 at a
 *            time, any number works) or the one for prompts (256 rows at a time on
 *            the tcgen05 tensor cores), instead of the call's own choice by its
 *            sizes -- for a caller that has measured its own.
 *   window   0, or with TF_KV_CAUSAL the number of latest tokens (its own
 *            included) that a row sees (any number: from max_len on, all).
 * Precision: q enters the tensor cores as fp16 after an exact power-of-two
 * scaling of its row (bf16 values keep all their bits, fp32 values are rounded
 * to 11), codes are exact there; each p times its page's value scale is rounded
 * to fp16 (11 bits) relative to the row's largest for the second product (11 bits
 * down to 2^-29 of it, nothing below 2^-40, and of a token whose p is below 2^-112 of
 * the row's largest perhaps nothing); scores, maxima, sums and accumulators
 * are fp32 (a score of 2^20 is held to 2^-3: larger ones are told apart no better
 * than fp32 does, but lose nothing else); out is rounded once to bf16.
 * A row's bits do not change from call to call with the same arguments; between
 * calls of another batch they may, within that precision, because sequences are
 * cut between the CTAs by the whole call's tokens.
 * The first call on a (device, stream) allocates the stream's workspace for the
 * parts of split sequences: some 41 MB, enough for every later call, held at the
 * same address until exit.  It must precede any graph capture on the stream (a
 * first call inside one is refused with TF_ECUDA and leaves the capture as it is);
 * a captured graph stays valid whatever is called on the stream afterwards.
 * Calls on one stream, and replays of the graphs captured on it, share that
 * workspace: replay them on that stream, or after one another.
 */
#define TF_IN_F32 4
#define TF_KV_CAUSAL 8
#define TF_KV_BY_ROWS 64
#define TF_KV_BY_TILES 128
int tf_kv_attend(const tf_kv *kv, const tf_kv_batch *batch, const void *q, int64_t q_stride, int heads, void *out,
                 int64_t out_stride, float scale, int window, int flags, void *stream);

/*
 * tf_sample -- one token per row of logits, from given random numbers.
 *   logits   [rows][vocab] fp32 (bf16 with TF_IN_BF16), `stride` elements apart;
 *            vocab up to 2^20.  NaN counts as -inf; -inf is never drawn.
 *   u        [rows] fp32 random numbers in [0, 1).
 *   temperature, top_k, top_p, min_p   [rows] each, or NULL for 1 / off.
 *   tokens   [rows] int32; probs [rows] fp32 or NULL: the token's probability
 *            among the tokens kept.
 * With z = (logit - max) * (1 / temperature) in fp32, a token's weight is the
 * whole number w = round(exp(z) * 2^31), so that sums are exact and do not
 * depend on their order.  Tokens are ranked by logit, equal ones by index (the
 * lower first).  top_k > 0 keeps the first top_k; top_p < 1 keeps of these the
 * shortest prefix whose sum reaches top_p times theirs (at least one token);
 * min_p keeps those of at least min_p times the largest weight (min_p above 1
 * counts as 1).  The token is the first, in index order, at which the running
 * sum of the kept weights exceeds u times their sum.  A temperature that is not
 * above 0, NaN included, takes the first largest logit (probability 1); one above
 * the largest float counts as that.  top_p or min_p of NaN are off.  A row of
 * -inf gives token -1 and probability 0.
 */
#define TF_IN_BF16 16
int tf_sample(const void *logits, int rows, int vocab, int64_t stride, const float *u, const float *temperature,
              const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens, float *probs, int flags,
              void *stream);

#ifdef __cplusplus
}
#endif
#endif
