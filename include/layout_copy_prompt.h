/*
 * layout_copy_prompt.h -- C ABI of attention over whole prompts.
 *
 *   lc_prompt_attend   attention of packed sequences of different lengths over
 *                      their own keys and values
 *
 * Queries, keys and values are packed: sequence b's queries are the rows
 * starts[b] .. starts[b+1]-1 of [n_tokens, n_q_heads, head_dim], its keys and
 * values the rows k_starts[b] .. k_starts[b+1]-1 of [n_keys, n_kv_heads,
 * head_dim] (k_starts NULL: starts).  Keys are as many as the queries for a
 * whole prompt, and more for a later piece of one, whose queries are the last
 * of its tokens: query i of nq sees, of nk keys, those up to i + nk - nq.
 *
 * Conventions are those of layout_copy_cache.h: strides count elements, the
 * struct is read during the call and not retained, launches are asynchronous
 * on `stream`, every function returns an lc_status and launches nothing when
 * it refuses.  The starts live on the device and are read by the kernel: one
 * outside 0 .. n_tokens (n_keys) is moved there; where one is below the one
 * before it nothing is computed and out stays as it was.  Both record
 * LC_ERR_CACHE_INDEX in the device error word (lc_last_device_error).
 */
#ifndef LAYOUT_COPY_PROMPT_H_
#define LAYOUT_COPY_PROMPT_H_

#include "layout_copy_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One call.
 *   type       LC_CACHE_BF16 or LC_CACHE_F16, of q, k, v and out
 *   *_stride   of token and head, elements of head_dim adjacent; lse: of token, heads
 *              adjacent
 *   n_q_heads  a multiple of n_kv_heads; query head i reads key head
 *              i / (n_q_heads / n_kv_heads)
 *   causal     not 0: keys after a query are not seen
 *   window     0, or how many keys are seen of those up to a query's own place
 *              (later ones, where not causal, are all seen)
 *   scale      of the dot products, finite, and so is its product with log2 e in float32
 *   lse        NULL, or receives log(sum_j exp(scale q . k_j))
 *
 * A query with no key to see gives zeros and the lse -inf.  Rows of out and lse
 * that are no sequence's are left as they were.  out shares no element with q (but for
 * out = q itself, with its strides), k or v, nor lse with them or out, nor either with the starts.  Rows of q, k and v lie on 16-byte boundaries (head_dim and strides
 * multiples of 8), as the copies of whole tiles need.  There is no backward pass.
 *
 * Logits, maxima and sums are float32; the weights are rounded once to the
 * values' 16-bit type for the second product (relative to a running maximum, so
 * that each is off by half a step of its own size; float16 weights below 2^-25 of
 * the largest by up to 2^-36 of it), and the output once more.  Exponentials and
 * logarithms are the hardware's approximate ones, and lse is off by up to a millionth beside
 * its logits' roundings.  What unseen keys and values
 * hold never reaches an output; a row that sees a value that is infinite or NaN
 * has no finite number in that column. */
typedef struct {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *starts;    /* [n_seqs + 1] */
    const int32_t *k_starts;  /* [n_seqs + 1] or NULL */
    int64_t n_tokens, n_keys;
    int32_t type;
    int32_t n_seqs;
    int32_t n_q_heads, n_kv_heads;
    int32_t head_dim;         /* a multiple of 8 up to LC_CACHE_MAX_DIM */
    int32_t causal;
    int32_t window;
    float scale;
    int64_t q_stride[2], k_stride[2], v_stride[2], out_stride[2];
    int64_t lse_stride;
} lc_prompt;

/* Errors: LC_ERR_NULL, LC_ERR_SHAPE (heads, head_dim, negative sizes), LC_ERR_TYPE,
 * LC_ERR_BAD_STRIDE (negative; 0 for a token or head among several), LC_ERR_ALIGN,
 * LC_ERR_OVERFLOW (2^30 tokens, keys or tiles, offsets past 2^60), LC_ERR_NOT_INJECTIVE (rows of out or lse
 * meet), LC_ERR_OVERLAP, LC_ERR_CUDA.  Waits inside the kernel are bounded
 * (LC_WAIT_TIMEOUT_NS, and up to 0.4 ms more: polls sleep); one that runs out sets LC_ERR_TIMEOUT
 * in the error word, and out and lse are then not to be used. */
int lc_prompt_attend(const lc_prompt *prompt, lc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYOUT_COPY_PROMPT_H_ */
