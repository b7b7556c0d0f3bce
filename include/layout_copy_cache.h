/*
 * layout_copy_cache.h -- C ABI of the paged key-value cache operators.
 *
 * A cache is a pool of pages, each holding page_size slots of n_kv_heads
 * heads of head_dim elements, for keys and for values.  The pages are
 * described the way a TileLayout describes a tensor: by element strides, so
 * [page, head, slot, dim] and [page, slot, head, dim] pools (or any other
 * order, or a slice of a larger pool) are the same call.  A page table names
 * each sequence's pages in order: slot j of sequence b is row j % page_size
 * of page page_table[b, j / page_size].
 *
 *   lc_cache_append   writes new tokens' rows into their slots
 *   lc_cache_attend   attention of one new token a sequence over its slots
 *   lc_cache_attend_tree  attention of a tree of drafted tokens a sequence
 *   lc_cache_accept   keeps the accepted path of the drafts, moved together
 *                     behind the tokens before them
 *   lc_cache_evict    keeps the slots of the largest accumulated weight and
 *                     the newest ones, moved together at the front
 *   lc_cache_reserve  page tables from lengths and a stack of free pages, and
 *                     the slots of packed tokens
 *   lc_cache_append_packed  writes packed tokens' rows into such slots
 *
 * Conventions are those of layout_copy.h: strides count elements, structs
 * are read during the call and not retained, pointers are device addresses
 * owned by the caller, launches are asynchronous on `stream`, every function
 * returns an lc_status and launches nothing when it refuses.  Lengths, page
 * tables and masks live on the device and are read by the kernels: a length
 * outside 0 .. pages_per_seq * page_size is clamped to it, a page id
 * outside 0 .. n_pages-1 makes its slots unseen (attend) or their rows
 * dropped (append, evict), and both record LC_ERR_CACHE_INDEX in the device
 * error word (lc_last_device_error).
 */
#ifndef LAYOUT_COPY_CACHE_H_
#define LAYOUT_COPY_CACHE_H_

#include "layout_copy.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head_dim. */
#define LC_CACHE_MAX_DIM 256

typedef enum {
    LC_CACHE_BF16 = 0,
    LC_CACHE_F16 = 1,
    /* E4M3 codes with one float32 scale a slot and head: the value is
     * code * scale.  lc_cache_append marks a row that holds an infinity or
     * NaN by a scale of NaN. */
    LC_CACHE_E4M3 = 2
} lc_cache_type;

typedef struct {
    void *k, *v;                 /* pools, aligned to their element */
    float *k_scale, *v_scale;    /* E4M3 only, else NULL */
    const int32_t *page_table;   /* [n_seqs, pages_per_seq], rows table_stride apart */
    int64_t table_stride;
    int64_t n_pages;             /* of the pools; at least 1 where sequences have slots */
    int32_t type;                /* lc_cache_type */
    int32_t n_seqs;
    int32_t n_kv_heads;
    int32_t page_size;
    int32_t head_dim;            /* 1 .. LC_CACHE_MAX_DIM, elements adjacent */
    int32_t pages_per_seq;
    int64_t k_stride[3], v_stride[3];             /* of page, head, slot; >= 0 */
    int64_t k_scale_stride[3], v_scale_stride[3]; /* the same, of the scales */
} lc_paged_cache;

/* Writes new tokens: for t < counts[b] (n_new where counts is NULL), the rows
 * k_new[b, t, h, :] and v_new[b, t, h, :] go to slot lengths[b] + t of
 * sequence b, and new_lengths[b] = lengths[b] + counts[b].  Tokens past the
 * sequence's capacity are dropped (LC_ERR_CACHE_INDEX in the error word) and
 * not counted; so are negative counts, and counts above n_new.
 *   type      LC_CACHE_BF16 or LC_CACHE_F16, of k_new and v_new: the cache's
 *             own, or either for an E4M3 cache, whose rows are quantised:
 *             scale = max(max |x| / 448, 2^-126) in float32, code = x / scale
 *             rounded to nearest even; a row with an infinity or NaN gets the
 *             scale NaN
 *   *_stride  of sequence, token, head
 *   new_lengths  shares no element with lengths or counts; where n_new is 0 it
 *             may be either's own buffer
 * Errors: LC_ERR_NULL, LC_ERR_SHAPE, LC_ERR_TYPE, LC_ERR_BAD_STRIDE,
 * LC_ERR_ALIGN, LC_ERR_OVERFLOW, LC_ERR_NOT_INJECTIVE, LC_ERR_OVERLAP
 * (new_lengths meets lengths or counts). */
int lc_cache_append(const lc_paged_cache *cache, const void *k_new, const void *v_new, int32_t type,
                    const int64_t k_stride[3], const int64_t v_stride[3], int32_t n_new, const int32_t *counts,
                    const int32_t *lengths, int32_t *new_lengths, lc_stream_t stream);

/* One attention call: n_q_heads query heads of one token a sequence, query
 * head i reading key head i / (n_q_heads / n_kv_heads).
 *   type       of q and out: the cache's own; LC_CACHE_BF16 for an E4M3 cache
 *   *_stride   of sequence and head (lse: of sequence, heads adjacent)
 *   out        may be q's own buffer with q's strides; else it shares no element
 *              with q
 *   mask       NULL, or one byte a slot ([n_seqs, capacity], rows mask_stride
 *              apart): slots of a zero byte are not seen
 *   window     0, or the number of newest slots that are seen
 *   scale      of the dot products
 *   lse        NULL, or receives log(sum_j exp(scale q . k_j)), -inf where no
 *              slot is seen (out is zero there)
 *   scores     NULL, or [n_seqs, n_kv_heads, capacity]: each seen slot's weight,
 *              summed over the query heads of its key head, is added to it
 *   workspace  at least lc_cache_attend_workspace(...) bytes, 256-byte aligned;
 *              calls that may overlap need one each.  Nothing is kept in it
 *              between calls.
 *
 * Logits, maxima and sums are float32, and the output is rounded once.  The
 * weights of a bfloat16 or float16 cache are multiplied with its values as sums
 * of two numbers of that type (within 2^-16 or 2^-22 of the weight); those of an
 * E4M3 cache as one float16 number (2^-11), and its queries as float16, scaled by
 * a power of two a head (elements below 2^-14 of the largest are off by up to
 * 2^-25 of it).  Exponentials and logarithms are the hardware's approximate ones.
 *
 * Workspace and kernels are chosen by the capacity, pages_per_seq * page_size,
 * not by the lengths: with scores the workspace takes 4 bytes a query head and
 * slot of it.  A descriptor of the table's first columns (and a mask and scores
 * of as many slots) serves sequences that are known to be shorter. */
typedef struct {
    const void *q;
    void *out;
    int32_t type;
    int32_t n_q_heads;
    int64_t q_stride[2], out_stride[2];
    const int32_t *lengths;
    const uint8_t *mask;
    int64_t mask_stride;
    int32_t window;
    float scale;
    float *lse;
    int64_t lse_stride;
    float *scores;
    int64_t scores_stride[2];
    void *workspace;
    int64_t workspace_bytes;
} lc_cache_query;

/* Bytes of workspace of lc_cache_attend, or -1 for arguments that it refuses. */
int64_t lc_cache_attend_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t with_scores);

/* Errors: LC_ERR_NULL, LC_ERR_SHAPE (n_q_heads no multiple of n_kv_heads,
 * negative window, sizes), LC_ERR_TYPE, LC_ERR_BAD_STRIDE, LC_ERR_ALIGN,
 * LC_ERR_OVERFLOW, LC_ERR_NOT_INJECTIVE, LC_ERR_OVERLAP (out meets q),
 * LC_ERR_WORKSPACE. */
int lc_cache_attend(const lc_paged_cache *cache, const lc_cache_query *query, lc_stream_t stream);

/* Most drafted tokens of a sequence in one call. */
#define LC_CACHE_MAX_DRAFTS 64

/* Attention of a tree of drafted tokens a sequence.  The drafts' rows are in the
 * cache already, as lc_cache_append leaves them: draft t of counts[b] sits in slot
 * lengths[b] - counts[b] + t.  It sees the slots before the drafts, its ancestors'
 * and its own.  (A chain, parents[t] = t - 1, is causal attention of several new
 * tokens.)
 *   parents    [n_seqs, n_drafts], rows parents_stride apart: a draft's parent, an
 *              earlier draft, or -1 where it follows the token before the drafts; any
 *              other value counts as -1 and records LC_ERR_CACHE_INDEX
 *   counts     [n_seqs], or NULL: n_drafts each, as far as the length goes; one outside 0 .. min(n_drafts,
 *              length) is clamped, with LC_ERR_CACHE_INDEX
 *   type       of q and out: the cache's own; LC_CACHE_BF16 for an E4M3 cache
 *   *_stride   of sequence, draft, head (lse: of sequence, draft, heads adjacent)
 *   out        shares no address range with q; neither out nor lse shares an element with the
 *              other, q, lengths, counts or parents.  (That they lie apart from the
 *              cache and the workspace is the caller's to see to.)
 *   window     0, or how many tokens are seen, a draft's own and its nearest ancestors
 *              first, then the newest before the drafts
 *   scale      of the dot products, finite, and so is its product with log2 e in float32
 *   lse        NULL, or receives log(sum_j exp(scale q . k_j))
 *   workspace  at least lc_cache_attend_tree_workspace(...) bytes, as lc_cache_attend's
 *
 * Rows of out and lse of drafts past a sequence's count are left as they were.
 * Roundings are lc_cache_attend's: float32 sums, weights of a bfloat16 or float16
 * cache as two numbers of its type, those of an E4M3 cache as one float16
 * number, its queries as float16 scaled by a power of two a row.  A row that
 * sees a value that is infinite or NaN has no finite number in that column. */
typedef struct {
    const void *q;
    void *out;
    int32_t type;
    int32_t n_q_heads;
    int32_t n_drafts;
    int32_t window;
    int64_t q_stride[3], out_stride[3];
    const int32_t *lengths, *counts, *parents;
    int64_t parents_stride;
    float scale;
    float *lse;
    int64_t lse_stride[2];
    void *workspace;
    int64_t workspace_bytes;
} lc_cache_tree;

/* Bytes of workspace of lc_cache_attend_tree, or -1 for arguments that it refuses. */
int64_t lc_cache_attend_tree_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t n_drafts);

/* Errors: as lc_cache_attend; LC_ERR_SHAPE also for n_drafts outside 0 ..
 * LC_CACHE_MAX_DRAFTS.  Waits inside the kernel are bounded (LC_WAIT_TIMEOUT_NS, and up to 0.4
 * ms more: polls sleep); one that runs out sets LC_ERR_TIMEOUT in the error word, and out and lse
 * are then not to be used. */
int lc_cache_attend_tree(const lc_paged_cache *cache, const lc_cache_tree *tree, lc_stream_t stream);

/* Keeps the drafts of a path and lets the others go: the i-th draft of the path
 * moves from slot before + path[b, i] to slot before + i of its sequence, before =
 * lengths[b] - counts[b], in both pools and their scales, and new_lengths[b] = before
 * + the path's length.  Slots past that hold what they held or what moved.
 *   path       [n_seqs, n_path], rows path_stride apart, n_path <= LC_CACHE_MAX_DRAFTS: drafts in rising
 *              order, ended by -1; one that does not rise or is no draft of the
 *              sequence ends the path too, and records LC_ERR_CACHE_INDEX
 *   counts     [n_seqs], the drafts a sequence has, or NULL: n_path each, as far as
 *              the length goes; clamped as in lc_cache_attend_tree
 *   new_lengths  [n_seqs], sharing no element with lengths, counts, path or the page table
 * The pages that hold the drafts must not be shared with another sequence.
 * Errors: as lc_cache_append. */
int lc_cache_accept(const lc_paged_cache *cache, const int32_t *lengths, const int32_t *counts, const int32_t *path,
                    int64_t path_stride, int32_t n_path, int32_t *new_lengths, lc_stream_t stream);

/* Writes packed tokens: row t of k_new and v_new, [n_tokens, n_kv_heads,
 * head_dim], goes to slot slots[t] of the pool, page * page_size + row, whose pages lc_cache_reserve
 * gives; -1 drops it, any other slot outside the pool does too, with LC_ERR_CACHE_INDEX. No two
 * tokens have one slot.  *_stride: of token and head.  The cache's page table
 * is not read.  Else as lc_cache_append. */
int lc_cache_append_packed(const lc_paged_cache *cache, const void *k_new, const void *v_new, int32_t type,
                           const int64_t k_stride[2], const int64_t v_stride[2], int32_t n_tokens, const int64_t *slots,
                           lc_stream_t stream);

/* Most sequences of one lc_cache_reserve. */
#define LC_CACHE_MAX_RESERVED 4096

/* Makes a page table hold the pages of lengths[b] + counts[b] tokens a sequence, and
 * tells where each of the new tokens goes.
 *   page_table   [n_seqs, pages_per_seq]: a sequence's pages, then -1
 *   new_table    the same afterwards; may be page_table itself (with its stride)
 *   free, n_free a stack of free pages of free_size entries and how many it has.  Pages past
 *                those that a sequence wants (one that has ended: length 0, count 0) go on
 *                top first, in the sequences' order; what is missing then comes off the top, in the
 *                same order
 *   new_n_free   how many the stack has afterwards
 *   new_lengths  lengths + counts of the sequences that are served, lengths of the others
 *   starts       [n_seqs + 1]: where each sequence's tokens begin among the packed ones
 *   slots, positions, seqs   [max_tokens], of every packed token: page * page_size +
 *                row, place in its sequence, sequence; -1 past the last
 * A sequence is not served, keeps the pages that it has (those past lengths + counts
 * have gone on the stack) and gets no tokens where its
 * pages do not last (those behind it that need pages are not served either), its
 * tokens pass pages_per_seq (then no page goes), or max_tokens ends; that records
 * LC_ERR_CACHE_INDEX, as a negative length or count (taken as 0) does.  All outputs and the stack lie
 * apart from one another and from what is read.
 * The stack's entries past its top and below free_size may change. */
typedef struct {
    const int32_t *page_table;
    int32_t *new_table;
    int64_t table_stride, new_table_stride;
    const int32_t *lengths, *counts;
    int32_t *free;
    const int32_t *n_free;
    int32_t *new_n_free, *new_lengths, *starts;
    int64_t *slots;
    int32_t *positions, *seqs;
    int64_t free_size;
    int32_t n_seqs, pages_per_seq, page_size, max_tokens;
} lc_cache_reservation;

/* Errors: LC_ERR_NULL, LC_ERR_SHAPE (sizes; more than LC_CACHE_MAX_RESERVED sequences),
 * LC_ERR_BAD_STRIDE, LC_ERR_ALIGN, LC_ERR_OVERFLOW, LC_ERR_NOT_INJECTIVE, LC_ERR_OVERLAP, LC_ERR_CUDA. */
int lc_cache_reserve(const lc_cache_reservation *reservation, lc_stream_t stream);

/* One eviction.  A sequence of n = lengths[b] <= budget slots keeps them all.
 * A longer one keeps, per key head, its `recent` newest slots and, of the
 * others, the budget - recent with the largest score (equal scores: the
 * lowest slots; NaN counts as the lowest score, -0 as 0).  The kept rows move to slots 0 ..
 * budget-1 in their order; rows past them keep what they held.  The pages
 * named by a sequence's table must not be shared with another sequence.
 *   scores      [n_seqs, n_kv_heads, capacity], read only
 *   kept        [n_seqs, n_kv_heads, budget] receives the old slot of every
 *               kept one, -1 past them
 *   new_scores  like scores, sharing no element with them: the kept slots'
 *               scores, then zeros
 *   new_lengths [n_seqs], sharing no element with lengths: min(n, budget)
 *   workspace   at least lc_cache_evict_workspace(...) bytes, 256-byte
 *               aligned, as lc_cache_attend's; may be NULL where that is 0 */
typedef struct {
    const int32_t *lengths;
    const float *scores;
    int64_t scores_stride[2];
    int32_t budget;
    int32_t recent;
    int32_t *kept;
    int64_t kept_stride[2];
    float *new_scores;
    int64_t new_scores_stride[2];
    int32_t *new_lengths;
    void *workspace;
    int64_t workspace_bytes;
} lc_cache_eviction;

/* Bytes of workspace of lc_cache_evict on this cache (0 where small sequences
 * are selected and moved in one launch), or -1 for arguments that it refuses. */
int64_t lc_cache_evict_workspace(const lc_paged_cache *cache, int32_t budget);

/* Errors: LC_ERR_NULL, LC_ERR_SHAPE (budget < 1, recent outside 0 .. budget,
 * sizes), LC_ERR_TYPE, LC_ERR_BAD_STRIDE, LC_ERR_ALIGN, LC_ERR_OVERFLOW,
 * LC_ERR_NOT_INJECTIVE, LC_ERR_WORKSPACE, LC_ERR_OVERLAP (new_scores or
 * new_lengths meets the old ones).  The move's waits for one another's reads
 * are bounded (LC_WAIT_TIMEOUT_NS).  One that runs out sets LC_ERR_TIMEOUT in
 * the error word and leaves the 32 slots that it was for as they were, in every
 * pool; all others hold their kept rows, and kept, new_scores and new_lengths
 * are written as ever.  That key head's rows are then to be given up. */
int lc_cache_evict(const lc_paged_cache *cache, const lc_cache_eviction *eviction, lc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYOUT_COPY_CACHE_H_ */
