// Attention of drafted trees over the cache: the checks, the workspace and the C
// entry points (lc_cache_attend_tree; the kernels are tree_attend.cuh).
#include <cmath>

#include "tensor_map.h"
#include "tree_attend.cuh"

namespace lc {

int launch_tree_bf16(const TreeArgs &a, cudaStream_t cs);
int launch_tree_f16(const TreeArgs &a, cudaStream_t cs);
int launch_tree_e4m3(const TreeArgs &a, cudaStream_t cs);

namespace {

// Offsets of the parts' maxima and sums, of the runs' cuts, and the end.
struct TreeSpace {
    int64_t ml, split, end;
    explicit TreeSpace(const CacheArgs &c) {
        const int64_t rows = int64_t(2) * kTrMostRuns * kTrRows;
        ml = rows * ((c.dim + 63) / 64 * 64 * 4);
        split = ml + rows * 8;
        end = split + kTrMostRuns * 16;
    }
};

// Pages x heads x slots x head_dim, in boxes of `box` slots of one head (16-bit elements: 64 columns of them).
bool map_pool(CUtensorMap *m, const lc_paged_cache &c, const void *p, const int64_t *st, int box) {
    EncodeTiledFn encode = encode_tiled();
    if (!encode) return false;
    const bool q8 = c.type == LC_CACHE_E4M3;
    const int64_t eb = q8 ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.n_kv_heads), static_cast<cuuint64_t>(c.n_pages)};
    const int64_t own = (c.head_dim * eb + 15) / 16 * 16;  // of a mode of one element, which has no stride
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.page_size > 1 ? st[2] * eb : own),
                                   static_cast<cuuint64_t>(c.n_kv_heads > 1 ? st[1] * eb : own),
                                   static_cast<cuuint64_t>(c.n_pages > 1 ? st[0] * eb : own)};
    const cuuint32_t shape[4] = {static_cast<cuuint32_t>(q8 ? c.head_dim : 64), static_cast<cuuint32_t>(box), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = q8                          ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : c.type == LC_CACHE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(m, type, 4, const_cast<void *>(p), dims, strides, shape, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int most_blocks(int64_t n_drafts, int group) { return static_cast<int>((n_drafts * group + kTrRows - 1) / kTrRows); }

}  // namespace

}  // namespace lc

extern "C" int64_t lc_cache_attend_tree_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t n_drafts) {
    using namespace lc;
    CacheArgs c;
    if (check_cache(cache, false, &c) || n_q_heads < 1 || n_q_heads % c.heads || n_drafts < 0 ||
        n_drafts > LC_CACHE_MAX_DRAFTS)
        return -1;
    return TreeSpace(c).end;
}

extern "C" int lc_cache_attend_tree(const lc_paged_cache *cache, const lc_cache_tree *q, lc_stream_t stream) {
    using namespace lc;
    TreeArgs a{};
    int st = check_cache(cache, false, &a.c);
    if (st) return st;
    if (!q) return LC_ERR_NULL;
    if (q->n_q_heads < 1 || q->n_q_heads % cache->n_kv_heads || q->window < 0 || q->n_drafts < 0 ||
        q->n_drafts > LC_CACHE_MAX_DRAFTS || !std::isfinite(q->scale * kLog2e))
        return LC_ERR_SHAPE;
    if (q->type != (cache->type == LC_CACHE_E4M3 ? LC_CACHE_BF16 : cache->type)) return LC_ERR_TYPE;
    if (cache->n_seqs == 0 || q->n_drafts == 0) return LC_OK;
    if (!q->q || !q->out || !q->lengths || !q->parents) return LC_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(q->q) | reinterpret_cast<uintptr_t>(q->out)) % 2 ||
        (reinterpret_cast<uintptr_t>(q->lengths) | reinterpret_cast<uintptr_t>(q->counts) |
         reinterpret_cast<uintptr_t>(q->parents) | reinterpret_cast<uintptr_t>(q->lse)) % 4)
        return LC_ERR_ALIGN;
    const int64_t ext[3] = {cache->n_seqs, q->n_drafts, q->n_q_heads};
    st = check_reach(3, ext, q->q_stride, cache->head_dim);
    if (!st) st = check_reach(3, ext, q->out_stride, cache->head_dim);
    if (!st) st = check_reach(1, ext, &q->parents_stride, q->n_drafts);
    if (!st && q->lse) st = check_reach(2, ext, q->lse_stride, q->n_q_heads);
    if (st) return st;
    if (!rows_apart(3, ext, q->out_stride, cache->head_dim) || (q->lse && !rows_apart(2, ext, q->lse_stride, q->n_q_heads)))
        return LC_ERR_NOT_INJECTIVE;
    // parts of q's rows are read while others' output is written: out lies apart from them, range from range
    int64_t q_top = 0, o_top = 0;
    for (int i = 0; i < 3; ++i) {
        q_top += (ext[i] - 1) * q->q_stride[i];
        o_top += (ext[i] - 1) * q->out_stride[i];
    }
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q->q), o0 = reinterpret_cast<uintptr_t>(q->out);
    if (q0 < o0 + 2 * (o_top + cache->head_dim) && o0 < q0 + 2 * (q_top + cache->head_dim)) return LC_ERR_OVERLAP;
    const Span out = span_of(q->out, ext[0], q->out_stride[0], cache->head_dim, 2, ext[1], q->out_stride[1], ext[2], q->out_stride[2]);
    const Span lse = span_of(q->lse, ext[0], q->lse_stride[0], ext[2], 4, ext[1], q->lse_stride[1]);
    const Span read[] = {span_of(q->lengths, 1, 0, ext[0], 4), span_of(q->counts, 1, 0, ext[0], 4),
                         span_of(q->parents, ext[0], q->parents_stride, ext[1], 4)};
    if (may_meet(lse, out) || may_meet(lse, span_of(q->q, ext[0], q->q_stride[0], cache->head_dim, 2, ext[1], q->q_stride[1], ext[2], q->q_stride[2])))
        return LC_ERR_OVERLAP;
    for (const Span &x : read)
        if (may_meet(out, x) || may_meet(lse, x)) return LC_ERR_OVERLAP;
    a.group = q->n_q_heads / cache->n_kv_heads;
    if (int64_t(q->n_drafts) * a.group > 1 << 24) return LC_ERR_OVERFLOW;
    a.most_blocks = most_blocks(q->n_drafts, a.group);
    const int64_t heads = int64_t(cache->n_seqs) * cache->n_kv_heads;
    const int keys = a.c.dim <= 128 ? 128 : 64;
    if (heads * a.most_blocks > 0x7fffffff / (a.c.cap / keys + 2)) return LC_ERR_OVERFLOW;  // (steps are counted in 32 bits)
    const TreeSpace space(a.c);
    if (!q->workspace) return LC_ERR_NULL;
    if (space.end > q->workspace_bytes) return LC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(q->workspace) % 256) return LC_ERR_ALIGN;
    if (a.c.cap == 0) return LC_OK;  // no slots: no drafts
    a.q = static_cast<const uint16_t *>(q->q);
    a.out = static_cast<uint16_t *>(q->out);
    a.lengths = q->lengths;
    a.counts = q->counts;
    a.parents = q->parents;
    a.lse = q->lse;
    for (int i = 0; i < 3; ++i) {
        a.qst[i] = q->q_stride[i];
        a.ost[i] = q->out_stride[i];
    }
    for (int i = 0; i < 2; ++i) a.lst[i] = q->lse_stride[i];
    a.parents_stride = q->parents_stride;
    a.drafts = q->n_drafts;
    a.q_heads = q->n_q_heads;
    a.group_div = make_fastdiv(static_cast<uint32_t>(a.group));
    a.window = q->window;
    // a scale of 0 is the smallest number there is, under which all logits are too small to tell, so that unseen slots' -infinity stays what it is
    a.scale2 = std::max(std::fabs(q->scale) * kLog2e, 0x1p-149f);
    a.negative = q->scale < 0.f;
    // (nor is it with what a row of q was divided by: a product of 2^-126 or more is never 0)
    a.q_least = std::max(-126, -126 - std::ilogb(a.scale2));
    const int eb = cache_elem_bytes(cache->type);
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    a.vec = a.c.dim * eb % 16 == 0 && rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 16) &&
            rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 16);
    a.q_vec = a.c.dim % 8 == 0 && rows_aligned(q->q, 3, ext, q->q_stride, 2, 16);
    a.out_vec = rows_aligned(q->out, 3, ext, q->out_stride, 2, 16);
    a.part = static_cast<float *>(q->workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(q->workspace) + space.ml);
    a.split = reinterpret_cast<int4 *>(static_cast<uint8_t *>(q->workspace) + space.split);
    a.limit_ns = wait_limit_ns();
    a.piece_div = make_fastdiv(static_cast<uint32_t>(std::max(a.c.dim / 16, 1)));
    // Tensor copies where rows lie on 16-byte boundaries, pages are whole eights of slots (which the swizzle needs) and
    // no stride is 0 or past what a tensor map holds: boxes of the largest power of two that divides a page and a step.
    // Otherwise 16 bytes or an element at a time.
    a.box = 1;
    bool boxes = a.vec && cache->page_size % 8 == 0;
    for (int i = 0; i < 3; ++i)
        for (const int64_t *pst : {cache->k_stride, cache->v_stride})
            if (pool[i] > 1 && (pst[i] == 0 || pst[i] >= int64_t(1) << 38)) boxes = false;
    if (boxes) {
        a.box = cache->page_size & -cache->page_size;
        a.box = std::min(a.box, keys);
        if (!map_pool(&a.km, *cache, cache->k, cache->k_stride, a.box) || !map_pool(&a.vm, *cache, cache->v, cache->v_stride, a.box))
            a.box = 1;
    }
    const auto launch = cache->type == LC_CACHE_BF16 ? launch_tree_bf16 : cache->type == LC_CACHE_F16 ? launch_tree_f16 : launch_tree_e4m3;
    return launch(a, reinterpret_cast<cudaStream_t>(stream));
}
