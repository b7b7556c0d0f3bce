// Prompt attention: the checks, the tensor maps and the C entry point
// (lc_prompt_attend; the kernel is prompt_attend.cuh).
#include <cmath>

#include "prompt_attend.cuh"
#include "tensor_map.h"

namespace lc {

int launch_prompt_bf16(const PromptArgs &a, int64_t items, cudaStream_t cs);
int launch_prompt_f16(const PromptArgs &a, int64_t items, cudaStream_t cs);

namespace {

// Tokens x heads x head_dim of 16-bit elements, in boxes of 64 columns.
bool map_rows(CUtensorMap *m, bool f16, const void *p, int64_t tokens, int heads, int dim, const int64_t *st, int box_heads,
              int box_tokens) {
    EncodeTiledFn encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(std::max<int64_t>(tokens, 1))};
    // a mode of one element has no stride of its own
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? st[1] : (dim + 7) / 8 * 8) * 2,
                                   static_cast<cuuint64_t>(tokens > 1 ? st[0] : (dim + 7) / 8 * 8) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    return encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p),
                  dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace lc

extern "C" int lc_prompt_attend(const lc_prompt *p, lc_stream_t stream) {
    using namespace lc;
    if (!p) return LC_ERR_NULL;
    if (p->type != LC_CACHE_BF16 && p->type != LC_CACHE_F16) return LC_ERR_TYPE;
    if (p->n_seqs < 0 || p->n_kv_heads < 1 || p->n_q_heads < 1 || p->n_q_heads % p->n_kv_heads || p->head_dim < 8 ||
        p->head_dim > LC_CACHE_MAX_DIM || p->head_dim % 8 || p->n_tokens < 0 || p->n_keys < 0 || p->window < 0 ||
        !std::isfinite(p->scale * kLog2e))
        return LC_ERR_SHAPE;
    if (p->n_tokens > 1 << 30 || p->n_keys > 1 << 30) return LC_ERR_OVERFLOW;
    if (p->n_seqs == 0 || p->n_tokens == 0) return LC_OK;
    if (!p->q || !p->out || !p->starts || (p->n_keys > 0 && (!p->k || !p->v))) return LC_ERR_NULL;
    const int64_t qext[2] = {p->n_tokens, p->n_q_heads}, kext[2] = {std::max<int64_t>(p->n_keys, 1), p->n_kv_heads};
    const int dim = p->head_dim;
    int st = check_reach(2, qext, p->q_stride, dim);
    if (!st) st = check_reach(2, kext, p->k_stride, dim);
    if (!st) st = check_reach(2, kext, p->v_stride, dim);
    if (!st) st = check_reach(2, qext, p->out_stride, dim);
    if (!st && p->lse) st = check_reach(1, qext, &p->lse_stride, p->n_q_heads);
    if (st) return st;
    for (int i = 0; i < 2; ++i) {
        if ((qext[i] > 1 && !p->q_stride[i]) || (kext[i] > 1 && (!p->k_stride[i] || !p->v_stride[i])))
            return LC_ERR_BAD_STRIDE;
        const int64_t most = int64_t(1) << 38;  // a tensor map's strides end at 2^40 bytes
        if ((qext[i] > 1 && p->q_stride[i] >= most) ||
            (kext[i] > 1 && (p->k_stride[i] >= most || p->v_stride[i] >= most)))
            return LC_ERR_OVERFLOW;
    }
    if (!rows_aligned(p->q, 2, qext, p->q_stride, 2, 16) || reinterpret_cast<uintptr_t>(p->out) % 2 ||
        (p->n_keys > 0 && (!rows_aligned(p->k, 2, kext, p->k_stride, 2, 16) ||
                           !rows_aligned(p->v, 2, kext, p->v_stride, 2, 16))) ||
        (reinterpret_cast<uintptr_t>(p->lse) | reinterpret_cast<uintptr_t>(p->starts) |
         reinterpret_cast<uintptr_t>(p->k_starts)) % 4)
        return LC_ERR_ALIGN;
    if (!rows_apart(2, qext, p->out_stride, dim) || (p->lse && !rows_apart(1, qext, &p->lse_stride, p->n_q_heads)))
        return LC_ERR_NOT_INJECTIVE;
    // a row of the queries' own buffer is written when its item has read it
    const bool in_place = p->out == p->q && (qext[0] == 1 || p->q_stride[0] == p->out_stride[0]) &&
                          (qext[1] == 1 || p->q_stride[1] == p->out_stride[1]);
    const Span out = span_of(p->out, qext[0], p->out_stride[0], dim, 2, qext[1], p->out_stride[1]);
    const Span lse = span_of(p->lse, qext[0], p->lse_stride, qext[1], 4);
    const Span q = span_of(p->q, qext[0], p->q_stride[0], dim, 2, qext[1], p->q_stride[1]);
    const Span read[] = {span_of(p->k, p->n_keys, p->k_stride[0], dim, 2, kext[1], p->k_stride[1]),
                         span_of(p->v, p->n_keys, p->v_stride[0], dim, 2, kext[1], p->v_stride[1]),
                         span_of(p->starts, 1, 0, p->n_seqs + int64_t(1), 4), span_of(p->k_starts, 1, 0, p->n_seqs + int64_t(1), 4)};
    if ((!in_place && may_meet(out, q)) || may_meet(lse, q) || may_meet(lse, out)) return LC_ERR_OVERLAP;
    for (const Span &x : read)
        if (may_meet(out, x) || may_meet(lse, x)) return LC_ERR_OVERLAP;
    PromptArgs a{};
    a.starts = p->starts;
    a.k_starts = p->k_starts;
    a.out = static_cast<uint16_t *>(p->out);
    a.lse = p->lse;
    a.v = static_cast<const uint16_t *>(p->v);
    for (int i = 0; i < 2; ++i) {
        a.ost[i] = p->out_stride[i];
        a.vst[i] = p->v_stride[i];
    }
    a.lse_stride = p->lse_stride;
    a.n_seqs = p->n_seqs;
    a.n_tokens = static_cast<int32_t>(p->n_tokens);
    a.n_keys = static_cast<int32_t>(p->n_keys);
    a.group = p->n_q_heads / p->n_kv_heads;
    a.heads_tile = std::min(a.group, kPrRows);
    a.head_blocks = (a.group + a.heads_tile - 1) / a.heads_tile;
    a.key_heads = p->n_kv_heads;
    a.tokens_tile = kPrRows / a.heads_tile;
    a.dim = dim;
    a.causal = p->causal != 0;
    a.window = std::min(p->window, 1 << 30);
    a.heads_div = make_fastdiv(static_cast<uint32_t>(a.heads_tile));
    const int64_t heads = int64_t(a.key_heads) * a.head_blocks;
    const int per = a.tokens_tile * (dim <= 128 ? 2 : 1);
    const int64_t pairs = p->n_tokens / per + p->n_seqs;
    if (heads > 0x3fffffff / pairs) return LC_ERR_OVERFLOW;
    a.pair_div = make_fastdiv(static_cast<uint32_t>(heads));
    // a scale of 0 is the smallest number there is, under which all logits are too small to tell, so that unseen keys' -infinity stays what it is
    a.scale2 = std::max(std::fabs(p->scale) * kLog2e, 0x1p-149f);
    a.negative = p->scale < 0.f;
    a.store = rows_aligned(p->out, 2, qext, p->out_stride, 2, 32) ? 32 : rows_aligned(p->out, 2, qext, p->out_stride, 2, 16) ? 16 : 2;
    a.limit_ns = wait_limit_ns();
    const bool f16 = p->type == LC_CACHE_F16, keys = p->n_keys > 0;
    const void *k = keys ? p->k : p->q, *v = keys ? p->v : p->q;
    if (!map_rows(&a.qm, f16, p->q, p->n_tokens, p->n_q_heads, dim, p->q_stride, a.heads_tile, a.tokens_tile) ||
        !map_rows(&a.km, f16, k, p->n_keys, keys ? p->n_kv_heads : 1, dim, p->k_stride, 1, kPrKeys) ||
        !map_rows(&a.vm, f16, v, p->n_keys, keys ? p->n_kv_heads : 1, dim, p->v_stride, 1, kPrKeys))
        return LC_ERR_CUDA;
    return (f16 ? launch_prompt_f16 : launch_prompt_bf16)(a, pairs * heads, reinterpret_cast<cudaStream_t>(stream));
}
