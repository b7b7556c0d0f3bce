// Attention of one new token a sequence over a paged key-value cache
// (lc_cache_attend):
//     x_j = scale * q . k_j,  w = softmax(x),  out = sum_j w_j v_j
// over the slots j that are seen, in float32.  A sequence and key head is one
// block: per query head, each warp keeps a running maximum, sum and output of
// the slots it takes (every fourth), joined through shared memory; a second
// pass over the keys adds the weights to `scores`.
#include <cmath>

#include "cache_common.cuh"

namespace lc {

constexpr int kAtThreads = 128;

struct AttendArgs {
    CacheArgs c;
    const uint16_t *q;
    uint16_t *out;
    const int32_t *lengths;
    const uint8_t *mask;
    float *lse, *scores;
    int64_t qst[2], ost[2], sst[2];
    int64_t mask_stride, lse_stride;
    int32_t q_heads, group, window;
    float scale;
    bool bf16;      // of q and out
    int32_t type;   // of the cache
};

__device__ __forceinline__ float to_float(uint16_t w, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
}

__device__ __forceinline__ float cache_value(const AttendArgs &a, const uint8_t *p, int64_t i) {
    if (a.type != LC_CACHE_E4M3) return to_float(reinterpret_cast<const uint16_t *>(p)[i], a.type == LC_CACHE_BF16);
    // sign and magnitude moved to bfloat16's places; the exponents' biases are 120 apart
    const uint32_t u = p[i];
    return __uint_as_float((u & 0x80u) << 24 | (u & 0x7fu) << 20) * 0x1p120f;
}

__global__ void __launch_bounds__(kAtThreads) k_cache_attend(const __grid_constant__ AttendArgs a) {
    __shared__ float so[4][LC_CACHE_MAX_DIM], sm[4], sl[4];
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / c.heads, h = blockIdx.x - b * c.heads;
    const int n = cache_length(c, a.lengths, b, kClassAttend);
    const int lo = a.window && a.window < n ? n - a.window : 0;
    extern __shared__ float lse_of[];  // per query head of the group
    // this lane's elements of query head g
    auto load_q = [&](int g, float (&x)[8]) {
        const uint16_t *q = a.q + b * a.qst[0] + (h * a.group + g) * a.qst[1];
        for (int i = 0; i < 8; ++i) x[i] = lane + 32 * i < c.dim ? to_float(q[lane + 32 * i], a.bf16) : 0.f;
    };
    // page of slot j, -1 where it is not seen
    auto find = [&](int j, int *row) {
        return a.mask && !a.mask[b * a.mask_stride + j] ? -1 : cache_page(c, b, j, row, kClassAttend);
    };
    auto score = [&](const float (&x)[8], int page, int row) {
        const int64_t at = row_offset(c.kst, page, h, row);
        float s = 0.f;
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < c.dim) s += x[i] * cache_value(a, c.k, at + lane + 32 * i);
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        return (c.ks ? s * c.ks[row_offset(c.kss, page, h, row)] : s) * a.scale;
    };
    float x[8];
    for (int g = 0; g < a.group; ++g) {
        const int hq = h * a.group + g;
        float m = -INFINITY, l = 0.f, o[8] = {};
        load_q(g, x);
        for (int j = lo + warp; j < n; j += 4) {
            int row;
            const int page = find(j, &row);
            if (page < 0) continue;
            const float s = score(x, page, row);
            const float top = fmaxf(m, s), safe = top == -INFINITY ? 0.f : top;
            const float keep = expf(m - safe), p = expf(s - safe);
            const float pv = c.vs ? p * c.vs[row_offset(c.vss, page, h, row)] : p;
            const int64_t at = row_offset(c.vst, page, h, row);
            l = l * keep + p;
            for (int i = 0; i < 8; ++i)
                if (lane + 32 * i < c.dim) o[i] = o[i] * keep + pv * cache_value(a, c.v, at + lane + 32 * i);
            m = top;
        }
        for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
        if (lane == 0) {
            sm[warp] = m;
            sl[warp] = l;
        }
        __syncthreads();
        float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        if (top == -INFINITY) top = 0.f;
        float total = 0.f;
        for (int w = 0; w < 4; ++w) total += sl[w] * expf(sm[w] - top);
        for (int i = threadIdx.x; i < c.dim; i += kAtThreads) {
            float y = 0.f;
            for (int w = 0; w < 4; ++w) y += so[w][i] * expf(sm[w] - top);
            y = total == 0.f ? 0.f : y / total;
            a.out[b * a.ost[0] + hq * a.ost[1] + i] =
                a.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
        }
        if (threadIdx.x == 0) {
            lse_of[g] = top + logf(total);
            if (a.lse) a.lse[b * a.lse_stride + hq] = lse_of[g];
        }
        __syncthreads();
    }
    if (!a.scores) return;
    for (int j = lo + warp; j < n; j += 4) {
        int row;
        const int page = find(j, &row);
        if (page < 0) continue;
        float w = 0.f;
        for (int g = 0; g < a.group; ++g) {
            load_q(g, x);
            const float s = score(x, page, row);
            if (lse_of[g] != -INFINITY) w += expf(s - lse_of[g]);
        }
        if (lane == 0) a.scores[b * a.sst[0] + h * a.sst[1] + j] += w;
    }
}

cudaError_t take_error_attend(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

extern "C" int64_t lc_cache_attend_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t with_scores) {
    (void)with_scores;
    lc::CacheArgs c;
    if (lc::check_cache(cache, false, &c) || n_q_heads < 1 || n_q_heads % c.heads) return -1;
    return 0;
}

extern "C" int lc_cache_attend(const lc_paged_cache *cache, const lc_cache_query *q, lc_stream_t stream) {
    using namespace lc;
    AttendArgs a{};
    int st = check_cache(cache, false, &a.c);
    if (st) return st;
    if (!q) return LC_ERR_NULL;
    if (q->n_q_heads < 1 || q->n_q_heads % cache->n_kv_heads || q->window < 0) return LC_ERR_SHAPE;
    if (q->type != (cache->type == LC_CACHE_E4M3 ? LC_CACHE_BF16 : cache->type)) return LC_ERR_TYPE;
    if (cache->n_seqs == 0) return LC_OK;
    if (!q->q || !q->out || !q->lengths) return LC_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(q->q) | reinterpret_cast<uintptr_t>(q->out)) % 2 ||
        (reinterpret_cast<uintptr_t>(q->lengths) | reinterpret_cast<uintptr_t>(q->lse) |
         reinterpret_cast<uintptr_t>(q->scores)) % 4)
        return LC_ERR_ALIGN;
    const int64_t qext[2] = {cache->n_seqs, q->n_q_heads}, kext[2] = {cache->n_seqs, cache->n_kv_heads};
    st = check_reach(2, qext, q->q_stride, cache->head_dim);
    if (!st) st = check_reach(2, qext, q->out_stride, cache->head_dim);
    if (!st && q->mask) st = check_reach(1, qext, &q->mask_stride, a.c.cap);
    if (!st && q->lse) st = check_reach(1, qext, &q->lse_stride, q->n_q_heads);
    if (!st && q->scores) st = check_reach(2, kext, q->scores_stride, a.c.cap);
    if (st) return st;
    if (!rows_apart(2, qext, q->out_stride, cache->head_dim) ||
        (q->lse && !rows_apart(1, qext, &q->lse_stride, q->n_q_heads)) ||
        (q->scores && !rows_apart(2, kext, q->scores_stride, std::max(a.c.cap, 1))))
        return LC_ERR_NOT_INJECTIVE;
    if (kext[0] * kext[1] > 0x7fffffff) return LC_ERR_OVERFLOW;
    if (q->n_q_heads / cache->n_kv_heads > 1024) return LC_ERR_SHAPE;
    const int64_t need = lc_cache_attend_workspace(cache, q->n_q_heads, q->scores != nullptr);
    if (need > 0 && !q->workspace) return LC_ERR_NULL;
    if (need > q->workspace_bytes) return LC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(q->workspace) % 256) return LC_ERR_ALIGN;
    a.q = static_cast<const uint16_t *>(q->q);
    a.out = static_cast<uint16_t *>(q->out);
    a.lengths = q->lengths;
    a.mask = q->mask;
    a.lse = q->lse;
    a.scores = q->scores;
    for (int i = 0; i < 2; ++i) {
        a.qst[i] = q->q_stride[i];
        a.ost[i] = q->out_stride[i];
        a.sst[i] = q->scores_stride[i];
    }
    a.mask_stride = q->mask_stride;
    a.lse_stride = q->lse_stride;
    a.q_heads = q->n_q_heads;
    a.group = q->n_q_heads / cache->n_kv_heads;
    a.window = q->window;
    a.scale = q->scale;
    a.bf16 = q->type == LC_CACHE_BF16;
    a.type = cache->type;
    k_cache_attend<<<static_cast<unsigned>(kext[0] * kext[1]), kAtThreads, 4 * a.group,
                     reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return finish_launch();
}
