// Eviction from a paged key-value cache by accumulated weight (lc_cache_evict).
//
// Per sequence and key head, of n > budget slots: the `recent` newest stay,
// and of the others the budget - recent of largest score, equal scores in
// slot order.  k_evict_select finds the score of the last one kept by radix
// selection, 8 bits of an order-preserving 32-bit key at a time, and writes
// the kept slots in ascending order (`kept`) with their scores;
// k_evict_move moves the rows.
//
// Rows move in place: the r-th kept slot goes to slot r, and kept[r] >= r, so
// a destination r never holds a row that a later rank j > r has yet to read
// (kept[j] >= j > r).  Reading a run of ranks, a barrier, writing it, and
// going on to the next run is therefore enough, and the columns of a row are
// independent of one another: a row's words are split over several blocks.
#include "cache_common.cuh"

namespace lc {

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 4;  // slots a thread looks at in one round of the ordered pass
constexpr int kMvThreads = 256;
constexpr int kMvPer = 8;   // words a thread holds at a time

struct EvictArgs {
    CacheArgs c;
    const int32_t *lengths;
    const float *scores;
    float *new_scores;
    int32_t *kept, *new_lengths;
    int64_t sst[2], nst[2], kst[2];  // sequence, head
    int32_t budget, recent;
    int32_t slices;      // blocks that share a row of one pool
    int32_t row_words;   // words of a row
};

// Larger scores have larger keys; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float s) {
    if (isnan(s)) s = __int_as_float(0xff800000);
    const uint32_t u = __float_as_uint(s + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

// Exclusive scan of one value a thread over the block; `total` is the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *warp_sums, uint32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    __syncthreads();  // warp_sums is free again
    return (warp ? before : 0) + s - x;
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictArgs a) {
    __shared__ uint32_t hist[256], warp_sums[32], chosen[2];
    const int t = threadIdx.x;
    const int b = blockIdx.x / a.c.heads, h = blockIdx.x - b * a.c.heads;
    const int n = cache_length(a.c, a.lengths, b, kClassEvict);
    const int m = min(n, a.budget);
    const float *scores = a.scores + b * a.sst[0] + h * a.sst[1];
    float *out = a.new_scores + b * a.nst[0] + h * a.nst[1];
    int32_t *kept = a.kept + b * a.kst[0] + h * a.kst[1];
    if (h == 0 && t == 0) a.new_lengths[b] = m;
    for (int i = m + t; i < a.budget; i += kSelThreads) kept[i] = -1;
    for (int i = m + t; i < a.c.cap; i += kSelThreads) out[i] = 0.f;
    if (n == m) {
        for (int i = t; i < m; i += kSelThreads) {
            kept[i] = i;
            out[i] = scores[i];
        }
        return;
    }
    // the key of the last slot kept among the first `cand`, and how many of
    // the slots with that key stay
    const int cand = n - a.recent;
    uint32_t need = a.budget - a.recent, prefix = 0;
    if (need) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (t < 256) hist[t] = 0;
            __syncthreads();
            for (int i = t; i < cand; i += kSelThreads) {
                const uint32_t key = score_key(scores[i]);
                if (shift == 24 || key >> (shift + 8) == prefix) atomicAdd(&hist[key >> shift & 255], 1u);
            }
            __syncthreads();
            // digits from the largest down: thread t stands for digit 255 - t
            const uint32_t mine = t < 256 ? hist[255 - t] : 0;
            uint32_t total;
            const uint32_t before = block_scan(mine, warp_sums, &total);
            if (t < 256 && before < need && before + mine >= need) {
                chosen[0] = 255 - t;
                chosen[1] = need - before;
            }
            __syncthreads();
            prefix = prefix << 8 | chosen[0];
            need = chosen[1];
            __syncthreads();
        }
    }
    // slots in order: `sure` are kept whatever else, of the `tied` ones the first `need`
    uint32_t sure = 0, tied = 0;
    const bool any = a.budget > a.recent;
    for (int base = 0; base < n; base += kSelThreads * kSelPer) {
        float s[kSelPer];
        uint32_t is[kSelPer], count = 0;  // 1: sure, 1 << 16: tied
#pragma unroll
        for (int j = 0; j < kSelPer; ++j) {
            const int i = base + t * kSelPer + j;
            s[j] = i < n ? scores[i] : 0.f;
            is[j] = 0;
            if (i >= cand)
                is[j] = i < n;
            else if (any) {
                const uint32_t key = score_key(s[j]);
                is[j] = key > prefix ? 1u : key == prefix ? 1u << 16 : 0u;
            }
            count += is[j];
        }
        uint32_t total;
        const uint32_t before = block_scan(count, warp_sums, &total);
        uint32_t g = sure + (before & 0xffff), e = tied + (before >> 16);
#pragma unroll
        for (int j = 0; j < kSelPer; ++j) {
            if (is[j] == 1 || (is[j] && e < need)) {
                const uint32_t r = g + min(e, need);
                kept[r] = base + t * kSelPer + j;
                out[r] = s[j];
            }
            g += is[j] & 0xffff;
            e += is[j] >> 16;
        }
        sure += total & 0xffff;
        tied += total >> 16;
    }
}

// Blocks (unit, pool, slice): the words [w0, w1) of every row of the unit's
// keys or values, or (E4M3, the last two of a unit) its scales.
template <typename T>
__device__ __forceinline__ void move_rows(const EvictArgs &a, T *pool, const int64_t *st, int64_t word_elems, int b,
                                          int h, int w0, int w1) {
    const CacheArgs &c = a.c;
    const int32_t *kept = a.kept + b * a.kst[0] + h * a.kst[1];
    const int words = w1 - w0;
    const int64_t items = int64_t(a.budget) * words;
    for (int64_t base = 0; base < items; base += kMvThreads * kMvPer) {
        T x[kMvPer];
        T *to[kMvPer];
#pragma unroll
        for (int j = 0; j < kMvPer; ++j) {
            const int64_t i = base + j * kMvThreads + threadIdx.x;
            to[j] = nullptr;
            if (i >= items) continue;
            const int r = static_cast<int>(i / words), w = w0 + static_cast<int>(i - int64_t(r) * words);
            const int from = kept[r];
            if (from == r) continue;
            int row_f, row_t;
            const int pf = cache_page(c, b, from, &row_f, kClassEvict), pt = cache_page(c, b, r, &row_t, kClassEvict);
            if (pf < 0 || pt < 0) continue;
            x[j] = pool[row_offset(st, pf, h, row_f) / word_elems + w];
            to[j] = pool + row_offset(st, pt, h, row_t) / word_elems + w;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMvPer; ++j)
            if (to[j]) *to[j] = x[j];
    }
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kMvThreads) k_evict_move(const __grid_constant__ EvictArgs a) {
    const CacheArgs &c = a.c;
    const int roles = 2 * a.slices + (Q8 ? 2 : 0);
    const int unit = blockIdx.x / roles, role = blockIdx.x - unit * roles;
    const int b = unit / c.heads, h = unit - b * c.heads;
    if (min(max(a.lengths[b], 0), c.cap) <= a.budget) return;
    if (Q8 && role >= 2 * a.slices) {
        const bool v = role & 1;
        move_rows<float>(a, v ? c.vs : c.ks, v ? c.vss : c.kss, 1, b, h, 0, 1);
        return;
    }
    const bool v = role >= a.slices;
    const int s = role - (v ? a.slices : 0);
    const int w0 = static_cast<int>(int64_t(a.row_words) * s / a.slices);
    const int w1 = static_cast<int>(int64_t(a.row_words) * (s + 1) / a.slices);
    move_rows<T>(a, reinterpret_cast<T *>(v ? c.v : c.k), v ? c.vst : c.kst, sizeof(T) / (Q8 ? 1 : 2), b, h, w0, w1);
}

cudaError_t take_error_evict(unsigned long long *v) { return take_module_error(v); }

namespace {

template <typename T, bool Q8>
int launch_evict(EvictArgs &a, int eb, cudaStream_t cs) {
    a.row_words = a.c.dim * eb / static_cast<int>(sizeof(T));
    const void *fn = reinterpret_cast<const void *>(&k_evict_move<T, Q8>);
    int sms, per;
    if (prepare(fn, kMvThreads, 0, 0, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
    // rows are split until the GPU is full, into parts of 64 bytes or more
    const int64_t units = int64_t(a.c.n_seqs) * a.c.heads;
    a.slices = 1;
    while (2 * units * a.slices < int64_t(sms) * per && a.row_words * static_cast<int>(sizeof(T)) >= 128 * a.slices)
        a.slices *= 2;
    const int64_t blocks = units * (2 * a.slices + (Q8 ? 2 : 0));
    if (blocks > 0x7fffffff) return LC_ERR_OVERFLOW;
    k_evict_select<<<static_cast<unsigned>(units), kSelThreads, 0, cs>>>(a);
    k_evict_move<T, Q8><<<static_cast<unsigned>(blocks), kMvThreads, 0, cs>>>(a);
    return finish_launch();
}

}  // namespace

}  // namespace lc

extern "C" int lc_cache_evict(const lc_paged_cache *cache, const lc_cache_eviction *e, lc_stream_t stream) {
    using namespace lc;
    EvictArgs a{};
    int st = check_cache(cache, true, &a.c);
    if (st) return st;
    if (!e) return LC_ERR_NULL;
    if (e->budget < 1 || e->recent < 0 || e->recent > e->budget) return LC_ERR_SHAPE;
    if (cache->n_seqs == 0) return LC_OK;
    if (!e->lengths || !e->kept || !e->new_lengths || (a.c.cap > 0 && (!e->scores || !e->new_scores)))
        return LC_ERR_NULL;
    if (e->lengths == e->new_lengths || (a.c.cap > 0 && e->scores == e->new_scores)) return LC_ERR_OVERLAP;
    if ((reinterpret_cast<uintptr_t>(e->lengths) | reinterpret_cast<uintptr_t>(e->scores) |
         reinterpret_cast<uintptr_t>(e->kept) | reinterpret_cast<uintptr_t>(e->new_scores) |
         reinterpret_cast<uintptr_t>(e->new_lengths)) % 4)
        return LC_ERR_ALIGN;
    const int64_t ext[2] = {cache->n_seqs, cache->n_kv_heads};
    st = check_reach(2, ext, e->scores_stride, a.c.cap);
    if (!st) st = check_reach(2, ext, e->new_scores_stride, a.c.cap);
    if (!st) st = check_reach(2, ext, e->kept_stride, e->budget);
    if (st) return st;
    if (!rows_apart(2, ext, e->new_scores_stride, std::max(a.c.cap, 1)) || !rows_apart(2, ext, e->kept_stride, e->budget))
        return LC_ERR_NOT_INJECTIVE;
    if (ext[0] * ext[1] > 0x7fffffff) return LC_ERR_OVERFLOW;
    a.lengths = e->lengths;
    a.scores = e->scores;
    a.new_scores = e->new_scores;
    a.kept = e->kept;
    a.new_lengths = e->new_lengths;
    for (int i = 0; i < 2; ++i) {
        a.sst[i] = e->scores_stride[i];
        a.nst[i] = e->new_scores_stride[i];
        a.kst[i] = e->kept_stride[i];
    }
    a.budget = e->budget;
    a.recent = e->recent;
    const int eb = cache_elem_bytes(cache->type);
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    const bool wide = a.c.dim * eb % 16 == 0 && rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 16) &&
                      rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 16);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (cache->type == LC_CACHE_E4M3)
        return wide ? launch_evict<uint4, true>(a, eb, cs) : launch_evict<uint8_t, true>(a, eb, cs);
    return wide ? launch_evict<uint4, false>(a, eb, cs) : launch_evict<uint16_t, false>(a, eb, cs);
}
