// The accepted drafts of a sequence move together behind the tokens before them
// (lc_cache_accept).
//
// The i-th draft of the path goes from slot before + path[i] to slot before + i.
// A path rises, so path[i] >= i: no row is written over before the rows behind it
// in the path, which lie further on, have been read.  One thread therefore moves 16 bytes of a
// (pool, head) along the whole path, kAcRows rows read before they are written, and
// threads need not wait for one another.  Rows that are in their place already are
// not touched.
//
// 192 sequences of up to 64 drafts, 8 heads of 128: 8.1 us for 48 MB, 6.0 TB/s; 4 sequences of 8:
// 3.0 us, the launch and three dependent reads.  kAcRows rows are on the way a thread:
// otherwise a path costs a read's latency a draft.
#include "cache_common.cuh"

namespace lc {

constexpr uint32_t kClassAccept = 0xf5;
constexpr int kAcThreads = 128;
constexpr int kAcRows = 8;

struct AcceptArgs {
    CacheArgs c;
    const int32_t *lengths, *counts, *path;
    int32_t *new_lengths;
    int64_t path_stride;
    int32_t n_path;
    int32_t eb;       // bytes of an element
    int32_t words;    // of a row
    int32_t items;    // words of a token's rows in both pools, and its scales
    int32_t blocks;   // of a sequence
    FastDiv word_div, block_div;
};

template <typename W>
__device__ __forceinline__ void move_along(const AcceptArgs &a, const int *from, const int *row_from, const int *row_to,
                                           const int *to, int n, uint8_t *pool, const int64_t *st, int head, int64_t byte,
                                           int eb) {
    auto at = [&](int page, int row) { return reinterpret_cast<W *>(pool + row_offset(st, page, head, row) * eb + byte); };
    for (int i0 = 0; i0 < n; i0 += kAcRows) {
        W w[kAcRows];
#pragma unroll
        for (int i = 0; i < kAcRows; ++i)
            if (i0 + i < n && from[i0 + i] >= 0) w[i] = *at(from[i0 + i], row_from[i0 + i]);
#pragma unroll
        for (int i = 0; i < kAcRows; ++i)
            if (i0 + i < n && from[i0 + i] >= 0) *at(to[i0 + i], row_to[i0 + i]) = w[i];
    }
}

// W: what a row is moved in, 16 bytes where it may be.
template <typename W>
__global__ void __launch_bounds__(kAcThreads) k_cache_accept(const __grid_constant__ AcceptArgs a) {
    __shared__ int from[LC_CACHE_MAX_DRAFTS], row_from[LC_CACHE_MAX_DRAFTS];  // page, -1: the row stays; row of it
    __shared__ int to[LC_CACHE_MAX_DRAFTS], row_to[LC_CACHE_MAX_DRAFTS];
    __shared__ uint32_t wrong[2];
    const CacheArgs &c = a.c;
    start_after_prior();
    const int t = threadIdx.x;
    const int b = static_cast<int>(fast_div(blockIdx.x, a.block_div)), block = blockIdx.x - b * a.blocks;
    const int n = cache_length(c, a.lengths, b, kClassAccept);
    const int want = a.counts ? a.counts[b] : min(a.n_path, n);
    const int count = min(max(want, 0), min(LC_CACHE_MAX_DRAFTS, n)), before = n - count;
    // the path ends at the first column that does not rise
    int p = -1;
    bool bad = false;
    if (t < LC_CACHE_MAX_DRAFTS) {
        if (t < a.n_path) {
            p = a.path[b * a.path_stride + t];
            const int last = t ? a.path[b * a.path_stride + t - 1] : -1;
            bad = p <= last || p >= count;
        } else {
            bad = true;
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, bad);
        if (t % 32 == 0) wrong[t / 32] = bits;
    }
    __syncthreads();
    const int m = wrong[0] ? __ffs(wrong[0]) - 1 : wrong[1] ? 31 + __ffs(wrong[1]) : LC_CACHE_MAX_DRAFTS;
    if (block == 0) {
        if (t == 0) {
            a.new_lengths[b] = before + m;
            if (count != want) report_error(LC_ERR_CACHE_INDEX, kClassAccept);
        }
        // (-1 ends a path; anything else that does not rise is an error)
        if (t == m && t < a.n_path && p != -1) report_error(LC_ERR_CACHE_INDEX, kClassAccept);
    }
    if (t < m) {
        int x = -1;
        if (p != t) {
            x = cache_page(c, b, before + p, &row_from[t], kClassAccept);
            to[t] = cache_page(c, b, before + t, &row_to[t], kClassAccept);
            if (to[t] < 0) x = -1;
        }
        from[t] = x;
    }
    __syncthreads();
    const int item = block * kAcThreads + t;
    if (item >= a.items) return;
    const int word = static_cast<int>(fast_div(item, a.word_div)), in = item - word * a.words;  // word: (pool, head)
    if (word < 2 * c.heads) {
        const bool is_v = word >= c.heads;
        move_along<W>(a, from, row_from, row_to, to, m, is_v ? c.v : c.k, is_v ? c.vst : c.kst, is_v ? word - c.heads : word,
                      int64_t(in) * sizeof(W), a.eb);
    } else {
        const int s = item - 2 * c.heads * a.words;  // E4M3: scales
        const bool is_v = s >= c.heads;
        move_along<float>(a, from, row_from, row_to, to, m, reinterpret_cast<uint8_t *>(is_v ? c.vs : c.ks),
                          is_v ? c.vss : c.kss, is_v ? s - c.heads : s, 0, 4);
    }
}

cudaError_t take_error_accept(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

extern "C" int lc_cache_accept(const lc_paged_cache *cache, const int32_t *lengths, const int32_t *counts,
                               const int32_t *path, int64_t path_stride, int32_t n_path, int32_t *new_lengths,
                               lc_stream_t stream) {
    using namespace lc;
    AcceptArgs a{};
    int st = check_cache(cache, true, &a.c);
    if (st) return st;
    if (n_path < 0 || n_path > LC_CACHE_MAX_DRAFTS) return LC_ERR_SHAPE;
    if (cache->n_seqs == 0) return LC_OK;
    if (!lengths || !new_lengths || (n_path > 0 && !path)) return LC_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(path) |
         reinterpret_cast<uintptr_t>(new_lengths)) % 4)
        return LC_ERR_ALIGN;
    const int64_t ext[1] = {cache->n_seqs};
    st = check_reach(1, ext, &path_stride, n_path);
    if (st) return st;
    // blocks read lengths, counts, paths and pages when others have written
    for (const int32_t *in : {lengths, counts})
        if (in && lists_meet(in, new_lengths, cache->n_seqs)) return LC_ERR_OVERLAP;
    if (n_path > 0) {
        const uintptr_t p0 = reinterpret_cast<uintptr_t>(path), l0 = reinterpret_cast<uintptr_t>(new_lengths);
        if (p0 < l0 + 4 * ext[0] && l0 < p0 + 4 * ((ext[0] - 1) * path_stride + n_path)) return LC_ERR_OVERLAP;
    }
    if (may_meet(span_of(new_lengths, 1, 0, ext[0], 4), span_of(cache->page_table, ext[0], cache->table_stride, cache->pages_per_seq, 4)))
        return LC_ERR_OVERLAP;
    a.lengths = lengths;
    a.counts = counts;
    a.path = path;
    a.new_lengths = new_lengths;
    a.path_stride = path_stride;
    a.n_path = n_path;
    const int eb = a.eb = cache_elem_bytes(cache->type);
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    const bool vec = a.c.dim * eb % 16 == 0 && rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 16) &&
                     rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 16);
    a.words = vec ? a.c.dim * eb / 16 : a.c.dim;
    const int64_t items = int64_t(2) * a.c.heads * (a.words + (cache->type == LC_CACHE_E4M3 ? 1 : 0));
    if (items > 1 << 28) return LC_ERR_OVERFLOW;
    a.items = static_cast<int32_t>(items);
    a.blocks = (a.items + kAcThreads - 1) / kAcThreads;
    if (int64_t(a.blocks) * cache->n_seqs > 0x7fffffff) return LC_ERR_OVERFLOW;
    a.word_div = make_fastdiv(static_cast<uint32_t>(a.words));
    a.block_div = make_fastdiv(static_cast<uint32_t>(a.blocks));
    const void *fn = vec       ? reinterpret_cast<const void *>(&k_cache_accept<uint4>)
                     : eb == 2 ? reinterpret_cast<const void *>(&k_cache_accept<uint16_t>)
                               : reinterpret_cast<const void *>(&k_cache_accept<uint8_t>);
    return launch_after(fn, static_cast<unsigned>(a.blocks * cache->n_seqs), kAcThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream), &a);
}
