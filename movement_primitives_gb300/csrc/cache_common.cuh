// What the paged-cache kernels share: the cache as a kernel parameter, slot
// addresses, the host checks of a cache descriptor, element conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "launch.h"
#include "layout_copy_cache.h"

namespace lc {

// Kernel classes in the device error word.
constexpr uint32_t kClassAppend = 0xf0, kClassAttend = 0xf1, kClassEvict = 0xf2;

// Kernels are launched to overlap the end of what precedes them on the stream
// (launch_after): the next one may be set up as soon as every block has come
// here, and this one touches no memory until all before it has ended and is
// visible.
__device__ __forceinline__ void start_after_prior() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct CacheArgs {
    uint8_t *k, *v;
    float *ks, *vs;
    const int32_t *table;
    int64_t table_stride, n_pages;
    int32_t n_seqs, heads, page, dim, per, cap;
    FastDiv page_div;
    int64_t kst[3], vst[3], kss[3], vss[3];  // elements: page, head, slot
};

// Length of sequence b, clamped to its capacity.
__device__ __forceinline__ int cache_length(const CacheArgs &c, const int32_t *lengths, int b, uint32_t cls) {
    const int n = lengths[b];
    const int m = min(max(n, 0), c.cap);
    if (n != m) report_error(LC_ERR_CACHE_INDEX, cls);
    return m;
}

// Page of slot j (0 <= j < cap) of sequence b, -1 when the table names none in
// the pool; `row` receives the slot's row in it.
__device__ __forceinline__ int cache_page(const CacheArgs &c, int b, int j, int *row, uint32_t cls) {
    const int i = static_cast<int>(fast_div(static_cast<uint32_t>(j), c.page_div));
    *row = j - i * c.page;
    const int p = c.table[b * c.table_stride + i];
    if (p >= 0 && p < c.n_pages) return p;
    report_error(LC_ERR_CACHE_INDEX, cls);
    return -1;
}

__device__ __forceinline__ int64_t row_offset(const int64_t *st, int page, int head, int row) {
    return page * st[0] + head * st[1] + row * st[2];
}

// ---- host ----------------------------------------------------------------

// Launches a kernel of one parameter struct that calls start_after_prior; in
// clusters of `cluster` blocks.
inline int launch_after(const void *fn, unsigned grid, unsigned threads, size_t smem, cudaStream_t cs, const void *arg,
                        unsigned cluster = 1) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = cs;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void *args[] = {const_cast<void *>(arg)};
    if (cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess) return LC_OK;
    cudaGetLastError();  // reported here: the next call's check does not see it
    return LC_ERR_CUDA;
}

inline int cache_elem_bytes(int type) { return type == LC_CACHE_E4M3 ? 1 : 2; }

// Largest element offset of extents `e` (>= 1 each) at strides `st` plus a
// last run of `run` elements; LC_ERR_BAD_STRIDE for a negative stride.
inline int check_reach(int n, const int64_t *e, const int64_t *st, int64_t run) {
    int64_t top = run;
    for (int i = 0; i < n; ++i) {
        int64_t x;
        if (st[i] < 0) return LC_ERR_BAD_STRIDE;
        if (!mul_ok_ext(e[i] - 1, st[i], &x) || !add_ok_ext(top, x, &top)) return LC_ERR_OVERFLOW;
    }
    return top > (int64_t(1) << 60) ? LC_ERR_OVERFLOW : LC_OK;
}

// Whether rows of `run` elements at these strides are apart: every stride,
// from the smallest up, clears what the smaller ones reach.
inline bool rows_apart(int n, const int64_t *e, const int64_t *st, int64_t run) {
    int at[4] = {0, 1, 2, 3};
    std::sort(at, at + n, [&](int a, int b) { return st[a] < st[b]; });
    int64_t span = run;
    for (int i = 0; i < n; ++i) {
        if (e[at[i]] <= 1) continue;
        if (st[at[i]] < span) return false;
        span += (e[at[i]] - 1) * st[at[i]];
    }
    return true;
}

// Whether `n` 4-byte elements at p and at q share any.
inline bool lists_meet(const void *p, const void *q, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return (a < b ? b - a : a - b) < static_cast<uint64_t>(n) * 4;
}

// Whether rows of `run` elements of eb bytes at p (strides st) share any with those
// at q (strides qst, rows apart), both of extents `e`.  Buffers whose ranges
// meet may still be apart, as two interleaved halves of one are.
inline bool rows_meet(const void *p, const int64_t *st, const void *q, const int64_t *qst, const int64_t *e,
                      int64_t run, int64_t eb = 4) {
    auto span = [&](const int64_t *s) { return (e[0] - 1) * s[0] + (e[1] - 1) * s[1] + run; };
    const int64_t d = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)) -
                       static_cast<int64_t>(reinterpret_cast<uintptr_t>(q))) / eb;
    if (d >= span(qst) || -d >= span(st)) return false;
    // q's rows from their larger step to the smaller one; a step of one row is none
    const int big = e[0] <= 1 ? 1 : e[1] <= 1 ? 0 : qst[0] < qst[1], small = 1 - big;
    // the steps i of `x` that rows at `at` could meet: two at most, since a row is no longer than a step
    auto meets = [&](int x, int64_t at, auto &&with) {
        if (e[x] <= 1) return with(at);
        const int64_t i0 = at >= 0 ? std::min(at / qst[x], e[x] - 1) : 0;
        const int64_t i1 = at + run > 0 ? std::min((at + run - 1) / qst[x], e[x] - 1) : 0;
        return with(at - i0 * qst[x]) || (i1 != i0 && with(at - i1 * qst[x]));
    };
    for (int64_t i = 0; i < e[0]; ++i)
        for (int64_t j = 0; j < e[1]; ++j)
            if (meets(big, d + i * st[0] + j * st[1], [&](int64_t at) {
                    return meets(small, at, [&](int64_t off) { return (off < 0 ? -off : off) < run; });
                }))
                return true;
    return false;
}

// Checks a cache descriptor and lays it out for the kernels.  `write`: the
// operator writes rows, which then have to be apart.
inline int check_cache(const lc_paged_cache *c, bool write, CacheArgs *a) {
    if (!c) return LC_ERR_NULL;
    if (c->type != LC_CACHE_BF16 && c->type != LC_CACHE_F16 && c->type != LC_CACHE_E4M3) return LC_ERR_TYPE;
    if (c->n_seqs < 0 || c->n_kv_heads < 1 || c->page_size < 1 || c->head_dim < 1 ||
        c->head_dim > LC_CACHE_MAX_DIM || c->pages_per_seq < 0 || c->n_pages < 0 || c->n_pages > 0x7fffffff)
        return LC_ERR_SHAPE;
    if (int64_t(c->page_size) * c->pages_per_seq > 0x7fff0000) return LC_ERR_OVERFLOW;
    if (c->n_seqs > 0 && c->pages_per_seq > 0 && c->n_pages < 1) return LC_ERR_SHAPE;
    if (c->n_pages > 0 && (!c->k || !c->v)) return LC_ERR_NULL;
    if (c->n_seqs > 0 && c->pages_per_seq > 0 && !c->page_table) return LC_ERR_NULL;
    const bool q8 = c->type == LC_CACHE_E4M3;
    if (q8 && c->n_pages > 0 && (!c->k_scale || !c->v_scale)) return LC_ERR_NULL;
    if (!q8 && (c->k_scale || c->v_scale)) return LC_ERR_TYPE;
    const int eb = cache_elem_bytes(c->type);
    const uintptr_t words = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v);
    const uintptr_t floats = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
                             reinterpret_cast<uintptr_t>(c->page_table);
    if (words % eb || floats % 4) return LC_ERR_ALIGN;
    const int64_t ext[3] = {std::max<int64_t>(c->n_pages, 1), c->n_kv_heads, c->page_size};
    const int64_t text[1] = {std::max<int64_t>(c->n_seqs, 1)}, tst[1] = {c->table_stride};
    int st = check_reach(3, ext, c->k_stride, c->head_dim);
    if (!st) st = check_reach(3, ext, c->v_stride, c->head_dim);
    if (!st && q8) st = check_reach(3, ext, c->k_scale_stride, 1);
    if (!st && q8) st = check_reach(3, ext, c->v_scale_stride, 1);
    if (!st) st = check_reach(1, text, tst, c->pages_per_seq);
    if (st) return st;
    if (write && (!rows_apart(3, ext, c->k_stride, c->head_dim) || !rows_apart(3, ext, c->v_stride, c->head_dim) ||
                  (q8 && (!rows_apart(3, ext, c->k_scale_stride, 1) || !rows_apart(3, ext, c->v_scale_stride, 1)))))
        return LC_ERR_NOT_INJECTIVE;
    a->k = static_cast<uint8_t *>(c->k);
    a->v = static_cast<uint8_t *>(c->v);
    a->ks = c->k_scale;
    a->vs = c->v_scale;
    a->table = c->page_table;
    a->table_stride = c->table_stride;
    a->n_pages = c->n_pages;
    a->n_seqs = c->n_seqs;
    a->heads = c->n_kv_heads;
    a->page = c->page_size;
    a->dim = c->head_dim;
    a->per = c->pages_per_seq;
    a->cap = c->page_size * c->pages_per_seq;
    a->page_div = make_fastdiv(static_cast<uint32_t>(c->page_size));
    for (int i = 0; i < 3; ++i) {
        a->kst[i] = c->k_stride[i];
        a->vst[i] = c->v_stride[i];
        a->kss[i] = q8 ? c->k_scale_stride[i] : 0;
        a->vss[i] = q8 ? c->v_scale_stride[i] : 0;
    }
    return LC_OK;
}

// Whether a base and its strides (elements of eb bytes; of extents e) keep
// every row on `bytes`-byte boundaries.
inline bool rows_aligned(const void *p, int n, const int64_t *e, const int64_t *st, int64_t eb, int64_t bytes) {
    if (reinterpret_cast<uintptr_t>(p) % bytes) return false;
    for (int i = 0; i < n; ++i)
        if (e[i] > 1 && st[i] * eb % bytes) return false;
    return true;
}

}  // namespace lc
