// New tokens' rows into the pages of a key-value cache (lc_cache_append).
//
// Row (b, t, h) of the new keys and values goes to slot lengths[b] + t of
// sequence b, as it is or quantised to E4M3:
//     scale = max(max_e |x_e| / 448, 2^-126),  code_e = e4m3(x_e / scale)
// in float32 (division and conversion round to nearest even), NaN as the scale
// where the largest magnitude is not finite.  A row's quotients share their
// divisor: with its rounded reciprocal r, q = x r and q + (x - q scale) r in
// fused operations is the rounded quotient (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), three
// operations on pairs of elements for a division's many; scales far out of
// range divide.
//
// One warp moves a token's rows of some heads in both pools: groups of 16, 8 or
// 4 lanes take a row, each lane 16 bytes of new elements at a time, with all
// loads before the first store.  Every byte is read and written once.
//
// Measured on GB300: 64 tokens of 8 heads of 128 as they are 1.9 us, the
// latency of three dependent reads; prompts of 8966 tokens into E4M3, 56 MB,
// 11.8 us (4.7 TB/s), 34 thousand tokens, 210 MB, 35 us (6.0 TB/s); the same as
// they are, 73 MB, 13.1 us (5.6 TB/s) and, 276 MB, 42 us (6.6 TB/s).  Packed tokens by
// their slots: 64 1.8 us, 9216 13.0 as they are and 11.8 into E4M3.  What is left
// above the copy's rate is the start and the tail of the launch.
#include <cuda_fp8.h>

#include "cache_common.cuh"

namespace lc {

constexpr int kApThreads = 128;
constexpr int64_t kApMany = 4 * 152 * 48;  // rows from which a warp takes several heads

struct AppendArgs {
    CacheArgs c;
    const uint16_t *k, *v;
    int64_t kst[3], vst[3];  // elements: sequence, token, head
    const int32_t *counts, *lengths;
    int32_t *new_lengths;
    const int64_t *slots;    // packed tokens: where they go (one "sequence" of n_new tokens)
    int32_t n_new;
    uint32_t items;          // n_seqs * n_new * head_div.d: a warp each
    FastDiv new_div, head_div;
};

// A bfloat16 (Q 1) or float16 (Q 2) element.
template <int Q>
__device__ __forceinline__ float value_of(uint32_t w) {
    return Q == 1 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}

__device__ __forceinline__ uint64_t twice(float x) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(x));
    return y;
}

// -x / d of two elements from d and minus its rounded reciprocal (see above).
// With these signs a zero's comes out negated like every other: the remainder
// of x = -0 and of x = +0 is +0, and the last sum adds two zeros of one sign.
__device__ __forceinline__ float2 minus_quotients(float2 x, uint64_t d, uint64_t minus_inverse) {
    float2 y;
    asm("{\n\t"
        ".reg .b64 x, q, rest;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mul.rn.f32x2 q, x, %5;\n\t"
        "fma.rn.f32x2 rest, q, %4, x;\n\t"
        "fma.rn.f32x2 q, rest, %5, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(x.x), "f"(x.y), "l"(d), "l"(minus_inverse));
    return y;
}

// x / d from d's rounded reciprocal.
__device__ __forceinline__ float rounded_quotient(float x, float d, float inverse) {
    const float q = x * inverse;
    return fmaf(fmaf(-q, d, x), inverse, q);
}

// One row's elements, as L lanes read them, to the pool: Q 0 unchanged, 1
// bfloat16 -> E4M3, 2 float16 -> E4M3.  NI: eights of elements a lane (rows of
// up to 8 L NI).  VEC: lane l holds eights l, l + L, .., else elements l + L j.
template <int Q, bool VEC, int NI, int L>
__device__ __forceinline__ void put_row(int dim, uint8_t *dst, float *scale_at, bool on, const uint16_t (&w)[8 * NI]) {
    const int lane = threadIdx.x & (L - 1);
    if constexpr (Q == 0) {
        if (!on) return;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if constexpr (VEC) {
                if (8 * (lane + L * i) < dim)
                    *reinterpret_cast<uint4 *>(dst + 16 * (lane + L * i)) = reinterpret_cast<const uint4 *>(w)[i];
            } else {
#pragma unroll
                for (int j = 8 * i; j < 8 * i + 8; ++j)
                    if (lane + L * j < dim) reinterpret_cast<uint16_t *>(dst)[lane + L * j] = w[j];
            }
        }
    } else {
        // the largest magnitude, by its bits: infinities and NaN are above every number
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4 * NI; ++j)
            top = __vmaxu2(top, reinterpret_cast<const uint32_t *>(w)[j] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float most = value_of<Q>(top);
        float scale;
        uint32_t code[4 * NI];
        auto encode = [&](auto &&quotients) {
#pragma unroll
            for (int j = 0; j < 4 * NI; ++j)
                code[j] = __nv_cvt_float2_to_fp8x2(
                    quotients(make_float2(value_of<Q>(w[2 * j]), value_of<Q>(w[2 * j + 1]))), __NV_SATFINITE,
                    __NV_E4M3);
        };
        // rows of zeros too, which heads past the last one look like
        if (__all_sync(0xffffffffu, most == 0.f || (most > 0x1p-90f && most < 0x1p90f))) {
            scale = fmaxf(rounded_quotient(most, 448.f, 1.f / 448.f), 0x1p-126f);
            const uint64_t d = twice(scale), minus_inverse = twice(-__frcp_rn(scale));
            encode([&](float2 x) { return minus_quotients(x, d, minus_inverse); });
#pragma unroll
            for (int j = 0; j < 4 * NI; ++j) code[j] ^= 0x8080u;
        } else {
            const bool fine = top < (Q == 1 ? 0x7f80u : 0x7c00u);
            scale = fine ? fmaxf(__fdiv_rn(most, 448.f), 0x1p-126f) : __int_as_float(0x7fc00000);
            encode([&](float2 x) { return make_float2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)); });
        }
        if (!on) return;
        if (lane == 0) *scale_at = scale;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if constexpr (VEC) {
                if (8 * (lane + L * i) < dim)
                    *reinterpret_cast<uint2 *>(dst + 8 * (lane + L * i)) =
                        make_uint2(code[4 * i] | code[4 * i + 1] << 16, code[4 * i + 2] | code[4 * i + 3] << 16);
            } else {
#pragma unroll
                for (int j = 8 * i; j < 8 * i + 8; ++j)
                    if (lane + L * j < dim) dst[lane + L * j] = static_cast<uint8_t>(code[j / 2] >> (8 * (j & 1)));
            }
        }
    }
}

// Page of a slot of the pool, -1 when there is none.
__device__ __forceinline__ int slot_page(const CacheArgs &c, int64_t slot, int *row) {
    const int64_t page = slot < 0 ? -1 : slot / c.page;
    *row = static_cast<int>(slot - page * c.page);
    if (slot != -1 && (page < 0 || page >= c.n_pages)) report_error(LC_ERR_CACHE_INDEX, kClassAppend);
    return page < c.n_pages ? static_cast<int>(page) : -1;
}

// A row by L lanes, so 32 / L rows at a time: keys' and values' of 16 / L
// heads, U times.  VEC: every row on both sides starts on the boundary of eight
// elements and holds whole eights.
template <int Q, bool VEC, int NI, int L, int U>
__global__ void __launch_bounds__(kApThreads) k_cache_append(const __grid_constant__ AppendArgs a) {
    constexpr int P = 16 / L;  // heads at a time
    const CacheArgs &c = a.c;
    start_after_prior();
    const int64_t thread = int64_t(blockIdx.x) * kApThreads + threadIdx.x;
    if (!a.slots && thread < c.n_seqs) {
        const int at = static_cast<int>(thread);
        const int n = cache_length(c, a.lengths, at, kClassAppend);
        const int m = a.counts ? min(max(a.counts[at], 0), a.n_new) : a.n_new;
        if ((a.counts && a.counts[at] != m) || m > c.cap - n) report_error(LC_ERR_CACHE_INDEX, kClassAppend);
        a.new_lengths[at] = n + min(m, c.cap - n);
    }
    const uint32_t item = static_cast<uint32_t>(thread / 32);
    if (item >= a.items) return;
    const uint32_t bt = fast_div(item, a.head_div);
    const int first = static_cast<int>(item - bt * a.head_div.d) * U * P, h0 = first + (threadIdx.x & 31) / (2 * L);
    const int b = static_cast<int>(fast_div(bt, a.new_div));
    const int t = static_cast<int>(bt - static_cast<uint32_t>(b) * a.n_new);
    int n = 0;
    if (!a.slots) {
        const int count = a.counts ? a.counts[b] : a.n_new;
        n = min(max(a.lengths[b], 0), c.cap);
        if (t >= min(count, c.cap - n)) return;
    }

    const int lane = threadIdx.x & (L - 1);
    const bool is_v = threadIdx.x & L;
    const int64_t head_stride = (is_v ? a.vst : a.kst)[2];
    const uint16_t *src = is_v ? a.v + b * a.vst[0] + t * a.vst[1] + h0 * head_stride
                               : a.k + b * a.kst[0] + t * a.kst[1] + h0 * head_stride;
    __align__(16) uint16_t w[U][8 * NI];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool on = h0 + u * P < c.heads;
            if constexpr (VEC) {
                uint4 q = make_uint4(0, 0, 0, 0);
                if (on && 8 * (lane + L * i) < c.dim)
                    q = *reinterpret_cast<const uint4 *>(src + u * P * head_stride + 8 * (lane + L * i));
                reinterpret_cast<uint4 *>(w[u])[i] = q;
            } else {
#pragma unroll
                for (int j = 8 * i; j < 8 * i + 8; ++j) {
                    const int e = lane + L * j;
                    w[u][j] = on && e < c.dim ? src[u * P * head_stride + e] : uint16_t(0);
                }
            }
        }
    int row;
    const int page = a.slots ? slot_page(c, a.slots[t], &row) : cache_page(c, b, n + t, &row, kClassAppend);
    if (page < 0) return;
    const int64_t *st = is_v ? c.vst : c.kst, *sst = is_v ? c.vss : c.kss;
    uint8_t *dst = (is_v ? c.v : c.k) + row_offset(st, page, h0, row) * (Q ? 1 : 2);
    float *scale_at = Q ? (is_v ? c.vs : c.ks) + row_offset(sst, page, h0, row) : nullptr;
    const int64_t dst_step = P * st[1] * (Q ? 1 : 2), scale_step = P * sst[1];
#pragma unroll
    for (int u = 0; u < U && first + u * P < c.heads; ++u, dst += dst_step, scale_at += Q ? scale_step : 0)
        put_row<Q, VEC, NI, L>(c.dim, dst, scale_at, h0 + u * P < c.heads, w[u]);
}

cudaError_t take_error_append(unsigned long long *v) { return take_module_error(v); }

namespace {

template <int Q, bool VEC, int NI, int L, int U>
int launch_append(AppendArgs &a, int64_t tokens, cudaStream_t cs) {
    constexpr int kHeads = U * 16 / L;
    const int per = (a.c.heads + kHeads - 1) / kHeads;
    a.items = static_cast<uint32_t>(tokens * per);
    a.head_div = make_fastdiv(static_cast<uint32_t>(per));
    const uint64_t threads = std::max<uint64_t>(uint64_t(a.items) * 32, a.c.n_seqs);
    return launch_after(reinterpret_cast<const void *>(&k_cache_append<Q, VEC, NI, L, U>),
                        static_cast<unsigned>((threads + kApThreads - 1) / kApThreads), kApThreads, 0, cs, &a);
}

template <int Q>
int launch_append_as(AppendArgs &a, int64_t tokens, bool vec, cudaStream_t cs) {
    if (!vec) return launch_append<Q, false, 2, 16, 1>(a, tokens, cs);
    // A head a warp until there are warps enough to fill the GPU, then four, and
    // of rows to quantise eight where there are as many heads and rows again.
    // The fewer lanes a row, the fewer instructions go into its scale and
    // addresses: prompts of 8966 tokens of 8 heads of 128 with 16 lanes a row
    // 14.9 us, 8 lanes 13.2, 4 lanes 11.9, 4 lanes and eight heads 11.8 (34 thousand
    // such tokens 43.8, 39.5 and 35.2, 4096 tokens 4.6, 4.4 and 4.8).
    const int64_t rows = tokens * a.c.heads;
    const bool many = rows >= kApMany;
    if constexpr (Q != 0) {
        if (many && a.c.heads >= 4) {
            const bool eight = a.c.heads > 4 && rows >= 2 * kApMany;
            if (a.c.dim > 128) return launch_append<Q, true, 4, 8, 2>(a, tokens, cs);
            if (a.c.dim > 64)
                return eight ? launch_append<Q, true, 4, 4, 2>(a, tokens, cs)
                             : launch_append<Q, true, 4, 4, 1>(a, tokens, cs);
            return eight ? launch_append<Q, true, 2, 4, 2>(a, tokens, cs)
                         : launch_append<Q, true, 2, 4, 1>(a, tokens, cs);
        }
    }
    const bool four = many && a.c.heads > 1;
    if (a.c.dim > 128)
        return four ? launch_append<Q, true, 2, 16, 4>(a, tokens, cs) : launch_append<Q, true, 2, 16, 1>(a, tokens, cs);
    return four ? launch_append<Q, true, 1, 16, 4>(a, tokens, cs) : launch_append<Q, true, 1, 16, 1>(a, tokens, cs);
}

}  // namespace

}  // namespace lc

extern "C" int lc_cache_append(const lc_paged_cache *cache, const void *k_new, const void *v_new, int32_t type,
                               const int64_t k_stride[3], const int64_t v_stride[3], int32_t n_new,
                               const int32_t *counts, const int32_t *lengths, int32_t *new_lengths,
                               lc_stream_t stream) {
    using namespace lc;
    AppendArgs a{};
    int st = check_cache(cache, true, &a.c);
    if (st) return st;
    if (n_new < 0) return LC_ERR_SHAPE;
    if (type != LC_CACHE_BF16 && type != LC_CACHE_F16) return LC_ERR_TYPE;
    const bool q8 = cache->type == LC_CACHE_E4M3;
    if (!q8 && type != cache->type) return LC_ERR_TYPE;
    if (cache->n_seqs == 0) return LC_OK;
    if (!lengths || !new_lengths || !k_stride || !v_stride || (n_new > 0 && (!k_new || !v_new))) return LC_ERR_NULL;
    // blocks read lengths and counts when others have written (no tokens: one thread a sequence does both)
    for (const int32_t *in : {lengths, counts})
        if (in && lists_meet(in, new_lengths, cache->n_seqs) && (n_new > 0 || in != new_lengths)) return LC_ERR_OVERLAP;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) % 2 ||
        (reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(lengths) |
         reinterpret_cast<uintptr_t>(new_lengths)) % 4)
        return LC_ERR_ALIGN;
    const int64_t ext[3] = {cache->n_seqs, std::max(n_new, 1), cache->n_kv_heads};
    st = check_reach(3, ext, k_stride, cache->head_dim);
    if (!st) st = check_reach(3, ext, v_stride, cache->head_dim);
    if (st) return st;
    int64_t rows;
    if (!mul_ok_ext(ext[0] * ext[2], n_new, &rows) || rows > (int64_t(1) << 31) - 1) return LC_ERR_OVERFLOW;
    a.k = static_cast<const uint16_t *>(k_new);
    a.v = static_cast<const uint16_t *>(v_new);
    for (int i = 0; i < 3; ++i) {
        a.kst[i] = k_stride[i];
        a.vst[i] = v_stride[i];
    }
    a.counts = counts;
    a.lengths = lengths;
    a.new_lengths = new_lengths;
    a.n_new = n_new;
    a.new_div = make_fastdiv(static_cast<uint32_t>(std::max(n_new, 1)));
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    const int eb = cache_elem_bytes(cache->type);
    const bool vec = cache->head_dim % 8 == 0 && rows_aligned(k_new, 3, ext, k_stride, 2, 16) &&
                     rows_aligned(v_new, 3, ext, v_stride, 2, 16) &&
                     rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 8 * eb) &&
                     rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 8 * eb);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int64_t tokens = ext[0] * n_new;
    if (!q8) return launch_append_as<0>(a, tokens, vec, cs);
    return type == LC_CACHE_BF16 ? launch_append_as<1>(a, tokens, vec, cs) : launch_append_as<2>(a, tokens, vec, cs);
}

extern "C" int lc_cache_append_packed(const lc_paged_cache *cache, const void *k_new, const void *v_new, int32_t type,
                                      const int64_t k_stride[2], const int64_t v_stride[2], int32_t n_tokens,
                                      const int64_t *slots, lc_stream_t stream) {
    using namespace lc;
    AppendArgs a{};
    int st = check_cache(cache, true, &a.c);
    if (st) return st;
    if (n_tokens < 0) return LC_ERR_SHAPE;
    if (type != LC_CACHE_BF16 && type != LC_CACHE_F16) return LC_ERR_TYPE;
    const bool q8 = cache->type == LC_CACHE_E4M3;
    if (!q8 && type != cache->type) return LC_ERR_TYPE;
    if (n_tokens == 0 || cache->n_pages == 0) return LC_OK;
    if (!k_new || !v_new || !k_stride || !v_stride || !slots) return LC_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) % 2 ||
        reinterpret_cast<uintptr_t>(slots) % 8)
        return LC_ERR_ALIGN;
    const int64_t ext[2] = {n_tokens, cache->n_kv_heads};
    st = check_reach(2, ext, k_stride, cache->head_dim);
    if (!st) st = check_reach(2, ext, v_stride, cache->head_dim);
    if (st) return st;
    if (ext[0] * ext[1] > (int64_t(1) << 31) - 1) return LC_ERR_OVERFLOW;
    a.k = static_cast<const uint16_t *>(k_new);
    a.v = static_cast<const uint16_t *>(v_new);
    for (int i = 0; i < 2; ++i) {
        a.kst[i + 1] = k_stride[i];
        a.vst[i + 1] = v_stride[i];
    }
    a.slots = slots;
    a.n_new = n_tokens;
    a.new_div = make_fastdiv(static_cast<uint32_t>(n_tokens));
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    const int eb = cache_elem_bytes(cache->type);
    const bool vec = cache->head_dim % 8 == 0 && rows_aligned(k_new, 2, ext, k_stride, 2, 16) &&
                     rows_aligned(v_new, 2, ext, v_stride, 2, 16) &&
                     rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 8 * eb) &&
                     rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 8 * eb);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!q8) return launch_append_as<0>(a, n_tokens, vec, cs);
    return type == LC_CACHE_BF16 ? launch_append_as<1>(a, n_tokens, vec, cs) : launch_append_as<2>(a, n_tokens, vec, cs);
}
