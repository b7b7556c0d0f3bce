// Cache attention: the joining of parts, the workspace and the C entry points
// (lc_cache_attend; the main kernels are cache_attend.cuh).
#include "cache_attend.cuh"

namespace lc {

// The whole row's maximum and sum of exponentials of a unit that was cut, by
// one warp from its parts.
struct Parts {
    int first, count;
    // the unit's first part is its run's second (the unit starts there), the
    // others their runs' first
    __device__ __forceinline__ int slot(int i) const { return 2 * (first + i) + (i == 0); }
};

__device__ __forceinline__ float2 join_ml(const AttendArgs &a, const Parts &p, int row) {
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < p.count; i += 32 * kAhead) {
        float2 v[kAhead];
        float most = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            v[k] = i + 32 * k < p.count ? a.part_ml[int64_t(p.slot(i + 32 * k)) * a.part_rows + row]
                                        : make_float2(-INFINITY, 0.f);
            most = fmaxf(most, v[k].x);
        }
        const float safe = most == -INFINITY ? 0.f : most;
        sum *= exp2_fast(top - safe);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) sum += v[k].y * exp2_fast(v[k].x - safe);
        top = most;
    }
    float most = top;
#pragma unroll
    for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    sum *= exp2_fast(top - (most == -INFINITY ? 0.f : most));
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return make_float2(most, sum);
}

// scores[b, h, j] += sum over the group's query heads of 2^(logit - lse), for
// one chunk of slots.
template <bool F16>
__device__ __forceinline__ void add_scores(const AttendArgs &a, uint32_t at, float *lse) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, threads = blockDim.x;
    const int units = a.c.heads * a.row_blocks;
    const uint32_t unit = fast_div(at, a.chunk_div);
    const int chunk = static_cast<int>(at - unit * a.chunk_div.d);
    const int b = static_cast<int>(fast_div(unit, a.head_div)), h = static_cast<int>(unit) - b * a.c.heads;
    int n;
    const int lo = seen_from(a, b, &n);
    const int i0 = chunk * threads * kScorePer;
    if (i0 >= n - lo) return;
    float w[kScorePer] = {};
    for (int g0 = 0; g0 < a.group; g0 += threads) {
        // the rows' log sums, a warp each
        const int gn = min(a.group - g0, threads);
        __syncthreads();
        for (int g = warp; g < gn; g += threads / 32) {
            const int rb = (g0 + g) / kAtRows;
            const int2 split = a.split[int64_t(b) * units + h * a.row_blocks + rb];
            float z;
            if (split.x < 0) {
                z = a.lse2[int64_t(b) * a.q_heads + h * a.group + g0 + g];
            } else {
                const float2 v = join_ml(a, Parts{split.x, split.y - split.x + 1}, g0 + g - rb * kAtRows);
                z = log_sum<F16>(v.x, v.y);
            }
            if (lane == 0) lse[g] = z;
        }
        __syncthreads();
        const float *x = a.logits + (int64_t(b) * a.q_heads + h * a.group + g0) * a.logit_stride + i0 + t;
#pragma unroll 2
        for (int g = 0; g < gn; ++g, x += a.logit_stride) {
            const float z = lse[g];
            float y[kScorePer];
#pragma unroll
            for (int k = 0; k < kScorePer; ++k) y[k] = i0 + t + k * threads < n - lo ? x[k * threads] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kScorePer; ++k) w[k] += weight_of(y[k], z);
        }
    }
    float *to = a.scores + b * a.sst[0] + h * a.sst[1] + lo + i0 + t;
#pragma unroll
    for (int k = 0; k < kScorePer; ++k)
        if (i0 + t + k * threads < n - lo) to[k * threads] += w[k];
}

// The first score_blocks blocks (with scores), one a (sequence, key head,
// chunk of slots), add the weights.  The join_blocks after them join the parts
// of the rows (sequence, query head) whose units were cut, in their order, and
// write the zeros of sequences with nothing to see: warp w of the i-th takes
// row i + w join_blocks (w < join_rows); a row of many parts is left for the
// whole block, several parts at a time.
template <bool F16>
__global__ void __launch_bounds__(kJoinMost) k_attend_join(const __grid_constant__ AttendArgs a) {
    extern __shared__ float acc[];  // four floats a thread
    __shared__ int whole_block[kJoinRows];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, threads = blockDim.x;
    start_after_prior();
    if (blockIdx.x < a.score_blocks) {
        add_scores<F16>(a, blockIdx.x, acc);
        return;
    }
    const int units = a.c.heads * a.row_blocks, quads = a.part_pitch / 4;
    struct Row {
        int b, hq, row;
        Parts parts;  // count 0: nothing to join
        int n, lo;
    };
    auto row_of = [&](int w) {
        Row r{};
        const uint32_t at = blockIdx.x - a.score_blocks + static_cast<uint32_t>(w) * a.join_blocks;
        if (at >= static_cast<uint32_t>(a.c.n_seqs) * a.q_heads) {
            r.n = 1;  // no such row
            return r;
        }
        r.b = static_cast<int>(fast_div(at, a.q_div));
        r.hq = static_cast<int>(at) - r.b * a.q_heads;
        const int h = static_cast<int>(fast_div(r.hq, a.group_div)), g = r.hq - h * a.group;
        r.row = g % kAtRows;
        const int2 split = a.split[int64_t(r.b) * units + h * a.row_blocks + g / kAtRows];
        r.lo = seen_from(a, r.b, &r.n);
        if (r.lo < r.n && split.x >= 0) r.parts = Parts{split.x, split.y - split.x + 1};
        return r;
    };
    auto part = [&](const Row &r, int i, int col, float safe, float4 &y) {
        const int64_t at = int64_t(r.parts.slot(i)) * a.part_rows + r.row;
        const float f = exp2_fast(a.part_ml[at].x - safe);
        const float4 z = *reinterpret_cast<const float4 *>(a.part + at * a.part_pitch + col);
        y.x += z.x * f;
        y.y += z.y * f;
        y.z += z.z * f;
        y.w += z.w * f;
    };
    auto put = [&](const Row &r, int col, float x) {
        if (col < a.c.dim) a.out[r.b * a.ost[0] + r.hq * a.ost[1] + col] = static_cast<uint16_t>(pack2<F16>(x, 0.f));
    };
    auto put_lse = [&](const Row &r, float2 v) {
        if (a.lse) a.lse[r.b * a.lse_stride + r.hq] = log_sum<F16>(v.x, v.y) * kLn2;
    };
    if (warp < a.join_rows) {
        const Row r = row_of(warp);
        const bool many = r.parts.count > (a.join_rows > 1 ? kJoinFew : 0);
        if (lane == 0) whole_block[warp] = many;
        if (r.lo >= r.n) {
            for (int i = lane; i < a.c.dim; i += 32) put(r, i, 0.f);
            if (lane == 0) put_lse(r, make_float2(0.f, 0.f));
        } else if (r.parts.count && !many) {
            const float2 v = join_ml(a, r.parts, r.row);
            const float safe = v.x == -INFINITY ? 0.f : v.x, f = v.y == 0.f ? 0.f : 1.f / v.y;
            for (int col = 4 * lane; col < a.part_pitch; col += 128) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int i = 0; i < r.parts.count; ++i) part(r, i, col, safe, y);
                put(r, col, y.x * f);
                put(r, col + 1, y.y * f);
                put(r, col + 2, y.z * f);
                put(r, col + 3, y.w * f);
            }
            if (lane == 0) put_lse(r, v);
        }
    }
    __syncthreads();
    const int lanes = threads / quads;  // parts read at a time; threads past them only write
    const int col = t % quads * 4, first = t / quads;
    for (int w = 0; w < a.join_rows; ++w) {
        if (!whole_block[w]) continue;
        const Row r = row_of(w);
        const float2 v = join_ml(a, r.parts, r.row);  // by every warp for itself
        const float safe = v.x == -INFINITY ? 0.f : v.x, f = v.y == 0.f ? 0.f : 1.f / v.y;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = first < lanes ? first : r.parts.count; i < r.parts.count; i += lanes) part(r, i, col, safe, y);
        __syncthreads();
        *reinterpret_cast<float4 *>(acc + first * a.part_pitch + col) = y;
        __syncthreads();
        for (int i = t; i < a.c.dim; i += threads) {
            float s = 0.f;
            for (int k = 0; k < lanes; ++k) s += acc[k * a.part_pitch + i];
            put(r, i, s * f);
        }
        if (t == 0) put_lse(r, v);
    }
}

cudaError_t take_error_attend(unsigned long long *v) { return take_module_error(v); }

int launch_attend_bf16(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs);
int launch_attend_f16(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs);
int launch_attend_e4m3(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs);

namespace {

// How a call of these sizes goes: a block or a cluster a unit, or runs; with
// runs, or with scores, it needs a workspace of these offsets and this end.
struct AttendSpace {
    bool vec;      // rows of the pools are whole 16-byte words on 16-byte boundaries
    bool warp_units;  // a unit a warp
    int unit_blocks;  // 0: by runs
    int part_rows, dim;
    int64_t part, ml, split, lse2, logits, end, logit_stride;
};

bool attend_space(const lc_paged_cache &cache, const CacheArgs &c, int q_heads, int window, bool scores,
                  AttendSpace *s) {
    const int eb = cache_elem_bytes(cache.type);
    const int64_t pool[3] = {cache.n_pages, cache.n_kv_heads, cache.page_size};
    s->vec = c.dim * eb % 16 == 0 && rows_aligned(cache.k, 3, pool, cache.k_stride, eb, 16) &&
             rows_aligned(cache.v, 3, pool, cache.v_stride, eb, 16);
    s->dim = padded_dim(c.dim, s->vec);
    const int tok = step_slots(s->dim, cache_elem_bytes(cache.type)), group = q_heads / c.heads;
    const int64_t units = c.heads * ((int64_t(group) + kAtRows - 1) / kAtRows), heads = int64_t(c.n_seqs) * q_heads;
    // scores of a key head whose query heads are several units' need the
    // second launch
    s->unit_blocks = 0;
    s->warp_units = false;
    const int64_t steps = ((window ? std::min(window, c.cap) : c.cap) + int64_t(tok) - 1) / tok;
    if (s->vec && !(scores && group > kAtRows)) {
        const int64_t all = c.n_seqs * units;
        int n = 1;
        while (2 * n <= kUnitCluster && n * kAtWarps < steps && all * 2 * n <= kUnitBlocks) n *= 2;
        if (steps <= int64_t(kUnitSteps) * kAtWarps * n) {
            s->unit_blocks = n;
            const int64_t rounds = (all - 1) / kUnitBlocks + 1, deal = (steps + kAtWarps - 1) / kAtWarps;
            const int64_t warps = kAtWarps * kUnitBlocks;
            s->warp_units = n == 1 && unit_by_warp(s->dim, group) &&
                            std::max(all, warps) * (kUnitCost + steps) < warps * rounds * (kUnitCost + deal);
        }
    }
    s->part_rows = std::min(group, kAtRows);
    const int64_t parts = s->unit_blocks ? 0 : int64_t(2) * kAtMaxRuns * s->part_rows;
    s->part = 0;
    s->ml = s->part + parts * s->dim * 4;
    s->split = s->ml + round256(parts * 8);
    s->lse2 = round256(s->split + (s->unit_blocks ? 0 : c.n_seqs * units * 8));
    s->logits = round256(s->lse2 + (scores ? heads * 4 : 0));
    s->logit_stride = int64_t(c.cap) + tok;  // a unit's last step is written whole
    int64_t logits;
    if (!mul_ok_ext(heads, s->logit_stride * 4, &logits)) return false;
    return add_ok_ext(s->logits, scores ? logits : 0, &s->end) && s->end < int64_t(1) << 60;
}

}  // namespace

}  // namespace lc

extern "C" int64_t lc_cache_attend_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t with_scores) {
    lc::CacheArgs c;
    lc::AttendSpace s;
    if (lc::check_cache(cache, false, &c) || n_q_heads < 1 || n_q_heads % c.heads ||
        !lc::attend_space(*cache, c, n_q_heads, 0, with_scores != 0, &s))
        return -1;
    return s.end;
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
        (q->scores && a.c.cap > 0 && !rows_apart(2, kext, q->scores_stride, a.c.cap)))
        return LC_ERR_NOT_INJECTIVE;
    // a row of the queries' own buffer is written when all that read it have
    const bool in_place = q->out == q->q && (qext[0] == 1 || q->q_stride[0] == q->out_stride[0]) &&
                          (qext[1] == 1 || q->q_stride[1] == q->out_stride[1]);
    if (!in_place && rows_meet(q->q, q->q_stride, q->out, q->out_stride, qext, cache->head_dim, 2))
        return LC_ERR_OVERLAP;
    AttendSpace space;
    const int64_t chunks = (int64_t(a.c.cap) + kJoinLeast * kScorePer - 1) / (kJoinLeast * kScorePer);
    if (!attend_space(*cache, a.c, q->n_q_heads, q->window, q->scores != nullptr, &space) ||
        qext[0] * qext[1] > 0x3fffffff || (q->scores && chunks && kext[0] * kext[1] > 0x3fffffff / chunks))
        return LC_ERR_OVERFLOW;
    if (space.end > 0 && !q->workspace) return LC_ERR_NULL;
    if (space.end > q->workspace_bytes) return LC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(q->workspace) % 256) return LC_ERR_ALIGN;
    a.q = static_cast<const uint16_t *>(q->q);
    a.out = static_cast<uint16_t *>(q->out);
    a.lengths = q->lengths;
    a.mask = q->mask;
    a.lse = q->lse;
    a.scores = a.c.cap ? q->scores : nullptr;
    for (int i = 0; i < 2; ++i) {
        a.qst[i] = q->q_stride[i];
        a.ost[i] = q->out_stride[i];
        a.sst[i] = q->scores_stride[i];
    }
    a.mask_stride = q->mask_stride;
    a.lse_stride = q->lse_stride;
    a.q_heads = q->n_q_heads;
    a.group = q->n_q_heads / cache->n_kv_heads;
    a.row_blocks = (a.group + kAtRows - 1) / kAtRows;
    a.window = q->window;
    a.scale2 = q->scale * kLog2e;
    a.q_wide = a.c.dim % 4 == 0 && rows_aligned(q->q, 2, qext, q->q_stride, 2, 8);
    uint8_t *ws = static_cast<uint8_t *>(q->workspace);
    a.part = reinterpret_cast<float *>(ws + space.part);
    a.part_ml = reinterpret_cast<float2 *>(ws + space.ml);
    a.split = reinterpret_cast<int2 *>(ws + space.split);
    a.lse2 = reinterpret_cast<float *>(ws + space.lse2);
    a.logits = a.scores ? reinterpret_cast<float *>(ws + space.logits) : nullptr;
    a.logit_stride = space.logit_stride;
    a.part_rows = space.part_rows;
    a.part_pitch = space.dim;
    a.warp_units = space.warp_units;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    int runs = 0;
    const auto launch = cache->type == LC_CACHE_BF16  ? launch_attend_bf16
                        : cache->type == LC_CACHE_F16 ? launch_attend_f16
                                                      : launch_attend_e4m3;
    st = launch(a, space.unit_blocks, space.vec, &runs, cs);
    if (st || space.unit_blocks) return st;
    // a row a block, as wide as lets all rows run at once: few rows have many
    // parts each, which a wide block reads more of at a time; rows past that
    // share blocks of the least width, a warp each
    const int64_t rows = qext[0] * qext[1];
    int threads = kJoinMost;
    while (threads > kJoinLeast && rows * threads > 152 * 1024) threads /= 2;
    a.join_rows = rows * threads > 152 * 1024 ? kJoinRows : 1;
    a.join_blocks = static_cast<int32_t>((rows + a.join_rows - 1) / a.join_rows);
    const int chunks_of = a.scores ? (a.c.cap + threads * kScorePer - 1) / (threads * kScorePer) : 0;
    a.chunk_div = make_fastdiv(static_cast<uint32_t>(std::max(chunks_of, 1)));
    a.head_div = make_fastdiv(static_cast<uint32_t>(a.c.heads));
    a.q_div = make_fastdiv(static_cast<uint32_t>(a.q_heads));
    a.group_div = make_fastdiv(static_cast<uint32_t>(a.group));
    a.score_blocks = static_cast<uint32_t>(kext[0] * kext[1] * chunks_of);
    const int64_t blocks = int64_t(a.score_blocks) + a.join_blocks;
    const void *join = cache->type == LC_CACHE_F16 ? reinterpret_cast<const void *>(&k_attend_join<true>)
                                                   : reinterpret_cast<const void *>(&k_attend_join<false>);
    return launch_after(join, static_cast<unsigned>(blocks), threads, threads * 16, cs, &a);
}
