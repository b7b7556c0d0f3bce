// Page tables that hold the pages of the sequences' lengths, and the slot of every
// packed token (lc_cache_reserve).
//
// What each sequence has and wants, and the sums over the sequences before it (pages
// given back, pages taken, tokens), decide where every page and token goes; every
// block of the cluster works them out for itself, since they are a few numbers a
// sequence: one pass of sums where all are served, else one after another.  Pages
// given back are written to the stack first, then the cluster meets, then tables and slots
// are written, each block its share.  A sequence's pages come first in its row, so
// what it has is found by looking where its length says, and else by a search of 32
// places at a time.
//
// What bounds it is the chain of dependent reads (length, row, stack, page), not the
// bytes: a step of 64 sequences is a block of 256 threads, whose barriers are
// cheaper than 1024's; many tokens or a table written anew take a cluster, every thread with
// kRsAtOnce reads on the way (256 sequences with 65792 tokens: 14.4 us, with four reads the same, with two 16.7, with
// a row of 1024 pages by one read after another a lane 20.7; 64 sequences of a token: 5.8 us).  Clusters of 16
// changed nothing.
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace lc {

namespace cg = cooperative_groups;

constexpr uint32_t kClassReserve = 0xf6;
constexpr int kRsThreads = 1024, kRsFew = 256;  // few: of a block for up to as many sequences
constexpr int kRsCluster = 8;
constexpr int kRsAtOnce = 8;

struct ReserveArgs {
    const int32_t *table, *lengths, *counts, *n_free;
    int32_t *new_table, *free, *new_n_free, *new_lengths, *starts, *positions, *seqs;
    int64_t *slots;
    int64_t table_stride, new_stride, free_size;
    int32_t n_seqs, per, page, n_tokens;
    FastDiv page_div;
};

// Sum of x over the threads before this one and its own; `all`: over the block.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *warps, T *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T w = lane < static_cast<int>(blockDim.x >> 5) ? warps[lane] : T(0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T o = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += o;
        }
        warps[lane] = w;
    }
    __syncthreads();
    *all = warps[31];
    return x + (warp ? warps[warp - 1] : T(0));
}

// The same where not all are served: the tokens of those who are (first, start and *pages_taken: theirs).
__device__ __noinline__ int reserve_in_turn(const ReserveArgs &a, const int *held, int *want, int *first, int *count, int *start,
                                            int *warps, int64_t *wide, int top, int *pages_taken) {
    const int t = threadIdx.x, threads = blockDim.x;
    auto error = [&] {
        if (blockIdx.x == 0) report_error(LC_ERR_CACHE_INDEX, kClassReserve);
    };
    int all;
    // who gets pages: in order, as long as they last, and whoever needs none
    int taken = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += threads) {
        const int b = b0 + t;
        int need = 0;
        if (b < a.n_seqs && count[b] >= 0) need = max(want[b] - held[b], 0);
        const int upto = block_scan(need, warps, &all);
        if (need > 0 && taken + int64_t(upto) > top) {
            error();
            count[b] = -1;
        }
        taken += all;
        __syncthreads();
    }
    // tokens, as far as the packed lists go
    int64_t asked = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += threads) {
        const int b = b0 + t;
        const int64_t c = b < a.n_seqs ? max(count[b], 0) : 0;
        int64_t most;
        const int64_t upto = block_scan(c, wide, &most);
        if (c > 0 && asked + upto > a.n_tokens) {
            error();
            count[b] = -1;
        }
        asked += most;
        __syncthreads();
    }
    // where pages and tokens of those who are served begin
    int tokens = 0;
    taken = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += threads) {
        const int b = b0 + t;
        int need = 0, c = 0;
        if (b < a.n_seqs) {
            if (count[b] < 0) want[b] = min(want[b], held[b]);  // (what it gave back above stays given)
            need = max(want[b] - held[b], 0);
            c = max(count[b], 0);
        }
        const int pages = block_scan(need, warps, &all);
        if (b < a.n_seqs) first[b] = taken + pages - need;
        taken += all;
        const int upto = block_scan(c, warps, &all);
        if (b < a.n_seqs) start[b] = tokens + upto - c;
        tokens += all;
    }
    *pages_taken = taken;
    return tokens;
}

__global__ void __launch_bounds__(kRsThreads) k_cache_reserve(const __grid_constant__ ReserveArgs a) {
    extern __shared__ int shared[];
    __shared__ int warps[32], searches;
    __shared__ int64_t wide[32];
    __shared__ int4 sums[2][32];
    __shared__ uint32_t token_sums[2][32];
    int *const held = shared, *const want = held + a.n_seqs, *const first = want + a.n_seqs;  // pages; pages taken before
    int *const count = first + a.n_seqs, *const start = count + a.n_seqs;                      // tokens; n_seqs + 1
    int *const back = start + a.n_seqs + 1, *const length = back + a.n_seqs;                    // pages given back before
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, threads = blockDim.x;
    const int blocks = gridDim.x, block = blockIdx.x;
    const int cap = a.per * a.page;
    auto error = [&] {
        if (block == 0) report_error(LC_ERR_CACHE_INDEX, kClassReserve);
    };
    auto pages_of = [&](int tokens) { return static_cast<int>(fast_div(tokens + a.page - 1, a.page_div)); };
    if (t == 0) searches = 0;
    start_after_prior();
    const int free_raw = *a.n_free;
    __syncthreads();
    // what every sequence has: looked for where its length says, searched for where it is not there
    for (int b = t; b < a.n_seqs; b += threads) {
        const int n = a.lengths[b], m = a.counts[b], len = min(max(n, 0), cap);
        length[b] = len;
        const int32_t *row = a.table + b * a.table_stride;
        const int guess = pages_of(len);
        const bool right = (guess == 0 || row[guess - 1] >= 0) && (guess == a.per || row[guess] < 0);
        held[b] = guess;
        int c = max(m, 0);
        if (n != len || m < 0) error();
        if (c > cap - len) {
            error();
            c = -1;  // refused
        }
        count[b] = c;
        if (!right) first[atomicAdd(&searches, 1)] = b;
    }
    __syncthreads();
    for (int i = warp; i < searches; i += threads / 16) {  // two at a time
        const int other = min(i + threads / 32, searches - 1), b[2] = {first[i], first[other]};
        int lo[2] = {0, 0}, hi[2] = {a.per, a.per};  // pages before lo, none from hi on
        while (lo[0] < hi[0] || lo[1] < hi[1]) {
            int step[2];
            bool there[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                step[k] = (hi[k] - lo[k] + 31) / 32;
                const int at = lo[k] + lane * step[k];
                there[k] = at < hi[k] && a.table[b[k] * a.table_stride + at] >= 0;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int n = __popc(__ballot_sync(0xffffffffu, there[k]));
                if (n == 0) {
                    hi[k] = lo[k];
                } else {
                    const int last = lo[k] + (n - 1) * step[k];  // a page there
                    hi[k] = min(hi[k], last + step[k]);
                    lo[k] = last + 1;
                }
            }
        }
        if (lane < 2) held[b[lane]] = lo[lane];
    }
    __syncthreads();
    const int n_free = static_cast<int>(min(int64_t(max(free_raw, 0)), a.free_size));
    if (free_raw != n_free && t == 0) error();
    // pages given back, pages taken and tokens, in the sequences' order, as if all were served
    int sum = 0, taken = 0;
    int64_t asked = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += threads) {
        const int b = b0 + t;
        // (tokens in 32 bits, which wrap, and their halves' sums, which tell whether they did)
        const int warps_used = min((a.n_seqs - b0 + 31) / 32, threads / 32);
        int over = 0, need = 0;
        uint32_t c = 0;
        if (b < a.n_seqs) {
            want[b] = count[b] < 0 ? held[b] : pages_of(length[b] + count[b]);
            over = max(held[b] - want[b], 0);
            need = max(want[b] - held[b], 0);
            c = max(count[b], 0);
        }
        int over_upto = over, need_upto = need;
        uint32_t c_upto = c;
        if (warp < warps_used) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, over_upto, d), n = __shfl_up_sync(0xffffffffu, need_upto, d);
                const uint32_t m = __shfl_up_sync(0xffffffffu, c_upto, d);
                if (lane >= d) {
                    over_upto += o;
                    need_upto += n;
                    c_upto += m;
                }
            }
            const uint32_t low = __reduce_add_sync(0xffffffffu, c & 0xffff), high = __reduce_add_sync(0xffffffffu, c >> 16);
            if (lane == 31) {
                sums[b0 ? 1 : 0][warp] = make_int4(over_upto, need_upto, static_cast<int>(low), static_cast<int>(high));
                token_sums[b0 ? 1 : 0][warp] = c_upto;
            }
        }
        __syncthreads();
        // what the warps before have, and all of them
        int4 of = make_int4(0, 0, 0, 0);
        uint32_t tokens_of = 0;
        if (lane < warps_used) {
            of = sums[b0 ? 1 : 0][lane];
            tokens_of = token_sums[b0 ? 1 : 0][lane];
        }
        const int over_all = __reduce_add_sync(0xffffffffu, of.x), need_all = __reduce_add_sync(0xffffffffu, of.y);
        const int64_t c_all = static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(of.z))) +
                              (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(of.w))) << 16);
        if (warp < warps_used) {
            const bool earlier = lane < warp;
            over_upto += __reduce_add_sync(0xffffffffu, earlier ? of.x : 0);
            need_upto += __reduce_add_sync(0xffffffffu, earlier ? of.y : 0);
            c_upto += __reduce_add_sync(0xffffffffu, earlier ? tokens_of : 0u);
        }
        if (b0) __syncthreads();  // (the second set of sums is used again)
        if (b < a.n_seqs) {
            back[b] = sum + over_upto - over;
            first[b] = taken + need_upto - need;
            start[b] = static_cast<int>(static_cast<uint32_t>(asked) + c_upto - c);
        }
        sum += over_all;
        taken += need_all;
        asked += c_all;
    }
    const int top = static_cast<int>(min(int64_t(n_free) + sum, a.free_size));
    if (n_free + int64_t(sum) > a.free_size && t == 0) error();
    int tokens = static_cast<int>(asked);
    if (taken > top || asked > a.n_tokens) {
        tokens = reserve_in_turn(a, held, want, first, count, start, warps, wide, top, &taken);
    }
    if (t == 0) start[a.n_seqs] = tokens;
    __syncthreads();
    // pages given back
    for (int b = block * (threads / 32) + warp; b < a.n_seqs; b += blocks * (threads / 32)) {
        const int32_t *row = a.table + b * a.table_stride;
        for (int j0 = want[b] + lane; j0 < held[b]; j0 += 32 * kRsAtOnce) {
            int x[kRsAtOnce];
#pragma unroll
            for (int i = 0; i < kRsAtOnce; ++i) x[i] = j0 + 32 * i < held[b] ? row[j0 + 32 * i] : -1;
#pragma unroll
            for (int i = 0; i < kRsAtOnce; ++i) {
                const int64_t at = int64_t(n_free) + back[b] + j0 + 32 * i - want[b];
                if (j0 + 32 * i < held[b] && at < a.free_size) a.free[at] = x[i];
            }
        }
    }
    if (blocks > 1) {
        cg::this_cluster().sync();
    } else {
        __syncthreads();
    }
    auto page_at = [&](int b, int j) {  // what is not in the old table comes off the stack
        return j < held[b] ? a.table[b * a.table_stride + j] : a.free[top - 1 - (first[b] + j - held[b])];
    };
    const bool in_place = a.new_table == a.table;
    for (int b = block * (threads / 32) + warp; b < a.n_seqs; b += blocks * (threads / 32)) {
        int32_t *row = a.new_table + b * a.new_stride;
        const int upto = in_place ? max(held[b], want[b]) : a.per;
        for (int j0 = (in_place ? min(held[b], want[b]) : 0) + lane; j0 < upto; j0 += 32 * kRsAtOnce) {
            int x[kRsAtOnce];
#pragma unroll
            for (int i = 0; i < kRsAtOnce; ++i) x[i] = j0 + 32 * i < want[b] ? page_at(b, j0 + 32 * i) : -1;
#pragma unroll
            for (int i = 0; i < kRsAtOnce; ++i)
                if (j0 + 32 * i < upto) row[j0 + 32 * i] = x[i];
        }
        if (lane == 0) a.new_lengths[b] = length[b] + max(count[b], 0);
    }
    const int stride = blocks * threads;
    for (int b = block * threads + t; b <= a.n_seqs; b += stride) a.starts[b] = start[b];
    if (block == 0 && t == 0) *a.new_n_free = top - taken;
    // a warp 32 x kRsAtOnce tokens in a row
    for (int64_t at = (int64_t(block) * (threads / 32) + warp) * 32 * kRsAtOnce; at < a.n_tokens; at += int64_t(stride) * kRsAtOnce) {
        const int i0 = static_cast<int>(at);
        // the sequences of the first and the last of them, by half a warp each: the last that begins there or before
        int lo = 0, hi = a.n_seqs;
        const int64_t edge = lane < 16 ? at : at + 32 * kRsAtOnce - 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (start[mid] <= edge) lo = mid;
            else hi = mid;
        }
        const int from = __shfl_sync(0xffffffffu, lo, 0), upto = __shfl_sync(0xffffffffu, lo, 31) + 1;
        int page[kRsAtOnce], row[kRsAtOnce], position[kRsAtOnce], seq[kRsAtOnce];
#pragma unroll
        for (int k = 0; k < kRsAtOnce; ++k) {
            const int i = i0 + k * 32 + lane;
            page[k] = position[k] = seq[k] = -1;
            row[k] = 0;
            if (at + k * 32 + lane < tokens) {
                lo = from;
                hi = upto;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (start[mid] <= i) lo = mid;
                    else hi = mid;
                }
                seq[k] = lo;
                position[k] = length[lo] + i - start[lo];
                const int j = static_cast<int>(fast_div(position[k], a.page_div));
                row[k] = position[k] - j * a.page;
                page[k] = page_at(lo, j);
            }
        }
#pragma unroll
        for (int k = 0; k < kRsAtOnce; ++k) {
            const int64_t i = at + k * 32 + lane;
            if (i < a.n_tokens) {
                a.slots[i] = page[k] >= 0 ? int64_t(page[k]) * a.page + row[k] : -1;
                a.positions[i] = position[k];
                a.seqs[i] = seq[k];
            }
        }
    }
}

cudaError_t take_error_reserve(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

extern "C" int lc_cache_reserve(const lc_cache_reservation *r, lc_stream_t stream) {
    using namespace lc;
    if (!r) return LC_ERR_NULL;
    if (r->n_seqs < 0 || r->n_seqs > LC_CACHE_MAX_RESERVED || r->pages_per_seq < 0 || r->page_size < 1 ||
        r->max_tokens < 0 || r->free_size < 0)
        return LC_ERR_SHAPE;
    if (int64_t(r->page_size) * r->pages_per_seq > 0x7fff0000 || r->free_size > 0x7fff0000 ||
        int64_t(r->n_seqs) * r->pages_per_seq > 0x7fff0000)
        return LC_ERR_OVERFLOW;
    if (!r->n_free || !r->new_n_free || !r->starts || (r->free_size > 0 && !r->free) ||
        (r->n_seqs > 0 && (!r->lengths || !r->counts || !r->new_lengths)) ||
        (r->n_seqs > 0 && r->pages_per_seq > 0 && (!r->page_table || !r->new_table)) ||
        (r->max_tokens > 0 && (!r->slots || !r->positions || !r->seqs)))
        return LC_ERR_NULL;
    uintptr_t words = 0;
    for (const void *p : {static_cast<const void *>(r->page_table), static_cast<const void *>(r->lengths),
                          static_cast<const void *>(r->counts), static_cast<const void *>(r->n_free),
                          static_cast<const void *>(r->new_table), static_cast<const void *>(r->free),
                          static_cast<const void *>(r->new_n_free), static_cast<const void *>(r->new_lengths),
                          static_cast<const void *>(r->starts), static_cast<const void *>(r->positions),
                          static_cast<const void *>(r->seqs)})
        words |= reinterpret_cast<uintptr_t>(p);
    if (words % 4 || reinterpret_cast<uintptr_t>(r->slots) % 8) return LC_ERR_ALIGN;
    const int64_t ext[1] = {std::max(r->n_seqs, 1)};
    int st = check_reach(1, ext, &r->table_stride, r->pages_per_seq);
    if (!st) st = check_reach(1, ext, &r->new_table_stride, r->pages_per_seq);
    if (st) return st;
    if (!rows_apart(1, ext, &r->new_table_stride, r->pages_per_seq)) return LC_ERR_NOT_INJECTIVE;
    // what is written lies apart from what is read and from one another, but for a table changed in place
    struct Range {
        const void *p;
        int64_t bytes;
    };
    const int64_t n = r->n_seqs;
    const bool in_place = r->new_table == r->page_table && (n <= 1 || r->table_stride == r->new_table_stride);
    const Range out[] = {{r->new_table, n && r->pages_per_seq ? ((n - 1) * r->new_table_stride + r->pages_per_seq) * 4 : 0},
                         {r->free, int64_t(r->free_size) * 4},
                         {r->new_n_free, 4},
                         {r->new_lengths, n * 4},
                         {r->starts, (n + 1) * 4},
                         {r->slots, int64_t(r->max_tokens) * 8},
                         {r->positions, int64_t(r->max_tokens) * 4},
                         {r->seqs, int64_t(r->max_tokens) * 4}};
    const Range in[] = {{r->page_table, in_place || !n || !r->pages_per_seq ? 0 : ((n - 1) * r->table_stride + r->pages_per_seq) * 4},
                        {r->lengths, n * 4},
                        {r->counts, n * 4},
                        {r->n_free, 4}};
    auto meet = [](const Range &x, const Range &y) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(x.p), q = reinterpret_cast<uintptr_t>(y.p);
        return x.bytes > 0 && y.bytes > 0 && p < q + y.bytes && q < p + x.bytes;
    };
    for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
        for (const Range &x : in)
            if (meet(out[i], x)) return LC_ERR_OVERLAP;
        for (size_t j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return LC_ERR_OVERLAP;
    }
    ReserveArgs a{};
    a.table = r->page_table;
    a.new_table = r->new_table;
    a.table_stride = r->table_stride;
    a.new_stride = r->new_table_stride;
    a.lengths = r->lengths;
    a.counts = r->counts;
    a.free = r->free;
    a.free_size = r->free_size;
    a.n_free = r->n_free;
    a.new_n_free = r->new_n_free;
    a.new_lengths = r->new_lengths;
    a.starts = r->starts;
    a.slots = r->slots;
    a.positions = r->positions;
    a.seqs = r->seqs;
    a.n_seqs = r->n_seqs;
    a.per = r->pages_per_seq;
    a.page = r->page_size;
    a.n_tokens = r->max_tokens;
    a.page_div = make_fastdiv(static_cast<uint32_t>(r->page_size));
    const int smem = (7 * r->n_seqs + 1) * 4;
    int sms = 0, per_sm = 0;
    const void *fn = reinterpret_cast<const void *>(&k_cache_reserve);
    if (prepare(fn, kRsThreads, smem, smem, &sms, &per_sm) != cudaSuccess) return LC_ERR_CUDA;
    const int64_t work = (in_place ? 0 : n * r->pages_per_seq) + r->max_tokens;
    const int blocks = work > 8 * kRsThreads ? kRsCluster : 1, threads = blocks == 1 && n <= kRsFew ? kRsFew : kRsThreads;
    return launch_after(fn, blocks, threads, smem, reinterpret_cast<cudaStream_t>(stream), &a, blocks);
}
