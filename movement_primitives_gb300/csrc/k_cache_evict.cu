// Eviction from a paged key-value cache by accumulated weight
// (lc_cache_evict).
//
// Per sequence and key head (a unit), of n > budget slots: the `recent` newest
// stay, and of the others the budget - recent of largest score, equal scores
// in slot order.
//
// select_slots, by a block or a cluster of blocks a unit, finds the score of
// the last slot kept by radix selection on an order-preserving 32-bit key
// (digits of 11, 11 and 10 bits from the top, the first one's histogram made
// as the scores come in), then writes the kept slots in ascending order
// (`kept`) with their scores.  The scores are read from memory once and their
// keys kept in shared memory; the blocks of a cluster take a run of slots each
// and add up their histograms through distributed shared memory.
//
// Small units select and move in one launch (k_evict_small); others select
// with k_evict_select and move with k_evict_move.
//
// k_evict_move moves the rows, 32 ranks (a chunk) a block at a time.  Rows
// move in place: the r-th kept slot goes to slot r, and kept[r] >= r, so slot
// r may still hold a row that a rank j < r has yet to read, never one of a
// later rank.  A chunk therefore reads its rows into shared memory without
// waiting, publishes that it has, and before writing waits for the chunks that
// hold the ranks of the slots it writes over (at most two, which the selection
// leaves in `rank_at`).  Chunks are handed out in order by an atomic counter,
// and waits go to lower chunks only, whose reads wait for nothing: no wait can
// be circular, whichever blocks run.  Every row that moves is read and written
// once.
//
// Measured on GB300: 15 sequences of up to 16384 bfloat16 slots of 8 heads cut
// to 4096, 403 MB moved, 90 us: the selection 18 us (bound by the latency of
// its passes over the keys, each a barrier of the block or cluster), the move 72
// us (5.6 TB/s).  One sequence of 131071 E4M3 slots cut to 32768, 138 MB, 59 us:
// 25 us of selection on 64 blocks, 34 us of rows of 128 bytes.  Four sequences of
// 1500 cut to 1024, 34 MB, in one launch 15.5 us.
#include <cooperative_groups.h>

#include <type_traits>

#include "cache_common.cuh"

namespace lc {

namespace cg = cooperative_groups;

constexpr int kSelBins = 2048;      // 64 groups of 32
constexpr int kSelRound = 2048;     // slots are dealt to blocks in so many
constexpr int kSelKeys = 48 * 1024; // keys a block holds in shared memory
constexpr int kSelEase = 16384;     // keys a block rather holds
constexpr int kSelCluster = 8;      // blocks of a unit at most
constexpr int kSelLeast = 4096;     // slots a block of a cluster has at least
constexpr int kSmThreads = 512;     // of a block that selects and moves
constexpr int kSmAhead = 4;         // words a thread reads at a time there
constexpr int kSmBlocks = 304;      // two an SM
constexpr int kSmSlots = 8192;      // of such a block's unit at most
constexpr int kSmMoved = 128 * 1024; // bytes that such a block moves at most, or twice that
constexpr int kMvThreads = 64;      // a warp a pool where the rows' places are found
constexpr int kMvRows = 32;         // ranks of a chunk (the selection writes rank_at once every 32 slots)

struct EvictArgs {
    CacheArgs c;
    const int32_t *lengths;
    const float *scores;
    float *new_scores;
    int32_t *kept, *new_lengths;
    int64_t sst[2], nst[2], kst[2];  // sequence, head
    int32_t budget, recent;
    int32_t chunks;          // of a unit: ceil(budget / kMvRows)
    FastDiv unit_div, head_div, word_div;  // units; key heads; words (VEC: of 16 bytes) of a row
    int32_t slices, held_keys;             // of k_evict_small; word_div is then of twice a slice's words
    uint64_t wait_ns;
    // workspace
    uint32_t *ticket;        // the next chunk
    uint32_t *done;          // [unit][chunk]: its rows have been read
    int32_t *rank_at;        // [unit][chunk + 1]: kept slots below slot kMvRows * chunk
};

// Larger scores have larger keys; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float s) {
    const uint32_t u = __float_as_uint(fmaxf(s, -INFINITY) + 0.f);  // the maximum is not the NaN
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// From the largest down: the one of 32 lanes' counts that holds the need-th,
// and how many of it are needed.
__device__ __forceinline__ int pick(uint32_t count, uint32_t *need) {
    const int lane = threadIdx.x & 31;
    uint32_t upto = count;  // lanes lane .. 31
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_down_sync(0xffffffffu, upto, o);
        if (lane + o < 32) upto += y;
    }
    const uint32_t above = upto - count;
    const int at = __ffs(__ballot_sync(0xffffffffu, above < *need && upto >= *need)) - 1;
    *need -= __shfl_sync(0xffffffffu, above, at);
    return at;
}

// Finds the slots that stay of one unit's first n > budget ones: stay(rank,
// slot, score) of each, and rank(k, r), the rank r of slot kMvRows k, for every
// such slot.  By THREADS threads, or with CLUSTER by a cluster of `parts`
// blocks, this one the `part`-th.  HELD: the keys of a block's slots fit its
// shared memory (`keys`); else every pass reads the scores again.
template <bool HELD, int THREADS, bool CLUSTER, typename Stay, typename Rank>
__device__ __forceinline__ void select_slots(const EvictArgs &a, int parts, int part, int n, const float *scores,
                                             uint32_t *keys, Stay &&stay, Rank &&rank) {
    constexpr int kWarps = THREADS / 32;
    __shared__ uint32_t hist[2][kSelBins], groups[2][64], chosen[3][3], counts[2];
    __shared__ uint2 warp_counts[kWarps];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // f of each of the first `count` blocks' copies of a shared array
    auto for_blocks = [&](int count, const uint32_t *own, auto &&f) {
        if constexpr (CLUSTER) {
#pragma unroll
            for (int r = 0; r < kSelCluster; ++r)
                if (r < count) f(static_cast<const uint32_t *>(cg::this_cluster().map_shared_rank(own, r)));
        } else if (count) {
            f(own);
        }
    };
    // this block's slots [s0, s1), a run of `run` for each warp
    const int rounds = (n - 1) / kSelRound + 1, each = (rounds + parts - 1) / parts, run = each * (kSelRound / kWarps);
    const int s0 = static_cast<int>(lmin(int64_t(part) * each * kSelRound, n));
    const int s1 = static_cast<int>(lmin(s0 + int64_t(each) * kSelRound, n));
    const int cand = n - a.recent;          // slots below it compete
    const int c1 = max(min(s1, cand), s0);  // this block's competing ones end there
    auto key_of = [&](int i) { return HELD ? keys[i - s0] : score_key(scores[i]); };

    // the key of the last slot kept among the competing, and how many with
    // that key stay
    uint32_t need = a.budget - a.recent, prefix = 0;
    const bool any = need > 0;
    for (int i = t; i < kSelBins; i += THREADS) hist[0][i] = 0;
    __syncthreads();
    // the first digit's histogram as the keys come in
#pragma unroll 8
    for (int i = s0 + t; i < s1; i += THREADS) {
        const uint32_t key = score_key(scores[i]);
        if (HELD) keys[i - s0] = key;
        if (any && i < c1) atomicAdd(&hist[0][key >> 21], 1u);
    }
    if (any) {
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
            const int shift = kShift[pass], bits = kBits[pass];
            uint32_t *mine = hist[pass & 1];  // the cluster may still read the other one
            if (pass) {
                for (int i = t; i < kSelBins; i += THREADS) mine[i] = 0;
                __syncthreads();
#pragma unroll 8
                for (int i = s0 + t; i < c1; i += THREADS) {
                    const uint32_t key = key_of(i);
                    if (key >> (shift + bits) == prefix) atomicAdd(&mine[key >> shift & ((1u << bits) - 1)], 1u);
                }
            }
            __syncthreads();
            // bins in 64 groups of 32: the cluster adds up the groups, then the bins of one
            for (int g = warp; g < 64; g += kWarps) {
                const uint32_t sum = __reduce_add_sync(0xffffffffu, mine[32 * g + lane]);
                if (lane == 0) groups[pass & 1][g] = sum;
            }
            if constexpr (CLUSTER)
                cg::this_cluster().sync();
            else
                __syncthreads();
            if (warp == 0) {
                uint32_t low = 0, high = 0, bin = 0, left = need;
                for_blocks(parts, groups[pass & 1], [&](const uint32_t *other) {
                    low += other[lane];
                    high += other[32 + lane];
                });
                const bool upper = __reduce_add_sync(0xffffffffu, high) >= left;
                if (!upper) left -= __reduce_add_sync(0xffffffffu, high);
                const int group = pick(upper ? high : low, &left) + (upper ? 32 : 0);
                for_blocks(parts, mine, [&](const uint32_t *other) { bin += other[32 * group + lane]; });
                if (lane == pick(bin, &left)) {
                    chosen[pass][0] = 32 * group + lane;
                    chosen[pass][1] = left;
                    chosen[pass][2] = bin == left;  // all of that digit stay
                }
            }
            __syncthreads();
            prefix = prefix << bits | chosen[pass][0];
            need = chosen[pass][1];
            if (chosen[pass][2]) {
                // every key from this prefix up stays (it is above 0: not all that compete stay),
                // none of a tie
                prefix = (prefix << shift) - 1;
                need = 0;
                break;
            }
        }
    } else {
        __syncthreads();
    }
    // Slots in order: `sure` are kept whatever else, of the `tied` ones the
    // first `need`.  Each warp counts its run's, then writes from the counts
    // before it.
    const int w0 = static_cast<int>(lmin(s0 + int64_t(warp) * run, s1));
    const int w1 = static_cast<int>(lmin(w0 + int64_t(run), s1));
    const uint32_t above = any ? prefix : 0xffffffffu;  // competing slots of larger keys are sure
    const bool ties = any && need > 0;
    uint32_t sure = 0, tied = 0;
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = key_of(i);
        sure += key > (i < c1 ? above : 0);  // (every score's key is above 0)
        if (ties) tied += i < c1 && key == prefix;
    }
    sure = __reduce_add_sync(0xffffffffu, sure);
    if (ties) tied = __reduce_add_sync(0xffffffffu, tied);
    if (lane == 0) warp_counts[warp] = make_uint2(sure, tied);
    __syncthreads();
    sure = tied = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint2 v = warp_counts[w];
        if (w < warp) {
            sure += v.x;
            tied += v.y;
        }
        if (CLUSTER && t == 0) {
            counts[0] = (w ? counts[0] : 0) + v.x;
            counts[1] = (w ? counts[1] : 0) + v.y;
        }
    }
    if constexpr (CLUSTER) {  // and the blocks before
        cg::this_cluster().sync();
        for_blocks(part, counts, [&](const uint32_t *other) {
            sure += other[0];
            tied += other[1];
        });
    }
    // 128 slots at a time, four adjacent ones a lane: the lanes' counts of sure
    // and (from bit 16) tied ones, scanned, give each its rank.  Most calls have
    // no ties to tell apart, and half the instructions.
    auto place = [&](auto with_ties) {
        constexpr bool TIES = decltype(with_ties)::value;
        for (int i0 = w0; i0 < w1; i0 += 128) {
            const int i = i0 + 4 * lane;
            uint32_t key[4] = {}, count = 0;
            if (i < w1) {
                if constexpr (HELD) {
                    *reinterpret_cast<uint4 *>(key) = *reinterpret_cast<const uint4 *>(keys + (i - s0));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i + j < w1) key[j] = score_key(scores[i + j]);
                }
            }
            bool is_sure[4], is_tied[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                is_sure[j] = key[j] > (i + j < c1 ? above : i + j < w1 ? 0u : 0xffffffffu);
                is_tied[j] = TIES && i + j < c1 && key[j] == prefix;
                count += (is_sure[j] ? 1u : 0u) + (is_tied[j] ? 1u << 16 : 0u);
            }
            uint32_t upto = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            uint32_t g = sure + (upto - count & 0xffff), e = tied + (upto - count >> 16);
            // every eighth lane's first slot starts 32 of them
            if ((lane & 7) == 0 && i < w1) rank(i / kMvRows, g + (TIES ? min(e, need) : 0));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (is_sure[j] || (is_tied[j] && e < need)) {
                    // a positive score is its key but for the top bit; others are read again
                    stay(g + (TIES ? min(e, need) : 0), i + j,
                         key[j] > 0x80000000u ? __uint_as_float(key[j] ^ 0x80000000u) : scores[i + j]);
                }
                g += is_sure[j];
                if (TIES) e += is_tied[j];
            }
            const uint32_t all_of = __shfl_sync(0xffffffffu, upto, 31);
            sure += all_of & 0xffff;
            tied += all_of >> 16;
        }
    };
    if (ties)
        place(std::true_type{});
    else
        place(std::false_type{});
    if constexpr (CLUSTER) cg::this_cluster().sync();  // no block leaves while another reads its shared memory
}

// THREADS: 512, two blocks an SM, or 1024.
template <bool HELD, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_evict_select(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = cluster.num_blocks(), part = cluster.block_rank();
    const int t = threadIdx.x;
    const int unit = blockIdx.x / parts;
    const int b = unit / a.c.heads, h = unit - b * a.c.heads;
    start_after_prior();
    const int n = cache_length(a.c, a.lengths, b, kClassEvict);
    const int m = min(n, a.budget);
    const float *scores = a.scores + b * a.sst[0] + h * a.sst[1];
    float *out = a.new_scores + b * a.nst[0] + h * a.nst[1];
    int32_t *kept = a.kept + b * a.kst[0] + h * a.kst[1];
    int32_t *rank_at = a.rank_at + int64_t(unit) * (a.chunks + 1);
    // what needs no selection, dealt to the cluster's threads
    const int all = parts * THREADS, at = part * THREADS + t;
    if (h == 0 && at == 0) a.new_lengths[b] = m;
    if (unit == 0 && at == 0) *a.ticket = 0;
    for (int i = at; i < a.chunks; i += all) a.done[int64_t(unit) * a.chunks + i] = 0;
    for (int i = m + at; i < a.budget; i += all) kept[i] = -1;
#pragma unroll 4
    for (int i = m + at; i < a.c.cap; i += all) out[i] = 0.f;
    if (n == m) {  // the same for the whole cluster
        for (int i = at; i < m; i += all) {
            kept[i] = i;
            out[i] = scores[i];
        }
        return;
    }
    for (int i = (n - 1) / kMvRows + 1 + at; i <= a.chunks; i += all) rank_at[i] = m;
    auto stay = [&](uint32_t r, int slot, float score) {
        kept[r] = slot;
        out[r] = score;
    };
    auto rank = [&](int k, uint32_t r) {
        if (k <= a.chunks) rank_at[k] = r;
    };
    if (parts > 1)
        select_slots<HELD, THREADS, true>(a, parts, part, n, scores, keys, stay, rank);
    else
        select_slots<HELD, THREADS, false>(a, 1, 0, n, scores, keys, stay, rank);
}

// Selection and move of small units in one launch, without a workspace.
// `slices` blocks a unit each select for themselves (the first writes kept,
// new_scores and new_lengths) and move a share of every row's words, of the key
// and of the value: the columns of a row are independent, so the blocks need
// nothing of one another.  A block moves runs of words in rank order, a run's
// reads before its writes (a barrier between them); the next run's reads need
// not wait for these: the source slot of rank j that moves is above j, and no
// rank up to j writes there.  A block moves about 9 GB/s (one run in flight,
// and its barrier), which is why units of many bytes a block do not come here.
template <int EB>
__global__ void __launch_bounds__(kSmThreads, 2) k_evict_small(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];
    const CacheArgs &c = a.c;
    int32_t *list = reinterpret_cast<int32_t *>(keys + a.held_keys);
    const int t = threadIdx.x;
    const int unit = blockIdx.x / a.slices, slice = blockIdx.x - unit * a.slices;
    const int b = unit / c.heads, h = unit - b * c.heads;
    start_after_prior();
    const int n = cache_length(c, a.lengths, b, kClassEvict);
    const int m = min(n, a.budget);
    const float *scores = a.scores + b * a.sst[0] + h * a.sst[1];
    float *out = a.new_scores + b * a.nst[0] + h * a.nst[1];
    int32_t *kept = a.kept + b * a.kst[0] + h * a.kst[1];
    if (slice == 0) {
        if (h == 0 && t == 0) a.new_lengths[b] = m;
        for (int i = m + t; i < a.budget; i += kSmThreads) kept[i] = -1;
        for (int i = m + t; i < c.cap; i += kSmThreads) out[i] = 0.f;
        if (n == m)
            for (int i = t; i < m; i += kSmThreads) {
                kept[i] = i;
                out[i] = scores[i];
            }
    }
    if (n == m) return;
    select_slots<true, kSmThreads, false>(
        a, 1, 0, n, scores, keys,
        [&](uint32_t r, int slot, float score) {
            list[r] = slot;
            if (slice == 0) {
                kept[r] = slot;
                out[r] = score;
            }
        },
        [](int, uint32_t) {});
    __syncthreads();

    // the slice's words of a rank: `words` of its key, then as many of its value
    const int words = a.word_div.d / 2, items = a.budget * 2 * words;
    for (int base = 0; base < items; base += kSmThreads * kSmAhead) {
        uint4 x[kSmAhead];
        uint8_t *to[kSmAhead];
#pragma unroll
        for (int k = 0; k < kSmAhead; ++k) {
            const int at = base + k * kSmThreads + t;
            to[k] = nullptr;
            if (at >= items) continue;
            const int r = static_cast<int>(fast_div(static_cast<uint32_t>(at), a.word_div));
            const int from = list[r];
            if (from == r) continue;
            int row_f, row_t;
            const int pf = cache_page(c, b, from, &row_f, kClassEvict), pt = cache_page(c, b, r, &row_t, kClassEvict);
            if (pf < 0 || pt < 0) continue;
            int w = at - r * 2 * words;
            const bool v = w >= words;
            w = w - (v ? words : 0) + slice * words;
            uint8_t *pool = (v ? c.v : c.k) + 16 * w;
            const int64_t *st = v ? c.vst : c.kst;
            x[k] = *reinterpret_cast<const uint4 *>(pool + row_offset(st, pf, h, row_f) * EB);
            to[k] = pool + row_offset(st, pt, h, row_t) * EB;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSmAhead; ++k)
            if (to[k]) *reinterpret_cast<uint4 *>(to[k]) = x[k];
    }
    if constexpr (EB == 1) {  // the scales: the keys' by the first slice, the values' by the last
        for (int v = 0; v < 2; ++v) {
            if (slice != (v ? a.slices - 1 : 0)) continue;
            float *pool = v ? c.vs : c.ks;
            const int64_t *st = v ? c.vss : c.kss;
            for (int base = 0; base < a.budget; base += kSmThreads) {
                const int r = base + t, from = r < a.budget ? list[r] : r;
                float x = 0.f, *to = nullptr;
                if (from != r) {
                    int row_f, row_t;
                    const int pf = cache_page(c, b, from, &row_f, kClassEvict);
                    const int pt = cache_page(c, b, r, &row_t, kClassEvict);
                    if (pf >= 0 && pt >= 0) {
                        x = pool[row_offset(st, pf, h, row_f)];
                        to = pool + row_offset(st, pt, h, row_t);
                    }
                }
                __syncthreads();
                if (to) *to = x;
            }
        }
    }
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(uint32_t *p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// VEC: rows are whole 16-byte words on 16-byte boundaries; else they move an
// element at a time.
template <int EB, bool VEC>
__global__ void __launch_bounds__(kMvThreads, 16) k_evict_move(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint8_t rows[];  // [pool][row][pitch]
    __shared__ int64_t from[2 * kMvRows], to[2 * kMvRows];  // bytes; from -1: the row stays, or has no place
    __shared__ float scales[2][kMvRows];
    __shared__ uint32_t next;
    __shared__ int late;
    const CacheArgs &c = a.c;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int pitch = (c.dim * EB + 15) / 16 * 16;
    const uint32_t units = static_cast<uint32_t>(c.n_seqs) * c.heads;
    const int64_t tickets = int64_t(units) * a.chunks;
    start_after_prior();
    if (t == 0) next = atomicAdd(a.ticket, 1u);
    __syncthreads();
    int64_t ticket = next;
    while (ticket < tickets) {
        uint32_t coming = 0;
        if (t == 0) coming = atomicAdd(a.ticket, 1u);
        // the units' chunks in turn: the chunks in flight are of many units
        const uint32_t chunk = fast_div(static_cast<uint32_t>(ticket), a.unit_div);
        const uint32_t unit = static_cast<uint32_t>(ticket) - chunk * units;
        const int b = static_cast<int>(fast_div(unit, a.head_div)), h = static_cast<int>(unit) - b * c.heads;
        const int n = min(max(a.lengths[b], 0), c.cap);
        if (n > a.budget) {
            // warp w finds the rows' places in pool w, a lane each
            const int r = static_cast<int>(chunk) * kMvRows + lane;
            const int64_t *st = warp ? c.vst : c.kst, *sst = warp ? c.vss : c.kss;
            int64_t f = -1, o = 0, scale_to = 0;
            if (r < a.budget) {
                const int src = a.kept[b * a.kst[0] + h * a.kst[1] + r];
                if (src != r) {
                    int row_f, row_t;
                    const int pf = cache_page(c, b, src, &row_f, kClassEvict);
                    const int pt = cache_page(c, b, r, &row_t, kClassEvict);
                    if (pf >= 0 && pt >= 0) {
                        f = row_offset(st, pf, h, row_f) * EB;
                        o = row_offset(st, pt, h, row_t) * EB;
                        if (EB == 1) {
                            scales[warp][lane] = (warp ? c.vs : c.ks)[row_offset(sst, pf, h, row_f)];
                            scale_to = row_offset(sst, pt, h, row_t);
                        }
                    }
                }
            }
            from[warp * kMvRows + lane] = f;
            to[warp * kMvRows + lane] = o;
            __syncthreads();
            const uint32_t words = a.word_div.d, items = 2 * kMvRows * words;
#pragma unroll 4
            for (uint32_t i = t; i < items; i += kMvThreads) {
                const uint32_t row = fast_div(i, a.word_div), w = i - row * words;
                if (from[row] < 0) continue;
                const uint8_t *src = (row < kMvRows ? c.k : c.v) + from[row];
                uint8_t *at = rows + row * pitch;
                if constexpr (VEC)
                    ptx::cp_async16(ptx::smem_addr(at + 16 * w), src + 16 * w);
                else if constexpr (EB == 2)
                    reinterpret_cast<uint16_t *>(at)[w] = reinterpret_cast<const uint16_t *>(src)[w];
                else
                    at[w] = src[w];
            }
            ptx::cp_async_commit();
            ptx::cp_async_wait<0>();
            __syncthreads();  // all rows have been read
            uint32_t *done = a.done + int64_t(unit) * a.chunks;
            if (t == 0) {
                store_release(done + chunk, 1);
                // the chunks whose rows sit in the slots written next
                const int32_t *rank = a.rank_at + int64_t(unit) * (a.chunks + 1) + chunk;
                const int first = rank[0] / kMvRows;
                const int last = min((rank[1] - 1) / kMvRows, static_cast<int>(chunk) - 1);
                bool ok = true;
                for (int k = first; k <= last && ok; ++k) {
                    if (load_acquire(done + k)) continue;
                    const uint64_t t0 = ptx::global_timer_ns();
                    uint32_t polls = 0;
                    while (!load_acquire(done + k)) {
                        if (++polls >= ptx::kMaxPolls || ptx::global_timer_ns() - t0 > a.wait_ns) {
                            report_error(LC_ERR_TIMEOUT, kClassEvict);
                            ok = false;
                            break;
                        }
                    }
                }
                late = !ok;
            }
            __syncthreads();
            if (!late) {
#pragma unroll 4
                for (uint32_t i = t; i < items; i += kMvThreads) {
                    const uint32_t row = fast_div(i, a.word_div), w = i - row * words;
                    if (from[row] < 0) continue;
                    uint8_t *dst = (row < kMvRows ? c.k : c.v) + to[row];
                    const uint8_t *at = rows + row * pitch;
                    if constexpr (VEC)
                        *reinterpret_cast<uint4 *>(dst + 16 * w) = *reinterpret_cast<const uint4 *>(at + 16 * w);
                    else if constexpr (EB == 2)
                        reinterpret_cast<uint16_t *>(dst)[w] = reinterpret_cast<const uint16_t *>(at)[w];
                    else
                        dst[w] = at[w];
                }
                if (EB == 1 && f >= 0) (warp ? c.vs : c.ks)[scale_to] = scales[warp][lane];
            }
        }
        if (t == 0) next = coming;
        __syncthreads();  // rows, from and to are free again
        ticket = next;
        __syncthreads();
    }
}

cudaError_t take_error_evict(unsigned long long *v) { return take_module_error(v); }

namespace {

// How a call of these sizes goes: in one launch of `slices` blocks a unit, or
// (0) in two with a workspace of these offsets and this end.  One launch takes
// units of at most kSmSlots slots, whose selections the blocks can afford to
// repeat, and kSmMoved bytes a block; twice the bytes where these are half the
// slots or fewer and every SM has a block.  Bfloat16 rows of 128, one launch against
// two: 8 heads of 4 sequences of 2000 cut to 1000, 16.4 against 21.2 us; 8 of
// 4000 to 1000, 26 against 32; 64 of 256 to 128, 23 against 30; 128 of 8000 to
// 64, 52 against 61; 300 of 1000 to 500, 242 against 262; at the bounds 4 of 8000
// to 2000, 33 against 34, and 8 of 4000 to 2000, 41 against 42.  Past them, 4 of up
// to 16384 to 4096, 59 against 40; 4 of 8000 to 4000, 50 against 43.
struct EvictSpace {
    bool vec;  // rows of the pools are whole 16-byte words on 16-byte boundaries
    int slices, held_keys;
    int64_t done, rank_at, end;
};

EvictSpace evict_space(const lc_paged_cache &cache, const CacheArgs &c, int budget) {
    const int64_t units = int64_t(c.n_seqs) * c.heads, chunks = (int64_t(budget) + kMvRows - 1) / kMvRows;
    const int eb = cache_elem_bytes(cache.type);
    const int64_t pool[3] = {cache.n_pages, cache.n_kv_heads, cache.page_size};
    EvictSpace s{};
    s.vec = c.dim * eb % 16 == 0 && rows_aligned(cache.k, 3, pool, cache.k_stride, eb, 16) &&
            rows_aligned(cache.v, 3, pool, cache.v_stride, eb, 16);
    const int64_t held = (int64_t(c.cap) + kSelRound - 1) / kSelRound * kSelRound;
    const int words = c.dim * eb / 16;
    if (s.vec && held <= kSmSlots) {
        int slices = 1;  // as many as the row's words divide into, of 32 bytes or more
        while (words % (2 * slices) == 0 && words / (2 * slices) >= 2 && units * 2 * slices <= kSmBlocks) slices *= 2;
        const bool filled = units * slices > kSmBlocks / 2;
        const int most = held <= kSmSlots / 2 && filled ? 2 * kSmMoved : kSmMoved;
        if (int64_t(budget) * 2 * 16 * words / slices <= most) {
            s.slices = slices;
            s.held_keys = static_cast<int>(held);
            return s;
        }
    }
    s.done = 256;  // behind the ticket
    s.rank_at = s.done + round256(units * chunks * 4);
    s.end = s.rank_at + round256(units * (chunks + 1) * 4);
    return s;
}

template <int EB>
int launch_evict_small(EvictArgs &a, cudaStream_t cs) {
    a.word_div = make_fastdiv(static_cast<uint32_t>(2 * (a.c.dim * EB / 16 / a.slices)));
    const void *fn = reinterpret_cast<const void *>(&k_evict_small<EB>);
    int sms, per;
    constexpr int kMost = 4 * (kSmSlots + kSmMoved / 32);  // half the slots: twice the ranks
    if (prepare(fn, kSmThreads, 0, kMost, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
    return launch_after(fn, static_cast<unsigned>(int64_t(a.c.n_seqs) * a.c.heads * a.slices), kSmThreads,
                        4 * (size_t(a.held_keys) + a.budget), cs, &a);
}

template <int EB, bool VEC>
int launch_evict(EvictArgs &a, cudaStream_t cs) {
    const int64_t units = int64_t(a.c.n_seqs) * a.c.heads;
    const int smem = 2 * kMvRows * ((a.c.dim * EB + 15) / 16 * 16);
    a.unit_div = make_fastdiv(static_cast<uint32_t>(units));
    a.head_div = make_fastdiv(static_cast<uint32_t>(a.c.heads));
    a.word_div = make_fastdiv(static_cast<uint32_t>(VEC ? a.c.dim * EB / 16 : a.c.dim));
    int sms, per, move_per;
    const void *move = reinterpret_cast<const void *>(&k_evict_move<EB, VEC>);
    if (prepare(move, kMvThreads, smem, smem, &sms, &move_per) != cudaSuccess) return LC_ERR_CUDA;
    // Selection.  Clusters where there are few units and many slots, a block an
    // SM at most (of 16 blocks, which are no longer portable, measured slower:
    // 45 against 27 us for 8 units of 131071 slots), and where a block would hold
    // more than kSelEase keys, twice that where it has an SM to itself: two
    // blocks share an SM and hide each other's barriers (320 units of 20000 slots
    // 48 against 57 us, 800 of them 92 against 111, 160 of 50000 77 against 122;
    // but 32 of 98340 34.3 with 256 blocks and 32.5 with 128).  Where blocks have an
    // SM each and many slots a thread, 1024 threads (26 against 31 us).
    int parts = 1;
    while (parts < kSelCluster && units * parts * 2 <= sms && a.c.cap / (2 * parts) >= kSelLeast) parts *= 2;
    const int rounds = a.c.cap ? (a.c.cap - 1) / kSelRound + 1 : 0;
    auto keys_held = [&] { return int64_t(rounds + parts - 1) / parts * kSelRound; };
    while (parts < kSelCluster && keys_held() > (units * parts <= sms ? 2 * kSelEase : kSelEase)) parts *= 2;
    const int64_t hold = keys_held();
    const bool held = hold <= kSelKeys;
    const int threads = units * parts <= sms && hold > 4096 ? 1024 : 512;
    const void *forms[2][2] = {{reinterpret_cast<const void *>(&k_evict_select<false, 512>),
                                reinterpret_cast<const void *>(&k_evict_select<false, 1024>)},
                               {reinterpret_cast<const void *>(&k_evict_select<true, 512>),
                                reinterpret_cast<const void *>(&k_evict_select<true, 1024>)}};
    const void *sel = forms[held][threads == 1024];
    if (prepare(sel, threads, 0, kSelKeys * 4, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
    const int st = launch_after(sel, static_cast<unsigned>(units * parts), threads,
                                held ? static_cast<size_t>(hold) * 4 : 0, cs, &a, parts);
    if (st) return st;
    const int64_t blocks = std::min<int64_t>(units * a.chunks, int64_t(sms) * move_per);
    return launch_after(move, static_cast<unsigned>(blocks), kMvThreads, smem, cs, &a);
}

}  // namespace

}  // namespace lc

extern "C" int64_t lc_cache_evict_workspace(const lc_paged_cache *cache, int32_t budget) {
    lc::CacheArgs c;
    if (lc::check_cache(cache, true, &c) || budget < 1) return -1;
    return lc::evict_space(*cache, c, budget).end;
}

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
    if (lists_meet(e->lengths, e->new_lengths, cache->n_seqs)) return LC_ERR_OVERLAP;
    if ((reinterpret_cast<uintptr_t>(e->lengths) | reinterpret_cast<uintptr_t>(e->scores) |
         reinterpret_cast<uintptr_t>(e->kept) | reinterpret_cast<uintptr_t>(e->new_scores) |
         reinterpret_cast<uintptr_t>(e->new_lengths)) % 4)
        return LC_ERR_ALIGN;
    const int64_t ext[2] = {cache->n_seqs, cache->n_kv_heads};
    st = check_reach(2, ext, e->scores_stride, a.c.cap);
    if (!st) st = check_reach(2, ext, e->new_scores_stride, a.c.cap);
    if (!st) st = check_reach(2, ext, e->kept_stride, e->budget);
    if (st) return st;
    if ((a.c.cap > 0 && !rows_apart(2, ext, e->new_scores_stride, a.c.cap)) ||
        !rows_apart(2, ext, e->kept_stride, e->budget))
        return LC_ERR_NOT_INJECTIVE;
    if (a.c.cap > 0 && rows_meet(e->scores, e->scores_stride, e->new_scores, e->new_scores_stride, ext, a.c.cap))
        return LC_ERR_OVERLAP;
    const int64_t units = ext[0] * ext[1], chunks = (int64_t(e->budget) + kMvRows - 1) / kMvRows;
    // the tickets that running blocks draw past the last one stay in 32 bits
    // too
    if (units > 0x0fffffff || units * chunks > 0xf0000000ll) return LC_ERR_OVERFLOW;
    const EvictSpace space = evict_space(*cache, a.c, e->budget);
    if (space.end > 0 && !e->workspace) return LC_ERR_NULL;
    if (space.end > e->workspace_bytes) return LC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(e->workspace) % 256) return LC_ERR_ALIGN;
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
    a.chunks = static_cast<int32_t>(chunks);
    a.wait_ns = wait_limit_ns();
    uint8_t *ws = static_cast<uint8_t *>(e->workspace);
    a.ticket = reinterpret_cast<uint32_t *>(ws);
    a.done = reinterpret_cast<uint32_t *>(ws + space.done);
    a.rank_at = reinterpret_cast<int32_t *>(ws + space.rank_at);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool q8 = cache->type == LC_CACHE_E4M3;
    if (space.slices) {
        a.slices = space.slices;
        a.held_keys = space.held_keys;
        return q8 ? launch_evict_small<1>(a, cs) : launch_evict_small<2>(a, cs);
    }
    if (q8) return space.vec ? launch_evict<1, true>(a, cs) : launch_evict<1, false>(a, cs);
    return space.vec ? launch_evict<2, true>(a, cs) : launch_evict<2, false>(a, cs);
}
