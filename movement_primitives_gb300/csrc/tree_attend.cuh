// Attention of a tree of drafted tokens a sequence over a paged key-value
// cache (lc_cache_attend_tree):
//     x_tj = scale * q_t . k_j,  w = softmax_j(x),  out_t = sum_j w_tj v_j
// over the slots j that draft t sees: those before the drafts, and the slots
// of its ancestors and its own.
//
// Mathematics.  The drafts x query heads of one key head are the rows of tiles of
// 128.  A tile goes through its sequence's slots in steps: S = Q K^T into tensor
// memory, one thread a row turns S into weights 2^(x - m) relative to a running
// maximum m (that follows the maximum only when that has grown by 2^kRise; the
// output is then rescaled) and adds them up, and P V is added to the output in tensor
// memory.  Two S take turns, so that a step's first product runs during the
// softmax of the step before.  Which drafts a draft descends from is a word of 64
// bits; the words come from the parents by doubling: what an ancestor sees joins
// in, then its ancestor is asked.
//
// A weight enters the second product as two numbers of the values' 16-bit type, its
// leading bits and the rounded rest (within 2^-16 or 2^-22 of it), two products:
// memory bounds the pass, so the second costs nothing up to about 128 rows, and the output's own
// rounding is the only one that shows.  E4M3 codes become float16 numbers on their
// way into shared memory, exactly; the keys' scales multiply the logits, the
// values' join the weights as 2^(x + log2 |s| - mv) with a maximum mv of that exponent;
// these weights are one float16 number each.
//
// Work.  A (sequence, key head, tile of rows) is a unit; the steps of all units, laid
// end to end, are cut into equal runs, one a block, found from the lengths on
// the device.  A unit inside one run is finished there; a cut one leaves
// parts in the workspace, which k_tree_join joins in their order, so results do not
// depend on timing.  Eight warps of a block bring the rows of keys and values in
// by asynchronous 16-byte copies (a row's place comes from the page table, which
// tensor copies could not follow), several tiles ahead; one thread issues the
// products; four warps do the softmax.
#pragma once

#include "cache_common.cuh"
#include "tensor_core.cuh"

namespace lc {

constexpr uint32_t kClassTree = 0xf4;
constexpr int kTrRows = 128;
constexpr int kTrDrafts = LC_CACHE_MAX_DRAFTS;
constexpr int kTrItems = 4;      // pieces that the scheduling warp may be ahead
constexpr int kTrMasked = 4;     // steps of a piece that some row sees in part: two at either end at most
constexpr int kTrAux = 8;        // steps whose slots' scales and presence are held
constexpr int kTrLoaders = 8;
constexpr int kTrMostRuns = 160;
constexpr int kTrLeast = 2;      // steps of a run

struct TreeArgs {
    CacheArgs c;
    const uint16_t *q;
    uint16_t *out;
    const int32_t *lengths, *counts, *parents;
    float *lse;
    int64_t qst[3], ost[3], lst[2];   // sequence, draft, head
    int64_t parents_stride;
    int32_t drafts, q_heads, group, window;
    FastDiv group_div;
    float scale2;           // |scale| log2 e
    int32_t negative;
    int32_t vec, q_vec, out_vec;  // rows of the pools, of q and of out are whole 16-byte words on 16-byte boundaries
    int32_t runs;           // blocks of the main kernel
    int32_t most_blocks;    // tiles of rows a key head at most
    float *part;            // [2 runs][dim / 4 rounded up to 16][128 rows][4]
    float2 *part_ml;        // [2 runs][128]
    uint64_t limit_ns;
};

// A sequence's share.
struct TreeSeq {
    int n, count, begin;    // slots, drafts, the first slot that any draft sees
    int blocks, steps;      // tiles of rows a key head, steps of a tile
};

template <int KEYS>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs &a, int b) {
    TreeSeq s;
    const int length = a.lengths[b];
    s.n = min(max(length, 0), a.c.cap);
    if (s.n != length) note_error(LC_ERR_CACHE_INDEX, kClassTree);
    const int want = a.counts ? a.counts[b] : min(a.drafts, s.n);
    s.count = min(max(want, 0), min(a.drafts, s.n));
    if (s.count != want) note_error(LC_ERR_CACHE_INDEX, kClassTree);
    s.begin = a.window ? max(s.n - s.count + 1 - a.window, 0) : 0;
    s.blocks = (s.count * a.group + kTrRows - 1) / kTrRows;
    s.steps = s.count ? (s.n - s.begin + KEYS - 1) / KEYS : 0;
    return s;
}

// Steps of all units, and of those of the sequences before `upto`, by a warp.
template <int KEYS>
__device__ __forceinline__ int64_t tree_steps(const TreeArgs &a, int upto, int64_t *before) {
    const int lane = threadIdx.x & 31;
    int64_t all = 0, some = 0;
#pragma unroll 1
    for (int b = lane; b < a.c.n_seqs; b += 32) {
        const TreeSeq s = tree_seq<KEYS>(a, b);
        const int64_t w = int64_t(s.steps) * s.blocks * a.c.heads;
        all += w;
        if (b < upto) some += w;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, d);
        some += __shfl_xor_sync(0xffffffffu, some, d);
    }
    if (before) *before = some;
    return all;
}

// Runs that `all` steps are cut into, and where run r begins.
__device__ __forceinline__ int tree_runs(const TreeArgs &a, int64_t all) {
    const int64_t most = (all + kTrLeast - 1) / kTrLeast;
    return most < a.runs ? static_cast<int>(most) : a.runs;
}
__device__ __forceinline__ int64_t run_begin(int64_t all, int runs, int r) { return all * r / runs; }

// A piece of a run: steps first .. first + steps - 1 of a unit.
struct TreeItem {
    int32_t b, head, row0;      // row0: the tile's first row, draft * group + query head of the group
    int32_t n, count, begin;
    int32_t first, steps;
    int32_t part;               // where its part goes, -1 for a whole unit
    int32_t end;
    int32_t bad_steps;
    uint32_t last_tile;
    int32_t bad_step[kTrMasked];
    uint32_t bad[kTrMasked][4];     // values that are not finite, of masked steps
    uint64_t kin[kTrDrafts];        // the drafts that a draft sees
    int32_t from[kTrDrafts];        // the first slot before the drafts that it sees
};

template <int NC, bool Q8>
struct TreeShape {
    static constexpr int KEYS = NC <= 2 ? 128 : 64;        // slots of a step: two tiles and more have to fit
    static constexpr int CHUNK = KEYS * 128;               // bytes of 64 columns of a tile
    static constexpr int TILE = NC * CHUNK;
    static constexpr int QCHUNK = kTrRows * 128;
    static constexpr int Q = NC * QCHUNK;
    static constexpr int RAW = !Q8 ? 0 : NC == 4 ? 3 : 4;     // E4M3 tiles under way
    static constexpr int RAW_TILE = TILE / 2;
    static constexpr int SHARED = 9216 + (Q8 ? kTrAux * KEYS * 8 : 0);  // the block of barriers and items, and 1024 for alignment
    static constexpr int FIT = (232448 - SHARED - Q - RAW * RAW_TILE) / TILE;
    // (what kTrAux holds is read before tiles this far on are started)
    static constexpr int SLOTS = Q8 ? (FIT < 6 ? FIT : 6) : (FIT < 12 ? FIT : 12);
    static constexpr int LAG = Q8 ? RAW - 1 : SLOTS / 2;   // tiles under way
    static constexpr int SMEM = Q + RAW * RAW_TILE + SLOTS * TILE + SHARED;
    static constexpr int THREADS = 32 * (4 + kTrLoaders + 2);
    static constexpr int O = 256;                          // first output column of tensor memory
    static_assert(SLOTS >= 3 && LAG < SLOTS + (Q8 ? RAW : 0), "keys of two steps and values of one");
};

struct TreeShared {
    uint64_t ring_full[12], ring_empty[12];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];  // of every other step
    uint64_t item_full[kTrItems], item_empty[kTrItems];
    uint64_t drain;
    uint32_t tmem;
    uint32_t there[kTrAux][4];      // the slots of a step that exist and whose pages do
    float q_scale[2][kTrRows];      // E4M3: what a row of q was divided by
    TreeItem item[kTrItems];
};
static_assert(sizeof(TreeShared) <= 8192, "the shared block has 8192 bytes");

__device__ __forceinline__ float tr_exp2(float x) {  // 2 ulp, 0 for -infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t tr_pack(float lo, float hi) {
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
// Two numbers >= 0 as the sums of two each: the leading bits, and what they leave, rounded.
template <bool F16>
__device__ __forceinline__ void tr_split(float lo, float hi, uint32_t *lead, uint32_t *rest) {
    float2 v;
    if constexpr (F16) {
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(*lead) : "f"(hi), "f"(lo));
        v = __half22float2(*reinterpret_cast<const __half2 *>(lead));
    } else {
        *lead = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
        v = make_float2(__uint_as_float(*lead << 16), __uint_as_float(*lead & 0xffff0000u));
    }
    *rest = tr_pack<F16>(lo - v.x, hi - v.y);
}
__device__ __forceinline__ uint32_t tr_halves(uint32_t codes) {  // two E4M3 codes (the low 16 bits) as float16, exactly
    uint32_t v;
    asm("{.reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c;}" : "=r"(v) : "r"(codes));
    return v;
}
__device__ __forceinline__ void tr_copy16(uint32_t dst, const void *src, bool real) {  // zeros where there is nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
    return v;
}

// The kernel's warps go through different code at the same time: what is rare, or
// may be a loop, is kept out of line or rolled, since instructions that do not fit the
// cache bounded the first form (195 KB of them, 20 cycles an instruction).

// 16 bytes of a row, element by element where they may not be read at once.
template <int EB>
__device__ __noinline__ uint4 tree_piece(const uint8_t *row, int col, int dim) {
    uint64_t w[2] = {0, 0};
#pragma unroll 1
    for (int i = 0; i < 16 / EB; ++i)
        if (col + i < dim) {
            const uint64_t v = EB == 2 ? *reinterpret_cast<const uint16_t *>(row + (col + i) * 2) : row[col + i];
            if (i * EB < 8) w[0] |= v << i * EB * 8;
            else w[1] |= v << (i * EB - 8) * 8;
        }
    return make_uint4(static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[0] >> 32), static_cast<uint32_t>(w[1]),
                      static_cast<uint32_t>(w[1] >> 32));
}

// The drafts that each draft of a sequence sees, and from where on it sees what was before them; by a warp, two drafts a lane.
__device__ __forceinline__ void tree_kin(const TreeArgs &a, TreeItem &it) {
    const int lane = threadIdx.x & 31, before = it.n - it.count;
    const int32_t *parents = a.parents + it.b * a.parents_stride;
    uint64_t kin[2];
    int up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        kin[i] = uint64_t(1) << t;
        up[i] = -1;
        if (t < it.count) {
            const int p = parents[t];
            if (p >= -1 && p < t) up[i] = p;
            else note_error(LC_ERR_CACHE_INDEX, kClassTree);
        }
    }
#pragma unroll 1
    for (int round = 0; round < 6; ++round) {
        uint64_t k[2];
        int u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int src = up[i] & 31;
            const uint64_t k0 = __shfl_sync(0xffffffffu, kin[0], src), k1 = __shfl_sync(0xffffffffu, kin[1], src);
            const int u0 = __shfl_sync(0xffffffffu, up[0], src), u1 = __shfl_sync(0xffffffffu, up[1], src);
            k[i] = up[i] < 0 ? 0 : up[i] < 32 ? k0 : k1;
            u[i] = up[i] < 0 ? -1 : up[i] < 32 ? u0 : u1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kin[i] |= k[i];
            up[i] = u[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i, depth = __popcll(kin[i]);
        // parents come before their children: the farthest ancestors are the lowest bits
        if (a.window)
            for (int d = depth; d > a.window; --d) kin[i] &= kin[i] - 1;
        it.kin[t] = kin[i];
        it.from[t] = a.window ? min(max(before + depth - a.window, 0), before) : 0;
    }
}

// The values of a slot, and of an element 0 or what is not finite.
template <int EB>
__device__ __noinline__ const uint8_t *tree_value(const TreeArgs &a, int b, int head, int slot) {
    int r = 0;
    const int page = cache_page(a.c, b, slot, &r, kClassTree);
    return page < 0 ? nullptr : a.c.v + row_offset(a.c.vst, page, head, r) * EB;
}
template <int KV>
__device__ __noinline__ float tree_unusual(const uint8_t *v, int e) {
    if constexpr (KV == LC_CACHE_E4M3) {
        return (v[e] & 0x7f) == 0x7f ? NAN : 0.f;
    } else {
        const uint32_t u = reinterpret_cast<const uint16_t *>(v)[e];
        constexpr uint32_t kExp = KV == LC_CACHE_F16 ? 0x7c00u : 0x7f80u;
        if ((u & kExp) != kExp) return 0.f;
        return KV == LC_CACHE_F16 ? __half2float(__ushort_as_half(u)) : __uint_as_float(u << 16);
    }
}

template <int KV, int NC>
__global__ void __launch_bounds__(TreeShape<NC, KV == LC_CACHE_E4M3>::THREADS, 1)
    k_tree_attend(const __grid_constant__ TreeArgs a) {
    constexpr bool Q8 = KV == LC_CACHE_E4M3, M16 = KV != LC_CACHE_BF16;  // float16 products
    using S = TreeShape<NC, Q8>;
    constexpr int KEYS = S::KEYS, EB = Q8 ? 1 : 2;
    // weights are up to 2^(kLift + kRise): float16 has few exponents, so small ones are lifted into them; others are
    // lowered, as sums are, so that those of the type's largest values stay in float32
    constexpr float kRise = M16 ? 2.f : 8.f, kLift = M16 ? 12.f : -40.f, kSumLift = Q8 ? -40.f : kLift;
    extern __shared__ uint8_t raw_smem[];
    const uint32_t base = (ptx::smem_addr(raw_smem) + 1023) & ~1023u;
    const uint32_t q_s = base, ring_s = q_s + S::Q, raw_s = ring_s + S::SLOTS * S::TILE;
    uint8_t *const after = raw_smem + (base - ptx::smem_addr(raw_smem)) + S::Q + S::SLOTS * S::TILE + S::RAW * S::RAW_TILE;
    TreeShared &sh = *reinterpret_cast<TreeShared *>(after);
    float *const aux = reinterpret_cast<float *>(after + 8192);  // E4M3: [kTrAux][keys' scales, log2 of values'][KEYS]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](const uint64_t &b) { return ptx::smem_addr(&b); };

    if (warp == 4 + kTrLoaders) tc::alloc(ptx::smem_addr(&sh.tmem), 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::SLOTS; ++i) {
            ptx::mbar_init(bar(sh.ring_full[i]), kTrLoaders);
            ptx::mbar_init(bar(sh.ring_empty[i]), 1);
        }
        ptx::mbar_init(bar(sh.q_full), kTrLoaders);
        ptx::mbar_init(bar(sh.q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(sh.s_full[i]), 1);
            ptx::mbar_init(bar(sh.p_full[i]), 4);
            ptx::mbar_init(bar(sh.o_full[i]), 1);
        }
        for (int i = 0; i < kTrItems; ++i) {
            ptx::mbar_init(bar(sh.item_full[i]), 1);
            ptx::mbar_init(bar(sh.item_empty[i]), 4 + kTrLoaders + 1);
        }
        ptx::mbar_init(bar(sh.drain), 1);
        ptx::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    start_after_prior();

    bool ok = true;  // no wait of this thread has run out
    auto wait = [&](const uint64_t &b, uint32_t n) {  // for phase n (counted from 0)
        if (ok && !ptx::mbar_wait_step(bar(b), n & 1, a.limit_ns)) {
            ok = false;
            note_error(LC_ERR_TIMEOUT, kClassTree);
        }
        return ok;
    };
    // a warp's wait: one lane polls, for the others' polls take turns with what else the shared memory does
    auto wait_warp = [&](const uint64_t &b, uint32_t n) {
        if (lane == 0) wait(b, n);
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
        return ok;
    };
    auto done_warp = [&](const uint64_t &b, uint32_t n) {
        int d = 0;
        if (lane == 0) d = ptx::mbar_try_wait(bar(b), n & 1);
        return __shfl_sync(0xffffffffu, d, 0) != 0;
    };
    auto arrive = [&](const uint64_t &b) {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar(b)) : "memory");
    };
    auto arrive_warp = [&](const uint64_t &b) {
        __syncwarp();
        if (lane == 0) arrive(b);
    };
    // whether some row of a piece sees a step in part
    auto masked = [&](const TreeItem &it, int slot0) {
        return slot0 + KEYS > it.n - it.count || (a.window && slot0 < it.n - it.count + kTrDrafts - a.window);
    };

    if (warp == 4 + kTrLoaders + 1) {
        // scheduling: the pieces of this block's run
        int64_t at = 0;
        const int64_t all = tree_steps<KEYS>(a, 0, nullptr);
        const int runs = tree_runs(a, all);
        int64_t from = 0, to = 0;
        if (static_cast<int>(blockIdx.x) < runs) {
            from = run_begin(all, runs, blockIdx.x);
            to = run_begin(all, runs, blockIdx.x + 1);
        }
        uint32_t i = 0;
        auto post = [&](auto &&fill) {
            const int s = i % kTrItems;
            if (i >= kTrItems && !wait_warp(sh.item_empty[s], i / kTrItems - 1)) return;
            fill(sh.item[s]);
            arrive_warp(sh.item_full[s]);
            ++i;
        };
#pragma unroll 1
        for (int b0 = 0; b0 < a.c.n_seqs && from < to && ok; b0 += 32) {
            TreeSeq s{};
            if (b0 + lane < a.c.n_seqs) s = tree_seq<KEYS>(a, b0 + lane);
            const int64_t w = int64_t(s.steps) * s.blocks * a.c.heads;
            int64_t upto = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            while (from < to && ok) {
                const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && at + upto > from);
                if (!hit) break;
                const int l = __ffs(hit) - 1;
                const int steps = __shfl_sync(0xffffffffu, s.steps, l), blocks = __shfl_sync(0xffffffffu, s.blocks, l);
                const int n = __shfl_sync(0xffffffffu, s.n, l), count = __shfl_sync(0xffffffffu, s.count, l);
                const int begin = __shfl_sync(0xffffffffu, s.begin, l);
                const int64_t in = from - at - __shfl_sync(0xffffffffu, upto - w, l);
                const int unit = static_cast<int>(in / steps), first = static_cast<int>(in - int64_t(unit) * steps);
                const int take = static_cast<int>(min(to - from, int64_t(steps - first)));
                post([&](TreeItem &it) {
                    if (lane == 0) {
                        it.b = b0 + l;
                        it.head = unit / blocks;
                        it.row0 = unit % blocks * kTrRows;
                        it.n = n;
                        it.count = count;
                        it.begin = begin;
                        it.first = first;
                        it.steps = take;
                        it.part = take == steps ? -1 : 2 * static_cast<int>(blockIdx.x) + (first == 0);
                        it.end = 0;
                        it.bad_steps = 0;
                    }
                    if (lane < 4 * kTrMasked) it.bad[lane / 4][lane % 4] = 0;
                    __syncwarp();
                    tree_kin(a, it);
                });
                from += take;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (ok) post([&](TreeItem &it) { if (lane == 0) it.end = 1; });
    } else if (warp >= 4 && warp < 4 + kTrLoaders) {
        // loads
        constexpr int RW = KEYS / kTrLoaders, PR = S::TILE / KEYS / 16 * EB / 2;  // rows of a warp, 16-byte pieces of a row
        constexpr int ITER = RW * PR / 32;
        const int lw = warp - 4, dim = a.c.dim, dim16 = (dim + 15) / 16 * 16;
        const uint8_t *const pool[2] = {a.c.k, a.c.v};
        uint32_t issued = 0, given = 0, n_q = 0;  // tiles started and given to the products, tiles of q
        uint32_t back = 0, done = 0;              // items given back, and whose tiles have all been started
        // of the tiles under way: values of masked steps (item * kTrMasked + entry, else -1); E4M3 values: the warp's rows
        // whose scale is negative
        int32_t note[S::LAG + 1];
        uint32_t flip[S::LAG + 1];
#pragma unroll
        for (int i = 0; i <= S::LAG; ++i) {
            note[i] = -1;
            flip[i] = 0;
        }
        auto piece_of = [&](int i, int *row, int *col) {  // i-th piece of this lane: row of the warp, first element
            const int at = i * 32 + lane;
            *row = at / PR;
            *col = at % PR * (16 / EB);
        };
        auto tile_at = [&](uint32_t slot, int row, int col) {  // where 8 elements go
            return ring_s + slot * S::TILE + col / 64 * S::CHUNK + row * 128 + ((col / 8 & 7) ^ (row & 7)) * 16;
        };
        // looks a masked step's values through: what is not finite becomes 0 and is noted
        auto look = [&](uint4 &x, int where, int row) {
            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (Q8) {
                    const uint32_t nan = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    if (nan) {
                        found = true;
                        w[e] &= ~(nan | (nan - (nan >> 7)));
                    }
                } else {
                    constexpr uint32_t kExp = M16 ? 0x7c00u : 0x7f80u;
                    if ((w[e] & kExp) == kExp) {
                        found = true;
                        w[e] &= 0xffff0000u;
                    }
                    if ((w[e] & kExp << 16) == kExp << 16) {
                        found = true;
                        w[e] &= 0xffffu;
                    }
                }
            }
            if (found) atomicOr(&sh.item[where / kTrMasked].bad[where % kTrMasked][row >> 5], 1u << (row & 31));
            return found;
        };
        // the oldest tile under way has landed: gives it to the products
        auto give = [&]() {
            const uint32_t slot = given % S::SLOTS;
            const int32_t where = note[0];
            const uint32_t signs = flip[0];
#pragma unroll
            for (int i = 0; i < S::LAG; ++i) {
                note[i] = note[i + 1];
                flip[i] = flip[i + 1];
            }
            if constexpr (Q8) {
                if (given >= S::SLOTS && !wait_warp(sh.ring_empty[slot], given / S::SLOTS - 1)) return;
#pragma unroll 2
                for (int i = 0; i < ITER; ++i) {
                    int row, col;
                    piece_of(i, &row, &col);
                    if (col >= dim16) continue;
                    uint4 x = ld_shared16(raw_s + given % S::RAW * S::RAW_TILE + ((lw * ITER + i) * 32 + lane) * 16);
                    if (where >= 0) look(x, where, lw * RW + row);
                    const uint32_t sign = (signs >> row & 1) ? 0x80008000u : 0u;
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(&x);
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[2 * e] = tr_halves(w[e]) ^ sign;
                        y[2 * e + 1] = tr_halves(w[e] >> 16) ^ sign;
                    }
                    st_shared16(tile_at(slot, lw * RW + row, col), make_uint4(y[0], y[1], y[2], y[3]));
                    st_shared16(tile_at(slot, lw * RW + row, col + 8), make_uint4(y[4], y[5], y[6], y[7]));
                }
            } else if (where >= 0) {
#pragma unroll 1
                for (int i = 0; i < ITER; ++i) {
                    int row, col;
                    piece_of(i, &row, &col);
                    if (col >= dim16) continue;
                    const uint32_t at = tile_at(slot, lw * RW + row, col);
                    uint4 x = ld_shared16(at);
                    if (look(x, where, lw * RW + row)) st_shared16(at, x);
                }
            }
            tc::fence_async_smem();
            arrive_warp(sh.ring_full[slot]);
            ++given;
            // an item is given back when its last values, which may be noted in it, have landed
            if (back < done && given == sh.item[back % kTrItems].last_tile) {
                arrive_warp(sh.item_empty[back % kTrItems]);
                ++back;
            }
        };
        // gives the tiles that have landed, or waits for all of them
        auto settle = [&](bool all) {
            if (all) ptx::cp_async_wait<0>();
            else ptx::cp_async_wait<S::LAG>();
            const uint32_t to = all ? issued : issued - S::LAG;
#pragma unroll 1
            while (given < to && ok) give();
        };
        auto flush = [&] { settle(true); };
        // starts a tile of pool w from the rows at `from`
        auto start = [&](int w, int64_t from, int32_t where, uint32_t signs) {
            const uint32_t slot = issued % S::SLOTS;
            if (!Q8 && issued >= S::SLOTS && !wait_warp(sh.ring_empty[slot], issued / S::SLOTS - 1)) return;
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                int row, col;
                piece_of(i, &row, &col);
                const int64_t r = __shfl_sync(0xffffffffu, from, row);
                if (col >= dim16) continue;
                const uint32_t dst = Q8 ? raw_s + issued % S::RAW * S::RAW_TILE + ((lw * ITER + i) * 32 + lane) * 16
                                        : tile_at(slot, lw * RW + row, col);
                const bool real = r >= 0 && col < dim;
                const uint8_t *src = pool[w] + (real ? r * EB : 0);
                if (a.vec) tr_copy16(dst, src + (real ? col * EB : 0), real);
                else st_shared16(dst, real ? tree_piece<EB>(src, col, dim) : make_uint4(0, 0, 0, 0));
            }
            ptx::cp_async_commit();
#pragma unroll
            for (int i = 0; i <= S::LAG; ++i)
                if (issued - given == static_cast<uint32_t>(i)) {
                    note[i] = where;
                    flip[i] = signs;
                }
            ++issued;
            if (issued - given > S::LAG) settle(false);
        };
        uint32_t step_no = 0;  // steps of all pieces
        for (uint32_t i = 0; ok; ++i) {
            if (!done_warp(sh.item_full[i % kTrItems], i / kTrItems)) flush();
            if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
            TreeItem &it = sh.item[i % kTrItems];
            if (it.end) break;
            const int b = it.b, head = it.head, n = it.n, slot_first = it.begin + it.first * KEYS, steps = it.steps;
            int entry = 0;
            int64_t v_off = -1, v_next = -1;   // rows of the values of the step whose keys were started last, and the one before
            uint32_t signs = 0, signs_next = 0;
            // a page id a lane, a step ahead
            auto page_id = [&](int j, int *row) {
                const int slot = slot_first + j * KEYS + lw * RW + lane;
                *row = 0;
                if (lane >= RW || j >= steps || slot >= n) return -1;
                const int at = static_cast<int>(fast_div(slot, a.c.page_div));
                *row = slot - at * a.c.page;
                const int id = a.c.table[b * a.c.table_stride + at];
                if (id >= 0 && id < a.c.n_pages) return id;
                note_error(LC_ERR_CACHE_INDEX, kClassTree);
                return -1;
            };
            int row = 0, page = page_id(0, &row);
            auto load_q = [&] {
                if (n_q && !done_warp(sh.q_empty, n_q - 1)) {
                    flush();  // its last keys among them
                    if (!wait_warp(sh.q_empty, n_q - 1)) return;
                }
                // the rows of q: a row a warp at a time, eight on the way
                constexpr int PQ = NC * 8;
#pragma unroll 1
                for (int r0 = 0; r0 < kTrRows / kTrLoaders; r0 += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int at = it.row0 + lw * (kTrRows / kTrLoaders) + r0 + r;
                        const int t = static_cast<int>(fast_div(at, a.group_div)), g = at - t * a.group;
                        x[r] = make_uint4(0, 0, 0, 0);
                        if (t < it.count && lane * 8 < dim) {
                            const uint16_t *from = a.q + b * a.qst[0] + t * a.qst[1] + (int64_t(head) * a.group + g) * a.qst[2];
                            if (a.q_vec) x[r] = *reinterpret_cast<const uint4 *>(from + lane * 8);
                            else x[r] = tree_piece<2>(reinterpret_cast<const uint8_t *>(from), lane * 8, dim);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int at = lw * (kTrRows / kTrLoaders) + r0 + r;
                        if constexpr (Q8) {
                            // bfloat16 to float16 of a row whose largest element is between 1 and 2
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x[r]);
                            float f[8], most = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                f[2 * e] = __uint_as_float(w[e] << 16);
                                f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                                most = fmaxf(most, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
                            }
                            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
                            int ex = static_cast<int>(top >> 23) - 127;
                            ex = min(max(ex, -126), 126);
                            const float div = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = tr_pack<true>(f[2 * e] * div, f[2 * e + 1] * div);
                            if (lane == 0) sh.q_scale[i & 1][at] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                        }
                        if (lane < PQ)
                            st_shared16(q_s + lane / 8 * S::QCHUNK + at * 128 + ((lane & 7) ^ (at & 7)) * 16, x[r]);
                    }
                }
                tc::fence_async_smem();
                arrive_warp(sh.q_full);
                ++n_q;
            };
            // tiles in their order: K0 K1 V0 K2 V1 ...
#pragma unroll 1
            for (int p = 0; p < 2 * steps && ok; ++p) {
                const bool is_k = p == 0 || (p & 1 && p < 2 * steps - 1);
                const int j = is_k ? (p + 1) / 2 : p == 2 * steps - 1 ? steps - 1 : p / 2 - 1;
                int64_t from;
                int32_t where = -1;
                uint32_t sign = 0;
                if (is_k) {
                    from = page >= 0 ? row_offset(a.c.kst, page, head, row) : -1;
                    v_off = v_next;
                    signs = signs_next;
                    v_next = page >= 0 ? row_offset(a.c.vst, page, head, row) : -1;
                    const int x = step_no % kTrAux;
                    const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & ((1u << RW) - 1);
                    if (lane == 0) {
                        if constexpr (RW == 16) reinterpret_cast<uint16_t *>(sh.there[x])[lw] = static_cast<uint16_t>(there);
                        else reinterpret_cast<uint8_t *>(sh.there[x])[lw] = static_cast<uint8_t>(there);
                    }
                    if constexpr (Q8) {
                        float ks = 0.f, vs = 0.f;
                        if (page >= 0) {
                            ks = a.c.ks[row_offset(a.c.kss, page, head, row)];
                            vs = a.c.vs[row_offset(a.c.vss, page, head, row)];
                        }
                        signs_next = __ballot_sync(0xffffffffu, vs < 0.f);
                        if (lane < RW) {
                            float lv;
                            asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(fabsf(vs)));
                            aux[(x * 2) * KEYS + lw * RW + lane] = ks;
                            aux[(x * 2 + 1) * KEYS + lw * RW + lane] = lv;
                        }
                    }
                    page = page_id(j + 1, &row);
                    ++step_no;
                } else {
                    const bool last = j + 1 == steps;
                    from = last ? v_next : v_off;
                    sign = last ? signs_next : signs;
                    const int slot0 = slot_first + j * KEYS;
                    if (masked(it, slot0) && entry < kTrMasked) {
                        where = static_cast<int>(i % kTrItems) * kTrMasked + entry;
                        if (lw == 0 && lane == 0) it.bad_step[entry] = slot0;
                        ++entry;
                        if (lw == 0 && lane == 0) it.bad_steps = entry;
                    }
                    if (last) {  // before it is started: that may give the item back
                        if (lane == 0) it.last_tile = issued + 1;  // (every warp the same)
                        __syncwarp();
                        ++done;
                    }
                }
                start(is_k ? 0 : 1, from, where, sign);
                if (p == 0 && ok) load_q();
            }
        }
        if (ok) flush();
        ptx::cp_async_wait<0>();
    } else if (warp == 4 + kTrLoaders) {
        // products
        if (lane == 0) {
            const uint32_t qk = tc::instr_desc(M16, KEYS, false, a.negative);
            const uint32_t pv = tc::instr_desc(M16, (a.c.dim + 15) / 16 * 16, true, false);
            const int k_steps = (a.c.dim + 15) / 16;
            uint32_t pos = 0, n_q = 0, n_p = 0;
            for (uint32_t i = 0;; ++i) {
                if (!wait(sh.item_full[i % kTrItems], i / kTrItems)) break;
                const int steps = sh.item[i % kTrItems].steps, end = sh.item[i % kTrItems].end;
                arrive(sh.item_empty[i % kTrItems]);
                if (end) break;
                const uint32_t p0 = pos, t0 = n_p;
                pos += 2 * steps;
                // places in the ring: K0 K1 V0 K2 V1 ...
                auto key_place = [&](int j) { return p0 + (j ? 2 * j - 1 : 0); };
                auto value_place = [&](int j) { return p0 + (j + 1 < steps ? 2 * j + 2 : 2 * j + 1); };
                auto first_product = [&](int j) {
                    const uint32_t p = key_place(j), tile = ring_s + p % S::SLOTS * S::TILE;
                    const int to = (t0 + j) & 1;
                    wait(sh.ring_full[p % S::SLOTS], p / S::SLOTS);
                    if (!ok) return;
                    tc::fence_after();
#pragma unroll 1
                    for (int k = 0; k < k_steps; ++k)
                        tc::mma_ss(tmem + to * 128, tc::smem_desc(q_s + k / 4 * S::QCHUNK + (k & 3) * 32, 16),
                                   tc::smem_desc(tile + k / 4 * S::CHUNK + (k & 3) * 32, 16), qk, k > 0);
                    tc::commit(bar(sh.s_full[to]));
                    tc::commit(bar(sh.ring_empty[p % S::SLOTS]));
                    if (j + 1 == steps) tc::commit(bar(sh.q_empty));
                };
                wait(sh.q_full, n_q++);
                if (!ok) break;
                tc::fence_after();
                for (int j = 0; j < 2 && j < steps && ok; ++j) first_product(j);
                for (int j = 0; j < steps && ok; ++j) {
                    const int buf = n_p & 1;
                    const uint32_t p = value_place(j), tile = ring_s + p % S::SLOTS * S::TILE;
                    wait(sh.ring_full[p % S::SLOTS], p / S::SLOTS);
                    wait(sh.p_full[buf], n_p++ >> 1);
                    if (!ok) break;
                    tc::fence_after();
#pragma unroll 1
                    for (int half = 0; half < (Q8 ? 1 : 2); ++half)
#pragma unroll
                        for (int k = 0; k < KEYS / 16; ++k)
                            tc::mma_ts(tmem + S::O, tmem + buf * 128 + k / 2 * 32 + half * 16 + (k & 1) * 8,
                                       tc::smem_desc(tile + k * 2048, S::CHUNK), pv, j > 0 || half > 0 || k > 0);
                    tc::commit(bar(sh.ring_empty[p % S::SLOTS]));
                    tc::commit(bar(sh.o_full[buf]));
                    if (j + 2 < steps) first_product(j + 2);
                }
                if (!ok) break;
            }
            // products in flight end before the tensor memory is given back
            ok = true;
            tc::commit(bar(sh.drain));
            wait(sh.drain, 0);
        }
    } else if (warp < 4) {
        // softmax and outputs, a thread a row
        const int row = warp * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);
        uint32_t n_s = 0;
        for (uint32_t i = 0; ok; ++i) {
            if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
            const TreeItem &it = sh.item[i % kTrItems];
            if (it.end) break;
            const int steps = it.steps, slot_first = it.begin + it.first * KEYS, before = it.n - it.count;
            const int at = it.row0 + row, t = static_cast<int>(fast_div(at, a.group_div)), g = at - t * a.group;
            const bool real = t < it.count;
            const bool some = __any_sync(0xffffffffu, real);
            const uint64_t kin = real ? it.kin[t] : 0;
            const int from = real ? it.from[t] : 0;
            float m = -INFINITY, less = -kSumLift, l = 0.f, mv = -INFINITY, less_v = -kLift;
            float scale2 = a.scale2;
            // the slots of 32 from slot0 that this row sees
            auto seen = [&](int slot0) {
                const int lo = max(from - slot0, 0), hi = min(before - slot0, 32);  // before the drafts
                uint32_t bits = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0;
                const int d = before - slot0;
                if (d < 32 && d > -64) bits |= static_cast<uint32_t>(d >= 0 ? kin << d : kin >> -d);
                return bits;
            };
            for (int j = 0; j < steps; ++j) {
                const int buf = n_s & 1, slot0 = slot_first + j * KEYS;
                const uint32_t s_at = lanes + buf * 128;
                if (!wait_warp(sh.s_full[buf], n_s >> 1)) break;
                const int x_at = n_s % kTrAux;
                ++n_s;
                if (Q8 && j == 0) scale2 = a.scale2 * sh.q_scale[i & 1][row];
                if (some) {
                    tc::fence_after();
                    const bool cut = masked(it, slot0);
                    bool part = cut;
#pragma unroll
                    for (int c = 0; c < KEYS / 32; ++c) part |= sh.there[x_at][c] != 0xffffffffu;
                    const float *ks = aux + (x_at * 2) * KEYS, *lv = ks + KEYS;
                    (void)ks;
                    (void)lv;
                    // the largest logits
                    float tops[4], tops_v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tops[k] = tops_v[k] = -INFINITY;
                    auto load = [&](uint32_t (&x)[32], int c) {
                        tc::ld32(x, s_at + c * 32);
                        tc::wait_ld(x);
                        if constexpr (Q8) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 s = *reinterpret_cast<const float4 *>(ks + c * 32 + e);
                                x[e] = __float_as_uint(__uint_as_float(x[e]) * (s.x * scale2));
                                x[e + 1] = __float_as_uint(__uint_as_float(x[e + 1]) * (s.y * scale2));
                                x[e + 2] = __float_as_uint(__uint_as_float(x[e + 2]) * (s.z * scale2));
                                x[e + 3] = __float_as_uint(__uint_as_float(x[e + 3]) * (s.w * scale2));
                            }
                        }
                        if (part) {
                            const uint32_t bits = sh.there[x_at][c] & (cut ? seen(slot0 + 32 * c) : 0xffffffffu);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(bits & 1u << e)) x[e] = 0xff800000u;
                        }
                    };
#pragma unroll 1
                    for (int c = 0; c < KEYS / 32; ++c) {
                        uint32_t x[32];
                        load(x, c);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            if constexpr (Q8) {
                                const float4 s = *reinterpret_cast<const float4 *>(lv + c * 32 + e);
                                const float sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    tops[k] = fmaxf(tops[k], __uint_as_float(x[e + k]));
                                    // (a slot that is not seen may have any scale)
                                    const float y = __uint_as_float(x[e + k]) + sv[k];
                                    tops_v[k] = fmaxf(tops_v[k], part && x[e + k] == 0xff800000u ? -INFINITY : y);
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], __uint_as_float(x[e + k]));
                            }
                        }
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    float top_v = fmaxf(fmaxf(tops_v[0], tops_v[1]), fmaxf(tops_v[2], tops_v[3]));
                    if constexpr (!Q8) {
                        top *= scale2;
                        top_v = top;
                    }
                    const bool rise = real && (top_v > mv + kRise || (mv == -INFINITY && top_v > mv));
                    if (Q8 && real && top > m) {
                        l *= tr_exp2(m - top);
                        m = top;
                        less = top - kSumLift;
                    }
                    if (__any_sync(0xffffffffu, rise)) {
                        const float f = rise ? tr_exp2(mv - top_v) : 1.f;
                        if (rise) {
                            mv = top_v;
                            less_v = top_v - kLift;
                            if (!Q8) {
                                l *= f;
                                m = mv;
                                less = less_v;
                            }
                        }
                        if (j > 0) {
                            if (!wait_warp(sh.o_full[n_s & 1], n_s - 2 >> 1)) break;
                            tc::fence_after();
#pragma unroll 1
                            for (int c = 0; c < (a.c.dim + 31) / 32; ++c) {
                                uint32_t o[32];
                                tc::ld32(o, lanes + S::O + c * 32);
                                tc::wait_ld(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st32(lanes + S::O + c * 32, o);
                            }
                        }
                    }
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 scale = make_float2(scale2, scale2), off2 = make_float2(-less, -less);
                    // the weights of 32 slots take the columns of their logits: 16 of leading numbers, 16 of the rests
#pragma unroll 1
                    for (int c = 0; c < KEYS / 32; ++c) {
                        uint32_t x[32], p[16], rest[16];
                        load(x, c);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 y = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                            if constexpr (Q8) {
                                const float2 s = *reinterpret_cast<const float2 *>(lv + c * 32 + e);
                                float2 z;
                                z.x = x[e] == 0xff800000u ? 0.f : tr_exp2(y.x + s.x - less_v);
                                z.y = x[e + 1] == 0xff800000u ? 0.f : tr_exp2(y.y + s.y - less_v);
                                p[e / 2] = tr_pack<true>(z.x, z.y);
                                y.x = tr_exp2(y.x - less);
                                y.y = tr_exp2(y.y - less);
                            } else {
                                y = tc::fma2(y, scale, off2);
                                y.x = tr_exp2(y.x);
                                y.y = tr_exp2(y.y);
                                tr_split<M16>(y.x, y.y, &p[e / 2], &rest[e / 2]);
                            }
                            sum[e >> 1 & 1] = tc::add2(sum[e >> 1 & 1], y);
                        }
                        tc::st16(s_at + c * 32, p);
                        if constexpr (!Q8) tc::st16(s_at + c * 32 + 16, rest);
                    }
                    const float2 both = tc::add2(sum[0], sum[1]);
                    l += both.x + both.y;
                    tc::wait_st();
                    tc::fence_before();
                }
                arrive_warp(sh.p_full[buf]);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (!wait_warp(sh.o_full[n_s - 1 & 1], n_s - 1 >> 1)) break;
            if (some) {
                tc::fence_after();
                const int hq = it.head * a.group + g;
                const bool none = l == 0.f;
                float f = none ? 0.f : 1.f / l;
                if (it.part >= 0) f = 1.f;
                if (Q8) f *= mv == -INFINITY ? 0.f : exp2f(less_v - less);  // the output was relative to mv
                uint16_t *out = a.out + it.b * a.ost[0] + t * a.ost[1] + hq * a.ost[2];
#pragma unroll 1
                for (int c = 0; c < (a.c.dim + 31) / 32; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    tc::ld32(o, lanes + S::O + c * 32);
                    tc::wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
                    for (int n = 0; n < it.bad_steps; ++n)
#pragma unroll 1
                        for (int w = 0; w < 4; ++w)
#pragma unroll 1
                            for (uint32_t left = it.bad[n][w]; left; left &= left - 1) {
                                const int slot = it.bad_step[n] + w * 32 + __ffs(left) - 1;
                                if (!real || !(seen(slot) & 1)) continue;
                                const uint8_t *v = tree_value<EB>(a, it.b, it.head, slot);
                                if (!v) continue;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (c * 32 + e < a.c.dim)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) + tree_unusual<KV>(v, c * 32 + e));
                            }
                    if (!real) {
                    } else if (it.part >= 0) {
                        float4 *to = reinterpret_cast<float4 *>(a.part) + (int64_t(it.part) * NC * 16 + c * 8) * kTrRows + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            to[e * kTrRows] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                          __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[k] = tr_pack<KV == LC_CACHE_F16>(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
                            uint16_t *to = out + c * 32 + e;
                            if (a.out_vec && c * 32 + e + 8 <= a.c.dim) {
                                *reinterpret_cast<uint4 *>(to) = make_uint4(y[0], y[1], y[2], y[3]);
                            } else {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (c * 32 + e + k < a.c.dim) to[k] = static_cast<uint16_t>(y[k / 2] >> (k & 1) * 16);
                            }
                        }
                    }
                }
                if (real && it.part >= 0) {
                    a.part_ml[int64_t(it.part) * kTrRows + row] = make_float2(m == -INFINITY ? -INFINITY : less, l);
                } else if (real && a.lse) {
                    a.lse[it.b * a.lst[0] + t * a.lst[1] + hq] =
                        none ? -INFINITY : (less + kSumLift + log2f(l * exp2f(-kSumLift))) * 0.6931471805599453f;
                }
            }
            arrive_warp(sh.item_empty[i % kTrItems]);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 4 + kTrLoaders) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// Joins the parts of the units that were cut, in their order: a block a unit and 32 rows, a warp some columns.
template <int KV, int NC>
__global__ void __launch_bounds__(256) k_tree_join(const __grid_constant__ TreeArgs a) {
    constexpr int KEYS = TreeShape<NC, KV == LC_CACHE_E4M3>::KEYS;
    constexpr float kSumLift = KV == LC_CACHE_F16 ? 12.f : -40.f;
    __shared__ int64_t all_s, before_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    start_after_prior();
    const int group = blockIdx.x % 4, unit = blockIdx.x / 4;
    const int block = unit % a.most_blocks, head = unit / a.most_blocks % a.c.heads, b = unit / a.most_blocks / a.c.heads;
    const TreeSeq s = tree_seq<KEYS>(a, b);
    const int row0 = block * kTrRows + group * 32;
    if (row0 >= s.count * a.group) return;
    if (warp == 0) {
        int64_t before;
        const int64_t all = tree_steps<KEYS>(a, b, &before);
        if (lane == 0) {
            all_s = all;
            before_s = before;
        }
    }
    __syncthreads();
    const int64_t all = all_s, u0 = before_s + (int64_t(head) * s.blocks + block) * s.steps, u1 = u0 + s.steps;
    const int runs = tree_runs(a, all);
    // the runs that hold its first and its last step
    auto run_of = [&](int64_t x) {
        int r = static_cast<int>(x * runs / all);
        while (run_begin(all, runs, r + 1) <= x) ++r;
        while (run_begin(all, runs, r) > x) --r;
        return r;
    };
    const int r0 = run_of(u0), r1 = run_of(u1 - 1);
    if (r0 == r1) return;
    const int at = row0 + lane, t = static_cast<int>(fast_div(at, a.group_div)), g = at - t * a.group;
    if (t >= s.count) return;
    const int row = group * 32 + lane;
    auto slot = [&](int r) { return int64_t(2 * r + (r == r0)); };
    float top = -INFINITY, l = 0.f;
    for (int r = r0; r <= r1; ++r) top = fmaxf(top, a.part_ml[slot(r) * kTrRows + row].x);
    const float safe = top == -INFINITY ? 0.f : top;
    for (int r = r0; r <= r1; ++r) {
        const float2 v = a.part_ml[slot(r) * kTrRows + row];
        l += v.y * tr_exp2(v.x - safe);
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = a.out + b * a.ost[0] + t * a.ost[1] + (int64_t(head) * a.group + g) * a.ost[2];
    for (int c = warp; c * 4 < a.c.dim; c += 8) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = r0; r <= r1; ++r) {
            const float w = tr_exp2(a.part_ml[slot(r) * kTrRows + row].x - safe);
            const float4 z = reinterpret_cast<const float4 *>(a.part)[(slot(r) * NC * 16 + c) * kTrRows + row];
            y.x += z.x * w;
            y.y += z.y * w;
            y.z += z.z * w;
            y.w += z.w * w;
        }
        const float v[4] = {y.x * f, y.y * f, y.z * f, y.w * f};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c * 4 + e < a.c.dim) out[c * 4 + e] = static_cast<uint16_t>(tr_pack<KV == LC_CACHE_F16>(v[e], 0.f));
    }
    if (warp == 0 && a.lse)
        a.lse[b * a.lst[0] + t * a.lst[1] + head * a.group + g] =
            l == 0.f ? -INFINITY : (top + kSumLift + log2f(l * exp2f(-kSumLift))) * 0.6931471805599453f;
}

// What a call needs of the workspace, and its launch.
template <int KV, int NC>
int launch_tree_shape(const TreeArgs &a, cudaStream_t cs) {
    using S = TreeShape<NC, KV == LC_CACHE_E4M3>;
    const void *fn = reinterpret_cast<const void *>(&k_tree_attend<KV, NC>);
    int sms = 0, per_sm = 0;
    if (prepare(fn, S::THREADS, S::SMEM, S::SMEM, &sms, &per_sm) != cudaSuccess) return LC_ERR_CUDA;
    TreeArgs b = a;
    const int64_t units = int64_t(a.c.n_seqs) * a.c.heads * a.most_blocks;
    const int64_t steps = units * ((int64_t(a.c.cap) + S::KEYS - 1) / S::KEYS);
    b.runs = static_cast<int32_t>(std::min<int64_t>(std::min(sms, kTrMostRuns), (steps + kTrLeast - 1) / kTrLeast));
    const int st = launch_after(fn, b.runs, S::THREADS, S::SMEM, cs, &b);
    if (st) return st;
    return launch_after(reinterpret_cast<const void *>(&k_tree_join<KV, NC>), static_cast<unsigned>(units * 4), 256, 0, cs, &b);
}

template <int KV>
int launch_tree_type(const TreeArgs &a, cudaStream_t cs) {
    switch ((a.c.dim + 63) / 64) {
        case 1: return launch_tree_shape<KV, 1>(a, cs);
        case 2: return launch_tree_shape<KV, 2>(a, cs);
        case 3: return launch_tree_shape<KV, 3>(a, cs);
        default: return launch_tree_shape<KV, 4>(a, cs);
    }
}

}  // namespace lc
