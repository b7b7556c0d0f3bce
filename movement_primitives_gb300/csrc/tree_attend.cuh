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
// values' the weights, which are one float16 number each, relative to a maximum mv of x
// + log2 |s|: of a bound of it, the largest x and the largest scale of a step, while
// scales of a step lie within 2^kNear of one another, and of the maximum itself where
// they do not.
//
// Work.  A (sequence, key head, tile of rows) is a unit; the steps of all units, laid
// end to end, are cut into equal runs, one a block, found from the lengths on
// the device.  A unit inside one run is finished there; a cut one leaves
// parts in the workspace, which k_tree_join joins in their order, so results do not
// depend on timing.  Where pages allow it (launcher) keys and values come by tensor
// copies, boxes of a page's slots, else four warps bring them in by asynchronous 16-byte
// copies or an element at a time, several tiles ahead; those warps also bring in the rows of q and turn
// E4M3 codes into float16.  One warp issues the products; eight do the softmax, two of
// them a row's (each half of the slots; they exchange their maxima).
//
// What bounds it, by GB300 figures of the kernels alone.  16 sequences of up to 4096
// slots, 8 key heads of 128, 64 rows each, bfloat16 (143 MB): 44 us, 3.3 TB/s, where a steady step runs at
// the memory's rate; the rest is the scheduler's reads, the first rows, the parts' way through
// the L2 and the joining (6 us).  12 sequences of up to 32767, 128 rows, E4M3 (443 MB): 217 us, bound by the
// softmax warps (3400 of 3900 cycles a step): two multiplications by scales more than
// in bfloat16, beside the conversions.  One of 301 slots: 10 us, the chain from the
// lengths to the output.  By copies of the four warps alone the first took 84 us and the second 678.
#pragma once

#include <cuda.h>

#include "cache_common.cuh"
#include "tensor_core.cuh"

namespace lc {

constexpr uint32_t kClassTree = 0xf4;
constexpr int kTrRows = 128;
constexpr int kTrDrafts = LC_CACHE_MAX_DRAFTS;
constexpr int kTrItems = 4;      // pieces that the scheduling warp may be ahead
constexpr int kTrMasked = 4;     // steps of a piece that some row sees in part: two at either end at most
constexpr int kTrAux = 8;        // steps whose slots' scales and presence are held
constexpr int kTrLoaders = 4;    // warps
constexpr int kTrSoft = 8;       // warps: two a 32 rows, each half of a step's slots
constexpr int kTrMostRuns = 160;
constexpr float kNear = 8.f, kFar = 60.f;  // log2 of scales that are near one another, and of ones that are not too far from 1

template <int KV>
constexpr float kTrLift = KV == LC_CACHE_BF16 ? -24.f : 8.f;  // log2 of what weights are multiplied by

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
    int32_t q_least;        // E4M3: log2 of what rows of q are divided by at least
    int32_t vec, q_vec, out_vec;  // rows of the pools, of q and of out are whole 16-byte words on 16-byte boundaries
    int32_t runs, least;    // blocks of the main kernel; steps of a run at least
    int32_t whole;          // not 0: units are not cut, nothing is joined
    int32_t most_blocks;    // tiles of rows a key head at most
    int4 *split;            // [runs]: the unit that is cut at the run's end (sequence, -1 for none, head, tile), its last run
    float *part;            // [2 runs][dim / 4 rounded up to 16][128 rows][4]
    float2 *part_ml;        // [2 runs][128]
    int32_t box;            // slots of a tensor copy
    FastDiv piece_div;      // by the 16-byte pieces of a row of codes
    uint64_t limit_ns;
    CUtensorMap km, vm;
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
    s.begin = a.window ? max(s.n - s.count + 1 - a.window, 0) / a.box * a.box : 0;
    s.blocks = (s.count * a.group + kTrRows - 1) / kTrRows;
    s.steps = s.count ? (s.n - s.begin + KEYS - 1) / KEYS : 0;
    return s;
}

// Steps of all units (where they stay whole: units), by a warp.
template <int KEYS>
__device__ __forceinline__ int tree_steps(const TreeArgs &a, const TreeSeq &first) {  // (of the sequence of this lane's number)
    const int lane = threadIdx.x & 31;
    auto of = [&](const TreeSeq &s) { return (a.whole ? min(s.steps, 1) : s.steps) * s.blocks * a.c.heads; };
    int all = of(first);
#pragma unroll 4
    for (int b = lane + 32; b < a.c.n_seqs; b += 32) {
        const TreeSeq s = tree_seq<KEYS>(a, b);
        all += of(s);
    }
    return __reduce_add_sync(0xffffffffu, all);
}

// The runs that `all` steps are cut into: run r begins at r * each + min(r, more).
struct TreeRuns {
    int runs, each, more;
    __device__ __forceinline__ TreeRuns(const TreeArgs &a, int all)
        : runs(min((all + a.least - 1) / a.least, a.runs)), each(all / max(runs, 1)), more(all - each * max(runs, 1)) {}
    __device__ __forceinline__ int begin(int r) const { return r * each + min(r, more); }
    __device__ __forceinline__ int of(int step) const {
        const int wide = more * (each + 1);
        return step < wide ? step / (each + 1) : more + (step - wide) / each;
    }
};

// A piece of a run: steps first .. first + steps - 1 of a unit.
struct TreeItem {
    int32_t b, head, row0;      // row0: the tile's first row, draft * group + query head of the group
    int32_t n, count, begin;
    int32_t first, steps;
    int32_t part;               // where its part goes, -1 for a whole unit
    int32_t end;
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
    static constexpr int SHARED = 12288 + (Q8 ? kTrAux * KEYS * 12 : 0);  // the block of barriers and items, and 1024 for alignment
    static constexpr int FIT = (232448 - SHARED - Q - RAW * RAW_TILE) / TILE;
    // (what kTrAux holds is read before tiles this far on are started)
    static constexpr int SLOTS = Q8 ? (FIT < 6 ? FIT : 6) : (FIT < 12 ? FIT : 12);
    static constexpr int LAG = Q8 ? RAW - 1 : SLOTS / 2;   // tiles under way
    static constexpr int SMEM = Q + RAW * RAW_TILE + SLOTS * TILE + SHARED;
    static constexpr int THREADS = 32 * (kTrSoft + kTrLoaders + 4);  // products, scheduling, two idle
    static constexpr int O = 256;                          // first output column of tensor memory
    static_assert(SLOTS >= 3 && LAG < SLOTS + (Q8 ? RAW : 0), "keys of two steps and values of one");
};

struct TreeShared {
    uint64_t ring_full[12], ring_empty[12];
    uint64_t q_full, q_empty;
    uint64_t raw_full[4], raw_empty[4];
    uint64_t s_full[2], p_full[2], o_full[2];  // of every other step
    uint64_t item_full[kTrItems], item_empty[kTrItems], kin_full[kTrItems];
    uint64_t pair[4];               // of the two warps of 32 rows
    uint64_t drain;
    uint32_t tmem;
    float top[2][2][kTrRows], top_v[2][2][kTrRows];  // [step parity][half of the slots][row]
    float sum[2][kTrRows];
    uint32_t there[kTrAux][4];      // the slots of a step that exist and whose pages do
    float2 range[kTrAux][kTrLoaders];  // E4M3: largest and least log2 of a step's values' scales, NaN for far ones
    float q_scale[2][kTrRows];      // E4M3: what a row of q was divided by
    TreeItem item[kTrItems];
};
static_assert(sizeof(TreeShared) <= 11264, "the shared block has 11264 bytes");

__device__ __forceinline__ float tr_exp2(float x) {  // 2 ulp, 0 for -infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float tr_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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
__device__ __forceinline__ void tr_halves(uint32_t codes, uint32_t *lo, uint32_t *hi) {  // four E4M3 codes as float16, exactly
    asm("{.reg .b16 c, d; mov.b32 {c, d}, %2; cvt.rn.f16x2.e4m3x2 %0, c; cvt.rn.f16x2.e4m3x2 %1, d;}"
        : "=r"(*lo), "=r"(*hi)
        : "r"(codes));
}
__device__ __forceinline__ void tr_copy16(uint32_t dst, const void *src, bool real) {  // zeros where there is nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_global16(void *dst, uint4 v, bool does) {  // by predicate: the warp stays together
    asm volatile("{.reg .pred p; setp.ne.b32 p, %5, 0; @p st.global.v4.b32 [%0], {%1, %2, %3, %4};}" ::"l"(dst), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w), "r"(static_cast<uint32_t>(does))
                 : "memory");
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

// Values that are not finite become 0; whether there was one.
template <int KV>
__device__ __forceinline__ bool tree_clean(uint4 &x) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    bool found = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t off;  // of the elements that are not finite, all bits
        if constexpr (KV == LC_CACHE_E4M3) {
            const uint32_t nan = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            off = nan | (nan - (nan >> 7));
        } else {
            constexpr uint32_t kExp = KV == LC_CACHE_F16 ? 0x7c00u : 0x7f80u;
            off = ((w[e] & kExp) == kExp ? 0xffffu : 0u) | ((w[e] & kExp << 16) == kExp << 16 ? 0xffff0000u : 0u);
        }
        found |= off != 0;
        w[e] &= ~off;
    }
    return found;
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

// The rows of q of a piece into shared memory, RQ a warp from row0 on: float16 copies of bfloat16 rows for E4M3 caches,
// divided by a power of two so that a row's largest element is between 1 and 2 (`scale`: by which; rows that are smaller than that, and zeros, by 2^q_least).
template <int KV, int NC, int RQ>
__device__ __forceinline__ void tree_query(const TreeArgs &a, const TreeItem &it, int row0, uint32_t q_s, float *scale) {
    constexpr bool Q8 = KV == LC_CACHE_E4M3;
    constexpr int PQ = NC * 8, CHUNK = kTrRows * 128;  // 16-byte pieces of a row; bytes of 64 columns
    const int lane = threadIdx.x & 31;
    auto q_at = [&](int r, int piece) {
        return q_s + piece / 8 * CHUNK + (row0 + r) * 128 + ((piece & 7) ^ (r & 7)) * 16;
    };
    auto q_piece = [&](int r, int col) {
        const int at = it.row0 + row0 + r, t = static_cast<int>(fast_div(at, a.group_div)), g = at - t * a.group;
        const bool real = t < it.count && col < a.c.dim;
        const uint16_t *from = a.q + (real ? it.b * a.qst[0] + t * a.qst[1] + (int64_t(it.head) * a.group + g) * a.qst[2] + col : 0);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (a.q_vec) {
            if (real) x = *reinterpret_cast<const uint4 *>(from);
        } else if (real) {
            x = tree_piece<2>(reinterpret_cast<const uint8_t *>(from - col), col, a.c.dim);
        }
        return x;
    };
    if constexpr (!Q8) {
#pragma unroll 1
        for (int r0 = 0; r0 < RQ; r0 += 16) {  // 16 rows on the way at once, 4 NC pieces a lane
            uint4 x[4 * NC];
#pragma unroll
            for (int k = 0; k < 4 * NC; ++k) x[k] = q_piece(r0 + (k * 32 + lane) / PQ, (k * 32 + lane) % PQ * 8);
#pragma unroll
            for (int k = 0; k < 4 * NC; ++k) st_shared16(q_at(r0 + (k * 32 + lane) / PQ, (k * 32 + lane) % PQ), x[k]);
        }
    } else {
#pragma unroll 1
        for (int r0 = 0; r0 < RQ; r0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = q_piece(r0 + r, lane * 8);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                uint32_t *w = reinterpret_cast<uint32_t *>(&x[r]);
                uint32_t most = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) most = max(most, max(w[e] << 16 & 0x7fffffffu, w[e] & 0x7fff0000u));
                most = __reduce_max_sync(0xffffffffu, most);
                const int ex = min(max(static_cast<int>(most >> 23) - 127, a.q_least), 126);
                const float div = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = tr_pack<true>(__uint_as_float(w[e] << 16) * div, __uint_as_float(w[e] & 0xffff0000u) * div);
                scale[row0 + r0 + r] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);  // (by all lanes)
                if (lane < PQ) st_shared16(q_at(r0 + r, lane), x[r]);
            }
        }
    }
    tc::fence_async_smem();
}

// TMA: pages come by tensor copies, a box of a page's slots each, which a warp issues (E4M3 ones go through four more
// that convert them); else element by element or 16 bytes, by four warps.
template <int KV, int NC, bool TMA>
__global__ void __launch_bounds__(TreeShape<NC, KV == LC_CACHE_E4M3>::THREADS, 1)
    k_tree_attend(const __grid_constant__ TreeArgs a) {
    constexpr bool Q8 = KV == LC_CACHE_E4M3, M16 = KV != LC_CACHE_BF16;  // float16 products
    using S = TreeShape<NC, Q8>;
    constexpr int KEYS = S::KEYS, EB = Q8 ? 1 : 2;
    constexpr int kIssuer = kTrSoft + kTrLoaders + 2;  // the warp that issues tensor copies
    // weights are up to 2^(kLift + kRise): float16 has few exponents, so small ones are lifted into them; others are
    // lowered, as sums are, so that those of the type's largest values stay in float32 (2^24 of them, 2^16 where the
    // maximum is 2^kRise behind), and by no more: exponents below 32 lose 2^-20, below 64 2^-19
    constexpr float kRise = M16 ? 6.f : 8.f, kLift = kTrLift<KV>, kSumLift = Q8 ? 0.f : kLift;
    extern __shared__ uint8_t raw_smem[];
    const uint32_t base = (ptx::smem_addr(raw_smem) + 1023) & ~1023u;
    const uint32_t q_s = base, ring_s = q_s + S::Q, raw_s = ring_s + S::SLOTS * S::TILE;
    uint8_t *const after = raw_smem + (base - ptx::smem_addr(raw_smem)) + S::Q + S::SLOTS * S::TILE + S::RAW * S::RAW_TILE;
    TreeShared &sh = *reinterpret_cast<TreeShared *>(after);
    float *const aux = reinterpret_cast<float *>(after + 11264);  // E4M3: [kTrAux][keys' scales, values', log2 of those][KEYS]
    // (shuffled, so that the compiler knows a warp's branches on it to be the whole warp's)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    auto bar = [&](const uint64_t &b) { return ptx::smem_addr(&b); };

    if (warp == kTrSoft + kTrLoaders) tc::alloc(ptx::smem_addr(&sh.tmem), 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::SLOTS; ++i) {
            ptx::mbar_init(bar(sh.ring_full[i]), TMA && !Q8 ? 1 : kTrLoaders);
            ptx::mbar_init(bar(sh.ring_empty[i]), 1);
        }
        ptx::mbar_init(bar(sh.q_full), kTrLoaders);
        for (int i = 0; i < S::RAW; ++i) {
            ptx::mbar_init(bar(sh.raw_full[i]), 1);
            ptx::mbar_init(bar(sh.raw_empty[i]), kTrLoaders);
        }
        ptx::mbar_init(bar(sh.q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(sh.s_full[i]), 1);
            ptx::mbar_init(bar(sh.p_full[i]), kTrSoft);
            ptx::mbar_init(bar(sh.o_full[i]), 1);
        }
        for (int i = 0; i < kTrItems; ++i) {
            ptx::mbar_init(bar(sh.item_full[i]), 1);
            // the softmax's, the products', and what brings the tiles
            ptx::mbar_init(bar(sh.item_empty[i]), kTrSoft + 1 + kTrLoaders + TMA);
            ptx::mbar_init(bar(sh.kin_full[i]), 1);
            ptx::mbar_init(bar(sh.pair[i]), 2);
        }
        ptx::mbar_init(bar(sh.drain), 1);
        ptx::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (joining blocks that come early take what this one needs)

    bool ok = true;  // no wait of this warp has run out
    auto arrive_warp = [&](const uint64_t &b) { tc::arrive(bar(b)); };
    auto wait_warp = [&](const uint64_t &b, uint32_t n) {  // for phase n (counted from 0)
        if (ok && !tc::wait(bar(b), n, a.limit_ns)) {
            ok = false;
            note_error(LC_ERR_TIMEOUT, kClassTree);
        }
        return ok;
    };
    auto drained = [&](const uint64_t &b, uint32_t n) {  // what was started ends, however short the limit
        if (!tc::wait(bar(b), n, max(a.limit_ns, uint64_t(2000000000)))) note_error(LC_ERR_TIMEOUT, kClassTree);
    };
    auto done_warp = [&](const uint64_t &b, uint32_t n) { return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar(b), n & 1)) != 0; };
    // whether some row of a piece sees a step in part
    auto masked = [&](const TreeItem &it, int slot0) {
        return slot0 + KEYS > it.n - it.count || (a.window && slot0 < it.n - it.count + kTrDrafts - a.window);
    };

    // of a block's registers the softmax threads take the larger part (512 x 128 = 256 x 152 + 256 x 104)
    auto few_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); };
    if (warp == kTrSoft + kTrLoaders + 1) {
        few_registers();
        // scheduling: the pieces of this block's run
        int at = 0, from = 0, to = 0;
        int4 cut = make_int4(-1, 0, 0, 0);  // for the joining
        TreeSeq seq0{};
        if (lane < a.c.n_seqs) seq0 = tree_seq<KEYS>(a, lane);
        const TreeRuns runs(a, tree_steps<KEYS>(a, seq0));
        if (static_cast<int>(blockIdx.x) < runs.runs) {
            from = runs.begin(blockIdx.x);
            to = runs.begin(blockIdx.x + 1);
        }
        uint32_t i = 0;
        auto post = [&](auto &&fill) {
            const int s = i % kTrItems;
            if (i >= kTrItems && !wait_warp(sh.item_empty[s], i / kTrItems - 1)) return;
            TreeItem &it = sh.item[s];
            fill(it);
            arrive_warp(sh.item_full[s]);
            if (!it.end) {  // only the softmax waits for this
                tree_kin(a, it);
                arrive_warp(sh.kin_full[s]);
            }
            ++i;
        };
#pragma unroll 1
        for (int b0 = 0; b0 < a.c.n_seqs && from < to && ok; b0 += 32) {
            const TreeSeq s = seq0;
            seq0 = TreeSeq{};  // the next 32, read while these are gone through
            if (b0 + 32 + lane < a.c.n_seqs) seq0 = tree_seq<KEYS>(a, b0 + 32 + lane);
            const int w = (a.whole ? min(s.steps, 1) : s.steps) * s.blocks * a.c.heads;
            int upto = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            while (from < to && ok) {
                const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && at + upto > from);
                if (!hit) break;
                const int l = __ffs(hit) - 1;
                const int steps = __shfl_sync(0xffffffffu, s.steps, l), blocks = __shfl_sync(0xffffffffu, s.blocks, l);
                const int n = __shfl_sync(0xffffffffu, s.n, l), count = __shfl_sync(0xffffffffu, s.count, l);
                const int begin = __shfl_sync(0xffffffffu, s.begin, l);
                const int in = from - at - __shfl_sync(0xffffffffu, upto - w, l);
                const int unit = a.whole ? in : in / steps, first = a.whole ? 0 : in - unit * steps;
                const int take = a.whole ? steps : min(to - from, steps - first);
                if (first == 0 && take < steps) cut = make_int4(b0 + l, unit / blocks, unit % blocks, runs.of(from + steps - 1));
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
                    }
                    if (lane < 4 * kTrMasked) it.bad[lane / 4][lane % 4] = 0;
                    __syncwarp();
                });
                from += a.whole ? 1 : take;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (ok) post([&](TreeItem &it) { if (lane == 0) it.end = 1; });
        if (!a.whole) a.split[blockIdx.x] = cut;  // (by every lane)
    } else if (TMA && warp == kIssuer) {
        few_registers();
        if constexpr (TMA) {
            // tensor copies: a lane looks after 4 (2) slots, and issues the box that begins with them
            constexpr int G = KEYS / 32;
            uint32_t step_no = 0;
            int b = 0, head = 0, n = 0, slot_first = 0, steps = 0;
            int page = 0, row = 0, page_next = 0, row_next = 0, page_v = 0, row_v = 0;  // (n_pages: nowhere, read as zeros)
            const int nowhere = static_cast<int>(a.c.n_pages);
            bool here_next = false;
            float ks[G], vs[G];
            const int64_t last_at = int64_t(a.c.n_seqs - 1) * a.c.table_stride + a.c.per - 1;  // of the table
            auto page_id = [&](int j) {
                const int slot = slot_first + j * KEYS + lane * G;
                const bool here = j < steps && slot < n;
                const int at = static_cast<int>(fast_div(slot, a.c.page_div));
                row_next = here ? slot - at * a.c.page : 0;
                page_next = a.c.table[here ? b * a.c.table_stride + at : last_at];
                here_next = here;
            };
            auto turn_page = [&](int j) {  // step j's page and scales, and the next one's page asked for
                const bool good = page_next >= 0 && page_next < a.c.n_pages;
                if (__any_sync(0xffffffffu, here_next && !good)) note_error(LC_ERR_CACHE_INDEX, kClassTree);
                page = here_next && good ? page_next : nowhere;
                row = row_next;
                if constexpr (Q8) {
                    const int from = page != nowhere ? page : 0;
                    const int64_t k_at = row_offset(a.c.kss, from, head, row), v_at = row_offset(a.c.vss, from, head, row);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const bool there = page != nowhere && slot_first + j * KEYS + lane * G + g < n;
                        const float k = a.c.ks[k_at + g * a.c.kss[2]], v = a.c.vs[v_at + g * a.c.vss[2]];
                        ks[g] = there ? k : 0.f;
                        vs[g] = there ? v : 0.f;
                    }
                }
                page_id(j + 1);
            };
            const uint32_t tile_bytes = Q8 ? KEYS * a.c.dim : S::TILE;
            const int boxes = KEYS / a.box, lanes_box = a.box / G;
            constexpr uint32_t M = Q8 ? (S::RAW ? S::RAW : 1) : S::SLOTS;  // tiles under way at most
            uint32_t at = 0, round = 0;  // the next tile's place among them, and how often that has been used
            auto issue = [&](const CUtensorMap &map, int at_page, int at_row) {
                __syncwarp();
                const uint32_t full = bar(Q8 ? sh.raw_full[0] : sh.ring_full[0]) + at * 8;
                tc::expect(full, tile_bytes);
                const uint32_t dst = Q8 ? raw_s + at * S::RAW_TILE : ring_s + at * S::TILE;
#pragma unroll 1
                for (int k = 0; k < boxes; ++k) {
                    const int pg = __shfl_sync(0xffffffffu, at_page, k * lanes_box);
                    const int rw = __shfl_sync(0xffffffffu, at_row, k * lanes_box);
                    if constexpr (Q8) {
                        tc::load_4d(dst + k * a.box * a.c.dim, &map, 0, rw, head, pg, full);
                    } else {
#pragma unroll
                        for (int c = 0; c < NC; ++c) tc::load_4d(dst + c * S::CHUNK + k * a.box * 128, &map, c * 64, rw, head, pg, full);
                    }
                }
                if (++at == M) {
                    at = 0;
                    ++round;
                }
            };
            auto room = [&] {  // for the next tile
                return round == 0 || wait_warp(*((Q8 ? sh.raw_empty : sh.ring_empty) + at), round - 1);
            };
            for (uint32_t i = 0; ok; ++i) {
                if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
                const TreeItem &it = sh.item[i % kTrItems];
                if (it.end) break;
                b = (it.b);
                head = (it.head);
                n = (it.n);
                slot_first = (it.begin + it.first * KEYS);
                steps = (it.steps);
                arrive_warp(sh.item_empty[i % kTrItems]);
                page_id(0);
                turn_page(0);
#pragma unroll 1
                for (int p = 0; p < 2 * steps; ++p) {  // K0 K1 V0 K2 V1 ...
                    if (!room()) break;
                    const bool is_k = p == 0 || (p & 1 && p < 2 * steps - 1);
                    if (is_k) {
                        const int j = (p + 1) / 2, slot0 = slot_first + j * KEYS, x = step_no % kTrAux;
                        // which slots there are: bits of those before the end whose pages there are
                        const uint32_t pages = __ballot_sync(0xffffffffu, page != nowhere), word = lane % (KEYS / 32);
                        uint32_t bits = 0;
#pragma unroll
                        for (int k = 0; k < 32 / G; ++k) bits |= (pages >> (word * (32 / G) + k) & 1) * (((1u << G) - 1) << k * G);
                        const int left = min(max(n - slot0 - static_cast<int>(word) * 32, 0), 32);
                        bits &= left ? 0xffffffffu >> (32 - left) : 0u;
                        sh.there[x][word] = bits;  // (eight lanes the same)
                        if constexpr (Q8) {
                            float most = -INFINITY, least = INFINITY;
                            bool odd = false;
#pragma unroll
                            for (int g = 0; g < G; ++g) {
                                float lv;
                                asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(fabsf(vs[g])));
                                aux[(x * 3) * KEYS + lane * G + g] = ks[g];
                                aux[(x * 3 + 1) * KEYS + lane * G + g] = vs[g];
                                aux[(x * 3 + 2) * KEYS + lane * G + g] = lv;
                                if (page != nowhere && vs[g] != 0.f) {
                                    most = fmaxf(most, lv);
                                    least = fminf(least, lv);
                                    odd |= !(fabsf(lv) <= kFar);
                                }
                            }
                            // by quarters of the warp: the largest and the least, NaN where there is a far one
#pragma unroll
                            for (int d = 4; d; d >>= 1) {
                                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                                least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
                            }
                            odd = __any_sync(0xffffffffu, odd);
                            if (lane % 8 == 0) sh.range[x][lane / 8] = odd ? make_float2(NAN, NAN) : make_float2(most, least);
                        }
                        const int k_page = page, k_row = row;
                        if (p == 0) {
                            page_v = page;
                            row_v = row;
                        }
                        turn_page(j + 1);
                        ++step_no;
                        issue(a.km, k_page, k_row);
                        if (p > 0) {  // the values of the step before follow, then this step's are next
                            if (!room()) break;
                            issue(a.vm, page_v, row_v);
                            page_v = k_page;
                            row_v = k_row;
                            ++p;
                        }
                    } else {
                        issue(a.vm, page_v, row_v);
                    }
                }
            }
            // copies in flight end before the block does
            for (uint32_t k = 0; k < M; ++k) {
                const uint32_t used = round + (k < at);
                if (used) drained(*((Q8 ? sh.raw_full : sh.ring_full) + k), used - 1);
            }
        }
    } else if (TMA && warp >= kTrSoft && warp < kTrSoft + kTrLoaders) {
        few_registers();
        if constexpr (TMA) {
            // the rows of q; E4M3: codes to float16, every lane the same pieces of a tile, 16 codes each
            const int lw = warp - kTrSoft, pieces = KEYS * a.c.dim / 16;
            uint32_t tiles = 0;
            (void)pieces;
            (void)tiles;
            for (uint32_t i = 0; ok; ++i) {
                if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
                TreeItem &it = sh.item[i % kTrItems];
                if (it.end) break;
                const int steps = it.steps, slot_first = it.begin + it.first * KEYS;
                int entry = 0;
                if (i && !wait_warp(sh.q_empty, i - 1)) break;
                tree_query<KV, NC, kTrRows / kTrLoaders>(a, it, lw * (kTrRows / kTrLoaders), q_s, sh.q_scale[i & 1]);
                arrive_warp(sh.q_full);
                if constexpr (Q8) {
#pragma unroll 1
                    for (int p = 0; p < 2 * steps; ++p, ++tiles) {
                        const uint32_t slot = tiles % S::SLOTS, raw = tiles % S::RAW;
                        if (!wait_warp(sh.raw_full[raw], tiles / S::RAW)) break;
                        if (tiles >= S::SLOTS && !wait_warp(sh.ring_empty[slot], tiles / S::SLOTS - 1)) break;
                        int where = -1, there = 0;  // there: rows that somebody may see
                        if (p && (!(p & 1) || p == 2 * steps - 1)) {  // values
                            const int slot0 = slot_first + (p == 2 * steps - 1 ? steps - 1 : p / 2 - 1) * KEYS;
                            if (masked(it, slot0) && entry < kTrMasked) where = entry++;
                            there = it.n - slot0;
                        }
                        const uint32_t from = raw_s + raw * S::RAW_TILE, to = ring_s + slot * S::TILE;
                        if (where >= 0) {
#pragma unroll 1
                            for (int k = lw * 32 + lane; k < pieces; k += 32 * kTrLoaders) {
                                uint4 x = ld_shared16(from + k * 16);
                                if (tree_clean<KV>(x)) {
                                    const int row = static_cast<int>(fast_div(k, a.piece_div));
                                    if (row < there) atomicOr(&it.bad[where][row >> 5], 1u << (row & 31));
                                    st_shared16(from + k * 16, x);
                                }
                            }
                            __syncwarp();
                        }
                        // (lanes past the last piece convert that one too: no branch parts the warp)
#pragma unroll 1
                        for (int k0 = lw * 32 + lane; k0 < pieces + lane; k0 += 4 * 32 * kTrLoaders) {
                            uint4 x[4];
                            int k[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                k[g] = min(k0 + g * 32 * kTrLoaders, pieces - 1);
                                x[g] = ld_shared16(from + k[g] * 16);
                            }
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const int row = static_cast<int>(fast_div(k[g], a.piece_div)), piece = k[g] - row * static_cast<int>(a.piece_div.d);
                                const uint32_t *w = reinterpret_cast<const uint32_t *>(&x[g]);
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 4; ++e) tr_halves(w[e], &y[2 * e], &y[2 * e + 1]);
                                const uint32_t at = to + piece / 4 * S::CHUNK + row * 128 + ((piece & 3) * 2 ^ (row & 7)) * 16;
                                st_shared16(at, make_uint4(y[0], y[1], y[2], y[3]));
                                st_shared16(at ^ 16, make_uint4(y[4], y[5], y[6], y[7]));
                            }
                        }
                        tc::fence_async_smem();
                        arrive_warp(sh.ring_full[slot]);
                        arrive_warp(sh.raw_empty[raw]);
                    }
                }
                arrive_warp(sh.item_empty[i % kTrItems]);
            }
        }
    } else if (!TMA && warp >= kTrSoft && warp < kTrSoft + kTrLoaders) {
        few_registers();
        if constexpr (!TMA) {
            // loads
            constexpr int RW = KEYS / kTrLoaders, PR = S::TILE / KEYS / 16 * EB / 2;  // rows of a warp, 16-byte pieces of a row
            constexpr int ITER = RW * PR / 32;
            const int lw = warp - kTrSoft, dim = a.c.dim, dim16 = (dim + 15) / 16 * 16;
            const uint8_t *const pool[2] = {a.c.k, a.c.v};
            uint32_t issued = 0, given = 0, n_q = 0;  // tiles started and given to the products, tiles of q
            uint32_t back = 0, done = 0;              // items given back, and whose tiles have all been started
            int32_t note[S::LAG + 1];  // of the tiles under way: values of masked steps (item * kTrMasked + entry, else -1)
#pragma unroll
            for (int i = 0; i <= S::LAG; ++i) note[i] = -1;
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
                const bool found = tree_clean<KV>(x);
                if (found) atomicOr(&sh.item[where / kTrMasked].bad[where % kTrMasked][row >> 5], 1u << (row & 31));
                return found;
            };
            // the oldest tile under way has landed: gives it to the products
            auto give = [&]() {
                const uint32_t slot = given % S::SLOTS;
                const int32_t where = note[0];
#pragma unroll
                for (int i = 0; i < S::LAG; ++i) note[i] = note[i + 1];
                if constexpr (Q8) {
                    if (given >= S::SLOTS && !wait_warp(sh.ring_empty[slot], given / S::SLOTS - 1)) return;
                    const uint32_t from = raw_s + given % S::RAW * S::RAW_TILE + (lw * ITER * 32 + lane) * 16;
                    if (where >= 0) {
#pragma unroll 1
                        for (int i = 0; i < ITER; ++i) {
                            int row, col;
                            piece_of(i, &row, &col);
                            if (col >= dim16) continue;
                            uint4 x = ld_shared16(from + i * 512);
                            if (look(x, where, lw * RW + row)) st_shared16(from + i * 512, x);
                        }
                    }
#pragma unroll
                    for (int i0 = 0; i0 < ITER; i0 += 4) {
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4 && i0 + i < ITER; ++i) x[i] = ld_shared16(from + (i0 + i) * 512);
#pragma unroll
                        for (int i = 0; i < 4 && i0 + i < ITER; ++i) {
                            int row, col;
                            piece_of(i0 + i, &row, &col);
                            if (col >= dim16) continue;
                            const uint32_t *w = reinterpret_cast<const uint32_t *>(&x[i]);
                            uint32_t y[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) tr_halves(w[e], &y[2 * e], &y[2 * e + 1]);
                            const uint32_t at = tile_at(slot, lw * RW + row, col);
                            st_shared16(at, make_uint4(y[0], y[1], y[2], y[3]));
                            st_shared16(at ^ 16, make_uint4(y[4], y[5], y[6], y[7]));  // (col is a multiple of 16)
                        }
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
            // Where a row has a power of two of pieces, a lane's are all the same column, and rows eight apart lie alike.
            constexpr int SPOTS = PR >= 32 ? 8 : 8 * PR / 32 > 0 ? 8 * PR / 32 : 1;
            const bool plain = a.vec && dim == dim16;
            const int first_col = lane % PR * (16 / EB);
            uint32_t spot[SPOTS];
#pragma unroll
            for (int i = 0; i < SPOTS; ++i) {
                const int row = i * (32 / PR) + lane / PR;
                spot[i] = tile_at(0, lw * RW + row, first_col) - ring_s;
            }
            // starts a tile of pool w from the rows at `from`
            auto start = [&](int w, int64_t from, int32_t where) {
                const uint32_t slot = issued % S::SLOTS;
                if (!Q8 && issued >= S::SLOTS && !wait_warp(sh.ring_empty[slot], issued / S::SLOTS - 1)) return;
                if (32 % PR == 0 && plain && __all_sync(0xffffffffu, from >= 0 || lane >= RW)) {
                    // every lane the same piece of one row after another: a pointer by shuffle, two additions and a copy
                    const uint8_t *const mine = pool[w] + from * EB;
                    const uint32_t dst = Q8 ? raw_s + issued % S::RAW * S::RAW_TILE + (lw * ITER * 32 + lane) * 16 : ring_s + slot * S::TILE;
#pragma unroll
                    for (int i0 = 0; i0 < ITER; i0 += 8) {
                        const uint8_t *src[8];
#pragma unroll
                        for (int i = 0; i < 8 && i0 + i < ITER; ++i)
                            src[i] = reinterpret_cast<const uint8_t *>(__shfl_sync(
                                0xffffffffu, reinterpret_cast<uint64_t>(mine), (i0 + i) * (32 / PR) + lane / PR));
#pragma unroll
                        for (int i = 0; i < 8 && i0 + i < ITER; ++i)
                            if (first_col < dim)
                                ptx::cp_async16(Q8 ? dst + (i0 + i) * 512 : dst + spot[i % SPOTS] + (i0 + i) / SPOTS * SPOTS * (32 / PR) * 128,
                                                src[i] + first_col * EB);
                    }
                } else {
                // the rows' places, eight ahead of their copies
#pragma unroll
                for (int i0 = 0; i0 < ITER; i0 += 8) {
                    int64_t place[8];
#pragma unroll
                    for (int i = 0; i < 8 && i0 + i < ITER; ++i) {
                        int row, col;
                        piece_of(i0 + i, &row, &col);
                        place[i] = __shfl_sync(0xffffffffu, from, row);
                    }
#pragma unroll
                    for (int i = 0; i < 8 && i0 + i < ITER; ++i) {
                        int row, col;
                        piece_of(i0 + i, &row, &col);
                        if (col >= dim16) continue;
                        const uint32_t dst = Q8 ? raw_s + issued % S::RAW * S::RAW_TILE + ((lw * ITER + i0 + i) * 32 + lane) * 16
                                                : tile_at(slot, lw * RW + row, col);
                        const bool real = place[i] >= 0 && col < dim;
                        const uint8_t *src = pool[w] + (real ? place[i] * EB : 0);
                        if (a.vec) tr_copy16(dst, src + (real ? col * EB : 0), real);
                        else st_shared16(dst, real ? tree_piece<EB>(src, col, dim) : make_uint4(0, 0, 0, 0));
                    }
                }
                }
                ptx::cp_async_commit();
#pragma unroll
                for (int i = 0; i <= S::LAG; ++i)
                    if (issued - given == static_cast<uint32_t>(i)) note[i] = where;
                ++issued;
            };
            uint32_t step_no = 0;  // steps of all pieces
            uint32_t i = 0;        // pieces taken
            // the piece: its next tile in the order K0 K1 V0 K2 V1 ..., 2 * steps when all have been started
            TreeItem *it = nullptr;
            int b = 0, head = 0, n = 0, slot_first = 0, steps = 0, p = 0, entry = 0;
            bool q_due = false, end = false;
            int64_t v_off = -1, v_next = -1;   // rows of the values of the step whose keys were started last, and the one before
            // of this lane's slots: pages two steps ahead, scales one
            int row = 0, page = -1, row_next = 0, page_next = -1;
            float ks = 0.f, vs = 0.f;
            auto page_id = [&](int j) {
                const int slot = slot_first + j * KEYS + lw * RW + lane;
                page_next = -1;
                if (lane >= RW || j >= steps || slot >= n) return;
                const int at = static_cast<int>(fast_div(slot, a.c.page_div));
                row_next = slot - at * a.c.page;
                page_next = a.c.table[b * a.c.table_stride + at];
                if (page_next >= 0 && page_next < a.c.n_pages) return;
                page_next = -1;
                note_error(LC_ERR_CACHE_INDEX, kClassTree);
            };
            auto turn_page = [&](int j) {  // step j's page and scales, and the next one's page asked for
                page = page_next;
                row = row_next;
                if constexpr (Q8) {
                    ks = vs = 0.f;
                    if (page >= 0) {
                        ks = a.c.ks[row_offset(a.c.kss, page, head, row)];
                        vs = a.c.vs[row_offset(a.c.vss, page, head, row)];
                    }
                }
                page_id(j + 1);
            };
            // one thing after another -- a piece taken, its q, a tile started -- and then the tiles that have landed are
            // given on, all but the newest LAG, or all where the next thing is not to be had yet
#pragma unroll 1
            while (ok && !end) {
                uint32_t keep = S::LAG;
                bool q_here = false;
                if (q_due) {
                    if (n_q && issued != given && !done_warp(sh.q_empty, n_q - 1)) {
                        keep = 0;  // its last keys among them
                    } else {
                        if (n_q && !wait_warp(sh.q_empty, n_q - 1)) break;
                        constexpr int RQ = kTrRows / kTrLoaders;
                        tree_query<KV, NC, RQ>(a, *it, lw * RQ, q_s, sh.q_scale[(i - 1) & 1]);
                        ++n_q;
                        keep = 0;  // and the keys that were started before them
                        q_due = false;
                        q_here = true;
                    }
                } else if (p == 2 * steps) {
                    if (issued != given && !done_warp(sh.item_full[i % kTrItems], i / kTrItems)) {
                        keep = 0;
                    } else {
                        if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
                        it = &sh.item[i % kTrItems];
                        ++i;
                        if (it->end) {
                            end = true;
                            keep = 0;
                        } else {
                            b = it->b;
                            head = it->head;
                            n = it->n;
                            slot_first = it->begin + it->first * KEYS;
                            steps = it->steps;
                            p = entry = 0;
                            page_id(0);
                            turn_page(0);
                        }
                    }
                } else {
                    const bool is_k = p == 0 || (p & 1 && p < 2 * steps - 1);
                    const int j = is_k ? (p + 1) / 2 : p == 2 * steps - 1 ? steps - 1 : p / 2 - 1;
                    int64_t from;
                    int32_t where = -1;
                    if (is_k) {
                        from = page >= 0 ? row_offset(a.c.kst, page, head, row) : -1;
                        v_off = v_next;
                        v_next = page >= 0 ? row_offset(a.c.vst, page, head, row) : -1;
                        const int x = step_no % kTrAux;
                        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                        if (lane == 0) {
                            if constexpr (RW == 32) sh.there[x][lw] = there;
                            else reinterpret_cast<uint16_t *>(sh.there[x])[lw] = static_cast<uint16_t>(there);
                        }
                        if constexpr (Q8) {
                            float lv;
                            asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(fabsf(vs)));
                            if (lane < RW) {
                                aux[(x * 3) * KEYS + lw * RW + lane] = ks;
                                aux[(x * 3 + 1) * KEYS + lw * RW + lane] = vs;
                                aux[(x * 3 + 2) * KEYS + lw * RW + lane] = lv;
                            }
                            // a step's largest logarithm, where they are all near one another (else NaN)
                            const bool counts = page >= 0 && vs != 0.f;
                            float most = counts ? lv : -INFINITY, least = counts ? lv : INFINITY;
#pragma unroll
                            for (int d = 16; d; d >>= 1) {
                                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                                least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
                            }
                            const bool odd = __any_sync(0xffffffffu, counts && !(fabsf(lv) <= kFar));
                            if (lane == 0) sh.range[x][lw] = odd ? make_float2(NAN, NAN) : make_float2(most, least);
                        }
                        turn_page(j + 1);
                        ++step_no;
                    } else {
                        const bool last = j + 1 == steps;
                        from = last ? v_next : v_off;
                        const int slot0 = slot_first + j * KEYS;
                        if (masked(*it, slot0) && entry < kTrMasked) {
                            where = static_cast<int>((i - 1) % kTrItems) * kTrMasked + entry;
                            ++entry;
                        }
                        if (last) {  // before it is started: that may give the item back
                            if (lane == 0) it->last_tile = issued + 1;  // (every warp the same)
                            __syncwarp();
                            ++done;
                        }
                    }
                    start(is_k ? 0 : 1, from, where);
                    if (!ok) break;
                    q_due = p == 0;
                    ++p;
                }
                if (issued - given > keep || q_here) {
                    if (keep) ptx::cp_async_wait<S::LAG>();
                    else ptx::cp_async_wait<0>();
#pragma unroll 1
                    while (issued - given > keep && ok) give();
                }
                if (q_here && ok) {
                    tc::fence_async_smem();
                    arrive_warp(sh.q_full);
                }
            }
            ptx::cp_async_wait<0>();
        }
    } else if (warp == kTrSoft + kTrLoaders) {
        few_registers();
        // products, by the whole warp
        const uint32_t tm = (tmem);
        const uint32_t q_desc = tc::smem_desc(q_s, 16), k_desc = tc::smem_desc(ring_s, 16), v_desc = tc::smem_desc(ring_s, S::CHUNK);
        const uint32_t qk = tc::instr_desc(M16, KEYS, false, a.negative);
        const uint32_t pv = tc::instr_desc(M16, (a.c.dim + 15) / 16 * 16, true, false);
        const int k_steps = (a.c.dim + 15) / 16;
        auto wait_all = [&](const uint64_t &b, uint32_t n) {
            wait_warp(b, n);
            tc::fence_after();
            return ok;
        };
        // tiles come in the order in which they are used, K0 K1 V0 K2 V1 ...
        uint32_t slot = 0, phase = 0, n_q = 0, n_p = 0;
        auto take = [&]() {  // the next tile's slot, when it is there
            const uint32_t s = slot;
            wait_all(sh.ring_full[slot], phase);
            if (++slot == S::SLOTS) {
                slot = 0;
                phase ^= 1;
            }
            return s;
        };
        for (uint32_t i = 0;; ++i) {
            if (!wait_all(sh.item_full[i % kTrItems], i / kTrItems)) break;
            const uint32_t steps = (sh.item[i % kTrItems].steps), end = (sh.item[i % kTrItems].end);
            arrive_warp(sh.item_empty[i % kTrItems]);
            if (end) break;
            const uint32_t t0 = n_p;  // steps before this piece: the S buffers go on in turn
            if (!wait_all(sh.q_full, n_q++)) break;
#pragma unroll 1
            for (uint32_t j = 0; j < steps + 2 && ok; ++j) {
                // what a step needs is there before its weights are waited for, and what it has used is given back when its
                // products are on their way
                const bool more = j < steps;
                uint32_t sv = 0, sk = 0;
                if (j >= 2) sv = take();
                if (more) sk = take();
                if (!ok) break;
                if (j >= 2) {
                    const uint32_t buf = n_p & 1, values = v_desc + sv * (S::TILE / 16);
                    if (!wait_all(sh.p_full[buf], n_p++ >> 1)) break;
#pragma unroll 1
                    for (int rest = 0; rest < (Q8 ? 1 : 2); ++rest)
#pragma unroll
                        for (int k = 0; k < KEYS / 16; ++k)  // 16 slots, 2048 bytes, on
                            tc::mma_ts(tm + S::O, tm + buf * 128 + rest * 16 + k / 2 * 32 + (k & 1) * 8, values + 128 * k, pv,
                                       j > 2 || rest > 0 || k > 0);
                    tc::commit(bar(sh.o_full[0]) + buf * 8);
                }
                if (more) {
                    const uint32_t to = (t0 + j) & 1, keys = k_desc + sk * (S::TILE / 16);
#pragma unroll
                    for (int k = 0; k < NC * 4; ++k)  // 16 columns, 32 bytes, on
                        if (k < k_steps)
                            tc::mma_ss(tm + to * 128, q_desc + k / 4 * (S::QCHUNK / 16) + (k & 3) * 2,
                                       keys + k / 4 * (S::CHUNK / 16) + (k & 3) * 2, qk, k > 0);
                    tc::commit(bar(sh.s_full[0]) + to * 8);
                    tc::commit(bar(sh.ring_empty[0]) + sk * 8);
                    if (j + 1 == steps) tc::commit(bar(sh.q_empty));
                }
                if (j >= 2) tc::commit(bar(sh.ring_empty[0]) + sv * 8);
            }
            if (!ok) break;
        }
        // products in flight end before the tensor memory is given back
        tc::commit(bar(sh.drain));
        drained(sh.drain, 0);
        tc::fence_after();
    } else if (warp < kTrSoft) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        // softmax and outputs: a thread a row and half of a step's slots
        constexpr int HALF = KEYS / 64;  // 32-slot pieces of a half
        const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);
        uint32_t n_s = 0, n_pair = 0, ring = 0;
        // the two warps of 32 rows have both written what the other reads
        auto meet = [&] {
            arrive_warp(sh.pair[quarter]);
            return wait_warp(sh.pair[quarter], n_pair++);
        };
        for (uint32_t i = 0; ok; ++i) {
            if (!wait_warp(sh.item_full[i % kTrItems], i / kTrItems)) break;
            TreeItem &it = sh.item[i % kTrItems];
            if (it.end) break;
            if (!wait_warp(sh.kin_full[i % kTrItems], i / kTrItems)) break;
            const int steps = it.steps, slot_first = it.begin + it.first * KEYS, before = it.n - it.count;
            const uint32_t ring0 = ring;
            ring += 2 * steps;
            int n_bad = 0;
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
#pragma unroll 1
            for (int j = 0; j < steps; ++j) {
                const int buf = n_s & 1, slot0 = slot_first + j * KEYS;
                const uint32_t s_at = lanes + buf * 128;
                if (!wait_warp(sh.s_full[buf], n_s >> 1)) break;
                const int x_at = n_s % kTrAux;
                ++n_s;
                if (Q8 && j == 0) scale2 = a.scale2 * sh.q_scale[i & 1][row];
                if (masked(it, slot0) && n_bad < kTrMasked) {
                    if constexpr (TMA && !Q8) {
                        // values that some row does not see are multiplied by weights of 0 there: what is not finite becomes 0,
                        // and is added at the end where it is seen.  (What their place in the ring held before has been used.)
                        // A warp every other 64 columns, by the largest exponents.
                        if (row < KEYS) {
                            const uint32_t place = ring0 + (j + 1 < steps ? 2 * j + 2 : 2 * j + 1), v_at = ring_s + place % S::SLOTS * S::TILE;
                            if (!wait_warp(sh.ring_full[place % S::SLOTS], place / S::SLOTS)) break;
                            constexpr uint32_t kExp = M16 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
                            for (int c = half; c < NC; c += 2) {
                                const uint32_t piece = v_at + c * S::CHUNK + row * 128;
                                uint4 v[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) v[k] = ld_shared16(piece + (k ^ (row & 7)) * 16);
                                uint32_t most = 0;
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                                                   __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
                                const bool found = (most & 0xffffu) >= kExp || most >> 16 >= kExp;
                                if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
                                    for (int k = 0; k < 8; ++k) {
                                        uint4 x = ld_shared16(piece + k * 16);
                                        tree_clean<KV>(x);
                                        st_shared16(piece + k * 16, x);
                                    }
                                    // (not of slots behind the sequence, which nobody sees)
                                    atomicOr(&it.bad[n_bad][quarter], __ballot_sync(0xffffffffu, found && slot0 + row < it.n));
                                    tc::fence_async_smem();
                                }
                            }
                        }
                    }
                    if (lane == 0 && warp == 0) it.bad_step[n_bad] = slot0;
                    ++n_bad;
                }
                if (some) {
                    tc::fence_after();
                    const bool cut = masked(it, slot0);
                    bool part = cut;
#pragma unroll
                    for (int c = 0; c < KEYS / 32; ++c) part |= sh.there[x_at][c] != 0xffffffffu;
                    const float *const ks = aux + x_at * 3 * KEYS, *const vs = ks + KEYS, *const lv = vs + KEYS;
                    (void)vs;
                    const float2 scale = make_float2(scale2, scale2);
                    // the logits, not scaled by scale2 yet, and the largest (a maximum passes NaN by: the weights will show it)
                    uint32_t x[HALF][32], bits[HALF];
                    float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < HALF; ++c) tc::ld32(x[c], s_at + (half * HALF + c) * 32);
#pragma unroll
                    for (int c = 0; c < HALF; ++c) {
                        const int c32 = half * HALF + c;
                        bits[c] = sh.there[x_at][c32] & (cut ? seen(slot0 + 32 * c32) : 0xffffffffu);
                    }
#pragma unroll
                    for (int c = 0; c < HALF; ++c) tc::wait_ld(x[c]);
#pragma unroll
                    for (int c = 0; c < HALF; ++c) {
                        const int s32 = (half * HALF + c) * 32;
                        if constexpr (Q8) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 s = *reinterpret_cast<const float4 *>(ks + s32 + e);
                                const float2 u = tc::mul2(make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), make_float2(s.x, s.y));
                                const float2 v = tc::mul2(make_float2(__uint_as_float(x[c][e + 2]), __uint_as_float(x[c][e + 3])), make_float2(s.z, s.w));
                                x[c][e] = __float_as_uint(u.x);
                                x[c][e + 1] = __float_as_uint(u.y);
                                x[c][e + 2] = __float_as_uint(v.x);
                                x[c][e + 3] = __float_as_uint(v.y);
                            }
                        }
                        if (part) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(bits[c] & 1u << e)) x[c][e] = 0xff800000u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            tops[0] = tr_max3(tops[0], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                            tops[1] = tr_max3(tops[1], __uint_as_float(x[c][e + 2]), __uint_as_float(x[c][e + 3]));
                        }
                    }
                    float top = fmaxf(tops[0], tops[1]), top_v = 0.f;
                    // E4M3: the largest logarithm of the step's scales; `wide` where they do not lie near one another
                    float most = -INFINITY;
                    bool wide = false;
                    if constexpr (Q8) {
                        float least = INFINITY;
#pragma unroll
                        for (int k = 0; k < kTrLoaders; ++k) {
                            const float2 r = sh.range[x_at][k];
                            wide |= !(r.x == r.x);
                            most = fmaxf(most, r.x);
                            least = fminf(least, r.y);
                        }
                        // (a maximum far from the logits' is one that such scales have left)
                        wide |= most == -INFINITY || most - least > kNear ||
                                __any_sync(0xffffffffu, real && mv != -INFINITY && !(fabsf(mv - m) <= kFar + 2 * kNear));
                        if (wide) {
                            top_v = -INFINITY;
#pragma unroll
                            for (int c = 0; c < HALF; ++c)
#pragma unroll
                                for (int e = 0; e < 32; ++e)  // (-infinity where not seen, and no sum with infinity counts)
                                    top_v = fmaxf(top_v, fmaf(__uint_as_float(x[c][e]), scale2, lv[(half * HALF + c) * 32 + e]));
                        }
                    }
                    const int turn = n_pair & 1;
                    sh.top[turn][half][row] = top;
                    if (Q8 && wide) sh.top_v[turn][half][row] = top_v;
                    if (!meet()) break;
                    top = fmaxf(top, sh.top[turn][1 - half][row]) * scale2;
                    top_v = !Q8 ? top : wide ? fmaxf(top_v, sh.top_v[turn][1 - half][row]) : top + most;
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
                            for (int c = half; c < (a.c.dim + 31) / 32; c += 2) {
                                uint32_t o[32];
                                tc::ld32(o, lanes + S::O + c * 32);
                                tc::wait_ld(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st32(lanes + S::O + c * 32, o);
                            }
                        }
                    }
                    // the weights of 32 slots take the columns of their logits: 16 of leading numbers, 16 of the rests
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 off = make_float2(-less, -less);
                    // E4M3: weights relative to mv, for the sum too (its factor follows), but where scales are not near one
                    // another: there each exponential of its own
                    const float2 off_v = make_float2(-less_v, -less_v);
                    (void)off_v;
#pragma unroll
                    for (int c = 0; c < HALF; ++c) {
                        const int s32 = (half * HALF + c) * 32;
                        uint32_t p[16], rest[16];
                        if (Q8 && wide) {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float2 z = make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                                float2 y = tc::fma2(z, scale, off), v = tc::add2(tc::fma2(z, scale, off_v), *reinterpret_cast<const float2 *>(lv + s32 + e));
                                y.x = tr_exp2(y.x);
                                y.y = tr_exp2(y.y);
                                sum[e >> 1 & 1] = tc::add2(sum[e >> 1 & 1], y);
                                const float2 sv = *reinterpret_cast<const float2 *>(vs + s32 + e);
                                p[e / 2] = tr_pack<true>(copysignf(tr_exp2(v.x), sv.x), copysignf(tr_exp2(v.y), sv.y));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                                if constexpr (Q8) s = *reinterpret_cast<const float4 *>(vs + s32 + e);
#pragma unroll
                                for (int k = 0; k < 4; k += 2) {
                                    float2 y = tc::fma2(make_float2(__uint_as_float(x[c][e + k]), __uint_as_float(x[c][e + k + 1])), scale,
                                                        Q8 ? off_v : off);
                                    y.x = tr_exp2(y.x);
                                    y.y = tr_exp2(y.y);
                                    sum[k / 2] = tc::add2(sum[k / 2], y);
                                    if constexpr (Q8) {
                                        const float2 v = tc::mul2(y, k ? make_float2(s.z, s.w) : make_float2(s.x, s.y));
                                        p[(e + k) / 2] = tr_pack<true>(v.x, v.y);
                                    } else {
                                        tr_split<M16>(y.x, y.y, &p[(e + k) / 2], &rest[(e + k) / 2]);
                                    }
                                }
                            }
                        }
                        if constexpr (Q8) {
                            if (part) {  // a slot that is not seen may have any scale
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    p[e] &= (bits[c] & 1u << 2 * e ? 0xffffu : 0u) | (bits[c] & 2u << 2 * e ? 0xffff0000u : 0u);
                            }
                        }
                        tc::st16(s_at + s32, p);
                        if constexpr (!Q8) tc::st16(s_at + s32 + 16, rest);
                    }
                    const float2 both = tc::add2(sum[0], sum[1]);
                    l += (both.x + both.y) * (Q8 && !wide ? tr_exp2(less_v - less) : 1.f);
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
                sh.sum[half][row] = l;
                if (!meet()) break;
                l = sh.sum[0][row] + sh.sum[1][row];
                const int hq = it.head * a.group + g;
                const bool none = l == 0.f;
                float f = none ? 0.f : 1.f / l;
                if (it.part >= 0) f = 1.f;
                if (Q8) f *= mv == -INFINITY ? 0.f : exp2f(less_v - less);  // the output was relative to mv
                uint16_t *out = a.out + it.b * a.ost[0] + t * a.ost[1] + hq * a.ost[2];
                uint32_t any_bad = 0;
                for (int n = 0; n < n_bad; ++n) any_bad |= it.bad[n][0] | it.bad[n][1] | it.bad[n][2] | it.bad[n][3];
                // 16 columns at a time, a warp every other 32 of them: short code, since the roles' code does not fit the
                // instruction cache together
#pragma unroll 1
                for (int c = 2 * half; c < (a.c.dim + 15) / 16; c += c & 1 ? 3 : 1) {
                    uint32_t o[16];
                    __syncwarp();
                    tc::ld16(o, lanes + S::O + c * 16);
                    tc::wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
                    for (int n = 0; any_bad && n < n_bad; ++n)
#pragma unroll 1
                        for (int w = 0; w < 4; ++w)
#pragma unroll 1
                            for (uint32_t left = it.bad[n][w]; left; left &= left - 1) {
                                const int slot = it.bad_step[n] + w * 32 + __ffs(left) - 1;
                                if (!real || !(seen(slot) & 1)) continue;
                                const uint8_t *v = tree_value<EB>(a, it.b, it.head, slot);
                                if (!v) continue;
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (c * 16 + e < a.c.dim)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) + tree_unusual<KV>(v, c * 16 + e));
                            }
                    if (it.part >= 0) {
                        float4 *to = reinterpret_cast<float4 *>(a.part) + (int64_t(it.part) * NC * 16 + c * 4) * kTrRows + row;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            st_global16(to + e * kTrRows, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]), real);
                    } else {
                        const bool whole = a.out_vec && c * 16 + 16 <= a.c.dim;
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[k] = tr_pack<KV == LC_CACHE_F16>(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
                            uint16_t *to = out + c * 16 + e;
                            if (whole) {
                                st_global16(to, make_uint4(y[0], y[1], y[2], y[3]), real);
                            } else if (real) {
#pragma unroll 1
                                for (int k = 0; k < 8; ++k)
                                    if (c * 16 + e + k < a.c.dim)
                                        to[k] = static_cast<uint16_t>((k < 4 ? k < 2 ? y[0] : y[1] : k < 6 ? y[2] : y[3]) >> (k & 1) * 16);
                            }
                        }
                    }
                }
                if (half == 0 && real && it.part >= 0) {
                    a.part_ml[int64_t(it.part) * kTrRows + row] = make_float2(m == -INFINITY ? -INFINITY : less, l);
                } else if (half == 0 && real && a.lse) {
                    a.lse[it.b * a.lst[0] + t * a.lst[1] + hq] =
                        none ? -INFINITY : (less + kSumLift + log2f(l * exp2f(-kSumLift))) * 0.6931471805599453f;
                }
            }
            arrive_warp(sh.item_empty[i % kTrItems]);
        }
    } else {
        few_registers();
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kTrSoft + kTrLoaders) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// Joins the parts of the units that were cut, in their order: a block a cut (the end of a run), 32
// rows and 32 columns, a warp four columns, a lane a row.
template <int KV, int NC>
__global__ void __launch_bounds__(256) k_tree_join(const __grid_constant__ TreeArgs a) {
    constexpr int KEYS = TreeShape<NC, KV == LC_CACHE_E4M3>::KEYS;
    constexpr float kSumLift = KV == LC_CACHE_E4M3 ? 0.f : kTrLift<KV>;
    __shared__ float2 ml[8][32];
    __shared__ uint32_t cuts_of[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    start_after_prior();
    const int columns = blockIdx.x % (2 * NC), group = blockIdx.x / (2 * NC) % 4;
    // the block's cut, in the runs' order
    const uint32_t cuts = __ballot_sync(0xffffffffu, static_cast<int>(threadIdx.x) < a.runs && a.split[threadIdx.x].x >= 0);
    if (lane == 0) cuts_of[warp] = cuts;
    __syncthreads();
    int left = blockIdx.x / (8 * NC), run = 0;
    uint32_t bits = 0;
#pragma unroll
    for (int w = 7; w >= 0; --w) {  // (the words before w have `before` of them)
        int before = 0;
#pragma unroll
        for (int v = 0; v < w; ++v) before += __popc(cuts_of[v]);
        if (bits == 0 && left >= before) {
            left -= before;
            bits = cuts_of[w];
            run = w * 32;
            if (left >= __popc(bits)) return;  // fewer cuts than blocks for them
        }
    }
    for (; left; --left) bits &= bits - 1;
    run += __ffs(bits) - 1;
    const int4 cut = a.split[run];
    const int b = cut.x, head = cut.y, row0 = cut.z * kTrRows + group * 32;
    const TreeSeq s = tree_seq<KEYS>(a, b);
    if (row0 >= s.count * a.group || columns * 32 >= a.c.dim) return;
    const int row = group * 32 + lane, n = cut.w - run + 1;
    // the unit's first part is its run's second, the others their runs' first
    auto slot = [&](int i) { return int64_t(2) * (run + i) + (i == 0); };
    float top = -INFINITY, l = 0.f;
    for (int i = warp; i < n; i += 8) {
        const float2 v = a.part_ml[slot(i) * kTrRows + row];
        const float t = fmaxf(top, v.x), safe = t == -INFINITY ? 0.f : t;
        l = l * tr_exp2(top - safe) + v.y * tr_exp2(v.x - safe);
        top = t;
    }
    ml[warp][lane] = make_float2(top, l);
    __syncthreads();
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, ml[w][lane].x);
    const float safe = top == -INFINITY ? 0.f : top;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += ml[w][lane].y * tr_exp2(ml[w][lane].x - safe);
    const int c = columns * 8 + warp;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 *part = reinterpret_cast<const float4 *>(a.part) + int64_t(c) * kTrRows + row;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float w = tr_exp2(a.part_ml[slot(i) * kTrRows + row].x - safe);
        const float4 z = part[slot(i) * NC * 16 * kTrRows];
        y.x += z.x * w;
        y.y += z.y * w;
        y.z += z.z * w;
        y.w += z.w * w;
    }
    const int at = row0 + lane, t = static_cast<int>(fast_div(at, a.group_div)), g = at - t * a.group;
    if (t >= s.count) return;
    const float f = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = a.out + b * a.ost[0] + t * a.ost[1] + (int64_t(head) * a.group + g) * a.ost[2] + c * 4;
    const uint32_t lo = tr_pack<KV == LC_CACHE_F16>(y.x * f, y.y * f), hi = tr_pack<KV == LC_CACHE_F16>(y.z * f, y.w * f);
    if (a.out_vec && c * 4 + 4 <= a.c.dim) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
    } else {
        for (int e = 0; e < 4; ++e)
            if (c * 4 + e < a.c.dim) out[e] = static_cast<uint16_t>((e < 2 ? lo : hi) >> (e & 1) * 16);
    }
    if (c == 0 && a.lse)
        a.lse[b * a.lst[0] + t * a.lst[1] + head * a.group + g] =
            l == 0.f ? -INFINITY : (top + kSumLift + log2f(l * exp2f(-kSumLift))) * 0.6931471805599453f;
}

// What a call needs of the workspace, and its launch.
template <int KV, int NC>
int launch_tree_shape(const TreeArgs &a, cudaStream_t cs) {
    using S = TreeShape<NC, KV == LC_CACHE_E4M3>;
    const void *fn = a.box > 1 ? reinterpret_cast<const void *>(&k_tree_attend<KV, NC, true>)
                               : reinterpret_cast<const void *>(&k_tree_attend<KV, NC, false>);
    int sms = 0, per_sm = 0;
    if (prepare(fn, S::THREADS, S::SMEM, S::SMEM, &sms, &per_sm) != cudaSuccess) return LC_ERR_CUDA;
    TreeArgs b = a;
    const int64_t units = int64_t(a.c.n_seqs) * a.c.heads * a.most_blocks;
    const int64_t steps = units * ((int64_t(a.c.cap) + S::KEYS - 1) / S::KEYS);
    // Steps of a run: one, so that a few short sequences take as many blocks as there are steps (a sequence of 300 slots, 2
    // key heads of 64: 10.3 us, 12.8 with two); two past 128 elements a head, whose parts are twice as large and whose joining
    // is as long as a step (8 windows of 1024, 192 rows of 256: 23 us, 2 more with one).
    // Units stay whole, and nothing is joined by a second launch, where the table's columns are few steps: up to four
    // (2 units of 3 steps of 64 elements a head: 9.3 us, cut 9.8, and 3 us less on the host; 128 of 3 steps of 128: 12.0 and 17.7;
    // of 4 in E4M3 2 units take 17.5 cut 15.3, which few units lose by this rule, 128 units 19.2 and 29.1), and up to eight where units take more than half of the
    // blocks (128 units: 17.7 and 24.9; 2 units of 8 steps 16.6 and 12.5).
    const int64_t most = (int64_t(a.c.cap) + S::KEYS - 1) / S::KEYS;
    b.whole = most <= (units <= sms && 2 * units > sms ? 8 : 4);
    b.least = NC <= 2 || b.whole ? 1 : 2;
    b.runs = static_cast<int32_t>(std::min<int64_t>(std::min(sms, kTrMostRuns), b.whole ? units : (steps + b.least - 1) / b.least));
    const int st = launch_after(fn, b.runs, S::THREADS, S::SMEM, cs, &b);
    if (st || b.whole) return st;
    return launch_after(reinterpret_cast<const void *>(&k_tree_join<KV, NC>), static_cast<unsigned>(std::min<int64_t>(b.runs, units) * 8 * NC), 256,
                        0, cs, &b);
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
