// Attention over whole prompts (lc_prompt_attend):
//     x_ij = scale * q_i . k_j,  w = softmax_j(x),  out_i = sum_j w_ij v_j
// over the keys j of the query's own sequence that are seen.
//
// Mathematics.  A tile of 128 rows (query tokens x the query heads of one key
// head) goes through its keys 128 at a time: S = Q K^T into tensor memory, one
// thread a row turns S into weights 2^(x - m) relative to a running maximum m
// and adds them up, P V is added to the output in tensor memory.  m follows the
// maximum only when that has grown by 2^kRise (the output is then rescaled);
// until then weights up to 2^kRise are as good as weights up to 1.
//
// Both products are fifth-generation tensor-core instructions: Q and K come
// from shared memory, P from the tensor memory that held S, V from shared
// memory in its own [key, dim] order.  Two row tiles take turns on the tensor
// cores: while one tile's products run, the other's softmax does.  Past 128
// elements a head the outputs of two tiles do not fit; one tile then has two S
// and runs the next tile's first product during the softmax.
//
// What bounds it, by GB300 figures of the kernel alone: a long causal prompt (11585
// tokens, 32 heads of 128, float16) runs at 1690 TFLOP/s (652 us), 87 % of the rate of a large library
// product: tensor cores and exponentials (16 a cycle and SM) both take a step's 2048 cycles; call after call the
// power limit leaves 1550.  24
// prompts of up to 2048, 32 on 8 heads: 1213 TFLOP/s; of an item's 24 thousand cycles 5 to 8 thousand are
// its first weights, its masked steps and its output.  Windows at 80 elements a head (6 prompts behind 3001
// keys, 1024 seen: 48 to 55 us) no one unit bounds: the exponentials would take 23, the rest is items' starts and
// outputs, three rounds of items where 2.2 would do, and steps in which one of two tiles sees nothing.  Past
// 128 elements a head: 8192 tokens, 16 heads of 256, 549 us (1000 TFLOP/s).  A short prompt: 6.5 us,
// the chain of launch, starts, copies, one step and output.
// Waits are by votes and arrivals by predicates, so that warps stay together: a lane that
// polls alone parts its warp, and every exchange after it cost 250 cycles (the long prompt took 896
// us, and 665 without).
//
// A weight is rounded to the values' 16-bit type for the second product: with
// independent roundings that adds as much as the output's own rounding does
// (errors against 64 bits 1.4 times a 32-bit softmax's rounded once); a second
// number a weight would make the tensor cores' work half as much again.
#pragma once

#include <cuda.h>

#include "cache_common.cuh"
#include "layout_copy_prompt.h"
#include "tensor_core.cuh"

namespace lc {

constexpr uint32_t kClassPrompt = 0xf3;
constexpr int kPrRows = 128;   // rows of a tile
constexpr int kPrKeys = 128;   // keys of a step
constexpr int kPrChunk = kPrKeys * 128;  // bytes of 64 columns of a tile
constexpr int kPrItems = 3;    // items that the scheduling warp may be ahead
constexpr int kPrMasked = 6;   // steps of an item whose values are looked through: three at either end of its keys at most
constexpr int kPrTurns = kPrItems + 1;  // items whose unusual values are held: one tile may be as many ahead of the other

struct PromptArgs {
    const int32_t *starts, *k_starts;
    uint16_t *out;
    float *lse;
    const uint16_t *v;
    int64_t ost[2], vst[2];
    int64_t lse_stride;
    int32_t n_seqs, n_tokens, n_keys;
    int32_t group, heads_tile, head_blocks, key_heads;  // query heads: a key head's, a tile's; tiles a key head's need
    int32_t tokens_tile;                                // query tokens of a tile
    int32_t dim, causal, window;
    FastDiv heads_div;                                  // by heads_tile
    FastDiv pair_div;                                   // by key_heads * head_blocks
    float scale2;                                       // |scale| log2 e
    int32_t negative;                                   // scale < 0
    int32_t store;                                      // bytes of a store to out: 32, 16
    uint64_t limit_ns;
    CUtensorMap qm, km, vm;
};

// What one item is: up to two row tiles, the steps of keys that they see.
struct PromptItem {
    int32_t q0, nq;     // the sequence's first query row and its queries
    int32_t k0, nk;
    int32_t t0;         // first query token of the item
    int32_t key_head, head0;  // first query head of the tile within its group
    int32_t first, steps;     // steps of 128 keys, from the sequence's first key
    int32_t end;        // not 0: there is no further item
};

template <int NC>
struct PromptShape {
    static constexpr int TILES = NC <= 2 ? 2 : 1;          // row tiles of an item
    static constexpr int CPS = NC <= 2 ? NC : 1;           // 64-column chunks of a ring slot
    static constexpr int SPT = NC / CPS;                   // slots of a tile of keys or values
    static constexpr int SLOT = CPS * kPrChunk;
    static constexpr int Q = TILES * NC * kPrChunk;
    static constexpr int SLOTS = (232448 - 2048 - Q) / SLOT < 10 ? (232448 - 2048 - Q) / SLOT : 10;
    static constexpr int SMEM = Q + SLOTS * SLOT + 2048;   // 1024 of them for alignment
    static constexpr int SOFT = 4 * TILES;                 // softmax warps
    static constexpr int THREADS = 32 * (SOFT + 4);        // products, loads, scheduling, a second tile's products
    static constexpr int O = 256;                          // first output column of tensor memory
    // The softmax waits for a step's values by their phase's parity, so the phase before, of the tile that came SLOTS
    // places earlier, has to be known to be over.  Logits seen mean that the tiles up to their keys have come, since
    // the products take tiles in the ring's order.  LATE: how many tiles before the values lies the newest one that
    // is not known to have come.  With two row tiles that is this step's keys (K V K V: two before).  With one
    // (K K V K V) the values of the step before were waited for, and it is this step's keys, three before, or where
    // this step's logits are waited for first the next step's, one before.
    static constexpr bool LOGITS_FIRST = TILES == 1;
    static constexpr int LATE = TILES == 2 ? 2 : LOGITS_FIRST ? 1 : 3;
    static_assert(SLOTS >= (LATE + 1) * SPT, "a values' wait may pass by the phase before");
};

struct PromptShared {
    uint64_t ring_full[10], ring_empty[10];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_half[2], p_full[2];  // weights of the first 64 keys, of all
    uint64_t o_full[2];              // of a tile's item; with one tile of every other step
    uint64_t item_full[kPrItems], item_empty[kPrItems];
    uint64_t turn[2];                // of a tile's products, when the other's are on their way
    uint64_t drain[2];
    PromptItem item[kPrItems];
    uint32_t bad[kPrTurns][kPrMasked][4];   // [item's turn][masked step][rows of 32]: values that are not finite
    int32_t bad_step[kPrTurns][kPrMasked];
    uint32_t bad_any[kPrTurns][4];
    uint32_t tmem;
};
static_assert(sizeof(PromptShared) <= 1024, "the shared block has 1024 bytes");

__device__ __forceinline__ float pr_exp2(float x) {  // 2 ulp, 0 for -infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pr_pack(float lo, float hi) {
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
__device__ __forceinline__ float pr_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// ---- scheduling ------------------------------------------------------------

// Up to 32 sequences' items are taken from the longest to the shortest: a sequence's tiles are
// counted from its last one down: the last one's level is the tiles of keys
// that come before the sequence's end, the one before it has a level less.  With more of them
// a block has many items, and they are taken in the sequences' order, the last tile of each first: to look
// for the longest of 2000 sequences of 20 tokens took 16 ms, in order the call takes 0.36 ms.  (33 of 1000 tokens each, where
// the order does not matter: 258 and 252 us.  Ragged ones pay for it where the longest come last: 64 of up to 2048, 32 heads
// of 128, take 440 us so, 404 to 411 in rising, falling or mixed order.)
struct PromptSeq {
    int level, tiles;
    bool fell;  // it ends before it begins
};

template <int TILES>
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs &a, int b, PromptItem *it) {
    const int32_t *ks = a.k_starts ? a.k_starts : a.starts;
    const int k_most = a.n_keys;
    const int r0 = a.starts[b], r1 = a.starts[b + 1], s0 = ks[b], s1 = ks[b + 1];
    const int q0 = min(max(r0, 0), a.n_tokens), q1 = min(max(r1, q0), a.n_tokens);
    const int k0 = min(max(s0, 0), k_most), k1 = min(max(s1, k0), k_most);
    const bool fell = min(max(r1, 0), a.n_tokens) < q0 || min(max(s1, 0), k_most) < k0;
    if (q0 != r0 || q1 != r1 || k0 != s0 || k1 != s1) note_error(LC_ERR_CACHE_INDEX, kClassPrompt);
    if (it) {
        it->q0 = q0;
        it->nq = q1 - q0;
        it->k0 = k0;
        it->nk = k1 - k0;
    }
    const int per = TILES * a.tokens_tile;
    return PromptSeq{(max(k1 - k0, 1) - 1) / per, (q1 - q0 + per - 1) / per, fell};
}

// Tiles of a sequence at level x or above.
__device__ __forceinline__ int prompt_above(const PromptArgs &a, const PromptSeq &s, int x) {
    if (x <= 0) return s.tiles;
    if (!a.causal) return s.level >= x ? s.tiles : 0;
    return min(max(s.level - x + 1, 0), s.tiles);
}

// Where a block has come to among the sequences: 32 of them, a lane each.
struct PromptCursor {
    PromptSeq mine;
    int b0;
    uint32_t before;  // tiles of the sequences before them
    bool fell;        // starts fall somewhere: sequences share rows, so there is no answer, and no bound on the tiles
};

template <int TILES>
__device__ __forceinline__ PromptCursor prompt_begin(const PromptArgs &a) {
    const int lane = threadIdx.x & 31;
    PromptCursor c{{0, 0, false}, 0, 0, false};
    if (lane < a.n_seqs) c.mine = prompt_seq<TILES>(a, lane, nullptr);
    bool fell = c.mine.fell;
#pragma unroll 4
    for (int b = 32 + lane; b < a.n_seqs; b += 32) fell |= prompt_seq<TILES>(a, b, nullptr).fell;
    c.fell = __any_sync(0xffffffffu, fell);
    return c;
}

// Item `at` of all, by one warp; `at` only rises.
template <int TILES>
__device__ __forceinline__ void prompt_item(const PromptArgs &a, uint32_t at, PromptCursor &c, PromptItem *it) {
    const int lane = threadIdx.x & 31;
    uint32_t pair = fast_div(at, a.pair_div);
    const int which = static_cast<int>(at - pair * a.pair_div.d);
    auto scan = [&](uint32_t n) {  // over the lanes up to this one
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, n, d);
            if (lane >= d) n += o;
        }
        return n;
    };
    it->end = 1;
    if (c.fell) return;
    int tile = 0, seq = 0;
    if (a.n_seqs <= 32) {
        auto total = [&](int x) { return __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(prompt_above(a, c.mine, x))); };
        if (pair >= total(0)) return;
        // the highest level x with more than `pair` tiles at it or above
        int lo = 0, hi = a.n_keys / (TILES * a.tokens_tile) + 1;
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (total(mid) > pair) lo = mid;
            else hi = mid;
        }
        pair -= total(lo + 1);  // of the tiles at level `lo`, in the sequences' order
        const uint32_t n = prompt_above(a, c.mine, lo) - prompt_above(a, c.mine, lo + 1), upto = scan(n);
        seq = __ffs(__ballot_sync(0xffffffffu, upto > pair)) - 1;
        // tiles of the level begin where those above it, at the sequence's end, leave off
        const int from = a.causal ? c.mine.tiles - prompt_above(a, c.mine, lo) : 0;
        tile = __shfl_sync(0xffffffffu, from + static_cast<int>(pair - (upto - n)), seq);
    } else {
        uint32_t upto;
        for (;;) {
            upto = scan(c.mine.tiles);
            const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
            if (pair < c.before + all) break;
            c.before += all;
            c.b0 += 32;
            if (c.b0 >= a.n_seqs) return;
            c.mine = PromptSeq{0, 0, false};
            if (c.b0 + lane < a.n_seqs) c.mine = prompt_seq<TILES>(a, c.b0 + lane, nullptr);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, c.before + upto > pair)) - 1;
        tile = __shfl_sync(0xffffffffu, static_cast<int>(c.before + upto - pair) - 1, src);
        seq = c.b0 + src;
    }
    it->end = 0;
    prompt_seq<TILES>(a, seq, it);
    it->key_head = which / a.head_blocks;
    it->head0 = which % a.head_blocks * a.heads_tile;
    it->t0 = tile * TILES * a.tokens_tile;
    // the keys that any of its rows sees
    const int last = min(it->t0 + TILES * a.tokens_tile, it->nq) - 1, shift = it->nk - it->nq;
    const int end = a.causal ? min(max(last + shift + 1, 0), it->nk) : it->nk;
    const int begin = a.window ? max(it->t0 + shift - a.window + 1, 0) : 0;
    it->first = begin / kPrKeys;
    it->steps = max((end + kPrKeys - 1) / kPrKeys - it->first, 0);
}

// ---- the kernel ------------------------------------------------------------

// A value that is not finite, 0 for others.
template <bool F16>
__device__ __noinline__ float prompt_unusual(uint32_t bits) {
    constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
    if ((bits & kExp) != kExp) return 0.f;
    return F16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float(bits << 16);
}

// Place in the ring, of an item's first slot, of step j's keys or values (in
// slots of a tile): with two row tiles K0 V0 K1 V1 ..., with one K0 K1 V0 K2 V1 ...
template <int TILES>
__device__ __forceinline__ int key_place(int j) { return TILES == 2 ? 2 * j : j ? 2 * j - 1 : 0; }
template <int TILES>
__device__ __forceinline__ int value_place(int j, int steps) {
    return TILES == 2 ? 2 * j + 1 : j + 1 < steps ? 2 * j + 2 : 2 * j + 1;
}

template <bool F16, int NC>
__global__ void __launch_bounds__(PromptShape<NC>::THREADS, 1) k_prompt_attend(const __grid_constant__ PromptArgs a) {
    using S = PromptShape<NC>;
    constexpr int TILES = S::TILES;
    // weights are up to 2^(kLift + kRise): float16 has few exponents, so small ones are lifted into them; others are
    // lowered so that sums of the type's largest values stay in float32 (2^24 of them, 2^16 where the maximum is
    // 2^kRise behind).  By no more than that: exponents of all weights that count, down to 2^-8 of the largest, are below 32
    // and lose 2^-20; below 64 they would lose 2^-19, 1.3e-6 of the log sum of a single key.  (Lowering by a
    // multiplication loses nothing and took 3 to 7 % longer.)
    constexpr float kRise = F16 ? 4.f : 8.f, kLift = F16 ? 11.f : -24.f, kDrop = F16 ? 0x1p-11f : 0x1p24f;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (ptx::smem_addr(raw) + 1023) & ~1023u;
    const uint32_t q_s = base, ring_s = base + S::Q;
    PromptShared &sh = *reinterpret_cast<PromptShared *>(raw + (base - ptx::smem_addr(raw)) + S::Q + S::SLOTS * S::SLOT);
    // (shuffled, so that the compiler knows a warp's branches on it to be the whole warp's)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    auto bar = [&](const uint64_t &b) { return ptx::smem_addr(&b); };

    if (warp == S::SOFT) tc::alloc(ptx::smem_addr(&sh.tmem), 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::SLOTS; ++i) {
            ptx::mbar_init(bar(sh.ring_full[i]), 1);
            ptx::mbar_init(bar(sh.ring_empty[i]), TILES);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(sh.q_full[i]), 1);
            ptx::mbar_init(bar(sh.q_empty[i]), 1);
            ptx::mbar_init(bar(sh.s_full[i]), 1);
            ptx::mbar_init(bar(sh.p_half[i]), 4);
            ptx::mbar_init(bar(sh.p_full[i]), 4);
            ptx::mbar_init(bar(sh.o_full[i]), 1);
        }
        for (int i = 0; i < kPrItems; ++i) {
            ptx::mbar_init(bar(sh.item_full[i]), 1);
            ptx::mbar_init(bar(sh.item_empty[i]), S::SOFT + 1 + TILES);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(sh.turn[i]), 1);
            ptx::mbar_init(bar(sh.drain[i]), 1);
        }
        ptx::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    start_after_prior();

    bool ok = true;  // no wait of this warp has run out
    auto arrive_warp = [&](const uint64_t &b) { tc::arrive(bar(b)); };
    auto wait_warp = [&](const uint64_t &b, uint32_t n) {  // for phase n (counted from 0)
        if (ok && !tc::wait(bar(b), n, a.limit_ns)) {
            ok = false;
            note_error(LC_ERR_TIMEOUT, kClassPrompt);
        }
        return ok;
    };

    auto drained = [&](const uint64_t &b, uint32_t n) {  // what was started ends, however short the limit
        if (!tc::wait(bar(b), n, max(a.limit_ns, uint64_t(2000000000)))) note_error(LC_ERR_TIMEOUT, kClassPrompt);
    };

    // of a block's registers the softmax threads take the larger part (384 x 168 = 256 x 216 + 128 x 72)
    auto few_registers = [] {
        if constexpr (TILES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    };
    if (warp < S::SOFT) {
        if constexpr (TILES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // softmax and outputs: row tile t, a thread a row
        const int t = TILES == 2 ? warp >> 2 : 0, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const int token = static_cast<int>(fast_div(row, a.heads_div)), head = row - token * a.heads_tile;
        uint32_t n_s = 0, n_o = 0, pos = 0;
        for (uint32_t i = 0; ok; ++i) {
            if (!wait_warp(sh.item_full[i % kPrItems], i / kPrItems)) break;
            const PromptItem it = sh.item[i % kPrItems];
            arrive_warp(sh.item_empty[i % kPrItems]);
            if (it.end) break;
            const uint32_t p0 = pos;
            pos += 2 * it.steps;
            const int tile0 = it.t0 + t * a.tokens_tile;
            if (tile0 >= it.nq) continue;
            const int shift = it.nk - it.nq, mine = tile0 + token;
            const bool real = token < a.tokens_tile && mine < it.nq && it.head0 + head < a.group;
            auto keys_end = [&](int x) { return a.causal ? min(max(x + shift + 1, 0), it.nk) : it.nk; };
            auto keys_begin = [&](int x) { return a.window ? max(x + shift - a.window + 1, 0) : 0; };
            const int hi = keys_end(min(mine, it.nq - 1)), lo = keys_begin(min(mine, it.nq - 1));
            // keys in [all_lo, all_hi) are seen by every row of the tile, and of the item
            const int tile_last = min(tile0 + a.tokens_tile, it.nq) - 1;
            const int all_hi = keys_end(tile0), all_lo = keys_begin(tile_last);
            const int item_hi = keys_end(it.t0);
            const int item_lo = keys_begin(min(it.t0 + TILES * a.tokens_tile, it.nq) - 1);
            const int first_seen = keys_begin(it.t0), last_seen = keys_end(min(it.t0 + TILES * a.tokens_tile, it.nq) - 1);
            const int turn = i % kPrTurns;
            float m = -INFINITY, less = -kLift, l = 0.f;
            int n_bad = 0;
            if (t == 0) {
                if (lane == 0) sh.bad_any[turn][warp & 3] = 0;
                __syncwarp();
            }
            auto wait_values = [&](int j) {
                for (int c = 0; c < S::SPT; ++c) {
                    const uint32_t at = (p0 + value_place<TILES>(j, it.steps)) * S::SPT + c;
                    wait_warp(sh.ring_full[at % S::SLOTS], at / S::SLOTS);
                }
            };
            for (int j = 0; j < it.steps; ++j) {
                const int key0 = (it.first + j) * kPrKeys, buf = TILES == 2 ? t : n_s & 1;
                auto wait_logits = [&] {
                    if (!wait_warp(sh.s_full[buf], TILES == 2 ? n_s : n_s >> 1)) return false;
                    ++n_s;
                    tc::fence_after();
                    return true;
                };
                // (with one tile in every step, masked or not: the next step's wait counts on it)
                if (S::LOGITS_FIRST && !wait_logits()) break;
                if (TILES == 1) wait_values(j);
                if (t == 0 && (key0 < item_lo || key0 + kPrKeys > item_hi)) {
                    // values that some row does not see are multiplied by weights of 0 there: what is not finite
                    // becomes 0, and is added at the end where it is seen
                    const uint32_t p = p0 + value_place<TILES>(j, it.steps);
                    if (TILES == 2) wait_values(j);
                    constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
                    auto row_at = [&](int c) {
                        return raw + (ring_s - ptx::smem_addr(raw)) + (p * S::SPT + c / S::CPS) % S::SLOTS * S::SLOT +
                               c % S::CPS * kPrChunk + row * 128;
                    };
                    uint32_t most = 0;  // the row's largest exponents, of even and odd columns
#pragma unroll 1
                    for (int c = 0; c < NC; ++c) {
                        const uint8_t *v = row_at(c);
                        uint4 x[8];
#pragma unroll
                        for (int g = 0; g < 8; ++g) x[g] = *reinterpret_cast<const uint4 *>(v + (g ^ (row & 7)) * 16);
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            most = __vmaxu2(most, __vmaxu2(__vmaxu2(x[g].x & 0x7fff7fffu, x[g].y & 0x7fff7fffu),
                                                           __vmaxu2(x[g].z & 0x7fff7fffu, x[g].w & 0x7fff7fffu)));
                    }
                    const bool found = (most & 0xffffu) >= kExp || most >> 16 >= kExp;
                    if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
                        for (int c = 0; c < NC; ++c)
#pragma unroll 1
                            for (int g = 0; g < 8; ++g) {
                                uint4 *at = reinterpret_cast<uint4 *>(row_at(c) + (g ^ (row & 7)) * 16);
                                uint4 x = *at;
                                uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((w[e] & kExp) == kExp) w[e] &= 0xffff0000u;
                                    if ((w[e] & kExp << 16) == kExp << 16) w[e] &= 0xffffu;
                                }
                                *at = x;
                            }
                        tc::fence_async_smem();
                    }
                    // what some row sees is added at the end (not the rows behind the sequence, of whatever they hold)
                    const int key = key0 + row;
                    const uint32_t rows = __ballot_sync(0xffffffffu, found && key >= first_seen && key < last_seen);
                    sh.bad[turn][n_bad][warp & 3] = rows;  // (by every lane)
                    sh.bad_step[turn][n_bad] = j;
                    sh.bad_any[turn][warp & 3] |= rows ? 1u << n_bad : 0u;
                    n_bad = min(n_bad + 1, kPrMasked - 1);
                }
                if (!S::LOGITS_FIRST && !wait_logits()) break;
                const uint32_t s_at = lanes + buf * 128;
                // 32 logits come while the maximum of the 32 before is taken
                uint32_t x[4][32];
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const bool cut = key0 < all_lo || key0 + kPrKeys > all_hi;
                tc::ld32(x[0], s_at);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tc::wait_ld(x[c]);
                    if (c < 3) tc::ld32(x[c + 1], s_at + c * 32 + 32);
                    if (cut) {
                        const int from = lo - key0 - c * 32, to = hi - key0 - c * 32;
                        const uint32_t bits = (from >= 32 ? 0u : 0xffffffffu << max(from, 0)) &
                                              (to <= 0 ? 0u : 0xffffffffu >> (32 - min(to, 32)));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(bits & 1u << e)) x[c][e] = 0xff800000u;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        tops[0 + 2 * (c & 1)] = pr_max3(tops[0 + 2 * (c & 1)], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                        tops[1 + 2 * (c & 1)] = pr_max3(tops[1 + 2 * (c & 1)], __uint_as_float(x[c][e + 2]), __uint_as_float(x[c][e + 3]));
                    }
                }
                const float top = pr_max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]) * a.scale2;
                const bool rise = real && (top > m + kRise || (m == -INFINITY && top > m));
                if (__any_sync(0xffffffffu, rise)) {
                    const float f = rise ? pr_exp2(m - top) : 1.f;
                    l *= f;
                    if (rise) {
                        m = top;
                        less = top - kLift;
                    }
                    if (j > 0) {
                        if (TILES == 1) {  // the product before this step's; with two tiles S came after it
                            if (!wait_warp(sh.o_full[n_s & 1], n_s - 2 >> 1)) break;
                            tc::fence_after();
                        }
                        const uint32_t o_at = lanes + S::O + t * NC * 64;
#pragma unroll 1
                        for (int c = 0; c < (a.dim + 31) / 32; ++c) {
                            uint32_t o[32];
                            tc::ld32(o, o_at + c * 32);
                            tc::wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::st32(o_at + c * 32, o);
                        }
                    }
                }
                const float2 scale = make_float2(a.scale2, a.scale2), off = make_float2(-less, -less);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 y = tc::fma2(make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), scale, off);
                        y.x = pr_exp2(y.x);
                        y.y = pr_exp2(y.y);
                        sum[e >> 1 & 1] = tc::add2(sum[e >> 1 & 1], y);
                        p[e / 2] = pr_pack<F16>(y.x, y.y);
                    }
                    tc::st16(s_at + c * 16, p);
                    if (c == 1) {
                        tc::wait_st();
                        tc::fence_before();
                        arrive_warp(sh.p_half[buf]);
                    }
                }
                const float2 both = tc::add2(sum[0], sum[1]);
                l += both.x + both.y;
                tc::wait_st();
                tc::fence_before();
                arrive_warp(sh.p_full[buf]);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // output
            if (it.steps) {
                if (!(TILES == 2 ? wait_warp(sh.o_full[t], n_o++) : wait_warp(sh.o_full[n_s - 1 & 1], n_s - 1 >> 1))) break;
                tc::fence_after();
            }
            const int64_t at = it.q0 + mine;
            const int hq = it.key_head * a.group + it.head0 + head;
            uint16_t *out = a.out + at * a.ost[0] + hq * a.ost[1];
            const float f = l == 0.f ? 0.f : 1.f / l;
            uint32_t bad = 0;
            if (it.steps)
                for (int w = 0; w < 4; ++w) bad |= sh.bad_any[turn][w];
#pragma unroll 1
            for (int c = 0; c < (a.dim + 31) / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (it.steps) {
                    tc::ld32(o, lanes + S::O + t * NC * 64 + c * 32);
                    tc::wait_ld(o);
                }
                if (l == 0.f) {  // nothing to see
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
#pragma unroll 1
                for (uint32_t left = bad; left; left &= left - 1) {
                    const int n = __ffs(left) - 1, key0 = (it.first + sh.bad_step[turn][n]) * kPrKeys;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w)
#pragma unroll 1
                        for (uint32_t keys = sh.bad[turn][n][w]; keys; keys &= keys - 1) {
                            const int key = key0 + w * 32 + __ffs(keys) - 1;
                            if (!real || key < lo || key >= hi) continue;
                            const uint16_t *v = a.v + (it.k0 + key) * a.vst[0] + it.key_head * a.vst[1] + c * 32;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c * 32 + e < a.dim) o[e] = __float_as_uint(__uint_as_float(o[e]) + prompt_unusual<F16>(v[e]));
                        }
                }
                if (real) {
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    uint32_t y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        y[k] = pr_pack<F16>(__uint_as_float(o[e + 2 * k]) * f, __uint_as_float(o[e + 2 * k + 1]) * f);
                    uint16_t *to = out + c * 32 + e;
                    if (a.store == 32 && c * 32 + e + 16 <= a.dim) {
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(y[0]),
                                     "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                                     : "memory");
                    } else if (a.store >= 16) {
                        if (c * 32 + e + 8 <= a.dim) *reinterpret_cast<uint4 *>(to) = make_uint4(y[0], y[1], y[2], y[3]);
                        if (c * 32 + e + 16 <= a.dim)
                            *reinterpret_cast<uint4 *>(to + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (c * 32 + e + k < a.dim) to[k] = static_cast<uint16_t>(y[k / 2] >> (k & 1) * 16);
                    }
                }
                }
            }
            if (a.lse && real)
                a.lse[at * a.lse_stride + hq] = l == 0.f ? -INFINITY : (less + kLift + log2f(l * kDrop)) * 0.6931471805599453f;
        }
    } else if (warp == S::SOFT + 2) {
        few_registers();
        // scheduling: items dealt in turn, every other round backwards, so that none gets the longest of each
        PromptCursor cursor = prompt_begin<TILES>(a);
        for (uint32_t i = 0; ok; ++i) {
            const uint32_t at = i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            PromptItem it{};
            prompt_item<TILES>(a, at, cursor, &it);
            const int s = i % kPrItems;
            if (i >= kPrItems && !wait_warp(sh.item_empty[s], i / kPrItems - 1)) break;
            if (lane == 0) sh.item[s] = it;
            arrive_warp(sh.item_full[s]);
            if (it.end) break;
        }
    } else if (warp == S::SOFT + 1) {
        few_registers();
        // loads, by the whole warp
        uint32_t slot = 0, round = 0, tiles_q[2] = {0, 0};  // the next slot of the ring, how often it has been used
        for (uint32_t i = 0;; ++i) {
            if (!wait_warp(sh.item_full[i % kPrItems], i / kPrItems)) break;
            const PromptItem &item = sh.item[i % kPrItems];
            const uint32_t end = (item.end), steps = (item.steps), key_head = (item.key_head);
            const int head0 = key_head * a.group + (item.head0);
            const int q0 = (item.q0 + item.t0), left = (item.nq - item.t0);
            const int key0 = (item.k0 + item.first * kPrKeys);
            arrive_warp(sh.item_empty[i % kPrItems]);
            if (end) break;
            if (!steps) continue;
            auto load_q = [&](int t) {
                if (t * a.tokens_tile >= left) return;
                if (tiles_q[t] && !wait_warp(sh.q_empty[t], tiles_q[t] - 1)) return;
                ++tiles_q[t];
                tc::expect(bar(sh.q_full[t]), NC * 128 * a.heads_tile * a.tokens_tile);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    tc::load_3d(q_s + (t * NC + c) * kPrChunk, &a.qm, c * 64, head0, q0 + t * a.tokens_tile, bar(sh.q_full[t]));
            };
            auto load_tile = [&](const CUtensorMap &m, uint32_t j) {
#pragma unroll
                for (int p = 0; p < S::SPT; ++p) {
                    if (!ok || (round && !wait_warp(sh.ring_empty[slot], round - 1))) return;
                    const uint32_t full = bar(sh.ring_full[0]) + slot * 8;
                    tc::expect(full, S::SLOT);
#pragma unroll
                    for (int c = 0; c < S::CPS; ++c)
                        tc::load_3d(ring_s + slot * S::SLOT + c * kPrChunk, &m, (p * S::CPS + c) * 64, key_head,
                                    key0 + j * kPrKeys, full);
                    if (++slot == S::SLOTS) {
                        slot = 0;
                        ++round;
                    }
                }
            };
            load_q(0);
            load_tile(a.km, 0);
            if constexpr (TILES == 2) load_q(1);
#pragma unroll 1
            for (uint32_t j = 0; j < steps && ok; ++j) {  // K0 V0 K1 V1 ..., with one tile K0 K1 V0 K2 V1 ...
                if (j) load_tile(a.km, j);
                if constexpr (TILES == 2) load_tile(a.vm, j);
                else if (j) load_tile(a.vm, j - 1);
            }
            if constexpr (TILES == 1) load_tile(a.vm, steps - 1);
            if (!ok) break;
        }
        // copies in flight end before the block does, also where only another warp's wait has run out
        for (uint32_t s = 0; s < S::SLOTS; ++s) {
            const uint32_t used = round + (s < slot);
            if (used) drained(sh.ring_full[s], used - 1);
        }
        for (int t = 0; t < TILES; ++t)
            if (tiles_q[t]) drained(sh.q_full[t], tiles_q[t] - 1);
    } else if (warp == S::SOFT || (TILES == 2 && warp == S::SOFT + 3)) {
        few_registers();
        // products, by the whole warp.  With two row tiles a warp a tile, so that one's waits and bookkeeping pass while
        // the other's products run; the tiles take turns, else both come to do their softmax at the same time and leave
        // the tensor cores idle meanwhile (a fifth slower, as is one warp for both).
        const int t = warp != S::SOFT;
        const uint32_t tm = (tmem);
        const uint32_t q_desc = tc::smem_desc(q_s, 16), k_desc = tc::smem_desc(ring_s, 16);
        const uint32_t v_desc = tc::smem_desc(ring_s, kPrChunk);
        const uint32_t qk = tc::instr_desc(F16, kPrKeys, false, a.negative);
        const int k_steps = (a.dim + 15) / 16;
        // of the values' columns a full slot, and what is left for the last
        const uint32_t pv_full = tc::instr_desc(F16, S::CPS * 64, true, false);
        const uint32_t pv_last = tc::instr_desc(F16, (a.dim - (NC - S::CPS) * 64 + 15) / 16 * 16, true, false);
        auto wait_all = [&](const uint64_t &b, uint32_t n) {
            wait_warp(b, n);
            tc::fence_after();
            return ok;
        };
        // tiles come in the order in which they are used: their first slot and the phase of its barriers
        uint32_t slot = 0, phase = 0;
        auto step = [&](uint32_t s, int c) { return s + c < S::SLOTS ? s + c : s + c - S::SLOTS; };
        auto take = [&]() {  // the next tile's first slot, when it is there
            const uint32_t s = slot;
#pragma unroll
            for (int c = 0; c < S::SPT; ++c) {
                wait_all(sh.ring_full[slot], phase);
                if (++slot == S::SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            return s;
        };
        auto free_tile = [&](uint32_t s) {
#pragma unroll
            for (int c = 0; c < S::SPT; ++c) tc::commit(bar(sh.ring_empty[0]) + step(s, c) * 8);
        };
        // S = Q K^T of row tile t into S buffer `to`
        auto first_product = [&](int t, int to, uint32_t s) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const uint32_t q = q_desc + (t * NC + c) * (kPrChunk / 16);
                const uint32_t k = k_desc + step(s, c / S::CPS) * (S::SLOT / 16) + c % S::CPS * (kPrChunk / 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 16 columns, 32 bytes, on
                    if (c * 4 + i < k_steps) tc::mma_ss(tm + to * 128, q + 2 * i, k + 2 * i, qk, c + i > 0);
            }
        };
        // O += P V; the weights of 64 keys are multiplied while those of the others are made
        uint32_t n_turn = 0;
        auto my_turn = [&] { return t == 0 ? n_turn == 0 || wait_all(sh.turn[0], n_turn - 1) : wait_all(sh.turn[1], n_turn); };
        auto your_turn = [&] {
            ++n_turn;
            arrive_warp(sh.turn[1 - t]);
        };
        auto second_product = [&](int t, int from, uint32_t n, uint32_t s, bool add, bool turns) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (!wait_all(h ? sh.p_full[from] : sh.p_half[from], n)) return;
                if (turns && h == 0 && !my_turn()) return;
#pragma unroll
                for (int c = 0; c < NC; c += S::CPS) {
                    const uint32_t d = tm + S::O + t * NC * 64 + c * 64, w = tm + from * 128 + h * (kPrKeys / 4);
                    const uint32_t v = v_desc + step(s, c / S::CPS) * (S::SLOT / 16) + h * (kPrKeys / 2 * 128 / 16);
#pragma unroll
                    for (int k = 0; k < kPrKeys / 32; ++k)  // 16 keys, 2048 bytes, on
                        tc::mma_ts(d, w + k * 8, v + 128 * k, c + S::CPS < NC ? pv_full : pv_last, add || h + k > 0);
                }
            }
        };
        uint32_t n_q = 0, n_p = 0;
        for (uint32_t i = 0;; ++i) {
            if (!wait_all(sh.item_full[i % kPrItems], i / kPrItems)) break;
            const PromptItem &it = sh.item[i % kPrItems];
            const uint32_t end = (it.end), steps = (it.steps);
            const uint32_t two = (TILES == 2 && it.t0 + a.tokens_tile < it.nq);
            arrive_warp(sh.item_empty[i % kPrItems]);
            if (end) break;
            if (!steps) continue;
            if constexpr (TILES == 2) {
                uint32_t k = take();
                const bool mine = t == 0 || two;
                if (mine) {
                    if (!wait_all(sh.q_full[t], n_q++) || (two && !my_turn())) break;
                    first_product(t, t, k);
                    if (two) your_turn();
                    tc::commit(bar(sh.s_full[0]) + t * 8);
                    if (steps == 1) tc::commit(bar(sh.q_empty[0]) + t * 8);
                }
                free_tile(k);
#pragma unroll 1
                for (uint32_t j = 0; j < steps && ok; ++j) {
                    // what a step needs is there before its weights are waited for, and what it has used is given back when
                    // all its products are on their way: between the two only products
                    const bool more = j + 1 < steps;
                    const uint32_t v = take();
                    if (more) k = take();
                    if (mine) {
                        second_product(t, t, n_p++, v, j > 0, two);
                        if (!ok) break;
                        if (more) first_product(t, t, k);
                        if (two) your_turn();
                        tc::commit((more ? bar(sh.s_full[0]) : bar(sh.o_full[0])) + t * 8);
                        if (j + 2 == steps) tc::commit(bar(sh.q_empty[0]) + t * 8);
                    }
                    free_tile(v);
                    if (more) free_tile(k);
                }
            } else {
                wait_all(sh.q_full[0], n_q++);
                const uint32_t t0 = n_p;  // steps before this item: the S buffers go on in turn
                uint32_t k = 0;
#pragma unroll 1
                for (uint32_t j = 0; j < steps + 2 && ok; ++j) {
                    const bool more = j < steps;
                    uint32_t v = 0;
                    if (j >= 2) v = take();
                    if (more) k = take();
                    if (!ok) break;
                    if (j >= 2) {
                        const uint32_t buf = n_p & 1;
                        second_product(0, buf, n_p++ >> 1, v, j > 2, false);
                        if (!ok) break;
                        tc::commit(bar(sh.o_full[0]) + buf * 8);
                    }
                    if (more) {
                        first_product(0, (t0 + j) & 1, k);
                        tc::commit(bar(sh.s_full[0]) + ((t0 + j) & 1) * 8);
                    }
                    if (j >= 2) free_tile(v);
                    if (more) free_tile(k);
                    if (j + 1 == steps) tc::commit(bar(sh.q_empty[0]));
                }
            }
            if (!ok) break;
        }
        // products in flight end before the tensor memory is given back
        tc::commit(bar(sh.drain[0]) + t * 8);
        drained(sh.drain[t], 0);
        tc::fence_after();
    } else {
        few_registers();
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == S::SOFT) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

template <bool F16, int NC>
int launch_prompt_shape(const PromptArgs &a, int64_t items, cudaStream_t cs) {
    using S = PromptShape<NC>;
    const void *fn = reinterpret_cast<const void *>(&k_prompt_attend<F16, NC>);
    int sms = 0, per_sm = 0;
    if (prepare(fn, S::THREADS, S::SMEM, S::SMEM, &sms, &per_sm) != cudaSuccess) return LC_ERR_CUDA;
    return launch_after(fn, static_cast<unsigned>(std::min<int64_t>(items, sms)), S::THREADS, S::SMEM, cs, &a);
}

template <bool F16>
int launch_prompt_type(const PromptArgs &a, int64_t items, cudaStream_t cs) {
    switch ((a.dim + 63) / 64) {
        case 1: return launch_prompt_shape<F16, 1>(a, items, cs);
        case 2: return launch_prompt_shape<F16, 2>(a, items, cs);
        case 3: return launch_prompt_shape<F16, 3>(a, items, cs);
        default: return launch_prompt_shape<F16, 4>(a, items, cs);
    }
}

}  // namespace lc
