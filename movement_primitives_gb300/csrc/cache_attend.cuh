// Attention of one new token a sequence over a paged key-value cache
// (lc_cache_attend):
//     x_j = scale * q . k_j,  w = softmax(x),  out = sum_j w_j v_j
// over the slots j that are seen.
//
// Mathematics.  One pass over the keys and values: a warp keeps, for up to 16
// query heads of one key head, the running maximum m of the logits (in base 2:
// x_j log2 e), the sum l of 2^(x_j - m) and the output o of the slots it has
// taken, all in float32, and rescales l and o when m grows.  Parts (m, l, o)
// of one row join as sums weighted by 2^(m - max m).
//
// Both products are warp-level matrix instructions (mma.sync m16n8k16) with
// the cache as the 16-row operand: 16 slots x 16 columns of the keys by 8
// query heads, and 16 columns x 16 slots of the values by 8 query heads, so
// that up to 8 query heads a key head cost one instruction where heads as rows
// would cost two.  The logits' fragment becomes the second product's operand
// by one 8 x 8 transpose across lanes (movmatrix) a slot octet and number.  With G
// query heads a key head the pass does G operations a byte of 16-bit cache, so
// memory bounds it up to the 16 heads of a unit and the accumulators fit
// registers.
//
// A weight enters the second product as two numbers of the values' 16-bit type,
// its leading bits (8 in bfloat16, 11 in float16) and what they leave, rounded:
// together within 2^-16 and 2^-22 of it, so that the output's own rounding is the
// only one that shows (one rounded number a weight: errors against 64 bits 7 to
// 20 % larger, 3 to 4 % less time for short units, none for full batches).  Neither
// is negative, nor zero for a weight above 0 (in float16, above 2^-38 of the
// largest), so that an infinite value stays one.  The sum l takes the weights
// whole.  Float16 has few exponents, so its weights are lifted by 2^14: the largest
// is 2^14, and one of 2^-38 of it is still held to a bit, so that a million slots
// together lose nothing to an outlier above them.  Others are lowered by 2^-31, so
// that sums of as many slots as there can be stay in float32 whatever the values
// are; what is lost is below 2^-95 of the largest.
//
// E4M3 codes are float16 numbers, converted exactly two at a time; their
// products run in float16.  The keys' scales multiply the logits.  The values'
// scales s_j join the weights as 2^(x_j + log2 |s_j| - mv), mv the running
// maximum of that exponent (lifted as above): the largest weight is the same
// whatever the scales; o is kept relative to mv.  These weights are one float16
// number each: 2^-11 is an eighth of the bfloat16 output's rounding, and a second
// number would go into the pass that instructions bound.
//
// Work.  Slots are taken in steps of TOK by one warp.  A (sequence, key head,
// block of 16 query heads) is a unit; the steps of all units, laid end to end,
// are cut into equal runs, one a warp, whatever the lengths: the warps find
// their run from the lengths on the device.  A unit inside one run is finished
// there; one that is cut leaves parts in the workspace, which k_attend_join
// joins in their order, so results do not depend on timing.  Each warp streams
// its run through a ring of its own in shared memory (cp.async, 16 bytes a
// lane, rows swizzled for ldmatrix) that runs ahead across units, with no
// barrier between warps.  Where units are short (kUnitSteps) a block, a cluster
// of blocks (few units) or a warp (many) takes one instead, joined in shared
// memory, with no second launch.
//
// Measured on GB300 (device time a call; the copy peak is 6678 GB/s): 64
// sequences of up to 8192 slots, 32 query on 8 key heads of 128 bfloat16, 1.09
// GB, 167 us (6.5 TB/s, 98 %); one sequence of 131071 float16 slots, 537 MB, 89
// us (6.0 TB/s; 9 us of it the launch and the joining of 152 parts a row); 16
// sequences of up to 2048, 71 MB, 21.5 us, about half of it what a call costs
// whatever its size: the lengths, the pages, the first rows and the parts are
// read one after the other, about a microsecond each.  E4M3 at 8 query heads a
// key head, 148 MB, 44 us with weights collected: a step of 8 KiB takes 930
// instructions, and with two warps a scheduler their latency bounds it
// (issue slots 46 % busy).
#pragma once

#include <cooperative_groups.h>

#include <cmath>
#include <type_traits>

#include "cache_common.cuh"

namespace lc {

namespace cg = cooperative_groups;

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
// Blocks of an SM (at least; registers) and steps in a warp's ring.  Measured
// on 1.09 GB of bfloat16 (64 sequences of up to 8192 slots, dim 128) and on
// 0.27 GB of dim 64: 2 blocks x 2 steps 167 and 51 us; x 3 steps 176 and 52; 3
// blocks x 2 steps 208 (fewer registers) and 62.  More streams do not hide more
// latency, they cost the memory its order.
constexpr int kAtBlocks = 2, kAtStages = 2;
constexpr int kAtRows = 16;        // query heads of a unit at most
constexpr int kAtMaxBlocks = 608;  // of the main kernel; sizes the workspace
constexpr int kAtMaxRuns = kAtMaxBlocks * kAtWarps;
constexpr int kJoinLeast = 128, kJoinMost = 1024;  // threads of a joining block
constexpr int kJoinRows = kJoinLeast / 32;  // rows of a block of the least width
constexpr int kJoinFew = 32;       // parts of a row that one warp joins
constexpr int kScorePer = 4;       // slots of a thread (4, 8, 16: 43.7, 45.4, 53 us
                                   // of 32 E4M3 sequences with scores)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A run takes at least this many steps: shorter ones leave more parts to join
// than the further warps save, longer ones leave warps idle.  Of 1, 2, 4, 6, 8
// steps: one sequence of 32000 slots, 16 query heads on one key head 36, 32,
// 23, 24, 24 us; of 8000 slots, 8 key heads 14.9, 14.8, 14.9, 17.2, 18.8.
constexpr int kAtMinSteps = 4;
// A unit is one block's, or a cluster's of up to kUnitCluster blocks while
// there are kUnitBlocks at most, where a warp then takes kUnitSteps steps or
// fewer: one launch and no parts in memory, but units of unlike lengths are
// not evened out.  GPU time against runs: 8 units of 64 steps of 16 KiB, weights
// collected, 15.2 and 23.1 us; 96 units of up to 50 steps of 5 KiB 11.4 and 13.2
// (the host saves 5 us of a launch too); at 16 steps a warp, 84 units of up to 125
// steps 21.8 and 14.1, 128 units of up to 128 steps of 8 KiB 27.4 and 21.7.
constexpr int kUnitSteps = 8, kUnitBlocks = 304, kUnitCluster = 8;
// Where a unit would be one block's, it is one warp's instead if that is
// sooner, counting kUnitCost steps for what a unit costs besides its own: the
// blocks' rounds of kUnitBlocks units against the warps' of four times as many.
// A warp against a block: 1000 sequences of up to 64 slots of 8 key heads 43
// and 97 us, 600 of up to 500 (E4M3) 79 and 110, 100 of 200 (E4M3) 13.9 and 15.2,
// but 40 of up to 250 19.9 and 9.5; at the boundary 100 of 200 (bfloat16) 19.4 and
// 18.0, 76 of up to 100 10.4 and 10.0.
constexpr int kUnitCost = 2;
// The largest shape's registers hold no second form of the end.
constexpr __host__ __device__ bool unit_by_warp(int padded, int rows) { return padded < 256 || rows <= 8; }

struct AttendArgs {
    CacheArgs c;
    const uint16_t *q;
    uint16_t *out;
    const int32_t *lengths;
    const uint8_t *mask;
    float *lse, *scores;
    int64_t qst[2], ost[2], sst[2];
    int64_t mask_stride, lse_stride;
    int32_t q_heads, group, window;
    int32_t row_blocks;   // units of one key head
    float scale2;         // scale * log2 e
    bool q_wide;          // rows of q on 8-byte boundaries
    bool warp_units;      // k_attend_unit: a unit a warp
    // workspace
    float *part;          // [2 runs][part_rows][part_pitch]
    float2 *part_ml;      // [2 runs][part_rows]
    int2 *split;          // per unit: first and last run of a unit that is cut, first -1 when it is not
    float *lse2;          // [sequence, query head], base 2, of units that are not cut (with scores)
    float *logits;        // [sequence, query head, logit_stride], base 2, from the first slot seen (with scores)
    int64_t logit_stride;
    int32_t part_rows, part_pitch;
    // of k_attend_join
    int32_t join_blocks, join_rows;
    uint32_t score_blocks;
    FastDiv chunk_div, head_div, q_div, group_div;
};

// Slots of a step: of 8 KiB where the shapes allow, but 32 of E4M3 rows of 192
// (12 KiB; for 32 sequences of up to 8000 slots of 8 key heads in [head, slot]
// order 16 of them take 90 us and 32 of them 77, in [slot, head] order 93 either
// way; of bfloat16 rows of 96, the same 192 bytes, 65 and 66).
constexpr int step_slots(int padded, int elem_bytes) {
    return padded * elem_bytes <= (elem_bytes == 1 ? 192 : 128) ? 32 : 16;
}

// Steps in a warp's ring where a unit is a block's: few steps, whose latency
// counts.
template <int DP, int KV>
constexpr int kUnitStages = DP * (KV == LC_CACHE_E4M3 ? 1 : 2) > 256 || DP == 192 ? 2 : 3;

// head_dim as the kernels take it.  Columns past head_dim cost products and
// registers, not bytes: 2 sequences of up to 99459 float16 slots, 16 query heads
// a key head of 192, padded to 256 299 us, to 192 157; 7 sequences of up to 1999,
// 12 heads of 80, to 128 15.4, to 96 14.1.  Rows that are read element by element
// are slower than either and have fewer forms.
inline int padded_dim(int dim, bool vec) {
    if (vec && dim > 64 && dim <= 96) return 96;
    if (vec && dim > 128 && dim <= 192) return 192;
    return dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
}

// Shapes of one instantiation.  DP: head_dim rounded up (padded_dim); KV: an
// lc_cache_type; NG: query heads in eights (1, 2); STAGES: steps in a warp's
// ring.
template <int DP, int KV, int NG, int STAGES>
struct AtShape {
    static constexpr int EB = KV == LC_CACHE_E4M3 ? 1 : 2;
    static constexpr int RB = DP * EB;                       // bytes of a row
    static constexpr int CH = RB / 16;                       // its 16-byte chunks
    static constexpr int TOK = step_slots(DP, EB);
    static constexpr int STEP = 2 * TOK * RB;                // keys, then values
    static constexpr int ST = STAGES;
    static constexpr int SC = KV == LC_CACHE_E4M3 ? 2 * TOK * 4 : 0;  // scales of a step
    static constexpr int WARP_BYTES = ST * (STEP + SC);
    static constexpr int OP = DP + 4;                        // floats between the heads of a warp's output
    static constexpr int SMEM = kAtWarps * WARP_BYTES;
    static_assert(8 * NG * OP * 4 <= WARP_BYTES, "a warp's output is staged in its ring");
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t (&b)[2]) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Two numbers >= 0 as the sums of two each: `lead`, their leading bits, and
// `rest`, the remainders, rounded, but above 0 for a number above 0.
template <bool F16>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t *lead, uint32_t *rest) {
    constexpr float kLeast = F16 ? 0x1p-24f : 0x1p-133f;  // the type's smallest step
    float2 v;
    if constexpr (F16) {
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(*lead) : "f"(hi), "f"(lo));
        v = __half22float2(*reinterpret_cast<const __half2 *>(lead));
    } else {
        *lead = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
        v = make_float2(__uint_as_float(*lead << 16), __uint_as_float(*lead & 0xffff0000u));
    }
    *rest = pack2<F16>(fmaxf(lo - v.x, fminf(lo, kLeast)), fmaxf(hi - v.y, fminf(hi, kLeast)));
}

// Two E4M3 codes (the low 16 bits) as float16, exactly.
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t codes) {
    uint32_t v;
    asm("{.reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c;}" : "=r"(v) : "r"(codes));
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp, 0 for -infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_fast(float x) {  // -infinity for 0
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of the largest weight of a row's sum l (see above), and the logarithm,
// base 2, of the whole sum from l and the maximum that it is relative to: the
// factor is taken out first, whose digits would cost the logarithm some of its.
constexpr __host__ __device__ float sum_lift(bool f16) { return f16 ? 14.f : -31.f; }
template <bool F16>
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.f ? -INFINITY : m + sum_lift(F16) + log2f(l * (F16 ? 0x1p-14f : 0x1p31f));
}

// The slots [lo, n) that sequence b's query sees (before the mask).
__device__ __forceinline__ int seen_from(const AttendArgs &a, int b, int *n) {
    *n = cache_length(a.c, a.lengths, b, kClassAttend);
    return a.window && a.window < *n ? *n - a.window : 0;
}

// A place in the steps of all units: step `t` of `steps` of unit `unit` of
// sequence b.
struct Place {
    int b, unit, t, steps, lo, n;
};

template <int TOK>
__device__ __forceinline__ void enter_sequence(const AttendArgs &a, Place &p) {
    p.lo = seen_from(a, p.b, &p.n);
    p.steps = (p.n - p.lo + TOK - 1) / TOK;
}

// To the next step; there has to be one.
template <int TOK>
__device__ __forceinline__ void next_step(const AttendArgs &a, int units, Place &p) {
    if (++p.t < p.steps) return;
    p.t = 0;
    if (++p.unit < units) return;
    p.unit = 0;
    do {
        ++p.b;
        enter_sequence<TOK>(a, p);
    } while (p.steps == 0);
}

template <int DP, int KV, int NG, bool VEC, int STAGES>
struct Attend {
    using S = AtShape<DP, KV, NG, STAGES>;
    static constexpr bool F16 = KV == LC_CACHE_F16, Q8 = KV == LC_CACHE_E4M3;
    static constexpr bool M16 = F16 || Q8;       // the matrix instructions' type is float16
    // log2 of the largest weight: of the second product, and of the sum l
    static constexpr float kLift = sum_lift(M16), kSumLift = sum_lift(F16);
    static constexpr int KS = DP / 16;           // 16-wide pieces of a row
    static constexpr int MT = S::TOK / 16;       // 16-slot pieces of a step

    const AttendArgs &a;
    const int lane;
    uint8_t *ring;        // this warp's
    uint32_t ring_s;
    uint32_t *seen_bits;  // this warp's, one word a stage

    // the unit: sequence, query heads, the first of them
    int b, rows, q0;

    uint32_t qb[KS][NG][2];
    float o[KS][NG][4], l[NG][2];
    float m[NG][2];        // the running maximum of the logits less kSumLift, which l and o are relative to
    float q_scale[NG][2];  // E4M3: what the float16 queries are to be multiplied by, times scale2
    float mv[NG][2];       // E4M3: that of logit + log2 |value scale|, less kLift, which o is relative to

    // the pages of a step's slots, one a lane, read one step ahead of its rows
    int next_page, next_row, next_head;
    bool next_seen;

    __device__ __forceinline__ static uint32_t swz(int row, int chunk) {
        if constexpr (S::RB % 128 == 0) return (chunk ^ (row & 7)) * 16;
        if constexpr (S::RB % 64 == 0) return (chunk ^ (row >> 1 & 3)) * 16;
        return (chunk ^ (row >> 2 & 1)) * 16;  // rows of 96 bytes
    }

    // The value column that row g (+ 8 i) of 16-wide piece c stands for: E4M3
    // columns come in adjacent pairs.
    __device__ __forceinline__ static int col_of(int c, int g, int i) {
        return Q8 ? 16 * c + 2 * g + i : 16 * c + g + 8 * i;
    }

    // Query heads as the 16 x 8 operand: head lane / 4, columns k = 2q, 2q +
    // 1, 2q + 8, 2q + 9 of each 16-wide piece; for E4M3 keys, which come four
    // adjacent columns a lane, 4q .. 4q + 3.
    __device__ __forceinline__ void load_q() {
        const int q = lane & 3;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int head = 8 * g + (lane >> 2);
            const uint16_t *p = a.q + b * a.qst[0] + (q0 + min(head, rows - 1)) * a.qst[1];
            const bool on = head < rows;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int c0 = 16 * ks + (Q8 ? 4 * q : 2 * q), c1 = c0 + (Q8 ? 2 : 8);
                uint32_t x, y;
                if (a.q_wide) {  // whole fours of columns on 8-byte boundaries
                    if (Q8) {
                        uint2 v = make_uint2(0, 0);
                        if (on && c0 < a.c.dim) v = *reinterpret_cast<const uint2 *>(p + c0);
                        x = v.x;
                        y = v.y;
                    } else {
                        x = on && c0 < a.c.dim ? *reinterpret_cast<const uint32_t *>(p + c0) : 0;
                        y = on && c1 < a.c.dim ? *reinterpret_cast<const uint32_t *>(p + c1) : 0;
                    }
                } else {
                    auto at = [&](int i) { return on && i < a.c.dim ? static_cast<uint32_t>(p[i]) : 0u; };
                    x = at(c0) | at(c0 + 1) << 16;
                    y = at(c1) | at(c1 + 1) << 16;
                }
                qb[ks][g][0] = x;
                qb[ks][g][1] = y;
            }
        }
        if constexpr (Q8) {
            // bfloat16 to float16, each head divided by the power of two at or below its largest
            // magnitude: exact but for elements below 2^-14 of it, which are off by at most 2^-25
            // of it
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t top = 0;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = max(top, max(qb[ks][g][i] & 0x7fffu, qb[ks][g][i] >> 16 & 0x7fffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = min(max(top >> 7, 1u), 253u);  // 1 / 2^(e - 127) is a normal number too
                const float down = __uint_as_float((254 - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t v = qb[ks][g][i];
                        qb[ks][g][i] =
                            pack2<true>(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
                    }
                // logits come by columns: heads 2 q, 2 q + 1
#pragma unroll
                for (int u = 0; u < 2; ++u) q_scale[g][u] = a.scale2 * __shfl_sync(0xffffffffu, up, (2 * q + u) * 4);
            }
        }
    }

    // Reads the page of this lane's slot of the step that starts at slot j0 of
    // sequence pb.
    __device__ __forceinline__ void find_pages(int pb, int head, int j0, int n) {
        const int j = j0 + lane;
        next_page = -1;
        next_row = 0;
        next_head = head;
        next_seen = false;
        if (lane < S::TOK && j < n) {
            const int i = static_cast<int>(fast_div(static_cast<uint32_t>(j), a.c.page_div));
            next_row = j - i * a.c.page;
            next_page = a.c.table[pb * a.c.table_stride + i];
            next_seen = !a.mask || a.mask[pb * a.mask_stride + j];
        }
    }

    // Starts the copies of the step whose pages find_pages read, into `stage`.
    __device__ __forceinline__ void issue(int stage) {
        const bool in_pool = next_page >= 0 && next_page < a.c.n_pages;
        if (next_seen && !in_pool) report_error(LC_ERR_CACHE_INDEX, kClassAttend);
        const bool seen = next_seen && in_pool;
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        int64_t ko = 0, vo = 0;
        if (seen) {
            ko = row_offset(a.c.kst, next_page, next_head, next_row);
            vo = row_offset(a.c.vst, next_page, next_head, next_row);
        }
        uint8_t *dst = ring + stage * (S::STEP + S::SC);
        const uint32_t dst_s = ring_s + stage * (S::STEP + S::SC);
        if (lane == 0) seen_bits[stage] = bits;
        if constexpr (Q8)
            if (lane < S::TOK) {
                const float *ks = a.c.ks + (seen ? row_offset(a.c.kss, next_page, next_head, next_row) : 0);
                const float *vs = a.c.vs + (seen ? row_offset(a.c.vss, next_page, next_head, next_row) : 0);
                cp_async4_zfill(dst_s + S::STEP + 4 * lane, ks, seen);
                cp_async4_zfill(dst_s + S::STEP + 4 * (S::TOK + lane), vs, seen);
            }
        if constexpr (VEC) {
            const int chunks = a.c.dim * S::EB / 16;
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int i = 0; i < S::TOK * S::CH / 32; ++i) {
                    const int at = i * 32 + lane, row = at / S::CH, chunk = at % S::CH;
                    const int64_t off = __shfl_sync(0xffffffffu, side ? vo : ko, row);
                    const bool real = (bits >> row & 1) && chunk < chunks;
                    cp_async16_zfill(dst_s + side * S::TOK * S::RB + row * S::RB + swz(row, chunk),
                                     (side ? a.c.v : a.c.k) + off * S::EB + (real ? chunk * 16 : 0), real);
                }
        } else {
#pragma unroll 1
            for (int side = 0; side < 2; ++side)
#pragma unroll 1
                for (int row = 0; row < S::TOK; ++row) {
                    const int64_t off = __shfl_sync(0xffffffffu, side ? vo : ko, row);
                    const uint8_t *src = (side ? a.c.v : a.c.k) + off * S::EB;
                    for (int e = lane; e < DP; e += 32) {
                        const bool real = (bits >> row & 1) && e < a.c.dim;
                        uint8_t *to = dst + side * S::TOK * S::RB + row * S::RB + swz(row, e * S::EB / 16) +
                                      e * S::EB % 16;
                        if constexpr (Q8)
                            *to = real ? src[e] : uint8_t(0);
                        else
                            *reinterpret_cast<uint16_t *>(to) =
                                real ? reinterpret_cast<const uint16_t *>(src)[e] : uint16_t(0);
                    }
                }
        }
    }

    __device__ __forceinline__ void begin_unit(int seq, int unit) {
        b = seq;
        const int h = a.row_blocks == 1 ? unit : unit / a.row_blocks, rb = unit - h * a.row_blocks;
        q0 = h * a.group + rb * kAtRows;
        rows = min(a.group - rb * kAtRows, kAtRows);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[g][i] = mv[g][i] = -INFINITY;
                l[g][i] = 0.f;
            }
#pragma unroll
        for (int c = 0; c < KS; ++c)
#pragma unroll
            for (int g = 0; g < NG; ++g) o[c][g][0] = o[c][g][1] = o[c][g][2] = o[c][g][3] = 0.f;
        load_q();
    }

    // Takes the step in `stage`, the unit's slots from `at` on (counted from
    // the first seen).
    __device__ __forceinline__ void take(int stage, int at) {
        const uint32_t bits = seen_bits[stage];
        if (!a.logits && bits == 0) return;
        const int slot = lane >> 2, q = lane & 3, mat = lane >> 3;
        const uint32_t ks_s = ring_s + stage * (S::STEP + S::SC), vs_s = ks_s + S::TOK * S::RB;
        const float *scales = reinterpret_cast<const float *>(ring + stage * (S::STEP + S::SC) + S::STEP);

        // logits: x[t][g][0, 1] of slot 16 t + lane / 4, [2, 3] of the slot 8 on; query heads 8 g +
        // 2 q, + 1
        float x[MT][NG][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int g = 0; g < NG; ++g) x[t][g][0] = x[t][g][1] = x[t][g][2] = x[t][g][3] = 0.f;
            const int row = 16 * t + (lane & 7) + (mat & 1) * 8;
            if constexpr (Q8) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t r[4];
                    ldsm_x4(r, ks_s + row * S::RB + swz(row, ks + (mat >> 1)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a0 = e4m3_halves(r[2 * i]), a2 = e4m3_halves(r[2 * i] >> 16);
                        const uint32_t a1 = e4m3_halves(r[2 * i + 1]), a3 = e4m3_halves(r[2 * i + 1] >> 16);
#pragma unroll
                        for (int g = 0; g < NG; ++g) mma16816<true>(x[t][g], a0, a1, a2, a3, qb[ks + i][g]);
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t r[4];
                    ldsm_x4(r, ks_s + row * S::RB + swz(row, 2 * ks + (mat >> 1)));
#pragma unroll
                    for (int g = 0; g < NG; ++g) mma16816<F16>(x[t][g], r[0], r[1], r[2], r[3], qb[ks][g]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 16 * t + slot + 8 * i;
                const float f = Q8 ? scales[col] : 1.f;
                const bool on = bits >> col & 1;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        x[t][g][2 * i + u] = on ? x[t][g][2 * i + u] * (Q8 ? q_scale[g][u] * f : a.scale2) : -INFINITY;
            }
        }
        if (a.logits) {
            float *to = a.logits + (int64_t(b) * a.q_heads + q0) * a.logit_stride + at;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int head = 8 * g + 2 * q + u;
                    if (head < rows)
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                to[head * a.logit_stride + 16 * t + slot + 8 * i] = x[t][g][2 * i + u];
                }
            if (bits == 0) return;
        }
        // running maximum, sum and rescaling of the output
        auto warp_max = [](float v) {
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        };
        // E4M3: the values' scales, whose logarithms join the logits for the second product
        float sv[MT][2], lv[MT][2];
        if constexpr (Q8) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sv[t][i] = scales[S::TOK + 16 * t + slot + 8 * i];
                    lv[t][i] = log2_fast(fabsf(sv[t][i]));
                }
        }
        bool grown = false;
        float keep[NG][2];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float top = fmaxf(x[0][g][u], x[0][g][2 + u]);
#pragma unroll
                for (int t = 1; t < MT; ++t) top = fmaxf(top, fmaxf(x[t][g][u], x[t][g][2 + u]));
                top = warp_max(top) - kSumLift;
                keep[g][u] = 1.f;
                if (top > m[g][u]) {
                    const float k = exp2_fast(m[g][u] - top);
                    m[g][u] = top;
                    l[g][u] *= k;
                    if (!Q8) {
                        keep[g][u] = k;
                        grown = true;
                    }
                }
                const float safe = m[g][u] == -INFINITY ? 0.f : m[g][u];
                float sum = 0.f;
                if constexpr (Q8) {
                    float topv = -INFINITY;
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            sum += exp2_fast(x[t][g][2 * i + u] - safe);
                            x[t][g][2 * i + u] += lv[t][i];
                            topv = fmaxf(topv, x[t][g][2 * i + u]);
                        }
                    topv = warp_max(topv) - kLift;
                    if (topv > mv[g][u]) {
                        keep[g][u] = exp2_fast(mv[g][u] - topv);
                        mv[g][u] = topv;
                        grown = true;
                    }
                    const float safe_v = mv[g][u] == -INFINITY ? 0.f : mv[g][u];
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            x[t][g][2 * i + u] = copysignf(exp2_fast(x[t][g][2 * i + u] - safe_v), sv[t][i]);
                } else {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            x[t][g][2 * i + u] = exp2_fast(x[t][g][2 * i + u] - safe);
                            sum += x[t][g][2 * i + u];
                        }
                }
                l[g][u] += sum;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int c = 0; c < KS; ++c)
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[c][g][i] *= keep[g][i & 1];
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            uint32_t p[NG][2], rest[NG][2];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // slots lane / 4 of two heads -> head lane / 4 of two slots
                    if constexpr (Q8) {
                        p[g][i] = transpose8(pack2<true>(x[t][g][2 * i], x[t][g][2 * i + 1]));
                    } else {
                        split2<F16>(x[t][g][2 * i], x[t][g][2 * i + 1], &p[g][i], &rest[g][i]);
                        p[g][i] = transpose8(p[g][i]);
                        rest[g][i] = transpose8(rest[g][i]);
                    }
                }
            if constexpr (Q8) {
                // slots 0-7 and 8-15 of two 16-wide pieces; a register holds two adjacent columns
                // of two slots
                const int row = 16 * t + (lane & 7) + (mat & 1) * 8;
#pragma unroll
                for (int c = 0; c < KS; c += 2) {
                    uint32_t r[4];
                    ldsm_x4_t(r, vs_s + row * S::RB + swz(row, c + (mat >> 1)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t lo = __byte_perm(r[2 * i], 0, 0x3120), hi = __byte_perm(r[2 * i + 1], 0, 0x3120);
                        const uint32_t a0 = e4m3_halves(lo), a1 = e4m3_halves(lo >> 16);
                        const uint32_t a2 = e4m3_halves(hi), a3 = e4m3_halves(hi >> 16);
#pragma unroll
                        for (int g = 0; g < NG; ++g) mma16816<true>(o[c + i][g], a0, a1, a2, a3, p[g]);
                    }
                }
            } else {
                const int row = 16 * t + (lane & 7) + (mat >> 1) * 8;
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    uint32_t r[4];
                    ldsm_x4_t(r, vs_s + row * S::RB + swz(row, 2 * c + (mat & 1)));
#pragma unroll
                    for (int g = 0; g < NG; ++g) mma16816<F16>(o[c][g], r[0], r[1], r[2], r[3], p[g]);
#pragma unroll
                    for (int g = 0; g < NG; ++g) mma16816<F16>(o[c][g], r[0], r[1], r[2], r[3], rest[g]);
                }
            }
        }
    }

    // The lanes' sums become the warp's; the output relative to m.
    __device__ __forceinline__ void total() {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[g][u] += __shfl_xor_sync(0xffffffffu, l[g][u], d);
                if constexpr (Q8) {
                    const float f = mv[g][u] == -INFINITY ? 0.f : exp2f(mv[g][u] - m[g][u]);
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        o[c][g][u] *= f;
                        o[c][g][2 + u] *= f;
                    }
                }
            }
    }

    // Writes the finished unit (slot < 0), or its part.
    __device__ __forceinline__ void write(int slot) {
        const int row = lane >> 2, q = lane & 3;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int head = 8 * g + 2 * q + u;
                if (head >= rows) continue;
                const float sum = l[g][u], top = m[g][u];
                if (slot >= 0) {
                    const int64_t at = int64_t(slot) * a.part_rows + head;
                    float *to = a.part + at * a.part_pitch;
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        to[col_of(c, row, 0)] = o[c][g][u];
                        to[col_of(c, row, 1)] = o[c][g][2 + u];
                    }
                    if (row == 0) a.part_ml[at] = make_float2(top, sum);
                } else {
                    const float f = sum == 0.f ? 0.f : 1.f / sum;
                    uint16_t *to = a.out + b * a.ost[0] + (q0 + head) * a.ost[1];
#pragma unroll
                    for (int c = 0; c < KS; ++c)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int col = col_of(c, row, i);
                            if (col < a.c.dim) to[col] = static_cast<uint16_t>(pack2<F16>(o[c][g][2 * i + u] * f, 0.f));
                        }
                    if (row == 0) write_lse(q0 + head, top, sum);
                }
            }
    }

    __device__ __forceinline__ float write_lse(int hq, float top, float sum) const {
        const float lse = log_sum<F16>(top, sum);
        if (a.lse) a.lse[b * a.lse_stride + hq] = lse * kLn2;
        if (a.logits) a.lse2[int64_t(b) * a.q_heads + hq] = lse;
        return lse;
    }
};

// One run a warp.
template <int DP, int KV, int NG, bool VEC>
__global__ void __launch_bounds__(kAtThreads, kAtBlocks) k_attend(const __grid_constant__ AttendArgs a) {
    using A = Attend<DP, KV, NG, VEC, kAtStages>;
    using S = typename A::S;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t seen_bits[kAtWarps * S::ST];
    __shared__ long long warp_sums[kAtWarps], upto[kAtThreads];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int units = a.c.heads * a.row_blocks;
    start_after_prior();

    // the steps up to the sequences of each thread: thread t stands for `per`
    // of them
    const int per = (a.c.n_seqs + kAtThreads - 1) / kAtThreads;
    long long incl = 0;
    for (int b = min(t * per, a.c.n_seqs); b < min(t * per + per, a.c.n_seqs); ++b) {
        int n;
        const int lo = seen_from(a, b, &n);
        incl += (n - lo + S::TOK - 1) / S::TOK;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) {
        if (w < warp) incl += warp_sums[w];
        total += warp_sums[w];
    }
    upto[t] = incl * units;
    total *= units;
    __syncthreads();

    // this warp's run [f0, f1) and the place it starts at
    const long long runs =
        min(static_cast<long long>(gridDim.x) * kAtWarps, (total + kAtMinSteps - 1) / kAtMinSteps);
    const int run = blockIdx.x * kAtWarps + warp;
    if (run >= runs) return;
    const long long f0 = total * run / runs, f1 = total * (run + 1) / runs;
    int owner = 0;  // the thread whose sequences hold f0
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) owner += __popc(__ballot_sync(0xffffffffu, upto[32 * w + lane] <= f0));
    long long base = owner ? upto[owner - 1] : 0;
    Place c{};
    for (c.b = owner * per;; ++c.b) {
        enter_sequence<S::TOK>(a, c);
        const long long size = static_cast<long long>(c.steps) * units;
        if (f0 < base + size) break;
        base += size;
    }
    c.unit = static_cast<int>((f0 - base) / c.steps);
    c.t = static_cast<int>(f0 - base - static_cast<long long>(c.unit) * c.steps);

    A u{a, lane, smem + warp * S::WARP_BYTES, ptx::smem_addr(smem + warp * S::WARP_BYTES), seen_bits + warp * S::ST};
    int left = static_cast<int>(f1 - f0), ahead = left;  // steps to take, and to find pages for
    Place p = c;
    bool found = false;  // a step's pages are at hand
    auto find = [&] {
        found = ahead > 0;
        if (!found) return;
        u.find_pages(p.b, a.row_blocks == 1 ? p.unit : p.unit / a.row_blocks, p.lo + p.t * S::TOK, p.n);
        if (--ahead > 0) next_step<S::TOK>(a, units, p);
    };
    find();
#pragma unroll 1
    for (int i = 0; i < S::ST - 1; ++i) {
        if (found) {
            u.issue(i);
            find();
        }
        ptx::cp_async_commit();
    }
    int stage = 0, fill = S::ST - 1;
    while (left > 0) {
        const int t0 = c.t, t1 = min(c.steps, t0 + left);
        u.begin_unit(c.b, c.unit);
#pragma unroll 1
        for (int k = t0; k < t1; ++k) {
            if (found) {
                u.issue(fill);
                find();
            }
            ptx::cp_async_commit();
            ptx::cp_async_wait<S::ST - 1>();
            __syncwarp();
            u.take(stage, k * S::TOK);
            __syncwarp();
            stage = stage + 1 == S::ST ? 0 : stage + 1;
            fill = fill + 1 == S::ST ? 0 : fill + 1;
        }
        u.total();
        const bool first = t0 == 0, last = t1 == c.steps;
        if (lane == 0) {
            int2 *split = a.split + int64_t(c.b) * units + c.unit;
            if (first) split->x = last ? -1 : run;
            if (last) split->y = run;
        }
        u.write(first && last ? -1 : 2 * run + first);
        left -= t1 - t0;
        if (left > 0) {
            c.t = t1 - 1;
            next_step<S::TOK>(a, units, c);
        }
    }
}

// The weight of a slot from its logit and its row's log sum, both base 2.  A
// slot that is not seen (logit -infinity) has none whatever the sum is: it is
// NaN where a seen slot's logit is, -infinity where nothing is seen.
__device__ __forceinline__ float weight_of(float logit, float lse) {
    return logit == -INFINITY ? 0.f : exp2_fast(logit - lse);
}

// Adds the weights of a unit's slots, seen from c.lo on, to the scores: the
// share of the `t`-th of `threads`.
template <typename Lse>
__device__ __forceinline__ void add_weights(const AttendArgs &a, const Place &c, int h, int q0, int rows, int t,
                                            int threads, Lse &&lse_of) {
    const float *x = a.logits + (int64_t(c.b) * a.q_heads + q0) * a.logit_stride;
    float *to = a.scores + c.b * a.sst[0] + h * a.sst[1] + c.lo;
    const int n = c.n - c.lo;
    for (int i0 = t; i0 < n; i0 += kScorePer * threads) {
        float w[kScorePer], old[kScorePer];
#pragma unroll
        for (int k = 0; k < kScorePer; ++k) {
            w[k] = 0.f;
            old[k] = i0 + k * threads < n ? to[i0 + k * threads] : 0.f;
        }
        for (int g = 0; g < rows; ++g, x += a.logit_stride) {
            const float lse = lse_of(g);
            float y[kScorePer];
#pragma unroll
            for (int k = 0; k < kScorePer; ++k) y[k] = i0 + k * threads < n ? x[i0 + k * threads] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kScorePer; ++k) w[k] += weight_of(y[k], lse);
        }
        x -= rows * a.logit_stride;
#pragma unroll
        for (int k = 0; k < kScorePer; ++k)
            if (i0 + k * threads < n) to[i0 + k * threads] = old[k] + w[k];
    }
}

// One unit a block, or a cluster of blocks, its steps dealt to the warps in
// turn; their results are joined in shared memory, the blocks' through
// distributed shared memory, each block writing a share.  Or (warp_units) one
// unit a warp.
template <int DP, int KV, int NG>
__global__ void __launch_bounds__(kAtThreads) k_attend_unit(const __grid_constant__ AttendArgs a) {
    using A = Attend<DP, KV, NG, true, kUnitStages<DP, KV>>;
    using S = typename A::S;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t seen_bits[kAtWarps * S::ST];
    __shared__ float2 ml[kAtWarps][8 * NG], block_ml[8 * NG];
    __shared__ float lse_of[8 * NG];
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = cluster.num_blocks(), part = cluster.block_rank();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int units = a.c.heads * a.row_blocks;
    start_after_prior();
    Place c{};
    const bool by_warp = unit_by_warp(DP, 8 * NG) && a.warp_units;
    const int at_unit = by_warp ? blockIdx.x * kAtWarps + warp : blockIdx.x / parts;
    if (at_unit >= a.c.n_seqs * units) return;  // warps of no unit, past every barrier
    c.b = at_unit / units;
    c.unit = at_unit - c.b * units;
    enter_sequence<S::TOK>(a, c);
    A u{a, lane, smem + warp * S::WARP_BYTES, ptx::smem_addr(smem + warp * S::WARP_BYTES), seen_bits + warp * S::ST};
    const int h = a.row_blocks == 1 ? c.unit : c.unit / a.row_blocks;
    const int first = by_warp ? 0 : part * kAtWarps + warp, stride = by_warp ? 1 : parts * kAtWarps;
    int ahead = first;
    auto find = [&] {
        if (ahead < c.steps) u.find_pages(c.b, h, c.lo + ahead * S::TOK, c.n);
    };
    auto issue = [&](int stage) {
        if (ahead < c.steps) {
            u.issue(stage);
            ahead += stride;
            find();
        }
        ptx::cp_async_commit();
    };
    find();
#pragma unroll 1
    for (int i = 0; i < S::ST - 1; ++i) issue(i);
    u.begin_unit(c.b, c.unit);
    int stage = 0, fill = S::ST - 1;
#pragma unroll 1
    for (int k = first; k < c.steps; k += stride) {
        issue(fill);
        ptx::cp_async_wait<S::ST - 1>();
        __syncwarp();
        u.take(stage, k * S::TOK);
        __syncwarp();
        stage = stage + 1 == S::ST ? 0 : stage + 1;
        fill = fill + 1 == S::ST ? 0 : fill + 1;
    }
    u.total();
    if (by_warp) {
        u.write(-1);
        if (!a.logits) return;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float lse = log_sum<A::F16>(u.m[g][i], u.l[g][i]);
                if (lane < 4) ml[warp][8 * g + 2 * lane + i].x = lse;
            }
        __syncwarp();
        add_weights(a, c, h, u.q0, u.rows, lane, 32, [&](int g) { return ml[warp][g].x; });
        return;
    }
    float *mine = reinterpret_cast<float *>(u.ring);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int head = 8 * g + 2 * (lane & 3) + i, row = lane >> 2;
            if (row == 0) ml[warp][head] = make_float2(u.m[g][i], u.l[g][i]);
#pragma unroll
            for (int k = 0; k < A::KS; ++k) {
                mine[head * S::OP + A::col_of(k, row, 0)] = u.o[k][g][i];
                mine[head * S::OP + A::col_of(k, row, 1)] = u.o[k][g][2 + i];
            }
        }
    __syncthreads();
    // (m, l, o) of one head and four columns from `n` parts
    auto join = [&](int n, auto &&ml_of, auto &&o_of, float2 *v, float (&y)[4]) {
        float top = -INFINITY, sum = 0.f;
        y[0] = y[1] = y[2] = y[3] = 0.f;
        for (int i = 0; i < n; ++i) top = fmaxf(top, ml_of(i).x);
        const float safe = top == -INFINITY ? 0.f : top;
        for (int i = 0; i < n; ++i) {
            const float2 w = ml_of(i);
            const float f = exp2_fast(w.x - safe);
            const float4 z = o_of(i);
            sum += w.y * f;
            y[0] += z.x * f;
            y[1] += z.y * f;
            y[2] += z.z * f;
            y[3] += z.w * f;
        }
        *v = make_float2(top, sum);
    };
    auto put = [&](int head, int col, float2 v, const float (&y)[4]) {
        const float f = v.y == 0.f ? 0.f : 1.f / v.y;
        uint16_t *to = a.out + c.b * a.ost[0] + (u.q0 + head) * a.ost[1];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < a.c.dim) to[col + i] = static_cast<uint16_t>(pack2<A::F16>(y[i] * f, 0.f));
        if (col == 0) {
            const float lse = u.write_lse(u.q0 + head, v.x, v.y);
            if (parts == 1) lse_of[head] = lse;  // a cluster's blocks form all heads' below
        }
    };
    for (int at = t; at < u.rows * (DP / 4); at += kAtThreads) {
        const int head = at / (DP / 4), col = at % (DP / 4) * 4;
        float2 v;
        float y[4];
        join(kAtWarps, [&](int w) { return ml[w][head]; },
             [&](int w) {
                 return *reinterpret_cast<const float4 *>(smem + w * S::WARP_BYTES + (head * S::OP + col) * 4);
             },
             &v, y);
        if (parts == 1) {
            put(head, col, v, y);
        } else {  // in the place of the first warp's, which only this thread reads
            *reinterpret_cast<float4 *>(smem + (head * S::OP + col) * 4) = make_float4(y[0], y[1], y[2], y[3]);
            if (col == 0) block_ml[head] = v;
        }
    }
    if (parts > 1) {
        cluster.sync();
        for (int at = part * kAtThreads + t; at < u.rows * (DP / 4); at += parts * kAtThreads) {
            const int head = at / (DP / 4), col = at % (DP / 4) * 4;
            float2 v;
            float y[4];
            join(parts, [&](int r) { return cluster.map_shared_rank(block_ml, r)[head]; },
                 [&](int r) {
                     const uint8_t *other = cluster.map_shared_rank(smem, r);
                     return *reinterpret_cast<const float4 *>(other + (head * S::OP + col) * 4);
                 },
                 &v, y);
            put(head, col, v, y);
        }
    }
    if (a.logits) {
        if (parts > 1 && t < u.rows) {  // every block needs every head's
            float top = -INFINITY, sum = 0.f;
            for (int r = 0; r < parts; ++r) top = fmaxf(top, cluster.map_shared_rank(block_ml, r)[t].x);
            for (int r = 0; r < parts; ++r) {
                const float2 v = cluster.map_shared_rank(block_ml, r)[t];
                sum += v.y * exp2_fast(v.x - (top == -INFINITY ? 0.f : top));
            }
            lse_of[t] = log_sum<A::F16>(top, sum);
        }
        __syncthreads();
        add_weights(a, c, h, u.q0, u.rows, part * kAtThreads + t, parts * kAtThreads,
                    [&](int g) { return lse_of[g]; });
    }
    if (parts > 1) cluster.sync();  // no block leaves while another reads its shared memory
}

// One warp instantiation's launches: one block a unit (VEC only), or one run a
// warp.
template <int DP, int KV, int NG, bool VEC>
int launch_attend(const AttendArgs &a, int unit_blocks, int *runs, cudaStream_t cs) {
    using S = AtShape<DP, KV, NG, kAtStages>;
    const int64_t units = int64_t(a.c.n_seqs) * a.c.heads * a.row_blocks;
    int sms, per;
    if constexpr (VEC) {
        if (unit_blocks) {
            constexpr int kBytes = AtShape<DP, KV, NG, kUnitStages<DP, KV>>::SMEM;
            const void *fn = reinterpret_cast<const void *>(&k_attend_unit<DP, KV, NG>);
            if (prepare(fn, kAtThreads, kBytes, kBytes, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
            if (a.warp_units)
                return launch_after(fn, static_cast<unsigned>((units + kAtWarps - 1) / kAtWarps), kAtThreads, kBytes,
                                    cs, &a);
            return launch_after(fn, static_cast<unsigned>(units * unit_blocks), kAtThreads, kBytes, cs, &a,
                                unit_blocks);
        }
    }
    const void *fn = reinterpret_cast<const void *>(&k_attend<DP, KV, NG, VEC>);
    if (prepare(fn, kAtThreads, S::SMEM, S::SMEM, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
    // no more blocks than are resident at once, nor than the steps of full
    // sequences
    const int64_t most = units * ((a.c.cap + S::TOK - 1) / S::TOK);
    const int64_t grid = std::max<int64_t>(
        1, std::min<int64_t>({int64_t(sms) * per, kAtMaxBlocks,
                              (most + kAtMinSteps * kAtWarps - 1) / (kAtMinSteps * kAtWarps)}));
    *runs = static_cast<int>(grid) * kAtWarps;
    return launch_after(fn, static_cast<unsigned>(grid), kAtThreads, S::SMEM, cs, &a);
}

// The main launch for one cache type; `runs` receives the runs of a launch by
// runs.
template <int KV>
int launch_attend_type(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs) {
    auto heads = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        if (a.group <= 8)
            return vec ? launch_attend<DP, KV, 1, true>(a, unit_blocks, runs, cs)
                       : launch_attend<DP, KV, 1, false>(a, unit_blocks, runs, cs);
        return vec ? launch_attend<DP, KV, 2, true>(a, unit_blocks, runs, cs)
                   : launch_attend<DP, KV, 2, false>(a, unit_blocks, runs, cs);
    };
    auto wide_heads = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        return a.group <= 8 ? launch_attend<DP, KV, 1, true>(a, unit_blocks, runs, cs)
                            : launch_attend<DP, KV, 2, true>(a, unit_blocks, runs, cs);
    };
    switch (padded_dim(a.c.dim, vec)) {
        case 64: return heads(std::integral_constant<int, 64>{});
        case 96: return wide_heads(std::integral_constant<int, 96>{});
        case 128: return heads(std::integral_constant<int, 128>{});
        case 192: return wide_heads(std::integral_constant<int, 192>{});
        default: return heads(std::integral_constant<int, 256>{});
    }
}

}  // namespace lc
