// Attention of one new token a sequence over a paged key-value cache
// (lc_cache_attend):
//     x_j = scale * q . k_j,  w = softmax(x),  out = sum_j w_j v_j
// over the slots j that are seen.
//
// Mathematics.  One pass over the keys and values: a warp keeps, for up to 16
// query heads of one key head, the running maximum m of the logits (in base
// 2: x_j log2 e), the sum l of 2^(x_j - m) and the output o of the slots it
// has taken, all in float32, and rescales l and o when m grows.  Parts
// (m, l, o) of one row join as sums weighted by 2^(m - max m).
//
// Both products are matrix instructions of 16 query heads by 8 slots (or 8
// columns of the values) by 16: with 16 query heads or fewer a key head the
// pass does at most 16 operations a byte, so memory bounds it and warp-level
// matrix instructions (mma.sync) are far from their rate; the rows of
// absent heads are zeros.  The weights are rounded to the values' 16-bit type
// for the second product (at most 2^-9 / 2^-12 of each weight, no more than the rounding
// of the output); the sum l takes them unrounded.
//
// Work.  A tile is W steps of TOK slots, a step a warp.  Every (sequence, key
// head, block of 16 query heads) is a unit of ceil(slots / tile) tiles; the tiles of all units,
// laid end to end, are cut into equal runs, one a block, whatever the
// lengths: the blocks find their run from the lengths on the device.  A unit
// inside one run is finished there; one that is cut leaves parts in the
// workspace, which k_attend_join joins in block order, so results do not
// depend on timing.  Each warp streams its own steps through a ring of its
// own in shared memory (cp.async, 16 bytes a lane, rows swizzled for
// ldmatrix), with no barrier between warps inside a unit.
#include <cmath>

#include "cache_common.cuh"

namespace lc {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kAtRows = 16;        // query heads of a unit
constexpr int kAtMaxBlocks = 608;  // of the main kernel; sizes the workspace
constexpr int kJoinThreads = 256;
constexpr int kScoreThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Tiles a block gets at least: below it, the parts' joining costs more than
// further blocks save.
constexpr int kAtMinTiles = 4;

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
    bool bf16;            // of q and out
    // workspace
    float *part;          // [2 blocks][kAtRows][part_pitch]
    float2 *part_ml;      // [2 blocks][kAtRows]
    int2 *split;          // per unit: first and last block of a unit that is cut, first -1 when it is not
    float *lse2;          // [sequence, query head], base 2 (with scores)
    float *logits;        // [sequence, query head, logit_stride], base 2, from the first slot seen (with scores)
    int64_t logit_stride;
    int32_t part_pitch;
};

// Shapes of one instantiation.  DP: head_dim rounded up (64, 128, 256); KV: an
// lc_cache_type.  A step is 8 KiB where the shapes allow, and the ring holds 24 KiB a warp:
// with four warps a block and two blocks an SM (one for 16-bit rows of 512
// bytes), 128 KiB and more are in flight on each SM.
template <int DP, int KV>
struct AtShape {
    static constexpr int EB = KV == LC_CACHE_E4M3 ? 1 : 2;
    static constexpr int RB = DP * EB;                       // bytes of a row
    static constexpr int CH = RB / 16;                       // its 16-byte chunks
    static constexpr int TOK = 8192 / (2 * RB) >= 32 ? 32 : 16;
    static constexpr int STEP = 2 * TOK * RB;                // keys, then values
    static constexpr int ST = STEP <= 4096 ? 6 : 3;          // steps in the ring
    static constexpr int SC = KV == LC_CACHE_E4M3 ? 2 * TOK * 4 : 0;  // scales of a step
    static constexpr int TILE = kAtWarps * TOK;
    static constexpr int WARP_BYTES = ST * (STEP + SC);
    static constexpr int OP = DP + 8;                        // floats between the rows of a warp's output
    static constexpr int SMEM = kAtWarps * WARP_BYTES;
    static_assert(kAtRows * OP * 4 <= WARP_BYTES, "a warp's output is staged in its ring");
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
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Four E4M3 codes (bytes 0..3 of r) as two bfloat16 pairs: even = (0, 2), odd = (1,
// 3).  Sign and magnitude move to bfloat16's places (the same exponent
// layout, three of its seven fraction bits), and one exact product by 2^120
// makes up for the biases, 7 and 127.
__device__ __forceinline__ void e4m3_pairs(uint32_t r, uint32_t &even, uint32_t &odd) {
    const uint32_t e = (r & 0x00800080u) << 8 | (r & 0x007f007fu) << 4;
    const uint32_t o = (r & 0x80008000u) | (r >> 4 & 0x07f007f0u);
    const uint32_t k = 0x7b807b80u;  // 2^120 twice
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(k));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(k));
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp, 0 for -infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The slots [lo, n) that sequence b's query sees (before the mask).
__device__ __forceinline__ int seen_from(const AttendArgs &a, int b, int *n) {
    *n = cache_length(a.c, a.lengths, b, kClassAttend);
    return a.window && a.window < *n ? *n - a.window : 0;
}
__device__ __forceinline__ int tiles_of(const AttendArgs &a, int b, int tile) {
    int n;
    const int lo = seen_from(a, b, &n);
    return (n - lo + tile - 1) / tile;
}

template <int DP, int KV, bool VEC, bool SCORES>
struct Attend {
    using S = AtShape<DP, KV>;
    static constexpr bool F16 = KV == LC_CACHE_F16, Q8 = KV == LC_CACHE_E4M3;
    static constexpr int KS = DP / 16;           // 16-wide pieces of a row
    static constexpr int NT = S::TOK / 8;        // 8-slot pieces of a step

    const AttendArgs &a;
    const int lane, warp;
    uint8_t *ring;        // this warp's
    uint32_t ring_s;
    uint32_t *seen_bits;  // this warp's, one word a stage

    // the unit
    int b, h, rows, q0;   // sequence, key head, query heads, the first of them
    int lo, n;

    uint32_t qa[KS][4];
    float o[DP / 8][4], m[2], l[2];

    // a step's page, read one step ahead of its rows
    int next_page, next_row;
    bool next_seen;

    __device__ __forceinline__ static uint32_t swz(int row, int chunk) {
        return S::RB >= 128 ? (chunk ^ (row & 7)) * 16 : (chunk ^ (row >> 1 & 3)) * 16;
    }

    // columns of the values that fragment column 2 q (+1) of 8-wide piece j stands for
    __device__ __forceinline__ static int col_of(int j, int q, int i) {
        return Q8 ? 16 * (j >> 1) + 4 * q + 2 * i + (j & 1) : 8 * j + 2 * q + i;
    }

    __device__ __forceinline__ uint32_t q_pair(const uint16_t *row, int c0, int c1) const {
        const uint32_t x = c0 < a.c.dim ? row[c0] : 0, y = c1 < a.c.dim ? row[c1] : 0;
        return x | y << 16;
    }

    __device__ __forceinline__ void load_q() {
        const int g = lane >> 2, q = lane & 3;
        const uint16_t *p0 = a.q + b * a.qst[0] + (q0 + min(g, rows - 1)) * a.qst[1];
        const uint16_t *p1 = a.q + b * a.qst[0] + (q0 + min(g + 8, rows - 1)) * a.qst[1];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // 16 columns as the matrix instruction's k = 2q, 2q + 1, 2q + 8, 2q + 9; E4M3 keys come
            // four adjacent columns a lane, pairs (0, 2) and (1, 3)
            const int c = 16 * ks + (Q8 ? 4 * q : 2 * q);
            const int d1 = Q8 ? 2 : 1, e0 = Q8 ? 1 : 8, e1 = Q8 ? 3 : 9;
            qa[ks][0] = g < rows ? q_pair(p0, c, c + d1) : 0;
            qa[ks][1] = g + 8 < rows ? q_pair(p1, c, c + d1) : 0;
            qa[ks][2] = g < rows ? q_pair(p0, c + e0, c + e1) : 0;
            qa[ks][3] = g + 8 < rows ? q_pair(p1, c + e0, c + e1) : 0;
        }
    }

    __device__ __forceinline__ int step_slot(int tile) const { return lo + tile * S::TILE + warp * S::TOK; }

    // Reads the page of this lane's slot of a step.
    __device__ __forceinline__ void find_page(int j0) {
        const int j = j0 + lane;
        next_page = -1;
        next_row = 0;
        next_seen = false;
        if (lane < S::TOK && j < n) {
            const int i = static_cast<int>(fast_div(static_cast<uint32_t>(j), a.c.page_div));
            next_row = j - i * a.c.page;
            next_page = a.c.table[b * a.c.table_stride + i];
            next_seen = !a.mask || a.mask[b * a.mask_stride + j];
        }
    }

    // Starts the copies of the step whose pages find_page read, into `stage`.
    __device__ __forceinline__ void issue(int stage) {
        const bool in_pool = next_page >= 0 && next_page < a.c.n_pages;
        if (next_seen && !in_pool) report_error(LC_ERR_CACHE_INDEX, kClassAttend);
        const bool seen = next_seen && in_pool;
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        int64_t ko = 0, vo = 0;
        if (seen) {
            ko = row_offset(a.c.kst, next_page, h, next_row);
            vo = row_offset(a.c.vst, next_page, h, next_row);
        }
        uint8_t *dst = ring + stage * (S::STEP + S::SC);
        const uint32_t dst_s = ring_s + stage * (S::STEP + S::SC);
        if (lane == 0) seen_bits[stage] = bits;
        if constexpr (Q8)
            if (lane < S::TOK) {
                const float *ks = a.c.ks + (seen ? row_offset(a.c.kss, next_page, h, next_row) : 0);
                const float *vs = a.c.vs + (seen ? row_offset(a.c.vss, next_page, h, next_row) : 0);
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

    // Takes the step in `stage`; its first slot is `j0`.
    __device__ __forceinline__ void take(int stage, int j0) {
        const uint32_t bits = seen_bits[stage];
        if (!SCORES && bits == 0) return;
        const int q = lane & 3, mat = lane >> 3;
        const uint32_t ks_s = ring_s + stage * (S::STEP + S::SC), vs_s = ks_s + S::TOK * S::RB;
        const float *scales = reinterpret_cast<const float *>(ring + stage * (S::STEP + S::SC) + S::STEP);

        float x[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            if constexpr (Q8) {
                const int row = 8 * t + (lane & 7) + (mat & 1) * 8;
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t r[4], e, d;
                    ldsm_x4(r, ks_s + row * S::RB + swz(row, ks + (mat >> 1)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e4m3_pairs(r[i], e, d);
                        mma16816<false>(x[t + (i & 1)], qa[ks + (i >> 1)], e, d);
                    }
                }
            } else {
                const int row = 8 * t + (lane & 7) + (mat >> 1) * 8;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t r[4];
                    ldsm_x4(r, ks_s + row * S::RB + swz(row, 2 * ks + (mat & 1)));
                    mma16816<F16>(x[t], qa[ks], r[0], r[1]);
                    mma16816<F16>(x[t + 1], qa[ks], r[2], r[3]);
                }
            }
        }
        const bool high = rows > 8;  // rows 8 .. 15 hold query heads
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 8 * t + 2 * q + i;
                const float f = Q8 ? a.scale2 * scales[col] : a.scale2;
                const bool on = bits >> col & 1;
                x[t][i] = on ? x[t][i] * f : -INFINITY;
                x[t][i + 2] = on && high ? x[t][i + 2] * f : -INFINITY;
            }
        if constexpr (SCORES) {
            float *to = a.logits + (int64_t(b) * a.q_heads + q0) * a.logit_stride + (j0 - lo);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = (lane >> 2) + 8 * i;
                    if (row < rows)
                        *reinterpret_cast<float2 *>(to + row * a.logit_stride + 8 * t + 2 * q) =
                            make_float2(x[t][2 * i], x[t][2 * i + 1]);
                }
            if (bits == 0) return;
        }
        // running maximum, sum and rescaling of the output
        bool grown = false;
        float keep[2] = {1.f, 1.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i && !high) break;
            float top = x[0][2 * i];
#pragma unroll
            for (int t = 0; t < NT; ++t) top = fmaxf(top, fmaxf(x[t][2 * i], x[t][2 * i + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > m[i]) {
                keep[i] = exp2_fast(m[i] - top);
                m[i] = top;
                grown = true;
            }
            const float safe = m[i] == -INFINITY ? 0.f : m[i];
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    x[t][2 * i + u] = exp2_fast(x[t][2 * i + u] - safe);
                    sum += x[t][2 * i + u];
                }
            l[i] = l[i] * keep[i] + sum;
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) {
                o[j][0] *= keep[0];
                o[j][1] *= keep[0];
                o[j][2] *= keep[1];
                o[j][3] *= keep[1];
            }
        }
        if (!high) {
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][2] = x[t][3] = 0.f;
        }
        if constexpr (Q8) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float s = scales[S::TOK + 8 * t + 2 * q + u];
                    x[t][u] *= s;
                    x[t][2 + u] *= s;
                }
        }
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            const uint32_t p[4] = {pack2<F16>(x[t][0], x[t][1]), pack2<F16>(x[t][2], x[t][3]),
                                   pack2<F16>(x[t + 1][0], x[t + 1][1]), pack2<F16>(x[t + 1][2], x[t + 1][3])};
            const int row = 8 * t + (lane & 7) + (mat & 1) * 8;
#pragma unroll
            for (int c = 0; c < S::CH; c += 2) {
                uint32_t r[4];
                ldsm_x4_t(r, vs_s + row * S::RB + swz(row, c + (mat >> 1)));
                if constexpr (Q8) {
                    uint32_t e0, d0, e1, d1;
                    e4m3_pairs(r[0], e0, d0);
                    e4m3_pairs(r[1], e1, d1);
                    mma16816<false>(o[2 * c], p, e0, e1);
                    mma16816<false>(o[2 * c + 1], p, d0, d1);
                    e4m3_pairs(r[2], e0, d0);
                    e4m3_pairs(r[3], e1, d1);
                    mma16816<false>(o[2 * c + 2], p, e0, e1);
                    mma16816<false>(o[2 * c + 3], p, d0, d1);
                } else {
                    mma16816<F16>(o[c], p, r[0], r[1]);
                    mma16816<F16>(o[c + 1], p, r[2], r[3]);
                }
            }
        }
    }

    // Takes this warp's steps of tiles [t0, t1) of the unit.
    __device__ __forceinline__ void stream(int t0, int t1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        find_page(step_slot(t0));
        int ahead = t0;
#pragma unroll 1
        for (int i = 0; i < S::ST - 1; ++i, ++ahead) {
            if (ahead < t1) {
                issue(i);
                if (ahead + 1 < t1) find_page(step_slot(ahead + 1));
            }
            ptx::cp_async_commit();
        }
        load_q();
        int stage = 0, fill = S::ST - 1;
#pragma unroll 1
        for (int t = t0; t < t1; ++t, ++ahead) {
            if (ahead < t1) {
                issue(fill);
                if (ahead + 1 < t1) find_page(step_slot(ahead + 1));
            }
            ptx::cp_async_commit();
            ptx::cp_async_wait<S::ST - 1>();
            __syncwarp();
            take(stage, step_slot(t));
            __syncwarp();
            stage = stage + 1 == S::ST ? 0 : stage + 1;
            fill = fill + 1 == S::ST ? 0 : fill + 1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
    }

    // Joins the warps' (m, l, o); writes the unit's result, or its part to `slot` (>= 0).
    __device__ __forceinline__ void finish(uint8_t *smem, float2 *ml, int slot) {
        const int g = lane >> 2, q = lane & 3;
        float *mine = reinterpret_cast<float *>(ring);
        if (q == 0) {
            ml[warp * kAtRows + g] = make_float2(m[0], l[0]);
            ml[warp * kAtRows + g + 8] = make_float2(m[1], l[1]);
        }
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mine[g * S::OP + col_of(j, q, i)] = o[j][i];
                mine[(g + 8) * S::OP + col_of(j, q, i)] = o[j][2 + i];
            }
        __syncthreads();
        for (int at = threadIdx.x; at < rows * (DP / 4); at += kAtThreads) {
            const int row = at / (DP / 4), col = at % (DP / 4) * 4;
            float top = -INFINITY, total = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) top = fmaxf(top, ml[w * kAtRows + row].x);
            const float safe = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                const float2 v = ml[w * kAtRows + row];
                const float f = exp2_fast(v.x - safe);
                const float4 z =
                    *reinterpret_cast<const float4 *>(smem + w * S::WARP_BYTES + (row * S::OP + col) * 4);
                total += v.y * f;
                y.x += z.x * f;
                y.y += z.y * f;
                y.z += z.z * f;
                y.w += z.w * f;
            }
            if (slot >= 0) {
                *reinterpret_cast<float4 *>(a.part + (int64_t(slot) * kAtRows + row) * a.part_pitch + col) = y;
                if (col == 0) a.part_ml[slot * kAtRows + row] = make_float2(top, total);
            } else {
                const float f = total == 0.f ? 0.f : 1.f / total;
                const float z[4] = {y.x * f, y.y * f, y.z * f, y.w * f};
                uint16_t *to = a.out + b * a.ost[0] + (q0 + row) * a.ost[1];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < a.c.dim) to[col + i] = static_cast<uint16_t>(pack2<F16>(z[i], 0.f));
                if (col == 0) {
                    const float lse = total == 0.f ? -INFINITY : top + log2f(total);
                    if (a.lse) a.lse[b * a.lse_stride + q0 + row] = lse * kLn2;
                    if (SCORES) a.lse2[int64_t(b) * a.q_heads + q0 + row] = lse;
                }
            }
        }
        __syncthreads();  // the rings are free again
    }
};

template <int DP, int KV, bool VEC, bool SCORES>
__global__ void __launch_bounds__(kAtThreads) k_attend(const __grid_constant__ AttendArgs a) {
    using A = Attend<DP, KV, VEC, SCORES>;
    using S = typename A::S;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 ml[kAtWarps * kAtRows];
    __shared__ uint32_t seen_bits[kAtWarps * S::ST];
    __shared__ long long warp_sums[kAtWarps], run_base;
    __shared__ int run_seq;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int units = a.c.heads * a.row_blocks;

    // this block's run of tiles: thread t stands for `per` sequences
    const int per = (a.c.n_seqs + kAtThreads - 1) / kAtThreads;
    const int s0 = min(t * per, a.c.n_seqs), s1 = min(s0 + per, a.c.n_seqs);
    long long mine = 0;
    for (int b = s0; b < s1; ++b) mine += tiles_of(a, b, S::TILE);
    long long incl = mine;
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
    total *= units;
    const long long blocks = min(static_cast<long long>(gridDim.x), (total + kAtMinTiles - 1) / kAtMinTiles);
    if (blockIdx.x >= blocks) return;
    const long long f0 = total * blockIdx.x / blocks, f1 = total * (blockIdx.x + 1) / blocks;
    long long base = (incl - mine) * units;
    if (f0 >= base && f0 < incl * units) {
        int b = s0;
        for (;; ++b) {
            const long long size = static_cast<long long>(tiles_of(a, b, S::TILE)) * units;
            if (f0 < base + size) break;
            base += size;
        }
        run_seq = b;
        run_base = base;
    }
    __syncthreads();

    A u{a, lane, warp, smem + warp * S::WARP_BYTES, ptx::smem_addr(smem + warp * S::WARP_BYTES),
        seen_bits + warp * S::ST};
    long long f = f0;
    u.b = run_seq;
    u.lo = seen_from(a, u.b, &u.n);
    int tiles = (u.n - u.lo + S::TILE - 1) / S::TILE;
    int unit = static_cast<int>((f - run_base) / tiles);
    int t0 = static_cast<int>(f - run_base - static_cast<long long>(unit) * tiles);
    while (f < f1) {
        if (unit == units) {  // the next sequence that has tiles
            do {
                ++u.b;
                u.lo = seen_from(a, u.b, &u.n);
                tiles = (u.n - u.lo + S::TILE - 1) / S::TILE;
            } while (tiles == 0);
            unit = 0;
        }
        const int t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + (f1 - f)));
        u.h = unit / a.row_blocks;
        const int rb = unit - u.h * a.row_blocks;
        u.q0 = u.h * a.group + rb * kAtRows;
        u.rows = min(a.group - rb * kAtRows, kAtRows);
        u.stream(t0, t1);
        const bool whole = t0 == 0 && t1 == tiles;
        if (t == 0) {
            int2 *split = a.split + int64_t(u.b) * units + unit;
            if (t0 == 0) split->x = whole ? -1 : static_cast<int>(blockIdx.x);
            if (t1 == tiles) split->y = static_cast<int>(blockIdx.x);
        }
        __syncthreads();
        u.finish(smem, ml, whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (t0 == 0));
        f += t1 - t0;
        t0 = 0;
        ++unit;
    }
}

// Joins the parts of a query head whose unit was cut, in block order, and
// writes the zeros of sequences with nothing to see.  A block a (sequence, query head): the parts' maxima
// and sums first, then their outputs, several parts at a time.
template <bool F16>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const __grid_constant__ AttendArgs a) {
    __shared__ float red[kJoinThreads / 32], acc[kJoinThreads * 4];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int b = blockIdx.x / a.q_heads, hq = blockIdx.x - b * a.q_heads;
    const int h = hq / a.group, rb = (hq - h * a.group) / kAtRows, row = (hq - h * a.group) % kAtRows;
    const int units = a.c.heads * a.row_blocks;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint16_t *out = a.out + b * a.ost[0] + hq * a.ost[1];
    int n;
    const int lo = seen_from(a, b, &n);
    if (lo >= n) {
        for (int i = t; i < a.c.dim; i += kJoinThreads) out[i] = 0;
        if (t == 0 && a.lse) a.lse[b * a.lse_stride + hq] = -INFINITY;
        return;
    }
    const int2 split = a.split[int64_t(b) * units + h * a.row_blocks + rb];
    if (split.x < 0) return;
    // the unit's first part is its block's second (it starts there), the others their blocks' first
    const int parts = split.y - split.x + 1;
    auto slot = [&](int i) { return 2 * (split.x + i) + (i == 0); };
    auto reduce = [&](float x, bool is_max) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, x, d);
            x = is_max ? fmaxf(x, y) : x + y;
        }
        __syncthreads();
        if (lane == 0) red[warp] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int w = 1; w < kJoinThreads / 32; ++w) x = is_max ? fmaxf(x, red[w]) : x + red[w];
        return x;
    };
    float top = -INFINITY, total = 0.f;
    for (int i = t; i < parts; i += kJoinThreads) top = fmaxf(top, a.part_ml[slot(i) * kAtRows + row].x);
    top = reduce(top, true);
    const float safe = top == -INFINITY ? 0.f : top;
    for (int i = t; i < parts; i += kJoinThreads) {
        const float2 v = a.part_ml[slot(i) * kAtRows + row];
        total += v.y * exp2_fast(v.x - safe);
    }
    total = reduce(total, false);
    const int quads = a.part_pitch / 4, lanes = kJoinThreads / quads;  // parts read at a time
    const int col = t % quads * 4, first = t / quads;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = first; i < parts; i += lanes) {
        const float f = exp2_fast(a.part_ml[slot(i) * kAtRows + row].x - safe);
        const float4 z = *reinterpret_cast<const float4 *>(
            a.part + (int64_t(slot(i)) * kAtRows + row) * a.part_pitch + col);
        y.x += z.x * f;
        y.y += z.y * f;
        y.z += z.z * f;
        y.w += z.w * f;
    }
    *reinterpret_cast<float4 *>(acc + first * a.part_pitch + col) = y;
    __syncthreads();
    const float f = total == 0.f ? 0.f : 1.f / total;
    for (int i = t; i < a.c.dim; i += kJoinThreads) {
        float s = 0.f;
        for (int k = 0; k < lanes; ++k) s += acc[k * a.part_pitch + i];
        out[i] = static_cast<uint16_t>(pack2<F16>(s * f, 0.f));
    }
    if (t == 0) {
        const float lse = total == 0.f ? -INFINITY : top + log2f(total);
        if (a.lse) a.lse[b * a.lse_stride + hq] = lse * kLn2;
        if (a.logits) a.lse2[int64_t(b) * a.q_heads + hq] = lse;
    }
}

// scores[b, h, j] += sum over the group's query heads of 2^(logit - lse).
__global__ void __launch_bounds__(kScoreThreads) k_attend_scores(const __grid_constant__ AttendArgs a, int chunks) {
    const int unit = blockIdx.x / chunks, chunk = blockIdx.x - unit * chunks;
    const int b = unit / a.c.heads, h = unit - b * a.c.heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int n;
    const int lo = seen_from(a, b, &n);
    const int i = chunk * kScoreThreads + threadIdx.x;
    if (i >= n - lo) return;
    const float *x = a.logits + (int64_t(b) * a.q_heads + h * a.group) * a.logit_stride + i;
    const float *lse2 = a.lse2 + int64_t(b) * a.q_heads + h * a.group;
    float w = 0.f;
#pragma unroll 4
    for (int g = 0; g < a.group; ++g) {
        const float z = lse2[g];
        const float e = exp2_fast(x[g * a.logit_stride] - z);
        w += z == -INFINITY ? 0.f : e;
    }
    a.scores[b * a.sst[0] + h * a.sst[1] + lo + i] += w;
}

cudaError_t take_error_attend(unsigned long long *v) { return take_module_error(v); }

namespace {

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Workspace of a call: offsets of its pieces, and their end.
struct AttendSpace {
    int64_t part, ml, split, lse2, logits, end, logit_stride;
};

bool attend_space(const CacheArgs &c, int q_heads, bool scores, AttendSpace *s) {
    const int64_t slots = 2 * kAtMaxBlocks * kAtRows;
    const int64_t group = q_heads / c.heads, units = c.heads * ((group + kAtRows - 1) / kAtRows);
    int64_t heads, logits;
    s->part = 0;
    s->ml = s->part + slots * padded_dim(c.dim) * 4;
    s->split = s->ml + slots * 8;
    s->lse2 = round256(s->split + c.n_seqs * units * 8);
    heads = int64_t(c.n_seqs) * q_heads;
    s->logits = round256(s->lse2 + (scores ? heads * 4 : 0));
    // the last tile's steps write whole steps: up to a tile past the capacity
    s->logit_stride = (int64_t(c.cap) + 3) / 4 * 4 + 32 * kAtWarps;
    if (!mul_ok_ext(heads, s->logit_stride * 4, &logits)) return false;
    return add_ok_ext(s->logits, scores ? logits : 0, &s->end) && s->end < int64_t(1) << 60;
}

cudaError_t launch_after(const void *fn, unsigned grid, unsigned threads, cudaStream_t cs, void **args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = cs;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int DP, int KV, bool VEC, bool SCORES>
int launch_attend(AttendArgs &a, cudaStream_t cs) {
    using S = AtShape<DP, KV>;
    const void *fn = reinterpret_cast<const void *>(&k_attend<DP, KV, VEC, SCORES>);
    int sms, per;
    if (prepare(fn, kAtThreads, S::SMEM, S::SMEM, &sms, &per) != cudaSuccess) return LC_ERR_CUDA;
    // no more blocks than are resident at once, nor than the tiles of full sequences
    const int64_t most = int64_t(a.c.n_seqs) * a.c.heads * a.row_blocks * ((a.c.cap + S::TILE - 1) / S::TILE);
    const int64_t grid = std::max<int64_t>(
        1, std::min<int64_t>({int64_t(sms) * per, kAtMaxBlocks, (most + kAtMinTiles - 1) / kAtMinTiles}));
    k_attend<DP, KV, VEC, SCORES><<<static_cast<unsigned>(grid), kAtThreads, S::SMEM, cs>>>(a);
    void *args[] = {&a, nullptr};
    const void *join = KV == LC_CACHE_F16 ? reinterpret_cast<const void *>(&k_attend_join<true>)
                                          : reinterpret_cast<const void *>(&k_attend_join<false>);
    if (launch_after(join, static_cast<unsigned>(a.c.n_seqs * a.q_heads), kJoinThreads, cs, args) != cudaSuccess)
        return LC_ERR_CUDA;
    if (SCORES) {
        int chunks = (a.c.cap + kScoreThreads - 1) / kScoreThreads;
        args[1] = &chunks;
        const void *sc = reinterpret_cast<const void *>(&k_attend_scores);
        if (launch_after(sc, static_cast<unsigned>(a.c.n_seqs * a.c.heads * chunks), kScoreThreads, cs, args) !=
            cudaSuccess)
            return LC_ERR_CUDA;
    }
    return finish_launch();
}

template <int DP, int KV>
int launch_attend_as(AttendArgs &a, bool vec, cudaStream_t cs) {
    if (vec) return a.scores ? launch_attend<DP, KV, true, true>(a, cs) : launch_attend<DP, KV, true, false>(a, cs);
    return a.scores ? launch_attend<DP, KV, false, true>(a, cs) : launch_attend<DP, KV, false, false>(a, cs);
}

template <int KV>
int launch_attend_dim(AttendArgs &a, bool vec, cudaStream_t cs) {
    switch (padded_dim(a.c.dim)) {
        case 64: return launch_attend_as<64, KV>(a, vec, cs);
        case 128: return launch_attend_as<128, KV>(a, vec, cs);
        default: return launch_attend_as<256, KV>(a, vec, cs);
    }
}

}  // namespace

}  // namespace lc

extern "C" int64_t lc_cache_attend_workspace(const lc_paged_cache *cache, int32_t n_q_heads, int32_t with_scores) {
    lc::CacheArgs c;
    lc::AttendSpace s;
    if (lc::check_cache(cache, false, &c) || n_q_heads < 1 || n_q_heads % c.heads ||
        !lc::attend_space(c, n_q_heads, with_scores != 0, &s))
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
        (q->scores && !rows_apart(2, kext, q->scores_stride, std::max(a.c.cap, 1))))
        return LC_ERR_NOT_INJECTIVE;
    AttendSpace space;
    const int64_t chunks = (int64_t(a.c.cap) + kScoreThreads - 1) / kScoreThreads;
    if (!attend_space(a.c, q->n_q_heads, q->scores != nullptr, &space) || qext[0] * qext[1] > 0x7fffffff ||
        (q->scores && chunks && kext[0] * kext[1] > 0x7fffffff / chunks))
        return LC_ERR_OVERFLOW;
    if (!q->workspace) return LC_ERR_NULL;
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
    a.bf16 = q->type == LC_CACHE_BF16;
    uint8_t *ws = static_cast<uint8_t *>(q->workspace);
    a.part = reinterpret_cast<float *>(ws + space.part);
    a.part_ml = reinterpret_cast<float2 *>(ws + space.ml);
    a.split = reinterpret_cast<int2 *>(ws + space.split);
    a.lse2 = reinterpret_cast<float *>(ws + space.lse2);
    a.logits = a.scores ? reinterpret_cast<float *>(ws + space.logits) : nullptr;
    a.logit_stride = space.logit_stride;
    a.part_pitch = padded_dim(a.c.dim);
    const int eb = cache_elem_bytes(cache->type);
    const int64_t pool[3] = {cache->n_pages, cache->n_kv_heads, cache->page_size};
    const bool vec = a.c.dim * eb % 16 == 0 && rows_aligned(cache->k, 3, pool, cache->k_stride, eb, 16) &&
                     rows_aligned(cache->v, 3, pool, cache->v_stride, eb, 16);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    switch (cache->type) {
        case LC_CACHE_BF16: return launch_attend_dim<LC_CACHE_BF16>(a, vec, cs);
        case LC_CACHE_F16: return launch_attend_dim<LC_CACHE_F16>(a, vec, cs);
        default: return launch_attend_dim<LC_CACHE_E4M3>(a, vec, cs);
    }
}
