// Attention over the 4-bit cache (layout and what a code stands for: kv4.cuh).
// Per (row, query head) -- a "column" -- at position p, over keys t = 0..p of its
// KV head, with k_t = z + s n per group of 64 dims (unrounded):
//   x_t = log2(e)/sqrt(128) (q . k_t)
//       = F sum_g s_tg (q' . n_tg) + sum_g z_tg Q_g,     Q_g = log2(e)/sqrt(128) sum_{d in g} q_d
//   P_t = 2^(x_t - m),  l = sum P_t
//   out_d = (sum_t P_t s_tg n_td + sum_t P_t z_tg) / l     (g the group of d)
//
// The sums over codes run on the tensor cores (m16n8k16, fp16 in, fp32 out), keys
// and then dims on the 16-row side, eight columns on the 8-wide side.  A code needs
// no conversion: n in the low bits of a 16-bit half is the fp16 number n 2^-24, and
// shifted left by four n 2^-20, so "word & 0x000f000f" is a fragment of two codes
// and the powers of two go into q' and into the end of the unit.  q' is q times a
// power of two that puts its largest number at 2^13..2^14 (exact in fp16 but for
// numbers 2^-26 and less of the largest); scales, zeros, weights, maxima and sums
// are fp32.
//
// The weights' operand is w = fp16(P s c), c a power of two per column and group: one rounding
// of 2^-11 relative, below the output's 2^-8, at half the tensor work of a split into two
// numbers.  The sum over the zeros takes P unrounded, so the error goes with P s n and a dim
// that stands for exact zeros stays exact.  c is set, up or down, so that the largest w of 32 keys is 2^6..2^7:
// at a unit's start, whenever m moves (which makes what came before smaller), and when a w
// passes 2^15; the running output moves with it.  So products P s down to 2^-20 of the group's
// largest keep fp16's full 11 bits and smaller ones an absolute 2^-31 of it.  m moves only
// when an x_t passes it by 8.  Both decisions are a column's own, so a column's bits do not
// depend on its neighbours.
//
// Split.  A unit is some steps of 32 keys of a KV head for up to eight columns, taken by
// one warp with a fresh (m, l, c, output).  A second kernel joins the units: groups of 8,
// then the groups, in order.  A unit's length comes from the row's position and the
// cache's heads, so a row's bits do not depend on what else the call holds or how its
// units are spread: the grid is persistent, each warp takes an equal share of the call's
// work one unit after the other, and meets no other warp.  A warp's keys come by bulk
// copies that one of its lanes asks for, into shared memory that no other warp reads.
//
// What bounds it.  One row over a long cache: after some 4 us (launch, parameters,
// queries, the table, the first keys) the warps take a step in 1.15 us each, 7.3 TB/s
// over all of them, until the cache is read; the join adds 5 us.  131,072 positions of 8
// KV heads, seven query heads each (151 MB): 34 us, 4.4 TB/s on the whole.  Windows and
// batches of short caches: the half-rate pipes that take codes apart and make operands
// of them (some 700 cycles of a scheduler per 32 keys and eight columns, of which the
// tensor pipe has 380), a unit's start and end (1.2 us of a warp: its code comes from
// beyond the first instruction cache) and the partials, 4 KB per unit and eight columns,
// which the join reads back: 16 rows over 4,096 keys 24 us, 16 rows over up to 8,192 each 31 us.
#include <algorithm>
#include <cfloat>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "tma.cuh"
#include "warp_mma.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kStepKeys = 32;                      // two blocks of the cache
constexpr int kStepBytes = 2 * kBlockBytes;        // 4,608
// Steps of a unit, by the position of the row that attends and the cache's heads:
// as long as that leaves every warp of a full grid at most one unit, but not below a
// shortest: more steps mean fewer starts and partials, fewer mean more warps for one short
// cache.  8 KV heads, seven query heads each, graph replays.  Shortest before position 8,192,
// with 3 | 4 | 5 | 6 | 8 steps: one row over 4,096 keys 8.1 | 8.2 | 9.0 | 9.8 | 11.2 us, 16 rows
// over up to 8,192 each 33.9 | 31.4 | 34.0 | 30.3 | 33.8 us, a window of 16 rows over 4,096 26.1 |
// 24.1 | 23.6 | 23.4 | 25.1 us (1 KV head, one row over 4,096: 8.1 | 7.8 | 8.6 | 9.5 | 10.9 us; 64
// of one query each, 16 rows over up to 8,192: 174 | 174 | 173 | 174 | 170 us).  From there on, with
// 6 | 8 | 10 | 12: one row over 9,000 keys 11.4 | 11.7 | 13.1 | 14.6 us, rows over 1 to 32,000 keys
// 47.2 | 45.2 | 42.6 | 42.9 us, a window of 16 rows over 20,000 75.8 | 68.4 | 66.8 | 72.1 us (1 KV
// head, one row over 131,072: 19.3 | 17.1 | 17.8 | 18.3 us).  One row over 131,072 keys of 8 heads with
// 8 steps, two or three units to a warp: 43.9 us, with 18 and one unit: 34.1 us.
constexpr int kSpread = 152 * 12;                  // warps of the full grid
__host__ inline int unit_steps(int pos, int n_kv) {
    const int most = kSpread / n_kv, steps = pos / kStepKeys + 1;
    return std::max(pos < 8192 ? 4 : 8, (steps + most - 1) / most);
}
constexpr int kWarps = 4;                          // of a CTA
// CTAs of an SM and steps of a warp's ring.  168 registers a thread allow three CTAs (four, at
// 128, spill).  16 rows over up to 8,192 keys each with rings of 2 | 3 | 4: 31.4 | 32.7 | 35.8 us,
// with two CTAs and rings of 4 | 6: 38.3 | 39.9 us.
constexpr int kCtas = 3, kStages = 2;
constexpr int kFan = 8;                           // units joined at a time
// Warps of a CTA of the join, on a grid of at most a CTA per SM, or more.  On the larger ones with
// 2 | 4 | 8 | 16: 16 rows over up to 8,192 keys 33.0 | 31.4 | 33.2 | 33.3 us, rows over 1 to 32,000
// 53.7 | 45.2 | 45.5 | 48.6 us, a window of 16 rows over 4,096 24.7 | 24.1 | 23.2 | 23.3 us (groups of 16
// units, 2 | 4 | 16 warps: the first 31.5 | 33.2 | 33.1 us).
constexpr int kJoinWarps = 16, kManyJoinWarps = 4;
constexpr int kGroupBytes = 36 * 16;               // a joined group: 32 float4, eight maxima, eight sums
constexpr int kMaxJoinBytes = (kSpread + kFan - 1) / kFan * kGroupBytes;
constexpr float kLog2eOverSqrtD = 0.12751743074640502f;
constexpr float kLazy = 8.f;                   // log2
constexpr float kUnset = -FLT_MAX;             // m before the first visible key
constexpr float kTopW = 32784.f;               // w above this moves c: those that fp16 rounds to more than 2^15
constexpr float kLoCode = 16777216.f;          // codes as fp16 numbers: n 2^-24 in bits 0..3,
constexpr float kHiCode = 1048576.f;           // n 2^-20 in bits 4..7

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 0xff) - 127; }

// 1 / 2^e for a power of two of -126..126 (0 and 2^127 do not come).
__device__ __forceinline__ float inv_pow2(float p) { return __uint_as_float(0x7f000000u - __float_as_uint(p)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Operands of a word's eight codes (bytes of two): "lo" the low codes of bytes 0 and 2
// (lo[0]) and 1 and 3 (lo[1]), "both" the whole bytes, "hi" = both - lo the high codes,
// 16 n.  The subtraction and the byte selection cost less of the half-rate logic pipe
// than a shift and four masks.
struct Codes {
    uint32_t lo[2], both[2];
};
__device__ __forceinline__ Codes codes(uint32_t x) {
    Codes c;
    c.both[0] = x & 0x00ff00ffu;
    c.both[1] = __byte_perm(x, 0, 0x4341);
    c.lo[0] = x & 0x000f000fu;
    c.lo[1] = c.both[1] & 0x000f000fu;
    return c;
}
__device__ __forceinline__ uint32_t hi_codes(uint32_t both, uint32_t lo) {
    uint32_t h;
    asm("sub.u32 %0, %1, %2;" : "=r"(h) : "r"(both), "r"(lo));
    return h;
}

// Key (0..15) of row r of a step's 16-row tiles.  With this order and the cache's
// exchange of row halves, a quarter warp's 16-byte key loads (rows 2i, 2i+1) and a
// half warp's 8-byte value loads (rows 2t of four lanes) cover all banks once.
__device__ __forceinline__ int key_of_row(int r) { return (r & 8) + ((((r >> 1) & 3) ^ (r & 1)) | ((r & 1) << 2)); }

// Maximum over a column's eight lanes (same lane & 3).
__device__ __forceinline__ float col_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
// Of two numbers, neither below 0: the upper halves of their bits.
__device__ __forceinline__ uint32_t col_max2(float lo, float hi) {
    uint32_t x = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    x = __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float col_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// ---- a warp's state ------------------------------------------------------------------
// Lane (g, t) = (lane / 4, lane % 4) holds, per tile of eight columns, columns 2t and
// 2t + 1; of the output, tile d = 4 gr + n of eight (gr the group of dims): dims
// 64 gr + 8 g + n ([0], [1]: the two columns) and 64 gr + 8 g + 4 + n ([2], [3]).  This is
// the layout of every partial output, in registers, shared and global memory
// ([tile][8][lane] of float4), until the last join writes rows of dims.

struct Query {
    uint32_t b[8][2];  // q' as operands: [word of a key's row x weight of its codes]
    float Q0[2], Q1[2], F[2];
    int pos[2];        // position of the column's row, -1 for a column past the last
};

struct State {
    float m[2], l[2], c[2][2], za[2][2];  // [column], c and za [column][group]; l and za: this lane's keys only
    float o[8][4];  // sums over codes, in units of c and of the codes: tiles 2i the low codes, 2i + 1 whole bytes
};

__device__ __forceinline__ void reset(State& e) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        e.m[j] = kUnset;
        e.l[j] = 0.f;
        e.c[j][0] = e.c[j][1] = pow2(100);
        e.za[j][0] = e.za[j][1] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) e.o[d][0] = e.o[d][1] = e.o[d][2] = e.o[d][3] = 0.f;
}

// The 32 keys from position k0, whose two blocks are at buf.  EDGE: some column does
// not see all of them; what it does not see takes no part, whatever its bytes.
// first: the unit's first step.  (A body of its own for that costs more in
// instruction cache misses than its tests.)
template <bool EDGE>
__device__ __forceinline__ void step(State& e, const Query& q, const char* buf, int k0, bool first) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int krow = key_of_row(g);  // rows g and g + 8 of the tiles: keys krow, krow + 8
    const int k_at = krow * kRowBytes + ((t ^ (krow & 2)) << 4);
    // ---- code sums of the scores, a group of dims apart ----
    float acc[2][2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][0][i] = acc[b][1][i] = 0.f;
        const uint4 ka = *reinterpret_cast<const uint4*>(buf + b * kBlockBytes + k_at);
        const uint4 kc = *reinterpret_cast<const uint4*>(buf + b * kBlockBytes + k_at + 8 * kRowBytes);
        const uint32_t x[4] = {ka.x, ka.y, ka.z, ka.w}, y[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const Codes cx = codes(x[w]), cy = codes(y[w]);
            const uint32_t hx0 = hi_codes(cx.both[0], cx.lo[0]), hx1 = hi_codes(cx.both[1], cx.lo[1]);
            const uint32_t hy0 = hi_codes(cy.both[0], cy.lo[0]), hy1 = hi_codes(cy.both[1], cy.lo[1]);
            mma_f16(acc[b][w & 1], cx.lo[0], cy.lo[0], cx.lo[1], cy.lo[1], q.b[2 * w][0], q.b[2 * w][1]);
            mma_f16(acc[b][w & 1], hx0, hy0, hx1, hy1, q.b[2 * w + 1][0], q.b[2 * w + 1][1]);
        }
    }
    // ---- scores and weights: [block][key half][column] ----
    const char* meta = buf + kMetaOff + krow * kMetaBytes;
    auto k_meta = [&](int b, int hk) {
        return *reinterpret_cast<const uint2*>(meta + b * kBlockBytes + hk * 8 * kMetaBytes);
    };
    auto v_meta = [&](int b, int hk) {
        return *reinterpret_cast<const uint2*>(meta + kHalfBlock + b * kBlockBytes + hk * 8 * kMetaBytes);
    };
    uint32_t wb[2][2][2];  // weights' operands [block][group][key half]
    // rows of this lane a column does not see
    auto hidden = [&](int j, int b, int hk) { return k0 + 16 * b + 8 * hk + krow > q.pos[j]; };
    float p[2][2][2], raw[2][2][2], top[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int hk = 0; hk < 2; ++hk) {
            const uint2 km = k_meta(b, hk);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ts = fmaf(lo_f(km.y), acc[b][1][2 * hk + j], lo_f(km.x) * acc[b][0][2 * hk + j]);
                const float z = fmaf(hi_f(km.y), q.Q1[j], hi_f(km.x) * q.Q0[j]);
                raw[b][hk][j] = fmaf(q.F[j], ts, z);
            }
        }
    if (EDGE) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (hidden(j, b, hk)) raw[b][hk][j] = -INFINITY;
    }
    auto weights = [&](int b, int hk) {  // w = P c s
        const uint2 vm = v_meta(b, hk);
        float w[2][2];  // [group][column]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[0][j] = p[b][hk][j] * e.c[j][0] * lo_f(vm.x);
            w[1][j] = p[b][hk][j] * e.c[j][1] * lo_f(vm.y);
        }
        if (EDGE) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (hidden(j, b, hk)) w[0][j] = w[1][j] = 0.f;
        }
        wb[b][0][hk] = pack_half(w[0][0], w[0][1]);
        wb[b][1][hk] = pack_half(w[1][0], w[1][1]);
    };
#pragma unroll
    for (int j = 0; j < 2; ++j)
        top[j] = fmaxf(fmaxf(raw[0][0][j], raw[0][1][j]), fmaxf(raw[1][0][j], raw[1][1][j]));
    bool move = first;
    if (!first) {
        uint32_t top2 = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) {
#pragma unroll
                for (int j = 0; j < 2; ++j) p[b][hk][j] = ex2(raw[b][hk][j] - e.m[j]);
                weights(b, hk);
                // w >= 0: fp16 order is the order of the bits
                top2 = __vimax3_u16x2(top2, wb[b][0][hk], wb[b][1][hk]);
            }
        // 2^15 is 0x7800 (a NaN, above it, counts too and stays one); w is above it where it was above kTopW
        move = __any_sync(0xffffffffu, top[0] > e.m[0] + kLazy || top[1] > e.m[1] + kLazy ||
                                           (top2 & 0xffffu) > 0x7800u || top2 > 0x7800ffffu);
    }
    // A score passes m by more than 8, or a w passes 2^15: m, c and the running sums move in the
    // columns where it does.  A unit's first step sets them.  Where m moves, the keys before lose
    // weight, and c, which they had set, is chosen anew.
    if (move) {
        // What the output holds, by column: of both groups the upper halves of the largest number (0: nothing yet).
        uint32_t held[2] = {0, 0};
        float to[2][2];  // the output's factors [column][group]
        if (!first) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                held[j] = col_max2(fmaxf(fmaxf(e.o[1][j], e.o[1][2 + j]), fmaxf(e.o[3][j], e.o[3][2 + j])),
                                   fmaxf(fmaxf(e.o[5][j], e.o[5][2 + j]), fmaxf(e.o[7][j], e.o[7][2 + j])));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float high = col_max(top[j]);
            const bool up = high > e.m[j] + kLazy;
            float al = 1.f;
            if (up) {
                al = ex2(e.m[j] - high);
                e.m[j] = high;
                e.l[j] *= al;
                e.za[j][0] *= al;
                e.za[j][1] *= al;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) p[b][hk][j] = ex2(raw[b][hk][j] - e.m[j]);
            float ps[2] = {0.f, 0.f};  // largest P s 2^-20 (which cannot overflow), by group
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) {
                    const uint2 vm = v_meta(b, hk);
                    const float pk = p[b][hk][j] * pow2(-20);
                    if (!EDGE || !hidden(j, b, hk)) {
                        ps[0] = fmaxf(ps[0], pk * lo_f(vm.x));
                        ps[1] = fmaxf(ps[1], pk * lo_f(vm.y));
                    }
                }
            const uint32_t most = col_max2(ps[0], ps[1]);
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                const bool over = __ballot_sync(0xffffffffu, ps[gr] * e.c[j][gr] > kTopW * pow2(-20)) & (0x11111111u << t);
                // In units of ps, what is held is a bound on its largest product, at most 16 times the unit's keys
                // too large.  c follows it only where that is 2^20 times the new products (it is in fp32,
                // and this bounds it too), so the largest product is at 2^6 or above.
                const float kept = (gr ? hi_f(held[j]) : lo_f(held[j])) * al * inv_pow2(e.c[j][gr]);
                const int x = max(exponent(gr ? hi_f(most) : lo_f(most)), exponent(kept) - 20);
                to[j][gr] = al;
                if ((up || over) && x < 128) {  // 128: an infinity, whose output is not finite anyway
                    const float now = pow2(max(-100, min(100, 6 - 20 - x)));
                    to[j][gr] = fminf(al * now * inv_pow2(e.c[j][gr]), FLT_MAX);  // finite where the output is 0
                    e.c[j][gr] = now;
                }
            }
        }
        if (!first) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k) e.o[d][k] *= to[k & 1][d >> 2];
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) weights(b, hk);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int hk = 0; hk < 2; ++hk) {
            const uint2 vm = v_meta(b, hk);
            float z[2][2] = {{hi_f(vm.x), hi_f(vm.y)}, {hi_f(vm.x), hi_f(vm.y)}};  // [column][group]
            if (EDGE) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (hidden(j, b, hk)) z[j][0] = z[j][1] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                e.l[j] += p[b][hk][j];
                e.za[j][0] = fmaf(p[b][hk][j], z[j][0], e.za[j][0]);
                e.za[j][1] = fmaf(p[b][hk][j], z[j][1], e.za[j][1]);
            }
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) wb[b][gr][hk] = wm::movmatrix_t(wb[b][gr][hk]);
        }
    // ---- code sums of the output ----
    const char* vb = buf + kHalfBlock + ((g ^ ((t & 2) << 1)) << 3);
#pragma unroll
    for (int b = 0; b < 2; ++b, vb += kBlockBytes) {
        const uint2 v0 = *reinterpret_cast<const uint2*>(vb + t * kRowBytes);              // row 2t: key t
        const uint2 v1 = *reinterpret_cast<const uint2*>(vb + ((t ^ 1) + 4) * kRowBytes);  // row 2t + 1: key (t ^ 1) + 4
        const uint2 v2 = *reinterpret_cast<const uint2*>(vb + (t + 8) * kRowBytes);
        const uint2 v3 = *reinterpret_cast<const uint2*>(vb + ((t ^ 1) + 12) * kRowBytes);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
            const uint32_t e0 = gr ? v0.y : v0.x, e1 = gr ? v1.y : v1.x, e2 = gr ? v2.y : v2.x, e3 = gr ? v3.y : v3.x;
            const uint32_t x0 = __byte_perm(e0, e1, 0x5410), x1 = __byte_perm(e0, e1, 0x7632);
            const uint32_t x2 = __byte_perm(e2, e3, 0x5410), x3 = __byte_perm(e2, e3, 0x7632);
            const Codes y0 = codes(x0), y1 = codes(x1), y2 = codes(x2), y3 = codes(x3);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma_f16(e.o[gr * 4 + 2 * i], y0.lo[i], y1.lo[i], y2.lo[i], y3.lo[i], wb[b][gr][0], wb[b][gr][1]);
                mma_f16(e.o[gr * 4 + 2 * i + 1], y0.both[i], y1.both[i], y2.both[i], y3.both[i], wb[b][gr][0],
                        wb[b][gr][1]);
            }
        }
    }
}

// The two blocks of a step from global to shared memory, asked for by one lane.
__device__ __forceinline__ void ask_step(char* dst, const char* src, uint64_t* full) {
    mbar_arrive_expect_tx(full, kStepBytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(kStepBytes), "r"(smem_u32(full))
                 : "memory");
}

// A unit's end, in place: l over the column's lanes, o from code units and c to the
// output's own scale, the zeros' sums added.  Of the pairs of tiles, the whole bytes
// less the low codes leave the high ones (with the rounding of both sums: a sixteenth of the low
// codes' comes into the dim above, 2^-24 relative and less).
__device__ __forceinline__ void finish(State& e) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        e.l[j] = col_sum(e.l[j]);
        const float z[2] = {col_sum(e.za[j][0]), col_sum(e.za[j][1])};
        const float inv[2] = {inv_pow2(e.c[j][0]), inv_pow2(e.c[j][1])};  // c >= 2^-100
#pragma unroll
        for (int d = 0; d < 8; d += 2)
#pragma unroll
            for (int k = j; k < 4; k += 2) {
                const float lo = inv[d >> 2] * kLoCode, hi = inv[d >> 2] * kHiCode;
                e.o[d + 1][k] = fmaf(e.o[d + 1][k] - e.o[d][k], hi, z[d >> 2]);
                e.o[d][k] = fmaf(e.o[d][k], lo, z[d >> 2]);
            }
    }
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

__device__ __forceinline__ float4 f4(const float (&o)[4]) { return make_float4(o[0], o[1], o[2], o[3]); }

// What the kernels are told.  A part is a stream's rows whose units have the same length; its
// work is a row of places, pitch_set for a set of (columns, KV head), pitch for a unit.  What a
// warp needs of a part is together, so that it costs few misses of the constant cache.
struct Part {
    const char* heads;             // tile 0 of the layer
    const int* table;
    size_t page_bytes;             // of the layer: n_kv tiles
    unsigned last_page;            // what an entry of the table outside the cache is taken for
    int row0, pos0, rows;
    int unit, nu;                  // steps of a unit, units of a set
    int pitch, pitch_set, set0;    // set0: sets of columns before the part
};
struct Call {
    int n_parts, n_kv, group, group_inv;  // query heads per KV head; 65536 / group, rounded up
    int per_sm, direct, max_units;        // CTAs of an SM; every set has one unit, whose warp writes the output
    int end;                              // places of the call: share for each warp, share_rest over
    unsigned share, share_rest;
    const bf16* q;
    long ldq;
    bf16* out;
    long ldo;
    float *pm, *pl, *po;
    int* status;
    int lose;                             // of a probe: the step that a warp never gets, polls of a wait
    unsigned wait_limit;
    int start[kMaxParts];                 // a part's first place
    Part part[kMaxParts];
};

// c / (query heads per KV head), c below 4,096.
__device__ __forceinline__ int row_of(const Call& a, int c) { return (c * a.group_inv) >> 16; }

// A (part, KV head, columns) set of a call.
struct Set {
    int p, h, c0, nc;      // columns c0 .. c0 + nc - 1 of part p
    int r0, pos0, nu, id;  // the part's first row and position, its units; the set's partials
    int unit, last;        // steps of a unit; position of the columns' last row
    int pitch;
};

// The first unit from place `i` on, in order of part, columns, KV head, unit; `i` becomes
// the place where it starts, or the call's end if there is none.
__device__ __forceinline__ int find(const Call& a, int& i, Set& x) {
    int p = 0;
    while (true) {
        while (p + 1 < a.n_parts && i >= a.start[p + 1]) ++p;
        const Part& q = a.part[p];
        x.p = p;
        x.r0 = q.row0;
        x.pos0 = q.pos0;
        x.unit = q.unit;
        x.nu = q.nu;
        x.pitch = q.pitch;
        const unsigned r = i - a.start[p], sh = r / (unsigned)q.pitch_set, chunk = sh / (unsigned)a.n_kv;
        const int first = a.start[p] + (int)sh * q.pitch_set;
        const int u = (unsigned)(i - first + q.pitch - 1) / (unsigned)q.pitch;
        if (u < x.nu) {
            i = first + u * q.pitch;
            x.h = sh - chunk * a.n_kv;
            x.c0 = chunk * 8;
            x.nc = min(8, q.rows * a.group - x.c0);
            x.id = (q.set0 + chunk) * a.n_kv + x.h;
            x.last = x.pos0 + row_of(a, x.c0 + x.nc - 1);
            return u;
        }
        i = first + q.pitch_set;
        if (i >= a.end) return 0;
    }
}

__device__ __forceinline__ size_t partial(const Call& a, const Set& x, int u) {
    return (size_t)x.id * a.max_units + u;
}

// The queries of a set: asked for (ask_query) before the keys, which they would
// otherwise wait behind, and made operands (load_query) when they are there.  Lane
// (g, t) holds column g's dims of its words of a key's row: 16t..16t+15 and 64+16t..64+16t+15.
struct RawQuery {
    uint4 w[4];
};
__device__ __forceinline__ void ask_query(RawQuery& r, const Call& a, const Set& x) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int c = x.c0 + g, G = a.group;
    const bool in = g < x.nc;
    const bf16* q = a.q + (in ? (long)(x.r0 + row_of(a, c)) * a.ldq + (x.h * G + c - row_of(a, c) * G) * kHeadDim : 0) + 16 * t;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        r.w[w] = in ? *reinterpret_cast<const uint4*>(q + (w & 1) * 64 + (w >> 1) * 8) : make_uint4(0, 0, 0, 0);
}

// q' by the power of two that its largest number asks for; the groups' sums by the
// tensor cores from the same operands (ones, and 16 for the codes' high halves).
__device__ __forceinline__ void load_query(Query& q, const RawQuery& r, const Call& a, const Set& x) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    uint32_t top = 0;  // of the absolute values' bits
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint4 v = r.w[w];
        top = __vimax3_u16x2(top, v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
        top = __vimax3_u16x2(top, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
    }
    uint32_t m = max(top & 0xffffu, top >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = max(-100, min(126, 13 - ((int)(m >> 7) - 127)));
    const float up = pow2(e), up4 = pow2(e - 4);
    float sum[2][4];
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) sum[gr][0] = sum[gr][1] = sum[gr][2] = sum[gr][3] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint4 v = r.w[w];
        q.b[2 * w][0] = pack_half(lo_f(v.x) * up, lo_f(v.z) * up);
        q.b[2 * w][1] = pack_half(lo_f(v.y) * up, lo_f(v.w) * up);
        q.b[2 * w + 1][0] = pack_half(hi_f(v.x) * up4, hi_f(v.z) * up4);
        q.b[2 * w + 1][1] = pack_half(hi_f(v.y) * up4, hi_f(v.w) * up4);
        mma_f16(sum[w & 1], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, q.b[2 * w][0], q.b[2 * w][1]);
        mma_f16(sum[w & 1], 0x4c004c00u, 0x4c004c00u, 0x4c004c00u, 0x4c004c00u, q.b[2 * w + 1][0],
                q.b[2 * w + 1][1]);
    }
    const float f = pow2(24 - e) * kLog2eOverSqrtD;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        q.F[j] = __shfl_sync(0xffffffffu, f, (2 * t + j) * 4);
        q.Q0[j] = sum[0][j] * (q.F[j] * pow2(-24));
        q.Q1[j] = sum[1][j] * (q.F[j] * pow2(-24));
        const int cc = 2 * t + j;
        q.pos[j] = cc < x.nc ? x.pos0 + row_of(a, x.c0 + cc) : -1;
    }
}

// Rows of the output of this lane's two columns of a tile (nullptr past the last column).
struct OutRows {
    bf16* r[2];
};
__device__ __forceinline__ OutRows out_rows(const Call& a, const Set& x) {
    const int G = a.group;
    OutRows o;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = 2 * (threadIdx.x & 3) + j, c = x.c0 + col, row = row_of(a, c);
        o.r[j] = col < x.nc ? a.out + (long)(x.r0 + row) * a.ldo + (x.h * G + c - row * G) * kHeadDim : nullptr;
    }
    return o;
}
// Tile d of them, from its output and the columns' 1 / l.
__device__ __forceinline__ void put_out(const OutRows& o, int d, float4 O, const float (&R)[2]) {
    const int dim = 64 * (d >> 2) + 8 * ((threadIdx.x & 31) >> 2) + (d & 3);
    if (o.r[0]) {
        o.r[0][dim] = rn(O.x * R[0]);
        o.r[0][dim + 4] = rn(O.z * R[0]);
    }
    if (o.r[1]) {
        o.r[1][dim] = rn(O.y * R[1]);
        o.r[1][dim + 4] = rn(O.w * R[1]);
    }
}

// The fetching side of a warp: lane 0, its state in shared memory.  Steps are fetched in
// runs: a unit's steps within a page.  The page of a run is looked up in the cache's table
// when the run before it begins, so that no fetch waits for the table.
struct Fetch {
    const char* next;       // the step to fetch,
    int run, idle;          // steps left of its run; stages that there was no step for
    int page;               // where the table's entry for the run after it arrives:
    int next_run, k, left;  // its steps (0: none), its position, its unit's steps from there on,
    int item, u, nu, unit;  // its unit: place, number, the set's units and their steps,
    int last, pitch;        // the set's last position
    const char* heads;      // tile 0 of its layer and head
    const int* table;
    size_t page_bytes;
    unsigned last_page;
    int asked;              // of a probe: steps asked for
};
__device__ __forceinline__ void ask_word(int* dst, const int* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ unsigned asked_word(const int* dst) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return *reinterpret_cast<const volatile unsigned*>(dst);
}

__device__ __forceinline__ void open_unit(Fetch* f, int v) {
    const int k = v * f->unit * kStepKeys, keys = f->last + 1 - k;
    f->u = v;
    f->k = k;
    // a unit of later rows may lie past the last position of these columns: no steps
    f->left = keys <= 0 ? 0 : min(f->unit, (keys + kStepKeys - 1) / kStepKeys);
}
__device__ __forceinline__ void open_set(const Call& a, Fetch* f, int item, const Set& x, int u) {
    const Part& p = a.part[x.p];
    f->heads = p.heads + x.h * kTileBytes;
    f->table = p.table;
    f->page_bytes = p.page_bytes;
    f->last_page = p.last_page;
    f->item = item;
    f->nu = x.nu;
    f->unit = x.unit;
    f->last = x.last;
    f->pitch = x.pitch;
    open_unit(f, u);
}
// The next run: of the unit, or of the next one with steps before place `end`.  Not inlined:
// a copy in each loop costs more in instruction cache misses than the call.
__device__ __noinline__ void open_run(const Call& a, Fetch* f, int end) {
    while (f->left == 0) {
        int item = f->item + f->pitch;
        if (f->u + 1 < f->nu) {
            if (item >= end) break;
            f->item = item;
            open_unit(f, f->u + 1);
        } else {
            Set x;  // the next set starts no later than a unit would
            item = f->item + 1;
            const int u = item < end ? find(a, item, x) : 0;
            if (item >= end) break;
            open_set(a, f, item, x, u);
        }
    }
    f->next_run = min(f->left, (kPage - f->k % kPage) / kStepKeys);
    if (f->left > 0) ask_word(&f->page, f->table + f->k / kPage);
}

constexpr int kWarpBytes = (kStages * (kStepBytes + 8) + (int)sizeof(Fetch) + 127) / 128 * 128;  // ring, its barriers, Fetch

// PROBE: every warp that has a step number a.lose announces it and does not copy it, so that the wait
// for it runs out, after a.wait_limit polls.
template <bool PROBE>
__global__ void __launch_bounds__(kWarps * 32, kCtas) units_kernel(const __grid_constant__ Call a) {
    extern __shared__ __align__(128) char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a full grid: the warps that a scheduler of an SM gets (CTAs b, b + SMs, ...; the same warp of each) take
    // neighbouring shares, so that their sum differs by at most one unit between schedulers
    const unsigned per = a.per_sm, sms = gridDim.x / per, shares = gridDim.x * kWarps;
    const unsigned share = ((blockIdx.x % sms) * kWarps + warp) * per + blockIdx.x / sms;
    // floor(share * end / shares), in 32 bits
    int i = (int)(share * a.share + share * a.share_rest / shares);
    const int end = (int)((share + 1) * a.share + (share + 1) * a.share_rest / shares);
    char* buf = smem + warp * kWarpBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(buf + kStages * kStepBytes);
    Fetch* f = reinterpret_cast<Fetch*>(full + kStages);
    Set x;
    int u = 0;
    if (i < end) u = find(a, i, x);
    if (i < end && lane == 0) {
        for (int k = 0; k < kStages; ++k) mbar_init(&full[k], 1);
        mbar_init_fence();
        f->run = f->idle = 0;
        if (PROBE) f->asked = 0;
        open_set(a, f, i, x, u);
    }
    pdl_wait();  // memory from here on
    pdl_trigger();
    if (i >= end) return;  // no unit starts in the share

    const unsigned page0 = load_word(a.part[x.p].table + min(u * x.unit * kStepKeys, x.last) / kPage);
    RawQuery raw;
    ask_query(raw, a, x);  // before the keys, which they would wait behind
    int fslot = 0;
    auto wait = [&](int slot, uint32_t phase) { return mbar_wait(&full[slot], phase, a.status, PROBE ? a.wait_limit : kMbarSpinLimit); };
    auto ask = [&](int slot, const char* src) {  // lane 0
        if (PROBE && f->asked++ == a.lose)
            mbar_arrive_expect_tx(&full[slot], kStepBytes);
        else
            ask_step(buf + slot * kStepBytes, src, &full[slot]);
    };
    auto fetch = [&]() {
        if (lane == 0) {
            int run = f->run;
            const char* src = f->next;
            if (run == 0) {
                run = f->next_run;
                if (run > 0) {
                    src = f->heads + min(asked_word(&f->page), f->last_page) * f->page_bytes + f->k % kPage / kBlockPos * kBlockBytes;
                    f->k += run * kStepKeys;
                    f->left -= run;
                    open_run(a, f, end);
                }
            }
            if (run > 0) {
                ask(fslot, src);
                f->next = src + kStepBytes;
                f->run = run - 1;
            } else {
                ++f->idle;
            }
        }
        if (++fslot == kStages) fslot = 0;
    };
    int asked = 0;
    if (lane == 0) {
        if (f->left > 0) {  // the first run, at once
            const int run = min(f->left, (kPage - f->k % kPage) / kStepKeys);
            asked = min(run, kStages);
            const char* src = f->heads + min(page0, f->last_page) * f->page_bytes + f->k % kPage / kBlockPos * kBlockBytes;
            for (int k = 0; k < asked; ++k, src += kStepBytes) ask(k, src);
            f->next = src;
            f->run = run - asked;
            f->k += run * kStepKeys;
            f->left -= run;
        }
        open_run(a, f, end);
    }
    __syncwarp();
    asked = __shfl_sync(0xffffffffu, asked, 0);
    fslot = asked == kStages ? 0 : asked;
#pragma unroll 1
    for (int k = asked; k < kStages; ++k) fetch();
    Query q;
    State e;
    int slot = 0;
    uint32_t phase = 0;
    bool there = true;  // until a wait gives up, which status then says
    bool fresh = true;  // the set's queries are to be made operands
#pragma unroll 1
    while (true) {
        if (fresh) load_query(q, raw, a, x);
        const int p_first = x.pos0 + row_of(a, x.c0), keys = x.unit * kStepKeys;
        const int k0 = u * keys, k1 = min(k0 + keys, x.last + 1);
        reset(e);
        auto steps = [&](auto edge) {
#pragma unroll 1
            for (int k = k0; k < k1; k += kStepKeys) {
                there = there && __all_sync(0xffffffffu, wait(slot, phase));
                if (!there) continue;  // nothing more is asked for
                step<decltype(edge)::value>(e, q, buf + slot * kStepBytes, k, k == k0);
                __syncwarp();  // the stage has been read
                fetch();
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        };
        // one body for all steps of a unit: fetching a second one costs more than it saves
        if (k0 + keys - 1 > p_first)
            steps(Bool<true>());
        else
            steps(Bool<false>());
        finish(e);
        if (a.direct) {
            const OutRows o = out_rows(a, x);
            const float R[2] = {1.f / e.l[0], 1.f / e.l[1]};
#pragma unroll
            for (int d = 0; d < 8; ++d) put_out(o, d, f4(e.o[d]), R);
        } else {
            const size_t at = partial(a, x, u);
#pragma unroll
            for (int d = 0; d < 8; ++d) reinterpret_cast<float4*>(a.po)[at * 256 + d * 32 + lane] = f4(e.o[d]);
            if (lane < 4) {
                *reinterpret_cast<float2*>(a.pm + at * 8 + 2 * lane) = make_float2(e.m[0], e.m[1]);
                *reinterpret_cast<float2*>(a.pl + at * 8 + 2 * lane) = make_float2(e.l[0], e.l[1]);
            }
        }
        if (u + 1 < x.nu) {
            i += x.pitch;
            if (i >= end) break;
            fresh = false;
            raw = RawQuery{};  // or its registers would be held through the unit
            ++u;
        } else {
            if (++i >= end) break;
            fresh = true;
            u = find(a, i, x);
            if (i >= end) break;
            ask_query(raw, a, x);
        }
    }
    if (!there && lane == 0) {  // the copies in flight end before the CTA does, or these waits run out too:
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int k = f->idle; k < kStages; ++k) {  // every stage with a step, from the one that was waited for on
            wait(slot, phase);
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
}

// Joins n <= kFan partials of one tile in order, by one warp.  Partial i's eight maxima
// and sums are at pm, pl + 8 i, this lane's output at po + 256 i; all
// loads are in flight at once.  Lane 8 a + c holds column c of partials a, a + 4, ...
__device__ __forceinline__ void join(const float* pm, const float* pl, const float4* po, int n,
                                     float (&M)[2], float (&L)[2], float4& O) {
    const int lane = threadIdx.x & 31, t = lane & 3, c = lane & 7, a = lane >> 3;
    constexpr int kR = kFan / 4;
    float m[kR], l[kR];
    float4 v[kFan];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const bool in = 4 * r + a < n;
        m[r] = in ? load_l2(pm + (4 * r + a) * 8 + c) : kUnset;
        l[r] = in ? load_l2(pl + (4 * r + a) * 8 + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kFan; ++i) v[i] = load_l2(po + min(i, n - 1) * 256);  // past n: weight 0 below
    float top = m[0];
#pragma unroll
    for (int r = 1; r < kR; ++r) top = fmaxf(top, m[r]);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
#pragma unroll
    for (int r = 0; r < kR; ++r) m[r] = 4 * r + a < n ? ex2(m[r] - top) : 0.f;  // the partial's weight
    L[0] = L[1] = 0.f;
    O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kFan; ++i) {
        const int from = (i & 3) * 8 + 2 * t;
        const float w0 = __shfl_sync(0xffffffffu, m[i >> 2], from), w1 = __shfl_sync(0xffffffffu, m[i >> 2], from + 1);
        L[0] = fmaf(__shfl_sync(0xffffffffu, l[i >> 2], from), w0, L[0]);
        L[1] = fmaf(__shfl_sync(0xffffffffu, l[i >> 2], from + 1), w1, L[1]);
        O.x = fmaf(v[i].x, w0, O.x);
        O.y = fmaf(v[i].y, w1, O.y);
        O.z = fmaf(v[i].z, w0, O.z);
        O.w = fmaf(v[i].w, w1, O.w);
    }
    M[0] = __shfl_sync(0xffffffffu, top, 2 * t);
    M[1] = __shfl_sync(0xffffffffu, top, 2 * t + 1);
}

// One tile (of a set's eight) per CTA: its warps join groups of kFan units, warp 0 the
// groups.  A group's loads are all in flight at once, so the kernel costs about two
// round trips to the L2, however many units.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Call a) {
    extern __shared__ __align__(16) float4 js[];  // [group]: 32 x float4 output, then 8 + 8 maxima and sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int d = blockIdx.x % 8, set = blockIdx.x / 8;
    int p = 0;
    while (p + 1 < a.n_parts && set >= a.part[p + 1].set0 * a.n_kv) ++p;
    Set x;
    int at0 = a.start[p] + (set - a.part[p].set0 * a.n_kv) * a.part[p].pitch_set;
    find(a, at0, x);
    const int groups = (x.nu + kFan - 1) / kFan;
    constexpr int kGroup4 = 36;  // float4 of a group
    pdl_wait();
    float M[2], L[2];
    float4 O;
#pragma unroll 1
    for (int gi = warp; gi < groups; gi += blockDim.x / 32) {
        const size_t at = partial(a, x, gi * kFan);
        join(a.pm + at * 8, a.pl + at * 8, reinterpret_cast<const float4*>(a.po) + at * 256 + d * 32 + lane,
             min(kFan, x.nu - gi * kFan), M, L, O);
        if (groups > 1) {
            js[gi * kGroup4 + lane] = O;
            float2* ml = reinterpret_cast<float2*>(js + gi * kGroup4 + 32);
            if (lane < 4) {
                ml[t] = make_float2(M[0], M[1]);
                ml[4 + t] = make_float2(L[0], L[1]);
            }
        }
    }
    if (groups > 1) {
        __syncthreads();
        if (warp) return;
        M[0] = M[1] = kUnset;
#pragma unroll 4
        for (int gi = 0; gi < groups; ++gi) {
            const float2 m = reinterpret_cast<const float2*>(js + gi * kGroup4 + 32)[t];
            M[0] = fmaxf(M[0], m.x);
            M[1] = fmaxf(M[1], m.y);
        }
        L[0] = L[1] = 0.f;
        O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int gi = 0; gi < groups; ++gi) {
            const float2* ml = reinterpret_cast<const float2*>(js + gi * kGroup4 + 32);
            const float2 m = ml[t], l = ml[4 + t];
            const float4 v = js[gi * kGroup4 + lane];
            const float w0 = ex2(m.x - M[0]), w1 = ex2(m.y - M[1]);
            L[0] = fmaf(l.x, w0, L[0]);
            L[1] = fmaf(l.y, w1, L[1]);
            O.x = fmaf(v.x, w0, O.x);
            O.y = fmaf(v.y, w1, O.y);
            O.z = fmaf(v.z, w0, O.z);
            O.w = fmaf(v.w, w1, O.w);
        }
    } else if (warp) {
        return;
    }
    // Only now: set up earlier, the next kernel's CTAs take the place of joins that have not begun.
    // 16 rows over up to 8,192 keys, call after call: 31.4 us, with a trigger at the top 38.0 (one row
    // over 4,096 keys 8.2 | 7.6, over 131,072 34.1 | 33.0).
    pdl_trigger();
    const float inv[2] = {1.f / L[0], 1.f / L[1]};
    put_out(out_rows(a, x), d, O, inv);
}

cudaLaunchConfig_t cfg(int grid, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr, bool pdl) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = 1;
    }
    return c;
}

template <class K>
cudaError_t allow_smem(K* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

int attn_max_units(int positions, int n_kv) {
    const int steps = (positions + kStepKeys - 1) / kStepKeys;  // short units before 8,192 positions, 256 steps
    return std::max((std::min(steps, 256) + 3) / 4, std::min((steps + 7) / 8, kSpread / n_kv));
}

cudaError_t init_attn() {
    cudaError_t e = allow_smem(units_kernel<false>, kWarps * kWarpBytes);
    if (e == cudaSuccess) e = allow_smem(units_kernel<true>, kWarps * kWarpBytes);
    if (e == cudaSuccess) e = allow_smem(join_kernel, kMaxJoinBytes);
    return e;
}

cudaError_t launch_attn(const AttnArgs& a, int sms, cudaStream_t st, bool pdl) {
    const Rows& m = a.rows;
    if (m.n_rows < 1) return cudaSuccess;
    const int G = a.n_q / m.n_kv;
    Call c;
    c.n_kv = m.n_kv;
    c.group = G;
    c.group_inv = (65536 + G - 1) / G;
    c.max_units = a.max_units;
    c.q = a.q;
    c.ldq = a.ldq;
    c.out = a.out;
    c.ldo = a.ldo;
    c.pm = a.pm;
    c.pl = a.pl;
    c.po = a.po;
    c.status = a.status;
    c.lose = a.lose;
    c.wait_limit = a.wait_limit;
    // A stream whose rows lie on both sides of a change of the unit's length (always at a multiple of 32) is
    // two parts.  The work in places where a unit is its steps and one more (its start and end), a set's last
    // unit as long as it is and two more (the set's queries):
    int n = 0, most = 1, sets = 0, units = 0, places = 0, top_unit = 0, low_unit = 1 << 20;
    int steps[kMaxParts];
    for (int s = 0; s < m.n_streams; ++s) {
        int rows = m.row_start[s + 1] - m.row_start[s], row = m.row_start[s], pos = m.pos0[s];
        while (rows > 0) {
            Part& p = c.part[n];
            p.unit = unit_steps(pos, m.n_kv);
            p.rows = unit_steps(pos + rows - 1, m.n_kv) == p.unit ? rows : (pos + rows - 1) / kStepKeys * kStepKeys - pos;
            p.row0 = row;
            p.pos0 = pos;
            p.heads = m.kv[s].pages + (size_t)m.layer * m.kv[s].n_pages * m.n_kv * kTileBytes;
            p.table = m.kv[s].table;
            p.page_bytes = (size_t)m.n_kv * kTileBytes;
            p.last_page = m.kv[s].n_pages - 1;
            p.set0 = sets;
            steps[n] = (pos + p.rows - 1) / kStepKeys + 1;
            p.nu = (steps[n] + p.unit - 1) / p.unit;
            const int chunks = (p.rows * G + 7) / 8;
            sets += chunks;
            units += chunks * m.n_kv * p.nu;
            places += chunks * m.n_kv * (steps[n] + p.nu + 2);
            most = std::max(most, p.nu);
            top_unit = std::max(top_unit, p.unit);
            low_unit = std::min(low_unit, p.unit);
            rows -= p.rows;
            row += p.rows;
            pos += p.rows;
            ++n;
        }
    }
    c.n_parts = n;
    // As many warps as there are units, one each, or a full grid whose warps share the places; or the units,
    // if all have the same steps and that leaves the warp with the most work less.  By
    // units | by places: 16 rows over up to 8,192 keys 31.4 | 32.4 us, 16 rows of one stream over 4,096 keys,
    // which the rule shares by places, 23.4 | 24.1 us, rows over 1 to 32,000 keys 45.6 | 45.2 us.
    const int full = sms * kCtas, need = (units + kWarps - 1) / kWarps, warps = full * kWarps;
    c.per_sm = need < full ? 1 : kCtas;
    bool count = need <= full;
    if (!count && top_unit == low_unit)
        count = (units + warps - 1) / warps * (top_unit + 1) < (places + warps - 1) / warps + top_unit;
    int at = 0;  // below 2^29: at most 160 sets of columns, 64 heads, 2^15 steps and as many units
    for (int i = 0; i < n; ++i) {
        Part& p = c.part[i];
        p.pitch = count ? 1 : p.unit + 1;
        p.pitch_set = count ? p.nu : steps[i] + p.nu + 2;
        c.start[i] = at;
        at += (p.rows * G + 7) / 8 * m.n_kv * p.pitch_set;
    }
    c.end = at;
    const unsigned shares = (need < full ? need : full) * kWarps;
    c.share = at / shares;
    c.share_rest = at % shares;
    c.direct = most == 1;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t g = cfg(need < full ? need : full, kWarps * 32, kWarps * kWarpBytes, st, attr, pdl);
    const cudaError_t e = a.probe ? cudaLaunchKernelEx(&g, units_kernel<true>, c) : cudaLaunchKernelEx(&g, units_kernel<false>, c);
    if (e != cudaSuccess || c.direct) return e;
    const int groups = (most + kFan - 1) / kFan;
    g = cfg(sets * m.n_kv * 8, std::min(groups, sets * m.n_kv * 8 > sms ? kManyJoinWarps : kJoinWarps) * 32,
            groups > 1 ? groups * kGroupBytes : 0, st, attr, true);
    return cudaLaunchKernelEx(&g, join_kernel, c);
}

}  // namespace kv4
}  // namespace tfl
