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
// The weights' operand is w = fp16(P s c), c a power of two per column: one rounding
// of 2^-11 relative, far below the output's 2^-8, at half the tensor work of a split
// into two numbers.  c starts so that the first 32 keys' largest w is 2^6..2^7 and
// moves (with the running output) only when a w passes 2^15, so products down to
// 2^-21 of the largest keep fp16's full 11 bits and smaller ones an absolute 2^-31
// of the largest.  Likewise m moves only when an x_t passes it by 8.  Both decisions
// are a column's own, so a column's bits do not depend on its neighbours.
//
// Split.  An element is 64 keys at absolute positions, taken by one warp in two
// steps of 32 with a fresh (m, l, c, output); a unit is eight elements (512 keys),
// folded in order of position; units are joined in groups of 16 and then the groups,
// by the last CTA to arrive, in order whoever it is.  So the bits depend on the
// position alone, while the work is spread in one of two ways (launch_attn):
//   wide   an element per warp, a unit per CTA of eight warps: short caches, where
//          there are few units and a call's time is one CTA's latency;
//   deep   a unit per warp, four units per CTA, keys and values through a ring of the
//          warp's own: no barrier until the CTA's end, queries prepared once per 512
//          keys: many units.
// A warp's keys come through cp.async into shared memory that no other warp reads.
#include <cfloat>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "warp_mma.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kStepKeys = 32;                      // two blocks of the cache
constexpr int kStepBytes = 2 * kBlockBytes;        // 4,608
constexpr int kElemKeys = 64;
constexpr int kElemSteps = kElemKeys / kStepKeys;  // 2
constexpr int kElems = 8;                          // elements of a unit
constexpr int kUnit = kElems * kElemKeys;          // 512 keys
constexpr int kWideWarps = kElems;
constexpr int kDeepWarps = 4;                      // units of a CTA
constexpr int kDeepStages = 2;                     // steps of a deep warp's ring
constexpr int kFan = 16;                           // units (then groups of units) joined at a time
constexpr long kDeepUnits = 1000;                  // (unit, KV head) pairs of a call from which units go to single warps
constexpr float kLog2eOverSqrtD = 0.12751743074640502f;
constexpr float kLazy = 8.f;                   // log2
constexpr float kUnset = -FLT_MAX;             // m before the first visible key
constexpr float kTopW = 32768.f;               // w above this moves c
constexpr float kLoCode = 16777216.f;          // codes as fp16 numbers: n 2^-24 in bits 0..3,
constexpr float kHiCode = 1048576.f;           // n 2^-20 in bits 4..7

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 0xff) - 127; }

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

// The same with c = 0 before.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

template <int NT>
struct Query {
    uint32_t b[NT][8][2];  // q' as operands: [word of a key's row x weight of its codes]
    float Q0[NT][2], Q1[NT][2], F[NT][2];
    int pos[NT][2];        // position of the column's row, -1 for a column past the last
};

template <int NT>
struct Elem {
    float m[NT][2], l[NT][2], c[NT][2], za[NT][2][2];  // l and za: this lane's keys only
    float o[NT][8][4];                                 // sums over codes, in units of c and of the codes
};

// A unit's fold of its elements.
template <int NT>
struct Fold {
    float M[NT][2], L[NT][2], Z[NT][2][2];
};

template <int NT>
__device__ __forceinline__ void load_query(Query<NT>& q, const AttnArgs& a, int r0, int G, int h, int c0, int nc,
                                           int pos0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = c0 + nt * 8 + g;
        float x[4][8];
        float amax = 0.f, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // the dims of this lane's words of a key's row
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (nt * 8 + g < nc)
                raw = *reinterpret_cast<const uint4*>(a.q + (long)(r0 + c / G) * a.ldq + (h * G + c % G) * kHeadDim +
                                                      (w & 1) * 64 + 16 * t + (w >> 1) * 8);
            const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[w][2 * i] = lo_f(u[i]);
                x[w][2 * i + 1] = hi_f(u[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(x[w][i]));
                sum[w & 1] += x[w][i];
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
            sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
        }
        const int e = max(-100, min(126, 13 - exponent(amax)));
        const float up = pow2(e), up4 = pow2(e - 4);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            q.b[nt][2 * w][0] = pack_half(x[w][0] * up, x[w][4] * up);
            q.b[nt][2 * w][1] = pack_half(x[w][2] * up, x[w][6] * up);
            q.b[nt][2 * w + 1][0] = pack_half(x[w][1] * up4, x[w][5] * up4);
            q.b[nt][2 * w + 1][1] = pack_half(x[w][3] * up4, x[w][7] * up4);
        }
        const float f = pow2(24 - e) * kLog2eOverSqrtD;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int from = (2 * t + j) * 4;
            q.F[nt][j] = __shfl_sync(0xffffffffu, f, from);
            q.Q0[nt][j] = __shfl_sync(0xffffffffu, sum[0] * kLog2eOverSqrtD, from);
            q.Q1[nt][j] = __shfl_sync(0xffffffffu, sum[1] * kLog2eOverSqrtD, from);
            const int cc = nt * 8 + 2 * t + j;
            q.pos[nt][j] = cc < nc ? pos0 + (c0 + cc) / G : -1;
        }
    }
}

template <int NT>
__device__ __forceinline__ void reset(Elem<NT>& e) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            e.m[nt][j] = kUnset;
            e.l[nt][j] = 0.f;
            e.c[nt][j] = pow2(100);
            e.za[nt][j][0] = e.za[nt][j][1] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) e.o[nt][d][0] = e.o[nt][d][1] = e.o[nt][d][2] = e.o[nt][d][3] = 0.f;
    }
}

// The 32 keys from position k0, whose two blocks are at buf.  EDGE: some column does
// not see all of them; what it does not see takes no part, whatever its bytes.
// FIRST: the element's first step (what e held does not matter).
template <int NT, bool EDGE, bool FIRST>
__device__ __forceinline__ void step(Elem<NT>& e, const Query<NT>& q, const char* buf, int k0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int krow = key_of_row(g);  // rows g and g + 8 of the tiles: keys krow, krow + 8
    const int k_at = krow * kRowBytes + ((t ^ (krow & 2)) << 4);
    // ---- code sums of the scores, a group of dims apart ----
    float acc[2][NT][2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint4 ka = *reinterpret_cast<const uint4*>(buf + b * kBlockBytes + k_at);
        const uint4 kc = *reinterpret_cast<const uint4*>(buf + b * kBlockBytes + k_at + 8 * kRowBytes);
        const uint32_t x[4] = {ka.x, ka.y, ka.z, ka.w}, y[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x8 = x[w] >> 8, y8 = y[w] >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float(&ac)[4] = acc[b][nt][w & 1];
                const uint32_t a0 = x[w] & 0x000f000fu, a1 = y[w] & 0x000f000fu, a2 = x8 & 0x000f000fu,
                               a3 = y8 & 0x000f000fu;
                if (w < 2)
                    mma_f16_first(ac, a0, a1, a2, a3, q.b[nt][2 * w][0], q.b[nt][2 * w][1]);
                else
                    mma_f16(ac, a0, a1, a2, a3, q.b[nt][2 * w][0], q.b[nt][2 * w][1]);
                mma_f16(ac, x[w] & 0x00f000f0u, y[w] & 0x00f000f0u, x8 & 0x00f000f0u, y8 & 0x00f000f0u,
                        q.b[nt][2 * w + 1][0], q.b[nt][2 * w + 1][1]);
            }
        }
    }
    // ---- scores and weights: [block][key half] ----
    const char* meta = buf + kMetaOff + krow * kMetaBytes;
    auto k_meta = [&](int b, int hk) {
        return *reinterpret_cast<const uint2*>(meta + b * kBlockBytes + hk * 8 * kMetaBytes);
    };
    auto v_meta = [&](int b, int hk) {
        return *reinterpret_cast<const uint2*>(meta + kHalfBlock + b * kBlockBytes + hk * 8 * kMetaBytes);
    };
    uint32_t wb[NT][2][2][2];  // weights' operands [block][group][key half]
    // rows of this lane a column does not see
    auto hidden = [&](int nt, int j, int b, int hk) { return EDGE && k0 + 16 * b + 8 * hk + krow > q.pos[nt][j]; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float x[2][2][2], ts[2][2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) {
                const uint2 km = k_meta(b, hk);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ts[b][hk][j] = fmaf(lo_f(km.y), acc[b][nt][1][2 * hk + j], lo_f(km.x) * acc[b][nt][0][2 * hk + j]);
            }
        // x_t of a key, less m if `less`
        auto score = [&](int b, int hk, int j, bool less) {
            const uint2 km = k_meta(b, hk);
            float z = less ? fmaf(hi_f(km.x), q.Q0[nt][j], -e.m[nt][j]) : hi_f(km.x) * q.Q0[nt][j];
            z = fmaf(hi_f(km.y), q.Q1[nt][j], z);
            const float r = fmaf(q.F[nt][j], ts[b][hk][j], z);
            return hidden(nt, j, b, hk) ? -INFINITY : r;
        };
        if (FIRST) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float high = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        x[b][hk][j] = score(b, hk, j, false);
                        high = fmaxf(high, x[b][hk][j]);
                    }
                high = fmaxf(col_max(high), kUnset);  // -inf (nothing seen): unset
                e.m[nt][j] = high;
                float ps = 0.f;
                e.l[nt][j] = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        const uint2 vm = v_meta(b, hk);
                        const float p = ex2(x[b][hk][j] - high);  // <= 1
                        x[b][hk][j] = p;
                        e.l[nt][j] += p;
                        if (!hidden(nt, j, b, hk)) ps = fmaxf(ps, fmaxf(p * lo_f(vm.x), p * lo_f(vm.y)));
                    }
                ps = col_max(ps);
                e.c[nt][j] = pow2(max(-126, min(100, 6 - exponent(ps))));
            }
        } else {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        x[b][hk][j] = score(b, hk, j, true);
                        top = fmaxf(top, x[b][hk][j]);
                    }
            if (__any_sync(0xffffffffu, top > kLazy)) {  // m moves in the columns that a score passes by more
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float raw[2][2], over = -INFINITY, high = -INFINITY;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int hk = 0; hk < 2; ++hk) {
                            raw[b][hk] = score(b, hk, j, false);
                            over = fmaxf(over, x[b][hk][j]);
                            high = fmaxf(high, raw[b][hk]);
                        }
                    over = col_max(over);
                    high = col_max(high);
                    if (over > kLazy) {
                        const float al = ex2(e.m[nt][j] - high);
                        e.m[nt][j] = high;
                        e.l[nt][j] *= al;
                        e.za[nt][j][0] *= al;
                        e.za[nt][j][1] *= al;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            e.o[nt][d][j] *= al;
                            e.o[nt][d][2 + j] *= al;
                        }
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int hk = 0; hk < 2; ++hk) x[b][hk][j] = raw[b][hk] - high;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        x[b][hk][j] = ex2(x[b][hk][j]);
                        e.l[nt][j] += x[b][hk][j];
                    }
        }
        // x holds the weights P; w = P c s, the zeros' sums
        auto weights = [&](int b, int hk, bool zeros) {
            const uint2 vm = v_meta(b, hk);
            float w[2][2];  // [group][column]
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = x[b][hk][j], pc = p * e.c[nt][j];
                const bool out = hidden(nt, j, b, hk);
                if (zeros) {
                    const bool start = FIRST && b == 0 && hk == 0;
                    e.za[nt][j][0] = fmaf(p, out ? 0.f : hi_f(vm.x), start ? 0.f : e.za[nt][j][0]);
                    e.za[nt][j][1] = fmaf(p, out ? 0.f : hi_f(vm.y), start ? 0.f : e.za[nt][j][1]);
                }
                w[0][j] = out ? 0.f : pc * lo_f(vm.x);
                w[1][j] = out ? 0.f : pc * lo_f(vm.y);
            }
            wb[nt][b][0][hk] = pack_half(w[0][0], w[0][1]);
            wb[nt][b][1][hk] = pack_half(w[1][0], w[1][1]);
        };
        uint32_t top2 = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) {
                weights(b, hk, true);
                // w >= 0: fp16 order is the order of the bits
                if (!FIRST) top2 = __vmaxu2(top2, __vmaxu2(wb[nt][b][0][hk], wb[nt][b][1][hk]));
            }
        // 2^15 is 0x7800 (a NaN, above it, comes here too and stays NaN)
        if (!FIRST && __any_sync(0xffffffffu, (top2 & 0xffffu) > 0x7800u || top2 > 0x7800ffffu)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float wt = 0.f, ps = 0.f;  // largest w, and largest P s 2^-20 (which cannot overflow)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        const uint2 vm = v_meta(b, hk);
                        const float p = x[b][hk][j], pc = p * e.c[nt][j];
                        if (!hidden(nt, j, b, hk)) {
                            wt = fmaxf(wt, fmaxf(pc * lo_f(vm.x), pc * lo_f(vm.y)));
                            ps = fmaxf(ps, fmaxf(p * (lo_f(vm.x) * pow2(-20)), p * (lo_f(vm.y) * pow2(-20))));
                        }
                    }
                wt = col_max(wt);
                ps = col_max(ps);
                if (wt > kTopW && ps < INFINITY) {
                    const float nc = pow2(max(-126, min(100, 6 - 20 - exponent(ps))));
                    const float ratio = nc * (1.f / e.c[nt][j]);  // powers of two: exact, or 0
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        e.o[nt][d][j] *= ratio;
                        e.o[nt][d][2 + j] *= ratio;
                    }
                    e.c[nt][j] = nc;
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) weights(b, hk, false);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) wb[nt][b][gr][hk] = wm::movmatrix_t(wb[nt][b][gr][hk]);
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
            uint32_t x0 = __byte_perm(e0, e1, 0x5410), x1 = __byte_perm(e0, e1, 0x7632);
            uint32_t x2 = __byte_perm(e2, e3, 0x5410), x3 = __byte_perm(e2, e3, 0x7632);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&lo)[4] = e.o[nt][gr * 4 + n];
                    float(&hi)[4] = e.o[nt][gr * 4 + n + 1];
                    const uint32_t w0 = wb[nt][b][gr][0], w1 = wb[nt][b][gr][1];
                    if (FIRST && b == 0) {
                        mma_f16_first(lo, x0 & 0x000f000fu, x1 & 0x000f000fu, x2 & 0x000f000fu, x3 & 0x000f000fu, w0, w1);
                        mma_f16_first(hi, x0 & 0x00f000f0u, x1 & 0x00f000f0u, x2 & 0x00f000f0u, x3 & 0x00f000f0u, w0, w1);
                    } else {
                        mma_f16(lo, x0 & 0x000f000fu, x1 & 0x000f000fu, x2 & 0x000f000fu, x3 & 0x000f000fu, w0, w1);
                        mma_f16(hi, x0 & 0x00f000f0u, x1 & 0x00f000f0u, x2 & 0x00f000f0u, x3 & 0x00f000f0u, w0, w1);
                    }
                }
                x0 >>= 8;
                x1 >>= 8;
                x2 >>= 8;
                x3 >>= 8;
            }
        }
    }
}

template <int NT, bool FIRST>
__device__ __forceinline__ void any_step(Elem<NT>& e, const Query<NT>& q, const char* buf, int k0, int p_first) {
    if (k0 + kStepKeys - 1 > p_first)
        step<NT, true, FIRST>(e, q, buf, k0);
    else
        step<NT, false, FIRST>(e, q, buf, k0);
}

// The two blocks of a step from global to shared memory, by one warp.
__device__ __forceinline__ void copy_step(char* dst, const char* src) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < kStepBytes / 512; ++j)
        wm::cp_async16_zfill(dst + (j * 32 + lane) * 16, src + (j * 32 + lane) * 16, true);
    static_assert(kStepBytes % 512 == 0, "whole rounds of 32 lanes");
}

// One element into the fold of (M) of a column: the weights of what is folded so far and of the element.
__device__ __forceinline__ void fold_max(float& M, float m, float& a, float& b) {
    const float n = fmaxf(M, m);
    a = ex2(M - n);
    b = ex2(m - n);
    M = n;
}

__device__ __forceinline__ float4 fold4(float4 O, const float (&o)[4], const float (&a)[2], const float (&b)[2]) {
    return make_float4(fmaf(o[0], b[0], O.x * a[0]), fmaf(o[1], b[1], O.y * a[1]), fmaf(o[2], b[0], O.z * a[0]),
                       fmaf(o[3], b[1], O.w * a[1]));
}

// Tile d's output from its fold: code units, and the zeros' sums of its two columns.
__device__ __forceinline__ float4 finish4(float4 O, int d, const float (&z)[2]) {
    const float k = (d & 1) ? kHiCode : kLoCode;
    return make_float4(fmaf(O.x, k, z[0]), fmaf(O.y, k, z[1]), fmaf(O.z, k, z[0]), fmaf(O.w, k, z[1]));
}

// The last of `n` CTAs that call this for one counter (which returns to 0).
__device__ __forceinline__ bool last_of(unsigned* counter, int n, int* flag) {
    __syncthreads();  // the CTA's partials are written
    if (threadIdx.x == 0) {
        __threadfence();
        *flag = atomicInc(counter, (unsigned)n - 1u) == (unsigned)n - 1u;
        __threadfence();
    }
    __syncthreads();
    return *flag != 0;
}

// Joins n partials (in order) of tile d of a set, by one warp: partial i's maxima and
// sums at pm / pl + i * ts * 8 (eight columns), its output at po + i * ts * 256 float4.
__device__ __forceinline__ void join(const float* pm, const float* pl, const float4* po, int d, int n, int ts,
                                     float (&M)[2], float (&L)[2], float4& O) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    const float2* mp = reinterpret_cast<const float2*>(pm) + t;
    const float2* lp = reinterpret_cast<const float2*>(pl) + t;
    const float4* op = po + d * 32 + lane;
    M[0] = M[1] = kUnset;
    for (int i = 0; i < n; i += kFan) {
        float2 m[kFan];
#pragma unroll
        for (int k = 0; k < kFan; ++k)
            if (i + k < n) m[k] = __ldcg(mp + (size_t)(i + k) * ts * 4);
#pragma unroll
        for (int k = 0; k < kFan; ++k)
            if (i + k < n) {
                M[0] = fmaxf(M[0], m[k].x);
                M[1] = fmaxf(M[1], m[k].y);
            }
    }
    L[0] = L[1] = 0.f;
    O = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kB = 8;
    for (int i = 0; i < n; i += kB) {
        float2 m[kB], l[kB];
        float4 v[kB];
#pragma unroll
        for (int k = 0; k < kB; ++k)
            if (i + k < n) {
                m[k] = __ldcg(mp + (size_t)(i + k) * ts * 4);
                l[k] = __ldcg(lp + (size_t)(i + k) * ts * 4);
                v[k] = __ldcg(op + (size_t)(i + k) * ts * 256);
            }
#pragma unroll
        for (int k = 0; k < kB; ++k)
            if (i + k < n) {
                const float w0 = ex2(m[k].x - M[0]), w1 = ex2(m[k].y - M[1]);
                L[0] = fmaf(l[k].x, w0, L[0]);
                L[1] = fmaf(l[k].y, w1, L[1]);
                O.x = fmaf(v[k].x, w0, O.x);
                O.y = fmaf(v[k].y, w1, O.y);
                O.z = fmaf(v[k].z, w0, O.z);
                O.w = fmaf(v[k].w, w1, O.w);
            }
    }
}

// Tile d's part of the output rows, into shared memory [column][128] bf16.
__device__ __forceinline__ void put_out(bf16* rows, int d, float4 O, const float (&L)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    bf16* o = rows + 2 * t * kHeadDim + 64 * (d >> 2) + 8 * g + (d & 3);
    o[0] = rn(O.x / L[0]);
    o[kHeadDim] = rn(O.y / L[1]);
    o[4] = rn(O.z / L[0]);
    o[kHeadDim + 4] = rn(O.w / L[1]);
}

constexpr int kScalars = 10;  // per lane and tile: m, l, 1/c (two each), zeros' sums (four)

template <int NT, bool DEEP>
struct Smem {
    static constexpr int kWarpsOf = DEEP ? kDeepWarps : kWideWarps;
    static constexpr int kBuf = DEEP ? kDeepStages * kStepBytes + NT * 4096 : kElemSteps * kStepBytes;  // a warp's
    static constexpr int kScalarBytes = DEEP ? 0 : kWarpsOf * NT * kScalars * 32 * 4;
    static constexpr int kOut = NT * 8 * kHeadDim * 2;
    static constexpr int kBytes = kWarpsOf * kBuf + kScalarBytes + kOut;
};
static_assert(Smem<2, false>::kBuf >= 2 * 4096, "a wide warp's output fits its buffer");

// NT tiles of eight columns.
template <int NT, bool DEEP>
__global__ void __launch_bounds__(Smem<NT, DEEP>::kWarpsOf * 32, DEEP ? (NT == 1 ? 4 : 2) : (NT == 1 ? 2 : 1))
    attn_kernel(const __grid_constant__ AttnArgs a) {
    using S = Smem<NT, DEEP>;
    constexpr int W = S::kWarpsOf;
    extern __shared__ __align__(128) char smem[];
    __shared__ int flag;
    const Rows& rm = a.rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int G = a.n_q / rm.n_kv;

    // which (stream, head, columns, unit or four units)
    int s = 0;
    while (s + 1 < rm.n_streams && (int)blockIdx.x >= a.item_start[s + 1]) ++s;
    const int r0 = rm.row_start[s], R = rm.row_start[s + 1] - r0, pos0 = rm.pos0[s];
    const int chunks = (R * G + NT * 8 - 1) / (NT * 8);
    int item = blockIdx.x - a.item_start[s];
    const int chunk = item % chunks;
    item /= chunks;
    const int h = item % rm.n_kv;
    item /= rm.n_kv;
    const int c0 = chunk * NT * 8, nc = min(NT * 8, R * G - c0);  // columns c0 .. c0 + nc - 1 of the stream
    const int p_first = pos0 + c0 / G, p_last = pos0 + (c0 + nc - 1) / G;
    const int nu = (pos0 + R - 1) / kUnit + 1;                    // units of the stream's items
    const int u = DEEP ? item * kDeepWarps + warp : item;         // a warp's (a CTA's) unit
    const int set = (a.set_start[s] + chunk) * rm.n_kv + h;       // this (stream, columns, head)

    char* buf = smem + warp * S::kBuf;
    bf16* rows = reinterpret_cast<bf16*>(smem + S::kBytes - S::kOut);
    const View& kv = rm.kv[s];
    const char* heads = kv.pages + ((size_t)rm.layer * kv.n_pages * rm.n_kv + h) * kTileBytes;
    auto src_of = [&](int page, int k) {  // the step from key k, on a physical page
        return heads + (size_t)page * rm.n_kv * kTileBytes + (k % kPage) / kBlockPos * kBlockBytes;
    };

    Query<NT> q;
    Elem<NT> e;
    float* pm = a.pm + ((size_t)set * a.max_units + u) * NT * 8;
    float* pl = a.pl + ((size_t)set * a.max_units + u) * NT * 8;
    float4* po = reinterpret_cast<float4*>(a.po) + ((size_t)set * a.max_units + u) * NT * 256;
    pdl_wait();

    if (!DEEP) {
        const int k0 = u * kUnit + warp * kElemKeys;
        const int steps = k0 > p_last ? 0 : min(kElemSteps, (p_last - k0) / kStepKeys + 1);
        if (steps) {
            const int page = __ldg(kv.table + k0 / kPage);
            copy_step(buf, src_of(page, k0));
            wm::cp_async_commit();
            if (steps > 1) copy_step(buf + kStepBytes, src_of(page, k0 + kStepKeys));
            wm::cp_async_commit();
        }
        load_query(q, a, r0, G, h, c0, nc, pos0);
        if (steps) {
            wm::cp_async_wait<1>();
            __syncwarp();
            any_step<NT, true>(e, q, buf, k0, p_first);
        } else {
            reset(e);
        }
        if (steps > 1) {
            wm::cp_async_wait<0>();
            __syncwarp();
            any_step<NT, false>(e, q, buf + kStepBytes, k0 + kStepKeys, p_first);
        }
        // ---- fold the elements: every warp puts its own down and takes tile `warp` of all ----
        float* sc = reinterpret_cast<float*>(smem + W * S::kBuf);  // [element][tile][scalar][lane]
        __syncwarp();  // the warp has read its keys
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float4* o = reinterpret_cast<float4*>(buf) + nt * 256 + lane;
#pragma unroll
            for (int d = 0; d < 8; ++d) o[d * 32] = make_float4(e.o[nt][d][0], e.o[nt][d][1], e.o[nt][d][2], e.o[nt][d][3]);
            float* x = sc + (warp * NT + nt) * kScalars * 32 + lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[(0 + j) * 32] = e.m[nt][j];
                x[(2 + j) * 32] = e.l[nt][j];
                x[(4 + j) * 32] = 1.f / e.c[nt][j];
                x[(6 + j) * 32] = e.za[nt][j][0];
                x[(8 + j) * 32] = e.za[nt][j][1];
            }
        }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float M[2] = {kUnset, kUnset}, L[2] = {0.f, 0.f}, Z[2] = {0.f, 0.f};
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float* x = sc + (w * NT + nt) * kScalars * 32 + lane;
                const float4 v = *(reinterpret_cast<const float4*>(smem + w * S::kBuf) + nt * 256 + warp * 32 + lane);
                float al[2], be[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fold_max(M[j], x[(0 + j) * 32], al[j], be[j]);
                    L[j] = fmaf(x[(2 + j) * 32], be[j], L[j] * al[j]);
                    Z[j] = fmaf(x[(warp < 4 ? 6 + j : 8 + j) * 32], be[j], Z[j] * al[j]);
                    be[j] *= x[(4 + j) * 32];
                }
                const float o[4] = {v.x, v.y, v.z, v.w};
                O = fold4(O, o, al, be);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                L[j] = col_sum(L[j]);
                Z[j] = col_sum(Z[j]);
            }
            O = finish4(O, warp, Z);
            if (nu == 1) {
                put_out(rows + nt * 8 * kHeadDim, warp, O, L);
            } else {
                po[nt * 256 + warp * 32 + lane] = O;
                if (warp == 0 && lane < 4) {
                    *reinterpret_cast<float2*>(pm + nt * 8 + 2 * t) = make_float2(M[0], M[1]);
                    *reinterpret_cast<float2*>(pl + nt * 8 + 2 * t) = make_float2(L[0], L[1]);
                }
            }
        }
    } else {
        const int k0 = u * kUnit, k1 = min(k0 + kUnit, p_last + 1);
        const int steps = k1 > k0 ? (k1 - k0 + kStepKeys - 1) / kStepKeys : 0;
        int pages = 0;  // lane i: physical page of the unit's page i
        if (steps && lane < kUnit / kPage && k0 + lane * kPage < k1) pages = __ldg(kv.table + k0 / kPage + lane);
        auto fetch = [&](int i) {
            if (i < steps) {
                const int k = k0 + i * kStepKeys;
                copy_step(buf + (i % kDeepStages) * kStepBytes,
                          src_of(__shfl_sync(0xffffffffu, pages, (k - k0) / kPage), k));
            }
            wm::cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kDeepStages; ++i) fetch(i);
        load_query(q, a, r0, G, h, c0, nc, pos0);
        Fold<NT> f;
        float4* O = reinterpret_cast<float4*>(buf + kDeepStages * kStepBytes) + lane;  // the fold's output [tile][8][lane]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f.M[nt][j] = kUnset;
                f.L[nt][j] = f.Z[nt][j][0] = f.Z[nt][j][1] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) O[(nt * 8 + d) * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        static_assert(kElemSteps == 2 && kDeepStages == 2, "the loop's two steps and stages");
        for (int i = 0; i < steps; i += 2) {
            const int k = k0 + i * kStepKeys;
            wm::cp_async_wait<1>();
            __syncwarp();
            any_step<NT, true>(e, q, buf, k, p_first);
            __syncwarp();  // the stage has been read
            fetch(i + 2);
            if (i + 1 < steps) {
                wm::cp_async_wait<1>();
                __syncwarp();
                any_step<NT, false>(e, q, buf + kStepBytes, k + kStepKeys, p_first);
                __syncwarp();
            }
            fetch(i + 3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float al[2], be[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fold_max(f.M[nt][j], e.m[nt][j], al[j], be[j]);
                    f.L[nt][j] = fmaf(e.l[nt][j], be[j], f.L[nt][j] * al[j]);
                    f.Z[nt][j][0] = fmaf(e.za[nt][j][0], be[j], f.Z[nt][j][0] * al[j]);
                    f.Z[nt][j][1] = fmaf(e.za[nt][j][1], be[j], f.Z[nt][j][1] * al[j]);
                    be[j] *= 1.f / e.c[nt][j];
                }
#pragma unroll
                for (int d = 0; d < 8; ++d) O[(nt * 8 + d) * 32] = fold4(O[(nt * 8 + d) * 32], e.o[nt][d], al, be);
            }
        }
        if (u < nu) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float Z[2][2], L[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    L[j] = col_sum(f.L[nt][j]);
                    Z[0][j] = col_sum(f.Z[nt][j][0]);
                    Z[1][j] = col_sum(f.Z[nt][j][1]);
                }
#pragma unroll
                for (int d = 0; d < 8; ++d) po[(nt * 8 + d) * 32 + lane] = finish4(O[(nt * 8 + d) * 32], d, Z[d >> 2]);
                if (lane < 4) {
                    *reinterpret_cast<float2*>(pm + nt * 8 + 2 * t) = make_float2(f.M[nt][0], f.M[nt][1]);
                    *reinterpret_cast<float2*>(pl + nt * 8 + 2 * t) = make_float2(L[0], L[1]);
                }
            }
        }
    }
    pdl_trigger();

    // ---- join the units: groups of kFan, then the groups ----
    if (DEEP || nu > 1) {
        constexpr int kPer = DEEP ? kDeepWarps : 1;  // units of a CTA (a group is whole CTAs)
        static_assert(kFan % kDeepWarps == 0, "groups of whole CTAs");
        const int groups = (nu + kFan - 1) / kFan;
        const int gi = item * kPer / kFan, gn = min(kFan, nu - gi * kFan);
        unsigned* counters = a.counters + (size_t)set * a.max_counters;
        const int arrive = (gn + kPer - 1) / kPer;
        if (arrive > 1) {
            if (!last_of(counters + 1 + gi, arrive, &flag)) return;
        } else {
            __syncthreads();  // the other warps' partials
        }
        for (int level = 0; level < 2; ++level) {
            const bool final = level == 1 || groups == 1;
            const size_t base = level == 0 ? (size_t)set * a.max_units + gi * kFan : (size_t)set * a.max_groups;
            const float *jm = level == 0 ? a.pm : a.gm, *jl = level == 0 ? a.pl : a.gl;
            const float4* jo = reinterpret_cast<const float4*>(level == 0 ? a.po : a.go);
            for (int i = warp; i < NT * 8; i += W) {
                const int nt = i >> 3, d = i & 7;
                float M[2], L[2];
                float4 O;
                join(jm + (base * NT + nt) * 8, jl + (base * NT + nt) * 8, jo + (base * NT + nt) * 256, d,
                     level == 0 ? gn : groups, NT, M, L, O);
                if (final) {
                    put_out(rows + nt * 8 * kHeadDim, d, O, L);
                } else {
                    const size_t at = ((size_t)set * a.max_groups + gi) * NT + nt;
                    reinterpret_cast<float4*>(a.go)[at * 256 + d * 32 + lane] = O;
                    if (d == 0 && lane < 4) {
                        *reinterpret_cast<float2*>(a.gm + at * 8 + 2 * t) = make_float2(M[0], M[1]);
                        *reinterpret_cast<float2*>(a.gl + at * 8 + 2 * t) = make_float2(L[0], L[1]);
                    }
                }
            }
            if (final) break;
            if (!last_of(counters, groups, &flag)) return;
        }
    }
    // ---- rows of dims, out ----
    __syncthreads();
    for (int i = threadIdx.x; i < nc * 16; i += W * 32) {  // (column, 16 bytes)
        const int c = c0 + i / 16;
        *reinterpret_cast<uint4*>(a.out + (long)(r0 + c / G) * a.ldo + (h * G + c % G) * kHeadDim + i % 16 * 8) =
            *reinterpret_cast<const uint4*>(rows + i / 16 * kHeadDim + i % 16 * 8);
    }
}

template <int NT, bool DEEP>
cudaError_t init_one() {
    return cudaFuncSetAttribute(attn_kernel<NT, DEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<NT, DEEP>::kBytes);
}

}  // namespace

int attn_unit() { return kUnit; }
int attn_fan() { return kFan; }

cudaError_t init_attn() {
    cudaError_t e = init_one<1, false>();
    if (e == cudaSuccess) e = init_one<2, false>();
    if (e == cudaSuccess) e = init_one<1, true>();
    return e;
}

cudaError_t launch_attn(AttnArgs& a, cudaStream_t st, bool pdl) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    const Rows& m = a.rows;
    const int G = a.n_q / m.n_kv;
    // one tile of eight columns where every stream's rows fit it, else two: codes are then unpacked once for 16 columns
    int nt = 1;
    long units = 0;
    for (int s = 0; s < m.n_streams; ++s) {
        const int R = m.row_start[s + 1] - m.row_start[s];
        if (R * G > 8) nt = 2;
        if (R > 0) units += (long)m.n_kv * ((m.pos0[s] + R - 1) / kUnit + 1);
    }
    const bool deep = nt == 1 && units >= kDeepUnits;
    int items = 0, sets = 0;
    for (int s = 0; s < m.n_streams; ++s) {
        const int R = m.row_start[s + 1] - m.row_start[s];
        const int chunks = (R * G + nt * 8 - 1) / (nt * 8);
        a.item_start[s] = items;
        a.set_start[s] = sets;
        sets += chunks;
        if (R > 0) {
            const int nu = (m.pos0[s] + R - 1) / kUnit + 1;
            items += chunks * m.n_kv * (deep ? (nu + kDeepWarps - 1) / kDeepWarps : nu);
        }
    }
    a.item_start[m.n_streams] = items;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)items);
    c.blockDim = dim3((deep ? kDeepWarps : kWideWarps) * 32);
    c.dynamicSmemBytes = deep ? Smem<1, true>::kBytes : nt == 1 ? Smem<1, false>::kBytes : Smem<2, false>::kBytes;
    c.stream = st;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = 1;
    }
    if (deep) return cudaLaunchKernelEx(&c, attn_kernel<1, true>, a);
    return nt == 1 ? cudaLaunchKernelEx(&c, attn_kernel<1, false>, a) : cudaLaunchKernelEx(&c, attn_kernel<2, false>, a);
}

}  // namespace kv4
}  // namespace tfl
