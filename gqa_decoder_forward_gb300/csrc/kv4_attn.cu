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
// The weights' operand is w = fp16(P s c), c a power of two per column and warp:
// one rounding of 2^-11 relative, far below the output's 2^-8, at half the tensor
// work of a split into two numbers.  c starts so that the first keys' largest w is
// 2^6..2^7 and moves (with the running output) only when a w passes 2^15, so
// products down to 2^-21 of the largest keep fp16's full 11 bits and smaller ones an
// absolute 2^-31 of the largest.  Likewise m moves only when an x_t passes it by 8.
// Both decisions are a column's own, so a column's bits do not depend on its
// neighbours.
//
// Split: a unit is 512 keys of one KV head at absolute positions; each of a CTA's
// four warps takes one page of it (128 keys) alone, in steps of 16 keys (a block of
// the cache: 2,304 contiguous bytes), from its own shared-memory buffer, which
// cp.async fills before the first step: no barrier until the end of the unit, where
// the warps' (m, l, O) are joined in warp order.  Units are joined by the last CTA
// to finish: groups of 16 units first, then the groups (in order of position,
// whoever does it), so one launch does it all and the bits depend on the position
// alone.
#include <cfloat>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "warp_mma.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kWarps = 4;
constexpr int kWarpKeys = kPage;               // keys of a warp: one page
constexpr int kUnit = kWarps * kWarpKeys;      // keys of a CTA
constexpr int kSteps = kWarpKeys / kBlockPos;  // steps of 16 keys
constexpr int kThreads = kWarps * 32;
constexpr int kSmem = kWarps * kTileBytes;
constexpr int kFan = 16;                       // units (then groups of units) joined at a time
constexpr float kLog2eOverSqrtD = 0.12751743074640502f;
constexpr float kLazy = 8.f;                   // log2
constexpr float kUnset = -FLT_MAX;             // m before the first visible key
constexpr float kTopW = 32768.f;               // w above this moves c
constexpr float kLoCode = 16777216.f;          // codes as fp16 numbers: n 2^-24 in bits 0..3,
constexpr float kHiCode = 1048576.f;           // n 2^-20 in bits 4..7
constexpr int kCoStride = kHeadDim + 4;        // floats of a column's output in the warps' join

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

__device__ __forceinline__ void wait_step(int i) {
    using wm::cp_async_wait;
    switch (i) {
        case 0: cp_async_wait<7>(); break;
        case 1: cp_async_wait<6>(); break;
        case 2: cp_async_wait<5>(); break;
        case 3: cp_async_wait<4>(); break;
        case 4: cp_async_wait<3>(); break;
        case 5: cp_async_wait<2>(); break;
        case 6: cp_async_wait<1>(); break;
        default: cp_async_wait<0>(); break;
    }
    __syncwarp();
}
static_assert(kSteps == 8, "wait_step");

// Joins n partials of one column, in order, by one warp: lane i holds dims 4i..4i+3.
// The partials' maxima, sums and outputs are at pm[i], pl[i], po[128 i].
__device__ __forceinline__ void join(const float* pm, const float* pl, const float* po, int n, float& M, float& L,
                                     float4& O) {
    const int lane = threadIdx.x & 31;
    M = kUnset;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(pm + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    L = 0.f;
    O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < n; b += kFan) {
        const int k = min(kFan, n - b);
        float w = 0.f, l = 0.f;
        if (lane < k) {
            w = exp2f(__ldcg(pm + b + lane) - M);
            l = __ldcg(pl + b + lane);
        }
        float4 v[kFan];
#pragma unroll
        for (int i = 0; i < kFan; ++i)
            if (i < k) v[i] = __ldcg(reinterpret_cast<const float4*>(po + (size_t)(b + i) * kHeadDim) + lane);
#pragma unroll
        for (int i = 0; i < kFan; ++i)
            if (i < k) {
                const float wi = __shfl_sync(0xffffffffu, w, i);
                L = fmaf(__shfl_sync(0xffffffffu, l, i), wi, L);
                O.x = fmaf(v[i].x, wi, O.x);
                O.y = fmaf(v[i].y, wi, O.y);
                O.z = fmaf(v[i].z, wi, O.z);
                O.w = fmaf(v[i].w, wi, O.w);
            }
    }
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

// NT tiles of eight columns.
template <int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) attn_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(128) char smem[];
    __shared__ float sm_m[kWarps][NT * 8], sm_l[kWarps][NT * 8];
    __shared__ int flag;
    const Rows& rm = a.rows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.n_q / rm.n_kv;

    // which (stream, head, columns, unit)
    int s = 0;
    while (s + 1 < rm.n_streams && (int)blockIdx.x >= a.item_start[s + 1]) ++s;
    const int r0 = rm.row_start[s], R = rm.row_start[s + 1] - r0, pos0 = rm.pos0[s];
    const int chunks = (R * G + NT * 8 - 1) / (NT * 8);
    int item = blockIdx.x - a.item_start[s];
    const int chunk = item % chunks;
    item /= chunks;
    const int h = item % rm.n_kv, u = item / rm.n_kv;
    const int c0 = chunk * NT * 8, nc = min(NT * 8, R * G - c0);  // columns c0 .. c0 + nc - 1 of the stream
    const int p_first = pos0 + c0 / G, p_last = pos0 + (c0 + nc - 1) / G;
    const int nu_all = (pos0 + R - 1) / kUnit + 1;                // units of the stream's items
    const int k0 = u * kUnit + warp * kWarpKeys;
    const int nsteps = k0 > p_last ? 0 : min(kSteps, (p_last - k0) / kBlockPos + 1);

    pdl_wait();
    char* buf = smem + warp * kTileBytes;
    {
        const char* src = nsteps ? tile(rm.kv[s], rm.layer, rm.n_kv, k0, h) : nullptr;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i < nsteps) {
#pragma unroll
                for (int j = 0; j < 5; ++j) {
                    const int at = i * kBlockBytes + (j * 32 + lane) * 16;
                    if (j < 4 || lane < 16) wm::cp_async16_zfill(buf + at, src + at, true);
                }
            }
            wm::cp_async_commit();
        }
    }

    // queries: lane (g, t) holds column g's dims 16t..16t+15 and 64+16t..64+16t+15 as key-side operands
    uint32_t qb[NT][8][2];
    float Q0[NT][2], Q1[NT][2], F[NT][2];
    int cpos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = c0 + nt * 8 + g;
        float q[4][8];
        float amax = 0.f, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (nt * 8 + g < nc)
                raw = *reinterpret_cast<const uint4*>(a.q + (long)(r0 + c / G) * a.ldq + (h * G + c % G) * kHeadDim +
                                                      (w & 1) * 64 + 16 * t + (w >> 1) * 8);
            const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[w][2 * i] = lo_f(x[i]);
                q[w][2 * i + 1] = hi_f(x[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(q[w][i]));
                sum[w & 1] += q[w][i];
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
            qb[nt][2 * w][0] = pack_half(q[w][0] * up, q[w][4] * up);
            qb[nt][2 * w][1] = pack_half(q[w][2] * up, q[w][6] * up);
            qb[nt][2 * w + 1][0] = pack_half(q[w][1] * up4, q[w][5] * up4);
            qb[nt][2 * w + 1][1] = pack_half(q[w][3] * up4, q[w][7] * up4);
        }
        const float f = pow2(24 - e) * kLog2eOverSqrtD;
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // this lane's columns of the products: 2t, 2t + 1
            const int from = (2 * t + j) * 4;
            F[nt][j] = __shfl_sync(0xffffffffu, f, from);
            Q0[nt][j] = __shfl_sync(0xffffffffu, sum[0] * kLog2eOverSqrtD, from);
            Q1[nt][j] = __shfl_sync(0xffffffffu, sum[1] * kLog2eOverSqrtD, from);
            const int cc = nt * 8 + 2 * t + j;
            cpos[nt][j] = cc < nc ? pos0 + (c0 + cc) / G : -1;  // -1: sees nothing
        }
    }

    float m[NT][2], l[NT][2], c[NT][2], za[NT][2][2], ot[NT][8][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[nt][j] = kUnset;
            l[nt][j] = 0.f;
            c[nt][j] = pow2(100);
            za[nt][j][0] = za[nt][j][1] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ot[nt][i][0] = ot[nt][i][1] = ot[nt][i][2] = ot[nt][i][3] = 0.f;
    }

    const int krow = key_of_row(g);                  // rows g and g + 8: keys krow, krow + 8
    const int k_at = krow * kRowBytes + ((t ^ (krow & 2)) << 4);
    const int v_at0 = t * kRowBytes + ((g ^ ((t & 2) << 1)) << 3);            // row 2t: key t
    const int v_at1 = ((t ^ 1) + 4) * kRowBytes + ((g ^ ((t & 2) << 1)) << 3);  // row 2t + 1: key (t ^ 1) + 4

    for (int i = 0; i < nsteps; ++i) {
        wait_step(i);
        const char* kb = buf + i * kBlockBytes;
        const char* vb = kb + kHalfBlock;
        // ---- code sums of the scores, a group of dims apart ----
        float acc[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[nt][0][j] = acc[nt][1][j] = 0.f;
        {
            const uint4 ka = *reinterpret_cast<const uint4*>(kb + k_at);
            const uint4 kc = *reinterpret_cast<const uint4*>(kb + k_at + 8 * kRowBytes);
            const uint32_t x[4] = {ka.x, ka.y, ka.z, ka.w}, y[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t x8 = x[w] >> 8, y8 = y[w] >> 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(acc[nt][w & 1], x[w] & 0x000f000fu, y[w] & 0x000f000fu, x8 & 0x000f000fu,
                            y8 & 0x000f000fu, qb[nt][2 * w][0], qb[nt][2 * w][1]);
                    mma_f16(acc[nt][w & 1], x[w] & 0x00f000f0u, y[w] & 0x00f000f0u, x8 & 0x00f000f0u,
                            y8 & 0x00f000f0u, qb[nt][2 * w + 1][0], qb[nt][2 * w + 1][1]);
                }
            }
        }
        // ---- scores, weights ----
        uint2 km[2], vm[2];
#pragma unroll
        for (int hk = 0; hk < 2; ++hk) {
            km[hk] = *reinterpret_cast<const uint2*>(kb + kMetaOff + (krow + 8 * hk) * kMetaBytes);
            vm[hk] = *reinterpret_cast<const uint2*>(vb + kMetaOff + (krow + 8 * hk) * kMetaBytes);
        }
        const int kp = k0 + i * kBlockPos + krow;                    // position of rows g (and + 8)
        const bool edge = k0 + i * kBlockPos + kBlockPos - 1 > p_first;  // some column does not see every key
        uint32_t wb[NT][2][2];                                       // weights' operands: [group][keys 0-7 / 8-15]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[2][2], ts[2][2];
            bool move = false;
#pragma unroll
            for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ts[hk][j] = fmaf(lo_f(km[hk].y), acc[nt][1][2 * hk + j], lo_f(km[hk].x) * acc[nt][0][2 * hk + j]);
                    float z = fmaf(hi_f(km[hk].x), Q0[nt][j], -m[nt][j]);
                    z = fmaf(hi_f(km[hk].y), Q1[nt][j], z);
                    x[hk][j] = fmaf(F[nt][j], ts[hk][j], z);
                    if (edge && kp + 8 * hk > cpos[nt][j]) x[hk][j] = -INFINITY;
                    move |= x[hk][j] > kLazy;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float raw[2];
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        float z = hi_f(km[hk].x) * Q0[nt][j];
                        z = fmaf(hi_f(km[hk].y), Q1[nt][j], z);
                        raw[hk] = fmaf(F[nt][j], ts[hk][j], z);
                        if (edge && kp + 8 * hk > cpos[nt][j]) raw[hk] = -INFINITY;
                    }
                    const float over = col_max(fmaxf(x[0][j], x[1][j]));
                    const float top = col_max(fmaxf(raw[0], raw[1]));
                    if (over > kLazy) {  // the column's own lanes agree
                        const float al = ex2(m[nt][j] - top);
                        m[nt][j] = top;
                        l[nt][j] *= al;
                        za[nt][j][0] *= al;
                        za[nt][j][1] *= al;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            ot[nt][d][j] *= al;
                            ot[nt][d][2 + j] *= al;
                        }
                        x[0][j] = raw[0] - top;
                        x[1][j] = raw[1] - top;
                    }
                }
            }
            float w[2][2][2];  // [group][key half][column]
            float p[2][2];
            uint32_t top2 = 0;
#pragma unroll
            for (int hk = 0; hk < 2; ++hk) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    p[hk][j] = ex2(x[hk][j]);
                    l[nt][j] += p[hk][j];
                    const bool out = edge && kp + 8 * hk > cpos[nt][j];
                    const float pc = p[hk][j] * c[nt][j];
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        const uint32_t mt = gr ? vm[hk].y : vm[hk].x;
                        za[nt][j][gr] = fmaf(p[hk][j], out ? 0.f : hi_f(mt), za[nt][j][gr]);
                        w[gr][hk][j] = out ? 0.f : pc * lo_f(mt);
                    }
                }
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    wb[nt][gr][hk] = pack_half(w[gr][hk][0], w[gr][hk][1]);
                    top2 = __vmaxu2(top2, wb[nt][gr][hk]);  // w >= 0: fp16 order is the order of the bits
                }
            }
            // 2^15 is 0x7800 (NaN, above it, takes the slow path and stays NaN)
            if (__any_sync(0xffffffffu, (top2 & 0xffffu) > 0x7800u || (top2 >> 16) > 0x7800u)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float wt = 0.f, ps = 0.f;  // largest w, and largest P s 2^-20 (which cannot overflow)
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        const bool out = edge && kp + 8 * hk > cpos[nt][j];
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr) {
                            wt = fmaxf(wt, w[gr][hk][j]);
                            const float sc = out ? 0.f : lo_f(gr ? vm[hk].y : vm[hk].x);
                            ps = fmaxf(ps, p[hk][j] * (sc * pow2(-20)));
                        }
                    }
                    wt = col_max(wt);
                    ps = col_max(ps);
                    if (wt > kTopW && ps < INFINITY) {
                        const float nc_ = pow2(max(-126, min(100, 6 - 20 - exponent(ps))));
                        const float ratio = nc_ * (1.f / c[nt][j]);  // powers of two: exact, or 0
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            ot[nt][d][j] *= ratio;
                            ot[nt][d][2 + j] *= ratio;
                        }
                        c[nt][j] = nc_;
#pragma unroll
                        for (int hk = 0; hk < 2; ++hk) {
                            const bool out = edge && kp + 8 * hk > cpos[nt][j];
#pragma unroll
                            for (int gr = 0; gr < 2; ++gr)
                                w[gr][hk][j] = out ? 0.f : p[hk][j] * nc_ * lo_f(gr ? vm[hk].y : vm[hk].x);
                        }
                    }
                }
#pragma unroll
                for (int hk = 0; hk < 2; ++hk)
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) wb[nt][gr][hk] = pack_half(w[gr][hk][0], w[gr][hk][1]);
            }
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) wb[nt][gr][hk] = wm::movmatrix_t(wb[nt][gr][hk]);
        }
        // ---- code sums of the output: dims 64 gr + 8 g + n (rows g), + 4 (rows g + 8) ----
        uint2 v0 = *reinterpret_cast<const uint2*>(vb + v_at0);
        uint2 v1 = *reinterpret_cast<const uint2*>(vb + v_at1);
        uint2 v2 = *reinterpret_cast<const uint2*>(vb + v_at0 + 8 * kRowBytes);
        uint2 v3 = *reinterpret_cast<const uint2*>(vb + v_at1 + 8 * kRowBytes);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
            const uint32_t e0 = gr ? v0.y : v0.x, e1 = gr ? v1.y : v1.x, e2 = gr ? v2.y : v2.x, e3 = gr ? v3.y : v3.x;
            uint32_t x0 = __byte_perm(e0, e1, 0x5410), x1 = __byte_perm(e0, e1, 0x7632);
            uint32_t x2 = __byte_perm(e2, e3, 0x5410), x3 = __byte_perm(e2, e3, 0x7632);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(ot[nt][gr * 4 + n], x0 & 0x000f000fu, x1 & 0x000f000fu, x2 & 0x000f000fu,
                            x3 & 0x000f000fu, wb[nt][gr][0], wb[nt][gr][1]);
                    mma_f16(ot[nt][gr * 4 + n + 1], x0 & 0x00f000f0u, x1 & 0x00f000f0u, x2 & 0x00f000f0u,
                            x3 & 0x00f000f0u, wb[nt][gr][0], wb[nt][gr][1]);
                }
                x0 >>= 8;
                x1 >>= 8;
                x2 >>= 8;
                x3 >>= 8;
            }
        }
    }

    // ---- join the warps ----
    wm::cp_async_wait_all();
    __syncthreads();  // the buffers are free
    float* co = reinterpret_cast<float*>(smem);  // [warp][column][kCoStride]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = nt * 8 + 2 * t + j;
            const float inv = 1.f / c[nt][j];  // a power of two up to 2^126
            const float z0 = col_sum(za[nt][j][0]), z1 = col_sum(za[nt][j][1]);
            const float ls = col_sum(l[nt][j]);
            float* o = co + (warp * NT * 8 + col) * kCoStride + 8 * g;
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float z = gr ? z1 : z0;
                    const int k = 2 * half + j;
                    *reinterpret_cast<float4*>(o + 64 * gr + 4 * half) =
                        make_float4(fmaf(ot[nt][gr * 4][k] * kLoCode, inv, z), fmaf(ot[nt][gr * 4 + 1][k] * kHiCode, inv, z),
                                    fmaf(ot[nt][gr * 4 + 2][k] * kLoCode, inv, z),
                                    fmaf(ot[nt][gr * 4 + 3][k] * kHiCode, inv, z));
                }
            if (g == 0) {
                sm_m[warp][col] = m[nt][j];
                sm_l[warp][col] = ls;
            }
        }
    __syncthreads();
    for (int col = warp; col < nc; col += kWarps) {  // a warp per column, lane i dims 4i..4i+3
        float M = sm_m[0][col];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm_m[w][col]);
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wt = exp2f(sm_m[w][col] - M);
            const float4 v = *reinterpret_cast<const float4*>(co + (w * NT * 8 + col) * kCoStride + 4 * lane);
            L = fmaf(sm_l[w][col], wt, L);
            O.x = fmaf(v.x, wt, O.x);
            O.y = fmaf(v.y, wt, O.y);
            O.z = fmaf(v.z, wt, O.z);
            O.w = fmaf(v.w, wt, O.w);
        }
        const int row = r0 + (c0 + col) / G, hq = h * G + (c0 + col) % G;
        if (nu_all == 1) {
            __nv_bfloat162 b[2] = {__floats2bfloat162_rn(O.x / L, O.y / L), __floats2bfloat162_rn(O.z / L, O.w / L)};
            *reinterpret_cast<uint2*>(a.out + (long)row * a.ldo + hq * kHeadDim + 4 * lane) =
                *reinterpret_cast<uint2*>(b);
        } else {
            const size_t idx = ((size_t)row * a.n_q + hq) * a.max_units + u;
            *reinterpret_cast<float4*>(a.po + idx * kHeadDim + 4 * lane) = O;
            if (lane == 0) {
                a.pm[idx] = M;
                a.pl[idx] = L;
            }
        }
    }
    pdl_trigger();
    if (nu_all == 1) return;

    // ---- join the units: groups of kFan, then the groups ----
    const int groups = (nu_all + kFan - 1) / kFan;
    const int gi = u / kFan, gn = min(kFan, nu_all - gi * kFan);
    const int set = (a.set_start[s] + chunk) * rm.n_kv + h;  // this (stream, columns, head)
    unsigned* counters = a.counters + (size_t)set * a.max_counters;
    if (gn > 1 && !last_of(counters + 1 + gi, gn, &flag)) return;
    for (int level = 0; level < 2; ++level) {
        const bool final = level == 1 || groups == 1;
        for (int col = warp; col < nc; col += kWarps) {
            const int row = r0 + (c0 + col) / G, hq = h * G + (c0 + col) % G;
            const size_t cidx = (size_t)row * a.n_q + hq;
            const size_t base = level == 0 ? cidx * a.max_units + gi * kFan : cidx * a.max_groups;
            const float *pm = level == 0 ? a.pm : a.gm, *pl = level == 0 ? a.pl : a.gl, *po = level == 0 ? a.po : a.go;
            float M, L;
            float4 O;
            join(pm + base, pl + base, po + base * kHeadDim, level == 0 ? gn : groups, M, L, O);
            if (final) {
                __nv_bfloat162 b[2] = {__floats2bfloat162_rn(O.x / L, O.y / L),
                                       __floats2bfloat162_rn(O.z / L, O.w / L)};
                *reinterpret_cast<uint2*>(a.out + (long)row * a.ldo + hq * kHeadDim + 4 * lane) =
                    *reinterpret_cast<uint2*>(b);
            } else {
                const size_t gidx = cidx * a.max_groups + gi;
                *reinterpret_cast<float4*>(a.go + gidx * kHeadDim + 4 * lane) = O;
                if (lane == 0) {
                    a.gm[gidx] = M;
                    a.gl[gidx] = L;
                }
            }
        }
        if (final || !last_of(counters, groups, &flag)) return;
    }
}

}  // namespace

int attn_unit() { return kUnit; }
int attn_fan() { return kFan; }

cudaError_t init_attn() {
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return e;
}

cudaError_t launch_attn(AttnArgs& a, cudaStream_t st, bool pdl) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    const int G = a.n_q / a.rows.n_kv;
    // one tile of eight columns where every stream's rows fit it, else two: codes are then unpacked once for 16 columns
    int nt = 1;
    for (int s = 0; s < a.rows.n_streams; ++s)
        if ((a.rows.row_start[s + 1] - a.rows.row_start[s]) * G > 8) nt = 2;
    int items = 0, sets = 0;
    for (int s = 0; s < a.rows.n_streams; ++s) {
        const int R = a.rows.row_start[s + 1] - a.rows.row_start[s];
        const int chunks = (R * G + nt * 8 - 1) / (nt * 8);
        a.item_start[s] = items;
        a.set_start[s] = sets;
        sets += chunks;
        if (R > 0) items += chunks * a.rows.n_kv * ((a.rows.pos0[s] + R - 1) / kUnit + 1);
    }
    a.item_start[a.rows.n_streams] = items;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)items);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kSmem;
    c.stream = st;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = 1;
    }
    return nt == 1 ? cudaLaunchKernelEx(&c, attn_kernel<1>, a) : cudaLaunchKernelEx(&c, attn_kernel<2>, a);
}

}  // namespace kv4
}  // namespace tfl
