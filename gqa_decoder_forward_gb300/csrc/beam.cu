// Beam search's selection over beams and vocabulary.  A group's beams b, with
// running log-probabilities s_b and rows of logits z_b, offer the candidates
//   score(b, v) = s_b + (z_b[v] - max z_b) - log sum_w e^(z_b[w] - max z_b),
// for its n_out largest logits, and of all those the n_out best are kept, ordered by score and,
// where scores are equal, by the lower row and then the lower id.  An ended beam offers one candidate (eos, s_b).
//
// Two launches:
//   chunk (a CTA per 8,192 logits of a row, of 256 threads or, in small calls, 512): within a row the order by score is the order by
//         logit, so a chunk's n_out largest logits (ties to the lower id) are all that can be
//         chosen from it.  A logit and its place make one 32-bit key, order-preserving bf16 above
//         the inverted place, so that keys are never equal.  One read of the logits gives the largest, the
//         candidates and the sum of exponentials.
//   join  (a CTA per group): the rows' sums and logarithms; then the candidates that can be among the n_out best, by
//         bounds in fp32, as 64-bit scores, which are ranked by comparison.
//
// Sums.  Beams are compared by sums over whole rows, so a sum's error can change who is chosen: e^z is a
// table's 2^(j/32), held as two fp32 numbers, times a short series (P. T. P. Tang's table-driven method, ACM TOMS 15
// (1989)), since double-precision arithmetic runs at 1/64 of the fp32 rate here.  A chunk's terms are good to 2^-29, what
// the join computes from the sums to about 2^-40.  Sums are integers: a chunk's in units of 2^(E-49) with
// E = ceil(z_max log2 e) of the chunk, a row's in units of 2^(E-45), so they do not depend on the order of addition; 16 logits are
// added up in fp32 before, the same ones and in the same order in either size of CTA, so that a row's score does not depend on
// the rest of the call.  The largest logit is counted apart, so that a row in which nothing else counts has the score s_b itself.
//
// Bound and measured (ids of 166,912, replayed from a graph).  64 rows of 16 beams, 32 kept (21.4 MB, 3.2 us of copying): 25.9
// us, of which the chunks take 17: 40 instructions a logit, 15 of them the exponential's, in 62% of the issue slots; the
// rest is a second round of CTAs (1,344 chunks, six to an SM at a time), and phases of a CTA in which few warps work.  As long with
// eight or five CTAs an SM; with 19 chunks of 8,785 logits, so that all are there at once: 25.9.  The exponential as in the join: 34; one
// logit an instruction: 26.4.  Four rows of one search: 8.5 us, the latency of two launches and of steps that wait for one
// another: loads, the largest, the n_out best and the sum, then the join's lists.
#include "beam.cuh"
#include "pair.cuh"

namespace tfl {
namespace beam {
namespace {

constexpr int kJoinThreads = 512;
constexpr int kSumThreads = 512;         // sums of a chunk's exponentials, of the same 16 logits each however many threads there are
constexpr int kReach = 2 * kMaxOut;      // threads of a chunk whose logits may reach its threshold
constexpr unsigned kBad = 1u;            // flag: the chunk holds NaN or +Inf
constexpr int kIdBits = 18;
static_assert(kMaxBeams * kMaxChunks <= kJoinThreads, "a thread per chunk of a group");
static_assert(kMaxChunks * kChunk <= 1 << kIdBits && kMaxBeams <= 1 << (32 - kIdBits), "a candidate's place");

// 2^(j/32) as t (1 + r): t of fp32, r what it leaves.
__device__ const float2 kPow[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.059b0ep+0f, -0x1.947414p-25f}, {0x1.0b5586p+0f, 0x1.8d96d4p-25f}, {0x1.11301ep+0f, -0x1.dda2fcp-25f},
    {0x1.172b84p+0f, -0x1.9c0c22p-27f}, {0x1.1d4874p+0f, -0x1.a2fbb2p-25f}, {0x1.2387a6p+0f, 0x1.964904p-25f}, {0x1.29e9e0p+0f, -0x1.2b0dbcp-25f},
    {0x1.306fe0p+0f, 0x1.125002p-25f}, {0x1.371a74p+0f, -0x1.cde8cep-26f}, {0x1.3dea64p+0f, 0x1.370be4p-25f}, {0x1.44e086p+0f, 0x1.336de2p-30f},
    {0x1.4bfdaep+0f, -0x1.0a3550p-25f}, {0x1.5342b6p+0f, -0x1.c541b4p-26f}, {0x1.5ab07ep+0f, -0x1.00d8acp-27f}, {0x1.6247ecp+0f, -0x1.6cb284p-25f},
    {0x1.6a09e6p+0f, 0x1.26055cp-26f}, {0x1.71f75ep+0f, 0x1.8b2bb8p-26f}, {0x1.7a1148p+0f, -0x1.05cb44p-25f}, {0x1.82589ap+0f, -0x1.1c2142p-26f},
    {0x1.8ace54p+0f, 0x1.67a1cap-28f}, {0x1.93737cp+0f, -0x1.348e56p-25f}, {0x1.9c4918p+0f, 0x1.a3b5e4p-28f}, {0x1.a5503cp+0f, -0x1.0b7ec8p-25f},
    {0x1.ae89fap+0f, -0x1.f9c304p-27f}, {0x1.b7f770p+0f, -0x1.e4c886p-26f}, {0x1.c199bep+0f, -0x1.6961b4p-28f}, {0x1.cb720ep+0f, -0x1.b5151ep-28f},
    {0x1.d5818ep+0f, -0x1.a5217cp-28f}, {0x1.dfc974p+0f, -0x1.ab7132p-26f}, {0x1.ea4afap+0f, 0x1.61428ep-28f}, {0x1.f50766p+0f, -0x1.2ad5f8p-27f}};

constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0c0p-26f;
constexpr float kLog2eHi = 0x1.7154p+0f, kLog2eRest = 0x1.d94ae0p-18f;  // the same, 16 bits first
constexpr float kLn2 = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;
constexpr float kRound = 393216.f;  // 1.5 * 2^18: sums with it are multiples of 1/32

// e^z 2^-E as an unevaluated sum of two fp32 numbers, for |z| < 2^17; 0 where it is below 2^-60 (z = -inf
// too).  z log2 e = th + tl; th = k/32 + f exactly; (f + tl) ln 2 = xh + xl, at most 0.017; e^x - 1 by its series,
// whose terms from x^2 on fit fp32 (the sixth is below 2^-43).
__device__ __forceinline__ float2 exp_scaled(float z, int E, const float2* pow) {
    const float th = __fmul_rn(z, kLog2e);
    const float tl = __fmaf_rn(z, kLog2eLo, __fmaf_rn(z, kLog2e, -th));
    const float s = __fadd_rn(th, kRound);
    const float f = __fadd_rn(th, -__fadd_rn(s, -kRound));
    const int k = __float_as_int(s) - __float_as_int(kRound);
    const float xh = __fmul_rn(f, kLn2);
    float xl = __fmaf_rn(f, kLn2Lo, __fmaf_rn(f, kLn2, -xh));
    xl = __fmaf_rn(tl, kLn2, xl);
    float p = __fmaf_rn(xh, 1.f / 120.f, 1.f / 24.f);
    p = __fmaf_rn(p, xh, 1.f / 6.f);
    p = __fmaf_rn(p, xh, 0.5f);
    p = __fmul_rn(p, __fmul_rn(xh, xh));
    xl = __fmaf_rn(xh, xl, xl);
    const float uh = __fadd_rn(xh, p);
    const float ul = __fadd_rn(__fadd_rn(__fadd_rn(xh, -uh), p), xl);
    const float2 t = pow[k & 31];
    const float ph = __fmul_rn(t.x, uh);
    const float pl = __fmaf_rn(t.x, __fadd_rn(ul, __fmaf_rn(t.y, uh, t.y)), __fmaf_rn(t.x, uh, -ph));
    const float eh = __fadd_rn(t.x, ph);
    const float el = __fadd_rn(__fadd_rn(__fadd_rn(t.x, -eh), ph), pl);
    const int n = (k >> 5) - E;
    const bool any = th > -1e6f && n > -60;
    const float scale = __int_as_float((n + 127) << 23);
    return make_float2(any ? __fmul_rn(eh, scale) : 0.f, any ? __fmul_rn(el, scale) : 0.f);
}

// From this magnitude on, bf16 numbers are 64 and more below the largest if they are below it: only it counts in a sum.
constexpr float kHuge = 16384.f;
__device__ __forceinline__ int exponent_of(float z_max) { return (int)ceilf(__fmul_rn(z_max, kLog2e)); }

// Order-preserving 16 bits of a bf16 pattern, -0 as +0; 0 for -inf, which is no candidate.
__device__ __forceinline__ unsigned order_of(unsigned x) {
    if (x == 0xFF80u) return 0u;
    if (x == 0x8000u) x = 0u;
    return (x ^ ((x & 0x8000u) ? 0xFFFFu : 0x8000u)) & 0xFFFFu;
}
__device__ __forceinline__ float logit_of(unsigned order) {
    const unsigned x = (order & 0x8000u) ? order ^ 0x8000u : order ^ 0xFFFFu;
    return __uint_as_float((x & 0xFFFFu) << 16);
}

// Whether a row's logits matter: a beam that has ended, or whose score is -inf, has no use for them.
__device__ __forceinline__ bool row_live(const Args& a, int row) {
    return !(a.done && a.done[row] != 0) && a.scores[row] != -INFINITY;
}

// Eight logits as fp32.
__device__ __forceinline__ void unpack(const uint4& c, float (&z)[8]) {
    const unsigned x[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = __uint_as_float((e & 1) ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16);
}

// A logit and its place as one key: the order by value, then by the lower place; never equal to another.
__device__ __forceinline__ unsigned key_of(float z, int place) {
    const unsigned o = order_of(__float_as_uint(z) >> 16);
    return o ? (o << 16) | (0xFFFFu - (unsigned)place) : 0u;
}

__device__ __forceinline__ unsigned max2_nan(unsigned a, unsigned b) {
    unsigned r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of eight, as bf16 bits; NaN if one is.
__device__ __forceinline__ unsigned max8(const uint4& c) {
    const unsigned m = max2_nan(max2_nan(c.x, c.y), max2_nan(c.z, c.w));
    return max2_nan(m, __byte_perm(m, m, 0x1032)) & 0xFFFFu;
}

// With 256 threads the fewest instructions; with 512, where a CTA has an SM to itself, the shorter way (84 chunks: 8.75 and 8.5 us;
// 21: 8.7 and 8.3; 1,344: 26.0 and 28.7).
template <int kThreads>
__global__ void __launch_bounds__(kThreads) chunk_kernel(const __grid_constant__ Args a) {
    constexpr int kPer = kChunk / kThreads;  // logits of a thread, in 16-byte loads
    constexpr int kWarps = kThreads / 32;
    constexpr int kSums = kSumThreads / kThreads;  // sums of a thread: over its eights s, s + kSums, ...
    static_assert(kReach * (kPer / 8) <= kThreads, "an eight of theirs to a thread");
    // The chunk: thread t's i-th eight logits at [i][t].  Passes over them are loops, not a copy of their body for each logit
    // (straight-line code that runs once is fetched slower than it runs); held here, since other threads look at
    // some of them.
    __shared__ uint4 held[kPer / 8][kThreads];
    __shared__ unsigned pow_t[32];                    // 2^(j/32), as what is added to the bits of s: see the sum
    __shared__ float pow_r[32];                       // (a bank for each entry)
    __shared__ __align__(16) unsigned ext[kThreads];  // threads' maxima, extracted from warps
    __shared__ __align__(16) unsigned list[kReach * kPer];
    __shared__ unsigned long long sums[kWarps];
    __shared__ unsigned counts[kWarps], wmax[kWarps], bad_any, threshold;
    __shared__ int n_list, n_who;
    __shared__ unsigned short who[kReach];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.y, chunk = blockIdx.x, n = a.n_out;
    const float2 entry = kPow[lane];
    if (tid == 0) {
        n_list = n_who = 0;
        bad_any = 0u;
        threshold = 0u;
    }
    pdl_wait();
    pdl_trigger();
    const int at0 = chunk * kChunk, passes = (min(kChunk, a.V - at0) + kSumThreads * 8 - 1) / (kSumThreads * 8) * kSums;
    uint4 w[kPer / 8];
#pragma unroll
    for (int i = 0; i < kPer / 8; ++i) {
        const int at = at0 + (i * kThreads + tid) * 8;
        w[i] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        if (at < a.V) w[i] = *reinterpret_cast<const uint4*>(a.logits + (size_t)row * a.V + at);
    }
    if (tid < 32) {
        pow_t[tid] = __float_as_uint(entry.x) - (unsigned)(tid << 18) - (__float_as_uint(kRound) << 18);
        pow_r[tid] = entry.y;
    }
    if (!row_live(a, row)) return;
    bool bad = false;
    unsigned best = 0u, bests[kSums];  // the largest of all a thread's logits, and of each of its sums'
#pragma unroll
    for (int s = 0; s < kSums; ++s) {
        unsigned m2 = 0xFF80FF80u;
#pragma unroll
        for (int i = s; i < kPer / 8; i += kSums) {
            m2 = max2_nan(max2_nan(m2, w[i].x), max2_nan(w[i].y, max2_nan(w[i].z, w[i].w)));
            held[i][tid] = w[i];
        }
        m2 = max2_nan(m2, __byte_perm(m2, m2, 0x1032)) & 0xFFFFu;
        bad = bad || ((m2 & 0x7F80u) == 0x7F80u && m2 != 0xFF80u);  // a NaN, or +Inf
        bests[s] = order_of(m2);
        best = max(best, bests[s]);
    }
    const unsigned wm = __reduce_max_sync(0xffffffffu, best);
    __syncthreads();
    if (bad) bad_any = kBad;
    if (lane == 0) wmax[warp] = wm;
    __syncthreads();
    unsigned top = 0u;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = max(top, wmax[i]);
    const unsigned flags = bad_any;
    const int slot = row * a.chunks + chunk;
    unsigned* cand = a.cand + (size_t)slot * kMaxOut;
    if (flags || top == 0u) {  // not usable, or nothing but -inf
        if (tid < n) cand[tid] = 0u;
        if (tid == 0) {
            a.sum[slot] = 0ull;
            a.top[slot] = make_uint2(0u, flags);
        }
        return;
    }

    // The n best: a threshold that the maxima of at least n threads reach; then all logits from it on, which lie
    // in threads that reach it.  First from the best few threads of each warp.
    unsigned left = best ? (best << 16) | (0xFFFFu - tid) : 0u;
    const unsigned mine_key = left;
    const int r = min(32, (2 * n + kWarps - 1) / kWarps);
    for (int i = 0; i < r; ++i) {
        const unsigned m = __reduce_max_sync(0xffffffffu, left);
        if (lane == 0) ext[warp * r + i] = m;
        if (left == m) left = 0u;
    }
    __syncthreads();
    const auto nth = [&](int count) {  // the n-th largest of ext[0, count), which are distinct; 0 if there are fewer
        const unsigned k = tid < count ? ext[tid] : 0u;
        if (k) {
            int above = 0;
#pragma unroll 4
            for (int i = 0; i < count; ++i) above += ext[i] > k;
            if (above == n - 1) threshold = k;
        }
        __syncthreads();
    };
    nth(kWarps * r);
    unsigned limit = threshold & 0xFFFF0000u;
    unsigned reach = mine_key;
    // Few warps hold the candidates, one holds many that were not taken, or many threads tie: by every thread's
    // best logit and its place.  Either way at most kReach threads reach the limit.
    if (limit == 0u || __syncthreads_count(mine_key >= limit) > kReach) {
        unsigned k = 0u;
#pragma unroll 1
        for (int i = 0; i < kPer / 8; ++i) {
            float z[8];
            unpack(held[i][tid], z);
#pragma unroll
            for (int e = 0; e < 8; ++e) k = max(k, key_of(z[e], (i * kThreads + tid) * 8 + e));
        }
        __syncthreads();
        ext[tid] = reach = k;
        if (tid == 0) threshold = 0u;
        __syncthreads();
        nth(kThreads);
        limit = threshold;
    }
    limit = max(limit, 1u);
    // the eights of those threads, one to a thread of the CTA
    if (reach >= limit) who[atomicAdd(&n_who, 1)] = (unsigned short)tid;
    __syncthreads();
    if (tid < n_who * (kPer / 8)) {
        const int i = tid % (kPer / 8), t = who[tid / (kPer / 8)];
        const uint4 c = held[i][t];
        const float least = limit >> 16 ? logit_of(limit >> 16) : __uint_as_float(0xFF7FFFFFu);  // (or all but -inf)
        if (__uint_as_float(max8(c) << 16) >= least) {
            float z[8];
            unpack(c, z);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (z[e] >= least) {
                    const unsigned k = key_of(z[e], (i * kThreads + t) * 8 + e);
                    if (k >= limit) list[atomicAdd(&n_list, 1)] = k;
                }
        }
    }

    // How often the largest occurs, and the sum of e^z over the others: e^z 2^-E = t 2^n (1 + r) 2^g with
    // z log2 e = k/32 + g, as in exp_scaled but for (1 + r) 2^g - 1 in one fp32 number (good to 2^-29).  Of 16 logits at a time, with
    // the E of their own largest, in two fp32 sums: multiples of 2^-18 (exact: at most 16) and what they leave, at most 2^-19 a
    // term, so that what fp32 rounds is 2^-35 of their largest in all, however many terms there are below it.
    // Then integers.
    const float z_max = logit_of(top);
    const bool huge = fabsf(z_max) >= kHuge;
    const int E = huge ? 0 : exponent_of(z_max);
    unsigned count = 0u;
    unsigned long long mine = 0ull;
    float round;
    Pair whole, rest;
    const auto add = [&](const float(&z)[8]) {
        Pair x[4], g[4], t[4], p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = pair_of(z[2 * e], z[2 * e + 1]);
            const Pair s = fma2(x[e], pair_of(kLog2e), pair_of(round));                  // its low bits are k - 32 E_own
            g[e] = fma2(s, pair_of(-1.f), pair_of(round));
            g[e] = fma2(x[e], pair_of(kLog2eHi), g[e]);                                  // exact: 16 bits by 8
            g[e] = fma2(x[e], pair_of(kLog2eRest), g[e]);
            const float2 v = parts_of(s);
            const unsigned a = __float_as_uint(v.x), b = __float_as_uint(v.y);
            // s's low five bits are j, those above them the exponent: 18 bits up, with what pow_t takes off
            t[e] = pair_of(__uint_as_float(pow_t[a & 31u] + a * (1u << 18)), __uint_as_float(pow_t[b & 31u] + b * (1u << 18)));
            x[e] = pair_of(pow_r[a & 31u], pow_r[b & 31u]);
            p[e] = fma2(g[e], pair_of(0x1.3b2ab6p-7f), pair_of(0x1.c6b08ep-5f));         // ln2^4 / 24, ln2^3 / 6
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fma2(p[e], g[e], pair_of(0x1.ebfbe0p-3f));    // ln2^2 / 2
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fma2(p[e], g[e], pair_of(0x1.62e430p-1f));    // ln2
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = fma2(p[e], g[e], x[e]);
            const Pair q = add2(add2(fma2(t[e], p[e], t[e]), pair_of(48.f)), pair_of(-48.f));
            whole = add2(whole, q);
            p[e] = fma2(t[e], p[e], fma2(q, pair_of(-1.f), t[e]));
        }
        rest = add2(rest, add2(add2(p[0], p[1]), add2(p[2], p[3])));
    };
    // Logits below `cut` count as if they were there, which is nothing; so do the largest, in the warps that hold one.
    const bool holds = __any_sync(0xffffffffu, best == top);
    if (!huge || holds) {
#pragma unroll 1
        for (int s = 0; s < kSums; ++s) {
            const unsigned own = kSums > 1 && s > 0 ? bests[kSums - 1] : bests[0];
            const float z_own = fmaxf(own ? logit_of(own) : -INFINITY, z_max - 41.5f);
            const float cut = z_own - 41.5f;  // e^-41.5 for each of the up to 2^18 logits below: 2^-41 in all
            const int E_own = huge ? 0 : exponent_of(z_own);
            round = kRound - (float)E_own;
            whole = rest = 0ull;
#pragma unroll 1
            for (int i = s; i < passes; i += kSums) {
                float z[8];
                unpack(held[i][tid], z);
                if (holds) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        count += z[e] == z_max;
                        z[e] = z[e] == z_max ? cut : z[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = fmaxf(z[e], cut);
                if (!huge) add(z);
            }
            const float2 w2 = parts_of(whole), r2 = parts_of(rest);
            const float wholes = __fadd_rn(w2.x, w2.y), rests = __fadd_rn(r2.x, r2.y);
            if (!huge)
                mine += (unsigned long long)((((long long)(wholes * 262144.f) << 31) + __float2ll_rn(rests * 562949953421312.f)) >>
                                             (E - E_own));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
        sums[warp] = mine;
        counts[warp] = count;
    }
    __syncthreads();
    // (a thread to a logit: a few warps' work, beside which other CTAs' goes on)
    const int L = n_list;
    for (int e = tid; e < max(L, n); e += kThreads) {
        if (e < L) {
            const unsigned k = list[e];
            int above = 0;
#pragma unroll 4
            for (int i = 0; i < L; ++i) above += list[i] > k;
            if (above < n) cand[above] = k;
            if (above == 0) a.top[slot].x = k;
        } else {
            cand[e] = 0u;  // no candidate
        }
    }
    if (tid == 0) {
        unsigned long long s = 0ull;
        unsigned c = 0u;
        for (int i = 0; i < kWarps; ++i) {
            s += sums[i];
            c += counts[i];
        }
        a.sum[slot] = s;
        a.top[slot].y = c << 1;
    }
}

// s + e = a + b exactly, s rounded (D. E. Knuth, The Art of Computer Programming, vol. 2, 4.2.2).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float v = __fadd_rn(s, -a);
    e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -v)), __fadd_rn(b, -v));
}
// A score as 64 bits in the same order; 0 stands for no candidate (and is no finite score's).
__device__ __forceinline__ unsigned long long order_of(double s) {
    const long long b = __double_as_longlong(s == 0.0 ? 0.0 : s);
    return (unsigned long long)b ^ (b < 0 ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double score_of(unsigned long long o) {
    return __longlong_as_double((long long)(o ^ ((o >> 63) ? 0x8000000000000000ull : ~0ull)));
}

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a) {
    constexpr int kFinal = (kMaxOut - 1 + kMaxChunks) * kMaxOut;  // of the lists that are left in any case: see there
    __shared__ float2 pow[32];
    __shared__ float row_top[kMaxBeams], score[kMaxBeams];
    __shared__ float log_rest[kMaxBeams], log_low[kMaxBeams];  // log sum_w e^(z_w - z_max) of row b, as a sum
    __shared__ int live[kMaxBeams];                // 0: no candidate, 1: its logits, 2: it has ended
    __shared__ __align__(16) unsigned head[kJoinThreads];
    __shared__ unsigned cand[kFinal], place[kFinal];  // keys of the candidates left; row in the group, then id
    __shared__ int from[kFinal];                   // their lists: row << 16 | chunk
    __shared__ unsigned long long key[kFinal];
    __shared__ unsigned reach;                     // a score that n candidates reach, in order; 0: none
    __shared__ unsigned short deep[kJoinThreads];  // lists whose first four all count
    __shared__ int n_final, n_deep, bad_any;
    static_assert(kJoinThreads <= kFinal, "a key for each list");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x, B = a.beams, C = a.chunks, n = a.n_out, row0 = g * B;
    const float2 entry = kPow[lane];
    if (tid == 0) {
        n_final = n_deep = bad_any = 0;
    }
    pdl_wait();
    // a list for each chunk, whose best is the chunk's largest logit; neighbouring lists lie in different warps
    const int lists = B * C, my = lane * (kJoinThreads / 32) + warp;
    const unsigned* my_cand = a.cand + (size_t)(row0 * C + my) * kMaxOut;
    unsigned head_key = 0u;
    uint4 ahead = make_uint4(0u, 0u, 0u, 0u);  // the list's first four, asked for before it is known whether they count
    if (my < lists) {
        head_key = a.top[row0 * C + my].x;
        ahead = *reinterpret_cast<const uint4*>(my_cand);
    }
    if (tid < 32) pow[tid] = entry;
    __syncthreads();
    // rows: a warp each, a lane for each chunk
    for (int b = warp; b < B; b += kJoinThreads / 32) {
        const int row = row0 + b;
        const float s = a.scores[row];
        const bool ended = a.done && a.done[row] != 0;
        bool alive = row_live(a, row);
        bool bad = isnan(s) || s == INFINITY;
        unsigned t = 0u, count = 0u;
        unsigned long long sum = 0ull;
        if (alive && lane < C) {
            const uint2 v = a.top[row * C + lane];
            t = v.x;
            count = v.y >> 1;
            bad = bad || (v.y & kBad);
            sum = a.sum[row * C + lane];
        }
        bad = __any_sync(0xffffffffu, bad);
        const unsigned m = __reduce_max_sync(0xffffffffu, t);
        const float z = logit_of(t >> 16), z_max = logit_of(m >> 16);
        if (m == 0u) alive = false;          // nothing but -inf
        unsigned long long part = 0ull;      // of the sum of e^z over all but the row's largest, in units of 2^(E - 45)
        const bool largest = t >> 16 == m >> 16, usual = fabsf(z_max) < kHuge;
        const int E = usual ? exponent_of(z_max) : 0;
        if (t != 0u && usual) {
            const bool near = fabsf(z) < kHuge;  // (beyond, 64 and more below the row's largest: nothing, and not for exp_scaled)
            const int d = near ? E - exponent_of(z) : 64;
            part = d < 60 ? sum >> (4 + d) : 0ull;
            if (!largest && near) {
                const float2 e = exp_scaled(z, E, pow);
                part += (unsigned long long)count *
                        (unsigned long long)(__float2ll_rn(e.x * 35184372088832.f) + __float2ll_rn(e.y * 35184372088832.f));
            }
        }
        count = __reduce_add_sync(0xffffffffu, t != 0u && largest ? count : 0u);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        // log of the sum relative to the largest: S = count + the others' sum / e^z_max, which is 1 exactly where
        // nothing else counts; y = logf(S); S e^-y = 1 + w; log S = y + log(1 + w).  In sums of two fp32 numbers
        // (double-precision instructions take sixteen cycles of the SM each).
        float lh = 0.f, ll = 0.f;
        if (alive) {
            const float N = (float)count;
            float sh = N, sl = 0.f;
            if (usual) {
                const float2 r = exp_scaled(-z_max, -E, pow);
                const float uh = __ull2float_rn(part), ul = __ll2float_rn((long long)(part - __float2ull_rn(uh)));
                const float ph = __fmul_rn(uh, r.x);
                const float pl = __fmaf_rn(uh, r.y, __fmaf_rn(ul, r.x, __fmaf_rn(uh, r.x, -ph)));
                const float qh = __fmul_rn(ph, 0x1p-45f), ql = __fmul_rn(pl, 0x1p-45f);
                two_sum(N, qh, sh, sl);
                sl = __fadd_rn(sl, ql);
            }
            lh = logf(sh);
            const float2 e = exp_scaled(-lh, 0, pow);
            const float ph = __fmul_rn(sh, e.x);
            const float pl = __fmaf_rn(sh, e.y, __fmaf_rn(sl, e.x, __fmaf_rn(sh, e.x, -ph)));
            const float w = __fadd_rn(__fadd_rn(ph, -1.f), pl);
            ll = __fmaf_rn(-0.5f * w, w, w);
        }
        if (lane == 0) {
            if (bad) bad_any = 1;
            live[b] = ended ? 2 : alive ? 1 : 0;
            row_top[b] = z_max;
            score[b] = s;
            log_rest[b] = lh;
            log_low[b] = ll;
        }
    }
    __syncthreads();
    if (bad_any) {  // the group's ranking is undefined
        if (tid == 0) atomicOr(a.status, kStatusNonFinite);
        if (tid < n) {
            a.ids[g * n + tid] = a.parents[g * n + tid] = -1;
            a.out_scores[g * n + tid] = __int_as_float(0x7fffffff);
            if (a.out_done) a.out_done[g * n + tid] = 0;
        }
        return;
    }
    // The score of row b's logit of this order: added up in two fp32 numbers, as a 64-bit one in the end; in 64 bits from the start
    // where it, or the logit's distance from the largest, is beyond fp32's range.
    const auto score_at = [&](int b, unsigned order) {
        float dh, dl, uh, ul, vh, vl;
        two_sum(logit_of(order), -row_top[b], dh, dl);
        two_sum(dh, -log_rest[b], uh, ul);
        two_sum(score[b], uh, vh, vl);
        const float rest = __fadd_rn(vl, __fadd_rn(__fadd_rn(dl, ul), -log_low[b]));
        if (isinf(vh)) {
            const double d = (double)logit_of(order) - (double)row_top[b];
            return order_of((double)score[b] + (d - ((double)log_rest[b] + (double)log_low[b])));
        }
        return order_of((double)vh + (double)rest);
    };
    // Who can be among the n best, in fp32 with a margin (double precision is slow for all): a candidate's score lies
    // within `off` of `near`; the n-th largest of some candidates' lower ends is a score that n candidates reach.
    const auto bounds = [&](int b, unsigned order, float& low, float& high) {
        const float d = logit_of(order) - row_top[b], lg = log_rest[b], near = score[b] + (d - lg);
        const float off = (fabsf(score[b]) + fabsf(d) + lg) * 0x1p-21f;
        low = near - off;
        high = near + off;
    };
    const int my_row = my < lists ? my / C : 0, my_chunk = my - my_row * C;
    const bool ended = live[my_row] == 2;
    const bool exists = my < lists && (ended ? my_chunk == 0 && score[my_row] != -INFINITY : live[my_row] == 1 && head_key != 0u);
    float low = -INFINITY, high = -INFINITY;
    if (exists) {
        if (ended) low = high = score[my_row];
        else bounds(my_row, head_key >> 16, low, high);
    }
    const auto order_low = [](float low) {  // a lower end in order; 0 is none's
        const unsigned x = low == low ? __float_as_uint(low) : 0xFF800000u;
        return x ^ ((x >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    };
    // (the n-th largest of the best 2 n or more, of a few from each warp that has lists: what is reached by n of them is
    // reached.  Not where there are 64 candidates at most: one list of 32, 15.1 us with and 9.6 without; 21 lists of 4, 7.7
    // and 9.2 us; eight lists of 32, 12.1 us, and 16.2 with no more than four of a list)
    const int W = min(kJoinThreads / 32, lists), r = lists * n <= 64 ? 0 : min(32, (2 * n + W - 1) / W);
    unsigned left = exists ? order_low(low) : 0u;
    uint4 next = ahead;
    int depth = 0;
    for (int i = 0; i < r && warp < W; ++i) {
        const unsigned m = __reduce_max_sync(0xffffffffu, left);
        const unsigned who = __ballot_sync(0xffffffffu, left == m);
        if (lane == 0) head[warp * r + i] = m;
        if (m != 0u && lane == __ffs(who) - 1) {
            ++depth;
            next = make_uint4(next.y, next.z, next.w, 0u);
            left = 0u;
            if (depth < n && !ended) {  // (a list has n)
                if (depth % 4 == 0) next = *reinterpret_cast<const uint4*>(my_cand + depth);
                if (next.x != 0u) {
                    float lo, hi;
                    bounds(my_row, next.x >> 16, lo, hi);
                    left = order_low(lo);
                }
            }
        }
    }
    if (tid == 0) reach = 0u;
    __syncthreads();
    if (tid < W * r && head[tid] != 0u) {
        const unsigned mine = head[tid];
        int above = 0;
#pragma unroll 4
        for (int i = 0; i < W * r; ++i) above += head[i] > mine || (head[i] == mine && i < tid);
        if (above == n - 1) reach = mine;
    }
    __syncthreads();
    const float need = reach ? __uint_as_float(reach ^ ((reach >> 31) ? 0x80000000u : 0xFFFFFFFFu)) : -INFINITY;
    // The candidates that reach it: each list's thread looks at the first four.  Where they all do, eight lanes look at the rest
    // together, since one thread would wait for every four of them (32 kept of each of 64 small rows: 13.2 us, 10.7
    // so).
    const auto keep = [&](unsigned v, int list_row, int list_chunk) {
        const int e = atomicAdd(&n_final, 1);
        if (e < kFinal) {
            cand[e] = v;
            from[e] = list_row << 16 | list_chunk;
        }
    };
    const auto keep_four = [&](const uint4& four, int i, int list_row, int list_chunk, float least) {
        const unsigned v[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            if (i + k >= n || v[k] == 0u) return false;
            bounds(list_row, v[k] >> 16, lo, hi);
            if (hi < least) return false;  // as are those after it
            keep(v[k], list_row, list_chunk);
        }
        return true;
    };
    const auto gather = [&](bool mine, float least) {
        if (mine) {
            if (ended) keep(0u, my_row, my_chunk);
            else if (keep_four(ahead, 0, my_row, my_chunk, least) && n > 4) deep[atomicAdd(&n_deep, 1)] = (unsigned short)my;
        }
        __syncthreads();
        const int D = n_deep;
        for (int j = tid / 8; j < D; j += kJoinThreads / 8) {
            const int list = deep[j], i = 4 + (tid & 7) * 4;
            if (i < n)
                keep_four(*reinterpret_cast<const uint4*>(a.cand + (size_t)(row0 * C + list) * kMaxOut + i), i, list / C,
                          list % C, least);
        }
        if (D > 0) __syncthreads();
    };
    const auto exact = [&](int b, unsigned v) {
        return live[b] == 2 ? order_of((double)score[b]) : score_at(b, v >> 16);
    };
    gather(exists && !(high < need), need);
    if (n_final > kFinal) {
        // Scores without a difference to speak of: by the heads' exact scores.  A list is left unless n heads, hence n
        // candidates, come before all of it, by score or row (so n - 1 lists are left and those of one more row,
        // which are equal), or n heads of its own row do, by logit.
        const unsigned long long mine = exists ? exact(my_row, head_key) : 0ull;
        key[my] = mine;
        cand[my] = head_key;
        __syncthreads();
        if (tid == 0) n_final = n_deep = 0;
        int above = 0, own = 0;
        for (int i = 0; i < lists; ++i) {
            above += key[i] > mine || (key[i] == mine && i / C < my_row);
            own += i / C == my_row && i != my && key[i] != 0ull &&
                   (cand[i] >> 16 > head_key >> 16 || (cand[i] >> 16 == head_key >> 16 && i < my));
        }
        __syncthreads();
        gather(exists && above < n && own < n, -INFINITY);
    }
    const int L = n_final;
    for (int e = tid; e < L; e += kJoinThreads) {
        const int b = from[e] >> 16;
        key[e] = exact(b, cand[e]);
        place[e] = (unsigned)b << kIdBits |
                  (live[b] == 2 ? (unsigned)a.eos : (unsigned)(from[e] & 0xFFFF) * kChunk + (0xFFFFu - (cand[e] & 0xFFFFu)));
    }
    __syncthreads();
#pragma unroll 1
    for (bool again = false;; again = true) {
        bool odd = false;  // different logits of a row have equal scores
        for (int e0 = 0; e0 < L; e0 += kJoinThreads / 8) {  // eight lanes to a candidate
            const int e = e0 + tid / 8;
            const unsigned long long k = e < L ? key[e] : 0ull;
            const unsigned f = e < L ? place[e] : 0u;
            int at = 0;
            if (e < L)
#pragma unroll 4
                for (int i = tid & 7; i < L; i += 8) {
                    const unsigned long long o = key[i];
                    at += o > k;
                    if (o == k) {
                        at += place[i] < f;
                        odd = odd || (place[i] >> kIdBits == f >> kIdBits && cand[i] >> 16 != cand[e] >> 16);
                    }
                }
            at += __shfl_xor_sync(0xffffffffu, at, 1);
            at += __shfl_xor_sync(0xffffffffu, at, 2);
            at += __shfl_xor_sync(0xffffffffu, at, 4);
            if (k && (tid & 7) == 0 && at < n) {
                const int id = (int)(f & ((1u << kIdBits) - 1u)), b = (int)(f >> kIdBits);
                a.ids[g * n + at] = id;
                a.parents[g * n + at] = row0 + b;
                a.out_scores[g * n + at] = (float)score_of(k);
                if (a.out_done) a.out_done[g * n + at] = live[b] == 2 || id == a.eos;
            }
        }
        if (!__syncthreads_or(odd) || again) break;
        // a row offers its n largest logits: the others are none
        for (int e = tid; e < L; e += kJoinThreads) {
            int larger = 0;
            for (int i = 0; i < L; ++i)
                larger += place[i] >> kIdBits == place[e] >> kIdBits &&
                          (cand[i] >> 16 > cand[e] >> 16 || (cand[i] >> 16 == cand[e] >> 16 && place[i] < place[e]));
            if (larger >= n) key[e] = 0ull;
        }
        __syncthreads();
    }
    if (tid >= L && tid < n) {  // no candidate
        a.ids[g * n + tid] = a.parents[g * n + tid] = -1;
        a.out_scores[g * n + tid] = -INFINITY;
        if (a.out_done) a.out_done[g * n + tid] = 0;
    }
}

}  // namespace

cudaError_t launch(const Args& a, int sms, cudaStream_t st, bool pdl) {
    if (a.V % 8 != 0 || a.chunks > kMaxChunks) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(a.chunks, a.groups * a.beams);
    const bool alone = a.groups * a.beams * a.chunks <= sms;
    c.blockDim = dim3(alone ? 512 : 256);
    c.stream = st;
    c.attrs = attr;
    c.numAttrs = pdl ? 1 : 0;
    if (cudaError_t e = cudaLaunchKernelEx(&c, alone ? chunk_kernel<512> : chunk_kernel<256>, a)) return e;
    c.gridDim = dim3(a.groups);
    c.blockDim = dim3(kJoinThreads);
    c.numAttrs = 1;  // it waits for the chunks' end, and its stream has nothing else before it
    return cudaLaunchKernelEx(&c, join_kernel, a);
}

}  // namespace beam
}  // namespace tfl
