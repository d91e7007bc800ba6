// Attention of one new token per stream over a prefix cache that a group of streams
// shares and a tail cache of each stream's own: softmax(q k / sqrt(128)) v over the keys of
// both.  A group's queries of a KV head (streams x n_q / n_kv, at most 128 rows) are one
// operand of the tensor cores, so that the prefix is read once for all of them.
//
// Work is cut into units: a KV head's run of 128-key blocks of one prefix, with all rows of its
// group, or of one stream's tail, with that stream's rows.  A unit's length follows from its own
// cache's length alone, so that a row's result does not depend on the other streams of the call.
// Units leave (m, l, O) per row, which a second kernel joins in a fixed order:
// out = sum_u 2^(m_u - M) O_u / sum_u 2^(m_u - M) l_u.
//
// Persistent CTAs, one per SM, take units one after the other (tails first, then prefixes, the longest
// units before shorter ones).  256 threads:
//   warps 0-3  softmax, a thread per row (tensor-memory lane);
//   warp 4, 6  keys and values by TMA, a block = one cache page, rings of two and three;
//   warp 5     tensor memory and the MMAs: S = Q K^T (M = 128 rows, N = 128 keys) into one of two buffers,
//              one block ahead, then O += P V with the weights read from where the softmax wrote them over S;
//   warp 7     queries, a unit ahead.
// So loads, products and softmax of neighbouring blocks and units overlap.
//
// The softmax is the prompt attention's: a row keeps a reference m that moves only when a
// block's maximum exceeds it by 2^8; weights enter P V as hi = bf16(p) and lo = bf16(p - hi), so
// that they are not rounded to bf16 (two roundings to nearest leave 2^-17 of p); sums are fp32.
// O_hi = sum hi V and O_lo = sum lo V are accumulated apart and added at the end.  A unit of at
// most 64 rows has its queries twice, in rows r and 64 + r: the former give hi, the latter lo, and
// one product of 128 rows does for both, with the same bits as two (8 beams after 131,072 keys: 85 us, 98 with two products;
// 16 streams on four prompts of 300 to 31,999: 49.5 and 59.8; measured before the last steps).
//
// Bound and measured (33B heads: 56 on 8, one layer, replayed from a graph).  Eight beams after 131,072 keys: 83.5 us, 539 MB at
// 6.5 TB/s, 95% of a copy; the memory bounds it (a block's products take 1,800 cycles of the 2,950 that it takes to come).
// 16 beams after as many: 99 us; 112 rows' weights, which one warp per scheduler makes, take a little longer than their block.
// 16 beams 100 tokens after 8,192 keys: 20.3 us for 40.6 MB (6.0 us): three to four blocks per SM, of which the
// first comes after 4 us of launch, queries and page table, and the last weights, products, partials (8 MB, written and read) and
// the join follow one another.  Four beams 17 tokens after 1,000: 8.5 us, latency alone.
//   Tried: a CTA per unit with two halves of a row in two warpgroups (33 us for the 16 beams), units shared out evenly by their
// blocks over all caches (no gain, and a row's bits would depend on the others), several tails in one product (another
// stream's values times a weight of 0 are NaN where they are not finite).
#include <algorithm>

#include "pair.cuh"
#include "shared_attn.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace tfl {
namespace shared {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyWarp = 4, kMmaWarp = 5, kValueWarp = 6, kQueryWarp = 7;
constexpr int kBN = kPage;                // keys of a block
constexpr int kBox = 128 * 64 * 2;        // 16 KB: 128 rows x 64 columns, 128-byte swizzle
constexpr int kTile = 2 * kBox;
constexpr int kTmemCols = 512;            // two S / P, O_hi, O_lo: 128 columns each
constexpr float kScale = 0.12751743074640502f;  // log2(e) / sqrt(128)
constexpr float kRescale = 8.f;
constexpr int kKStages = 2, kVStages = 3;  // scores are a block ahead of outputs, so keys leave earlier

constexpr int kOffQ = 0, kOffK = 2 * kTile, kOffV = kOffK + kKStages * kTile, kOffBar = kOffV + kVStages * kTile;
constexpr int kBarBytes = 512;
constexpr int kSmem = 1024 + kOffBar + kBarBytes;

// A unit: blocks [b0, b0 + nb) of a segment whose valid keys are [lo, hi), for `rows` rows of a KV head from stream0 on.
struct Unit {
    int seg, head, stream0, rows;
    int b0, nb, lo, hi;
    int at;  // first partial row
};

struct Bars {
    uint64_t q_full[2], o_free[2];            // by item: queries in place; outputs read
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t v_clean[kVStages];               // of a block with values to be zeroed: done
    uint64_t s_full[2], p_full[2], o_full[2];  // by block: scores; weights; outputs
    uint64_t drain;
    Unit unit[2];                             // by unit: what it is, in place with its queries
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier area");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// A bounded wait (tma.cuh's mbar_wait, with the call's limit) that also ends when another role has given up.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, const UnitArgs& a, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1; i < a.spin_limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0u && (*abort || global_ns() - t0 > kMbarWaitNs)) break;
    }
    if (!*abort) atomicOr(a.status, kStatusDevice);
    *abort = 1;
    return false;
}

// 32 columns of the warp's tensor-memory lanes, a lane to a thread; not in r before tmem_ld_wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for the thread's tensor-memory loads; r, which they fill, is not used before.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[N]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A page table's entry.  (Tables are written when caches are made and never again.)
__device__ __forceinline__ int table_entry(const Seg& v, int page) {
    int x;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(x) : "l"(v.table + page) : "memory");
    return min(max(x, 0), v.n_pages - 1);
}

// x / d as the upper half of x * per; per = 2^32 / d, rounded up (0: d is 1), right for x and d below 2^16.
__device__ __forceinline__ int over(int x, unsigned per) { return per ? (int)__umulhi((unsigned)x, per) : x; }

__device__ __forceinline__ Unit unit_of(const UnitArgs& a, int it) {
    Unit x;
    int c = 0;
    while (c + 1 < a.n_segs && it >= a.seg[c + 1].item0) ++c;
    const Seg& s = a.seg[c];
    const int u = it - s.item0, unit = over(u, a.per_head);
    x.seg = c;
    x.head = u - unit * a.n_kv;
    x.stream0 = s.stream0;
    x.rows = s.rows;
    x.lo = s.lo;
    x.hi = s.hi;
    x.at = s.row0 + (x.head * s.units + unit) * s.rows;
    x.b0 = unit * s.len;
    x.nb = min(s.len, (s.hi + kBN - 1) / kBN - x.b0);
    return x;
}
__device__ __forceinline__ bool whole_block(const Unit& x, int b) {
    const int k0 = (x.b0 + b) * kBN;
    return k0 >= x.lo && k0 + kBN <= x.hi;
}

// Loads of one kind of a CTA's blocks into its ring, with what a page table says.
struct Loader {
    const UnitArgs& a;
    Bars& b;
    uint64_t *full, *empty;
    unsigned char* ring;
    int stages, kind;
    volatile int* abort;
    long long issued = 0;

    // The unit's next block: waits for its stage, then two boxes.  Returns whether it went on.
    __device__ __forceinline__ bool load(const Unit& x, int page) {
        const int st = (int)(issued % stages);
        if (issued >= stages && !await(&empty[st], (uint32_t)(issued / stages - 1) & 1u, a, abort)) return false;
        const CUtensorMap* map = &a.map[x.seg];
        const int row0 = ((a.layer * 2 + kind) * a.seg[x.seg].n_pages + page) * kPage;
        const uint64_t once = policy_evict_first();
        mbar_arrive_expect_tx(&full[st], kTile);
        tma_load_3d(ring + st * kTile, map, 0, x.head, row0, &full[st], once);
        tma_load_3d(ring + st * kTile + kBox, map, 64, x.head, row0, &full[st], once);
        ++issued;
        return true;
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Weights 2^(s log2(e) / sqrt(128) - ref) of a row's 128 scores at tensor-memory address at, written over them 32 at a time:
// the parts of them that the thread has, hi in the first 16 columns and lo in the next (or in the first, if it has lo
// alone).  Adds the weights to ls (of a thread that has hi).
constexpr int kHi = 1, kLo = 2;
template <int Parts>
__device__ __forceinline__ void weights(uint32_t at, float ref, Pair (&ls)[2]) {
#pragma unroll 1
    for (int c = 0; c < kBN; c += 32) {
        uint32_t sc[32], hi[16], lo[16];
        tmem_ld32_async(at + c, sc);
        tmem_ld_done(sc);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const Pair x = pair_of(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
            const float2 y = parts_of(fma2(x, pair_of(kScale), pair_of(-ref)));
            const float2 p = make_float2(ex2(y.x), ex2(y.y));
            const Pair both = pair_of(p.x, p.y);
            if (Parts & kHi) ls[e / 2 & 1] = add2(ls[e / 2 & 1], both);
            const uint32_t h = pack_rn(p.x, p.y);
            hi[e / 2] = h;
            if (Parts & kLo) {
                const float2 left =
                    parts_of(fma2(pair_of(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u)), pair_of(-1.f), both));
                lo[e / 2] = pack_rn(left.x, left.y);
            }
        }
        if (Parts & kHi) tmem_st16(at + c, hi);
        if (Parts & kLo) tmem_st16(at + c + (Parts & kHi ? 16 : 0), lo);
    }
}

// Probe: the loader of a.lose (2 k: the keys of a CTA's block k, 2 k + 1: its values) stops there, as if it had broken.
template <bool Probe>
__global__ void __launch_bounds__(kThreads, 1) unit_kernel(const __grid_constant__ UnitArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& b = *reinterpret_cast<Bars*>(base + kOffBar);
    volatile int* abort = &b.abort;
    const uint32_t su = smem_u32(base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.q_full[i], 1);
            mbar_init(&b.o_free[i], 4);
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_full[i], 4);
            mbar_init(&b.o_full[i], 1);
        }
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&b.k_full[i], 1);
            mbar_init(&b.k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&b.v_full[i], 1);
            mbar_init(&b.v_empty[i], 1);
            mbar_init(&b.v_clean[i], 1);
        }
        mbar_init(&b.drain, 1);
        b.abort = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&b.tmem, kTmemCols);
        tmem_relinquish();
    }
    const Unit x0 = unit_of(a, blockIdx.x);
    if (threadIdx.x == kKeyWarp * 32) prefetch_map(&a.map[x0.seg]);
    if (threadIdx.x == kQueryWarp * 32) prefetch_map(&a.qmap[a.seg[x0.seg].qmap]);
    int first_pages = 0;
    if ((warp == kKeyWarp || warp == kValueWarp) && lane < x0.nb) first_pages = table_entry(a.seg[x0.seg], x0.b0 + lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    bool mma_any = false;
    pdl_wait();
    pdl_trigger();  // the join's CTAs may be set up where there is room

    if (warp == kKeyWarp || warp == kValueWarp) {
        // ---------------- keys / values ----------------
        const bool values = warp == kValueWarp;
        Loader ld{a, b, values ? b.v_full : b.k_full, values ? b.v_empty : b.k_empty,
                  base + (values ? kOffV : kOffK), values ? kVStages : kKStages, values ? 1 : 0, abort};
        bool ok = true, lost = false;
        Unit x = x0;
        for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            if (i != blockIdx.x) x = unit_of(a, i);
            int pages = first_pages;
            for (int j = 0; j < x.nb && ok; ++j) {
                if (j % 32 == 0 && j + lane < x.nb && (j > 0 || i != blockIdx.x)) pages = table_entry(a.seg[x.seg], x.b0 + j + lane);
                const int page = __shfl_sync(0xffffffffu, pages, j % 32);
                const int st = (int)(ld.issued % ld.stages);
                const uint32_t phase = (uint32_t)(ld.issued / ld.stages) & 1u;
                if (Probe && ld.issued * 2 + (values ? 1 : 0) == a.lose) {  // the rest never comes
                    lost = true;
                    ok = false;
                    break;
                }
                if (lane == 0) ok = ok && !*abort && ld.load(x, page);
                else ++ld.issued;
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
                // values outside the cache's valid keys: exact zeros (the cache there holds anything)
                if (values && ok && !whole_block(x, j)) {
                    ok = __all_sync(0xffffffffu, await(&ld.full[st], phase, a, abort));
                    const int k0 = (x.b0 + j) * kBN;
                    for (int t = lane; t < kBN * 8; t += 32) {
                        const int k = k0 + (t >> 3);
                        if (k >= x.lo && k < x.hi) continue;
                        const uint32_t at = su + kOffV + st * kTile + (t >> 3) * 128 + (t & 7) * 16;
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0u) : "memory");
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + kBox), "r"(0u) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.v_clean[st]);
                }
            }
        }
        if (!ok && !lost) *abort = 1;
        // the last copies land before the CTA exits, whether or not they were used
        if (lane == 0)
            drain_ring(ld.full, ld.stages, (int)(ld.issued % ld.stages), (uint32_t)(ld.issued / ld.stages) & 1u, ld.issued,
                       a.status);
    } else if (warp == kMmaWarp) {
        // ---------------- products ----------------
        // The whole warp runs the loop and one lane issues: so descriptors stay warp-wide values.
        constexpr uint32_t idS = idesc_bf16_f32(kRows, kBN);
        constexpr uint32_t idPV = idesc_bf16_f32_bmn(kRows, kHeadDim);
        const bool leader = elect_one();
        const uint64_t q_desc = sdesc_sw128(su + kOffQ), k_desc = sdesc_sw128(su + kOffK);
        const uint64_t v_desc = sdesc_sw128_mn(su + kOffV, kBox);
        uint32_t n = 0, it = 0, cleaned = 0;                              // blocks and units so far; a bit per stage of values
        bool ok = true;
        bool last_first = false, last_whole = true, last_paired = false;  // of block n - 1
        uint32_t last_it = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, await(bar, parity & 1u, a, abort)) != 0;
        };
        // O += P V of block m, the last one whose scores were issued
        auto outputs = [&](uint32_t m) {
            const uint32_t st = m % kVStages, buf = m & 1u;
            if (!wait(&b.v_full[st], m / kVStages)) return false;
            if (!last_whole) {
                if (!wait(&b.v_clean[st], cleaned >> st)) return false;
                cleaned ^= 1u << st;
            }
            // the last unit's outputs have been read
            if (last_first && last_it > 0 && !wait(&b.o_free[(last_it - 1) & 1u], (last_it - 1) >> 1)) return false;
            if (!wait(&b.p_full[buf], m >> 1)) return false;
            tc_fence_after();
            const uint64_t vd = v_desc + st * (kTile >> 4);
            const uint32_t pt = tmem + 128 * buf;
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    tc_mma_bf16_ta(tmem + 256, pt + 32 * (kk >> 1) + 8 * (kk & 1), vd + kk * 128, idPV,
                                   (!last_first || kk > 0) ? 1u : 0u);
                if (!last_paired)
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        tc_mma_bf16_ta(tmem + 384, pt + 32 * (kk >> 1) + 16 + 8 * (kk & 1), vd + kk * 128, idPV,
                                       (!last_first || kk > 0) ? 1u : 0u);
                tc_commit(&b.o_full[buf]);
                tc_commit(&b.v_empty[st]);
            }
            __syncwarp();
            return true;
        };
        for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x, ++it) {
            // a unit's last outputs do not wait for the next one's queries and keys
            if (n > 0) ok = outputs(n - 1);
            ok = ok && wait(&b.q_full[it & 1u], it >> 1);
            const Unit x = b.unit[it & 1u];
            for (int j = 0; j < x.nb && ok; ++j) {
                const uint32_t st = n % kKStages, buf = n & 1u;
                // the buffer's last weights have been used
                ok = !__any_sync(0xffffffffu, *abort) && (n < 2 || wait(&b.o_full[buf], (n >> 1) - 1)) &&
                     wait(&b.k_full[st], n / kKStages);
                if (!ok) break;
                tc_fence_after();
                const uint64_t qd = q_desc + (it & 1u) * (kTile >> 4), kd = k_desc + st * (kTile >> 4);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk) {
                        const uint32_t step = (kk >> 2) * (kBox >> 4) + (kk & 3) * 2;
                        tc_mma_bf16(tmem + 128 * buf, qd + step, kd + step, idS, kk > 0 ? 1u : 0u);
                    }
                    tc_commit(&b.s_full[buf]);
                    tc_commit(&b.k_empty[st]);
                }
                __syncwarp();
                mma_any = true;
                if (j > 0) ok = outputs(n - 1);
                last_first = j == 0;
                last_paired = x.rows <= 64;
                last_whole = whole_block(x, j);
                last_it = it;
                ++n;
            }
        }
        if (ok && n > 0) ok = outputs(n - 1);
        if (!ok) *abort = 1;
        if (mma_any && leader) {  // every MMA issued completes before tensor memory is freed, whoever has given up since
            tc_commit(&b.drain);
            mbar_wait(&b.drain, 0u, a.status);
        }
    } else if (warp == kQueryWarp) {
        // ---------------- queries ----------------
        // Rows (stream, head) side by side; a unit of at most 64 has them twice.  Rows past the unit's hold anything: what
        // they give is not read.
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            Unit x = x0;
            for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x, ++it) {
                if (it > 0) x = unit_of(a, i);
                const uint32_t buf = it & 1u;
                if (it >= 2 && (*abort || !await(&b.o_free[buf], ((it >> 1) - 1) & 1u, a, abort))) {
                    ok = false;
                    break;
                }
                const CUtensorMap* map = &a.qmap[a.seg[x.seg].qmap];
                const int y = x.head * over(a.n_q, a.per_head), times = x.rows <= 64 ? 2 : 1;
                const uint64_t keep = policy_evict_last();
                b.unit[buf] = x;
                mbar_arrive_expect_tx(&b.q_full[buf], (uint32_t)(times * x.rows * kHeadDim * 2));
                for (int k = 0; k < times; ++k) {
                    unsigned char* to = base + kOffQ + buf * kTile + k * (kBox / 2);
                    tma_load_3d(to, map, 0, y, x.stream0, &b.q_full[buf], keep);
                    tma_load_3d(to + kBox, map, 64, y, x.stream0, &b.q_full[buf], keep);
                }
            }
            if (!ok) *abort = 1;
            drain_ring(b.q_full, 2, (int)(it & 1u), (it >> 1) & 1u, it, a.status);
        }
    } else {
        // ---------------- softmax ----------------
        const int t = threadIdx.x;
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        uint32_t n = 0, it = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < a.items; i += gridDim.x, ++it) {
            if (ok && (*abort || !await(&b.q_full[it & 1u], (it >> 1) & 1u, a, abort))) ok = false;
            const Unit x = ok ? b.unit[it & 1u] : unit_of(a, i);
            const bool paired = x.rows <= 64, low = paired && t >= 64;
            const int row = paired ? t & 63 : t;
            const bool warp_in = (paired ? warp & 1 : warp) * 32 < x.rows;  // the warp has rows of the unit
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < x.nb; ++j, ++n) {
                const uint32_t buf = n & 1u, rS = tmem + lane_off + 128 * buf;
                if (ok && (*abort || !await(&b.s_full[buf], (n >> 1) & 1u, a, abort))) ok = false;
                tc_fence_after();
                if (warp_in) {
                    // Two passes over the scores, 32 at a time, in loops: code that runs once is fetched slower than it runs,
                    // and many units have one block.
                    const int k0 = (x.b0 + j) * kBN;
                    const bool whole = k0 >= x.lo && k0 + kBN <= x.hi;
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < kBN; c += 32) {
                        uint32_t sc[32];
                        tmem_ld32_async(rS + c, sc);
                        tmem_ld_done(sc);
                        if (!whole) {  // keys outside the cache's valid ones: score -inf, hence weight 0
                            const int from = x.lo - (k0 + c), to = x.hi - (k0 + c);
                            uint32_t keep = from >= 32 || to <= 0 ? 0u : ~0u << max(from, 0);
                            if (to < 32) keep &= (1u << max(to, 0)) - 1u;
#pragma unroll
                            for (int e = 0; e < 32; ++e) sc[e] = (keep >> e) & 1u ? sc[e] : 0xFF800000u;
                            tmem_st32(rS + c, sc);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            mq[e / 2 & 3] = max3(mq[e / 2 & 3], __uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
                    }
                    if (!whole) tmem_st_wait();
                    const float bmax = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * kScale;
                    const bool rescale = bmax > m + kRescale;
                    const float alpha = rescale ? ex2(m - bmax) : 1.f;
                    // (a row without weights so far has an output of zeros, whatever it is multiplied by)
                    if (j > 0 && __any_sync(0xffffffffu, rescale && m != -INFINITY)) {
                        if (ok && !await(&b.o_full[buf ^ 1u], ((n - 1) >> 1) & 1u, a, abort)) ok = false;
                        tc_fence_after();
                        const int columns = paired ? kHeadDim : 2 * kHeadDim;
#pragma unroll 1
                        for (int c = 0; c < columns; c += 16) {
                            float v[16];
                            tmem_ld16(tmem + lane_off + 256 + c, v);
                            uint32_t o[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e] * alpha);
                            tmem_st16(tmem + lane_off + 256 + c, o);
                        }
                    }
                    if (rescale) {
                        l *= alpha;
                        m = bmax;
                    }
                    const float ref = m == -INFINITY ? 0.f : m;  // nothing but -inf so far: weights of 0
                    Pair ls[2] = {0ull, 0ull};
                    if (!paired) weights<kHi | kLo>(rS, ref, ls);
                    else if (low) weights<kLo>(rS, ref, ls);
                    else weights<kHi>(rS, ref, ls);
                    const float2 l0 = parts_of(ls[0]), l1 = parts_of(ls[1]);
                    l += (l0.x + l0.y) + (l1.x + l1.y);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_full[buf]);
            }
            // the unit's outputs, O_hi + O_lo: dims in groups of four, rows side by side
            if (ok && (*abort || !await(&b.o_full[(n - 1) & 1u], ((n - 1) >> 1) & 1u, a, abort))) ok = false;
            tc_fence_after();
            float4* po = reinterpret_cast<float4*>(a.po) + (size_t)x.at * (kHeadDim / 4) + row;
            const auto put = [&](int d, const uint32_t* u, const uint32_t* w) {  // dims 4 d .. 4 d + 3
                float4 v;
                v.x = __uint_as_float(u[0]) + __uint_as_float(w[0]);
                v.y = __uint_as_float(u[1]) + __uint_as_float(w[1]);
                v.z = __uint_as_float(u[2]) + __uint_as_float(w[2]);
                v.w = __uint_as_float(u[3]) + __uint_as_float(w[3]);
                po[(size_t)d * x.rows] = v;
            };
            if (paired) {
                // Of a row that is held twice, one thread adds dims 0-63 and the other 64-127: each hands the other's over
                // in the queries' place (their products have ended).
                uint4* given = reinterpret_cast<uint4*>(base + kOffQ + (it & 1u) * kTile) + row;
                const int own = low ? 64 : 0;
                uint32_t mine[64];
                if (warp_in) {
                    uint32_t v[64];
                    tmem_ld64_async(tmem + lane_off + 256 + (64 - own), v);
                    tmem_ld64_async(tmem + lane_off + 256 + own, mine);
                    tmem_ld_done(v);
                    tmem_ld_done(mine);
#pragma unroll
                    for (int d = 0; d < 16; ++d)
                        given[((64 - own) / 4 + d) * 64] = make_uint4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
                }
                named_barrier(1, 128);
                if (warp_in && row < x.rows) {
#pragma unroll
                    for (int d = 0; d < 16; ++d) {
                        const uint4 v = given[(own / 4 + d) * 64];
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        put(own / 4 + d, mine + 4 * d, w);
                    }
                }
            } else if (warp_in) {
#pragma unroll 1
                for (int c = 0; c < kHeadDim; c += 32) {
                    uint32_t hi[32], lo[32];
                    tmem_ld32_async(tmem + lane_off + 256 + c, hi);
                    tmem_ld32_async(tmem + lane_off + 384 + c, lo);
                    tmem_ld_done(hi);
                    tmem_ld_done(lo);
                    if (row < x.rows) {
#pragma unroll
                        for (int d = 0; d < 8; ++d) put(c / 4 + d, hi + 4 * d, lo + 4 * d);
                    }
                    __syncwarp();
                }
            }
            if (warp_in) {
                if (!low && row < x.rows) {
                    a.pm[x.at + row] = m;
                    a.pl[x.at + row] = l;
                }
            }
            tc_fence_before();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the next queries come over what was handed over
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.o_free[it & 1u]);
        }
        if (!ok) *abort = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- join ---------------------------------------------------------------------------------

constexpr int kJoinRows = 8;   // rows of a CTA: eight neighbouring rows of a unit are 128 bytes of each group of four dims
constexpr int kJoinThreads = kJoinRows * kHeadDim / 4;
constexpr int kFewUnits = 32, kMostUnits = 160;  // of a cache and head; a row has two caches

// A CTA takes eight rows of a (group, KV head) and an equal part of their dims, of Split parts.  A warp per row finds its
// units' weights; then a thread per (row, four dims) adds every Split-th unit in order, the prefix's first, and the
// Split sums are added in order.  The first outputs are asked for before the weights are known.
//   Split: 1 where the model's caches have few units, 8 where they have many, so that they are read by more SMs and in fewer
// round trips (one KV head, 16 streams after 131,072 keys, 147 units: 70 us with 1, 30 with 8; eight KV heads, 16 streams after
// 8,192, 17 units: 20.8 with 1, 24.0 with 8).
template <int Split>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ JoinArgs a) {
    constexpr int kDims = kHeadDim / 4 / Split;                                 // groups of four dims of a CTA
    constexpr int kBatch = Split == 1 ? 20 : 10;                                // outputs that a thread asks for at a time
    constexpr int kLaneUnits = 2 * (Split == 1 ? kFewUnits : kMostUnits) / 32;  // weights of a lane
    __shared__ float4 sums[Split == 1 ? 1 : kJoinThreads];
    extern __shared__ float weights[];  // [max_units][rows]
    const int G = a.n_q / a.n_kv, head = blockIdx.y;
    int g = 0, chunk = blockIdx.x;
    for (;; ++g) {
        const int chunks = ((a.first[g + 1] - a.first[g]) * G + kJoinRows - 1) / kJoinRows;
        if (chunk < chunks) break;
        chunk -= chunks;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = (a.first[g + 1] - a.first[g]) * G, up = a.p_units[g];
    const int p_row = a.p_row[g] + head * up * rows;
    const int part = threadIdx.x / (kJoinRows * kDims), k = threadIdx.x % kJoinRows;
    const int d = blockIdx.z * kDims + threadIdx.x / kJoinRows % kDims, r = min(chunk * kJoinRows + k, rows - 1);
    const int s = a.first[g] + r / G, i = r % G, tu = a.t_units[s], n = up + tu;
    const float4* po = reinterpret_cast<const float4*>(a.po);
    const float4* p_out = po + (size_t)p_row * 32 + (size_t)d * rows + r;
    const float4* t_out = po + (size_t)(a.t_row[s] + head * tu * G) * 32 + (size_t)d * G + i;
    const size_t p_step = (size_t)rows * 32, t_step = (size_t)G * 32;
    pdl_wait();
    pdl_trigger();
    float4 v[kBatch];
    const auto ask = [&](int u0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int u = u0 + j * Split;
            if (u < n) v[j] = __ldcg(u < up ? p_out + u * p_step : t_out + (u - up) * t_step);
        }
    };
    ask(part);
    const int wr = chunk * kJoinRows + warp;
    if (wr < rows) {
        const int ws = a.first[g] + wr / G, wn = up + a.t_units[ws];
        const int t_row = a.t_row[ws] + head * a.t_units[ws] * G + wr % G;
        float m[kLaneUnits], l[kLaneUnits], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int j = 0; j < kLaneUnits; ++j) {
            const int u = lane + 32 * j, at = u < up ? p_row + u * rows + wr : t_row + (u - up) * G;
            m[j] = u < wn ? __ldcg(a.pm + at) : -INFINITY;
            l[j] = u < wn ? __ldcg(a.pl + at) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kLaneUnits; ++j) M = fmaxf(M, m[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int j = 0; j < kLaneUnits; ++j)
            if (lane + 32 * j < wn) {
                m[j] = ex2(m[j] - M);
                L = fmaf(m[j], l[j], L);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
        for (int j = 0; j < kLaneUnits; ++j)
            if (lane + 32 * j < wn) weights[(lane + 32 * j) * kJoinRows + warp] = m[j] / L;
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u0 = part; u0 < n; u0 += kBatch * Split) {
        if (u0 > part) ask(u0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int u = u0 + j * Split;
            if (u >= n) break;
            const float x = weights[u * kJoinRows + k];
            o.x = fmaf(x, v[j].x, o.x);
            o.y = fmaf(x, v[j].y, o.y);
            o.z = fmaf(x, v[j].z, o.z);
            o.w = fmaf(x, v[j].w, o.w);
        }
    }
    if (Split > 1) {
        sums[threadIdx.x] = o;
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 1; p < Split; ++p) {
            const float4 x = sums[p * kJoinRows * kDims + threadIdx.x];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
    }
    if (chunk * kJoinRows + k < rows)
        *reinterpret_cast<uint2*>(a.out + (size_t)s * a.ldo + (size_t)(head * G + i) * kHeadDim + d * 4) =
            make_uint2(pack_rn(o.x, o.y), pack_rn(o.z, o.w));
}

// A unit has n blocks where the cache has at most this times n^2: a unit more costs the join about a 40th of a block's time, so that
// many heads' worth of SMs are not all used by one (one KV head, 10 streams after 18,962 keys, units of 1 | 2 | 3 blocks: 22.8 |
// 12.8 | 12.8 us; 4 after 30,000, 2 | 3 | 4: 13.9 | 11.7 | 12.1; 4 after 5,000, 1 | 2: 8.4 | 8.7).
constexpr int kUnitSquare = 48;
// Blocks of a tail's unit, at least.  Short units end soon where few tails are long; long ones leave fewer of them, in few rounds,
// where many are (eight KV heads, units of 1 | 2 | 4 blocks: one of five tails of 477 keys after 3,724 keys 15.7 | 16.8 | 19.7 us;
// eight of 700 after 1,000: 18.7 | 18.1 | 16.8; four of 4,000 alone: 23.2 | 23.1 | 20.1; one KV head, eight of 700: 7.8 | 9.0 |
// 11.5).
int tail_blocks(int blocks, int most) { return most > kFewUnits ? 1 : blocks <= 8 ? 2 : 4; }
// Units of a KV head that a cache is cut into at most: a CTA per SM over the heads.
int most_units(int n_kv, int sms) { return std::min(std::max(1, sms / n_kv), kMostUnits); }

}  // namespace

void plan(Call& call, int sms) {
    UnitArgs& a = call.unit;
    JoinArgs& j = call.join;
    const int G = a.n_q / a.n_kv, most = call.most_units = most_units(a.n_kv, sms);
    const auto per = [](int d) { return d == 1 ? 0u : (unsigned)((0xFFFFFFFFull + d) / d); };
    a.per_head = per(a.n_kv);
    a.n_segs = a.items = j.max_units = 0;
    a.lose = -1;
    a.spin_limit = kMbarSpinLimit;
    int row = 0;
    const auto add = [&](int cache, int stream0, int streams, int lo, int hi, bool tail) {
        const int blocks = (hi + kBN - 1) / kBN;
        if (blocks == 0) return 0;
        Seg& s = a.seg[a.n_segs++];
        s.cache = cache;
        s.qmap = cache < kMaxStreams && streams > 1 ? 1 + cache : 0;
        s.stream0 = stream0;
        s.rows = streams * G;
        s.lo = lo;
        s.hi = hi;
        s.len = std::max(tail ? tail_blocks(blocks, most) : 1, (blocks + most - 1) / most);
        while (kUnitSquare * s.len * s.len < blocks) ++s.len;
        s.units = (blocks + s.len - 1) / s.len;
        s.row0 = row;
        row += s.units * a.n_kv * s.rows;
        return s.units;
    };
    // Tails first: their work runs while the first keys and values of the prefixes come.  Then the longest units first.
    for (int g = 0; g < call.n_groups; ++g)
        for (int s = j.first[g]; s < j.first[g + 1]; ++s) {
            const int end = call.pos[s] + 1 - call.n_prefix[g] / kBN * kBN;
            const bool none = call.pos[s] + 1 == call.n_prefix[g];
            j.t_row[s] = row;
            j.t_units[s] = add(kMaxStreams + s, s, 1, call.n_prefix[g] % kBN, none ? 0 : end, true);
        }
    const int tails = a.n_segs;
    for (int g = 0; g < call.n_groups; ++g) {
        j.p_row[g] = row;
        j.p_units[g] = add(g, j.first[g], j.first[g + 1] - j.first[g], 0, call.n_prefix[g], false);
        for (int s = j.first[g]; s < j.first[g + 1]; ++s) j.max_units = std::max(j.max_units, j.p_units[g] + j.t_units[s]);
    }
    std::stable_sort(a.seg + tails, a.seg + a.n_segs, [](const Seg& x, const Seg& y) { return x.len > y.len; });
    for (int c = 0; c < a.n_segs; ++c) {
        a.seg[c].item0 = a.items;
        a.items += a.seg[c].units * a.n_kv;
    }
    call.grid = std::min(a.items, sms);
}

size_t max_partial_rows(int n_q, int n_kv, int streams, int sms) {
    return (size_t)2 * most_units(n_kv, sms) * streams * n_q;
}

cudaError_t init() {
    cudaError_t e = cudaFuncSetAttribute(unit_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return e ? e : cudaFuncSetAttribute(unit_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t launch(const Call& a, cudaStream_t st, bool pdl) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(a.grid);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kSmem;
    c.stream = st;
    c.attrs = attr;
    c.numAttrs = pdl ? 1 : 0;
    if (cudaError_t e = cudaLaunchKernelEx(&c, a.unit.lose >= 0 ? unit_kernel<true> : unit_kernel<false>, a.unit)) return e;
    const JoinArgs& j = a.join;
    int chunks = 0;
    for (int g = 0; g < a.n_groups; ++g)
        chunks += ((j.first[g + 1] - j.first[g]) * (j.n_q / j.n_kv) + kJoinRows - 1) / kJoinRows;
    const bool few = a.most_units <= kFewUnits;
    c.gridDim = dim3(chunks, j.n_kv, few ? 1 : 8);
    c.blockDim = dim3(kJoinThreads);
    c.dynamicSmemBytes = (size_t)kJoinRows * j.max_units * sizeof(float);
    c.numAttrs = 1;  // the units' end is all that it waits for
    return cudaLaunchKernelEx(&c, few ? join_kernel<1> : join_kernel<8>, j);
}

}  // namespace shared
}  // namespace tfl
