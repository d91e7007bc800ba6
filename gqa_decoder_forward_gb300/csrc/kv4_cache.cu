// Writing rows into the 4-bit cache and reading them back (layout and formula:
// kv4.cuh).  Most of the bytes are the dense side's (256 of a row of 128 bf16
// numbers against 72 held), of which a lane moves 16 at a time.
//
// Write: sixteen lanes take a head's key or value of a row: a lane loads eight bf16
// numbers, eight lanes find their group's minimum and maximum by shuffles, and each
// lane writes one 32-bit word of codes.  One token costs a launch (1.8 us in a graph);
// 2,048 rows of 8 heads (10.7 MB, 1.6 us of transfer) some 6 us: 303 instructions of a
// warp for two such row-heads, two in five of them on the half-rate pipes, and one load of a
// lane in flight.  Key and value in one lane share the index work but cost one token 0.7 us more.
// Read: a warp takes 16 positions of a block (1,152 contiguous bytes of the cache,
// half a block), a half warp a row at a time; a lane holds one word of eight rows, all in flight.
// 131,072 positions of 8 heads (688 MB): 101 us, 6.8 TB/s, what a copy takes; 8,192
// positions (43 MB): 8.7 us, 4.9 TB/s, the rest being launch and ramp.  (A warp per row:
// 196 us for the former.)
#include "kv4.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;   // of a CTA of the write, of one head's keys or values
constexpr float kRound = 12582912.f;   // 1.5 * 2^23, in bits 0x4b400000
constexpr uint32_t kRoundCodes = 0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8);  // (<< 12 and more: 0)

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight numbers x8 (loaded: raw) of a row to the half block hb.  All lanes of the warp call it.
__device__ __forceinline__ void write8(const bf16* x8, const uint4& raw, char* hb, int pos, bool live) {
    const int lane = threadIdx.x & 15;
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_f(w[i]);
        f[2 * i + 1] = hi_f(w[i]);
    }
    // (maximum, -minimum) of the group, two bf16 numbers in a word; a NaN stays one
    auto b2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    auto u2 = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
    auto most = [&](uint32_t x, uint32_t y) { return u2(__hmax2_nan(b2(x), b2(y))); };
    const uint32_t hi = most(most(w[0], w[1]), most(w[2], w[3]));
    const uint32_t lo = u2(__hmin2_nan(__hmin2_nan(b2(w[0]), b2(w[1])), __hmin2_nan(b2(w[2]), b2(w[3])))) ^ 0x80008000u;
    uint32_t m = most(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = most(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mn = -hi_f(m), span = lo_f(m) - mn;
    const bool bad = !(span < INFINITY);  // a NaN or an infinity in the group, or too wide
    const bf16 scale = rn(span / 15.f);
    const float sc = bf(scale);
    uint32_t code = 0;
    if (!bad && sc > 0.f) {
        // n = round_half_even((x - zero) / scale) by the reciprocal, as the low bits of 1.5 2^23 + n.  The
        // quotient's error, 2^-21 of at most 16, can only change n within 2^-17 of a half: there, and for
        // scales whose reciprocal overflows or that are so coarse that n could pass 15, the lane divides.
        const float r = __fdividef(1.f, sc);  // 0 where it overflows or nearly does
        bool near = !(sc >= 1.17549435e-38f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = f[i] - mn, u = fmaf(d, r, kRound), rest = fmaf(kRound - u, sc, d);
            near |= !(fabsf(rest) < 0.4999f * sc);
            code += __float_as_uint(u) << (4 * i);  // 0x4b400000 + n, whose sum comes off below
        }
        code -= kRoundCodes;
        if (near) {
            code = 0;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const float x = bf(x8[i]);  // read again: the lanes that come here are few
                const float q = fminf(rintf((x - mn) / sc), 15.f);  // x >= mn: not below 0
                code |= (uint32_t)q << (4 * i);
            }
        }
    }
    if (live) {
        *reinterpret_cast<uint32_t*>(hb + word_at(pos, lane & 7, lane >> 3)) = code;
        if ((lane & 7) == 0) {
            const uint32_t sb = bad ? 0u : (uint32_t)__bfloat16_as_ushort(scale);
            const uint32_t zb = bad ? 0x7fc0u : __float_as_uint(mn) >> 16;  // a bf16 number: exact
            *reinterpret_cast<uint32_t*>(hb + kMetaOff + (pos % kBlockPos) * kMetaBytes + (lane >> 3) * 4) =
                sb | (zb << 16);
        }
    }
}

__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteArgs a) {
    const int row = blockIdx.x * kRows + threadIdx.x / 16, lane = threadIdx.x & 15;
    const bool live = row < a.rows.n_rows;  // whole half-warps; the others take part in the shuffles
    const int r = min(row, a.rows.n_rows - 1), h = blockIdx.y >> 1, kind = blockIdx.y & 1;
    const int s = stream_of(a.rows, r);
    const int pos = a.rows.pos0[s] + (r - a.rows.row_start[s]);
    const long src = (a.wrap ? 2l * kPage * s + pos % kPage : r) * a.ld + (long)h * kHeadDim + lane * 8;
    const bf16* x8 = (kind ? a.v : a.k) + src;
    pdl_wait();  // memory from here on
    pdl_trigger();
    const uint4 raw = *reinterpret_cast<const uint4*>(x8);
    const View& kv = a.rows.kv[s];
    const unsigned page = page_of(kv, pos);
    write8(x8, raw, half_block(tile(kv, a.rows.layer, a.rows.n_kv, page, h), pos, kind), pos, live && page < (unsigned)kv.n_pages);
}

// Two bf16 numbers, each z + s n rounded once to fp32 and then to bf16.
__device__ __forceinline__ uint32_t two(uint32_t code, int i, float s, float z) {
    const float x = fmaf((float)((code >> (8 * i)) & 15u), s, z), y = fmaf((float)((code >> (8 * i + 4)) & 15u), s, z);
    __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&p);
}

// A warp per (block that a stream's rows touch, head, keys or values).
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 7, j = (lane >> 3) & 1;
    const int n_kv = a.rows.n_kv;
    int item = (int)((blockIdx.x * kThreads + threadIdx.x) / 32);
    const int kind = item & 1;
    item >>= 1;
    int s = 0;
    while (s + 1 < a.rows.n_streams && item >= a.item_start[s + 1]) ++s;
    item -= a.item_start[s];
    const bool none = s == a.rows.n_streams - 1 && item >= a.item_start[s + 1] - a.item_start[s];
    pdl_wait();  // memory from here on
    pdl_trigger();
    if (none) return;
    const int h = (int)((unsigned)item % (unsigned)n_kv), b = (int)((unsigned)item / (unsigned)n_kv);
    const int r0 = a.rows.row_start[s], pos0 = a.rows.pos0[s], end = pos0 + a.rows.row_start[s + 1] - r0;
    const int p0 = pos0 / kBlockPos * kBlockPos + b * kBlockPos;  // the block's first position
    const char* hb = half_block(tile(a.rows.kv[s], a.rows.layer, n_kv, page_of(a.rows.kv[s], p0), h), p0, kind);
    uint32_t code[8], meta[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // rows i * 2 + half: what was never written is read but not used
        const int r = 2 * i + half;
        code[i] = load_once(hb + word_at(r, c, j));
        meta[i] = load_word(hb + kMetaOff + r * kMetaBytes + j * 4);
    }
    bf16* out = (kind ? a.v : a.k) + (long)h * kHeadDim + j * 64 + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int p = p0 + 2 * i + half;
        if (p < pos0 || p >= end) continue;
        const float sc = lo_f(meta[i]), z = hi_f(meta[i]);
        uint4 o;
        o.x = two(code[i], 0, sc, z);
        o.y = two(code[i], 1, sc, z);
        o.z = two(code[i], 2, sc, z);
        o.w = two(code[i], 3, sc, z);
        __stcs(reinterpret_cast<uint4*>(out + (long)(r0 + p - pos0) * a.ld), o);
    }
}

__global__ void __launch_bounds__(kThreads) identity_kernel(int* table, int n) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) table[i] = i;
}

cudaLaunchConfig_t cfg(long blocks, cudaStream_t st, cudaLaunchAttribute* attr, bool pdl) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)blocks);
    c.blockDim = dim3(kThreads);
    c.stream = st;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = attr;
        c.numAttrs = 1;
    }
    return c;
}

}  // namespace

cudaError_t launch_write(const WriteArgs& a, cudaStream_t st, bool pdl) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t c = cfg((a.rows.n_rows + kRows - 1) / kRows, st, attr, pdl);
    c.gridDim.y = 2 * a.rows.n_kv;
    return cudaLaunchKernelEx(&c, write_kernel, a);
}

cudaError_t launch_read(ReadArgs& a, cudaStream_t st, bool pdl) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    int items = 0;
    for (int s = 0; s < a.rows.n_streams; ++s) {
        const int R = a.rows.row_start[s + 1] - a.rows.row_start[s], p = a.rows.pos0[s];
        a.item_start[s] = items;
        if (R > 0) items += ((p + R - 1) / kBlockPos - p / kBlockPos + 1) * a.rows.n_kv;
    }
    a.item_start[a.rows.n_streams] = items;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t c = cfg(((long)items * 2 * 32 + kThreads - 1) / kThreads, st, attr, pdl);
    return cudaLaunchKernelEx(&c, read_kernel, a);
}

cudaError_t launch_identity(int* table, int n, cudaStream_t st) {
    identity_kernel<<<(n + kThreads - 1) / kThreads, kThreads, 0, st>>>(table, n);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace tfl
