// Writing rows into the 4-bit cache and reading them back (layout and formula:
// kv4.cuh).  Sixteen lanes take one (row, head) of keys or values: a lane loads
// eight bf16 numbers (16 bytes), eight lanes find their group's minimum and
// maximum by shuffles, and each lane writes one 32-bit word of codes; the read
// goes the other way.
#include "kv4.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = kThreads / 16;  // (row, head) items of a CTA

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteArgs a) {
    pdl_wait();
    const int kind = blockIdx.y;
    const long item = (long)blockIdx.x * kItems + threadIdx.x / 16;
    const int lane = threadIdx.x & 15;
    const long n_items = (long)a.rows.n_rows * a.rows.n_kv;
    const bool live = item < n_items;  // whole half-warps; the others take part in the shuffles
    const long it = live ? item : n_items - 1;
    const int r = (int)(it / a.rows.n_kv), h = (int)(it % a.rows.n_kv);
    const int s = stream_of(a.rows, r);
    const int pos = a.rows.pos0[s] + (r - a.rows.row_start[s]);
    const long src = a.wrap ? 2l * kPage * s + pos % kPage : r;
    const bf16* x = (kind ? a.v : a.k) + src * a.ld + (long)h * kHeadDim + lane * 8;
    const uint4 raw = *reinterpret_cast<const uint4*>(x);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_f(w[i]);
        f[2 * i + 1] = hi_f(w[i]);
    }
    float mn = f[0], mx = f[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mn = fminf(mn, f[i]);
        mx = fmaxf(mx, f[i]);
        bad |= !(fabsf(f[i]) < INFINITY);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const unsigned bads = __ballot_sync(0xffffffffu, bad);
    bad = ((bads >> (threadIdx.x & 24)) & 0xffu) != 0;  // of this lane's eight
    const float span = mx - mn;
    bad |= !(span < INFINITY);
    const bf16 scale = rn(span / 15.f);
    const float sc = bf(scale);
    uint32_t code = 0;
    if (!bad && sc > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(rintf((f[i] - mn) / sc), 15.f);  // f >= mn: not below 0
            code |= (uint32_t)q << (4 * i);
        }
    }
    if (live) {
        char* hb = half_block(tile(a.rows.kv[s], a.rows.layer, a.rows.n_kv, pos, h), pos, kind);
        *reinterpret_cast<uint32_t*>(hb + word_at(pos, lane & 7, lane >> 3)) = code;
        if ((lane & 7) == 0) {
            const uint32_t sb = bad ? 0u : (uint32_t)__bfloat16_as_ushort(scale);
            const uint32_t zb = bad ? 0x7fc0u : __float_as_uint(mn) >> 16;  // a bf16 number: exact
            *reinterpret_cast<uint32_t*>(hb + kMetaOff + (pos % kBlockPos) * kMetaBytes + (lane >> 3) * 4) =
                sb | (zb << 16);
        }
    }
    pdl_trigger();
}

// Two bf16 numbers, each z + s n rounded once to fp32 and then to bf16.
__device__ __forceinline__ uint32_t two(uint32_t code, int i, float s, float z) {
    const float x = fmaf((float)((code >> (8 * i)) & 15u), s, z), y = fmaf((float)((code >> (8 * i + 4)) & 15u), s, z);
    __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&p);
}

__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    pdl_wait();
    const int kind = blockIdx.y;
    const long item = (long)blockIdx.x * kItems + threadIdx.x / 16;
    const int lane = threadIdx.x & 15;
    if (item < (long)a.rows.n_rows * a.rows.n_kv) {
        const int r = (int)(item / a.rows.n_kv), h = (int)(item % a.rows.n_kv);
        const int s = stream_of(a.rows, r);
        const int pos = a.rows.pos0[s] + (r - a.rows.row_start[s]);
        const char* hb = half_block(tile(a.rows.kv[s], a.rows.layer, a.rows.n_kv, pos, h), pos, kind);
        const uint32_t code = *reinterpret_cast<const uint32_t*>(hb + word_at(pos, lane & 7, lane >> 3));
        const uint32_t m =
            *reinterpret_cast<const uint32_t*>(hb + kMetaOff + (pos % kBlockPos) * kMetaBytes + (lane >> 3) * 4);
        const float sc = lo_f(m), z = hi_f(m);
        uint4 o;
        o.x = two(code, 0, sc, z);
        o.y = two(code, 1, sc, z);
        o.z = two(code, 2, sc, z);
        o.w = two(code, 3, sc, z);
        *reinterpret_cast<uint4*>((kind ? a.v : a.k) + (long)r * a.ld + (long)h * kHeadDim + lane * 8) = o;
    }
    pdl_trigger();
}

cudaLaunchConfig_t cfg(const Rows& r, cudaStream_t st, cudaLaunchAttribute* attr, bool pdl) {
    cudaLaunchConfig_t c = {};
    const long n = (long)r.n_rows * r.n_kv;
    c.gridDim = dim3((unsigned)((n + kItems - 1) / kItems), 2);
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
    cudaLaunchConfig_t c = cfg(a.rows, st, attr, pdl);
    return cudaLaunchKernelEx(&c, write_kernel, a);
}

cudaError_t launch_read(const ReadArgs& a, cudaStream_t st, bool pdl) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t c = cfg(a.rows, st, attr, pdl);
    return cudaLaunchKernelEx(&c, read_kernel, a);
}

}  // namespace kv4
}  // namespace tfl
