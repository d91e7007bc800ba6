// Attention over the 4-bit cache (layout and what a code stands for: kv4.cuh).
// Per (row, query head) at position p, over keys t = 0..p of its KV head:
//   s_t = (q . k_t) / sqrt(128),  P_t = e^(s_t - max s),  out = sum P_t v_t / sum P_t
// with k_t, v_t = zero + scale n unrounded, and everything in fp32.
//
// A CTA takes one page (128 keys) of one stream and KV head: a thread scores its
// key for every (row, head) pair of the group, then owns one output dim.  The
// partials (max, sum, output) of the pages are joined by a second kernel.
#include "kv4.cuh"

namespace tfl {
namespace kv4 {
namespace {

constexpr int kUnit = kPage;

__device__ __forceinline__ float meta_scale(uint32_t m) { return __uint_as_float(m << 16); }
__device__ __forceinline__ float meta_zero(uint32_t m) { return __uint_as_float(m & 0xffff0000u); }

__device__ __forceinline__ float block_reduce(float x, bool mx, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = mx ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    return mx ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) : (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ void __launch_bounds__(kPage) page_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float qs[kHeadDim], ps[kPage], red[4];
    pdl_wait();
    const Rows& m = a.rows;
    const int u = blockIdx.x, h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int r0 = m.row_start[s], R = m.row_start[s + 1] - r0, G = a.n_q / m.n_kv;
    const int k0 = u * kUnit, key = k0 + tid;
    if (R == 0 || k0 > m.pos0[s] + R - 1) return;
    char* t = tile(m.kv[s], m.layer, m.n_kv, k0, h);
    const char* hk = half_block(t, tid, 0);
    for (int c = 0; c < R * G; ++c) {
        const int r = r0 + c / G, hq = h * G + c % G, pos = m.pos0[s] + c / G;
        if (k0 > pos) continue;  // uniform
        __syncthreads();
        qs[tid] = bf(a.q[(long)r * a.ldq + hq * kHeadDim + tid]);
        __syncthreads();
        float sc = -INFINITY;
        if (key <= pos) {
            sc = 0.f;
            for (int j = 0; j < 2; ++j) {
                const uint32_t mt = *reinterpret_cast<const uint32_t*>(hk + kMetaOff + (tid % kBlockPos) * 8 + j * 4);
                float dot = 0.f, sum = 0.f;
                for (int ch = 0; ch < 8; ++ch) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(hk + word_at(tid, ch, j));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float qv = qs[j * 64 + ch * 8 + i];
                        dot = fmaf(qv, (float)((w >> (4 * i)) & 15u), dot);
                        sum += qv;
                    }
                }
                sc += meta_scale(mt) * dot + meta_zero(mt) * sum;
            }
            sc *= 0.08838834764831845f;
        }
        const float mx = block_reduce(sc, true, red);
        const float p = key <= pos ? expf(sc - mx) : 0.f;
        ps[tid] = p;
        const float l = block_reduce(p, false, red);
        float o = 0.f;
        const int n = min(kUnit, pos + 1 - k0);
        for (int i = 0; i < n; ++i) {
            const char* hv = half_block(t, i, 1);
            const uint32_t mt =
                *reinterpret_cast<const uint32_t*>(hv + kMetaOff + (i % kBlockPos) * 8 + (tid >> 6) * 4);
            const uint32_t w = *reinterpret_cast<const uint32_t*>(hv + word_at(i, (tid & 63) >> 3, tid >> 6));
            o = fmaf(ps[i], fmaf((float)((w >> (4 * (tid & 7))) & 15u), meta_scale(mt), meta_zero(mt)), o);
        }
        const size_t idx = ((size_t)r * a.n_q + hq) * a.max_units + u;
        a.po[idx * kHeadDim + tid] = o;
        if (tid == 0) {
            a.pm[idx] = mx;
            a.pl[idx] = l;
        }
    }
}

__global__ void __launch_bounds__(kHeadDim) join_kernel(const __grid_constant__ AttnArgs a) {
    pdl_wait();
    const int hq = blockIdx.x, r = blockIdx.y, d = threadIdx.x;
    const int s = stream_of(a.rows, r);
    const int nu = (a.rows.pos0[s] + r - a.rows.row_start[s]) / kUnit + 1;
    const size_t base = ((size_t)r * a.n_q + hq) * a.max_units;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int u = 0; u < nu; ++u) M = fmaxf(M, a.pm[base + u]);
    for (int u = 0; u < nu; ++u) {
        const float w = expf(a.pm[base + u] - M);
        L = fmaf(a.pl[base + u], w, L);
        O = fmaf(a.po[(base + u) * kHeadDim + d], w, O);
    }
    a.out[(long)r * a.ldo + hq * kHeadDim + d] = rn(O / L);
}

}  // namespace

int attn_unit() { return kUnit; }

cudaError_t init_attn() { return cudaSuccess; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st, bool) {
    if (a.rows.n_rows < 1) return cudaSuccess;
    int nu = 1;
    for (int s = 0; s < a.rows.n_streams; ++s) {
        const int last = a.rows.pos0[s] + a.rows.row_start[s + 1] - a.rows.row_start[s] - 1;
        if (last / kUnit + 1 > nu) nu = last / kUnit + 1;
    }
    page_kernel<<<dim3(nu, a.rows.n_kv, a.rows.n_streams), kPage, 0, st>>>(a);
    join_kernel<<<dim3(a.n_q, a.rows.n_rows), kHeadDim, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace tfl
