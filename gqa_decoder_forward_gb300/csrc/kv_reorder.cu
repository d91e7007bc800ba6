// Reordering of caches by parents: positions [begin[i], end[i]) of cache i become what
// cache parents[i] held there, in every layer, keys and values.  The parents are in device
// memory (a beam search's selection leaves them there), so which caches move is known to the
// kernel alone; a parent that is none of the call's caches (first .. first + n - 1), like a cache's own number, leaves the
// cache as it is.
//
// In place, whatever the parents (two caches may change places): a thread holds the same
// 16 bytes of every cache that has children and stores after it has loaded them all, and no
// other thread touches those bytes.  What bounds it is the memory: a moved row is written once,
// and read once however many children it has.
// Measured (33B shape, all layers, replayed from a graph): 16 caches, 200 positions, 894.6 MB: 138 us, 6.5 TB/s, 96%
// of a copy; 4 caches, 17 positions, 18.1 MB: 6.2 us, of which 2.7 are the memory's; two of the tiny model: 2.0 us, the launch.
#include "kv_reorder.cuh"

namespace tfl {
namespace {

constexpr int kMaxRun = 16;    // positions of a CTA, within one page
constexpr int kThreads = 256;

// Slots: caches of the call, at most (registers for what is held).
template <int Slots>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ char *to[kMaxStreams], *from[kMaxStreams];  // the run's first position, of a cache that takes, that gives
    __shared__ int first[kMaxStreams], last[kMaxStreams];  // 16-byte chunks of the run that cache i takes
    __shared__ int begin[kMaxStreams], end[kMaxStreams];   // the same that the k-th source gives, to any child
    __shared__ unsigned children[kMaxStreams];             // of the k-th source
    __shared__ int n_sources;
    const int run = a.run, runs = (a.hi - 1) / run - a.lo / run + 1;
    const int pos = (a.lo / run + blockIdx.x % runs) * run, lk = blockIdx.x / runs;
    const int row = a.n_kv * kHeadDim * 2 / 16;  // chunks of a position
    const int lane = threadIdx.x;
    pdl_wait();
    if (lane < 32) {
        const int i = lane;
        int p = -1, page = 0, b = 0, e = 0;
        if (i < a.n) {
            p = a.parents[i];
            p = p >= a.first && p - a.first < a.n ? p - a.first : -1;
            page = a.kv[i].table[pos / kPage];
            b = max(a.begin[i], pos) - pos;
            e = min(a.end[i], pos + run) - pos;
            if (p == i || b >= e) p = -1;  // stays
        }
        const int parent_page = __shfl_sync(0xffffffffu, page, max(p, 0));
        const auto at = [&](const KvView& v, int page) {
            return (char*)(v.pages + (((size_t)lk * v.n_pages + page) * kPage + pos % kPage) * (size_t)a.n_kv * kHeadDim);
        };
        if (p >= 0) {
            to[i] = at(a.kv[i], page);
            first[i] = b * row;
            last[i] = e * row;
        }
        // the sources: lanes with one parent find each other, and the lowest of them speaks for it
        const unsigned taking = __ballot_sync(0xffffffffu, p >= 0);
        const unsigned same = __match_any_sync(0xffffffffu, p) & taking;
        const bool speaks = p >= 0 && __ffs(same) - 1 == i;
        const unsigned speakers = __ballot_sync(0xffffffffu, speaks);
        const int k = __popc(speakers & ((1u << i) - 1u));
        __syncwarp();
        if (speaks) {
            from[k] = at(a.kv[p], parent_page);
            children[k] = same;
            int lo = 1 << 30, hi = 0;
            for (unsigned m = same; m; m &= m - 1) {
                lo = min(lo, first[__ffs(m) - 1]);
                hi = max(hi, last[__ffs(m) - 1]);
            }
            begin[k] = lo;
            end[k] = hi;
        }
        if (i == 0) n_sources = __popc(speakers);
    }
    __syncthreads();
    const int n = n_sources;
    for (int c = threadIdx.x; c < run * row; c += kThreads) {
        uint4 x[Slots];
#pragma unroll
        for (int k = 0; k < Slots; ++k)
            if (k < n && c >= begin[k] && c < end[k]) x[k] = __ldcs(reinterpret_cast<const uint4*>(from[k] + (size_t)c * 16));
#pragma unroll
        for (int k = 0; k < Slots; ++k) {
            if (k >= n) break;
            for (unsigned m = children[k]; m; m &= m - 1) {
                const int i = __ffs(m) - 1;
                if (c >= first[i] && c < last[i]) *reinterpret_cast<uint4*>(to[i] + (size_t)c * 16) = x[k];
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_reorder(ReorderArgs a, int sms, cudaStream_t st, bool pdl) {
    if (a.lo >= a.hi) return cudaSuccess;
    // Positions of a CTA: two passes of its threads, since a CTA's passes wait for one another (16 beams of the 33B
    // shape, 200 positions, with 8 | 4 | 2 passes: 149 | 139 | 138 us), or one if that gives every SM eight CTAs sooner
    // (4 beams, 17 positions: 8.1 us with eight, 5.9 with one).
    const int row = a.n_kv * kHeadDim * 2 / 16;
    const auto grid = [&](int run) { return ((a.hi - 1) / run - a.lo / run + 1) * a.layers * 2; };
    a.run = kMaxRun;
    while (a.run > 1 && a.run * row > 2 * kThreads) a.run /= 2;
    if (a.run > 1 && a.run * row > kThreads && grid(a.run) < 8 * sms) a.run /= 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)grid(a.run));
    c.blockDim = dim3(kThreads);
    c.stream = st;
    c.attrs = attr;
    c.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&c, a.n <= 4 ? reorder_kernel<4> : a.n <= 8 ? reorder_kernel<8> : reorder_kernel<16>, a);
}

}  // namespace tfl
