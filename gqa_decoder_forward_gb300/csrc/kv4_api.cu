// C entry points of the 4-bit cache (include/tfl.h): argument checks, sizes and
// enqueueing.  The kernels are in kv4_cache.cu and kv4_attn.cu.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "kv4.cuh"
#include "../../include/tfl.h"

namespace tfl {
int api_fail(int code, const char* msg);
void set_last_error(const char* msg);
}  // namespace tfl

using namespace tfl;

namespace {

constexpr int kMaxLayers = 1024;
constexpr int kMaxPositions = 1 << 20;
constexpr int kMaxAttnRowsPerStream = 16;

static_assert(kv4::kTileBytes == TFL_KV4_TILE && kv4::kGroup == TFL_KV4_GROUP && kPage == TFL_KV_PAGE, "tfl.h");

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return api_fail(code, buf);
}

int ok() {
    set_last_error("");
    return TFL_OK;
}

#define CK(call)                                                                                                     \
    do {                                                                                                             \
        cudaError_t e_ = (call);                                                                                     \
        if (e_ != cudaSuccess)                                                                                       \
            return fail(TFL_E_CUDA, "%s failed: %s (%s:%d)", #call, cudaGetErrorString(e_), __FILE__, __LINE__);     \
    } while (0)

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int pages_of(int max_positions) { return (max_positions + kPage - 1) / kPage; }

bool cache_sizes_ok(int layers, int n_kv, int head_dim, int max_positions) {
    return layers >= 1 && layers <= kMaxLayers && n_kv >= 1 && n_kv <= kv4::kMaxKvHeads && head_dim == kHeadDim &&
           max_positions >= 1 && max_positions <= kMaxPositions;
}

bool attn_sizes_ok(int n_q, int n_kv, int head_dim, int max_rows, int max_positions) {
    return n_kv >= 1 && n_kv <= kv4::kMaxKvHeads && n_q >= n_kv && n_q % n_kv == 0 &&
           n_q / n_kv <= kv4::kMaxGroupHeads && head_dim == kHeadDim && max_rows >= 1 && max_rows <= kMaxDecodeRows &&
           max_positions >= 1 && max_positions <= kMaxPositions;
}

// Workspace of an attention object (byte offsets, 256-byte aligned regions).
struct AttnLayout {
    size_t status, pm, pl, po, total;
    int units;
};

AttnLayout attn_layout(int n_q, int n_kv, int max_rows, int max_positions) {
    AttnLayout L;
    L.units = kv4::attn_max_units(max_positions, n_kv);
    // Tiles of eight columns over all sets.  A call has at most 16 streams, cut into 32 parts; a part
    // of R rows has ceil(R G / 8) tiles per KV head.
    const int G = n_q / n_kv;
    const size_t tiles = (size_t)n_kv * (std::min(max_rows, kv4::kMaxParts) + max_rows * G / 8);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = round256(off + bytes);
        return o;
    };
    L.status = take(256);
    L.pm = take(tiles * L.units * 8 * 4);
    L.pl = take(tiles * L.units * 8 * 4);
    L.po = take(tiles * L.units * 8 * kHeadDim * 4);
    L.total = off;
    return L;
}

// The current device, if it is one this library runs on.
int check_arch(int* dev) {
    CK(cudaGetDevice(dev));
    int major = 0, minor = 0;
    CK(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev));
    CK(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev));
    if (major != 10 || minor != 3)
        return fail(TFL_E_ARCH, "this library needs an sm_103 (GB300) GPU; device %d is sm_%d%d", *dev, major, minor);
    return TFL_OK;
}

// A call's first kernel may be set up while the stream's last one ends (every kernel here
// waits for that end before it touches memory).  Not on the legacy stream, which also
// waits for other streams.  Call after call without | with it: one token written and read
// back 4.3 | 3.5 us, one row attending 4,096 keys 8.6 | 8.2 us.
bool programmatic(void* stream) { return stream != nullptr && stream != (void*)cudaStreamLegacy; }

// Ends what cudaMemcpy and cudaMemset have left to do when they return (a small copy from pageable memory, or a
// memset, may still be on its way): streams that do not wait for the legacy one find it done.
cudaError_t settle(cudaError_t e) { return e == cudaSuccess ? cudaStreamSynchronize(cudaStreamLegacy) : e; }

bool bad_ptr(const void* p) { return !p || ((uintptr_t)p & 15u); }

bool bad_ld(size_t ld, int heads) { return ld < (size_t)heads * kHeadDim || ld % 8 != 0 || ld > ((size_t)1 << 40); }

// Fills the row map of a call, or fails.  max_rows: rows of one stream (0: as
// many as its capacity holds); unique: a cache may not appear twice.
int fill_rows(kv4::Rows& m, tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0, const int* rows,
              int max_rows, bool unique) {
    if (!kvs || !pos0 || !rows) return fail(TFL_E_ARG, "NULL kvs, pos0 or rows");
    if (n_streams < 1 || n_streams > kMaxStreams)
        return fail(TFL_E_ARG, "n_streams %d outside 1..%d", n_streams, kMaxStreams);
    std::memset(&m, 0, sizeof m);
    long total = 0;
    for (int s = 0; s < n_streams; ++s) {
        const tfl_kv4* kv = kvs[s];
        if (!kv) return fail(TFL_E_ARG, "stream %d: NULL cache", s);
        if (kv->n_kv != kvs[0]->n_kv || kv->device != kvs[0]->device)
            return fail(TFL_E_ARG, "stream %d: a cache of %d heads on device %d beside one of %d on device %d", s,
                        kv->n_kv, kv->device, kvs[0]->n_kv, kvs[0]->device);
        if (layer < 0 || layer >= kv->layers)
            return fail(TFL_E_ARG, "layer %d outside 0..%d of stream %d's cache", layer, kv->layers - 1, s);
        for (int t = 0; unique && t < s; ++t)
            if (kvs[t] == kv) return fail(TFL_E_ARG, "stream %d repeats the cache of stream %d", s, t);
        if (rows[s] < 0 || (max_rows && rows[s] > max_rows))
            return fail(TFL_E_ARG, "stream %d: %d rows outside 0..%d", s, rows[s], max_rows ? max_rows : kv->max_pos);
        if (pos0[s] < 0 || rows[s] > kv->max_pos || pos0[s] > kv->max_pos - rows[s])
            return fail(TFL_E_CAPACITY, "stream %d: %d rows from position %d pass the capacity %d", s, rows[s], pos0[s],
                        kv->max_pos);
        m.row_start[s] = (int)total;
        m.pos0[s] = pos0[s];
        m.kv[s] = kv->view();
        total += rows[s];
    }
    m.row_start[n_streams] = (int)total;  // at most 16 * 2^20
    m.n_streams = n_streams;
    m.n_rows = (int)total;
    m.n_kv = kvs[0]->n_kv;
    m.layer = layer;
    int dev = -1;
    CK(cudaGetDevice(&dev));
    if (dev != kvs[0]->device)
        return fail(TFL_E_ARG, "the caches are on device %d and the current device is %d", kvs[0]->device, dev);
    return TFL_OK;
}

int check_rows_tensors(const void* k, const void* v, size_t ld, int n_kv) {
    if (bad_ptr(k) || bad_ptr(v)) return fail(TFL_E_ARG, "k/v NULL or not 16-byte aligned");
    if (bad_ld(ld, n_kv))
        return fail(TFL_E_ARG, "ld %zu is less than %d heads of %d or not a multiple of 8", ld, n_kv, kHeadDim);
    return TFL_OK;
}

int attend(tfl_kv4_attn* attn, tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0, const int* rows,
           const void* q, size_t ldq, void* out, size_t ldo, void* stream, bool probe, int lose, int wait_limit) {
    if (!attn) return fail(TFL_E_ARG, "NULL attention object");
    kv4::AttnArgs a;
    if (int e = fill_rows(a.rows, kvs, n_streams, layer, pos0, rows, kMaxAttnRowsPerStream, false)) return e;
    if (attn->n_kv != a.rows.n_kv || attn->device != kvs[0]->device)
        return fail(TFL_E_ARG, "an attention object for %d KV heads on device %d, caches of %d heads on device %d",
                    attn->n_kv, attn->device, a.rows.n_kv, kvs[0]->device);
    if (a.rows.n_rows > attn->max_rows)
        return fail(TFL_E_ARG, "%d rows exceed the object's max_rows %d", a.rows.n_rows, attn->max_rows);
    for (int s = 0; s < n_streams; ++s)
        if (rows[s] > 0 && pos0[s] + rows[s] > attn->max_pos)
            return fail(TFL_E_CAPACITY, "stream %d: positions to %d pass the object's max_positions %d", s,
                        pos0[s] + rows[s] - 1, attn->max_pos);
    if (a.rows.n_rows == 0) return ok();  // whatever the tensors
    if (bad_ptr(q) || bad_ptr(out)) return fail(TFL_E_ARG, "q/out NULL or not 16-byte aligned");
    if (q == out) return fail(TFL_E_ARG, "q and out are the same memory");
    if (bad_ld(ldq, attn->n_q) || bad_ld(ldo, attn->n_q))
        return fail(TFL_E_ARG, "ldq %zu / ldo %zu: less than %d heads of %d or not a multiple of 8", ldq, ldo,
                    attn->n_q, kHeadDim);
    a.n_q = attn->n_q;
    a.q = (const bf16*)q;
    a.ldq = (long)ldq;
    a.out = (bf16*)out;
    a.ldo = (long)ldo;
    a.pm = attn->pm;
    a.pl = attn->pl;
    a.po = attn->po;
    a.max_units = attn->max_units;
    a.status = attn->status;
    a.probe = probe;
    a.lose = lose;
    a.wait_limit = (unsigned)wait_limit;
    CK(kv4::launch_attn(a, attn->sms, (cudaStream_t)stream, programmatic(stream)));
    return ok();
}

}  // namespace

extern "C" {

size_t tfl_kv4_bytes(int layers, int n_kv, int head_dim, int max_positions) {
    if (!cache_sizes_ok(layers, n_kv, head_dim, max_positions)) return 0;
    const size_t n = (size_t)pages_of(max_positions);
    return round256(n * 4) + (size_t)layers * n * n_kv * kv4::kTileBytes;
}

int tfl_kv4_alloc(int layers, int n_kv, int head_dim, int max_positions, void* dev_buf, size_t bytes, tfl_kv4** out) {
    if (!out) return fail(TFL_E_ARG, "out is NULL");
    *out = nullptr;
    if (!cache_sizes_ok(layers, n_kv, head_dim, max_positions))
        return fail(TFL_E_ARG,
                    "%d layers, %d heads of %d, %d positions refused: layers 1..%d, heads 1..%d of %d, positions 1..%d",
                    layers, n_kv, head_dim, max_positions, kMaxLayers, kv4::kMaxKvHeads, kHeadDim, kMaxPositions);
    if (bad_ptr(dev_buf)) return fail(TFL_E_ARG, "KV buffer NULL or not 16-byte aligned");
    const size_t need = tfl_kv4_bytes(layers, n_kv, head_dim, max_positions);
    if (bytes < need) return fail(TFL_E_WORKSPACE, "KV buffer %zu bytes < %zu needed", bytes, need);
    int dev = 0;
    if (int e = check_arch(&dev)) return e;
    const int n = pages_of(max_positions);
    tfl_kv4* kv = new (std::nothrow) tfl_kv4();
    int* ident = new (std::nothrow) int[n];
    if (!kv || !ident) {
        delete kv;
        delete[] ident;
        return fail(TFL_E_ARG, "out of host memory");
    }
    kv->device = dev;
    kv->layers = layers;
    kv->n_kv = n_kv;
    kv->max_pos = max_positions;
    kv->n_pages = n;
    kv->length = 0;
    kv->table = (int*)dev_buf;
    kv->pages = (char*)dev_buf + round256((size_t)n * 4);
    for (int i = 0; i < n; ++i) ident[i] = i;
    const cudaError_t ce = settle(cudaMemcpy(kv->table, ident, (size_t)n * 4, cudaMemcpyHostToDevice));
    delete[] ident;
    if (ce != cudaSuccess) {
        delete kv;
        return fail(TFL_E_CUDA, "writing the page table failed: %s", cudaGetErrorString(ce));
    }
    *out = kv;
    return ok();
}

void tfl_kv4_free(tfl_kv4* kv) { delete kv; }

int tfl_kv4_reset(tfl_kv4* kv, int keep) {
    if (!kv) return fail(TFL_E_ARG, "NULL KV object");
    if (keep < 0 || keep > kv->max_pos) return fail(TFL_E_ARG, "keep %d outside 0..%d", keep, kv->max_pos);
    kv->length = keep;
    return ok();
}

int tfl_kv4_length(const tfl_kv4* kv) { return kv ? kv->length : -1; }
int tfl_kv4_capacity(const tfl_kv4* kv) { return kv ? kv->max_pos : -1; }

int tfl_kv4_write(tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0, const int* rows, const void* k,
                  const void* v, size_t ld, void* stream) {
    kv4::WriteArgs a;
    if (int e = fill_rows(a.rows, kvs, n_streams, layer, pos0, rows, 0, true)) return e;
    if (a.rows.n_rows == 0) return ok();  // whatever the tensors
    if (int e = check_rows_tensors(k, v, ld, a.rows.n_kv)) return e;
    a.k = (const bf16*)k;
    a.v = (const bf16*)v;
    a.ld = (long)ld;
    a.wrap = 0;
    CK(kv4::launch_write(a, (cudaStream_t)stream, programmatic(stream)));
    return ok();
}

int tfl_kv4_read(tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0, const int* rows, void* k, void* v,
                 size_t ld, void* stream) {
    kv4::ReadArgs a;
    if (int e = fill_rows(a.rows, kvs, n_streams, layer, pos0, rows, 0, false)) return e;
    if (a.rows.n_rows == 0) return ok();  // whatever the tensors
    if (int e = check_rows_tensors(k, v, ld, a.rows.n_kv)) return e;
    if (k == v) return fail(TFL_E_ARG, "k and v are the same memory");
    a.k = (bf16*)k;
    a.v = (bf16*)v;
    a.ld = (long)ld;
    CK(kv4::launch_read(a, (cudaStream_t)stream, programmatic(stream)));
    return ok();
}

size_t tfl_kv4_attn_bytes(int n_q, int n_kv, int head_dim, int max_rows, int max_positions) {
    if (!attn_sizes_ok(n_q, n_kv, head_dim, max_rows, max_positions)) return 0;
    return attn_layout(n_q, n_kv, max_rows, max_positions).total;
}

int tfl_kv4_attn_init(int n_q, int n_kv, int head_dim, int max_rows, int max_positions, void* workspace,
                      size_t ws_bytes, tfl_kv4_attn** out) {
    if (!out) return fail(TFL_E_ARG, "out is NULL");
    *out = nullptr;
    if (!attn_sizes_ok(n_q, n_kv, head_dim, max_rows, max_positions))
        return fail(TFL_E_ARG,
                    "%d query / %d KV heads of %d, %d rows, %d positions refused: KV heads 1..%d of %d, 1..%d query "
                    "heads each, rows 1..%d, positions 1..%d",
                    n_q, n_kv, head_dim, max_rows, max_positions, kv4::kMaxKvHeads, kHeadDim, kv4::kMaxGroupHeads,
                    kMaxDecodeRows, kMaxPositions);
    if (!workspace || ((uintptr_t)workspace & 255u)) return fail(TFL_E_ARG, "workspace NULL or not 256-byte aligned");
    const size_t need = tfl_kv4_attn_bytes(n_q, n_kv, head_dim, max_rows, max_positions);
    if (ws_bytes < need) return fail(TFL_E_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    int dev = 0;
    if (int e = check_arch(&dev)) return e;
    int sms = 0;
    CK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    CK(kv4::init_attn());
    tfl_kv4_attn* a = new (std::nothrow) tfl_kv4_attn();
    if (!a) return fail(TFL_E_ARG, "out of host memory");
    a->device = dev;
    a->n_q = n_q;
    a->n_kv = n_kv;
    a->max_rows = max_rows;
    a->max_pos = max_positions;
    const AttnLayout L = attn_layout(n_q, n_kv, max_rows, max_positions);
    char* ws = (char*)workspace;
    a->max_units = L.units;
    a->pm = (float*)(ws + L.pm);
    a->pl = (float*)(ws + L.pl);
    a->po = (float*)(ws + L.po);
    a->sms = sms;
    a->status = (int*)(ws + L.status);
    const cudaError_t ce = settle(cudaMemset(a->status, 0, 256));
    if (ce != cudaSuccess) {
        delete a;
        return fail(TFL_E_CUDA, "clearing the status word failed: %s", cudaGetErrorString(ce));
    }
    *out = a;
    return ok();
}

int tfl_kv4_attn_status(tfl_kv4_attn* attn, void* stream) {
    if (!attn) return fail(TFL_E_ARG, "NULL attention object");
    CK(cudaStreamSynchronize((cudaStream_t)stream));
    int s = 0;
    CK(cudaMemcpy(&s, attn->status, 4, cudaMemcpyDeviceToHost));
    if (s == 0) return ok();
    CK(settle(cudaMemset(attn->status, 0, 4)));
    return fail(TFL_E_DEVICE, "a kernel gave up a bounded wait");
}

void tfl_kv4_attn_free(tfl_kv4_attn* attn) { delete attn; }

int tfl_kv4_attention(tfl_kv4_attn* attn, tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0,
                      const int* rows, const void* q, size_t ldq, void* out, size_t ldo, void* stream) {
    return attend(attn, kvs, n_streams, layer, pos0, rows, q, ldq, out, ldo, stream, false, 0, 0);
}

int tfl_kv4_wait_probe(tfl_kv4_attn* attn, tfl_kv4* const* kvs, int n_streams, int layer, const int* pos0,
                       const int* rows, const void* q, size_t ldq, void* out, size_t ldo, int lose, int spin_limit,
                       void* stream) {
    if (lose < 0) return fail(TFL_E_ARG, "step %d", lose);
    if (spin_limit < 1 || spin_limit > (1 << 20))
        return fail(TFL_E_ARG, "spin_limit %d outside 1..%d", spin_limit, 1 << 20);
    return attend(attn, kvs, n_streams, layer, pos0, rows, q, ldq, out, ldo, stream, true, lose, spin_limit);
}

}  // extern "C"
