// The 4-bit key/value cache: layout, quantisation formula and the arguments of
// its kernels (kv4_cache.cu: write and read; kv4_attn.cu: attention; kv4_api.cu:
// the C entry points).
//
// A cache holds, per (layer, page of 128 positions, KV head), one tile of
// 18,432 contiguous bytes: eight blocks of 16 positions, each block
//   16 rows of key codes (64 bytes each) | 16 key (scale, zero) pairs x 2 |
//   16 rows of value codes               | 16 value (scale, zero) pairs x 2
// so that a warp's 16 keys with everything that belongs to them are 2,304
// contiguous bytes.  A row's 128 codes sit in eight 8-byte chunks; chunk c holds
// dims 8c..8c+7 in its first 32-bit word and 64+8c..64+8c+7 in its second, the
// lowest dim in the lowest 4 bits, and is stored at chunk c ^ 4 for positions
// whose bit 1 is set (the exchange of halves lets the attention's 8-byte value
// loads of four positions hit distinct shared-memory banks).  Dims 0..63 and
// 64..127 are the two groups: bf16 scale and zero of group 0, then of group 1,
// eight bytes per position.
//
// Quantisation of a group of 64 bf16 numbers x (one position, one head):
//   zero = min x,  scale = bf16((max x - min x) / 15),
//   n = clamp(round_half_even((x - zero) / scale), 0, 15)   (0 when scale = 0)
// in fp32; the group stands for zero + scale n.  A group that holds a NaN or an
// infinity, or whose max - min overflows fp32, is stored with zero = NaN and
// scale = 0: it stands for NaN everywhere.
#pragma once

#include "common.cuh"

namespace tfl {
namespace kv4 {

constexpr int kGroup = 64;                     // dims that share a scale and a zero
constexpr int kBlockPos = 16;                  // positions of a block
constexpr int kRowBytes = kHeadDim / 2;        // codes of a row
constexpr int kMetaBytes = 8;                  // (scale, zero) of a row's two groups
constexpr int kMetaOff = kBlockPos * kRowBytes;               // within a half block
constexpr int kHalfBlock = kBlockPos * (kRowBytes + kMetaBytes);  // keys or values of a block: 1,152
constexpr int kBlockBytes = 2 * kHalfBlock;                   // 2,304
constexpr int kTileBytes = kPage / kBlockPos * kBlockBytes;   // 18,432
constexpr int kMaxKvHeads = 64;
constexpr int kMaxGroupHeads = 16;             // query heads per KV head

// One stream's cache.
struct View {
    char* pages;       // first tile
    const int* table;  // logical page -> physical page
    int n_pages;
    int pad_;
};

// Rows of one call, grouped by stream: rows [row_start[s], row_start[s+1])
// belong to stream s and sit at positions pos0[s], pos0[s]+1, ...
struct Rows {
    int n_streams;
    int n_rows;
    int n_kv;
    int layer;
    int row_start[kMaxStreams + 1];
    int pos0[kMaxStreams];
    View kv[kMaxStreams];
};

__device__ __forceinline__ int stream_of(const Rows& m, int r) {
    int s = 0;
    while (s + 1 < m.n_streams && r >= m.row_start[s + 1]) ++s;
    return s;
}

// Loads of what the kernel before may have written.  A kernel is set up while that one still runs, so
// its memory is not read-only for the kernel's life, which the read-only path (ld.global.nc) asks for: such a load
// could be moved before pdl_wait.  These stay behind it (volatile, as it is).
__device__ __forceinline__ uint32_t load_word(const void* p) {
    uint32_t x;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(x) : "l"(p));
    return x;
}
__device__ __forceinline__ uint32_t load_once(const void* p) {  // not to be kept in the caches
    uint32_t x;
    asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(x) : "l"(p));
    return x;
}
__device__ __forceinline__ float load_l2(const float* p) {
    float x;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x) : "l"(p));
    return x;
}
__device__ __forceinline__ float4 load_l2(const float4* p) {
    float4 x;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
    return x;
}

// The physical page of pos: below v.n_pages in a sound table.
__device__ __forceinline__ unsigned page_of(const View& v, int pos) { return load_word(v.table + pos / kPage); }

// The tile of (layer, page, head); of an entry outside the cache, one of the last page's.
__device__ __forceinline__ char* tile(const View& v, int layer, int n_kv, unsigned page, int head) {
    return v.pages + (((size_t)layer * v.n_pages + min(page, v.n_pages - 1u)) * n_kv + head) * (size_t)kTileBytes;
}

// The half block (kind 0: keys, 1: values) of a tile that holds pos.
__device__ __forceinline__ char* half_block(char* t, int pos, int kind) {
    return t + (pos % kPage) / kBlockPos * kBlockBytes + kind * kHalfBlock;
}

// Byte of 32-bit word j of chunk c in the row of pos.
__device__ __forceinline__ int word_at(int pos, int c, int j) {
    return (pos % kBlockPos) * kRowBytes + ((c ^ ((pos & 2) << 1)) << 3) + (j << 2);
}

struct WriteArgs {
    Rows rows;
    const bf16 *k, *v;   // row r at k + src_row * ld, head h at + 128 h
    long ld;
    int wrap;            // 0: src_row = r; 1: src_row = 2 * 128 s + position mod 128 (a page of its own per stream)
};
struct ReadArgs {
    Rows rows;
    bf16 *k, *v;         // row r at k + r * ld
    long ld;
    int item_start[kMaxStreams + 1];  // set by launch_read: first (block, head) of a stream
};
cudaError_t launch_write(const WriteArgs& a, cudaStream_t st, bool pdl);
cudaError_t launch_read(ReadArgs& a, cudaStream_t st, bool pdl);
cudaError_t launch_identity(int* table, int n, cudaStream_t st);  // table[i] = i

struct AttnArgs {
    Rows rows;
    int n_q;
    const bf16* q;
    long ldq;
    bf16* out;
    long ldo;
    // partials of (part, columns, KV head) "sets", per unit: maxima and sums
    // [set][unit][column], outputs [set][unit][tile][lane] of float4 (kv4_attn.cu)
    float *pm, *pl, *po;
    int max_units;
    int* status;         // device status word: a bounded wait that gives up raises kStatusDevice
    bool probe;          // a call in which a wait runs out: of step `lose` of every warp that has it,
    int lose;            // after wait_limit polls
    unsigned wait_limit;
};
constexpr int kMaxParts = 2 * kMaxStreams;  // attention may cut a call's streams in two
int attn_max_units(int positions, int n_kv);  // partials of a row's head over caches of up to so many positions
cudaError_t init_attn();
cudaError_t launch_attn(const AttnArgs& a, int sms, cudaStream_t st, bool pdl);

}  // namespace kv4
}  // namespace tfl

struct tfl_kv4 {
    int device;
    int layers, n_kv, max_pos, n_pages;
    int length;
    int* table;
    char* pages;
    tfl::kv4::View view() const { return tfl::kv4::View{pages, table, n_pages, 0}; }
};

struct tfl_kv4_attn {
    int device;
    int n_q, n_kv, max_rows, max_pos, max_units;
    int sms;  // of the device
    float *pm, *pl, *po;
    int* status;
};
