// What the kernels of the experts' products share: which rows belong to which
// expert, tiles of those rows, buffers, copies to LDS and the epilogue's small
// functions.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

#include <algorithm>
#include <cmath>

namespace moe {

// H and N: a tile's rows have to lie within 32-bit offsets of each other.
constexpr int32_t kMaxGemmChannels = 1 << 22;
constexpr int kMaxSegments = kMaxE + kMaxBalanceSlots;
constexpr int kXcds = 8;       // workgroups go round the XCDs in turn
constexpr int kCus = 256;      // workgroups that run at once, of one per CU
constexpr int kTileRows = 256; // token rows of a tile of long segments

// The rows of every expert: expert i's rows of a plain layout, or with
// seg_offset the (rank, segment) pairs of a balanced one.
struct Segments {
    const int32_t *count;      // [E]
    const int32_t *offset;     // [E+1]
    const int32_t *seg_offset; // [R*(E/R+B)+1] or null
    const int32_t *slot_expert;
    int32_t E, R, B, nseg;
    int64_t entries;           // S*K: at most this many rows are used
    int64_t max_count;         // at most this many in one segment
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

struct RowTile {
    int row0;      // first row of the receive buffer
    int rows;      // rows of the tile that hold an entry
    int expert;
    int ntile;     // which tile of the weights' rows
};

// Segment i's first row, and its number of rows or (balanced layout) the next
// segment's first row; past the last segment the last one's, without a branch
// around the loads.
__device__ __forceinline__ void load_segment(const Segments &a, int i, int &first, int &rows_or_end) {
    const int at = min(i, a.nseg - 1);
    const int32_t *const f = a.seg_offset != nullptr ? a.seg_offset : a.offset;
    const int32_t *const n = a.seg_offset != nullptr ? a.seg_offset + 1 : a.count;
    first = f[at];
    rows_or_end = n[at];
}
__device__ __forceinline__ int segment_rows(const Segments &a, int i, int first, int rows_or_end) {
    return i < a.nseg ? rows_or_end - (a.seg_offset != nullptr ? first : 0) : 0;
}

// find_tile with PER segments per lane (nseg <= 64 * PER).
template <int BM, int PER>
__device__ __forceinline__ bool find_tile_per(const Segments &a, int block, int tiles_n, RowTile &t) {
    const int lane = threadIdx.x & (kWave - 1);
    // every load at once: the whole search waits for memory one time
    int first[PER], n[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) load_segment(a, lane * PER + j, first[j], n[j]);
    int tiles = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        n[j] = segment_rows(a, lane * PER + j, first[j], n[j]);
        tiles += (n[j] + BM - 1) / BM;
    }
    const int upto = wave_inclusive_scan(tiles);
    const int total = __builtin_amdgcn_readlane(upto, kWave - 1) * tiles_n;
    const int run = (total + kXcds - 1) / kXcds, at_run = block / kXcds;
    const int tile = (block % kXcds) * run + at_run;
    if (at_run >= run || tile >= total) return false;
    const int row_tile = tile / tiles_n;
    const int owner = __builtin_ctzll(__ballot(upto > row_tile));
    // each lane looks among its own segments; the owner's answer counts
    int seg = 0, seg_first = 0, seg_n = 0, before = 0, at = upto - tiles;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (at <= row_tile) {
            seg = lane * PER + j;
            seg_first = first[j];
            seg_n = n[j];
            before = at;
        }
        at += (n[j] + BM - 1) / BM;
    }
    seg = __builtin_amdgcn_readlane(seg, owner);
    seg_first = __builtin_amdgcn_readlane(seg_first, owner);
    seg_n = __builtin_amdgcn_readlane(seg_n, owner);
    before = __builtin_amdgcn_readlane(before, owner);
    const int seg_tiles = (seg_n + BM - 1) / BM, local = tile - before * tiles_n, m = local % seg_tiles;
    t.ntile = local / seg_tiles;
    t.rows = min(BM, seg_n - m * BM);
    t.row0 = seg_first + m * BM;
    t.expert = seg;
    if (a.seg_offset != nullptr) {
        const int epr = a.E / a.R, r = seg / (epr + a.B), j = seg % (epr + a.B);
        t.expert = j < epr ? r * epr + j : __builtin_amdgcn_readfirstlane(a.slot_expert[r * a.B + j - epr]);
    }
    return true;
}

// Finds what workgroup `block` computes.  Tiles are numbered segment by
// segment, inside a segment weight tile by weight tile, inside that row tile
// (BM rows) by row tile, so that workgroups that run together share a weight
// tile.  Workgroups go round the XCDs in turn: each XCD takes one run of the
// tiles, and its L2 serves the neighbours.  Every lane of the wave calls it;
// false for a workgroup without a tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const Segments &a, int block, int tiles_n, RowTile &t) {
    if (a.nseg <= kWave) return find_tile_per<BM, 1>(a, block, tiles_n, t);
    if (a.nseg <= 4 * kWave) return find_tile_per<BM, 4>(a, block, tiles_n, t);
    return find_tile_per<BM, kMaxSegments / kWave>(a, block, tiles_n, t);
}

// g / (1 + exp(-g)) with the hardware's exponential and reciprocal: within
// (|g| + 4) units of 2^-23, far below the bf16 rounding that follows, in 5
// instructions instead of ~35 for the library's exponential and division.  The
// reciprocal has no subnormal results: from g = -126 ln 2 = -87.3 on down it is 0.
__device__ __forceinline__ float silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

__device__ __forceinline__ u32x2 pack_bf16x4(f32x4 v) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

// A raw buffer over `bytes` bytes: loads take a 32-bit offset per lane and read
// zeros, stores write nothing, where it lies past the end.  An offset that all
// lanes share is always smaller than `bytes`, or 0: whether the end is found there
// too does not matter then.
constexpr int kBufferRsrcWord3 = 0x00020000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, unsigned int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, static_cast<int>(bytes), kBufferRsrcWord3);
}

typedef __attribute__((address_space(3))) void lds_void;

// Copies 16 bytes per lane to 1 KiB of LDS at `to` (the same in every lane).
// ONCE: past the caches (non-temporal).
constexpr int kNonTemporal = 2;
template <bool ONCE = false>
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t b, u32x4 *to, unsigned int offset, int uniform_offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, reinterpret_cast<lds_void *>(reinterpret_cast<uintptr_t>(to)), 16,
                                             static_cast<int>(offset), uniform_offset, 0, ONCE ? kNonTemporal : 0);
}

// Orders the wave's own LDS accesses; nothing else uses the memory between.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Workgroup barrier that first waits until at most N of the wave's global
// loads, copies and stores are in flight (63: for none of them), and for its
// LDS accesses.  A fence would wait for every copy to LDS.
template <int N>
__device__ __forceinline__ void barrier_after() {
    static_assert(N < 64, "the count's six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4 << 14));   // vmcnt(N), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// Segments with the number of tiles before each (row tiles by weight tiles).
struct SegTable {
    int before[kMaxSegments + 1], first[kMaxSegments], rows[kMaxSegments];
};

// Tile number `tile` from the table; every lane calls it.
__device__ __forceinline__ RowTile tile_at(const Segments &a, const SegTable &segs, int tile) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.nseg + kWave - 1) / kWave;
    // the last lane, then the last of its segments, with at most `tile` tiles before it
    int from = segs.before[min(lane * per, a.nseg)];
    const int owner = kWave - 1 - __builtin_clzll(__ballot(from <= tile && lane * per < a.nseg));
    const int i = owner * per + lane;
    from = segs.before[min(i, a.nseg)];
    const int seg = owner * per + kWave - 1 - __builtin_clzll(__ballot(lane < per && i < a.nseg && from <= tile));
    const int n = __builtin_amdgcn_readfirstlane(segs.rows[seg]), before = __builtin_amdgcn_readfirstlane(segs.before[seg]);
    // local / seg_tiles is the weight tile's number, below 2^15: the estimate is within one
    const int seg_tiles = (n + kTileRows - 1) / kTileRows, local = tile - before;
    RowTile t;
    t.ntile = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<float>(local) * __builtin_amdgcn_rcpf(static_cast<float>(seg_tiles))));
    int m = local - t.ntile * seg_tiles;
    if (m < 0) {
        t.ntile -= 1;
        m += seg_tiles;
    } else if (m >= seg_tiles) {
        t.ntile += 1;
        m -= seg_tiles;
    }
    t.rows = min(kTileRows, n - m * kTileRows);
    t.row0 = __builtin_amdgcn_readfirstlane(segs.first[seg]) + m * kTileRows;
    t.expert = seg;
    if (a.seg_offset != nullptr) {
        const int epr = a.E / a.R, r = seg / (epr + a.B), j = seg % (epr + a.B);
        t.expert = j < epr ? r * epr + j : __builtin_amdgcn_readfirstlane(a.slot_expert[r * a.B + j - epr]);
    }
    return t;
}

// Most row tiles of BM rows that any routing of this shape can have.
inline int64_t most_tiles(const Segments &a, int BM) {
    const int64_t used = std::min<int64_t>(a.nseg, a.entries);
    return std::min(a.entries / BM + used, used * ((a.max_count + BM - 1) / BM));
}

// Segments with a row, if the routing is at random.
inline double used_segments(const Segments &a) {
    return std::max(1.0, a.nseg * -std::expm1(-static_cast<double>(a.entries) / a.nseg));
}

}  // namespace moe
