// Products of every expert's rows with its weights, both MXFP4.
//
// out[r][n] = sum over h of x[r][h] * w[e(r)][n][h], as scaled matrix
// instructions: v_mfma_scale 16x16x128 multiplies 16 weight rows by 16 token
// rows over 128 channels, each lane carrying 32 channels of one row (16 bytes
// of codes) and that block's scale byte, and sums in fp32.  Weights are the
// instruction's first operand, so a lane ends with four neighbouring channels
// of one token: one 8-byte store.
//
// Which rows belong to which expert is known on the device alone.  The grid
// holds enough workgroups for any routing; they find their tiles by a prefix sum
// over the segments' row counts.
//
// Two kernels: k_expert_stream for segments of few rows (the weights' bytes are
// the work), k_expert_tile for longer ones.
#include "expert_gemm.h"
#include "mx4.h"
#include "tile_copies.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kFp4 = 4;        // operand format code of the scaled matrix instructions: E2M1
constexpr int kMaxSegments = kMaxE + kMaxBalanceSlots;
constexpr int kXcds = 8;       // workgroups go round the XCDs in turn
constexpr int kStep = 128;     // channels of one matrix instruction

struct RowTile {
    int row0;      // first row of the receive buffer
    int rows;      // rows of the tile that hold an entry
    int expert;
    int ntile;     // which tile of the weights' rows
};

// Segment i's first row, and its number of rows or (balanced layout) the next
// segment's first row; past the last segment the last one's, without a branch
// around the loads.
__device__ __forceinline__ void load_segment(const ExpertGemmArgs &a, int i, int &first, int &rows_or_end) {
    const int at = min(i, a.nseg - 1);
    const int32_t *const f = a.seg_offset != nullptr ? a.seg_offset : a.offset;
    const int32_t *const n = a.seg_offset != nullptr ? a.seg_offset + 1 : a.count;
    first = f[at];
    rows_or_end = n[at];
}
__device__ __forceinline__ int segment_rows(const ExpertGemmArgs &a, int i, int first, int rows_or_end) {
    return i < a.nseg ? rows_or_end - (a.seg_offset != nullptr ? first : 0) : 0;
}

// find_tile with PER segments per lane (nseg <= 64 * PER).
template <int BM, int PER>
__device__ __forceinline__ bool find_tile_per(const ExpertGemmArgs &a, int block, int tiles_n, RowTile &t) {
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
__device__ __forceinline__ bool find_tile(const ExpertGemmArgs &a, int block, int tiles_n, RowTile &t) {
    if (a.nseg <= kWave) return find_tile_per<BM, 1>(a, block, tiles_n, t);
    if (a.nseg <= 4 * kWave) return find_tile_per<BM, 4>(a, block, tiles_n, t);
    return find_tile_per<BM, kMaxSegments / kWave>(a, block, tiles_n, t);
}

__device__ __forceinline__ i32x8 fp4_operand(u32x4 c) {
    return i32x8{static_cast<int>(c[0]), static_cast<int>(c[1]), static_cast<int>(c[2]), static_cast<int>(c[3]), 0, 0, 0, 0};
}

// g / (1 + exp(-g)) with the hardware's exponential and reciprocal: within
// (|g| + 4) units of 2^-23, far below the bf16 rounding that follows, in 5
// instructions instead of ~35 for the library's exponential and division.
__device__ __forceinline__ float silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

__device__ __forceinline__ u32x2 pack_bf16x4(f32x4 v) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

// A raw buffer over `bytes` bytes: loads take a 32-bit offset per lane and read
// zeros, stores write nothing, where it lies past the end.  An offset that all
// lanes share is always smaller than `bytes`: whether the end is found there too
// does not matter then.
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

// ---------------------------------------------------------------------------
// short segments
// ---------------------------------------------------------------------------

// 16 token rows by 32 weight rows; the four waves split the channels and join
// their sums in LDS.  The weights' bytes are the work, each read once, so what
// counts is to keep many of them in flight and to ask for whole lines: a unit
// (256 channels) of the 32 rows, 4 KB, is copied to the wave's own LDS in
// instructions of 8 whole 128-byte lines while the unit before it is
// multiplied, four workgroups of four such waves per CU.  (The operands' own
// order, straight to registers, asks for 64 pieces of 16 bytes per instruction:
// 432 us at the decode case, 1024 rows of 256 experts, H = 7168, 2 x 1024 weight
// rows, against 328 us here, 306 = 6.4 TB/s past the caches; 64 weight rows and two
// workgroups per CU took 350 us, two waves of 32 rows 339, one 348, eight 395.)
// The wave's channels' weight scales come in parts of 8 units; tokens and their
// scales, few and shared by every workgroup of the segment, go straight to
// registers.
constexpr int kStreamRows = 16;
constexpr int kStreamWaves = 4;
constexpr int kWTiles = 2;         // 16-row weight tiles (SWIGLU: half gate, half up)
constexpr int kUnitVecs = kWTiles * 16 * 8;
constexpr int kPartUnits = 8;      // units whose scales are in LDS

template <bool SWIGLU, bool ONCE>
__global__ __launch_bounds__(kStreamWaves * kWave, 4) void k_expert_stream(ExpertGemmArgs a, int tiles_n) {
    constexpr int kOutTiles = SWIGLU ? kWTiles / 2 : kWTiles;
    __shared__ u32x4 unit0[kStreamWaves][kUnitVecs], unit1[kStreamWaves][kUnitVecs];
    __shared__ unsigned int wscale[kStreamWaves][kWTiles * 16 * 2 * kPartUnits];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    RowTile t;
    if (!find_tile<kStreamRows>(a, blockIdx.x, tiles_n, t)) return;   // the same for every wave
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.ntile = __builtin_amdgcn_readfirstlane(t.ntile);
    const int n0 = t.ntile * (kOutTiles * 16);
    // lane = 16*g + r: row r of each operand, channels 32*g .. 32*g+31 of a step
    const int r = lane & 15, g = lane >> 4;
    const unsigned int half = a.H / 2, scales = a.H / kMx4Block;
    const unsigned int wrows = min(kOutTiles * 16, a.N - n0);           // past them zeros are read
    const size_t first = t.expert * (SWIGLU ? 2 * static_cast<size_t>(a.N) : a.N) + n0, up = first + (SWIGLU ? a.N : 0);
    const auto w_gate = buffer_of(a.w + first * half, wrows * half), w_up = buffer_of(a.w + up * half, wrows * half);
    const auto s_gate = buffer_of(a.ws + first * scales, wrows * scales), s_up = buffer_of(a.ws + up * scales, wrows * scales);
    const auto xb = buffer_of(a.x + static_cast<size_t>(t.row0) * half, t.rows * half);
    const auto xsb = buffer_of(a.xs + static_cast<size_t>(t.row0) * scales, t.rows * scales);
    const int steps = a.H / kStep, units = (steps + 1) / 2;
    const int begin = units * wave / kStreamWaves, end = units * (wave + 1) / kStreamWaves;
    // Copies of 8 weight rows: lane l's vector is row l/8, chunk c at place l%8;
    // chunk c (32 channels) of row q lies at c ^ (q % 8), so that eight rows'
    // chunk c are in eight different groups of banks.
    const int q8 = lane / 8;
    const unsigned int wo = q8 * half + ((lane & 7) ^ q8) * 16;
    const auto copy_unit = [&](int u, u32x4 *to) {
        // a last unit of 128 channels leaves the second half of each row alone
        const unsigned int gone = 2 * u + 1 >= steps && (((lane & 7) ^ q8) & 4) ? kPastEnd : 0u;
#pragma unroll
        for (int j = 0; j < kWTiles * 2; ++j) {
            const int row = 8 * j;
            const bool is_up = row >= kOutTiles * 16;
            copy_to_lds<ONCE>(is_up ? w_up : w_gate, to + row * 8, (wo + (is_up ? row - kOutTiles * 16 : row) * half) | gone, u * 128);
        }
    };
    // Scale words of 8 units from u0: row 16*i + lane/4, words 4*(lane%4) .. +3;
    // those past the row's end are not read.  Word d of row q lies at
    // d ^ (q % 16): 16 rows' word d are in 16 different banks.
    const auto load_part = [&](int u0) {
        u32x4 v[kWTiles];
        const int d0 = 4 * (lane & 3);
#pragma unroll
        for (int i = 0; i < kWTiles; ++i) {
            const bool is_up = i >= kOutTiles;
            const int q = (is_up ? i - kOutTiles : i) * 16 + lane / 4, word = 2 * u0 + d0;
            const unsigned int at = q * scales + 4u * word;
            const auto b = is_up ? s_up : s_gate;
            v[i] = u32x4{0u, 0u, 0u, 0u};
            if (word + 4 <= steps) {
                v[i] = __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(at), 0, 0);
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (word + j < steps) v[i][j] = __builtin_amdgcn_raw_buffer_load_b32(b, static_cast<int>(at + 4 * j), 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < kWTiles; ++i) {
            const int q = i * 16 + lane / 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) wscale[wave][q * 16 + ((d0 + j) ^ (q & 15))] = v[i][j];
        }
        wave_lds_fence();
    };
    f32x4 acc[kWTiles];
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Tokens {
        u32x4 x[2];
        u32x2 s;
    };
    // a token row's codes and scale words of a unit; a second step past the
    // row's end is not read
    const unsigned int xo = r * half + g * 16, xso = r * scales;
    const auto load_tokens = [&](int u) {
        const bool both = 2 * u + 1 < steps;
        Tokens v;
        v.x[0] = __builtin_amdgcn_raw_buffer_load_b128(xb, static_cast<int>(xo), u * 128, 0);
        v.s[0] = __builtin_amdgcn_raw_buffer_load_b32(xsb, static_cast<int>(xso), u * 8, 0);
        v.x[1] = u32x4{0u, 0u, 0u, 0u};
        v.s[1] = 0u;
        if (both) {
            v.x[1] = __builtin_amdgcn_raw_buffer_load_b128(xb, static_cast<int>(xo), u * 128 + 64, 0);
            v.s[1] = __builtin_amdgcn_raw_buffer_load_b32(xsb, static_cast<int>(xso), u * 8 + 4, 0);
        }
        return v;
    };
    const auto products = [&](int u, int u0, const u32x4 *from, const Tokens &tok) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (2 * u + h < steps) {
#pragma unroll
                for (int i = 0; i < kWTiles; ++i) {
                    const int q = i * 16 + r;
                    const u32x4 w = from[q * 8 + ((h * 4 + g) ^ (r & 7))];
                    const unsigned int s = wscale[wave][q * 16 + ((2 * (u - u0) + h) ^ r)];
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w), fp4_operand(tok.x[h]), acc[i], kFp4, kFp4,
                                                                             0, static_cast<int>(s >> (8 * g)), 0,
                                                                             static_cast<int>(tok.s[h] >> (8 * g)));
                }
            }
        }
        // the unit is read before anything is copied over it
#pragma unroll
        for (int i = 0; i < kWTiles; ++i) asm volatile("" : "+v"(acc[i]) : : "memory");
    };
    for (int u0 = begin; u0 < end; u0 += kPartUnits) {
        const int stop = min(end, u0 + kPartUnits);
        copy_unit(u0, unit0[wave]);
        if (u0 + 1 < stop) copy_unit(u0 + 1, unit1[wave]);
        Tokens now = load_tokens(u0);
        load_part(u0);
        for (int u = u0; u < stop; u += 2) {
            Tokens next = now;
            if (u + 1 < stop) next = load_tokens(u + 1);
            products(u, u0, unit0[wave], now);
            if (u + 2 < stop) copy_unit(u + 2, unit0[wave]);
            if (u + 1 < stop) {
                if (u + 2 < stop) now = load_tokens(u + 2);
                products(u + 1, u0, unit1[wave], next);
                if (u + 3 < stop) copy_unit(u + 3, unit1[wave]);
            }
        }
    }
    // the sums meet where the weights were
    __syncthreads();
    f32x4(*const part)[kWTiles][kWave] = reinterpret_cast<f32x4(*)[kWTiles][kWave]>(&unit0[0][0]);
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < kOutTiles; i += kStreamWaves) {
        f32x4 v = part[0][i][lane];
        f32x4 u{};
#pragma unroll
        for (int q = 1; q < kStreamWaves; ++q) v += part[q][i][lane];
        if constexpr (SWIGLU) {
            u = part[0][kOutTiles + i][lane];
#pragma unroll
            for (int q = 1; q < kStreamWaves; ++q) u += part[q][kOutTiles + i][lane];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * u[c];
        }
        const int n = n0 + i * 16 + 4 * g;
        if (r < t.rows && n < a.N)
            *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.out) + static_cast<size_t>(t.row0 + r) * a.N + n) =
                pack_bf16x4(v);
    }
}

// ---------------------------------------------------------------------------
// long segments
// ---------------------------------------------------------------------------

// A tile is up to 256 token rows by 256 weight rows.  One workgroup of eight
// waves per CU takes tile after tile: above 128 rows each wave multiplies 128
// token rows by 64 weight rows (128 accumulator registers), otherwise all (up to
// 128) by 32.
//
// A stage (256 channels, two steps) of both operands, up to 64 KB, is copied
// to LDS without passing registers while the stage before it is multiplied,
// across tiles too: the next tile's first stage is on its way during a tile's
// last products and its stores, so neither the search for a tile nor the first
// loads' latency is waited for more than once.  A copy instruction reads 8 whole
// 128-byte lines; the operands' own order, 16 rows to 16 neighbouring lanes,
// would read 64 pieces of 16 bytes.  The two stage buffers are objects of their
// own, so that the compiler, which waits for copies into what it reads, knows
// that the other buffer's copies may stay in flight.
//
// Measured at the prompt case (98304 rows, 64 experts, H = 2048, 2 x 1280
// weight rows, SwiGLU): weights straight to registers 396 us; 128 x 256 tiles
// of four waves, two workgroups per CU, one step per stage, three stages deep
// 336 us; this 309 us (3.3 PFLOP/s).  In copies that leave parts out: no stage
// copies 251, no LDS reads 295, no stores 281, products and barriers alone 170,
// stage copies alone 213.  A stage's copies take about 1.4 us with one stage in
// flight (a quarter of their lines come from beyond the L2), its products 1.1 us,
// and LDS holds no third stage; nothing runs beside a tile's stores.  Asking the
// L2 for lines one to three stages ahead (332 and more), reading operands across
// the barriers (330) and raising the waves' priority (320) did not help.
constexpr int kTileRows = 256;
constexpr int kTileWeights = 256;
constexpr int kTileThreads = kTileWaves * kWave;
constexpr int kCus = 256;                    // workgroups that run at once
constexpr int kStageVecs = (kTileRows + kTileWeights) * 8;   // 16-byte vectors: 128 bytes of every token row, then weight row

// A row's scale bytes of steps 4S .. 4S+3 (words d0 .. d3, byte g of each the
// block of lane group g) as one word per lane group, step s in byte s.
__device__ __forceinline__ u32x4 transpose_scales(u32x4 d) {
    const unsigned int a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
    const unsigned int b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    return u32x4{__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                 __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
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

struct TileLds {
    u32x4 *stage0, *stage1, *scale;   // scale: token rows, then weight rows
};

// What a tile's copies need besides the tile: this lane's first offsets into
// the weights' and the tokens' rows, and its row of scales.
struct TileCopies {
    unsigned int wo, xo, so;
    int slot;                                 // the scales' place in LDS
    __amdgpu_buffer_rsrc_t w[2], x, scales;   // this wave's first and last 16 weight rows, the token rows, this wave's scales
    bool wide;                                // more than 128 token rows
};

// First weight row of a tile, among all experts', and how many there are.
template <bool SWIGLU>
__device__ __forceinline__ size_t first_weight_row(const ExpertGemmArgs &a, const RowTile &t, unsigned int &rows) {
    constexpr int kOutRows = SWIGLU ? kTileWeights / 2 : kTileWeights;
    const int n0 = t.ntile * kOutRows;
    rows = min(kOutRows, a.N - n0);
    return t.expert * (SWIGLU ? 2 * static_cast<size_t>(a.N) : a.N) + n0;
}

// Lane l's vector of a copy: row l/8 of the eight, chunk c at place l%8, where
// chunk c (32 channels) of row q lies at c ^ (q % 8): eight rows' chunk c are
// then in eight different groups of banks (tile_copies.h).
template <bool SWIGLU>
__device__ __forceinline__ TileCopies tile_copies(const ExpertGemmArgs &a, const RowTile &t) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const unsigned int half = a.H / 2, scales = a.H / kMx4Block;
    const bool wide = t.rows > 128;
    TileCopies c;
    c.wo = first_weight(SWIGLU, wide, wave, lane) * half + lane_chunk(lane);
    c.xo = first_token(wave, lane) * half + lane_chunk(lane);
    // scales: a row per thread.  Waves 0 to 3 weight rows (SWIGLU: 0 and 1 gate,
    // 2 and 3 up), 4 to 7 token rows.
    if (wave >= 4) {
        c.so = (tid - 256) * scales;
        c.slot = tid - 256;
    } else {
        const int n = SWIGLU ? tid & 127 : tid, up = SWIGLU && wave >= 2 ? 1 : 0;
        c.so = n * scales;
        c.slot = kTileRows + (!SWIGLU ? n : (wide ? n / 32 * 64 + (n & 31) + up * 32 : n / 16 * 32 + (n & 15) + up * 16));
    }
    unsigned int rows;
    const size_t first = first_weight_row<SWIGLU>(a, t, rows), up_first = first + (SWIGLU ? a.N : 0);
    c.wide = wide;
    c.w[0] = buffer_of(a.w + (wide && (wave & 1) ? up_first : first) * half, rows * half);
    c.w[1] = buffer_of(a.w + (!wide || (wave & 1) ? up_first : first) * half, rows * half);
    c.x = buffer_of(a.x + static_cast<size_t>(t.row0) * half, t.rows * half);
    c.scales = wave >= 4 ? buffer_of(a.xs + static_cast<size_t>(t.row0) * scales, t.rows * scales)
                         : buffer_of(a.ws + (wave >= 2 ? up_first : first) * scales, rows * scales);
    return c;
}

// Copies channels 256*s .. of the tile into `stage`.  A last stage of 128
// channels leaves the second half of each row alone (the offset is past the
// end there).  Every copy's offset is made here from one per lane and operand:
// kept from stage to stage they would take a register each.
template <bool SWIGLU, int XCOPIES>
__device__ __forceinline__ void copy_stage(const ExpertGemmArgs &a, const TileCopies &c, int s, u32x4 *stage, bool wide) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int half = a.H / 2;
    const unsigned int gone = left_out(a.H, s, lane);
    unsigned int wo = c.wo, xo = c.xo;
    asm volatile("" : "+v"(wo), "+v"(xo));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const CopyAt at = copy_at(wo, weight_step(SWIGLU, wide, i, j), half, s, gone);
            copy_to_lds(c.w[i], stage + (kTileRows + wave * 32 + i * 16 + j * 8) * 8, at.lane, at.uniform);
        }
#pragma unroll
    for (int i = 0; i < XCOPIES; ++i) {
        const CopyAt at = copy_at(xo, token_step(i), half, s, gone);
        copy_to_lds(c.x, stage + (i * kTileWaves + wave) * 64, at.lane, at.uniform);
    }
}

// Scale words 4S .. 4S+3 of this thread's row; those past the row's end are
// not read.
__device__ __forceinline__ u32x4 load_scales(const ExpertGemmArgs &a, const TileCopies &c, int S) {
    const int steps = a.H / kStep;
    if (4 * S + 4 <= steps) return __builtin_amdgcn_raw_buffer_load_b128(c.scales, static_cast<int>(c.so), S * 16, 0);
    u32x4 d = {0u, 0u, 0u, 0u};
    d[0] = __builtin_amdgcn_raw_buffer_load_b32(c.scales, static_cast<int>(c.so), S * 16, 0);
    if (4 * S + 1 < steps) d[1] = __builtin_amdgcn_raw_buffer_load_b32(c.scales, static_cast<int>(c.so + 4), S * 16, 0);
    if (4 * S + 2 < steps) d[2] = __builtin_amdgcn_raw_buffer_load_b32(c.scales, static_cast<int>(c.so + 8), S * 16, 0);
    return d;
}

// Tile number `tile` from the table; every lane calls it.
__device__ __forceinline__ RowTile tile_at(const ExpertGemmArgs &a, const SegTable &segs, int tile) {
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

// One tile whose first stage is on its way to stage 0 and whose first scales
// are on their way to `first_scales`.  next_first() asks for the next tile's,
// into the same places.  TT token tiles of 16 rows and WT weight tiles per wave.
template <int TT, int WT, bool SWIGLU, typename NextFirst>
__device__ __forceinline__ void run_tile(const ExpertGemmArgs &a, const RowTile &t, const TileCopies &copies, const TileLds &lds,
                                         u32x4 &first_scales, NextFirst &&next_first) {
    constexpr int kWeightWaves = kTileWeights / (16 * WT), kX = WT == 4 ? 4 : (TT * 2 + kTileWaves - 1) / kTileWaves;
    constexpr bool kWide = WT == 4;
    constexpr int kOut = SWIGLU ? WT / 2 : WT;                 // 16-channel tiles of output per wave
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // what follows from it is made once per tile, not kept from tile to tile
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int ww = wave % kWeightWaves, q0 = (wave / kWeightWaves) * 128;   // the wave's weight rows and token rows
    const int r = lane & 15, g = lane >> 4;
    const int steps = a.H / kStep, stages = (steps + 1) / 2;
    f32x4 acc[TT][WT];
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < WT; ++i) acc[m][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    unsigned int sca[WT], scb[TT];
    // Where the lane's operands of either step of a stage and its scales begin:
    // values of their own, so that every read is one of them and a constant.
    int wat0 = (kTileRows + ww * WT * 16 + r) * 8 + (g ^ (r & 7)), wat1 = (kTileRows + ww * WT * 16 + r) * 8 + ((4 + g) ^ (r & 7));
    int xat0 = (q0 + r) * 8 + (g ^ (r & 7)), xat1 = (q0 + r) * 8 + ((4 + g) ^ (r & 7));
    int wsat = (kTileRows + ww * WT * 16 + r) * 4 + g, xsat = (q0 + r) * 4 + g;
    asm volatile("" : "+v"(wat0), "+v"(wat1), "+v"(xat0), "+v"(xat1), "+v"(wsat), "+v"(xsat));
    // Step h of a stage, the stage's byte b0 + h of the scales' words.
    const auto products = [&](const u32x4 *stage, auto byte_, int h) {
        constexpr int byte = decltype(byte_)::value;
        u32x4 wv[WT];
#pragma unroll
        for (int i = 0; i < WT; ++i) wv[i] = stage[(h ? wat1 : wat0) + i * 128];
#pragma unroll
        for (int m = 0; m < TT; ++m) {
            const u32x4 b = stage[(h ? xat1 : xat0) + m * 128];
#pragma unroll
            for (int i = 0; i < WT; ++i)
                acc[m][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wv[i]), fp4_operand(b), acc[m][i], kFp4,
                                                                            kFp4, byte, static_cast<int>(sca[i]), byte,
                                                                            static_cast<int>(scb[m]));
        }
        // a step's products stay in their step: the compiler would move them,
        // with their operands, behind the barriers
#pragma unroll
        for (int m = 0; m < TT; ++m)
#pragma unroll
            for (int i = 0; i < WT; ++i) asm volatile("" : "+v"(acc[m][i]));
    };
    lds.scale[copies.slot] = transpose_scales(first_scales);
    barrier_after<0>();                                        // stage 0 has arrived
    for (int s = 0; s < stages; s += 2) {
        const bool second = s + 1 < stages, more = s + 2 < stages;
        if (second) copy_stage<SWIGLU, kX>(a, copies, s + 1, lds.stage1, kWide);
        u32x4 next_scales = {0u, 0u, 0u, 0u};
        if (more) next_scales = load_scales(a, copies, s / 2 + 1);
        const unsigned int *p = reinterpret_cast<const unsigned int *>(lds.scale);
#pragma unroll
        for (int i = 0; i < WT; ++i) sca[i] = p[wsat + i * 64];
#pragma unroll
        for (int m = 0; m < TT; ++m) scb[m] = p[xsat + m * 64];
        products(lds.stage0, std::integral_constant<int, 0>{}, 0);
        if (2 * s + 1 < steps) products(lds.stage0, std::integral_constant<int, 1>{}, 1);
        barrier_after<0>();                                    // stage s + 1 has arrived, stage s and its scales are free
        if (more)
            copy_stage<SWIGLU, kX>(a, copies, s + 2, lds.stage0, kWide);
        else
            next_first();
        if (second) {
            products(lds.stage1, std::integral_constant<int, 2>{}, 0);
            if (2 * s + 3 < steps) products(lds.stage1, std::integral_constant<int, 3>{}, 1);
        }
        if (more) {
            lds.scale[copies.slot] = transpose_scales(next_scales);
            barrier_after<0>();                                // stage s + 2 has arrived, stage s + 1 is free
        }
    }
    barrier_after<63>();                                       // stage 1 is free; the next tile's first stage may be on its way
    // A lane holds token r of tile m, four channels from 4g of tile i.  Up to two
    // tiles at a time pass through LDS (4 KB of the wave's own) so that a store
    // instruction writes runs of whole rows.  Rows of kChunks 16-byte chunks,
    // chunk c of row q at c ^ turn(q), against bank conflicts.  Stores outside
    // the tile's rows fall past the buffer's end, those past N are sent there.  They
    // pass the caches: 470 MB of results 584 -> 573 us, 268 MB with the quantise
    // behind it 230 -> 214, 46 MB or less with it 1 % more.
    constexpr int kChunks = 2 * kOut, kRowsPerStore = kWave / kChunks;
    const auto turn = [](int q) { return (q * kChunks / 8) & (kChunks - 1); };
    const unsigned int row_bytes = static_cast<unsigned int>(a.N) * 2u;
    const auto ob = buffer_of(static_cast<char *>(a.out) + static_cast<size_t>(t.row0) * row_bytes, t.rows * row_bytes);
    const int n0 = (t.ntile * kWeightWaves + ww) * (kOut * 16);
    u32x4 *const mine = lds.stage1 + wave * 256;
#pragma unroll
    for (int m0 = 0; m0 < TT; m0 += 2) {
#pragma unroll
        for (int m = m0; m < m0 + 2; ++m) {
            const int q = (m - m0) * 16 + r;
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                f32x4 v = acc[m][i];
                if constexpr (SWIGLU) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * acc[m][i + kOut][c];
                }
                reinterpret_cast<u32x2 *>(mine)[(q * kChunks + ((2 * i + (g >> 1)) ^ turn(q))) * 2 + (g & 1)] = pack_bf16x4(v);
            }
        }
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < 32 / kRowsPerStore; ++j) {
            const int q = j * kRowsPerStore + lane / kChunks, c = lane % kChunks;
            const u32x4 v = mine[q * kChunks + (c ^ turn(q))];
            const int n = n0 + c * 8;
            const unsigned int at = n < a.N ? (q0 + m0 * 16 + q) * row_bytes + 2u * n : kPastEnd;
            __builtin_amdgcn_raw_buffer_store_b128(v, ob, static_cast<int>(at), 0, kNonTemporal);
        }
        wave_lds_fence();
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kTileThreads, 2) void k_expert_tile(ExpertGemmArgs a, int tiles_n) {
    __shared__ u32x4 stage0[kStageVecs], stage1[kStageVecs];
    __shared__ u32x4 scale[kTileRows + kTileWeights];
    __shared__ SegTable segs;
    __shared__ int2 s_scan[kTileWaves];
    const int tid = threadIdx.x;
    // the table: three segments per thread, every load at once
    constexpr int kPer = kMaxSegments / kTileThreads;
    int first[kPer], n[kPer], tiles = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) load_segment(a, tid * kPer + j, first[j], n[j]);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        n[j] = segment_rows(a, tid * kPer + j, first[j], n[j]);
        tiles += (n[j] + kTileRows - 1) / kTileRows;
    }
    int2 all;
    int at = block_exclusive_scan2<kTileWaves>(make_int2(tiles, 0), s_scan, all).x;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        if (i < a.nseg) {
            segs.before[i] = at * tiles_n;
            segs.first[i] = first[j];
            segs.rows[i] = n[j];
        }
        at += (n[j] + kTileRows - 1) / kTileRows;
    }
    if (tid == 0) segs.before[a.nseg] = all.x * tiles_n;
    __syncthreads();
    // Rounds of kCus tiles.  Runs of neighbouring tiles go to the workgroups of one
    // XCD, whose L2 then serves the tiles' common weights and tokens.  Where the
    // last round has at most a half or a quarter of them, its tiles are taken in
    // two or four parts of 128 or 64 token rows.  Measured without / with (us; E
    // experts, about m rows each): E=8 H=7168 N=2048 m=128 48 / 30, m=256 49 / 37,
    // m=1024 112 / 98; E=64 H=2048 N=1408 m=256 58 / 53; E=32 H=5120 N=1536 m=700
    // 133 / 126.
    const int total = __builtin_amdgcn_readfirstlane(all.x) * tiles_n;
    const int whole = total / kCus * kCus, rest = total - whole;
    const int halvings = rest * 4 <= kCus ? 2 : (rest * 2 <= kCus ? 1 : 0), items = whole + (rest << halvings);
    const int place = static_cast<int>(blockIdx.x) / kXcds, xcd = static_cast<int>(blockIdx.x) % kXcds;
    // What this workgroup takes in a round; false: nothing, then or later.
    const auto tile_of = [&](int round, RowTile &t) {
        const int left = min(items - round * kCus, kCus), run = (left + kXcds - 1) / kXcds, at = xcd * run + place;
        if (place >= run || at >= left) return false;
        const int item = round * kCus + at, cut = item < whole ? 0 : halvings;
        t = tile_at(a, segs, item - (cut ? item - whole - ((item - whole) >> cut) : 0));
        const int part_rows = kTileRows >> cut, skip = cut ? (((item - whole) & ((1 << cut) - 1)) * part_rows) : 0;
        t.row0 += skip;
        t.rows = __builtin_amdgcn_readfirstlane(min(t.rows - skip, part_rows));
        return t.rows > 0;
    };
    const TileLds lds{stage0, stage1, scale};
    RowTile t;
    if (!tile_of(0, t)) return;                                // the same for every wave
    u32x4 scales;
    {
        const TileCopies c = tile_copies<SWIGLU>(a, t);
        scales = load_scales(a, c, 0);
        copy_stage<SWIGLU, 4>(a, c, 0, stage0, c.wide);
    }
    for (int round = 1;; ++round) {
        const TileCopies copies = tile_copies<SWIGLU>(a, t);
        RowTile nt{};
        bool more = false;
        const auto next_first = [&]() {
            more = tile_of(round, nt);
            if (!more) return;
            const TileCopies nc = tile_copies<SWIGLU>(a, nt);
            scales = load_scales(a, nc, 0);
            copy_stage<SWIGLU, 4>(a, nc, 0, stage0, nc.wide);
        };
        if (t.rows > 128)
            run_tile<8, 4, SWIGLU>(a, t, copies, lds, scales, next_first);
        else if (t.rows > 64)
            run_tile<8, 2, SWIGLU>(a, t, copies, lds, scales, next_first);
        else if (t.rows > 32)
            run_tile<4, 2, SWIGLU>(a, t, copies, lds, scales, next_first);
        else
            run_tile<2, 2, SWIGLU>(a, t, copies, lds, scales, next_first);
        if (!more) return;
        t = nt;
    }
}

// Most row tiles of BM rows that any routing of this shape can have.
int64_t most_tiles(const ExpertGemmArgs &a, int BM) {
    const int64_t used = std::min<int64_t>(a.nseg, a.entries);
    return std::min(a.entries / BM + used, used * ((a.max_count + BM - 1) / BM));
}

// Segments with a row, if the routing is at random, and the bytes of their weights.
double used_segments(const ExpertGemmArgs &a) {
    return std::max(1.0, a.nseg * -std::expm1(-static_cast<double>(a.entries) / a.nseg));
}
double weight_bytes(const ExpertGemmArgs &a) { return used_segments(a) * (a.swiglu ? 2.0 : 1.0) * a.N * a.H * (17.0 / 32.0); }

// Weights that the Infinity Cache (256 MB) does not hold from call to call are
// read past the caches by the streaming kernel.  Ordinary / past the caches (us,
// 7168 x 2048 weights each): 24 experts with a row, 190 MB, 25.8 / 28.9; 35,
// 270 MB, 41.8 / 44.2; 55, 432 MB, 76 / 68.5; 252, 1.96 GB, 328 / 306.
bool weights_once(const ExpertGemmArgs &a) { return weight_bytes(a) > 320.0e6; }

// The rule between the two kernels: the sooner by these estimates, in
// microseconds, which near the crossing hold what was measured within about a
// fifth.  Experts with a row: as many as a routing at random leaves with one.
//   stream: a start of 4 us; a workgroup's work is one 16-row tile by 32 weight
//     rows, with about 7 steps' worth of its own start and end; 3200 such steps a
//     microsecond, or the weights at 6.0 TB/s (6.4 past the caches).
//   tile: a start of 6 us, then rounds of 256 workgroups one tile each, 0.38 us a
//     step and 0.0015 more for each row of a tile, or of a part of it in the last
//     round; or the weights at 5.2 TB/s.
// Measured, stream / tile (us; E experts with m rows each, M weight rows):
//   E=256 H=7168 M=2048  m=1 197 / 279   m=4 306 / 384   m=8 342 / 391   m=12 412 / 397
//   E=256 H=2048 M=7168  m=1 274 / 234   m=4 411 / 387   m=16 659 / 406
//   E=64  H=1024 M=4096  m=1 25 / 21     m=12 48 / 34
//   E=64  H=2048 M=2048  m=1 20 / 26     m=4 34 / 32     m=12 38 / 33
//   E=8   H=7168 M=2048  m=4 14 / 28     m=32 26 / 29    m=64 42 / 30    m=256 134 / 38
//   E=4   H=7168 M=512   m=128 16 / 28   m=256 24 / 29
bool long_segments(const ExpertGemmArgs &a) {
    if (a.entries == 0) return false;
    const double rows = static_cast<double>(a.entries), used = used_segments(a), weights = weight_bytes(a);
    const double M = a.swiglu ? 2.0 * a.N : a.N, steps = a.H / kStep;
    const double stream_tiles = std::max(used, rows / kStreamRows + used / 2), row_tiles = std::max(used, rows / kTileRows + used / 2);
    const double stream = 4 + std::max(stream_tiles * (M / (16 * kWTiles)) * (steps + 7) / 3200, weights / (weights_once(a) ? 6.4e6 : 6.0e6));
    const double tiles = row_tiles * std::ceil(M / kTileWeights), whole = std::floor(tiles / kCus), rest = tiles - whole * kCus;
    const double last_rows = rest * 4 <= kCus ? kTileRows / 4 : (rest * 2 <= kCus ? kTileRows / 2 : kTileRows);
    const auto step_us = [](double tile_rows) { return 0.38 + 0.0015 * tile_rows; };
    const double tile_rows = std::min(rows / used, static_cast<double>(kTileRows));
    const double rounds_us = whole * step_us(tile_rows) + (rest > 0 ? step_us(std::min(tile_rows, last_rows)) : 0);
    return 6 + std::max(steps * rounds_us, weights / 5.2e6) < stream;
}

struct Grid {
    int tiles_n;
    int64_t tiles;    // at most; a multiple of the XCD count
    int64_t blocks;
};
Grid grid_of(const ExpertGemmArgs &a) {
    const bool tiles = long_segments(a);
    const int weights = tiles ? kTileWeights : kWTiles * 16, out = a.swiglu ? weights / 2 : weights;
    Grid g;
    g.tiles_n = (a.N + out - 1) / out;
    const int64_t all = most_tiles(a, tiles ? kTileRows : kStreamRows) * g.tiles_n;
    g.tiles = (all + kXcds - 1) / kXcds * kXcds;
    g.blocks = tiles ? std::min<int64_t>(4 * g.tiles, kCus) : g.tiles;   // a tile may be taken in four parts
    return g;
}

}  // namespace

bool expert_gemm_grid_ok(const ExpertGemmArgs &a) {
    const Grid g = grid_of(a);
    return g.tiles <= INT32_MAX - kCus && g.blocks * std::max(kStreamWaves * kWave, kTileThreads) <= kMaxLaunchThreads;
}

hipError_t launch_expert_gemm_mx4(const ExpertGemmArgs &a, hipStream_t s) {
    const Grid g = grid_of(a);
    if (g.blocks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(g.blocks)), stream_block(kStreamWaves * kWave), tile_block(kTileThreads);
    if (long_segments(a)) {
        if (a.swiglu)
            hipLaunchKernelGGL(k_expert_tile<true>, grid, tile_block, 0, s, a, g.tiles_n);
        else
            hipLaunchKernelGGL(k_expert_tile<false>, grid, tile_block, 0, s, a, g.tiles_n);
    } else if (weights_once(a)) {
        if (a.swiglu)
            hipLaunchKernelGGL((k_expert_stream<true, true>), grid, stream_block, 0, s, a, g.tiles_n);
        else
            hipLaunchKernelGGL((k_expert_stream<false, true>), grid, stream_block, 0, s, a, g.tiles_n);
    } else {
        if (a.swiglu)
            hipLaunchKernelGGL((k_expert_stream<true, false>), grid, stream_block, 0, s, a, g.tiles_n);
        else
            hipLaunchKernelGGL((k_expert_stream<false, false>), grid, stream_block, 0, s, a, g.tiles_n);
    }
    return hipGetLastError();
}

}  // namespace moe
