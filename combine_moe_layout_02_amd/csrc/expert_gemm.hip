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
// holds enough workgroups for any routing; a workgroup finds its tile by
// scanning the segments' row counts (a wave-wide prefix sum), and one past the
// last tile returns.
//
// A workgroup takes 16 rows of one segment and 64 weight rows; its four waves
// split the channels and join their sums in LDS.
#include "expert_gemm.h"
#include "mx4.h"

#include <algorithm>
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

// find_tile with PER segments per lane (nseg <= 64 * PER).
template <int BM, int PER>
__device__ __forceinline__ bool find_tile_per(const ExpertGemmArgs &a, int block, int tiles_n, RowTile &t) {
    const int lane = threadIdx.x & (kWave - 1);
    // every load at once: the whole search waits for memory one time
    int first[PER], n[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = lane * PER + j;
        const bool in = i < a.nseg;
        first[j] = in ? (a.seg_offset != nullptr ? a.seg_offset[i] : a.offset[i]) : 0;
        n[j] = in ? (a.seg_offset != nullptr ? a.seg_offset[i + 1] : a.count[i]) : 0;
    }
    int tiles = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (a.seg_offset != nullptr) n[j] -= first[j];
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

constexpr int kStreamRows = 16;  // token rows of a workgroup
constexpr int kStreamWaves = 4;
constexpr int kWTiles = 4;     // 16-row weight tiles of a workgroup (SWIGLU: half gate, half up)

// U channel steps from step s: every load first, then the products.
template <int U>
__device__ __forceinline__ void stream_steps(const uint8_t *const (&wp)[kWTiles], const uint8_t *const (&wsp)[kWTiles],
                                             const uint8_t *xp, const uint8_t *xsp, int s, int shift,
                                             f32x4 (&acc)[kWTiles]) {
    u32x4 w[U][kWTiles], x[U];
    unsigned int ws[U][kWTiles], xs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < kWTiles; ++i) {
            w[u][i] = *reinterpret_cast<const u32x4 *>(wp[i] + static_cast<size_t>(s + u) * (kStep / 2));
            ws[u][i] = *reinterpret_cast<const unsigned int *>(wsp[i] + static_cast<size_t>(s + u) * 4);
        }
        x[u] = *reinterpret_cast<const u32x4 *>(xp + static_cast<size_t>(s + u) * (kStep / 2));
        xs[u] = *reinterpret_cast<const unsigned int *>(xsp + static_cast<size_t>(s + u) * 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < kWTiles; ++i)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w[u][i]), fp4_operand(x[u]), acc[i],
                                                                     kFp4, kFp4, 0, static_cast<int>(ws[u][i] >> shift),
                                                                     0, static_cast<int>(xs[u] >> shift));
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kStreamWaves * kWave) void k_expert_stream(ExpertGemmArgs a, int tiles_n) {
    constexpr int kOutTiles = SWIGLU ? kWTiles / 2 : kWTiles;
    __shared__ f32x4 part[kStreamWaves][kWTiles][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    RowTile t;
    if (!find_tile<kStreamRows>(a, blockIdx.x, tiles_n, t)) return;   // the same for every wave
    const int row0 = t.row0, rows = t.rows, expert = t.expert, n0 = t.ntile * (kOutTiles * 16);
    // lane = 16*g + r: row r of each operand, channels 32*g .. 32*g+31 of a step
    const int r = lane & 15, g = lane >> 4;
    const size_t half = a.H / 2, scales = a.H / kMx4Block;
    const size_t M = SWIGLU ? 2 * static_cast<size_t>(a.N) : a.N;
    const uint8_t *wp[kWTiles], *wsp[kWTiles];
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) {
        const int n = min(n0 + (i % kOutTiles) * 16 + r, a.N - 1);        // rows past N repeat the last one
        const size_t row = expert * M + n + (i >= kOutTiles ? a.N : 0);
        wp[i] = a.w + row * half + g * 16;
        wsp[i] = a.ws + row * scales;
    }
    const size_t xrow = row0 + min(r, rows - 1);
    const uint8_t *xp = a.x + xrow * half + g * 16, *xsp = a.xs + xrow * scales;
    f32x4 acc[kWTiles];
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = a.H / kStep;
    int s = steps * wave / kStreamWaves;
    const int end = steps * (wave + 1) / kStreamWaves;
    for (; s + 4 <= end; s += 4) stream_steps<4>(wp, wsp, xp, xsp, s, 8 * g, acc);
    for (; s < end; ++s) stream_steps<1>(wp, wsp, xp, xsp, s, 8 * g, acc);
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
        if (r < rows && n < a.N)
            *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.out) + static_cast<size_t>(row0 + r) * a.N + n) =
                pack_bf16x4(v);
    }
}

// ---------------------------------------------------------------------------
// long segments
// ---------------------------------------------------------------------------

// 128 token rows by 256 weight rows, four waves of 128 x 64 (128 accumulator
// registers).  A step (128 channels) is 16 KB of weights and 8 KB of tokens,
// copied to LDS without passing registers, three steps deep: a step's copies
// are issued two steps before its products.  Each copy instruction reads whole
// 64-byte runs (16 rows), which the operands' own order, 16 rows to 16
// neighbouring lanes, would not: loading weights straight into the operands'
// registers took 396 us at the prompt case (98304 rows, H = 2048, 2 x 1280
// weight rows of 64 experts) against 336 us here.  The compiler knows each
// stage as an object of its own and so waits for that stage's copies alone.
constexpr int kTileRows = 128;
constexpr int kTileWeights = 256; // 64 for each wave
constexpr int kTileWaves = 4;
constexpr int kStageVecs = (kTileRows + kTileWeights) * 4;   // 16-byte vectors: token rows, then weight rows

// A row's scale bytes of steps 4S .. 4S+3 (words d0 .. d3, byte g of each the
// block of lane group g) as one word per lane group, step s in byte s.
__device__ __forceinline__ u32x4 transpose_scales(u32x4 d) {
    const unsigned int a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
    const unsigned int b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    return u32x4{__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                 __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
}

// A raw buffer over `bytes` bytes: loads take a uniform base and a 32-bit
// offset per lane, and read zeros past the end.
constexpr int kBufferRsrcWord3 = 0x00020000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base, unsigned int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, static_cast<int>(bytes), kBufferRsrcWord3);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, unsigned int offset, int uniform_offset) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(offset), uniform_offset, 0);
}

typedef __attribute__((address_space(3))) void lds_void;

// Copies 16 bytes per lane to 1 KiB of LDS from `to` (the same in every lane).
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t b, u32x4 *to, unsigned int offset, int uniform_offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, reinterpret_cast<lds_void *>(reinterpret_cast<uintptr_t>(to)), 16,
                                             static_cast<int>(offset), uniform_offset, 0, 0);
}

// Workgroup barrier that first waits until at most N of the wave's global
// loads and copies are in flight, and for its LDS writes.  A fence would wait
// for every copy to LDS; here the ones that N leaves are for later steps.
template <int N>
__device__ __forceinline__ void barrier_after_copies() {
    static_assert(N < 16, "the low bits of the count alone");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070 | N);   // vmcnt(N), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// Orders the wave's own LDS accesses; nothing else uses the memory between.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// TT 16-row token tiles of the workgroup's rows.
template <int TT, bool SWIGLU>
__device__ __forceinline__ void tile_product(const ExpertGemmArgs &a, const RowTile &t, u32x4 *stage0, u32x4 *stage1,
                                             u32x4 *stage2, u32x4 *scale) {
    constexpr int kOutPerWave = SWIGLU ? 32 : 64;
    constexpr int kOutRows = kTileWaves * kOutPerWave;
    constexpr int kTokCopies = TT >= 4 ? TT / 4 : 1;   // a wave's copies of token rows per step
    constexpr int kCopies = 4 + kTokCopies;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const unsigned int half = a.H / 2, scales = a.H / kMx4Block;
    const size_t M = SWIGLU ? 2 * static_cast<size_t>(a.N) : a.N;
    const int n0 = t.ntile * kOutRows;
    const int steps = a.H / kStep;
    // Weight row j of the workgroup: wave j/64, tile (j/16)%4, row j%16 of it;
    // with SWIGLU tiles 2 and 3 are the up rows of tiles 0 and 1.  Rows past
    // the last one read as zeros.
    const size_t first = t.expert * M + n0;
    const unsigned int wrows = min(kOutRows, a.N - n0);
    const size_t up = SWIGLU ? a.N : 0;
    const auto w_gate = buffer_of(a.w + first * half, wrows * half), w_up = buffer_of(a.w + (first + up) * half, wrows * half);
    const auto s_gate = buffer_of(a.ws + first * scales, wrows * scales),
               s_up = buffer_of(a.ws + (first + up) * scales, wrows * scales);
    const auto xb = buffer_of(a.x + static_cast<size_t>(t.row0) * half, t.rows * half),
               xsb = buffer_of(a.xs + static_cast<size_t>(t.row0) * scales, t.rows * scales);
    const auto weight_row = [&](int j) -> unsigned int {
        return (j / 64) * kOutPerWave + (SWIGLU ? (j / 16) & 1 : (j / 16) & 3) * 16 + (j & 15);
    };
    // A copy instruction moves 16 rows: lane l fills vector l of the 64, row
    // l/4.  Chunk c (32 channels) of row q lies at 4q + (c ^ (q/2 % 4)), so that
    // eight rows' chunk c are in eight different groups of banks.
    const int q16 = lane / 4;
    const unsigned int chunk = ((lane & 3) ^ ((q16 >> 1) & 3)) * 16;
    unsigned int wo[4], xo[kTokCopies];
    int xat[kTokCopies];
#pragma unroll
    for (int i = 0; i < 4; ++i) wo[i] = weight_row(wave * 64 + i * 16 + q16) * half + chunk;
#pragma unroll
    for (int i = 0; i < kTokCopies; ++i) {
        xat[i] = (wave * kTokCopies + i) & (TT - 1);   // two waves copy the same rows where there are fewer tiles than waves
        xo[i] = (xat[i] * 16 + q16) * half + chunk;
    }
    // scales: a thread stages a weight row (with SWIGLU the first two waves the
    // gate rows, the others the up rows) and a token row; where there are more
    // threads than rows some stage the same one
    const int wrow = SWIGLU ? (tid & 127) / 32 * 64 + (tid >> 7) * 32 + (tid & 31) : tid;
    const unsigned int wso = weight_row(wrow) * scales, xso = (tid & (TT * 16 - 1)) * scales;
    const auto sb = SWIGLU && wave >= 2 ? s_up : s_gate;

    f32x4 acc[TT][4];
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 sw, sx;
    const auto copy_step = [&](int k, u32x4 *stage) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            copy_to_lds(i < 2 ? w_gate : w_up, stage + (kTileRows + wave * 64 + i * 16) * 4, wo[i], k * (kStep / 2));
#pragma unroll
        for (int i = 0; i < kTokCopies; ++i) copy_to_lds(xb, stage + xat[i] * 64, xo[i], k * (kStep / 2));
    };
    // Words past a row's end are another row's or zeros: nothing uses them.
    const auto load_s = [&](int S) {
        sw = load16(sb, wso, S * 16);
        sx = load16(xsb, xso, S * 16);
    };
    const auto store_s = [&]() {
        scale[kTileRows + wrow] = transpose_scales(sw);
        scale[tid & (TT * 16 - 1)] = transpose_scales(sx);
    };
    unsigned int sca[4], scb[TT];
    const auto read_s = [&]() {
        const unsigned int *p = reinterpret_cast<const unsigned int *>(scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) sca[i] = p[(kTileRows + wave * 64 + i * 16 + r) * 4 + g];
#pragma unroll
        for (int m = 0; m < TT; ++m) scb[m] = p[(m * 16 + r) * 4 + g];
    };
    // The products of step k, from `stage`.
    const auto products = [&](int k, const u32x4 *stage) {
        if ((k & 3) == 0) {
            read_s();
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) sca[i] >>= 8;
#pragma unroll
            for (int m = 0; m < TT; ++m) scb[m] >>= 8;
        }
        u32x4 wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[i] = stage[(kTileRows + wave * 64 + i * 16 + r) * 4 + (g ^ ((r >> 1) & 3))];
#pragma unroll
        for (int m = 0; m < TT; ++m) {
            const u32x4 b = stage[(m * 16 + r) * 4 + (g ^ ((r >> 1) & 3))];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[m][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wv[i]), fp4_operand(b), acc[m][i], kFp4,
                                                                            kFp4, 0, static_cast<int>(sca[i]), 0,
                                                                            static_cast<int>(scb[m]));
        }
        // a step's products stay in their step: the compiler would move them,
        // with their operands, behind the barrier
#pragma unroll
        for (int m = 0; m < TT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(acc[m][i]));
    };
    // Scales of the next four steps: asked for after the first of four, when
    // every wave has read the last ones, and stored in the third.
    const auto scales_early = [&](int k) {
        if ((k & 3) == 0 && k + 4 < steps) load_s(k / 4 + 1);
    };
    const auto scales_late = [&](int k) {
        if ((k & 3) == 2 && k + 2 < steps) store_s();
    };
    // A step with two more behind it; `next` gets step k+2.
    const auto step = [&](int k, const u32x4 *stage, u32x4 *next) {
        copy_step(k + 2, next);
        products(k, stage);
        scales_late(k);
        barrier_after_copies<kCopies>();   // step k+1 has arrived: only step k+2 is in flight
        scales_early(k);
    };
    const auto last_step = [&](int k, const u32x4 *stage, u32x4 *next) {
        if (k + 2 < steps) copy_step(k + 2, next);
        products(k, stage);
        scales_late(k);
        barrier_after_copies<0>();
        scales_early(k);
    };
    load_s(0);
    copy_step(0, stage0);
    store_s();
    if (steps > 1) {
        copy_step(1, stage1);
        barrier_after_copies<kCopies>();
    } else {
        barrier_after_copies<0>();
    }
    int k = 0;
    for (; k + 5 <= steps; k += 3) {
        step(k, stage0, stage2);
        step(k + 1, stage1, stage0);
        step(k + 2, stage2, stage1);
    }
    // one to four steps are left
    last_step(k, stage0, stage2);
    if (k + 1 < steps) last_step(k + 1, stage1, stage0);
    if (k + 2 < steps) last_step(k + 2, stage2, stage1);
    if (k + 3 < steps) last_step(k + 3, stage0, stage2);
    // A lane holds token r of tile m, four channels from 4g of tile i.  Two
    // tiles at a time pass through LDS (4 KB of the wave's own) so that a store
    // instruction writes runs of 64 channels (32 with SWIGLU) of a row.  Rows of
    // kChunks 16-byte chunks, chunk c of row q at c ^ (q % kChunks) (SWIGLU: of
    // q/2), against bank conflicts.  Stores outside the tile's rows fall past
    // the buffer's end, those past N are sent there.
    constexpr int kOut = SWIGLU ? 2 : 4, kChunks = 2 * kOut;
    const unsigned int row_bytes = static_cast<unsigned int>(a.N) * 2u;
    const __amdgpu_buffer_rsrc_t ob = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<char *>(a.out) + static_cast<size_t>(t.row0) * row_bytes, 0, static_cast<int>(t.rows * row_bytes),
        kBufferRsrcWord3);
    u32x4 *const mine = stage0 + wave * 256;
#pragma unroll
    for (int m0 = 0; m0 < TT; m0 += 2) {
#pragma unroll
        for (int m = m0; m < m0 + 2; ++m) {
            const int q = (m - m0) * 16 + r, turn = SWIGLU ? (q >> 1) & 3 : q & 7;
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                f32x4 v = acc[m][i];
                if constexpr (SWIGLU) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * acc[m][i + 2][c];
                }
                reinterpret_cast<u32x2 *>(mine)[(q * kChunks + ((2 * i + (g >> 1)) ^ turn)) * 2 + (g & 1)] = pack_bf16x4(v);
            }
        }
        wave_lds_fence();
        constexpr int kRowsPerStore = kWave / kChunks;
#pragma unroll
        for (int j = 0; j < 32 / kRowsPerStore; ++j) {
            const int q = j * kRowsPerStore + lane / kChunks, c = lane % kChunks;
            const u32x4 v = mine[q * kChunks + (c ^ (SWIGLU ? (q >> 1) & 3 : q & 7))];
            const int n = n0 + wave * kOutPerWave + c * 8;
            const unsigned int at = n < a.N ? (m0 * 16 + q) * row_bytes + 2u * n : ~0u - 15u;
            __builtin_amdgcn_raw_buffer_store_b128(v, ob, static_cast<int>(at), 0, 0);
        }
        wave_lds_fence();
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kTileWaves * kWave, 2) void k_expert_tile(ExpertGemmArgs a, int tiles_n) {
    __shared__ u32x4 stage0[kStageVecs], stage1[kStageVecs], stage2[kStageVecs];
    __shared__ u32x4 scale[kTileRows + kTileWeights];
    RowTile t;
    if (!find_tile<kTileRows>(a, blockIdx.x, tiles_n, t)) return;   // the same for every wave
    if (t.rows > 64)
        tile_product<8, SWIGLU>(a, t, stage0, stage1, stage2, scale);
    else if (t.rows > 32)
        tile_product<4, SWIGLU>(a, t, stage0, stage1, stage2, scale);
    else
        tile_product<2, SWIGLU>(a, t, stage0, stage1, stage2, scale);
}

// Most row tiles of BM rows that any routing of this shape can have.
int64_t most_tiles(const ExpertGemmArgs &a, int BM) {
    const int64_t used = std::min<int64_t>(a.nseg, a.entries);
    return std::min(a.entries / BM + used, used * ((a.max_count + BM - 1) / BM));
}

// The rule between the two kernels: rows per segment in use, on average.
bool long_segments(const ExpertGemmArgs &a) { return a.entries > 16 * std::min<int64_t>(a.nseg, a.entries); }

struct Grid {
    int tiles_n;
    int64_t blocks;   // a multiple of the XCD count
};
Grid grid_of(const ExpertGemmArgs &a) {
    const bool tiles = long_segments(a);
    const int weights = tiles ? kTileWeights : kWTiles * 16, out = a.swiglu ? weights / 2 : weights;
    Grid g;
    g.tiles_n = (a.N + out - 1) / out;
    g.blocks = (most_tiles(a, tiles ? kTileRows : kStreamRows) * g.tiles_n + kXcds - 1) / kXcds * kXcds;
    return g;
}

}  // namespace

bool expert_gemm_grid_ok(const ExpertGemmArgs &a) { return grid_of(a).blocks <= INT32_MAX; }

hipError_t launch_expert_gemm_mx4(const ExpertGemmArgs &a, hipStream_t s) {
    const Grid g = grid_of(a);
    if (g.blocks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(g.blocks)), stream_block(kStreamWaves * kWave), tile_block(kTileWaves * kWave);
    if (long_segments(a)) {
        if (a.swiglu)
            hipLaunchKernelGGL(k_expert_tile<true>, grid, tile_block, 0, s, a, g.tiles_n);
        else
            hipLaunchKernelGGL(k_expert_tile<false>, grid, tile_block, 0, s, a, g.tiles_n);
    } else if (a.swiglu) {
        hipLaunchKernelGGL(k_expert_stream<true>, grid, stream_block, 0, s, a, g.tiles_n);
    } else {
        hipLaunchKernelGGL(k_expert_stream<false>, grid, stream_block, 0, s, a, g.tiles_n);
    }
    return hipGetLastError();
}

}  // namespace moe
