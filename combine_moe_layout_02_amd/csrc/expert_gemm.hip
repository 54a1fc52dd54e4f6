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
constexpr int kXcds = 8;       // workgroups go round the XCDs in turn
constexpr int kStep = 128;     // channels of one matrix instruction

// Rows of segment i.
__device__ __forceinline__ int seg_rows(const ExpertGemmArgs &a, int i) {
    return a.seg_offset != nullptr ? a.seg_offset[i + 1] - a.seg_offset[i] : a.count[i];
}

struct RowTile {
    int row0;      // first row of the receive buffer
    int rows;      // rows of the tile that hold an entry
    int expert;
    int ntile;     // which tile of the weights' rows
};

// Finds what workgroup `block` computes.  Tiles are numbered segment by
// segment, inside a segment weight tile by weight tile, inside that row tile
// (BM rows) by row tile, so that workgroups that run together share a weight
// tile.  Workgroups go round the XCDs in turn: each XCD takes one run of the
// tiles, and its L2 serves the neighbours.  Every lane of the wave calls it;
// false for a workgroup without a tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertGemmArgs &a, int block, int tiles_n, RowTile &t) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.nseg + kWave - 1) / kWave;          // <= 24 segments per lane
    int tiles = 0;
    for (int i = lane * per; i < min(a.nseg, (lane + 1) * per); ++i) tiles += (seg_rows(a, i) + BM - 1) / BM;
    int upto = wave_inclusive_scan(tiles);
    const int total = __builtin_amdgcn_readlane(upto, kWave - 1) * tiles_n;
    const int run = (total + kXcds - 1) / kXcds, at_run = block / kXcds;
    const int tile = (block % kXcds) * run + at_run;
    if (at_run >= run || tile >= total) return false;
    const int row_tile = tile / tiles_n;
    const int owner = __builtin_ctzll(__ballot(upto > row_tile));
    const int before = __builtin_amdgcn_readlane(upto - tiles, owner);
    // the owner's segments, one per lane
    const int seg = owner * per + lane;
    const int n = lane < per && seg < a.nseg ? seg_rows(a, seg) : 0;
    tiles = (n + BM - 1) / BM;
    upto = wave_inclusive_scan(tiles);
    const int at = __builtin_ctzll(__ballot(before + upto > row_tile));
    const int seg_tiles = __builtin_amdgcn_readlane(tiles, at);
    const int local = tile - (before + __builtin_amdgcn_readlane(upto - tiles, at)) * tiles_n;
    const int m = local % seg_tiles;
    const int s = owner * per + at;
    t.ntile = local / seg_tiles;
    t.rows = min(BM, __builtin_amdgcn_readlane(n, at) - m * BM);
    if (a.seg_offset != nullptr) {
        const int epr = a.E / a.R, r = s / (epr + a.B), j = s % (epr + a.B);
        t.row0 = a.seg_offset[s] + m * BM;
        t.expert = j < epr ? r * epr + j : a.slot_expert[r * a.B + j - epr];
    } else {
        t.row0 = a.offset[s] + m * BM;
        t.expert = s;
    }
    // the same in every lane: into scalar registers, where the buffer
    // descriptors made from them have to be
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.ntile = __builtin_amdgcn_readfirstlane(t.ntile);
    return true;
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

constexpr int kTileRows = 128;    // token rows of a workgroup
constexpr int kTileWeights = 256; // weight rows of a workgroup: 64 for each wave
constexpr int kTileWaves = 4;
constexpr int kSuper = 4;         // steps whose scales are staged together: one byte of a word each

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

struct TileLds {
    u32x4 tok[2][kTileRows * 4];               // one step of every token row, 16-byte chunks
    u32x4 scale[2][kTileRows + kTileWeights];  // token rows, then weight rows
};

// TT 16-row token tiles of the workgroup's rows.
template <int TT, bool SWIGLU>
__device__ __forceinline__ void tile_product(const ExpertGemmArgs &a, const RowTile &t, TileLds &lds) {
    constexpr int kOutPerWave = SWIGLU ? 32 : 64;
    constexpr int kOutRows = kTileWaves * kOutPerWave;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const unsigned int half = a.H / 2, scales = a.H / kMx4Block;
    const size_t M = SWIGLU ? 2 * static_cast<size_t>(a.N) : a.N;
    const int n0 = t.ntile * kOutRows;
    const int steps = a.H / kStep, supers = (steps + kSuper - 1) / kSuper;
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
    unsigned int wo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wo[i] = weight_row(wave * 64 + i * 16 + r) * half + g * 16;
    // tokens: four lanes carry the 64 bytes of a row's step; chunk c of row q
    // lies at 4q + (c ^ (q/2 % 4)), so that eight rows' chunk c are in eight
    // different groups of banks
    constexpr int kTokLoads = (TT * 64 + 255) / 256;
    unsigned int xo[kTokLoads];
    int xslot[kTokLoads];
#pragma unroll
    for (int i = 0; i < kTokLoads; ++i) {
        const int q = ((i * 256 + tid) & (TT * 64 - 1)) / 4, c = tid & 3;
        xo[i] = q * half + c * 16;
        xslot[i] = 4 * q + (c ^ ((q >> 1) & 3));
    }
    // scales: a thread stages a weight row (with SWIGLU the first two waves the
    // gate rows, the others the up rows) and a token row.  Where there are more
    // threads than rows some stage the same one: branches around the loads
    // would let the compiler move products out of the steps.
    const int wrow = SWIGLU ? (tid & 127) / 32 * 64 + (tid >> 7) * 32 + (tid & 31) : tid;
    const unsigned int wso = weight_row(wrow) * scales, xso = (tid & (TT * 16 - 1)) * scales;
    const auto sb = SWIGLU && wave >= 2 ? s_up : s_gate;

    f32x4 acc[TT][4];
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 w[kSuper][4], x[2][kTokLoads], sw, sx;
    const auto load_w = [&](int k, u32x4 (&to)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = load16(i < 2 ? w_gate : w_up, wo[i], k * (kStep / 2));
    };
    const auto load_x = [&](int k, u32x4 (&to)[kTokLoads]) {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i)
            to[i] = load16(xb, xo[i], k * (kStep / 2));
    };
    const auto store_x = [&](int k, const u32x4 (&from)[kTokLoads]) {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i)
            lds.tok[k & 1][xslot[i]] = from[i];
    };
    // Steps past a row's end read whatever follows it: their scale bytes are 0
    // on both sides, and 2^-254 times any two codes is 0 in fp32.
    const auto load_s = [&](int S) {
        sw = load16(sb, wso, S * 16);
        sx = load16(xsb, xso, S * 16);
    };
    const auto store_s = [&](int S) {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const unsigned int keep = 4 * S + i < steps ? ~0u : 0u;
            sw[i] &= keep;
            sx[i] &= keep;
        }
        lds.scale[S & 1][kTileRows + wrow] = transpose_scales(sw);
        lds.scale[S & 1][tid & (TT * 16 - 1)] = transpose_scales(sx);
    };
    // One superstep; the last one requests nothing past the row's end.
    const auto super = [&](int S, auto is_last) {
        constexpr bool last = decltype(is_last)::value;
        unsigned int sca[4], scb[TT];
#pragma unroll
        for (int s = 0; s < kSuper; ++s) {
            const int k = kSuper * S + s;
            if (!last || s < 2) load_x(k + 2, x[s & 1]);
            if (!last || s < 2) load_w(k + 2, w[(s + 2) & 3]);
            if (s == 0) {
                if (!last) load_s(S + 1);
                const unsigned int *p = reinterpret_cast<const unsigned int *>(lds.scale[S & 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) sca[i] = p[(kTileRows + wave * 64 + i * 16 + r) * 4 + g];
#pragma unroll
                for (int m = 0; m < TT; ++m) scb[m] = p[(m * 16 + r) * 4 + g];
            }
            const u32x4 *tok = lds.tok[s & 1];
#pragma unroll
            for (int m = 0; m < TT; ++m) {
                const u32x4 b = tok[4 * (m * 16 + r) + (g ^ ((r >> 1) & 3))];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const i32x8 av = fp4_operand(w[s][i]), bv = fp4_operand(b);
                    const int sa = static_cast<int>(sca[i]), sx4 = static_cast<int>(scb[m]);
                    // the byte of a step is an immediate
                    acc[m][i] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[m][i], kFp4, kFp4, 0, sa, 0, sx4)
                              : s == 1 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[m][i], kFp4, kFp4, 1, sa, 1, sx4)
                              : s == 2 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[m][i], kFp4, kFp4, 2, sa, 2, sx4)
                                       : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[m][i], kFp4, kFp4, 3, sa, 3, sx4);
                }
            }
            // a step's products stay in their step: the scheduler would keep
            // them, with their operands, for behind the barriers
            __builtin_amdgcn_sched_barrier(0);
            if (!last || s < 3) {
                store_x(k + 1, x[(s + 1) & 1]);
                if (s == 3) store_s(S + 1);
                lds_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    load_s(0);
    load_x(0, x[0]);
    load_w(0, w[0]);
    load_x(1, x[1]);
    load_w(1, w[1]);
    store_s(0);
    store_x(0, x[0]);
    lds_barrier();
    for (int S = 0; S < supers - 1; ++S) super(S, std::false_type{});
    super(supers - 1, std::true_type{});
    // the sums stay where the products left them: without this the compiler
    // moves the last products behind the stores and keeps their operands
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(acc[m][i]));
    // Lane: token r of tile m, four channels from 4g of tile i.  Stores outside
    // the tile's rows fall past the buffer's end, those past N are sent there.
    constexpr int kOut = SWIGLU ? 2 : 4;
    const unsigned int row_bytes = static_cast<unsigned int>(a.N) * 2u;
    const __amdgpu_buffer_rsrc_t ob = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<char *>(a.out) + static_cast<size_t>(t.row0) * row_bytes, 0, static_cast<int>(t.rows * row_bytes),
        kBufferRsrcWord3);
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            f32x4 v = acc[m][i];
            if constexpr (SWIGLU) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * acc[m][i + 2][c];
            }
            const int n = n0 + wave * kOutPerWave + i * 16 + 4 * g;
            const unsigned int at = n < a.N ? (m * 16 + r) * row_bytes + 2u * n : ~0u - 7u;
            __builtin_amdgcn_raw_buffer_store_b64(pack_bf16x4(v), ob, static_cast<int>(at), 0, 0);
        }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kTileWaves * kWave, 2) void k_expert_tile(ExpertGemmArgs a, int tiles_n) {
    __shared__ TileLds lds;
    RowTile t;
    if (!find_tile<kTileRows>(a, blockIdx.x, tiles_n, t)) return;   // the same for every wave
    if (t.rows > 64)
        tile_product<8, SWIGLU>(a, t, lds);
    else if (t.rows > 32)
        tile_product<4, SWIGLU>(a, t, lds);
    else
        tile_product<2, SWIGLU>(a, t, lds);
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
