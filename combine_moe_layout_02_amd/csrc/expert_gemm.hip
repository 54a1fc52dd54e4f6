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

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kFp4 = 4;        // operand format code of the scaled matrix instructions: E2M1
constexpr int kRowTile = 16;   // token rows of a tile
constexpr int kStep = 128;     // channels of one matrix instruction

// Rows of segment i.
__device__ __forceinline__ int seg_rows(const ExpertGemmArgs &a, int i) {
    return a.seg_offset != nullptr ? a.seg_offset[i + 1] - a.seg_offset[i] : a.count[i];
}

// Finds row tile `tile` (BM rows, numbered segment by segment): its first row,
// how many of its rows hold an entry, and the expert.  Every lane of the wave
// calls it; false past the last tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertGemmArgs &a, int tile, int &row0, int &rows, int &expert) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.nseg + kWave - 1) / kWave;          // <= 24 segments per lane
    int tiles = 0;
    for (int i = lane * per; i < min(a.nseg, (lane + 1) * per); ++i) tiles += (seg_rows(a, i) + BM - 1) / BM;
    int upto = wave_inclusive_scan(tiles);
    if (tile >= __builtin_amdgcn_readlane(upto, kWave - 1)) return false;
    const int owner = __builtin_ctzll(__ballot(upto > tile));
    int left = tile - __builtin_amdgcn_readlane(upto - tiles, owner);
    // the owner's segments, one per lane
    const int seg = owner * per + lane;
    const int n = lane < per && seg < a.nseg ? seg_rows(a, seg) : 0;
    tiles = (n + BM - 1) / BM;
    upto = wave_inclusive_scan(tiles);
    const int at = __builtin_ctzll(__ballot(upto > left));
    left -= __builtin_amdgcn_readlane(upto - tiles, at);
    const int s = owner * per + at;
    rows = min(BM, __builtin_amdgcn_readlane(n, at) - left * BM);
    if (a.seg_offset != nullptr) {
        const int epr = a.E / a.R, r = s / (epr + a.B), j = s % (epr + a.B);
        row0 = a.seg_offset[s] + left * BM;
        expert = j < epr ? r * epr + j : a.slot_expert[r * a.B + j - epr];
    } else {
        row0 = a.offset[s] + left * BM;
        expert = s;
    }
    return true;
}

__device__ __forceinline__ i32x8 fp4_operand(u32x4 c) {
    return i32x8{static_cast<int>(c[0]), static_cast<int>(c[1]), static_cast<int>(c[2]), static_cast<int>(c[3]), 0, 0, 0, 0};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ u32x2 pack_bf16x4(f32x4 v) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

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
    int row0, rows, expert;
    if (!find_tile<kRowTile>(a, blockIdx.x / tiles_n, row0, rows, expert)) return;   // the same for every wave
    const int n0 = (blockIdx.x % tiles_n) * (kOutTiles * 16);
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

// Most row tiles of BM rows that any routing of this shape can have.
int64_t most_tiles(const ExpertGemmArgs &a, int BM) {
    const int64_t used = std::min<int64_t>(a.nseg, a.entries);
    return std::min(a.entries / BM + used, used * ((a.max_count + BM - 1) / BM));
}

int out_tile(const ExpertGemmArgs &a) { return (a.swiglu ? kWTiles / 2 : kWTiles) * 16; }

int64_t grid_of(const ExpertGemmArgs &a) {
    return most_tiles(a, kRowTile) * ((a.N + out_tile(a) - 1) / out_tile(a));
}

}  // namespace

bool expert_gemm_grid_ok(const ExpertGemmArgs &a) { return grid_of(a) <= INT32_MAX; }

hipError_t launch_expert_gemm_mx4(const ExpertGemmArgs &a, hipStream_t s) {
    const int64_t grid = grid_of(a);
    if (grid == 0) return hipSuccess;
    const int tiles_n = (a.N + out_tile(a) - 1) / out_tile(a);
    const dim3 block(kStreamWaves * kWave);
    if (a.swiglu)
        hipLaunchKernelGGL(k_expert_stream<true>, dim3(static_cast<unsigned>(grid)), block, 0, s, a, tiles_n);
    else
        hipLaunchKernelGGL(k_expert_stream<false>, dim3(static_cast<unsigned>(grid)), block, 0, s, a, tiles_n);
    return hipGetLastError();
}

}  // namespace moe
