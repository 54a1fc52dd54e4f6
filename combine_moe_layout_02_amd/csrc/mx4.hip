// MXFP4 rows: quantise, dequantise, and the dispatch that quantises on the way.
//
// Per 32 channels, scale = 2^(floor(log2(amax)) - 2) and code = E2M1(x / scale)
// (to nearest, ties to the even code, saturating at 6).  Nothing is summed: a
// row is read once and 17/64 of its bytes are written (once, or K times by the
// dispatch), so HBM bounds all three; at decode sizes it is the launch.
//
// A wave converts 2048 channels at a time in four steps of 16 bytes per lane,
// so that every load instruction reads 1 KiB in one run; the four lanes that
// share a block take the largest magnitude with two cross-lane swaps.  The
// codes, one word per lane and step, then pass through LDS (written and read
// by the same wave: no barrier) so that lane l owns the whole of block l and
// stores its 16 bytes of codes in one instruction, 1 KiB per wave.
//
// The wide side, bf16 rows, is read and written past the caches
// (non-temporal), the codes, a quarter as many and read again by the next
// product, are not.  65536 rows of 7168: quantise 203 us (5.9 TB/s) and
// dequantise 197 us (6.0), back to back 345 us, against 208, 209 and 429 us with
// ordinary accesses; codes stored non-temporally too 191, 197 and 388 us; 2048
// rows 7.5 and 6.8 against 7.7 and 7.9 us.  The dispatch reads rows K copies
// long: ordinary loads, non-temporal stores of codes (32.5 us at 4096 x 7168, K
// = 8, 5.7 TB/s; 38.8 with non-temporal loads, 40.5 with ordinary stores).
#include "mx4.h"

namespace moe {
namespace {

constexpr int kMx4Waves = 4;
constexpr int kXcds = 8;   // workgroups go round the XCDs in turn
constexpr int kSteps = 4;  // 16-byte vectors per lane and conversion

struct Mx4Stage {
    unsigned int code[kSteps * kWave];
    uint8_t scale[kWave];
};

// Orders the wave's own LDS accesses.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A value of another lane of the same four (DPP quad_perm).
template <int CTRL>
__device__ __forceinline__ unsigned int quad_swap(unsigned int v) {
    return static_cast<unsigned int>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// Which of the wave's vectors j*64 + lane from v0 to convert: those inside the
// array whose row holds an entry (src null: every row).
__device__ __forceinline__ void mx4_rows_in_use(const Mx4Args &a, int64_t v0, int64_t nvec, bool (&use)[kSteps]) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) use[j] = v0 + j * kWave + lane < nvec;
    if (a.src == nullptr) return;
    const int vec_per_row = a.H / 8;
    const int64_t row0 = v0 / vec_per_row;                            // the wave's first row
    const int rem0 = static_cast<int>(v0 - row0 * vec_per_row);
    int s[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) s[j] = use[j] ? a.src[row0 + (rem0 + j * kWave + lane) / vec_per_row] : -1;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) use[j] = s[j] >= 0;
}

// Converts the wave's vectors x[j] = vector j*64 + lane of 2048 consecutive
// channels; on return lane l has block l's 16 bytes of codes and its scale
// byte.  Every lane of the wave calls it.
__device__ __forceinline__ u32x4 mx4_wave_quantize(const u32x4 (&x)[kSteps], Mx4Stage &st, unsigned int &scale_byte) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        unsigned int m = mx4_absmax(x[j]);
        m = max(m, quad_swap<0xB1>(m));   // lanes 1, 0, 3, 2
        m = max(m, quad_swap<0x4E>(m));   // lanes 2, 3, 0, 1
        const unsigned int sb = mx4_scale_byte(m);
        st.code[j * kWave + lane] = mx4_encode8(x[j], sb);
        if ((lane & 3) == 0) st.scale[j * (kWave / 4) + lane / 4] = static_cast<uint8_t>(sb);
    }
    wave_lds_order();   // nothing else uses this stage
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = st.code[4 * lane + i];
    scale_byte = st.scale[lane];
    return c;
}

// Quantises vectors j*64 + lane of the 2048 channels from vector v0 of the
// array; use[j]: this lane's is to be converted.
__device__ __forceinline__ void quantize_2048(const Mx4Args &a, int64_t v0, const bool (&use)[kSteps], Mx4Stage &stage) {
    const int lane = threadIdx.x & (kWave - 1);
    const u32x4 *__restrict__ in = static_cast<const u32x4 *>(a.in) + v0;
    u32x4 x[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        x[j] = u32x4{0u, 0u, 0u, 0u};
        if (use[j]) x[j] = __builtin_nontemporal_load(in + j * kWave + lane);
    }
    // block l = vectors 4l .. 4l+3, all of one row: step l/16, lanes 4*(l%16) .. +3
    uint64_t ballot[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) ballot[j] = __ballot(use[j]);
    unsigned int sb;
    const u32x4 c = mx4_wave_quantize(x, stage, sb);
    const int j = lane / (kWave / 4);
    const uint64_t mine = j == 0 ? ballot[0] : (j == 1 ? ballot[1] : (j == 2 ? ballot[2] : ballot[3]));
    if ((mine >> (4 * (lane % (kWave / 4)))) & 1u) {
        static_cast<u32x4 *>(a.out)[v0 / 4 + lane] = c;
        a.out_scales[v0 / 4 + lane] = static_cast<uint8_t>(sb);
    }
}

// Dequantises the same vectors.  A lane expands one word of codes (8 channels,
// 16 bytes of bf16) per step, so the stores, four fifths of the bytes, are 1 KiB
// runs.
__device__ __forceinline__ void dequantize_2048(const Mx4Args &a, int64_t v0, const bool (&use)[kSteps]) {
    const int lane = threadIdx.x & (kWave - 1);
    const unsigned int *__restrict__ in = static_cast<const unsigned int *>(a.in) + v0;
    const uint8_t *__restrict__ sc = a.in_scales + v0 / 4;
    u32x4 *__restrict__ out = static_cast<u32x4 *>(a.out) + v0;
    unsigned int c[kSteps], sb[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const int v = j * kWave + lane;
        c[j] = use[j] ? in[v] : 0u;
        sb[j] = use[j] ? sc[v / 4] : 0u;
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const float scale = __uint_as_float(sb[j] == 0u ? 0x00400000u : sb[j] << 23);
        u32x4 o;
        o[0] = __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], scale, 0));
        o[1] = __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], scale, 1));
        o[2] = __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], scale, 2));
        o[3] = __builtin_bit_cast(unsigned int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], scale, 3));
        if (sb[j] == 255u) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        if (use[j]) __builtin_nontemporal_store(o, out + j * kWave + lane);
    }
}

// Rows lie end to end, so a wave takes 2048 consecutive channels of the whole
// array, whatever rows they belong to; with src, a lane's row is looked up.
template <bool QUANTIZE>
__global__ __launch_bounds__(kMx4Waves * kWave) void k_convert_mx4(Mx4Args a) {
    __shared__ __align__(16) Mx4Stage stage[QUANTIZE ? kMx4Waves : 1];
    const int wave = threadIdx.x / kWave;
    const int64_t nvec = a.rows * (a.H / 8);                          // 16-byte vectors
    const int64_t v0 = (static_cast<int64_t>(blockIdx.x) * kMx4Waves + wave) * (kSteps * kWave);
    if (v0 >= nvec) return;
    bool use[kSteps];
    mx4_rows_in_use(a, v0, nvec, use);
    if constexpr (QUANTIZE)
        quantize_2048(a, v0, use, stage[wave]);
    else
        dequantize_2048(a, v0, use);
}

// The same with a layout and rows of at least one wave's 2048 channels: a
// workgroup per row, its waves taking the row's chunks in turn, one lookup for
// the workgroup.  The rows in use begin each expert's segment, often a power of
// two apart, so that consecutive workgroups (which go to the XCDs in turn) would
// leave all of them to one or two XCDs: each XCD takes consecutive rows instead.
// 32768 rows of 7168, four of each 128 in use: quantise 62.5 -> 9.6 us, dequantise
// 32.0 -> 10.6 us (17.0 and 13.7 in the order of the rows); 40960 rows, 128 of
// each 160 in use: 109.6 -> 92.8 and 84.5 -> 82.0 us, at H = 2048 34.6 -> 28.8 and
// 26.5 -> 25.5 us.  Below that, waves would idle: at H = 1024 24.2 against 19.7
// and 19.4 against 12.6 us with the lookup per lane.
template <bool QUANTIZE>
__global__ __launch_bounds__(kMx4Waves * kWave) void k_convert_rows_mx4(Mx4Args a) {
    __shared__ __align__(16) Mx4Stage stage[QUANTIZE ? kMx4Waves : 1];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t row = static_cast<int64_t>(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    if (row >= a.rows || a.src[row] < 0) return;
    const int vec_per_row = a.H / 8;
    for (int c = wave * (kSteps * kWave); c < vec_per_row; c += kMx4Waves * (kSteps * kWave)) {
        bool use[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) use[j] = c + j * kWave + lane < vec_per_row;
        if constexpr (QUANTIZE) {
            quantize_2048(a, row * vec_per_row + c, use, stage[wave]);
            wave_lds_order();                                         // the stage is read before it is filled again
        } else {
            dequantize_2048(a, row * vec_per_row + c, use);
        }
    }
}

// One wave per (token, 2048-channel chunk), chunk-fastest as in the other
// dispatch kernels; the token's row indices are wave-uniform and read before
// the first store.
template <int K>
__global__ __launch_bounds__(kWave) void k_dispatch_mx4(DispatchMx4Args a, int nchunk) {
    __shared__ __align__(16) Mx4Stage stage;
    const int t = blockIdx.x / nchunk, c = blockIdx.x % nchunk, lane = threadIdx.x;
    const int nvec = a.H / 8, nblk = a.H / kMx4Block;
    const u32x4 *__restrict__ hid = static_cast<const u32x4 *>(a.hidden) + static_cast<size_t>(t) * nvec;
    const bool maps = a.recv_w != nullptr && a.topk_w != nullptr && c == 0 && lane < K;
    u32x4 x[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const int v = c * (kSteps * kWave) + j * kWave + lane;
        x[j] = u32x4{0u, 0u, 0u, 0u};
        if (v < nvec) x[j] = hid[v];
    }
    int p[K];
#pragma unroll
    for (int k = 0; k < K; ++k) p[k] = a.pos[static_cast<size_t>(t) * K + k];
    const float w = maps ? a.topk_w[static_cast<size_t>(t) * K + lane] : 0.0f;
    unsigned int sb;
    const u32x4 codes = mx4_wave_quantize(x, stage, sb);
    const int b = c * kWave + lane;
    if (b < nblk) {
        u32x4 *__restrict__ recv = static_cast<u32x4 *>(a.recv);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (p[k] >= 0) {
                __builtin_nontemporal_store(codes, recv + static_cast<size_t>(p[k]) * nblk + b);
                a.recv_scales[static_cast<size_t>(p[k]) * nblk + b] = static_cast<uint8_t>(sb);
            }
        }
    }
    if (maps) {
        int row = -1;
#pragma unroll
        for (int k = 0; k < K; ++k) row = lane == k ? p[k] : row;
        if (row >= 0) a.recv_w[row] = w;
    }
}

template <bool QUANTIZE>
hipError_t launch_convert(const Mx4Args &a, hipStream_t s) {
    constexpr int64_t kMaxRowBlocks = kMaxLaunchThreads / (kMx4Waves * kWave) / kXcds * kXcds;
    if (a.src != nullptr && a.H >= kMx4WaveChannels && a.rows <= kMaxRowBlocks) {
        const dim3 grid(static_cast<unsigned int>((a.rows + kXcds - 1) / kXcds * kXcds));
        hipLaunchKernelGGL(k_convert_rows_mx4<QUANTIZE>, grid, dim3(kMx4Waves * kWave), 0, s, a);
    } else {
        const int64_t per = int64_t(kMx4WaveChannels) * kMx4Waves;
        hipLaunchKernelGGL(k_convert_mx4<QUANTIZE>, dim3(static_cast<unsigned int>((a.rows * a.H + per - 1) / per)), dim3(kMx4Waves * kWave), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mx4(const Mx4Args &a, hipStream_t s) { return launch_convert<true>(a, s); }

hipError_t launch_dequantize_mx4(const Mx4Args &a, hipStream_t s) { return launch_convert<false>(a, s); }

hipError_t launch_dispatch_mx4(const DispatchMx4Args &a, hipStream_t s) {
    const int nchunk = (a.H + kMx4WaveChannels - 1) / kMx4WaveChannels;
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.S) * nchunk)), block(kWave);
#define MOE_MX4_CASE(N) \
    case N: hipLaunchKernelGGL(k_dispatch_mx4<N>, grid, block, 0, s, a, nchunk); break;
    switch (a.K) {
        MOE_MX4_CASE(1) MOE_MX4_CASE(2) MOE_MX4_CASE(3) MOE_MX4_CASE(4) MOE_MX4_CASE(5) MOE_MX4_CASE(6)
        MOE_MX4_CASE(7) MOE_MX4_CASE(8) MOE_MX4_CASE(9) MOE_MX4_CASE(10) MOE_MX4_CASE(11) MOE_MX4_CASE(12)
        MOE_MX4_CASE(13) MOE_MX4_CASE(14) MOE_MX4_CASE(15) MOE_MX4_CASE(16)
        default: return hipErrorInvalidValue;
    }
#undef MOE_MX4_CASE
    return hipGetLastError();
}

}  // namespace moe
