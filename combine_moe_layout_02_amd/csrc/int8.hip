// 8-bit integer rows: quantise, dequantise, and the dispatch that quantises on
// the way.
//
// Per row, scale = amax/127 and code = round(x / scale), ties to even, both
// divisions correctly rounded in fp32, so |code| <= 127 and a row's largest
// channel has code +-127.  A row with a NaN or an infinity gets scale NaN and
// codes 0: what is multiplied with it is NaN.  One workgroup per row: the row
// is read once and stays in registers (up to kHeld groups of 16 channels per
// lane; longer rows are read a second time), its largest magnitude is joined
// over the wave by lane swaps and over the waves in LDS.
//
// HBM bounds them: 98304 rows of 1408 81 us (5.1 TB/s), 32768 of 7168 117 us (6.0) and
// back 125 us (5.6; 98 where the same call before left its codes in the Infinity Cache),
// the dispatch of 4096 tokens of 7168 to eight rows each 51 us (5.8).  Of a layout's
// 32768 rows with 1024 in use 14 us, back 10, most of it workgroups that find nothing to
// do; two to eight rows a workgroup took 17 to 30, back 9 to 12 (and 99 to 102, not 98,
// with every row in use), and a wave for each row of a plain array was slower.
#include "int8.h"
#include "mx4.h"   // mx4_absmax

namespace moe {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kHeld = 2;        // groups of 16 channels a lane keeps
constexpr int kMaxWaves = 8;

// Largest of the wave's values, in every lane.
__device__ __forceinline__ unsigned int wave_max(unsigned int m) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) m = max(m, static_cast<unsigned int>(__shfl_xor(static_cast<int>(m), d)));
    return m;
}

// Codes of 16 channels.  The definition's quotient x / scale is a division, about
// ten instructions, and would bound the conversion (98304 rows of 1408: 106 us, not 81).
// With inv = 1/scale, fma(x, inv, 1.5 * 2^23) is x * inv rounded to an integer, ties
// to even, in the sum's low bits.  x * inv is within 2^-24 of itself of the exact
// quotient and the rounded quotient within as much, below 127 * 2^-23 together: where
// x * inv is further than 2^-14 from the middle of two integers both round alike.
// The others, one in 8000, are divided.  `exact`: a scale whose inverse is not to
// be had so well, below 2^-100, divides too.
__device__ __forceinline__ u32x4 codes16(u32x4 lo, u32x4 hi, float scale, float inv, bool exact) {
    constexpr float kShift = 12582912.0f;
    float f[16], t[16], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(lo[i]);
        f[2 * i + 1] = bf16_hi(lo[i]);
        f[8 + 2 * i] = bf16_lo(hi[i]);
        f[9 + 2 * i] = bf16_hi(hi[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        t[i] = __builtin_fmaf(f[i], inv, kShift);
        far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(f[i], inv, kShift - t[i])));
    }
    if (exact || far > 0.5f - 0x1p-14f) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            // a scale below fp32's normal range is rounded: its quotient may pass 127
            t[i] = fminf(fmaxf(__builtin_rintf(f[i] / scale), -127.0f), 127.0f) + kShift;
    }
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned int a = __float_as_uint(t[4 * i]), b = __float_as_uint(t[4 * i + 1]), d = __float_as_uint(t[4 * i + 2]), e = __float_as_uint(t[4 * i + 3]);
        c[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(e, d, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
    }
    return c;
}

// The largest of the workgroup's waves' values.
__device__ __forceinline__ unsigned int join_waves(unsigned int m) {
    __shared__ unsigned int part[kMaxWaves];
    const int waves = blockDim.x / kWave;
    if (waves == 1) return m;
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = m;
    __syncthreads();
    for (int w = 0; w < waves; ++w) m = max(m, part[w]);
    return m;
}

// Quantises one row of H channels with the whole workgroup; store(g, codes) for
// each group g of 16 channels that the lane owns.  Returns the row's scale.  ONCE:
// the row is read past the caches.
template <bool ONCE, typename Store>
__device__ __forceinline__ float quantize_row(const u32x4 *__restrict__ x, int H, Store &&store) {
    const int n16 = H / 16, threads = blockDim.x, tid = threadIdx.x;
    u32x4 lo[kHeld], hi[kHeld];
    unsigned int m = 0u;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int g = j * threads + tid;
        lo[j] = hi[j] = u32x4{0u, 0u, 0u, 0u};
        if (g < n16) {
            lo[j] = ONCE ? __builtin_nontemporal_load(x + 2 * g) : x[2 * g];
            hi[j] = ONCE ? __builtin_nontemporal_load(x + 2 * g + 1) : x[2 * g + 1];
        }
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) m = max(m, max(mx4_absmax(lo[j]), mx4_absmax(hi[j])));
    for (int g = kHeld * threads + tid; g < n16; g += threads) m = max(m, max(mx4_absmax(x[2 * g]), mx4_absmax(x[2 * g + 1])));
    m = join_waves(wave_max(m));
    const bool broken = m >= 0x7F80u;
    const float scale = broken ? __uint_as_float(0x7FC00000u) : __uint_as_float(m << 16) / 127.0f;
    const float inv = 1.0f / scale;
    const bool none = broken || m == 0u, exact = !(scale >= 0x1p-100f);
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int g = j * threads + tid;
        if (g < n16) store(g, none ? zero : codes16(lo[j], hi[j], scale, inv, exact));
    }
    for (int g = kHeld * threads + tid; g < n16; g += threads) store(g, none ? zero : codes16(x[2 * g], x[2 * g + 1], scale, inv, exact));
    return scale;
}

// Row of a workgroup: each XCD takes consecutive rows, since with a layout the
// rows in use often begin a power of two apart.
__device__ __forceinline__ int64_t row_of_block() {
    constexpr int kXcds = 8;
    return static_cast<int64_t>(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
}

__global__ __launch_bounds__(kMaxWaves * kWave) void k_quantize_i8(QuantizeI8Args a) {
    const int64_t row = row_of_block();
    if (row >= a.rows || (a.src != nullptr && a.src[row] < 0)) return;
    u32x4 *__restrict__ codes = static_cast<u32x4 *>(a.codes) + row * (a.H / 16);
    const float scale = quantize_row<true>(static_cast<const u32x4 *>(a.x) + row * (a.H / 8), a.H, [&](int g, u32x4 c) { codes[g] = c; });
    if (threadIdx.x == 0) a.scales[row] = scale;
}

__device__ __forceinline__ unsigned int bf16_pair(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned int, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__global__ __launch_bounds__(kMaxWaves * kWave) void k_dequantize_i8(DequantizeI8Args a) {
    const int64_t row = row_of_block();
    if (row >= a.rows || (a.src != nullptr && a.src[row] < 0)) return;
    const int n8 = a.H / 8;
    const u32x2 *__restrict__ codes = static_cast<const u32x2 *>(a.codes) + row * n8;
    u32x4 *__restrict__ out = static_cast<u32x4 *>(a.out) + row * n8;
    const float scale = a.scales[row];
    for (int v = threadIdx.x; v < n8; v += blockDim.x) {
        const u32x2 c = codes[v];
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = static_cast<int>(c[i / 2] << (i & 1 ? 0 : 16));   // the pair in the upper half
            o[i] = bf16_pair(static_cast<float>(w << 8 >> 24) * scale, static_cast<float>(w >> 24) * scale);
        }
        __builtin_nontemporal_store(o, out + v);
    }
}

template <int K>
__global__ __launch_bounds__(kMaxWaves * kWave) void k_dispatch_i8(DispatchI8Args a) {
    const int t = blockIdx.x;
    const int n16 = a.H / 16;
    int p[K];
#pragma unroll
    for (int k = 0; k < K; ++k) p[k] = a.pos[static_cast<size_t>(t) * K + k];
    u32x4 *__restrict__ recv = static_cast<u32x4 *>(a.recv);
    const float scale = quantize_row<false>(static_cast<const u32x4 *>(a.hidden) + static_cast<size_t>(t) * (a.H / 8), a.H, [&](int g, u32x4 c) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (p[k] >= 0) __builtin_nontemporal_store(c, recv + static_cast<size_t>(p[k]) * n16 + g);
    });
    if (threadIdx.x < K) {
        int row = -1;
#pragma unroll
        for (int k = 0; k < K; ++k) row = static_cast<int>(threadIdx.x) == k ? p[k] : row;
        if (row >= 0) {
            a.recv_scales[row] = scale;
            if (a.recv_w != nullptr && a.topk_w != nullptr) a.recv_w[row] = a.topk_w[static_cast<size_t>(t) * K + threadIdx.x];
        }
    }
}

// Waves of a row's workgroup: as few as keep the row in registers.
int row_waves(int32_t H) {
    const int n = (H / 16 + kHeld * kWave - 1) / (kHeld * kWave);
    return n < kMaxWaves ? n : kMaxWaves;
}

dim3 row_grid(int64_t rows) { return dim3(static_cast<unsigned int>((rows + 7) / 8 * 8)); }

}  // namespace

bool int8_rows_ok(int64_t rows, int32_t H) {
    return H >= 16 && H % 16 == 0 && H <= kMaxInt8Channels && rows >= 0 && rows <= kMaxLaunchThreads / (kMaxWaves * kWave) / 8 * 8;
}

hipError_t launch_quantize_i8(const QuantizeI8Args &a, hipStream_t s) {
    hipLaunchKernelGGL(k_quantize_i8, row_grid(a.rows), dim3(row_waves(a.H) * kWave), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dequantize_i8(const DequantizeI8Args &a, hipStream_t s) {
    hipLaunchKernelGGL(k_dequantize_i8, row_grid(a.rows), dim3(row_waves(a.H) * kWave), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dispatch_i8(const DispatchI8Args &a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned int>(a.S)), block(row_waves(a.H) * kWave);
#define MOE_I8_CASE(N) \
    case N: hipLaunchKernelGGL(k_dispatch_i8<N>, grid, block, 0, s, a); break;
    switch (a.K) {
        MOE_I8_CASE(1) MOE_I8_CASE(2) MOE_I8_CASE(3) MOE_I8_CASE(4) MOE_I8_CASE(5) MOE_I8_CASE(6)
        MOE_I8_CASE(7) MOE_I8_CASE(8) MOE_I8_CASE(9) MOE_I8_CASE(10) MOE_I8_CASE(11) MOE_I8_CASE(12)
        MOE_I8_CASE(13) MOE_I8_CASE(14) MOE_I8_CASE(15) MOE_I8_CASE(16)
        default: return hipErrorInvalidValue;
    }
#undef MOE_I8_CASE
    return hipGetLastError();
}

}  // namespace moe
