// Gradient of combine: of out[t] = sum over k of w[t,k] * y[pos[t,k]] (+ shared),
//   d_y[pos[t,k]] = bf16(w[t,k] * d_out[t]),
//   d_w[t,k] = sum over channels of d_out[t,c] * y[pos[t,k],c], 0 where pos is -1
// (d_shared is d_out itself).  Every row of y is read once, every row of d_y written
// once, d_out read once or (in_two) twice: HBM bounds it, 4096 tokens of 7168 with
// eight rows each 171 us, 6.2 TB/s.
//
// One workgroup per token; a wave takes every W-th chunk of 512 channels, 16
// bytes per lane, with all K gathers in flight before the first product, as in
// the forward.  A lane keeps K sums in fp32 over its chunks; they are joined over
// the lanes and then, in LDS, over the waves, in an order that does not depend
// on how the work runs.
#include "combine_backward.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 8;

__device__ __forceinline__ unsigned int bf16_pair(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned int, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

template <int K, bool ROWS, bool WEIGHTS>
__global__ __launch_bounds__(kMaxWaves * kWave) void k_combine_backward(CombineBackwardArgs a) {
    __shared__ float part[kMaxWaves][K];
    const int t = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    const int nvec = a.H / 8;
    // d_y may be y itself: a lane reads its channels of a row before it writes them
    const u32x4 *const d_out = static_cast<const u32x4 *>(a.d_out) + static_cast<size_t>(t) * nvec;
    const u32x4 *const y = static_cast<const u32x4 *>(a.y);
    u32x4 *const d_y = static_cast<u32x4 *>(a.d_y);
    int p[K];
    float w[K], sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        p[k] = a.pos[static_cast<size_t>(t) * K + k];
        w[k] = ROWS && a.w != nullptr ? a.w[static_cast<size_t>(t) * K + k] : 1.0f;
        sum[k] = 0.0f;
    }
    for (int v = wave * kWave + lane; v < nvec; v += waves * kWave) {
        const u32x4 d = d_out[v];
        u32x4 r[K];
        if constexpr (WEIGHTS) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                r[k] = u32x4{0u, 0u, 0u, 0u};
                if (p[k] >= 0) r[k] = __builtin_nontemporal_load(y + static_cast<size_t>(p[k]) * nvec + v);
            }
        }
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(d[i]);
            f[2 * i + 1] = bf16_hi(d[i]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (p[k] < 0) continue;                               // the same for the whole workgroup
            if constexpr (WEIGHTS) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[k] = __builtin_fmaf(f[2 * i], bf16_lo(r[k][i]), sum[k]);
                    sum[k] = __builtin_fmaf(f[2 * i + 1], bf16_hi(r[k][i]), sum[k]);
                }
            }
            if constexpr (ROWS) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = bf16_pair(w[k] * f[2 * i], w[k] * f[2 * i + 1]);
                __builtin_nontemporal_store(o, d_y + static_cast<size_t>(p[k]) * nvec + v);
            }
        }
    }
    if constexpr (WEIGHTS) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int s = kWave / 2; s > 0; s /= 2) sum[k] += __shfl_xor(sum[k], s);
            if (lane == 0) part[wave][k] = sum[k];
        }
        __syncthreads();
        if (threadIdx.x < K) {
            float v = 0.0f;
            for (int i = 0; i < waves; ++i) v += part[i][threadIdx.x];
            a.d_w[static_cast<size_t>(t) * K + threadIdx.x] = v;
        }
    }
}

// Rows of y and d_y that the caches do not keep are read in one launch and written
// in another: the memory turns from the one to the other less often, and d_out, the
// smaller part, is read twice.  One launch / two (us; S tokens, H channels, K rows
// each): S=256 H=7168 K=8, 29 MB, 13.9 / 15.5; S=1024 H=2048 K=6, 25 MB, 12.4 / 14.8;
// S=512 H=7168 K=8, 59 MB, 28.1 / 25.9; S=4096, 470 MB, 189 / 171; S=16384 H=2048
// K=6, 403 MB, 155 / 149.
bool in_two(const CombineBackwardArgs &a) { return 2.0 * a.S * a.K * a.H > 40.0e6; }

template <int K>
void launch(const CombineBackwardArgs &a, dim3 grid, dim3 block, hipStream_t s) {
    if (a.d_y != nullptr && a.d_w != nullptr && in_two(a)) {
        // d_y may be y: what reads it goes first
        CombineBackwardArgs weights = a, rows = a;
        weights.d_y = nullptr;
        rows.d_w = nullptr;
        launch<K>(weights, grid, block, s);
        launch<K>(rows, grid, block, s);
        return;
    }
    if (a.d_y == nullptr)
        hipLaunchKernelGGL((k_combine_backward<K, false, true>), grid, block, 0, s, a);
    else if (a.d_w == nullptr)
        hipLaunchKernelGGL((k_combine_backward<K, true, false>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_combine_backward<K, true, true>), grid, block, 0, s, a);
}

}  // namespace

bool combine_backward_grid_ok(int32_t S) { return S <= kMaxLaunchThreads / (kMaxWaves * kWave); }

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t s) {
    const int nchunk = (a.H / 8 + kWave - 1) / kWave;
    const dim3 grid(static_cast<unsigned>(a.S)), block(static_cast<unsigned>((nchunk < kMaxWaves ? nchunk : kMaxWaves) * kWave));
#define MOE_CASE(N) \
    case N: launch<N>(a, grid, block, s); break;
    switch (a.K) {
        MOE_CASE(1) MOE_CASE(2) MOE_CASE(3) MOE_CASE(4) MOE_CASE(5) MOE_CASE(6) MOE_CASE(7) MOE_CASE(8)
        MOE_CASE(9) MOE_CASE(10) MOE_CASE(11) MOE_CASE(12) MOE_CASE(13) MOE_CASE(14) MOE_CASE(15) MOE_CASE(16)
        default: return hipErrorInvalidValue;
    }
#undef MOE_CASE
    return hipGetLastError();
}

}  // namespace moe
