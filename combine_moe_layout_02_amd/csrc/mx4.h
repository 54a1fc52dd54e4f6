// MXFP4 rows (E2M1 codes, one E8M0 scale byte per 32 channels): launch
// declarations and the conversion of one lane's channels.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

namespace moe {

constexpr int kMx4Block = 32;             // channels per scale
constexpr int kMx4WaveChannels = 32 * kWave;  // channels a wave converts at a time: one block per lane

struct Mx4Args {
    const void *in;       // bf16 rows (quantise) or codes (dequantise)
    const uint8_t *in_scales;
    int64_t rows;
    int32_t H;
    const int32_t *src;   // [rows] or null
    void *out;            // codes or bf16 rows
    uint8_t *out_scales;
};

struct DispatchMx4Args {
    const void *hidden;   // [S,H] bf16
    int32_t S, H, K;
    const int32_t *pos;   // [S,K]
    const float *topk_w;  // [S,K] or null
    void *recv;           // [max_recv,H/2]
    uint8_t *recv_scales; // [max_recv,H/32]
    float *recv_w;        // [max_recv] or null
};

hipError_t launch_quantize_mx4(const Mx4Args &a, hipStream_t s);
hipError_t launch_dequantize_mx4(const Mx4Args &a, hipStream_t s);
hipError_t launch_dispatch_mx4(const DispatchMx4Args &a, hipStream_t s);

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Larger of the two bf16 magnitudes in each half of a word, as bits: without
// the sign bit, bf16 values order as integers, NaN above infinity above all.
__device__ __forceinline__ unsigned int mx4_absmax(u32x4 x) {
    unsigned int m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned int lo = x[i] & 0x7FFFu, hi = (x[i] >> 16) & 0x7FFFu;
        m = max(m, max(lo, hi));
    }
    return m;
}

// Scale byte of a block from its largest magnitude's bits: the exponent field
// less 2 (E2M1's largest exponent), not below 0, which is 2^-127; 255 for a
// block with a NaN or an infinity.  A subnormal bf16 has field 0 and every
// block below 2^-124 takes byte 0.
__device__ __forceinline__ unsigned int mx4_scale_byte(unsigned int absmax) {
    const unsigned int e = absmax >> 7;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// E2M1 codes of 8 consecutive bf16 channels (one 16-byte vector), the first in
// the lowest four bits.  The conversion instruction divides by the scale (the
// float's exponent alone counts), rounds to nearest even and saturates at 6.
__device__ __forceinline__ unsigned int mx4_encode8(u32x4 x, unsigned int scale_byte) {
    // byte 0 is 2^-127, a subnormal float
    const float scale = __uint_as_float(scale_byte == 0u ? 0x00400000u : scale_byte << 23);
    // words of their own: a bit cast of a vector's element reads element 0
    const unsigned int w0 = x[0], w1 = x[1], w2 = x[2], w3 = x[3];
    unsigned int c = 0u;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w0), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w1), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w2), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w3), scale, 3);
    return scale_byte == 255u ? 0u : c;
}

}  // namespace moe
