// 8-bit integer rows (symmetric codes, one fp32 scale per row): launch declarations.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

namespace moe {

constexpr int32_t kMaxInt8Channels = 1 << 22;   // of a row

struct QuantizeI8Args {
    const void *x;          // [rows,H] bf16
    int64_t rows;
    int32_t H;
    const int32_t *src;     // [rows] or null
    void *codes;            // [rows,H] int8
    float *scales;          // [rows]
};

struct DequantizeI8Args {
    const void *codes;
    const float *scales;
    int64_t rows;
    int32_t H;
    const int32_t *src;
    void *out;              // [rows,H] bf16
};

struct DispatchI8Args {
    const void *hidden;     // [S,H] bf16
    int32_t S, H, K;
    const int32_t *pos;     // [S,K]
    const float *topk_w;    // [S,K] or null
    void *recv;             // [max_recv,H] int8
    float *recv_scales;     // [max_recv]
    float *recv_w;          // [max_recv] or null
};

hipError_t launch_quantize_i8(const QuantizeI8Args &a, hipStream_t s);
hipError_t launch_dequantize_i8(const DequantizeI8Args &a, hipStream_t s);
hipError_t launch_dispatch_i8(const DispatchI8Args &a, hipStream_t s);
// Rows that one launch can number.
bool int8_rows_ok(int64_t rows, int32_t H);

}  // namespace moe
