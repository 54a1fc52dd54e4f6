// The experts' products on MXFP4 rows: launch declaration.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

namespace moe {

// H and N: a tile's rows have to lie within 32-bit offsets of each other.
constexpr int32_t kMaxGemmChannels = 1 << 22;

struct ExpertGemmArgs {
    const uint8_t *x;          // [max_recv,H/2] codes
    const uint8_t *xs;         // [max_recv,H/32] scale bytes
    const uint8_t *w;          // [E,M,H/2]
    const uint8_t *ws;         // [E,M,H/32]
    void *out;                 // [max_recv,N] bf16
    int32_t H, N;
    bool swiglu;               // M = 2N: gate rows, then up rows
    // segments: expert i's rows of a plain layout, or with seg_offset the
    // (rank, segment) pairs of a balanced one
    const int32_t *count;      // [E]
    const int32_t *offset;     // [E+1]
    const int32_t *seg_offset; // [R*(E/R+B)+1] or null
    const int32_t *slot_expert;
    int32_t E, R, B, nseg;
    int64_t entries;           // S*K: at most this many rows are used
    int64_t max_count;         // at most this many in one segment
};

hipError_t launch_expert_gemm_mx4(const ExpertGemmArgs &a, hipStream_t s);
// Whether the grid fits a launch for any routing of this shape.
bool expert_gemm_grid_ok(const ExpertGemmArgs &a);

}  // namespace moe
