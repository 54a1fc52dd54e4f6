// The experts' products on MXFP4 rows: launch declaration.
#pragma once

#include "expert_tiles.h"

namespace moe {

struct ExpertGemmArgs : Segments {
    const uint8_t *x;          // [max_recv,H/2] codes
    const uint8_t *xs;         // [max_recv,H/32] scale bytes
    const uint8_t *w;          // [E,M,H/2]
    const uint8_t *ws;         // [E,M,H/32]
    void *out;                 // [max_recv,N] bf16
    int32_t H, N;
    bool swiglu;               // M = 2N: gate rows, then up rows
};

hipError_t launch_expert_gemm_mx4(const ExpertGemmArgs &a, hipStream_t s);
// Whether the grid fits a launch for any routing of this shape.
bool expert_gemm_grid_ok(const ExpertGemmArgs &a);

}  // namespace moe
