// Gradient of combine: launch declaration.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

namespace moe {

struct CombineBackwardArgs {
    const void *d_out;    // [S,H] bf16
    int32_t S, H, K;
    const int32_t *pos;   // [S,K]
    const void *y;        // [max_recv,H] bf16, with d_w
    const float *w;       // [S,K] or null (weight 1)
    void *d_y;            // [max_recv,H] bf16 or null
    float *d_w;           // [S,K] or null
};

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t s);
bool combine_backward_grid_ok(int32_t S);

}  // namespace moe
