// Router and balance loss: launch declarations.
#pragma once

#include "launch_limit.h"
#include "moe_kernels.h"

namespace moe {

struct RouterArgs {
    const void *logits;        // [S,E]
    bool bf16;                 // the logits' (and d_logits') type: bf16, else fp32
    const uint8_t *mask;       // [S] or null
    int32_t S, E, K, n_groups, topk_groups;
    bool renorm;
    int32_t seq;               // tokens per sequence (> 0)
    int32_t G;                 // sequences
    float alpha;
    bool given;                // the routing is the caller's (given_idx [S,K], with the loss); else the router picks
    const int32_t *given_idx;
    int32_t *idx;              // [S,K]
    float *w;                  // [S,K]
    int32_t *count;            // [G,E], null: no loss
    float *coef;               // [G,E]
    float *loss;               // [1]
    // backward
    const int32_t *picked;     // [S,K] or null
    const float *picked_w;     // [S,K]
    const float *saved_coef;   // [G,E] or null
    const float *d_w;          // [S,K] or null
    const float *d_loss;       // [1] or null
    void *d_logits;            // [S,E]
};

size_t router_workspace_bytes(const RouterArgs &a);
bool router_grid_ok(const RouterArgs &a, bool loss);   // a launch can number that many threads
hipError_t launch_router(const RouterArgs &a, void *workspace, hipStream_t s);
hipError_t launch_router_backward(const RouterArgs &a, hipStream_t s);

}  // namespace moe
