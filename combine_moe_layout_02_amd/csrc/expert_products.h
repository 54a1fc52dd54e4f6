// The experts' products on bf16 and 8-bit integer rows, and their gradients:
// launch declaration.
#pragma once

#include "expert_tiles.h"

namespace moe {

// Channels of an 8-bit product: a sum of that many products of codes, -128
// included, stays in 32 bits.
constexpr int32_t kMaxInt8Inner = ((1 << 17) - 1) / 16 * 16;

enum class Product {
    kForward,      // out[r][c] = sum over h of x[r][h] * w[e][c][h]
    kForwardI8,    // the same in 8-bit integers, times the row's and the channel's scale
    kBackwardX,    // out[r][c] = sum over n of x[r][n] * w[e][n][c]   (x: d_out)
    kBackwardW,    // out[e][n][c] = sum over e's rows r of x[r][n] * w[r][c]   (x: d_out, w: the rows)
};

struct ProductArgs : Segments {
    Product kind;
    bool gated;              // forward: w holds `cols` gate rows, then `cols` up rows; kBackwardX: with pre_in
    bool out_f32;            // kBackwardW
    bool pre_f32;            // of pre_in and pre; bf16 otherwise
    int32_t inner;           // channels of a row of x: summed over, but for kBackwardW (its n)
    int32_t cols;            // channels of a row of out (c)
    const void *x, *w;
    const float *xs, *ws;    // kForwardI8: [max_recv], [E, cols or 2*cols]
    const void *pre_in;      // kBackwardX: [max_recv, 2*cols] or null
    void *pre;               // kForward, gated: [max_recv, 2*cols] or null
    void *out;               // rows of `cols`; of 2*cols for kBackwardX with pre_in
};

hipError_t launch_product(const ProductArgs &a, hipStream_t s);
// Whether the grid fits a launch for any routing of this shape.
bool product_grid_ok(const ProductArgs &a);

}  // namespace moe
