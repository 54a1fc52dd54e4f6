// Products of every expert's rows with its weights in bf16 and in 8-bit integers,
// and their gradients (expert_products.h has the formulas).
//
// Every form is out[q][c] = sum over k of X[q][k] * W[c][k] on the matrix
// instructions, 16x16x32 for bf16 and 16x16x64 for integers: either way a lane
// carries 16 bytes of k of one row of each operand.  W is the instruction's first
// operand, so that a lane ends with four neighbouring channels c of one row q.
#include "expert_products.h"

#include <type_traits>

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <bool I8>
using Acc = std::conditional_t<I8, i32x4, f32x4>;

template <bool I8>
__device__ __forceinline__ Acc<I8> multiply(u32x4 w, u32x4 x, Acc<I8> acc) {
    if constexpr (I8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}

// d silu(g) / dg = s * (1 + g * (1 - s)), s = sigmoid(g)
__device__ __forceinline__ void gated_gradient(float g, float u, float dh, float &dg, float &du) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
    dg = dh * u * s * (1.0f + g * (1.0f - s));
    du = dh * (g * s);
}

// 64 rows by 64 channels per workgroup, four waves of 16 rows each; steps of 64
// bytes of k go through LDS.
constexpr int kTile = 64;
constexpr int kPitch = 80;   // bytes of a row in LDS

template <Product KIND, bool GATED>
__global__ __launch_bounds__(256) void k_product_simple(ProductArgs a, int tiles_c) {
    constexpr bool kI8 = KIND == Product::kForwardI8, kForward = KIND == Product::kForward || kI8;
    constexpr int kSize = kI8 ? 1 : 2, kInner = 64 / kSize;
    constexpr bool kSplit = kForward && GATED;                  // half of the tile's channels gate, half up
    constexpr int kOut = kSplit ? kTile / 2 : kTile;
    __shared__ __align__(16) unsigned char xt[kTile * kPitch], wt[kTile * kPitch];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, r = lane & 15, g = lane >> 4;
    RowTile t{};
    if constexpr (KIND == Product::kBackwardW) {
        const int tiles_q = (a.inner + kTile - 1) / kTile;
        int b = blockIdx.x;
        t.ntile = b % tiles_c;
        b /= tiles_c;
        t.row0 = b % tiles_q * kTile;
        t.rows = min(kTile, a.inner - t.row0);
        t.expert = b / tiles_q;
        if (t.expert >= a.E) return;
    } else {
        if (!find_tile<kTile>(a, blockIdx.x, tiles_c, t)) return;
    }
    const int c0 = t.ntile * kOut;
    Acc<kI8> acc[4];
    for (int i = 0; i < 4; ++i) acc[i] = Acc<kI8>{0, 0, 0, 0};
    const auto products = [&]() {
        const u32x4 xv = *reinterpret_cast<const u32x4 *>(&xt[(wave * 16 + r) * kPitch + g * 16]);
        for (int i = 0; i < 4; ++i) acc[i] = multiply<kI8>(*reinterpret_cast<const u32x4 *>(&wt[(i * 16 + r) * kPitch + g * 16]), xv, acc[i]);
    };
    const u32x4 zero = {0u, 0u, 0u, 0u};
    // eight neighbouring channels of step row k go to eight rows of the tile
    const auto scatter = [&](unsigned char *to, int k, int c, u32x4 v) {
        const unsigned short *h = reinterpret_cast<const unsigned short *>(&v);
        for (int i = 0; i < 8; ++i) *reinterpret_cast<unsigned short *>(&to[(c + i) * kPitch + k * 2]) = h[i];
    };
    const int row = tid / 4, chunk = tid % 4, krow = tid / 8, cchunk = tid % 8 * 8;
    if constexpr (KIND == Product::kBackwardW) {
        const auto segment = [&](int first, int n) {
            for (int k0 = 0; k0 < n; k0 += kInner) {
                u32x4 xv = zero, wv = zero;
                if (k0 + krow < n) {
                    const size_t at = static_cast<size_t>(first) + k0 + krow;
                    if (t.row0 + cchunk < a.inner)
                        xv = *reinterpret_cast<const u32x4 *>(static_cast<const unsigned short *>(a.x) + at * a.inner + t.row0 + cchunk);
                    if (c0 + cchunk < a.cols)
                        wv = *reinterpret_cast<const u32x4 *>(static_cast<const unsigned short *>(a.w) + at * a.cols + c0 + cchunk);
                }
                __syncthreads();
                scatter(xt, krow, cchunk, xv);
                scatter(wt, krow, cchunk, wv);
                __syncthreads();
                products();
            }
        };
        if (a.seg_offset == nullptr) {
            segment(a.offset[t.expert], a.count[t.expert]);
        } else {
            const int epr = a.E / a.R, per = epr + a.B;
            const int home = t.expert / epr * per + t.expert % epr;
            segment(a.seg_offset[home], a.seg_offset[home + 1] - a.seg_offset[home]);
            for (int s = 0; s < a.R * a.B; ++s)
                if (a.slot_expert[s] == t.expert) {
                    const int i = s / a.B * per + epr + s % a.B;
                    segment(a.seg_offset[i], a.seg_offset[i + 1] - a.seg_offset[i]);
                }
        }
    } else {
        for (int k0 = 0; k0 < a.inner; k0 += kInner) {
            u32x4 xv = zero, wv = zero;
            const int k = k0 + chunk * (16 / kSize);
            if (row < t.rows && k < a.inner)
                xv = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.x) + ((static_cast<size_t>(t.row0) + row) * a.inner + k) * kSize);
            if constexpr (kForward) {
                const int half = kSplit && row >= kOut ? 1 : 0, c = c0 + row - half * kOut;
                if (c < a.cols && k < a.inner)
                    wv = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.w) +
                                                         ((static_cast<size_t>(t.expert) * (kSplit ? 2 : 1) + half) * a.cols + c) * a.inner * kSize + static_cast<size_t>(k) * kSize);
            } else {
                if (k0 + krow < a.inner && c0 + cchunk < a.cols)
                    wv = *reinterpret_cast<const u32x4 *>(static_cast<const unsigned short *>(a.w) +
                                                         (static_cast<size_t>(t.expert) * a.inner + k0 + krow) * a.cols + c0 + cchunk);
            }
            __syncthreads();
            *reinterpret_cast<u32x4 *>(&xt[row * kPitch + chunk * 16]) = xv;
            if constexpr (kForward)
                *reinterpret_cast<u32x4 *>(&wt[row * kPitch + chunk * 16]) = wv;
            else
                scatter(wt, krow, cchunk, wv);
            __syncthreads();
            products();
        }
    }
    const int q = wave * 16 + r;
    if (q >= t.rows) return;
    const size_t out_row = KIND == Product::kBackwardW ? static_cast<size_t>(t.expert) * a.inner + t.row0 + q : static_cast<size_t>(t.row0) + q;
    for (int i = 0; i < (kSplit ? 2 : 4); ++i) {
        const int c = c0 + i * 16 + 4 * g;
        if (c >= a.cols) continue;
        f32x4 v;
        for (int j = 0; j < 4; ++j) v[j] = static_cast<float>(acc[i][j]);
        if constexpr (kI8) {
            for (int j = 0; j < 4; ++j) v[j] = v[j] * a.xs[out_row] * a.ws[static_cast<size_t>(t.expert) * (kSplit ? 2 : 1) * a.cols + c + j];
        }
        if constexpr (kSplit) {
            f32x4 u;
            for (int j = 0; j < 4; ++j) u[j] = static_cast<float>(acc[i + 2][j]);
            if constexpr (kI8) {
                for (int j = 0; j < 4; ++j) u[j] = u[j] * a.xs[out_row] * a.ws[(static_cast<size_t>(t.expert) * 2 + 1) * a.cols + c + j];
            } else if (a.pre != nullptr) {
                unsigned short *const pre = static_cast<unsigned short *>(a.pre) + out_row * 2 * a.cols;
                *reinterpret_cast<u32x2 *>(pre + c) = pack_bf16x4(v);
                *reinterpret_cast<u32x2 *>(pre + a.cols + c) = pack_bf16x4(u);
            }
            for (int j = 0; j < 4; ++j) v[j] = silu(v[j]) * u[j];
        }
        if constexpr (KIND == Product::kBackwardX && GATED) {
            const unsigned short *const pre = static_cast<const unsigned short *>(a.pre_in) + out_row * 2 * a.cols;
            f32x4 dg, du;
            for (int j = 0; j < 4; ++j) {
                float x, y;
                gated_gradient(bf16_lo(pre[c + j]), bf16_lo(pre[a.cols + c + j]), v[j], x, y);
                dg[j] = x;
                du[j] = y;
            }
            unsigned short *const to = static_cast<unsigned short *>(a.out) + out_row * 2 * a.cols;
            *reinterpret_cast<u32x2 *>(to + c) = pack_bf16x4(dg);
            *reinterpret_cast<u32x2 *>(to + a.cols + c) = pack_bf16x4(du);
        } else if (KIND == Product::kBackwardW && a.out_f32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + out_row * a.cols + c) = v;
        } else {
            *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.out) + out_row * a.cols + c) = pack_bf16x4(v);
        }
    }
}

int64_t grid_of(const ProductArgs &a, int &tiles_c) {
    const bool split = a.gated && a.kind != Product::kBackwardX;
    const int out = split ? kTile / 2 : kTile;
    tiles_c = (a.cols + out - 1) / out;
    const int64_t rows = a.kind == Product::kBackwardW ? static_cast<int64_t>(a.E) * ((a.inner + kTile - 1) / kTile) : most_tiles(a, kTile);
    return (rows * tiles_c + kXcds - 1) / kXcds * kXcds;
}

}  // namespace

bool product_grid_ok(const ProductArgs &a) {
    int tiles_c;
    return grid_of(a, tiles_c) <= kMaxLaunchThreads / 256;
}

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
    int tiles_c;
    const int64_t blocks = grid_of(a, tiles_c);
    if (blocks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(blocks)), block(256);
#define MOE_PRODUCT(KIND, GATED) hipLaunchKernelGGL((k_product_simple<Product::KIND, GATED>), grid, block, 0, s, a, tiles_c)
    switch (a.kind) {
        case Product::kForward: if (a.gated) MOE_PRODUCT(kForward, true); else MOE_PRODUCT(kForward, false); break;
        case Product::kForwardI8: if (a.gated) MOE_PRODUCT(kForwardI8, true); else MOE_PRODUCT(kForwardI8, false); break;
        case Product::kBackwardX: if (a.gated) MOE_PRODUCT(kBackwardX, true); else MOE_PRODUCT(kBackwardX, false); break;
        case Product::kBackwardW: MOE_PRODUCT(kBackwardW, false); break;
    }
#undef MOE_PRODUCT
    return hipGetLastError();
}

}  // namespace moe
