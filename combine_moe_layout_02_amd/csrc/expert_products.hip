// Products of every expert's rows with its weights in bf16 and in 8-bit integers,
// and their gradients (expert_products.h has the formulas).
//
// Every form is out[q][c] = sum over k of X[q][k] * W[c][k] on the matrix
// instructions, 16x16x32 for bf16 and 16x16x64 for integers: either way a lane
// carries 16 bytes of k of one row of each operand.  W is the instruction's first
// operand, so that a lane ends with four neighbouring channels c of one row q.
//
//   form        X: rows q of          W: rows c of             k
//   forward     the receive buffer    the expert's weights     channels (neighbours)
//   backward x  d_out                 the weights, transposed  channels; W's rows are k
//   backward w  d_out, transposed     x, transposed            the expert's rows, of both
//
// An operand whose rows are k lies in memory with c (or q) as neighbours: it goes
// to LDS as it lies and is transposed on its way to the registers
// (ds_read_b64_tr_b16).
#include "expert_products.h"
#include "tile_copies.h"

#include <type_traits>

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
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

// d silu(g) / dg = s * (1 + g * (1 - s)), s = sigmoid(g), with the hardware's
// exponential and reciprocal as in silu().
__device__ __forceinline__ void gated_gradient(float g, float u, float dh, float &dg, float &du) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
    dg = dh * u * s * (1.0f + g * (1.0f - s));
    du = dh * (g * s);
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

// A tile is up to 256 rows q by 256 channels c.  One workgroup of eight waves per
// CU takes tile after tile; each wave holds 128 x 64 (128 accumulator registers),
// or for at most 128 rows all of them by 32 channels.  A stage, 128 bytes of k of
// every row (64 rows of k where those are the memory's rows), 64 KB, is copied to
// LDS while the stage before it is multiplied; it has two steps of 64 bytes.
constexpr int kGemmWaves = 8;
constexpr int kGemmThreads = kGemmWaves * kWave;
constexpr int kTileCols = 256;
constexpr int kOperandVecs = 2048;             // 16-byte vectors of one operand's stage
constexpr int kPairVecs = 2 * kOperandVecs;    // X, then W
constexpr int kStageK = 64;                    // rows of k of a stage of a transposed operand

template <Product KIND>
struct Form {
    static constexpr bool kI8 = KIND == Product::kForwardI8;
    static constexpr bool kForward = KIND == Product::kForward || kI8;
    static constexpr bool kXByK = KIND == Product::kBackwardW;      // X's rows in memory are k
    static constexpr bool kWByK = !kForward;
    static constexpr int kSize = kI8 ? 1 : 2;                       // bytes of an element
};

// Rows of k of a stage lie at a pitch of 512 bytes.  The transposing read's 16
// lanes of one group take four rows of k (its lanes' quarter of each 32 bytes);
// 32-byte block b of row k lies at b ^ turn(k), so that the eight rows that half a
// wave reads are in eight different groups of banks.
__device__ __forceinline__ int k_turn(int k) { return (k & 3) | (k >> 1 & 4); }

// Where a lane's operands lie.  K neighbours: row i*16 + r of the wave's, chunk
// 4h + g at (4h + g) ^ (r % 8).
template <bool BY_K>
struct Reader {
    int at[2];
    unsigned int base;
    __device__ __forceinline__ Reader(int first, int lane) {   // the wave's first row (of 16 * a power of two)
        const int r = lane & 15, g = lane >> 4;
        if constexpr (BY_K) {
            const int k = 8 * g + r / 4;
            base = static_cast<unsigned int>(k * 512 + ((first / 16) ^ k_turn(k)) * 32 + (r & 3) * 8);
        } else {
            at[0] = (first + r) * 8 + (g ^ (r & 7));
            at[1] = (first + r) * 8 + ((4 + g) ^ (r & 7));
        }
    }
    __device__ __forceinline__ u32x4 operator()(const u32x4 *stage, int h, int i) const {
        if constexpr (BY_K) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const char *const p = reinterpret_cast<const char *>(stage) + (base ^ static_cast<unsigned int>(i * 32)) + h * 16384;
            // rows 8g .. 8g+3 of the step, then 8g+4 .. 8g+7
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 2048));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a[0], a[1], b[0], b[1]};
        } else {
            return stage[at[h] + i * 128];
        }
    }
};

struct ProductTile {
    int row0, rows;    // rows q: of the receive buffer, or (kBackwardW) n
    int expert;
    int c0;            // first channel
    int first, end;    // kBackwardW: the expert's rows, but for its replicas'
};

// Asks for a tile's stages, one after the other.
template <Product KIND, bool GATED>
struct Feed {
    using F = Form<KIND>;
    static constexpr bool kSplit = F::kForward && GATED;
    unsigned int xo, wo;                 // this lane's first offsets
    __amdgpu_buffer_rsrc_t x, gate, up;  // K neighbours: the tile's rows; gate, then up weights
    const char *xk, *wk;                 // rows of k: the next stage's first
    int left;                            // rows of k, or bytes of k, not asked for yet
    int s;                               // stage
    int slot;                            // kBackwardW, balanced: replica slots looked at

    __device__ __forceinline__ bool next_run(const ProductArgs &a, const ProductTile &t) {
        if (a.seg_offset == nullptr) return false;
        const int lane = threadIdx.x & (kWave - 1), slots = a.R * a.B;
        while (slot < slots) {
            const int i = slot + lane;
            const uint64_t mine = __ballot(i < slots && a.slot_expert[min(i, slots - 1)] == t.expert);
            if (mine == 0) {
                slot += kWave;
                continue;
            }
            const int found = slot + __builtin_ctzll(mine);
            slot = found + 1;
            const int epr = a.E / a.R, seg = found / a.B * (epr + a.B) + epr + found % a.B;
            run(a, t, a.seg_offset[seg], a.seg_offset[seg + 1]);
            if (left > 0) return true;
        }
        return false;
    }
    __device__ __forceinline__ void run(const ProductArgs &a, const ProductTile &t, int first, int end) {
        first = __builtin_amdgcn_readfirstlane(first);
        left = __builtin_amdgcn_readfirstlane(end) - first;
        xk = static_cast<const char *>(a.x) + static_cast<size_t>(first) * a.inner * 2 + static_cast<size_t>(t.row0) * 2;
        wk = static_cast<const char *>(a.w) + static_cast<size_t>(first) * a.cols * 2 + static_cast<size_t>(t.c0) * 2;
    }

    __device__ __forceinline__ void start(const ProductArgs &a, const ProductTile &t) {
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize, cb = static_cast<unsigned int>(a.cols) * 2;
        // of eight rows of k neighbours: row lane/8, its chunk; of two rows of k: row
        // lane/32, its chunk (copy_k() has the rows that this wave takes)
        const int k = 2 * (wave & 1) + 8 * (wave >> 1 & 1) + 4 * (wave >> 2) + lane / 32;
        const unsigned int k_chunk = ((lane & 31) ^ (2 * k_turn(k))) * 16;
        s = 0;
        slot = 0;
        if constexpr (KIND == Product::kBackwardW) {
            xo = k * xb + k_chunk;
            wo = k * cb + k_chunk;
            run(a, t, t.first, t.end);
        } else {
            x = buffer_of(static_cast<const char *>(a.x) + static_cast<size_t>(t.row0) * xb, t.rows * xb);
            xo = (wave * 8 + lane / 8) * xb + lane_chunk(lane);
            if constexpr (F::kForward) {
                left = static_cast<int>(xb);
                const unsigned int wrows = min(kSplit ? kTileCols / 2 : kTileCols, a.cols - t.c0);
                const char *const first = static_cast<const char *>(a.w) + (static_cast<size_t>(t.expert) * (kSplit ? 2 : 1) * a.cols + t.c0) * xb;
                gate = buffer_of(first, wrows * xb);
                up = kSplit ? buffer_of(first + static_cast<size_t>(a.cols) * xb, wrows * xb) : gate;
                wo = lane / 8 * xb + lane_chunk(lane);
            } else {
                left = a.inner;
                wk = static_cast<const char *>(a.w) + static_cast<size_t>(t.expert) * a.inner * cb + static_cast<size_t>(t.c0) * 2;
                wo = k * cb + k_chunk;
            }
        }
    }

    // Rows of k `n` (at most 64) from `from`: the wave's copies take two rows each,
    // with the same turn.  Rows past the last read zeros.
    __device__ __forceinline__ void copy_k(const char *from, int n, unsigned int row_bytes, unsigned int first, u32x4 *to) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        // the first row begins at the tile's column: what follows it in memory belongs
        // to the buffer as far as the last row's end of the columns asked for
        const auto b = buffer_of(from, n > 0 ? static_cast<unsigned int>(n - 1) * row_bytes + k_bytes : 0u);
        const int k0 = 2 * (wave & 1) + 8 * (wave >> 1 & 1) + 4 * (wave >> 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dk = 16 * j;
            copy_to_lds(b, to + (k0 + dk) * 32, first + dk * row_bytes, 0);
        }
    }
    unsigned int k_bytes;

    // Whether there is another stage.
    __device__ __forceinline__ bool have(const ProductArgs &a, const ProductTile &t) {
        if constexpr (KIND == Product::kBackwardW)
            return left > 0 || next_run(a, t);
        else
            return left > 0;
    }
    __device__ __forceinline__ void step(const ProductArgs &a) {
        if constexpr (F::kXByK) xk += static_cast<size_t>(kStageK) * a.inner * 2;
        if constexpr (F::kWByK) wk += static_cast<size_t>(kStageK) * a.cols * 2;
        left -= F::kForward ? kStageBytes : kStageK;
        ++s;
    }

    // Asks for the next stage, if there is one, into `stage`; false if there is none.
    // XCOPIES: 8 rows of X per wave and copy.
    template <int XCOPIES>
    __device__ __forceinline__ bool copy(const ProductArgs &a, const ProductTile &t, u32x4 *stage, int wave_cols) {
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        if (!have(a, t)) return false;
        const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize, cb = static_cast<unsigned int>(a.cols) * 2;
        unsigned int x_lane = xo, w_lane = wo;
        asm volatile("" : "+v"(x_lane), "+v"(w_lane));    // offsets are made here, not kept in a register each
        if constexpr (F::kXByK) {
            const int n = min(left, kStageK);
            k_bytes = min(512u, xb - static_cast<unsigned int>(t.row0) * 2);
            copy_k(xk, n, xb, x_lane, stage);
            k_bytes = min(512u, cb - static_cast<unsigned int>(t.c0) * 2);
            copy_k(wk, n, cb, w_lane, stage + kOperandVecs);
        } else {
            const int bytes = F::kForward ? left : 2 * left;      // of k, from this stage on
            const unsigned int gone = static_cast<int>(lane_chunk(lane)) >= bytes ? kPastEnd : 0u;
#pragma unroll
            for (int j = 0; j < XCOPIES; ++j)
                copy_to_lds(x, stage + (j * kGemmWaves + wave) * 64, (x_lane + j * kGemmWaves * 8 * xb) | gone, s * kStageBytes);
            if constexpr (F::kForward) {
                // 32 rows of the tile; gated, the second half of a wave's channels (wave_cols)
                // are the up rows of the first
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    int row = wave * 32 + j * 8;
                    bool is_up = false;
                    if constexpr (kSplit) {
                        const int half = wave_cols / 2, of = row / wave_cols * half, in = row % wave_cols;
                        is_up = in >= half;
                        row = of + in - (is_up ? half : 0);
                    }
                    copy_to_lds(is_up ? up : gate, stage + kOperandVecs + (wave * 4 + j) * 64, (w_lane + row * xb) | gone, s * kStageBytes);
                }
            } else {
                k_bytes = min(512u, cb - static_cast<unsigned int>(t.c0) * 2);
                copy_k(wk, min(left, kStageK), cb, w_lane, stage + kOperandVecs);
            }
        }
        step(a);
        return true;
    }
};

// 16-byte chunk c of row q of a plane in LDS lies at c ^ turn(q), against bank
// conflicts: rows of CHUNKS chunks.
template <int CHUNKS>
__device__ __forceinline__ int plane_turn(int q) { return (CHUNKS >= 8 ? q : q * CHUNKS / 8) & (CHUNKS - 1); }

// Writes four neighbouring channels (from 4*g of tile i of 16) of row q.
template <int CHUNKS>
__device__ __forceinline__ void plane_put(u32x4 *plane, int q, int i, int g, f32x4 v) {
    reinterpret_cast<u32x2 *>(plane)[(q * CHUNKS + ((2 * i + (g >> 1)) ^ plane_turn<CHUNKS>(q))) * 2 + (g & 1)] = pack_bf16x4(v);
}

// Stores 32 rows of a plane: channels c0 .. of rows `row_bytes` apart, from row q0
// of `to`.  Rows outside the tile fall past the buffer's end, channels past `cols`
// are sent there.
template <int CHUNKS>
__device__ __forceinline__ void plane_store(const u32x4 *plane, __amdgpu_buffer_rsrc_t to, unsigned int row_bytes, int q0, int c0, int cols) {
    const int lane = threadIdx.x & (kWave - 1);
    constexpr int kRows = kWave / CHUNKS;
#pragma unroll
    for (int j = 0; j < 32 / kRows; ++j) {
        const int q = j * kRows + lane / CHUNKS, c = lane % CHUNKS;
        const u32x4 v = plane[q * CHUNKS + (c ^ plane_turn<CHUNKS>(q))];
        const unsigned int at = c0 + c * 8 < cols ? (q0 + q) * row_bytes + 2u * (c0 + c * 8) : kPastEnd;
        __builtin_amdgcn_raw_buffer_store_b128(v, to, static_cast<int>(at), 0, kNonTemporal);
    }
}

// What is done with a wave's sums: TT tiles of 16 rows from row q0 of the tile, WT
// tiles of 16 channels; n0: the first channel.  `mine`: 8 KB of LDS.
template <int TT, int WT, Product KIND, bool GATED>
__device__ __forceinline__ void finish(const ProductArgs &a, const ProductTile &t, Acc<Form<KIND>::kI8> (&acc)[TT][WT], int q0, int n0,
                                       u32x4 *mine) {
    using F = Form<KIND>;
    constexpr bool kSplit = F::kForward && GATED;
    constexpr int kOut = kSplit ? WT / 2 : WT, kChunks = 2 * kOut;
    const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
    const unsigned int row_bytes = static_cast<unsigned int>(a.cols) * 2u;
    const size_t first = KIND == Product::kBackwardW ? static_cast<size_t>(t.expert) * a.inner + t.row0 : static_cast<size_t>(t.row0);
    if constexpr (KIND == Product::kBackwardW) {
        if (a.out_f32) {
            // 16 bytes of one row per lane; a row's neighbours follow in the next store
            const auto to = buffer_of(static_cast<char *>(a.out) + first * row_bytes * 2, static_cast<unsigned int>(t.rows) * row_bytes * 2);
#pragma unroll
            for (int m = 0; m < TT; ++m)
#pragma unroll
                for (int i = 0; i < WT; ++i) {
                    const int c = n0 + i * 16 + 4 * g;
                    const unsigned int at = c < a.cols ? (q0 + m * 16 + r) * row_bytes * 2 + 4u * c : kPastEnd;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[m][i]), to, static_cast<int>(at), 0, 0);
                }
            return;
        }
    }
    if constexpr (KIND == Product::kBackwardX && GATED) {
        // the sums pass LDS in fp32: a lane then has eight neighbouring channels of a
        // row, and reads and writes 16 bytes of gate and up each
        constexpr int kF = 4 * WT, kRowsAt = kWave / (2 * WT);
        const auto pre = buffer_of(static_cast<const char *>(a.pre_in) + first * row_bytes * 2, static_cast<unsigned int>(t.rows) * row_bytes * 2);
        const auto to = buffer_of(static_cast<char *>(a.out) + first * row_bytes * 2, static_cast<unsigned int>(t.rows) * row_bytes * 2);
#pragma unroll
        for (int m0 = 0; m0 < TT; m0 += 2) {
#pragma unroll
            for (int m = m0; m < m0 + 2; ++m)
#pragma unroll
                for (int i = 0; i < WT; ++i) {
                    const int q = (m - m0) * 16 + r;
                    mine[q * kF + ((4 * i + g) ^ (r & (kF - 1)))] = __builtin_bit_cast(u32x4, acc[m][i]);
                }
            wave_lds_fence();
#pragma unroll
            for (int j = 0; j < 32 / kRowsAt; ++j) {
                const int q = j * kRowsAt + lane / (2 * WT), c = lane % (2 * WT);
                const f32x4 lo = __builtin_bit_cast(f32x4, mine[q * kF + ((2 * c) ^ (q & 15 & (kF - 1)))]);
                const f32x4 hi = __builtin_bit_cast(f32x4, mine[q * kF + ((2 * c + 1) ^ (q & 15 & (kF - 1)))]);
                const unsigned int at = n0 + c * 8 < a.cols ? (q0 + m0 * 16 + q) * row_bytes * 2 + 2u * (n0 + c * 8) : kPastEnd;
                const unsigned int at_up = at == kPastEnd ? kPastEnd : at + row_bytes;
                const u32x4 gv = __builtin_amdgcn_raw_buffer_load_b128(pre, static_cast<int>(at), 0, 0);
                const u32x4 uv = __builtin_amdgcn_raw_buffer_load_b128(pre, static_cast<int>(at_up), 0, 0);
                f32x4 dg[2], du[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float gf = e & 1 ? bf16_hi(gv[e / 2]) : bf16_lo(gv[e / 2]), uf = e & 1 ? bf16_hi(uv[e / 2]) : bf16_lo(uv[e / 2]);
                    float x, y;
                    gated_gradient(gf, uf, e < 4 ? lo[e & 3] : hi[e & 3], x, y);
                    dg[e / 4][e & 3] = x;
                    du[e / 4][e & 3] = y;
                }
                const u32x2 a0 = pack_bf16x4(dg[0]), a1 = pack_bf16x4(dg[1]), b0 = pack_bf16x4(du[0]), b1 = pack_bf16x4(du[1]);
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{a0[0], a0[1], a1[0], a1[1]}, to, static_cast<int>(at), 0, 0);
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{b0[0], b0[1], b1[0], b1[1]}, to, static_cast<int>(at_up), 0, 0);
            }
            wave_lds_fence();
        }
        return;
    }
    const auto to = buffer_of(static_cast<char *>(a.out) + first * row_bytes, static_cast<unsigned int>(t.rows) * row_bytes);
    const bool keep = kSplit && !F::kI8 && a.pre != nullptr;
    const auto pre = keep ? buffer_of(static_cast<char *>(a.pre) + first * row_bytes * 2, static_cast<unsigned int>(t.rows) * row_bytes * 2) : to;
    f32x4 ws[F::kI8 ? WT : 1];
    if constexpr (F::kI8) {
#pragma unroll
        for (int i = 0; i < WT; ++i) {
            const int c = n0 + (i % kOut) * 16 + 4 * g;
            const float *const from = a.ws + (static_cast<size_t>(t.expert) * (kSplit ? 2 : 1) + i / kOut) * a.cols;
            ws[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (c < a.cols)
#pragma unroll
                for (int e = 0; e < 4; ++e) ws[i][e] = from[c + e];
        }
    }
#pragma unroll
    for (int m0 = 0; m0 < TT; m0 += 2) {
#pragma unroll
        for (int m = m0; m < m0 + 2; ++m) {
            const int q = (m - m0) * 16 + r;
            float xs = 0.0f;
            if constexpr (F::kI8) {
                if (q0 + m * 16 + r < t.rows) xs = a.xs[first + q0 + m * 16 + r];
            }
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                f32x4 v, u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = static_cast<float>(acc[m][i][e]);
                    u[e] = static_cast<float>(acc[m][kSplit ? i + kOut : i][e]);
                    if constexpr (F::kI8) {
                        v[e] = v[e] * xs * ws[i][e];
                        u[e] = u[e] * xs * ws[kSplit ? i + kOut : i][e];
                    }
                }
                if constexpr (kSplit) {
                    if (keep) {
                        plane_put<kChunks>(mine + 32 * kChunks, q, i, g, v);
                        plane_put<kChunks>(mine + 64 * kChunks, q, i, g, u);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = silu(v[e]) * u[e];
                }
                plane_put<kChunks>(mine, q, i, g, v);
            }
        }
        wave_lds_fence();
        plane_store<kChunks>(mine, to, row_bytes, q0 + m0 * 16, n0, a.cols);
        if (keep) {
            plane_store<kChunks>(mine + 32 * kChunks, pre, 2 * row_bytes, q0 + m0 * 16, n0, a.cols);
            // up values lie `cols` channels further
            const auto pre_up = buffer_of(static_cast<char *>(a.pre) + first * row_bytes * 2 + row_bytes, static_cast<unsigned int>(t.rows) * row_bytes * 2 - row_bytes);
            plane_store<kChunks>(mine + 64 * kChunks, pre_up, 2 * row_bytes, q0 + m0 * 16, n0, a.cols);
        }
        wave_lds_fence();
    }
}

// One tile whose first stage, if it has one, is on its way to stage 0.
// next_first() asks for the next tile's, into the same place.
template <int TT, int WT, Product KIND, bool GATED, typename NextFirst>
__device__ __forceinline__ void run_tile(const ProductArgs &a, const ProductTile &t, Feed<KIND, GATED> &feed, bool any, u32x4 *stage0,
                                         u32x4 *stage1, NextFirst &&next_first) {
    using F = Form<KIND>;
    constexpr int kAcross = kTileCols / (16 * WT);                  // waves across the channels
    constexpr int kX = (TT * (kGemmWaves / kAcross) * 2 + kGemmWaves - 1) / kGemmWaves;
    constexpr bool kSplit = F::kForward && GATED;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // what follows from it is made once per tile, not kept from tile to tile
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int across = wave % kAcross, q0 = wave / kAcross * (16 * TT);
    const Reader<F::kXByK> xr(q0, lane);
    const Reader<F::kWByK> wr(across * 16 * WT, lane);
    Acc<F::kI8> acc[TT][WT];
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < WT; ++i) acc[m][i] = Acc<F::kI8>{0, 0, 0, 0};
    const auto products = [&](const u32x4 *stage, int h) {
        u32x4 w[WT];
#pragma unroll
        for (int i = 0; i < WT; ++i) w[i] = wr(stage + kOperandVecs, h, i);
#pragma unroll
        for (int m = 0; m < TT; ++m) {
            const u32x4 x = xr(stage, h, m);
#pragma unroll
            for (int i = 0; i < WT; ++i) acc[m][i] = multiply<F::kI8>(w[i], x, acc[m][i]);
        }
        // a step's products stay in their step: the compiler would move them,
        // with their operands, behind the barriers
#pragma unroll
        for (int m = 0; m < TT; ++m)
#pragma unroll
            for (int i = 0; i < WT; ++i) asm volatile("" : "+v"(acc[m][i]));
    };
    barrier_after<0>();                                            // stage 0 has arrived, stage 1 is free
    bool even = any;
    if (!even) next_first();
    while (even) {
        const bool odd = feed.template copy<kX>(a, t, stage1, 16 * WT);
        products(stage0, 0);
        products(stage0, 1);
        barrier_after<0>();                                        // stage 1 has arrived, stage 0 is free
        even = odd && feed.template copy<kX>(a, t, stage0, 16 * WT);
        if (!even) next_first();
        if (odd) {
            products(stage1, 0);
            products(stage1, 1);
        }
        if (even) barrier_after<0>();                              // stage 0 has arrived, stage 1 is free
    }
    barrier_after<63>();                                           // stage 1 is free
    finish<TT, WT, KIND, GATED>(a, t, acc, q0, t.c0 + across * (kSplit ? 8 : 16) * WT, stage1 + wave * 512);
}

template <Product KIND, bool GATED>
__global__ __launch_bounds__(kGemmThreads, 2) void k_product_tile(ProductArgs a, int tiles_c) {
    using F = Form<KIND>;
    constexpr bool kSplit = F::kForward && GATED;
    constexpr int kOutCols = kSplit ? kTileCols / 2 : kTileCols;
    constexpr bool kW = KIND == Product::kBackwardW;
    __shared__ u32x4 stage0[kPairVecs], stage1[kPairVecs];
    __shared__ SegTable segs;
    __shared__ int2 s_scan[kGemmWaves];
    const int tid = threadIdx.x;
    int total;
    const int tiles_q = (a.inner + kTileRows - 1) / kTileRows;   // kBackwardW
    if constexpr (kW) {
        total = a.E * tiles_q * tiles_c;
    } else {
        // the table: three segments per thread, every load at once
        constexpr int kPer = kMaxSegments / kGemmThreads;
        int first[kPer], n[kPer], tiles = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) load_segment(a, tid * kPer + j, first[j], n[j]);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            n[j] = segment_rows(a, tid * kPer + j, first[j], n[j]);
            tiles += (n[j] + kTileRows - 1) / kTileRows;
        }
        int2 all;
        int at = block_exclusive_scan2<kGemmWaves>(make_int2(tiles, 0), s_scan, all).x;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            if (i < a.nseg) {
                segs.before[i] = at * tiles_c;
                segs.first[i] = first[j];
                segs.rows[i] = n[j];
            }
            at += (n[j] + kTileRows - 1) / kTileRows;
        }
        if (tid == 0) segs.before[a.nseg] = all.x * tiles_c;
        __syncthreads();
        total = __builtin_amdgcn_readfirstlane(all.x) * tiles_c;
    }
    // Rounds of kCus tiles.  Runs of neighbouring tiles go to the workgroups of one
    // XCD, whose L2 then serves the tiles' common rows.  Where the last round has at
    // most a half or a quarter of them, its tiles are taken in two or four parts of
    // 128 or 64 rows.
    const int whole = total / kCus * kCus, rest = total - whole;
    const int halvings = rest * 4 <= kCus ? 2 : (rest * 2 <= kCus ? 1 : 0), items = whole + (rest << halvings);
    const int place = static_cast<int>(blockIdx.x) / kXcds, xcd = static_cast<int>(blockIdx.x) % kXcds;
    // What this workgroup takes in a round; false: nothing, then or later.
    const auto tile_of = [&](int round, ProductTile &t) {
        const int left = min(items - round * kCus, kCus), run = (left + kXcds - 1) / kXcds, at = xcd * run + place;
        if (place >= run || at >= left) return false;
        const int item = round * kCus + at, cut = item < whole ? 0 : halvings;
        const int tile = item - (cut ? item - whole - ((item - whole) >> cut) : 0);
        if constexpr (kW) {
            t.c0 = tile / tiles_q % tiles_c * kOutCols;
            t.row0 = tile % tiles_q * kTileRows;
            t.expert = tile / tiles_q / tiles_c;
            t.rows = min(kTileRows, a.inner - t.row0);
            if (a.seg_offset == nullptr) {
                t.first = a.offset[t.expert];
                t.end = t.first + a.count[t.expert];
            } else {
                const int epr = a.E / a.R, home = t.expert / epr * (epr + a.B) + t.expert % epr;
                t.first = a.seg_offset[home];
                t.end = a.seg_offset[home + 1];
            }
        } else {
            const RowTile rt = tile_at(a, segs, tile);
            t = ProductTile{rt.row0, rt.rows, rt.expert, rt.ntile * kOutCols, 0, 0};
        }
        const int part_rows = kTileRows >> cut, skip = cut ? (((item - whole) & ((1 << cut) - 1)) * part_rows) : 0;
        t.row0 += skip;
        t.rows = __builtin_amdgcn_readfirstlane(min(t.rows - skip, part_rows));
        return t.rows > 0;
    };
    // channels of a wave
    const auto cols_of = [](const ProductTile &t) { return t.rows > 128 ? 64 : 32; };
    ProductTile t;
    if (!tile_of(0, t)) return;                                    // the same for every wave
    {
        Feed<KIND, GATED> first;
        first.start(a, t);
        first.template copy<4>(a, t, stage0, cols_of(t));
    }
    for (int round = 1;; ++round) {
        Feed<KIND, GATED> feed;
        feed.start(a, t);
        const bool any = feed.have(a, t);
        if (any) feed.step(a);
        ProductTile nt{};
        bool more = false;
        const auto next_first = [&]() {
            more = tile_of(round, nt);
            if (!more) return;
            Feed<KIND, GATED> first;
            first.start(a, nt);
            first.template copy<4>(a, nt, stage0, cols_of(nt));
        };
        if (t.rows > 128)
            run_tile<8, 4, KIND, GATED>(a, t, feed, any, stage0, stage1, next_first);
        else if (t.rows > 64)
            run_tile<8, 2, KIND, GATED>(a, t, feed, any, stage0, stage1, next_first);
        else if (t.rows > 32)
            run_tile<4, 2, KIND, GATED>(a, t, feed, any, stage0, stage1, next_first);
        else
            run_tile<2, 2, KIND, GATED>(a, t, feed, any, stage0, stage1, next_first);
        if (!more) return;
        t = nt;
    }
}

int64_t grid_of(const ProductArgs &a, int &tiles_c, int64_t &tiles) {
    const bool split = a.gated && a.kind != Product::kBackwardX;
    const int out = split ? kTileCols / 2 : kTileCols;
    tiles_c = (a.cols + out - 1) / out;
    const int64_t rows = a.kind == Product::kBackwardW ? static_cast<int64_t>(a.E) * ((a.inner + kTileRows - 1) / kTileRows) : most_tiles(a, kTileRows);
    tiles = rows * tiles_c;
    return std::min<int64_t>(4 * tiles, kCus);               // a tile may be taken in four parts
}

}  // namespace

bool product_grid_ok(const ProductArgs &a) {
    int tiles_c;
    int64_t tiles;
    grid_of(a, tiles_c, tiles);
    return tiles <= INT32_MAX - kCus;
}

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
    int tiles_c;
    int64_t tiles;
    const int64_t blocks = grid_of(a, tiles_c, tiles);
    if (blocks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>((blocks + kXcds - 1) / kXcds * kXcds)), block(kGemmThreads);
#define MOE_PRODUCT(KIND, GATED) hipLaunchKernelGGL((k_product_tile<Product::KIND, GATED>), grid, block, 0, s, a, tiles_c)
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
