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
//
// Sums are fp32, or 32-bit integers, in an order that the layout alone decides.  A
// result is rounded once, to bf16: what the next product's instructions take.  The
// arguments of the activation may be kept in fp32, since their rounding would pass
// into the gradients besides that of the gradient's own rows.  With what lies between
// two products in bf16, a block's rows and gradients are 0.0023 to 0.0024 off 64 bits,
// with fp32 there 0.0017, which is the results' own rounding.
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
// or for at most 128 rows all of them by 32 channels.
//
// 128 bytes of k of every row (64 rows of k where those are the memory's rows), a
// whole line each, make a pair of stages.  The first stage multiplies half of each
// wave's rows q with its channels, the second the other half with the same
// channels, which stay in registers: so X is needed in two halves, one a stage
// later.  LDS holds two pairs, 128 KB: while one stage is multiplied what the next
// three need is on its way, across tiles too.
//
// 98304 rows of 64 experts, 2048 channels and 2 x 1408 (1.13 TFLOP, or half of it):
//   gate and up 945 us, down 479, x's gradient 933, the weights' 985 and 542:
//   1.05 to 1.22 PFLOP/s; 8-bit integers 530 and 312 us, 1.8 to 2.1 POP/s.  Four
//   experts of 4096 rows and 4096 x 4096 weights: 1.24 to 1.32 PFLOP/s, 2.4 to 2.5 POP/s.
//   One library product of all rows with one expert's weights: 1.28.
// In a tile's loop 128 channels of k take 2.85 to 3.1 us: 1.4 to 1.5 PFLOP/s, where the
// card's power holds the clock at about 1.9 GHz.  The first three such steps of a tile,
// whose copies wait behind the last tile's stores, take 0.3 us more each, the last
// products and the stores 3 to 4 us, pre in fp32 another 6, and a gradient through
// the activation 26 (785 us, where the product alone takes 540; 686 with pre in bf16):
// all workgroups reach it at one time, and 1.1 GB of pre and 0.55 of its gradient move in
// ten bursts at close to 6 TB/s, what memory gives; in the loops between it is nearly idle.
// Without copies, or without stores, the same loop takes 0.77 of the time.
// Slower, or no faster: four waves of 128 x 128 (registers spill where gated);
// stages of 64 bytes in a ring; the next tile's lines asked for ahead of it; waves
// that only copy; other cache policies of the stores; XCDs half a tile apart; tiles
// of more than 128 rows before the others, which evens out the workgroups' shares;
// pre asked for two or three rows ahead.
constexpr int kGemmWaves = 8;
constexpr int kGemmThreads = kGemmWaves * kWave;
constexpr int kTileCols = 256;
constexpr int kHalfVecs = 1024;                // 16-byte vectors of half of X of a pair
constexpr int kWVecs = 2048;                   // of W
constexpr int kPairBytes = 128;                // bytes of k of a pair
constexpr int kPairK = 64;                     // rows of k of a pair of a transposed operand
constexpr int kInFlight = 8;                   // a wave's copies of two stages: two of X, then two of X and four of W

template <Product KIND>
struct Form {
    static constexpr bool kI8 = KIND == Product::kForwardI8;
    static constexpr bool kForward = KIND == Product::kForward || kI8;
    static constexpr bool kXByK = KIND == Product::kBackwardW;      // X's rows in memory are k
    static constexpr bool kWByK = !kForward;
    static constexpr int kSize = kI8 ? 1 : 2;                       // bytes of an element
};

// Rows of k lie at a pitch of 512 bytes (W) or 256 (half of X).  The transposing
// read's 16 lanes of one group take four rows of k (its lanes' quarter of each 32
// bytes); 32-byte block b of row k lies at b ^ turn(k), so that the eight rows that
// half a wave reads are in eight different groups of banks.
__device__ __forceinline__ int k_turn(int k) { return (k & 3) | (k >> 1 & 4); }

// Where a lane's operands lie, of tiles of 16 rows (q or c) from `first` of the
// buffer's, at step h of the pair.  K neighbours: row r, chunk 4h + g at
// (4h + g) ^ (r % 8).
template <bool BY_K, int PITCH>
struct Reader {
    int at[2];
    unsigned int base;
    __device__ __forceinline__ Reader(int first, int lane) {   // first: 16 * a multiple of the power of two of tiles
        const int r = lane & 15, g = lane >> 4;
        if constexpr (BY_K) {
            const int k = 8 * g + r / 4;
            base = static_cast<unsigned int>(k * PITCH + ((first / 16) ^ k_turn(k)) * 32 + (r & 3) * 8);
        } else {
            at[0] = (first + r) * 8 + (g ^ (r & 7));
            at[1] = (first + r) * 8 + ((4 + g) ^ (r & 7));
        }
    }
    __device__ __forceinline__ u32x4 operator()(const u32x4 *buffer, int h, int i) const {
        if constexpr (BY_K) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const char *const p = reinterpret_cast<const char *>(buffer) + (base ^ static_cast<unsigned int>(i * 32)) + h * 32 * PITCH;
            // rows 8g .. 8g+3 of the step, then 8g+4 .. 8g+7
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * PITCH));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a[0], a[1], b[0], b[1]};
        } else {
            return buffer[at[h] + i * 128];
        }
    }
};

// The same in every lane: keeps descriptors and branches on the scalar side.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ const char *uniform(const char *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = static_cast<uint32_t>(uniform(static_cast<int>(v))), hi = static_cast<uint32_t>(uniform(static_cast<int>(v >> 32)));
    return reinterpret_cast<const char *>(hi << 32 | lo);
}

// A buffer over `n` (at most 64) rows of k from `from`; `bytes` of the last row
// belong to the tile.  Rows past the last read zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of_k(const char *from, int n, unsigned int bytes, unsigned int row_bytes) {
    return buffer_of(uniform(from), n > 0 ? static_cast<unsigned int>(n - 1) * row_bytes + bytes : 0u);
}

struct ProductTile {
    int row0, rows;    // rows q: of the receive buffer, or (kBackwardW) n
    int expert;
    int c0;            // first channel
    int first, end;    // kBackwardW: the expert's rows, but for its replicas'
};

// Asks for what a tile's stages need, pair by pair: W and the first half of X, then
// the second half.  Past the tile's last k it asks for zeros.
template <Product KIND, bool GATED>
struct Feed {
    using F = Form<KIND>;
    static constexpr bool kSplit = F::kForward && GATED;
    unsigned int xo, wo;                 // this lane's first offsets
    // K neighbours: X's first row, and of W the first row of each half of the wave's
    // copies, with the bytes from there to the tile's end; rows of k: the pair's first
    // row and the tile's bytes of each row
    const char *x, *w, *w1;
    unsigned int x_bytes, w_bytes, w1_bytes;
    int left;                            // rows of k, or bytes of k, from this pair on
    int at;                              // bytes of k before this pair
    int slot;                            // kBackwardW, balanced: replica slots looked at
    int row0, c0, expert;                // kBackwardW: of the tile

    // kBackwardW: rows first .. end-1 of the receive buffer
    __device__ __forceinline__ void run(const ProductArgs &a, int first, int end) {
        left = uniform(end - first);
        x = static_cast<const char *>(a.x) + (static_cast<size_t>(uniform(first)) * a.inner + row0) * 2;
        w = static_cast<const char *>(a.w) + (static_cast<size_t>(uniform(first)) * a.cols + c0) * 2;
    }
    __device__ __forceinline__ void next_run(const ProductArgs &a) {
        const int lane = threadIdx.x & (kWave - 1), slots = a.R * a.B;
        while (left <= 0 && slot < slots) {
            const int i = slot + lane;
            const uint64_t mine = __ballot(i < slots && a.slot_expert[min(i, slots - 1)] == expert);
            if (mine == 0) {
                slot += kWave;
                continue;
            }
            const int found = slot + __builtin_ctzll(mine);
            slot = found + 1;
            const int epr = a.E / a.R, seg = found / a.B * (epr + a.B) + epr + found % a.B;
            run(a, a.seg_offset[seg], a.seg_offset[seg + 1]);
        }
    }

    // A tile's first pair comes next.
    __device__ __forceinline__ void start(const ProductArgs &a, const ProductTile &t) {
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
        const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize, cb = static_cast<unsigned int>(a.cols) * 2;
        // W's rows of k: of the wave's copies of two rows, row lane/32 of the first and
        // its chunk
        const int k = 2 * (wave & 1) + 8 * (wave >> 1 & 1) + 4 * (wave >> 2) + lane / 32;
        const unsigned int k_chunk = ((lane & 31) ^ (2 * k_turn(k))) * 16;
        at = 0;
        slot = 0;
        if constexpr (KIND == Product::kBackwardW) {
            // half of X: two pieces of 128 bytes of each row of k, 256 apart; of the wave's
            // copies of four rows, row lane/16 of the first
            const int kx = 4 * wave + lane / 16, c = (lane & 15) ^ (2 * k_turn(kx));
            xo = kx * xb + (c >> 3) * 256 + (c & 7) * 16;
            wo = k * cb + k_chunk;
            x_bytes = min(512u, xb - static_cast<unsigned int>(t.row0) * 2);
            w_bytes = min(512u, cb - static_cast<unsigned int>(t.c0) * 2);
            row0 = t.row0;
            c0 = t.c0;
            expert = t.expert;
            run(a, t.first, t.end);
            if (a.seg_offset != nullptr) next_run(a);
        } else {
            x = static_cast<const char *>(a.x) + static_cast<size_t>(t.row0) * xb;
            x_bytes = t.rows * xb;
            // of copies of eight rows: row lane/8, its chunk
            xo = (wave * 8 + lane / 8) * xb + lane_chunk(lane);
            if constexpr (F::kForward) {
                left = static_cast<int>(xb);
                const bool wide = t.rows > 128;
                const WeightRows half = weight_rows(kSplit, wide, wave, 0), half1 = weight_rows(kSplit, wide, wave, 1);
                const int rows = min(kSplit ? kTileCols / 2 : kTileCols, a.cols - t.c0);
                const char *const first = static_cast<const char *>(a.w) + (static_cast<size_t>(t.expert) * (kSplit ? 2 : 1) * a.cols + t.c0) * xb;
                w = first + (static_cast<size_t>(half.up ? a.cols : 0) + half.first) * xb;
                w1 = first + (static_cast<size_t>(half1.up ? a.cols : 0) + half1.first) * xb;
                w_bytes = bytes_from(half.first, rows, xb);
                w1_bytes = bytes_from(half1.first, rows, xb);
                wo = lane / 8 * xb + lane_chunk(lane);
            } else {
                left = a.inner;
                w_bytes = min(512u, cb - static_cast<unsigned int>(t.c0) * 2);
                w = static_cast<const char *>(a.w) + (static_cast<size_t>(t.expert) * a.inner * a.cols + t.c0) * 2;
                wo = k * cb + k_chunk;
            }
        }
    }
    // The same, or zeros where no tile comes next.  (Without a branch: the two sides'
    // last stores would be joined, and what they store to kept in memory.)
    __device__ __forceinline__ void start_or_stop(const ProductArgs &a, const ProductTile &t) {
        start(a, t);
        const bool none = t.rows <= 0;
        left = none ? 0 : left;
        slot = none ? kMaxBalanceSlots : slot;
    }

    // kPastEnd for the lanes whose chunk of the pair lies past the row's end.
    __device__ __forceinline__ unsigned int gone() const {
        return past_row(F::kForward ? left : 2 * left, threadIdx.x & (kWave - 1));
    }

    // Half `half` of the pair's X.
    __device__ __forceinline__ void copy_x(const ProductArgs &a, u32x4 *to, int half) const {
        const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
        const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize;
        unsigned int x_lane = xo;
        asm volatile("" : "+v"(x_lane));                  // offsets are made here, not kept in a register each
        if constexpr (F::kXByK) {
            const auto b = rows_of_k(x, uniform(min(left, kPairK)), uniform(x_bytes), xb);
#pragma unroll
            for (int j = 0; j < 2; ++j) copy_to_lds(b, to + (j * 8 + wave) * 64, x_lane + j * 32 * xb + half * 128, 0);
        } else {
            // rows 0-63 and 128-191 of the tile, or those 64 further on
            const auto b = buffer_of(uniform(x), uniform(x_bytes));
            const unsigned int past = gone();
            const int shared = uniform(shared_offset(at, left, x_bytes));
#pragma unroll
            for (int j = 0; j < 2; ++j) copy_to_lds(b, to + (j * 8 + wave) * 64, (x_lane + (j * 128 + half * 64) * xb) | past, shared);
        }
    }
    // The pair's W.
    __device__ __forceinline__ void copy_w(const ProductArgs &a, u32x4 *to) const {
        const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
        unsigned int w_lane = wo;
        asm volatile("" : "+v"(w_lane));
        if constexpr (F::kWByK) {
            const unsigned int cb = static_cast<unsigned int>(a.cols) * 2;
            const auto b = rows_of_k(w, uniform(min(left, kPairK)), uniform(w_bytes), cb);
            const int k0 = 2 * (wave & 1) + 8 * (wave >> 1 & 1) + 4 * (wave >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_to_lds(b, to + (k0 + 16 * j) * 32, w_lane + 16 * j * cb, 0);
        } else {
            const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize, past = gone();
            const auto b = buffer_of(uniform(w), uniform(w_bytes)), b1 = buffer_of(uniform(w1), uniform(w1_bytes));
            const int shared = uniform(shared_offset(at, left, w_bytes)), shared1 = uniform(shared_offset(at, left, w1_bytes));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                copy_to_lds(b, to + (wave * 4 + j) * 64, (w_lane + j * 8 * xb) | past, shared);
                copy_to_lds(b1, to + (wave * 4 + 2 + j) * 64, (w_lane + j * 8 * xb) | past, shared1);
            }
        }
    }
    // What a pair's first stage needs, then what its second does.
    __device__ __forceinline__ void ask_first(const ProductArgs &a, u32x4 *x_to, u32x4 *w_to) const {
        copy_x(a, x_to, 0);
        copy_w(a, w_to);
    }
    __device__ __forceinline__ void ask_second(const ProductArgs &a, u32x4 *x_to) {
        copy_x(a, x_to, 1);
        if constexpr (F::kXByK) x += static_cast<size_t>(kPairK) * a.inner * 2;
        if constexpr (F::kWByK) w += static_cast<size_t>(kPairK) * a.cols * 2;
        at += kPairBytes;
        left -= F::kForward ? kPairBytes : kPairK;
        if constexpr (KIND == Product::kBackwardW) {
            if (a.seg_offset != nullptr) next_run(a);
        }
    }
};

// Pairs of a tile.
template <Product KIND>
__device__ __forceinline__ int pairs_of(const ProductArgs &a, const ProductTile &t) {
    if constexpr (Form<KIND>::kForward) return (a.inner * Form<KIND>::kSize + kPairBytes - 1) / kPairBytes;
    if constexpr (KIND == Product::kBackwardX) return (a.inner + kPairK - 1) / kPairK;
    int n = (t.end - t.first + kPairK - 1) / kPairK;
    if (a.seg_offset != nullptr) {
        const int lane = threadIdx.x & (kWave - 1), slots = a.R * a.B, epr = a.E / a.R;
        int mine = 0;
        for (int i = lane; i < slots; i += kWave)
            if (a.slot_expert[i] == t.expert) {
                const int seg = i / a.B * (epr + a.B) + epr + i % a.B;
                mine += (a.seg_offset[seg + 1] - a.seg_offset[seg] + kPairK - 1) / kPairK;
            }
        n += __builtin_amdgcn_readlane(wave_inclusive_scan(mine), kWave - 1);
    }
    return uniform(n);
}

// 16-byte chunk c of row q of a plane in LDS lies at c ^ turn(q), against bank
// conflicts: rows of CHUNKS chunks.
template <int CHUNKS>
__device__ __forceinline__ int plane_turn(int q) { return (CHUNKS >= 8 ? q : q * CHUNKS / 8) & (CHUNKS - 1); }

// Writes four neighbouring channels (from 4*g of tile i of 16) of row q.
template <int CHUNKS>
__device__ __forceinline__ void plane_put(u32x4 *plane, int q, int i, int g, f32x4 v) {
    reinterpret_cast<u32x2 *>(plane)[(q * CHUNKS + ((2 * i + (g >> 1)) ^ plane_turn<CHUNKS>(q))) * 2 + (g & 1)] = pack_bf16x4(v);
}

// Stores the 16 rows of a plane: channels c0 .. of rows `row_bytes` apart, from row
// q0 of `to`.  Rows outside the tile fall past the buffer's end, channels past
// `cols` are sent there.
template <int CHUNKS>
__device__ __forceinline__ void plane_store(const u32x4 *plane, __amdgpu_buffer_rsrc_t to, unsigned int row_bytes, int q0, int c0, int cols) {
    const int lane = threadIdx.x & (kWave - 1);
    constexpr int kRows = kWave / CHUNKS;
#pragma unroll
    for (int j = 0; j < (15 + kRows) / kRows; ++j) {
        const int q = j * kRows + lane / CHUNKS, c = lane % CHUNKS;
        const bool mine = kRows <= 16 || q < 16;
        const u32x4 v = plane[mine ? q * CHUNKS + (c ^ plane_turn<CHUNKS>(q)) : 0];
        const unsigned int at = mine && c0 + c * 8 < cols ? (q0 + q) * row_bytes + 2u * (c0 + c * 8) : kPastEnd;
        __builtin_amdgcn_raw_buffer_store_b128(v, to, static_cast<int>(at), 0, kNonTemporal);
    }
}

// What is done with a wave's sums: TT tiles of 16 rows from row q0 of the tile, WT
// tiles of 16 channels; n0: the first channel.  `mine`: 2 KB of LDS.
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
        // the sums pass LDS in fp32, 32 channels at a time: a lane then has eight
        // neighbouring channels of a row, and reads and writes whole 16 bytes of gate and up
        const auto to = buffer_of(static_cast<char *>(a.out) + first * row_bytes * 2, static_cast<unsigned int>(t.rows) * row_bytes * 2);
        const int q = lane / 4, c = lane & 3;
        const auto all_rows = [&](auto pre_f32_) {
            constexpr unsigned int kWide = decltype(pre_f32_)::value ? 2 : 1;   // vectors of eight channels of pre
            const unsigned int pre_bytes = row_bytes * 2 * kWide;
            const auto pre = buffer_of(static_cast<const char *>(a.pre_in) + first * pre_bytes, static_cast<unsigned int>(t.rows) * pre_bytes);
#pragma unroll
            for (int m = 0; m < TT; ++m) {
                u32x4 gv[WT / 2][kWide], uv[WT / 2][kWide];
                unsigned int at[WT / 2], at_up[WT / 2];
#pragma unroll
                for (int p = 0; p < WT / 2; ++p) {
                    const int n = n0 + p * 32 + c * 8;
                    at[p] = n < a.cols ? (q0 + m * 16 + q) * row_bytes * 2 + 2u * n : kPastEnd;
                    at_up[p] = n < a.cols ? at[p] + row_bytes : kPastEnd;
#pragma unroll
                    for (unsigned int e = 0; e < kWide; ++e) {
                        gv[p][e] = __builtin_amdgcn_raw_buffer_load_b128(pre, static_cast<int>(n < a.cols ? at[p] * kWide + e * 16 : kPastEnd), 0, 0);
                        uv[p][e] = __builtin_amdgcn_raw_buffer_load_b128(pre, static_cast<int>(n < a.cols ? at_up[p] * kWide + e * 16 : kPastEnd), 0, 0);
                    }
                }
#pragma unroll
                for (int p = 0; p < WT / 2; ++p) {
                    // eight chunks to the row
#pragma unroll
                    for (int i = 0; i < 2; ++i) mine[r * 8 + ((4 * i + g) ^ (r & 7))] = __builtin_bit_cast(u32x4, acc[m][2 * p + i]);
                    wave_lds_fence();
                    const f32x4 lo = __builtin_bit_cast(f32x4, mine[q * 8 + ((2 * c) ^ (q & 7))]);
                    const f32x4 hi = __builtin_bit_cast(f32x4, mine[q * 8 + ((2 * c + 1) ^ (q & 7))]);
                    wave_lds_fence();
                    const auto value = [&](const u32x4(&v)[kWide], int e) {
                        if constexpr (kWide == 2) return __builtin_bit_cast(f32x4, v[e / 4])[e & 3];
                        return e & 1 ? bf16_hi(v[0][e / 2]) : bf16_lo(v[0][e / 2]);
                    };
                    f32x4 dg[2], du[2];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float x, y;
                        gated_gradient(value(gv[p], e), value(uv[p], e), e < 4 ? lo[e & 3] : hi[e & 3], x, y);
                        dg[e / 4][e & 3] = x;
                        du[e / 4][e & 3] = y;
                    }
                    const u32x2 a0 = pack_bf16x4(dg[0]), a1 = pack_bf16x4(dg[1]), b0 = pack_bf16x4(du[0]), b1 = pack_bf16x4(du[1]);
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{a0[0], a0[1], a1[0], a1[1]}, to, static_cast<int>(at[p]), 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{b0[0], b0[1], b1[0], b1[1]}, to, static_cast<int>(at_up[p]), 0, 0);
                }
            }
        };
        if (a.pre_f32)
            all_rows(std::true_type{});
        else
            all_rows(std::false_type{});
        return;
    }
    const auto to = buffer_of(static_cast<char *>(a.out) + first * row_bytes, static_cast<unsigned int>(t.rows) * row_bytes);
    const bool keep = kSplit && !F::kI8 && a.pre != nullptr;
    const unsigned int pre_up_at = row_bytes * (a.pre_f32 ? 2 : 1), pre_bytes = pre_up_at * 2;   // up values lie `cols` channels further
    const auto pre = keep ? buffer_of(static_cast<char *>(a.pre) + first * pre_bytes, static_cast<unsigned int>(t.rows) * pre_bytes) : to;
    const auto pre_up = keep ? buffer_of(static_cast<char *>(a.pre) + first * pre_bytes + pre_up_at, static_cast<unsigned int>(t.rows) * pre_bytes - pre_up_at) : to;
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
    constexpr int kPlane = 16 * kChunks;
#pragma unroll
    for (int m = 0; m < TT; ++m) {
        const unsigned int row = static_cast<unsigned int>(q0 + m * 16);
        float xs = 0.0f;
        if constexpr (F::kI8) {
            if (static_cast<int>(row) + r < t.rows) xs = a.xs[first + row + r];
        }
        const auto sums = [&](int i) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = static_cast<float>(acc[m][i][e]);
                if constexpr (F::kI8) v[e] = v[e] * xs * ws[i][e];
            }
            return v;
        };
        if constexpr (kSplit) {
            if (keep && a.pre_f32) {
                // 16 bytes of one row per lane; a row's neighbours follow in the next store
#pragma unroll
                for (int i = 0; i < kOut; ++i) {
                    const int c = n0 + i * 16 + 4 * g;
                    const int at = static_cast<int>(c < a.cols ? (row + r) * pre_bytes + 4u * c : kPastEnd);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sums(i)), pre, at, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sums(i + kOut)), pre_up, at, 0, 0);
                }
            } else if (keep) {
#pragma unroll
                for (int i = 0; i < kOut; ++i) {
                    plane_put<kChunks>(mine, r, i, g, sums(i));
                    plane_put<kChunks>(mine + kPlane, r, i, g, sums(i + kOut));
                }
                wave_lds_fence();
                plane_store<kChunks>(mine, pre, pre_bytes, row, n0, a.cols);
                plane_store<kChunks>(mine + kPlane, pre_up, pre_bytes, row, n0, a.cols);
                wave_lds_fence();
            }
        }
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            f32x4 v = sums(i);
            if constexpr (kSplit) {
                const f32x4 u = sums(i + kOut);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = silu(v[e]) * u[e];
            }
            plane_put<kChunks>(mine, r, i, g, v);
        }
        wave_lds_fence();
        plane_store<kChunks>(mine, to, row_bytes, row, n0, a.cols);
        wave_lds_fence();
    }
}

// Waits until at most N of the wave's global loads, copies and stores are in
// flight.  They finish in order.
template <int N>
__device__ __forceinline__ void copies_arrived() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));   // vmcnt(N)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// The buffers of the two pairs.
struct Pairs {
    u32x4 *xa0, *xb0, *w0, *xa1, *xb1, *w1;
};

// One tile.  Its first pair and the first stage of its second have arrived; the next
// tile's are asked for when its own are.  Its pairs are taken two at a time: past
// the last one zeros are multiplied.  next_tile() makes `feed` the next tile's.
//
// The two waves of a SIMD take turns: while one group of four waves multiplies the
// other reads its operands of the next stage from LDS and asks for copies.  Each
// half step ends with a barrier of the workgroup; the second group begins half a
// step later.  Tiles of at most 64 rows have no second half of X and little to
// multiply: they take a pair at a time, every wave at once, with half the barriers.
template <int TT, int WT, Product KIND, bool GATED, typename NextTile, typename Ended>
__device__ __forceinline__ void run_tile(const ProductArgs &a, const ProductTile &t, Feed<KIND, GATED> &feed, int groups,
                                         const Pairs &lds, NextTile &&next_tile, Ended &&ended) {
    using F = Form<KIND>;
    constexpr int kAcross = kTileCols / (16 * WT);                  // waves across the channels
    constexpr bool kSplit = F::kForward && GATED;
    constexpr int kXT = TT < 4 ? TT : 4;                            // tiles of a half of X
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // what follows from it is made once per tile, not kept from tile to tile
    const int lane = tid & (kWave - 1);
    const int wave = uniform(tid / kWave);
    const bool second = wave >= kGemmWaves / 2;
    const int across = wave % kAcross, half = wave / kAcross, q0 = half * (16 * TT);
    const Reader<F::kXByK, 256> xr(half * 64, lane);
    const Reader<F::kWByK, 512> wr(across * 16 * WT, lane);
    Acc<F::kI8> acc[TT][WT];
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int i = 0; i < WT; ++i) acc[m][i] = Acc<F::kI8>{0, 0, 0, 0};
    u32x4 w[2][WT];
    // One stage: rows of the tiles m0 and on, from `x`.  settled: what the next stage
    // needs has arrived already.
    const auto stage = [&](const u32x4 *x_from, const u32x4 *w_from, auto m0_, bool settled, auto &&ask) {
        constexpr int m0 = decltype(m0_)::value;
        u32x4 x[2][kXT];
        if constexpr (m0 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < WT; ++i) w[h][i] = wr(w_from, h, i);
        }
        if constexpr (m0 < TT) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kXT; ++m) x[h][m] = xr(x_from, h, m);
        }
        ask();
        if (second && !settled) copies_arrived<kInFlight>();
        barrier_after<63>();
        if constexpr (m0 < TT) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kXT; ++m)
#pragma unroll
                    for (int i = 0; i < WT; ++i) acc[m0 + m][i] = multiply<F::kI8>(w[h][i], x[h][m], acc[m0 + m][i]);
            // a stage's products stay between their barriers
#pragma unroll
            for (int m = 0; m < kXT; ++m)
#pragma unroll
                for (int i = 0; i < WT; ++i) asm volatile("" : "+v"(acc[m0 + m][i]));
            __builtin_amdgcn_s_setprio(0);
        }
        if (!second && !settled) copies_arrived<kInFlight>();
        barrier_after<63>();
    };
    bool begun = false;
    if constexpr (TT <= 4) {
        const auto pair = [&](u32x4 *x_from, u32x4 *w_from, u32x4 *second_to, bool settled, bool last) {
            u32x4 x[2][kXT];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < WT; ++i) w[h][i] = wr(w_from, h, i);
#pragma unroll
                for (int m = 0; m < kXT; ++m) x[h][m] = xr(x_from, h, m);
            }
            barrier_after<63>();                                   // the pair is in registers
            feed.ask_second(a, second_to);
            if (last) next_tile();
            feed.ask_first(a, x_from, w_from);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < kXT; ++m)
#pragma unroll
                    for (int i = 0; i < WT; ++i) acc[m][i] = multiply<F::kI8>(w[h][i], x[h][m], acc[m][i]);
#pragma unroll
            for (int m = 0; m < kXT; ++m)
#pragma unroll
                for (int i = 0; i < WT; ++i) asm volatile("" : "+v"(acc[m][i]));
            if (!settled) copies_arrived<kInFlight>();
            barrier_after<63>();
        };
        do {
            pair(lds.xa0, lds.w0, lds.xb1, !begun, groups == 1);
            pair(lds.xa1, lds.w1, lds.xb0, false, false);
            begun = true;
        } while (--groups > 0);
        copies_arrived<0>();
        ended();
        finish<TT, WT, KIND, GATED>(a, t, acc, q0, t.c0 + across * (kSplit ? 8 : 16) * WT, lds.xb1 + wave * 128);
        return;
    }
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 4>;
    if (second) barrier_after<63>();
    do {
        stage(lds.xa0, lds.w0, First{}, !begun, [&]() { feed.ask_second(a, lds.xb1); });
        if (groups == 1) next_tile();
        stage(lds.xb0, lds.w0, Second{}, !begun, [&]() { feed.ask_first(a, lds.xa0, lds.w0); });
        stage(lds.xa1, lds.w1, First{}, false, [&]() { feed.ask_second(a, lds.xb0); });
        stage(lds.xb1, lds.w1, Second{}, false, [&]() { feed.ask_first(a, lds.xa1, lds.w1); });
        begun = true;
    } while (--groups > 0);
    if (!second) barrier_after<63>();
    copies_arrived<0>();
    ended();
    finish<TT, WT, KIND, GATED>(a, t, acc, q0, t.c0 + across * (kSplit ? 8 : 16) * WT, lds.xb1 + wave * 128);
}

template <Product KIND, bool GATED>
__global__ __launch_bounds__(kGemmThreads, 2) void k_product_tile(ProductArgs a, int tiles_c) {
    using F = Form<KIND>;
    constexpr bool kSplit = F::kForward && GATED;
    constexpr int kOutCols = kSplit ? kTileCols / 2 : kTileCols;
    constexpr bool kW = KIND == Product::kBackwardW;
    __shared__ u32x4 xa0[kHalfVecs], xb0[kHalfVecs], w0[kWVecs], xa1[kHalfVecs], xb1[kHalfVecs], w1[kWVecs];
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
    // What this workgroup takes in a round; nothing, then or later, where it has no rows.
    const auto tile_of = [&](int round) {
        ProductTile t{};                                           // rows 0: no tile
        const int left = min(items - round * kCus, kCus), run = (left + kXcds - 1) / kXcds, at = xcd * run + place;
        if (place >= run || at >= left) return t;
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
        t.rows = uniform(min(t.rows - skip, part_rows));
        t.row0 = uniform(t.row0 + skip);
        t.expert = uniform(t.expert);
        t.c0 = uniform(t.c0);
        if constexpr (kW) {
            t.first = uniform(t.first);
            t.end = uniform(t.end);
        }
        return t;
    };
    ProductTile t = tile_of(0);
    if (t.rows <= 0) return;                                       // the same for every wave
    const Pairs lds{xa0, xb0, w0, xa1, xb1, w1};
    Feed<KIND, GATED> feed;
    feed.start(a, t);
    feed.ask_first(a, xa0, w0);
    feed.ask_second(a, xb0);
    feed.ask_first(a, xa1, w1);
    ProductTile nt = tile_of(1);
    copies_arrived<0>();
    for (int round = 2;; ++round) {
        const int groups = max((pairs_of<KIND>(a, t) + 1) / 2, 1);
        const auto next_tile = [&]() { feed.start_or_stop(a, nt); };
        // the tile after the next one, before the stores, for which its search would wait
        ProductTile later{};
        const auto ended = [&]() { later = tile_of(round); };
        barrier_after<63>();                                       // every wave's copies are there, the last tile's results have left LDS
        if (t.rows > 128)
            run_tile<8, 4, KIND, GATED>(a, t, feed, groups, lds, next_tile, ended);
        else if (t.rows > 64)
            run_tile<8, 2, KIND, GATED>(a, t, feed, groups, lds, next_tile, ended);
        else if (t.rows > 32)
            run_tile<4, 2, KIND, GATED>(a, t, feed, groups, lds, next_tile, ended);
        else
            run_tile<2, 2, KIND, GATED>(a, t, feed, groups, lds, next_tile, ended);
        if (nt.rows <= 0) return;
        t = nt;
        nt = later;
    }
}

// ---------------------------------------------------------------------------
// forward products of short segments
// ---------------------------------------------------------------------------

// 16 token rows by 32 weight rows; the four waves split the channels and join
// their sums in LDS.  The weights' bytes are the work, each read once, so what
// counts is to keep many of them in flight and to ask for whole lines: a unit
// (128 bytes of k) of the 32 rows, 4 KB, is copied to the wave's own LDS in
// instructions of 8 whole lines while the unit before it is multiplied, four
// workgroups of four such waves per CU.  Tokens, few and shared by every workgroup
// of the segment, go straight to registers.  256 experts, 2048 x 7168 weights, four
// rows each: 1066 us, 7.0 TB/s of weights, what a plain read of such an array takes;
// in 8-bit integers 530.  One token's eight experts 34 us, from the Infinity Cache.
constexpr int kStreamRows = 16;
constexpr int kStreamWaves = 4;
constexpr int kWTiles = 2;                     // 16-row weight tiles (gated: a gate and an up tile)
constexpr int kUnitBytes = 128;                // of k: two steps
constexpr int kUnitVecs = kWTiles * 16 * 8;

template <Product KIND, bool GATED, bool ONCE>
__global__ __launch_bounds__(kStreamWaves * kWave, 4) void k_product_stream(ProductArgs a, int tiles_c) {
    using F = Form<KIND>;
    constexpr bool kI8 = F::kI8;
    constexpr int kOutTiles = GATED ? kWTiles / 2 : kWTiles;
    __shared__ u32x4 unit0[kStreamWaves][kUnitVecs], unit1[kStreamWaves][kUnitVecs];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
    RowTile t;
    if (!find_tile<kStreamRows>(a, blockIdx.x, tiles_c, t)) return;   // the same for every wave
    t.row0 = uniform(t.row0);
    t.rows = uniform(t.rows);
    t.expert = uniform(t.expert);
    t.ntile = uniform(t.ntile);
    const int n0 = t.ntile * (kOutTiles * 16);
    // lane = 16*g + r: row r of each operand, chunk g of a step
    const int r = lane & 15, g = lane >> 4;
    const unsigned int xb = static_cast<unsigned int>(a.inner) * F::kSize;
    const unsigned int wrows = min(kOutTiles * 16, a.cols - n0);      // past them zeros are read
    const char *const first = static_cast<const char *>(a.w) + (static_cast<size_t>(t.expert) * (GATED ? 2 : 1) * a.cols + n0) * xb;
    const auto w_gate = buffer_of(first, wrows * xb), w_up = buffer_of(first + (GATED ? static_cast<size_t>(a.cols) * xb : 0), wrows * xb);
    const auto xbuf = buffer_of(static_cast<const char *>(a.x) + static_cast<size_t>(t.row0) * xb, t.rows * xb);
    const int units = (xb + kUnitBytes - 1) / kUnitBytes;
    const int begin = units * wave / kStreamWaves, end = units * (wave + 1) / kStreamWaves;
    // Copies of 8 weight rows: lane l's vector is row l/8, chunk c at place l%8;
    // chunk c of row q lies at c ^ (q % 8).  Chunks past the row's end read zeros.
    const unsigned int chunk = lane_chunk(lane);
    const unsigned int wo = lane / 8 * xb + chunk;
    const auto copy_unit = [&](int u, u32x4 *to) {
        const int left = u < end ? static_cast<int>(xb) - u * kUnitBytes : 0, shared = shared_offset(u * kUnitBytes, left, wrows * xb);
        const unsigned int gone = past_row(left, lane);
#pragma unroll
        for (int j = 0; j < kWTiles * 2; ++j) {
            const int row = 8 * j;
            const bool is_up = row >= kOutTiles * 16;
            copy_to_lds<ONCE>(is_up ? w_up : w_gate, to + row * 8, (wo + (is_up ? row - kOutTiles * 16 : row) * xb) | gone, shared);
        }
    };
    Acc<kI8> acc[kWTiles];
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) acc[i] = Acc<kI8>{0, 0, 0, 0};
    struct Tokens {
        u32x4 x[2];
    };
    const unsigned int xo = r * xb + g * 16;
    const auto load_tokens = [&](int u) {
        Tokens v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned int at = static_cast<unsigned int>(u * kUnitBytes + h * 64);
            v.x[h] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, static_cast<int>(u >= end || at + g * 16 >= xb ? kPastEnd : xo), static_cast<int>(min(at, xb - 1)), 0);
        }
        return v;
    };
    const auto products = [&](const u32x4 *from, const Tokens &tok) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kWTiles; ++i) acc[i] = multiply<kI8>(from[(i * 16 + r) * 8 + ((h * 4 + g) ^ (r & 7))], tok.x[h], acc[i]);
        // the unit is read before anything is copied over it
#pragma unroll
        for (int i = 0; i < kWTiles; ++i) asm volatile("" : "+v"(acc[i]) : : "memory");
    };
    // Past the wave's last unit zeros are copied and multiplied: without branches the
    // loads in flight are counted.  Before a unit's products its copies are there:
    // in flight are the next one's four and its tokens' two loads.
    if (begin < end) {
        copy_unit(begin, unit0[wave]);
        Tokens now = load_tokens(begin);
        copy_unit(begin + 1, unit1[wave]);
        for (int u = begin; u < end; u += 2) {
            const Tokens next = load_tokens(u + 1);
            copies_arrived<kWTiles * 2 + 2>();
            products(unit0[wave], now);
            copy_unit(u + 2, unit0[wave]);
            now = load_tokens(u + 2);
            copies_arrived<kWTiles * 2 + 2>();
            products(unit1[wave], next);
            copy_unit(u + 3, unit1[wave]);
        }
        copies_arrived<0>();
    }
    // the sums meet where the weights were
    __syncthreads();
    Acc<kI8>(*const part)[kWTiles][kWave] = reinterpret_cast<Acc<kI8>(*)[kWTiles][kWave]>(&unit0[0][0]);
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < kOutTiles; i += kStreamWaves) {
        const int n = n0 + i * 16 + 4 * g;
        const bool mine = r < t.rows && n < a.cols;
        const size_t row = static_cast<size_t>(t.row0) + r;
        const auto sum = [&](int tile, int up) {
            Acc<kI8> v = part[0][tile][lane];
#pragma unroll
            for (int q = 1; q < kStreamWaves; ++q) v += part[q][tile][lane];
            f32x4 f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                f[c] = static_cast<float>(v[c]);
                if constexpr (kI8) {
                    if (mine) f[c] = f[c] * a.xs[row] * a.ws[(static_cast<size_t>(t.expert) * (GATED ? 2 : 1) + up) * a.cols + n + c];
                }
            }
            return f;
        };
        f32x4 v = sum(i, 0);
        if constexpr (GATED) {
            const f32x4 u = sum(kOutTiles + i, 1);
            if (!kI8 && a.pre != nullptr && mine) {
                const size_t at = row * 2 * a.cols + n;
                if (a.pre_f32) {
                    float *const pre = static_cast<float *>(a.pre) + at;
                    *reinterpret_cast<f32x4 *>(pre) = v;
                    *reinterpret_cast<f32x4 *>(pre + a.cols) = u;
                } else {
                    unsigned short *const pre = static_cast<unsigned short *>(a.pre) + at;
                    *reinterpret_cast<u32x2 *>(pre) = pack_bf16x4(v);
                    *reinterpret_cast<u32x2 *>(pre + a.cols) = pack_bf16x4(u);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * u[c];
        }
        if (mine) *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.out) + row * a.cols + n) = pack_bf16x4(v);
    }
}

// ---------------------------------------------------------------------------
// the rows' gradient of short segments
// ---------------------------------------------------------------------------

// The same for W's rows of k: 16 rows by 64 channels, a whole line of each of W's
// rows; a unit is 32 of those.  32-byte block b of row k lies at b ^ back_turn(k), so
// that the eight rows that half a wave's transposing read takes, 128 bytes apart,
// lie in eight different groups of banks.  A tile's workgroup walks all of k alone, in
// steps as long as a copy takes: with few rows there are too few of those for the
// chip (16 tokens, 16 experts, 2048 x 704: 25 us, here 9).  256 experts, 2048 x 7168
// weights, four rows each: 1164 us, 6.4 TB/s of weights.
constexpr int kBackTiles = 4;
constexpr int kBackCols = 16 * kBackTiles;
constexpr int kBackUnit = 32;                  // rows of k
static_assert(kBackUnit * 8 == kUnitVecs && kStreamWaves == kBackTiles, "a unit as long as the forward's; a wave joins a tile");
__device__ __forceinline__ int back_turn(int k) { return (k >> 1 & 1) | (k >> 2 & 2); }

template <bool GATED, bool ONCE>
__global__ __launch_bounds__(kStreamWaves * kWave, 4) void k_product_stream_back(ProductArgs a, int tiles_c) {
    __shared__ u32x4 unit0[kStreamWaves][kUnitVecs], unit1[kStreamWaves][kUnitVecs];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
    RowTile t;
    if (!find_tile<kStreamRows>(a, blockIdx.x, tiles_c, t)) return;   // the same for every wave
    t.row0 = uniform(t.row0);
    t.rows = uniform(t.rows);
    t.expert = uniform(t.expert);
    t.ntile = uniform(t.ntile);
    const int n0 = t.ntile * kBackCols;
    const int r = lane & 15, g = lane >> 4;
    const unsigned int xb = static_cast<unsigned int>(a.inner) * 2, cb = static_cast<unsigned int>(a.cols) * 2;
    const char *const first = static_cast<const char *>(a.w) + (static_cast<size_t>(t.expert) * a.inner * a.cols + n0) * 2;
    const unsigned int bytes = min(2u * kBackCols, cb - 2u * n0);
    const auto xbuf = buffer_of(static_cast<const char *>(a.x) + static_cast<size_t>(t.row0) * xb, t.rows * xb);
    const int units = (a.inner + kBackUnit - 1) / kBackUnit;
    const int begin = units * wave / kStreamWaves, end = units * (wave + 1) / kStreamWaves;
    // Copies of 8 rows of k: lane l's vector is of row l/8, place l%8.  Channels past the
    // last one read what follows them, and count for nothing.
    const unsigned int row = lane / 8 * cb, chunk = (((lane & 7) >> 1 ^ back_turn(lane / 8)) * 2 + (lane & 1)) * 16;
    const auto copy_unit = [&](int u, u32x4 *to) {
        const auto b = rows_of_k(first + static_cast<size_t>(u) * kBackUnit * cb, u < end ? min(a.inner - u * kBackUnit, kBackUnit) : 0, bytes, cb);
#pragma unroll
        for (int j = 0; j < kBackUnit / 8; ++j) copy_to_lds<ONCE>(b, to + j * 64, row + j * 8 * cb + (j & 1 ? chunk ^ 64u : chunk), 0);
    };
    f32x4 acc[kBackTiles];
#pragma unroll
    for (int i = 0; i < kBackTiles; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const unsigned int xo = r * xb + g * 16;
    const auto load_rows = [&](int u) {
        const unsigned int at = static_cast<unsigned int>(u) * kBackUnit * 2;
        return __builtin_amdgcn_raw_buffer_load_b128(xbuf, static_cast<int>(u >= end || at + g * 16 >= xb ? kPastEnd : xo), static_cast<int>(min(at, xb - 1)), 0);
    };
    // of tile i: rows 8g .. 8g+3 of k, then 8g+4 .. 8g+7
    const int k = 8 * g + r / 4;
    const unsigned int read = static_cast<unsigned int>(k * 128 + back_turn(k) * 32 + (r & 3) * 8);
    const auto products = [&](const u32x4 *from, u32x4 x) {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
#pragma unroll
        for (int i = 0; i < kBackTiles; ++i) {
            const char *const p = reinterpret_cast<const char *>(from) + (read ^ static_cast<unsigned int>(i * 32));
            const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
            const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 128)));
            acc[i] = multiply<false>(u32x4{lo[0], lo[1], hi[0], hi[1]}, x, acc[i]);
        }
        // the unit is read before anything is copied over it
#pragma unroll
        for (int i = 0; i < kBackTiles; ++i) asm volatile("" : "+v"(acc[i]) : : "memory");
    };
    // Past the wave's last unit zeros are copied and multiplied: without branches the
    // loads in flight are counted.  Before a unit's products its copies are there:
    // in flight are the next one's four and its row's load.
    if (begin < end) {
        copy_unit(begin, unit0[wave]);
        u32x4 now = load_rows(begin);
        copy_unit(begin + 1, unit1[wave]);
        for (int u = begin; u < end; u += 2) {
            const u32x4 next = load_rows(u + 1);
            copies_arrived<kBackUnit / 8 + 1>();
            products(unit0[wave], now);
            copy_unit(u + 2, unit0[wave]);
            now = load_rows(u + 2);
            copies_arrived<kBackUnit / 8 + 1>();
            products(unit1[wave], next);
            copy_unit(u + 3, unit1[wave]);
        }
        copies_arrived<0>();
    }
    // the sums meet where the weights were
    __syncthreads();
    f32x4(*const part)[kBackTiles][kWave] = reinterpret_cast<f32x4(*)[kBackTiles][kWave]>(&unit0[0][0]);
#pragma unroll
    for (int i = 0; i < kBackTiles; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    const int n = n0 + wave * 16 + 4 * g;
    if (r >= t.rows || n >= a.cols) return;
    f32x4 d = part[0][wave][lane];
#pragma unroll
    for (int q = 1; q < kStreamWaves; ++q) d += part[q][wave][lane];
    const size_t out_row = (static_cast<size_t>(t.row0) + r) * (GATED ? 2 : 1) * a.cols + n;
    unsigned short *const out = static_cast<unsigned short *>(a.out) + out_row;
    if constexpr (GATED) {
        f32x4 gate, up, dg, du;
        if (a.pre_f32) {
            const float *const pre = static_cast<const float *>(a.pre_in) + out_row;
            gate = *reinterpret_cast<const f32x4 *>(pre);
            up = *reinterpret_cast<const f32x4 *>(pre + a.cols);
        } else {
            const unsigned short *const pre = static_cast<const unsigned short *>(a.pre_in) + out_row;
            const u32x2 gw = *reinterpret_cast<const u32x2 *>(pre), uw = *reinterpret_cast<const u32x2 *>(pre + a.cols);
            gate = f32x4{bf16_lo(gw[0]), bf16_hi(gw[0]), bf16_lo(gw[1]), bf16_hi(gw[1])};
            up = f32x4{bf16_lo(uw[0]), bf16_hi(uw[0]), bf16_lo(uw[1]), bf16_hi(uw[1])};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x, y;
            gated_gradient(gate[e], up[e], d[e], x, y);
            dg[e] = x;
            du[e] = y;
        }
        *reinterpret_cast<u32x2 *>(out) = pack_bf16x4(dg);
        *reinterpret_cast<u32x2 *>(out + a.cols) = pack_bf16x4(du);
    } else {
        *reinterpret_cast<u32x2 *>(out) = pack_bf16x4(d);
    }
}

bool forward(const ProductArgs &a) { return a.kind == Product::kForward || a.kind == Product::kForwardI8; }

double weight_bytes(const ProductArgs &a) {
    return used_segments(a) * (a.gated && forward(a) ? 2.0 : 1.0) * a.cols * a.inner * (a.kind == Product::kForwardI8 ? 1.0 : 2.0);
}
// Weights that the Infinity Cache (256 MB) does not hold from call to call are
// read past the caches by the streaming kernel.
bool weights_once(const ProductArgs &a) { return weight_bytes(a) > 320.0e6; }

// The rule between the two kernels of a forward product, or of the rows' gradient: the
// sooner by these estimates, in microseconds.  Experts with a row: as many as a routing at random leaves with
// one.  Steps are of 64 bytes of k.
//   stream: a start of 4 us; a workgroup's work is one 16-row tile by 32 weight
//     rows (gradient: 64 channels), 3300 steps of such (1650) a microsecond, or the
//     weights at 7.0 TB/s.
//   tile: a start of 6 us, then rounds of 256 workgroups one tile each, 0.38 us a
//     step and 0.0018 more for each row of a tile, or of a part of it in the last
//     round; or the weights at 5.5 TB/s.
// Measured, stream / tile (us; E experts with m rows each, M weight rows; bf16):
//   E=256 H=7168 M=2048  m=4 1066 / 1351  m=16 1664 / 1370
//   E=256 H=1024 M=7168  m=4 561 / 642    E=256 H=2048 M=1536 m=16 356 / 354
//   E=64  H=2048 M=2816  m=6 107 / 171    m=24 205 / 172
//   E=8   H=7168 M=2048  m=2 30 / 87      m=8 34 / 88     m=32 55 / 97
//   E=4   H=7168 M=512   m=32 17 / 95     m=128 33 / 97
// The gradient of K channels with respect to H (m as a mean, routed at random):
//   E=256 K=7168 H=1024  m=4 603 / 565    K=2048 H=7168 m=4 1164 / 1225
//   E=64  K=2048 H=1408  m=6 60 / 76      m=24 127 / 82
//   E=64  K=2816 H=2048  m=6 127 / 123    m=24 231 / 126
//   E=16  K=512  H=264   m=32 9 / 13      K=528 H=512 m=32 7.6 / 12
//   E=16  K=2048 H=704   m=2 9 / 25       K=1024 H=704 m=64 14 / 20
//   E=8   K=7168 H=2048  m=4 38 / 70      K=4096 H=7168 m=4 95 / 83
//   E=4   K=4096 H=512   m=32 11 / 49     m=128 20 / 49
// Three of these it streams where tiles are sooner, by 7, 3 and 14 %: E=256 K=7168,
// E=64 K=2816 m=6 and E=8 K=4096.  The gradient streams weights at 4.9 to 6.4 TB/s, the
// estimate's 7.0 is the forward's.
// The weights' gradient has tiles alone.  A tile walks all of its expert's rows: of few
// experts with small weights there are too few for the chip (one expert, 65536 rows,
// 512 x 512: 815 us, 2048 x 1408: 972; eight experts of 8192 rows: 107 and, 1024 x 2048, 247).
bool long_segments(const ProductArgs &a) {
    const bool back = a.kind == Product::kBackwardX;
    if (a.kind == Product::kBackwardW) return true;
    if (a.entries == 0) return false;
    // a grid of tiles can always be numbered
    if (back && most_tiles(a, kStreamRows) * ((a.cols + kBackCols - 1) / kBackCols) > 1 << 20) return true;
    const double rows = static_cast<double>(a.entries), used = used_segments(a), weights = weight_bytes(a);
    const double M = a.gated && !back ? 2.0 * a.cols : a.cols, steps = a.inner * (a.kind == Product::kForwardI8 ? 1.0 : 2.0) / 64;
    const double stream_tiles = std::max(used, rows / kStreamRows + used / 2), row_tiles = std::max(used, rows / kTileRows + used / 2);
    const double stream = 4 + std::max(stream_tiles * (M / (16 * kWTiles)) * steps / 3300, weights / 7.0e6);
    const double tiles = row_tiles * std::ceil(M / kTileCols), whole = std::floor(tiles / kCus), rest = tiles - whole * kCus;
    const double last_rows = rest * 4 <= kCus ? kTileRows / 4 : (rest * 2 <= kCus ? kTileRows / 2 : kTileRows);
    const auto step_us = [](double tile_rows) { return 0.38 + 0.0018 * tile_rows; };
    const double tile_rows = std::min(rows / used, static_cast<double>(kTileRows));
    const double rounds_us = whole * step_us(tile_rows) + (rest > 0 ? step_us(std::min(tile_rows, last_rows)) : 0);
    return 6 + std::max(steps * rounds_us, weights / 5.5e6) < stream;
}

struct Grid {
    int tiles_c;
    int64_t tiles;     // at most
    int64_t blocks;
};
Grid grid_of(const ProductArgs &a) {
    const bool tiles = long_segments(a), split = a.gated && forward(a);
    const int cols = tiles ? kTileCols : (a.kind == Product::kBackwardX ? kBackCols : kWTiles * 16), out = split ? cols / 2 : cols;
    Grid g;
    g.tiles_c = (a.cols + out - 1) / out;
    const int64_t rows = a.kind == Product::kBackwardW ? static_cast<int64_t>(a.E) * ((a.inner + kTileRows - 1) / kTileRows)
                                                       : most_tiles(a, tiles ? kTileRows : kStreamRows);
    g.tiles = (rows * g.tiles_c + kXcds - 1) / kXcds * kXcds;
    g.blocks = tiles ? std::min<int64_t>(4 * g.tiles, kCus) : g.tiles;   // a tile may be taken in four parts
    return g;
}

}  // namespace

bool product_grid_ok(const ProductArgs &a) {
    const Grid g = grid_of(a);
    return g.tiles <= INT32_MAX - kCus && g.blocks * std::max(kStreamWaves * kWave, kGemmThreads) <= kMaxLaunchThreads;
}

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
    const Grid g = grid_of(a);
    if (g.blocks == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(g.blocks)), tile_block(kGemmThreads), stream_block(kStreamWaves * kWave);
    const bool tiles = long_segments(a), once = weights_once(a);
#define MOE_TILE(KIND, GATED) hipLaunchKernelGGL((k_product_tile<Product::KIND, GATED>), grid, tile_block, 0, s, a, g.tiles_c)
#define MOE_FORWARD(KIND, GATED)                                                                                              \
    do {                                                                                                                      \
        if (tiles)                                                                                                            \
            MOE_TILE(KIND, GATED);                                                                                            \
        else if (once)                                                                                                        \
            hipLaunchKernelGGL((k_product_stream<Product::KIND, GATED, true>), grid, stream_block, 0, s, a, g.tiles_c);       \
        else                                                                                                                  \
            hipLaunchKernelGGL((k_product_stream<Product::KIND, GATED, false>), grid, stream_block, 0, s, a, g.tiles_c);      \
    } while (0)
#define MOE_BACK(GATED)                                                                                                       \
    do {                                                                                                                      \
        if (tiles)                                                                                                            \
            MOE_TILE(kBackwardX, GATED);                                                                                      \
        else if (once)                                                                                                        \
            hipLaunchKernelGGL((k_product_stream_back<GATED, true>), grid, stream_block, 0, s, a, g.tiles_c);                 \
        else                                                                                                                  \
            hipLaunchKernelGGL((k_product_stream_back<GATED, false>), grid, stream_block, 0, s, a, g.tiles_c);                \
    } while (0)
    switch (a.kind) {
        case Product::kForward: if (a.gated) MOE_FORWARD(kForward, true); else MOE_FORWARD(kForward, false); break;
        case Product::kForwardI8: if (a.gated) MOE_FORWARD(kForwardI8, true); else MOE_FORWARD(kForwardI8, false); break;
        case Product::kBackwardX: if (a.gated) MOE_BACK(true); else MOE_BACK(false); break;
        case Product::kBackwardW: MOE_TILE(kBackwardW, false); break;
    }
#undef MOE_BACK
#undef MOE_FORWARD
#undef MOE_TILE
    return hipGetLastError();
}

}  // namespace moe
