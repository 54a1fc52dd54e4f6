// Where the products' copies to LDS read: offsets into a buffer that starts at the
// tile's first weight row or token row and ends behind its last.
//
// A copy instruction reads 8 rows of 128 bytes: lane l takes row l/8, and chunk c
// (16 bytes) of row q at place c ^ (q % 8).  A lane's own offset says which row
// and which chunk; the offset that all lanes share is the stage's place inside a
// row, so it is smaller than any buffer that holds a row; where a buffer holds none,
// or a copy lies behind the rows' ends, it is 0.
#pragma once

namespace moe {

constexpr unsigned int kPastEnd = ~0u - 15u;   // of every buffer
constexpr int kTileWaves = 8;
constexpr int kStageBytes = 128;               // of a row: 256 channels

struct CopyAt {
    unsigned int lane;
    int uniform;
};

// This lane's chunk of its row of eight.
__device__ __forceinline__ unsigned int lane_chunk(int lane) { return static_cast<unsigned int>((lane & 7) ^ (lane / 8)) * 16; }

// This lane's first weight row.  Weight row j of a tile belongs to wave j/64
// (wide: more than 128 token rows) or j/32 and is row j%16 of its 16-row tile;
// with SWIGLU the second half of a wave's tiles are the up rows of the first.
// Wave w copies rows 32*w .. 32*w+31.
__device__ __forceinline__ int first_weight(bool swiglu, bool wide, int wave, int lane) {
    return (swiglu ? (wide ? wave / 2 * 32 : wave * 16) : wave * 32) + lane / 8;
}
// What weight copy j of half i of the wave's 32 rows adds to it.
__device__ __forceinline__ int weight_step(bool swiglu, bool wide, int i, int j) { return swiglu && !wide ? 8 * j : 16 * i + 8 * j; }

// The same for token rows; copy i.
__device__ __forceinline__ int first_token(int wave, int lane) { return wave * 8 + lane / 8; }
__device__ __forceinline__ int token_step(int i) { return i * kTileWaves * 8; }

// kPastEnd for the lanes that a last stage of 128 channels leaves out: the second
// half of each row.
__device__ __forceinline__ unsigned int left_out(int H, int s, int lane) {
    return 256 * s + 128 >= H && (((lane & 7) ^ (lane / 8)) & 4) ? kPastEnd : 0u;
}

// Copy `step` rows behind the lane's first (at `first`) of stage s.
__device__ __forceinline__ CopyAt copy_at(unsigned int first, int step, int half, int s, unsigned int gone) {
    return CopyAt{(first + static_cast<unsigned int>(step) * half) | gone, s * kStageBytes};
}

// The products on bf16 and 8-bit integer rows take 128 bytes of every row at a time
// and go on past the rows' ends, where zeros are to be read.

// The offset that all lanes share, `at` bytes into the rows: 0 where nothing is
// left of them or the buffer is empty.
__device__ __forceinline__ int shared_offset(int at, int left, unsigned int buffer_bytes) {
    return left > 0 && buffer_bytes > 0 ? at : 0;
}

// kPastEnd for the lanes whose chunk lies behind the `left` bytes of a row.
__device__ __forceinline__ unsigned int past_row(int left, int lane) { return static_cast<int>(lane_chunk(lane)) >= left ? kPastEnd : 0u; }

// The 16 weight rows that half i of a wave's copies of 32 takes, of the tile's gate
// (or only) rows or of its up rows.  Gated, the second half of the rows that one
// wave multiplies (64, or 32 for at most 128 rows q: not wide) are the up rows of the first.
struct WeightRows {
    int first;
    bool up;
};
__device__ __forceinline__ WeightRows weight_rows(bool gated, bool wide, int wave, int i) {
    if (!gated) return WeightRows{wave * 32 + 16 * i, false};
    return wide ? WeightRows{(wave >> 1) * 32 + 16 * i, (wave & 1) != 0} : WeightRows{wave * 16, i != 0};
}

// Bytes of a buffer over the rows from `first` to the last of `rows`.
__device__ __forceinline__ unsigned int bytes_from(int first, int rows, unsigned int row_bytes) {
    return first < rows ? static_cast<unsigned int>(rows - first) * row_bytes : 0u;
}

}  // namespace moe
