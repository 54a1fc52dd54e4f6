// Where the long-segment kernel's copies to LDS read: offsets into a buffer that
// starts at the tile's first weight row or token row and ends behind its last.
//
// A copy instruction reads 8 rows of 128 bytes: lane l takes row l/8, and chunk c
// (16 bytes) of row q at place c ^ (q % 8).  A lane's own offset says which row
// and which chunk; the offset that all lanes share is the stage's place inside a
// row, so it is smaller than any buffer.
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

}  // namespace moe
