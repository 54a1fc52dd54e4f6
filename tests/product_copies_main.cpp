// Every offset of the bf16 and 8-bit products' copies that name a shared offset, checked on
// the host: tiles of all lengths and widths, every pair of stages from the first to those
// asked for behind the rows' ends, and where no tile comes next.
//
// A buffer of B bytes answers a read at lane + shared with zeros where lane >= B - shared;
// what it does where shared > B is nowhere written, so a shared offset lies inside its
// buffer or is 0.  A copy that is not past the end has to read the whole chunk it is for.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "tile_copies.h"

using namespace moe;

static long checked = 0;

struct Place {
    const char *what;
    int rows, row, at, row_bytes, wave, lane;
};

static void check(unsigned int lane_offset, int shared, unsigned int records, unsigned int row_in_buffer, unsigned int chunk, const Place &p) {
    const bool wanted = p.row < p.rows && p.at + static_cast<int>(chunk) < p.row_bytes;
    const char *wrong = nullptr;
    if (shared < 0 || (shared > 0 && static_cast<unsigned int>(shared) >= records)) {
        wrong = "the shared offset is not inside the buffer";
    } else {
        const bool reads = lane_offset < records - static_cast<unsigned int>(shared);
        const long byte = static_cast<long>(lane_offset) + shared;
        if (reads != wanted)
            wrong = reads ? "reads what it should not" : "does not read its chunk";
        else if (reads && byte != static_cast<long>(row_in_buffer) * p.row_bytes + p.at + chunk)
            wrong = "reads another chunk";
        else if (reads && byte + 16 > static_cast<long>(records))
            wrong = "passes the buffer's end";
    }
    ++checked;
    if (wrong != nullptr) {
        std::printf("%s: %s (row %d of %d, %d bytes a row, byte %d, chunk byte %u, wave %d, lane %d)\n", p.what, wrong, p.row, p.rows,
                    p.row_bytes, p.at, chunk, p.wave, p.lane);
        std::exit(1);
    }
}

// One wave's copies of one pair: 256 rows q, then the 256 weight rows, of which the tile holds `rows` and `wrows`.
static void tile_pair(int row_bytes, int at, int rows, int wrows, bool gated, int wave, int lane) {
    const int left = rows > 0 ? row_bytes - at : 0;
    const unsigned int xb = static_cast<unsigned int>(row_bytes), chunk = lane_chunk(lane), past = past_row(left, lane);
    const unsigned int x_bytes = static_cast<unsigned int>(rows) * xb, xo = (wave * 8 + lane / 8) * xb + chunk;
    for (int half = 0; half < 2; ++half)
        for (int j = 0; j < 2; ++j) {
            const int step = j * 128 + half * 64, row = wave * 8 + step + lane / 8;
            check((xo + step * xb) | past, shared_offset(at, left, x_bytes), x_bytes, row, chunk, Place{"rows q", rows, row, at, row_bytes, wave, lane});
        }
    const bool wide = rows > 128;
    const unsigned int wo = lane / 8 * xb + chunk;
    for (int i = 0; i < 2; ++i) {
        const WeightRows w = weight_rows(gated, wide, wave, i);
        // the tile's own order: gated, 32 gate rows then their 32 up rows (16 and 16 for at most 128 rows q)
        const int place = wave * 32 + i * 16, part = wide ? 32 : 16;
        const int first = !gated ? place : place / (2 * part) * part + place % part;
        const bool up = gated && place / part % 2;
        const unsigned int bytes = bytes_from(w.first, wrows, xb);
        if (w.first != first || w.up != up) {
            std::printf("weight rows %d, not %d (wave %d, half %d)\n", w.first, first, wave, i);
            std::exit(1);
        }
        for (int j = 0; j < 2; ++j) {
            const int in = j * 8 + lane / 8;
            check((wo + j * 8 * xb) | past, shared_offset(at, left, bytes), bytes, in, chunk,
                  Place{w.up ? "up rows" : "weight rows", rows > 0 ? wrows : 0, w.first + in, at, row_bytes, wave, lane});
        }
    }
}

// One wave's copies of one unit of the streaming kernel: 32 weight rows, or 16 gate rows and 16 up rows.
static void stream_unit(int row_bytes, int u, int end, int wrows, bool gated, int lane) {
    const unsigned int xb = static_cast<unsigned int>(row_bytes), chunk = lane_chunk(lane), bytes = wrows * xb;
    const int left = u < end ? row_bytes - u * 128 : 0;
    for (int j = 0; j < 4; ++j) {
        const int row = (gated ? 8 * j % 16 : 8 * j) + lane / 8;
        const Place p{"streamed rows", u < end ? wrows : 0, row, u * 128, row_bytes, 0, lane};
        check((lane / 8 * xb + chunk + (row - lane / 8) * xb) | past_row(left, lane), shared_offset(u * 128, left, bytes), bytes, row, chunk, p);
    }
}

int main() {
    const int widths[] = {16, 48, 112, 128, 144, 256, 528, 1152, 4096, 14336, 1 << 23};   // bytes of a row
    for (int row_bytes : widths) {
        const int pairs = (row_bytes + 127) / 128, taken = (pairs + 1) / 2 * 2;
        for (int pair : {0, 1, 2, pairs / 2, pairs - 2, pairs - 1, pairs, pairs + 1, taken, taken + 1, taken + 2}) {
            if (pair < 0) continue;
            const int at = pair * 128;
            for (int rows : {0, 1, 7, 8, 31, 33, 64, 65, 128, 129, 200, 255, 256})
                for (int wrows : {8, 16, 24, 40, 104, 120, 128, 136, 232, 248, 256})
                    for (int gated = 0; gated < 2; ++gated) {
                        if (gated && wrows > 128) continue;
                        for (int wave = 0; wave < kTileWaves; ++wave)
                            for (int lane = 0; lane < 64; ++lane) tile_pair(row_bytes, at, rows, wrows, gated, wave, lane);
                    }
        }
        for (int wave = 0; wave < 4; ++wave) {
            const int begin = pairs * wave / 4, end = pairs * (wave + 1) / 4;
            for (int u : {begin, begin + 1, end - 2, end - 1, end, end + 1, end + 2})
                for (int wrows : {8, 16, 24, 32})
                    for (int gated = 0; gated < 2; ++gated)
                        if (u >= begin && (!gated || wrows <= 16))
                            for (int lane = 0; lane < 64; ++lane) stream_unit(row_bytes, u, end, wrows, gated, lane);
        }
    }
    std::printf("%ld copies\n", checked);
    return 0;
}
