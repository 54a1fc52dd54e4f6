// Every offset of the long-segment product kernel's copies, checked on the host.
// A buffer of B bytes answers a read at lane + uniform with zeros where
// lane >= B - uniform; what it does where uniform > B is nowhere written, so no
// copy may get there.  A copy that is not past the end has to read the whole
// chunk it is for, inside its row.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "tile_copies.h"

using namespace moe;

static long checked = 0;

static void check(CopyAt at, unsigned int records, int rows, int half, int row, unsigned int chunk, int s, int H, const char *what) {
    const long steps = (H + 127) / 128;
    const bool wanted = row < rows && 2 * s + static_cast<int>(chunk >= 64) < steps;
    const long uniform = at.uniform;
    const char *wrong = nullptr;
    if (uniform < 0 || uniform >= static_cast<long>(records)) {
        wrong = "the shared offset is not inside the buffer";
    } else {
        const bool reads = at.lane < records - static_cast<unsigned int>(uniform);
        const long byte = static_cast<long>(at.lane) + uniform;
        if (reads != wanted)
            wrong = reads ? "reads what it should not" : "does not read its chunk";
        else if (reads && byte != static_cast<long>(row) * half + s * 128 + chunk)
            wrong = "reads another chunk";
        else if (reads && byte + 16 > static_cast<long>(records))
            wrong = "passes the buffer's end";
    }
    ++checked;
    if (wrong != nullptr) {
        std::printf("%s: %s (rows %d of %d bytes, row %d, chunk byte %u, stage %d, H %d)\n", what, wrong, rows, half, row, chunk, s, H);
        std::exit(1);
    }
}

int main() {
    const int channels[] = {128, 256, 384, 640, 2048, 7168, 1 << 22};
    const int lengths[] = {1, 2, 7, 8, 9, 16, 31, 33, 64, 65, 104, 127, 128, 129, 200, 255, 256};
    for (int H : channels) {
        const int half = H / 2, stages = (H + 255) / 256;
        for (int s : {0, 1, stages / 2, stages - 2, stages - 1}) {
            if (s < 0 || s >= stages) continue;
            for (int rows : lengths) {
                for (int wave = 0; wave < kTileWaves; ++wave) {
                    for (int lane = 0; lane < 64; ++lane) {
                        const unsigned int chunk = lane_chunk(lane), gone = left_out(H, s, lane);
                        const unsigned int records = static_cast<unsigned int>(rows) * half;
                        const unsigned int xo = first_token(wave, lane) * static_cast<unsigned int>(half) + chunk;
                        for (int i = 0; i < 4; ++i)
                            check(copy_at(xo, token_step(i), half, s, gone), records, rows, half, wave * 8 + i * 64 + lane / 8, chunk, s, H,
                                  "tokens");
                        if (rows % 8 != 0) continue;   // weight rows come in eights
                        for (int swiglu = 0; swiglu < 2; ++swiglu) {
                            for (int wide = 0; wide < 2; ++wide) {
                                if (swiglu && rows > 128) continue;
                                const unsigned int wo = first_weight(swiglu, wide, wave, lane) * static_cast<unsigned int>(half) + chunk;
                                for (int i = 0; i < 2; ++i)
                                    for (int j = 0; j < 2; ++j) {
                                        // the tile's own order: 16 rows of gate then 16 of up (or 32 and 32)
                                        const int at = wave * 32 + i * 16 + j * 8 + lane / 8;
                                        const int row = !swiglu ? at : (wide ? at / 64 * 32 + at % 32 : at / 32 * 16 + at % 16);
                                        check(copy_at(wo, weight_step(swiglu, wide, i, j), half, s, gone), records, rows, half, row, chunk, s, H,
                                              swiglu ? "gate or up rows" : "weight rows");
                                    }
                            }
                        }
                    }
                }
            }
        }
    }
    std::printf("%ld copies\n", checked);
    return 0;
}
