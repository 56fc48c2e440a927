// gdn_tiles.h - which tile and how many parts of K a gdn_linear_act call takes: host code alone, which a test compiles as well.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace gdn {

constexpr int kStepBytes = 128;  // of a row's K that a step of a tile takes

// The tile shapes, as launch_of has them.
enum Tile { kShort6, kShort4, k32x64, k64x64, k64x128, k128x128Deep, k128x128, k256x256 };
struct Choice {
    int tile, splits;
};

// A launch's tile and the parts of K, by what is expected of them.  Measured on products of 1 to 8191 rows, 5120 to 27648
// columns and K of 4096 to 13824 in the three types, in us:
// - Up to 64 rows the product is a stream of w.  The smallest tile that holds the rows spreads it over the most workgroups:
//   16 rows by 64 columns (16 x 5120 -> 12352 bf16: 26.7, with 32 rows 30.3), 32 by 64 (32 rows: 30.6, with 32 by 128 43.5),
//   64 by 64.  Six buffered tiles where workgroups are few (26.7 against 27.6 with four), four where there are more than 512
//   (16 x 512 -> 65536: 16.7 against 20.1).  Below 160 tiles K is cut into parts of at least 16 steps (1 x 13824 -> 5120 e4m3:
//   19 against 42; above, the join costs more than it gives: 193 tiles in two parts 32.4 against 26.7).
// - Beyond that a tile's step takes about `step` us with one workgroup to a CU, and `more` for each further 256 tiles; the join
//   reads what the parts write.  256 x 256 has the fewest bytes per flop and wins where its tiles fill whole rounds of
//   256 CUs (1024 x 5120 -> 2 x 13824 e4m3, 432 tiles: 153 against 196 with 128 x 128), 128 x 128 two to a CU in between
//   (4096 x 5120 -> 5120 bf16: 258 against 279), its three-buffer form where there is only one to a CU
//   (256 x 5120 -> 12352: 63 against 85), 64 x 128 and 64 x 64 below; parts of K where even those leave CUs idle
//   (1024 x 13824 -> 5120 i8, 80 tiles of 256 x 256: three parts 108, one 186; 128 x 128 in one part 125).
inline Choice choose_tile(int64_t M, int64_t N, int64_t K, int elem_bytes, bool gated)
{
    const int64_t steps = (K * elem_bytes + kStepBytes - 1) / kStepBytes, rows = gated ? 2 * N : N;
    if (M <= 64) {
        const int64_t tiles = (rows + 63) / 64;
        const int64_t most = M <= 32 ? 240 : 480;  // workgroups that splitting aims at
        const int splits = tiles >= 160 ? 1 : (int)std::max<int64_t>(1, std::min(steps / 16, (most + tiles - 1) / tiles));
        return {M > 32 ? k64x64 : M > 16 ? k32x64 : tiles > 512 ? kShort4 : kShort6, splits};
    }
    struct {
        int tile, bm, bn;
        double step, more;
        bool rounds;  // whole rounds of one workgroup to a CU
    } const shapes[] = {{k256x256, 256, 256, 1.8, 1.8, true}, {k128x128, 128, 128, 1.0, 0.62, false}, {k128x128Deep, 128, 128, 0.7, 0.7, true},
                        {k64x128, 64, 128, 0.5, 0.5, false}, {k64x64, 64, 64, 0.18, 0.4, false}};
    Choice best{k256x256, 1};
    double least = 1e30;
    for (const auto &t : shapes)
        for (int splits : {1, 2, 3, 4, 6, 8}) {
            if (splits > 1 && steps / splits < 8) break;
            const double tiles = (double)((M + t.bm - 1) / t.bm) * ((rows + t.bn - 1) / t.bn) * splits / 256;
            const double at_once = t.rounds ? t.step * std::ceil(tiles) : std::max(t.step, t.more * tiles);
            double us = at_once * (double)((steps + splits - 1) / splits);
            if (splits > 1) us += 5 + (double)splits * M * rows * 8 / 4e6;
            if (us < least) {
                least = us;
                best = {t.tile, splits};
            }
        }
    return best;
}

}  // namespace gdn
