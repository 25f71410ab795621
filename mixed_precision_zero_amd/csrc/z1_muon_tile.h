// z1_muon_tile.h -- which of Muon's kernels a list of matrices runs on, chosen
// on the host from the sizes alone: one workgroup's, or products of which tile
// side, split along their depth or not.  Plain C++, so that a test can ask
// without a GPU.  Not installed.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

namespace z1 {
namespace ops {

inline int64_t pad_to(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// A matrix is small when a workgroup of 8 waves holds all of its iteration:
// sides padded to 32, at most 4 blocks of 32 x 32 a wave, and X, X^T, A and B
// in LDS with rows 16 bytes longer than their data (so that consecutive rows
// start on other banks).
constexpr int kSmallLds = 160 * 1024 - 256;
inline bool muon_small(int64_t mp, int64_t np)
{
    return mp * np <= 32 * 1024 &&
           2 * (mp * (np + 8) + np * (mp + 8) + 2 * mp * (mp + 8)) <= kSmallLds;
}

// The tile side a product runs with (0: X X^T, 1: A A, 2: B X): the one with
// the smallest estimate of its time,
//   fixed + panels * (time of a 32-deep panel)   microseconds,
// where r = ceil(tiles / 256) tiles fall to the busiest compute unit and a
// panel takes 0.1 r for tiles of 64, max(0.43, 0.36 r - 0.3) for 128 (which
// overlap two or three to a unit) and 0.68, or 0.88 r from two on, for 256
// (one to a unit).  Measured (64 / 128 / 256, us): whole calls 2 x 333 x 1537
// 130 / 238 / 493, 4 x 1024^2 249 / 298 / 523, 1 x 2048^2 388 / 441 / 777,
// 24 x 2048^2 7936 / 6364 / 5551; single products of 2 x 2048 x 8192
// (128 / 256) 112 / 157, 34 / 53 and 207 / 181, of 4 x 2048^2 62 / 62, 63 / 65
// and 113 / 87, of 4096 x 11008 245 / 250, 99 / 104 and 472 / 401.
// passes: how often each panel is read, 3 for the wide products.
inline int pick_tile(int product, int32_t n, const int64_t *rows, const int64_t *cols, int passes = 1)
{
    static const struct {
        int side;
        double fixed;
    } kTiles[3] = {{64, 3.0}, {128, 6.0}, {256, 13.0}};
    int tile = 64;
    double best = 0.0;
    for (const auto &c : kTiles) {
        double tiles = 0.0, work = 0.0;
        for (int32_t i = 0; i < n; ++i) {
            const double m = (double)pad_to(std::min(rows[i], cols[i]), c.side);
            const double w = (double)pad_to(std::max(rows[i], cols[i]), c.side);
            const double q = m / c.side;
            const double t = product == 2 ? q * (w / c.side) : q * (q + 1) / 2;
            tiles += t;
            work += t * (product == 0 ? w : m) / 32 * passes;
        }
        if (n == 0)
            break;
        const double r = ceil(tiles / 256.0);
        const double panel = c.side == 64 ? 0.1 * r
                             : c.side == 128 ? std::max(0.43, 0.36 * r - 0.3)
                                             : (r > 1.0 ? 0.88 * r : 0.68);
        const double cost = c.fixed + work / tiles * panel;
        if (c.side == 64 || cost < best) {
            best = cost;
            tile = c.side;
        }
    }
    return tile;
}

// In how many pieces of its depth X X^T is computed, `tiles` tiles of side
// `tile` and at least `panels` panels of 32 deep (1: whole).  Few tiles leave
// most of the GPU idle while a few compute units read long panels: at least 16
// panels a piece, where what is saved is more than the join's 3 us
// (512 x 8192: 290 -> 189 us, 333 x 1537: 108 -> 103).
inline int32_t gram_splits(int tile, int64_t tiles, int64_t panels)
{
    if (tile != 64 || tiles == 0 || tiles > 128 || panels < 48)
        return 1;
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>(256 / tiles, panels / 16));
}

}  // namespace ops
}  // namespace z1
