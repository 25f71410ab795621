// z1_linear_tile.h -- on which tiles a product of z1_linear or z1_linear_grad runs,
// and in how many pieces of its depth: chosen on the host from sizes and type alone.
// Plain C++, so that a test can ask without a GPU.  Not installed.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

namespace z1 {
namespace ops {

struct TileChoice {
    int32_t tile;     // 64, 128 or 256; 0: none that can be launched
    int32_t splits;   // pieces of the depth
    int32_t piece;    // bytes of depth each of them takes, a multiple of 128
};

constexpr int64_t kMostGroups = (INT64_C(1) << 24) - 1;   // of a launch: 2^32 - 1 threads, 256 each

// The choice with the smallest estimate of its time in microseconds, for a product of
// P x Q elements and `bytes` of depth, fp32 or 16-bit.  With t workgroups to each of 256
// compute units, r = ceil(t) rounds where one takes a unit alone, and n panels of 128
// bytes a workgroup:
//   64    3.9 + 0.55 t + n max(0.14 + 0.08 t, 0.175 t)      up to three share a unit
//   128   2.5 + r (4.3 + n (t < 1 ? 0.33 + 0.15 t : 0.48))
//   256   r (14 + 1.45 n)
// and for s pieces a join of 4 + 8 s P Q / 4e6.  A panel of fp32 takes max(0.54, 0.5 t)
// and 1.95 r instead, and there are no 256 tiles of it.  Measured (64 / 128 / 256, us,
// bf16 forward): 2048^3 29 / 22 / 52, 1024 x 4096 -> 4096 55 / 37 / 83, 2048 x 576 -> 1536
// 9.2 / 11.3 / 29, 1000^3 7.5 / 12.6 / 35, 4096^3 197 / 150 / 117; fp32 1000^3 23 / 67,
// 2048^3 140 / 140.
//
// Only what a launch can hold is chosen from (a shallow product of 2^29 rows has 2^24
// tiles of 64 for 128 outputs), with pieces of less than 2^31 bytes.
inline TileChoice pick_product(int64_t P, int64_t Q, int64_t bytes, bool fp32)
{
    TileChoice best{0, 0, 0};
    double least = 0.0;
    const int64_t panels = std::max<int64_t>(1, (bytes + 127) / 128);
    for (const int side : {64, 128, 256}) {
        if (fp32 && side == 256)
            continue;
        const int64_t tiles = ((P + side - 1) / side) * ((Q + side - 1) / side);
        for (int64_t s = 1; s <= 64 && s <= panels; s = s < 4 ? s + 1 : s + s / 2) {
            if (tiles * s > kMostGroups || (s > 1 && (panels / s < 4 || tiles * s > 1024)))
                break;
            const int64_t piece = (panels + s - 1) / s;
            if (piece * 128 > INT32_MAX)
                continue;
            const double n = (double)piece, t = (double)(tiles * s) / 256.0, r = ceil(t);
            double cost;
            if (side == 64)
                cost = 3.9 + 0.55 * t + n * (fp32 ? std::max(0.54, 0.5 * t) : std::max(0.14 + 0.08 * t, 0.175 * t));
            else if (side == 128)
                cost = 2.5 + r * (4.3 + n * (fp32 ? 1.95 : t < 1.0 ? 0.33 + 0.15 * t : 0.48));
            else
                cost = r * (14.0 + 1.45 * n);
            if (s > 1)
                cost += 4.0 + 8e-6 * (double)s * (double)P * (double)Q / 4.0;
            if (least == 0.0 || cost < least) {
                least = cost;
                best = TileChoice{side, (int32_t)((panels + piece - 1) / piece), (int32_t)(piece * 128)};
            }
        }
    }
    return best;
}

}  // namespace ops
}  // namespace z1
