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
    int32_t tile;     // 64, 128 or 256
    int32_t splits;   // pieces of the depth
    int32_t piece;    // bytes of depth each of them takes, a multiple of 128
};

// The choice with the smallest estimate of its time in microseconds, for a product of
// P x Q elements and `bytes` of depth, fp32 or 16-bit.  With r = ceil(workgroups / 256)
// rounds and n panels of 128 bytes a workgroup:
//   64    4 + 0.55 r + n max(0.26, 0.2 r)     several workgroups share a compute unit
//   128   2.5 + r (4.3 + 0.46 n)
//   256   r (14 + 1.45 n)
// and for s pieces a join of 4 + 8 s P Q / 4e6.  fp32 products take 0.45 and 1.75 a
// panel and round instead, and have no 256 tiles.  Measured (64 / 128 / 256, us, bf16
// forward): 2048^3 32 / 21.5 / 48, 1024 x 4096 -> 4096 60 / 36 / 81, 2048 x 576 -> 1536
// 9.0 / 10.2 / 24, 4096^3 206 / 153 / 115, 16384 x 64 -> 4096 50 / 77 / 59.
inline TileChoice pick_product(int64_t P, int64_t Q, int64_t bytes, bool fp32)
{
    TileChoice best{64, 1, 128};
    double least = 0.0;
    const int64_t panels = std::max<int64_t>(1, (bytes + 127) / 128);
    for (const int side : {64, 128, 256}) {
        if (fp32 && side == 256)
            continue;
        const int64_t tiles = ((P + side - 1) / side) * ((Q + side - 1) / side);
        for (int64_t s = 1; s <= 64 && s <= panels; s = s < 4 ? s + 1 : s + s / 2) {
            if (s > 1 && (panels / s < 4 || tiles * s > 1024))
                break;
            const double n = (double)((panels + s - 1) / s), r = ceil((double)(tiles * s) / 256.0);
            double cost;
            if (side == 64)
                cost = 4.0 + 0.55 * r + n * std::max(fp32 ? 0.5 : 0.26, (fp32 ? 0.45 : 0.2) * r);
            else if (side == 128)
                cost = 2.5 + r * (4.3 + (fp32 ? 1.75 : 0.46) * n);
            else
                cost = r * (14.0 + 1.45 * n);
            if (s > 1)
                cost += 4.0 + 8e-6 * (double)s * (double)P * (double)Q / 4.0;
            if (least == 0.0 || cost < least) {
                least = cost;
                const int64_t piece = (panels + s - 1) / s;
                best = TileChoice{side, (int32_t)((panels + piece - 1) / piece), (int32_t)(piece * 128)};
            }
        }
    }
    return best;
}

}  // namespace ops
}  // namespace z1
