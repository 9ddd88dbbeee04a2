// qsdp_plan.h -- how the tiled products with coded weights are cut up.  Host code alone.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace onebit {

constexpr int kTileDepth = 64;  // of a step

// How a product is cut up: its tiles and how many workgroups share the depth of each.
struct TilePlan {
    int shape;
    int64_t tiles_m, tiles_n;
    int splits;
};

constexpr int kMostSplits = 16;

// Bytes of partial results at most: as many parts of the result, in whole tiles, but not more than 64 MB.
inline int64_t partial_room(int64_t tokens, int64_t width) {
    const int64_t m = tokens > 128 ? (tokens + 255) / 256 * 256 : (tokens + 63) / 64 * 64;
    const int64_t n = width > 256 ? (width + 255) / 256 * 256 : (width + 127) / 128 * 128;
    return std::min(m * n * 4 * kMostSplits, int64_t{1} << 26);
}

// Results of a workgroup, groups of waves that share its depth, and what a step takes (us), linear and
// gradient.
struct PlannedShape {
    int tm, tn, groups;
    float step[2];
};
constexpr PlannedShape kPlannedShapes[4] = {
    {256, 256, 1, {2.4f, 2.4f}}, {128, 128, 2, {1.55f, 1.9f}}, {64, 128, 2, {1.25f, 1.4f}}, {64, 64, 4, {1.6f, 1.8f}}};

// The cheapest by this estimate (us): a workgroup is alone on its compute unit, so there are as many rounds of
// workgroups as 256 (the whole GPU's units) go into them, of so many steps each.  The steps' times above are
// those of an earlier state of the kernels; what a step takes now, of whole calls in bf16 with 4 / 8 bits:
//   first shape   linear 2.2 / 2.1 (2048 x 16384 x 4096: 277 / 266 us in 2 x 64 steps), gradient 2.2 / 2.1 (4096 x
//                 1600 x 6400, 2 workgroups a tile: 121 / 118 in 50 and a join of 13) and 2.4 / 2.3 (500 x 1600
//                 x 50257, 16 of them: 134 / 124 in 50 and a join of 12)
//   second shape  linear 1.7 (1000 x 4096 x 4096: 56 in 32), gradient 1.7 / 1.6 (4096 x 1600 x 6400: 166 / 157 in 2 x 50)
//   third shape   linear 1.3 (512 x 4096 x 4096: 41 in 32; 333 x 4800 x 1600: 17 in 13), gradient 1.5 / 1.4 (512 x
//                 4096 x 4096: 46 / 44 in 32)
//   fourth shape  linear 1.6 (512 x 4096 x 4096: 50 in 2 x 16), gradient 1.9 (the same: 62 / 60)
// Choices up to 14% from the best one are known (787 x 7392 x 4551: 116 against 101.5 us).  Sharing a tile's depth
// costs a second launch and the partial results' way to memory and back: 2.5 us and 3 us for every 8 MB.
inline TilePlan tile_plan(int64_t tokens, int64_t width, int64_t depth, bool grad) {
    const int64_t steps = (depth + kTileDepth - 1) / kTileDepth;
    const int64_t room = partial_room(tokens, width);
    TilePlan best{};
    float least = 0.0f;
    for (int i = 0; i < 4; ++i) {
        const PlannedShape &p = kPlannedShapes[i];
        const int64_t m = (tokens + p.tm - 1) / p.tm, n = (width + p.tn - 1) / p.tn;
        for (int s = 1; s <= kMostSplits && s <= steps; s = s < 4 ? s + 1 : s < 8 ? s + 2 : s + 4) {
            if (s > 1 && m * n * s * p.tm * p.tn * 4 > room) break;
            const int64_t rounds = (m * n * s + 255) / 256;
            const int64_t each = ((steps + s - 1) / s + p.groups - 1) / p.groups;
            const float cost = (float)(rounds * each) * p.step[grad] +
                               (s > 1 ? 2.5f + (float)(s * tokens * width) * (4.0f * 3.0f / 8e6f) : 0.0f);
            if (least == 0.0f || cost < least) {
                least = cost;
                best = {i, m, n, s};
            }
        }
    }
    return best;
}

}  // namespace onebit
