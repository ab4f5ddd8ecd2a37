// Tiles of the gated MLP block's products and of the transposed ones, and the
// choice between them. Plain host code, shared by the argument checks, the
// workspace queries, the launchers and the CPU tests.
#pragma once

#include <stdint.h>

namespace bg {

enum GatedTile : int { GT_256x256, GT_160x256, GT_256x128, GT_128x256, GT_128x128, GT_128x128_3, GT_64x128, GT_TILES };
struct GatedTileSize {
    int bm, bn, threads;
};
constexpr GatedTileSize kGatedTiles[GT_TILES] = {{256, 256, 512}, {160, 256, 256}, {256, 128, 512}, {128, 256, 512},
                                                     {128, 128, 256}, {128, 128, 256}, {64, 128, 256}};

// Output columns of a tile of bn operand rows: a gated tile holds both products.
constexpr int tile_columns(int bn, bool gated) { return gated ? bn / 2 : bn; }

struct GatedPlan {
    int tile, splits;
};

inline uint64_t gated_ceil(uint64_t n, uint64_t by) { return (n + by - 1) / by; }

inline uint64_t gated_tiles(int tile, bool gated, uint32_t M, uint32_t N, uint32_t outputs) {
    const GatedTileSize& t = kGatedTiles[tile];
    return gated_ceil(M, t.bm) * gated_ceil(N, tile_columns(t.bn, gated)) * outputs;
}

// A launch holds fewer than 2^32 threads.
inline bool gated_launches(const GatedPlan& p, bool gated, uint32_t M, uint32_t N, uint32_t outputs) {
    return gated_tiles(p.tile, gated, M, N, outputs) * p.splits * kGatedTiles[p.tile].threads < ((uint64_t)1 << 32);
}

inline GatedPlan plan_of(bool gated, uint32_t M, uint32_t N, uint32_t steps, uint32_t outputs, uint32_t cus, int forced) {
    GatedPlan p{GT_256x256, 1};
    if (forced >= 0) {
        p.tile = forced % 16 < GT_TILES ? forced % 16 : GT_256x256;
        if (!gated && forced >= 16) p.splits = forced / 16;
    } else {
        if (gated_tiles(GT_256x256, gated, M, N, outputs) < cus) p.tile = M <= 64 ? GT_64x128 : GT_128x128;
        if (!gated) {
            const uint64_t n = gated_tiles(p.tile, gated, M, N, outputs);
            while (n * p.splits * 2 <= 2 * cus && p.splits < 16 && steps / (p.splits * 2) >= 4) p.splits *= 2;
        }
    }
    if (p.splits > (int)steps) p.splits = steps > 1 ? (int)steps : 1;
    return p;
}

}  // namespace bg
