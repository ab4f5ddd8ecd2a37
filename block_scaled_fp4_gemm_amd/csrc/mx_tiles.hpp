// Tiles of the MXFP4 products: the grid each one takes and the choice between
// them. Plain host code, shared by the argument checks, the launcher and the
// CPU tests.
#pragma once

#include <stdint.h>

namespace bg {

struct MxTile {
    int bm, bn;
    int whole, other;              // threads of a workgroup where K is whole steps of 256, and otherwise
    double fixed, alone, paired;   // dense: us per tile, and per step of 256 K elements alone on a compute unit
                                   // and as one of two (0: one workgroup fills a compute unit's LDS)
};

// Dense products, largest first; times fitted to 20 shapes from 32 x 4096 x
// 7168 to 4096 x 4096 x 8192, most within 10%.
enum MxDenseTile : int { MX_256x256, MX_256x128, MX_128x128, MX_64x64, MX_32x64, MX_DENSE_TILES };
constexpr MxTile kMxDense[MX_DENSE_TILES] = {{256, 256, 512, 256, 3.5, 2.15, 0},
                                             {256, 128, 512, 512, 3.2, 1.13, 0},
                                             {128, 128, 512, 256, 2.0, 0.61, 1.22},
                                             {64, 64, 256, 256, 1.5, 0.28, 0.47},
                                             {32, 64, 128, 128, 1.5, 0.23, 0.4}};

// Grouped products, smallest first.
enum MxGroupedTile : int { MX_G32x128, MX_G64x128, MX_G128x128, MX_GROUPED_TILES };
constexpr MxTile kMxGrouped[MX_GROUPED_TILES] = {{32, 128, 256, 256, 0, 0, 0},
                                                 {64, 128, 256, 256, 0, 0, 0},
                                                 {128, 128, 512, 256, 0, 0, 0}};

inline uint64_t mx_ceil(uint64_t n, uint64_t by) { return (n + by - 1) / by; }

// Tile rows of a grid. Grouped: every expert may end in a partly filled tile,
// and the XCDs take eight stretches of at least as many tiles as exist.
inline uint64_t mx_tiles_m(const MxTile& t, uint32_t M) { return mx_ceil(M, t.bm); }
inline uint64_t mx_tiles_m_grouped(const MxTile& t, uint32_t M, uint32_t E) {
    return mx_ceil((uint64_t)M / t.bm + (E < M ? E : M), 8) * 8;
}

// A launch holds fewer than 2^32 threads.
inline bool mx_launches(const MxTile& t, uint64_t tiles_m, uint32_t N, uint32_t K) {
    const uint64_t threads = K >= 512 && K % 256 == 0 ? t.whole : t.other;
    return tiles_m * mx_ceil(N, t.bn) * threads < ((uint64_t)1 << 32);
}

// Whether a launch holds the grid of any tile.
inline bool mx_dense_launches(uint32_t M, uint32_t N, uint32_t K) {
    for (const MxTile& t : kMxDense)
        if (mx_launches(t, mx_tiles_m(t, M), N, K)) return true;
    return false;
}

// Of the tiles whose grid a launch holds, the one whose time, counted in
// rounds over `cus` compute units, is least; -1 where none does.
inline int mx_dense_tile(uint32_t M, uint32_t N, uint32_t K, uint32_t cus) {
    const double steps = (double)mx_ceil(K, 256);
    int best = -1;
    double least = 0;
    for (int i = 0; i < MX_DENSE_TILES; ++i) {
        const MxTile& c = kMxDense[i];
        const uint64_t tiles_m = mx_tiles_m(c, M), n = tiles_m * mx_ceil(N, c.bn), cu = cus;
        if (!mx_launches(c, tiles_m, N, K)) continue;
        double t;
        if (c.paired == 0) {
            t = (double)mx_ceil(n, cu) * (c.fixed + steps * c.alone);
        } else {
            const uint64_t rest = n % (2 * cu);
            t = (double)(n / (2 * cu)) * (c.fixed + steps * c.paired);
            if (rest != 0) t += c.fixed + steps * (rest <= cu ? c.alone : c.paired);
        }
        if (best < 0 || t < least) best = i, least = t;
    }
    return best;
}

// By the rows an expert has on average. 256 experts of unequal load, N 1024, K
// 2048, us with 32 x 128, 64 x 128 and 128 x 128 tiles: 4 rows 54, 54, 60; 16 rows
// 59, 61, 68; 32 rows 68, 67, 72; 64 rows 95, 81, 80; 141 rows 158, 127, 107. N
// 2048: 4 rows 105, 106, 120; 32 rows 133, 130, 140; 64 rows 179, 156, 151. A
// larger tile where a launch does not hold that one's grid; -1 where none does.
inline int mx_grouped_tile(uint32_t M, uint32_t N, uint32_t K, uint32_t E) {
    const uint64_t mean = M / E;
    int i = mean < 16 ? MX_G32x128 : mean < 64 ? MX_G64x128 : MX_G128x128;
    while (i < MX_GROUPED_TILES && !mx_launches(kMxGrouped[i], mx_tiles_m_grouped(kMxGrouped[i], M, E), N, K)) ++i;
    return i < MX_GROUPED_TILES ? i : -1;
}

}  // namespace bg
