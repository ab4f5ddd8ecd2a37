// Tiles of the gated MLP block's products and of the transposed ones, and the
// choice between them. Plain host code, shared by the argument checks, the
// workspace queries, the launchers and the CPU tests.
#pragma once

#include <stdint.h>

namespace bg {

// us: per tile; per step of 64 with few tiles on the chip, with one on every
// compute unit, and, where two fit a unit's LDS, the tile and the step of a pair
// (0: one workgroup fills it). Medians over the three products, 32 to 1024 tiles
// and K 512 to 6144; the sum is within 10% of most of them, and 15% above the
// largest gated products (444 us for 5120 x 11008 x 2048, which takes 386).
struct GatedTileInfo {
    int bm, bn, threads;
    double fixed, few, full, pair_fixed, pair;
};
enum GatedTile : int { GT_256x256, GT_160x256, GT_256x128, GT_128x128, GT_128x128_DEEP, GT_64x128, GT_MIXED, GT_TILES };
constexpr GatedTileInfo kGatedTiles[GT_TILES] = {{256, 256, 512, 9.0, 1.25, 1.72, 0, 0},
                                                 {160, 256, 256, 7.5, 0.80, 1.20, 0, 0},
                                                 {256, 128, 512, 5.7, 0.68, 1.04, 0, 0},
                                                 {128, 128, 256, 4.0, 0.70, 0.78, 5.0, 1.02},
                                                 {128, 128, 512, 4.8, 0.41, 0.58, 0, 0},
                                                 {64, 128, 256, 4.4, 0.48, 0.52, 4.6, 0.69},
                                                 // 256 x 256 tiles, the last columns in 256 x 128: counted as the latter
                                                 {256, 128, 512, 0, 0, 0, 0, 0}};

// Rows that do not start at multiples of 16 bytes: 128 x 128 tiles, every step
// loaded through registers with checks.
constexpr GatedTileInfo kGuarded = {128, 128, 256, 4.0, 5.0, 5.5, 5.0, 6.5};

// Output columns of a tile of bn operand rows: a gated tile holds both products.
constexpr int tile_columns(int bn, bool gated) { return gated ? bn / 2 : bn; }

// Direct loads: rows `ld` elements apart start at multiples of 16 bytes, and a
// tile's rows lie within 32-bit offsets.
inline bool gated_direct(uint32_t ld) { return ld % 8 == 0 && (uint64_t)ld * 512 < ((uint64_t)1 << 31); }

struct GatedPlan {
    int tile, splits;
    uint32_t wide = 0;      // GT_MIXED: columns of 256 x 256 tiles
};

inline uint64_t gated_ceil(uint64_t n, uint64_t by) { return (n + by - 1) / by; }

inline uint64_t gated_tiles(int tile, bool gated, uint32_t M, uint32_t N, uint32_t outputs) {
    const GatedTileInfo& t = kGatedTiles[tile];
    return gated_ceil(M, t.bm) * gated_ceil(N, tile_columns(t.bn, gated)) * outputs;
}

// A launch holds fewer than 2^32 threads.
inline bool gated_launches(const GatedPlan& p, bool gated, uint32_t M, uint32_t N, uint32_t outputs) {
    return gated_tiles(p.tile, gated, M, N, outputs) * p.splits * kGatedTiles[p.tile].threads < ((uint64_t)1 << 32);
}

// The tile that every problem may fall back to, and whether a launch holds it:
// 256 x 256, or kGuarded's without direct loads (both bounds then).
constexpr int gated_last_tile(bool direct) { return direct ? GT_256x256 : GT_128x128; }
inline bool gated_fits(bool direct, bool gated, uint32_t M, uint32_t N, uint32_t outputs) {
    return gated_launches(GatedPlan{GT_256x256, 1}, gated, M, N, outputs) &&
           gated_launches(GatedPlan{gated_last_tile(direct), 1}, gated, M, N, outputs);
}

// n tiles of `steps` steps in rounds over the compute units.
inline double gated_us(const GatedTileInfo& t, uint64_t n, double steps, uint32_t cus) {
    const uint64_t slots = t.pair > 0 ? 2 * (uint64_t)cus : cus;
    const double round = t.pair > 0 ? t.pair_fixed + steps * t.pair : t.fixed + steps * t.full;
    const uint64_t rest = n % slots;
    double us = (double)(n / slots) * round;
    if (rest > cus)
        us += round;
    else if (rest != 0)
        us += t.fixed + steps * (t.few + (t.full - t.few) * (double)rest / cus);
    return us;
}

// GT_MIXED: whole rounds of 256 x 256 tiles (`fewer`: one less than there are); the
// columns that are left go in 256 x 128 tiles, first on the units that the last
// round leaves free. It saves most of a round that 256 x 256 tiles alone would
// fill to less than a half: 5120 x 11008 x 2048 as nn (860 of them, 3.4 rounds)
// 226 us, in 256 x 256 alone 241, in 256 x 128 alone 249; 2048 x 11008 x 5120 as
// tn (344, 1.3 rounds) 229, 264, 258 us; 12152 x 2672 x 5736 as tn, where one round
// less pays because the columns do not divide the rounds, 365, 445, 397 (all in one
// run; cards and clocks differ by 10%).
inline uint32_t mixed_columns(bool gated, uint32_t M, uint32_t N, uint32_t outputs, uint32_t cus, bool fewer) {
    const uint64_t column = gated_ceil(M, 256) * outputs, all = gated_ceil(N, tile_columns(256, gated));
    const uint64_t rounds = column * all / cus;
    if (rounds < (fewer ? 2 : 1)) return 0;
    return (uint32_t)((rounds - (fewer ? 1 : 0)) * cus / column);
}
inline double mixed_us(bool gated, uint32_t M, uint32_t N, double steps, uint32_t outputs, uint32_t cus, uint32_t wide) {
    const GatedTileInfo &w = kGatedTiles[GT_256x256], &t = kGatedTiles[GT_256x128];
    const uint64_t column = gated_ceil(M, 256) * outputs, done = (uint64_t)wide * tile_columns(256, gated);
    const uint64_t wides = column * wide, narrow = column * (done < N ? gated_ceil(N - done, tile_columns(128, gated)) : 0);
    const double round = w.fixed + steps * w.full;
    const uint64_t last = wides % cus, free = last ? cus - last : 0;      // of the last round
    double us = (double)gated_ceil(wides, cus) * round;
    const uint64_t beside = free * (uint64_t)(round / (t.fixed + steps * t.full));
    return us + (narrow > beside ? gated_us(t, narrow - beside, steps, cus) : 0.0);
}

// The planes of a split reduction: written by the product and read by their sum
// (at about 4 bytes a ps), and the second launch.
inline double planes_us(uint32_t M, uint32_t N, uint32_t outputs, int splits) {
    return splits == 1 ? 0.0 : 4.0 + (double)M * N * outputs * splits * 8e-6 / 4.0;
}

constexpr int kMaxSplits = 16;

// The tile, and the number of parts of the reduction (products without a
// workspace: one), whose time by the table is least. Without direct loads there is
// one tile (kGuarded, GT_128x128 by name). `forced` >= 0: tile forced % 16 and forced / 16 parts.
inline GatedPlan plan_of(bool gated, bool tn, bool direct, uint32_t M, uint32_t N, uint32_t steps, uint32_t outputs, uint32_t cus,
                         int forced, double* time = nullptr) {
    const int most = steps < 2 ? 1 : steps < (uint32_t)kMaxSplits ? (int)steps : kMaxSplits;
    const GatedPlan last{gated_last_tile(direct), 1};
    auto ok = [&](const GatedPlan& p) {
        return !(tn && p.tile == GT_160x256) && ((p.tile == last.tile && p.splits == 1) || gated_launches(p, gated, M, N, outputs));
    };
    if (forced >= 0) {
        GatedPlan p{direct && forced % 16 < GT_TILES ? forced % 16 : last.tile, 1};
        if (!gated && forced >= 16) p.splits = forced / 16 < most ? forced / 16 : most;
        if (p.tile == GT_MIXED) p.splits = 1, p.wide = (uint32_t)(gated_ceil(N, tile_columns(256, gated)) / 2);
        return ok(p) ? p : last;
    }
    GatedPlan best = last;
    double least = -1;
    for (int tile = direct ? 0 : GT_128x128; tile < (direct ? (int)GT_MIXED : GT_128x128 + 1); ++tile) {
        const GatedTileInfo& info = direct ? kGatedTiles[tile] : kGuarded;
        const uint64_t n = gated_tiles(tile, gated, M, N, outputs);
        for (int splits = 1; splits <= (gated ? 1 : most); ++splits) {
            // parts of less than four steps, or parts that no unit waits for, gain nothing
            if (splits > 1 && (steps / splits < (direct ? 4 : 1) || n * (splits - 1) >= 2 * (uint64_t)cus)) break;
            const GatedPlan p{tile, splits};
            if (!ok(p)) continue;
            const double us = gated_us(info, n * splits, (double)gated_ceil(steps ? steps : 1, splits), cus) +
                              planes_us(M, N, outputs, splits);
            if (least < 0 || us < least) best = p, least = us;
        }
    }
    for (int fewer = 0; direct && fewer < 2; ++fewer) {
        const GatedPlan p{GT_MIXED, 1, mixed_columns(gated, M, N, outputs, cus, fewer != 0)};
        if (p.wide == 0 || !ok(p)) continue;
        const double us = mixed_us(gated, M, N, steps ? steps : 1, outputs, cus, p.wide);
        if (us < least) best = p, least = us;
    }
    if (time != nullptr) *time = least;
    return best;
}

// Operands of a product whose rows do not start at multiples of 16 bytes are copied
// to rows that do, where the copy (elements read and written, one launch) and the
// product with direct loads take less than the product with guarded ones: 5120 x
// 11007 x 2048 as nn 250 us instead of 712, 2047 x 11007 x 5120 as tn 291 (1736),
// 64 x 2047 x 5461 29 (53), 1 x 11007 x 2048 32 (36), 512 x 513 x 1024 14.2 (15.7);
// but 300 x 301 x 303 14.8 (12.3 - 14), 30 x 1001 x 100 11.7 (9.6).
inline double aligned_copy_us(uint64_t elements) { return 4.0 + (double)elements * 4e-6 / 4.8; }

// An nn and a tn product in one launch of GT_128x128_DEEP tiles, where all their
// workgroups run at once: the parts of each whose longer time is least, with the
// us; splits 0 where they do not fit. m, n, steps, outputs: of each product.
struct PairPlan {
    int nn, tn;
    double us;
};
inline PairPlan pair_plan(const uint32_t (&m)[2], const uint32_t (&n)[2], const uint32_t (&steps)[2], const uint32_t (&outputs)[2],
                          uint32_t stacked, uint32_t cus) {
    const GatedTileInfo& t = kGatedTiles[GT_128x128_DEEP];
    uint64_t tiles[2];
    for (int i = 0; i < 2; ++i) tiles[i] = gated_tiles(GT_128x128_DEEP, false, m[i], n[i], outputs[i]);
    PairPlan best{0, 0, 0};
    for (uint32_t a = 1; a <= (uint32_t)kMaxSplits && tiles[0] * a < cus; ++a) {
        if (a > 1 && steps[0] / a < 4) break;
        for (uint32_t b = 1; b <= (uint32_t)kMaxSplits && tiles[0] * a + tiles[1] * b <= cus; ++b) {
            if (b > 1 && steps[1] / b < 4) break;
            const double sa = (double)gated_ceil(steps[0] ? steps[0] : 1, a), sb = (double)gated_ceil(steps[1] ? steps[1] : 1, b);
            const double us = t.fixed + t.full * (sa > sb ? sa : sb) +
                              (a > 1 || stacked > 1 ? planes_us(m[0], n[0], outputs[0], (int)a + 1) : 0.0) +
                              planes_us(m[1], n[1], outputs[1], (int)b);
            if (best.nn == 0 || us < best.us) best = PairPlan{(int)a, (int)b, us};
        }
    }
    return best;
}

}  // namespace bg
