// Sanitizer driver for the tile choice of the MXFP4 products (mx_tiles.hpp):
// every problem the header promises to run has a tile whose grid a launch
// holds, at the borders of the limits too, and ordinary problems take the tile
// their time asks for.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../block_scaled_fp4_gemm_amd/csrc/mx_tiles.hpp"

using namespace bg;

static const char* what = "";
static uint32_t m, n, k, e;

#define CHECK(cond)                                                                                           \
    do {                                                                                                      \
        if (!(cond)) {                                                                                        \
            std::fprintf(stderr, "%s:%d: check failed: %s (%s %ux%ux%u, %u experts)\n", __FILE__, __LINE__, #cond, what, m, n, k, e); \
            std::exit(1);                                                                                     \
        }                                                                                                     \
    } while (0)

static uint64_t ceil_div(uint64_t a, uint64_t b) { return a / b + (a % b != 0); }

int main() {
    const uint32_t sides[] = {1, 31, 32, 33, 64, 100, 128, 129, 255, 256, 257, 1000, 65535, 65536, 1u << 20, (1u << 22) + 1, 1u << 23,
                              (1u << 24) - 1, 1u << 28, (1u << 29) - 1, 1u << 29, (1u << 29) + 5, 1u << 30, (1u << 30) + 1, 0x7FFFFF00u, 0x7FFFFFFFu};
    const uint32_t depths[] = {0, 32, 480, 512, 544, 768, 1024, 1u << 24};
    const uint32_t experts[] = {1, 2, 3, 63, 64, 256, 1023, 1024};
    unsigned long long dense = 0, grouped = 0, refused = 0;
    for (uint32_t M : sides)
        for (uint32_t N : sides)
            for (uint32_t K : depths) {
                m = M, n = N, k = K, e = 1, what = "dense";
                const bool runs = mx_dense_launches(M, N, K);
                if (ceil_div(M, 256) * ceil_div(N, 256) < (1u << 23)) CHECK(runs);
                for (uint32_t cus : {1u, 256u, 304u}) {
                    const int i = mx_dense_tile(M, N, K, cus);
                    CHECK((i >= 0) == runs && i < MX_DENSE_TILES);
                    if (i < 0) continue;
                    const uint64_t tiles = ceil_div(M, kMxDense[i].bm) * ceil_div(N, kMxDense[i].bn);
                    const uint64_t threads = K % 256 == 0 && K >= 512 ? kMxDense[i].whole : kMxDense[i].other;
                    CHECK(tiles < (uint64_t)1 << 31);
                    CHECK(tiles * threads <= 0xFFFFFFFFull);
                }
                runs ? ++dense : ++refused;
                for (uint32_t E : experts) {
                    e = E, what = "grouped";
                    const int i = mx_grouped_tile(M, N, K, E);
                    CHECK(i < MX_GROUPED_TILES);
                    if ((M / 128 + (uint64_t)(E < M ? E : M) + 7) * ceil_div(N, 128) < (1u << 23)) CHECK(i >= 0);
                    if (i < 0) {
                        ++refused;
                        continue;
                    }
                    const MxTile& t = kMxGrouped[i];
                    const uint64_t tiles_m = mx_tiles_m_grouped(t, M, E);
                    // at least the tiles of any split of the rows over the experts, in eight equal stretches
                    CHECK(tiles_m % 8 == 0 && tiles_m >= M / t.bm + (uint64_t)(E < M ? E : M));
                    CHECK(tiles_m * ceil_div(N, t.bn) * (K % 256 == 0 && K >= 512 ? t.whole : t.other) <= 0xFFFFFFFFull);
                    ++grouped;
                }
            }
    // sizes of everyday use are far from the limits and keep their tiles
    what = "choice";
    CHECK(mx_dense_tile(4096, 4096, 8192, 256) == MX_256x256);
    CHECK(mx_dense_tile(5120, 11008, 2048, 256) == MX_128x128);
    CHECK(mx_dense_tile(128, 7168, 16384, 256) == MX_64x64);
    CHECK(mx_dense_tile(0x7FFFFFFFu, 0x7FFFFFFFu, 32, 256) == -1);
    CHECK(mx_dense_tile((1u << 29), 64, 32, 256) >= 0);
    CHECK(mx_grouped_tile(128, 2048, 2048, 256) == MX_G32x128);
    CHECK(mx_grouped_tile(256 * 16, 1024, 2048, 256) == MX_G64x128);
    CHECK(mx_grouped_tile(36080, 1024, 2048, 256) == MX_G128x128);
    CHECK(mx_grouped_tile(1u << 24, 4096, 2048, 256) == MX_G128x128);
    std::printf("mx_tiles sanitizer driver: ok, %llu dense, %llu grouped, %llu refused\n", dense, grouped, refused);
    return 0;
}
