// Host side of the product: which shape of the kernel a product takes.
#include "mhcm_internal.h"

namespace mhcpb {
namespace product {

namespace {
// A constant, not the GPU's: the split of a sum decides its order.
constexpr int64_t kBlocks = 152;

int64_t tiles_of(const Shape& s, int64_t tile_m, int64_t tile_n, int* m_tiles, int* n_tiles) {
    if (s.mode == kSideBySide) tile_n /= 2;
    const int64_t m = (s.M + tile_m - 1) / tile_m, n = (s.N + tile_n - 1) / tile_n;
    *m_tiles = (int)m;
    *n_tiles = (int)n;
    return s.mode == kSymmetric ? n * (n + 1) / 2 : m * n * (s.mode == kGroups ? 2 : 1);
}
}  // namespace

Choice choose(const Shape& s) {
    Choice c{};
    const int64_t pairs = tiles_of(s, 256, 256, &c.m_tiles, &c.n_tiles);
    if (s.M > 128 && pairs >= kBlocks / 4) {
        c.pair = true;
        c.split = 1;
        c.tiles = (int)pairs;
        c.grid = (int)(2 * (pairs < kBlocks / 2 ? pairs : kBlocks / 2));
        return c;
    }
    const int64_t tiles = tiles_of(s, 128, 128, &c.m_tiles, &c.n_tiles);
    const int64_t steps = (int64_t)s.k_steps * (s.mode == kLongK ? 2 : 1);
    c.tiles = (int)tiles;
    c.split = 1;
    while (c.split < 8 && tiles * c.split * 2 <= kBlocks && steps / (2 * c.split) >= 4) c.split *= 2;
    c.grid = c.tiles * c.split;
    return c;
}

}  // namespace product
}  // namespace mhcpb
