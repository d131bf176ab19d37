// Host side of the product: which shape of the kernel a product takes.
#include "mhcm_internal.h"

namespace mhcpb {
namespace product {

namespace {

// A constant, not the GPU's: the split of a sum decides its order.
constexpr int64_t kSms = 152;

int64_t over(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t tiles_of(const Shape& s, int64_t tile_m, int64_t tile_n) {
    const int64_t m = over(s.M, tile_m), n = over(s.N, tile_n);
    return s.mode == kSymmetric ? n * (n + 1) / 2 : m * n * (s.mode == kGroups ? 2 : 1);
}

// Clocks that a product takes, roughly: what each SM has to do one after another,
// at the rates that were seen (per SM and clock 46 bytes from L2, 24 from HBM, the
// MMA's 4096 products), and what a block's start and end cost.
constexpr double kFromL2 = 46, kFromHbm = 24, kStart = 6000, kStartAgain = 3000, kPairStart = 11000, kPairAgain = 3000;

double single_cost(const Shape& s, int64_t steps, int64_t tile_n, int split) {
    const int64_t columns = s.mode == kSideBySide ? 2 * tile_n : tile_n, rows = s.M < 128 ? s.M : 128;
    const int64_t blocks = tiles_of(s, 128, tile_n) * split, turns = over(blocks, kSms);
    // B is read once if there is one row of tiles, and then comes from HBM
    const double b_rate = s.M <= 128 ? kFromHbm : kFromL2;
    double step = columns * 128 / b_rate + rows * 128 / kFromL2;
    if (step < 2.0 * columns) step = 2.0 * columns;
    // two blocks or more share an SM: one's start and end are under another's products, or wait for a place
    return (double)turns * over(steps, split) * step + kStart + (turns - 1) * kStartAgain + 400.0 * (split - 1);
}

}  // namespace

Choice choose(Shape& s) {
    Choice c{};
    const bool side = s.mode == kSideBySide;
    const int64_t steps = (int64_t)s.k_steps * (s.mode == kLongK ? 2 : 1);

    const int64_t pair_n = side ? 128 : 256, pairs = tiles_of(s, 256, pair_n), waves = over(pairs, kSms / 2);
    const double pair_step = 32768 / kFromL2 < 512 ? 512 : 32768 / kFromL2;
    const double pair_cost = waves * steps * pair_step + kPairStart + (waves - 1) * kPairAgain;

    // single blocks: B's rows per tile free where its rows are k and C is not symmetric
    const bool free_n = !s.b_mn && s.mode != kSymmetric;
    const int64_t unit = side ? 8 : 16, most_n = side ? 128 : 256, fixed_n = side ? 64 : 128;
    double best = 1e300;
    for (int split = 1; split <= 8 && split <= steps; ++split)
        for (int64_t n = free_n ? unit : fixed_n; n <= (free_n ? most_n : fixed_n); n += unit) {
            const double cost = single_cost(s, steps, n, split);
            if (cost < best) {
                best = cost;
                s.tile_n = (int)n;
                s.split = split;
            }
        }
    if (s.M > 128 && pair_cost <= best) {
        c.pair = true;
        s.tile_n = (int)pair_n;
        s.split = 1;
        s.b_box = 0;
        s.m_tiles = (int)over(s.M, 256);
        s.n_tiles = (int)over(s.N, pair_n);
        s.tiles = (int)pairs;
        c.grid = (int)(2 * (pairs < kSms / 2 ? pairs : kSms / 2));
        return c;
    }
    const int columns = side ? 2 * s.tile_n : s.tile_n;
    s.m_tiles = (int)over(s.M, 128);
    s.n_tiles = (int)over(s.N, s.tile_n);
    s.tiles = (int)tiles_of(s, 128, s.tile_n);
    c.grid = s.tiles * s.split;
    s.b_box = free_n ? s.tile_n : 0;
    s.b_bytes = free_n ? (uint32_t)columns * 128 : 2 * kBoxBytes;
    s.tmem_columns = 32;
    while (s.tmem_columns < columns) s.tmem_columns *= 2;
    s.part_row = (columns + 31) / 32 * 32 + 4;   // 4 more: vectors of neighbouring rows in different banks
    // stages: as many as fit, for one block per SM or for two
    const uint32_t fixed = 2048, stage = 2 * kBoxBytes + s.b_bytes;
    const uint32_t part = (uint32_t)((s.M < 128 ? (s.M + 31) / 32 * 32 : 128) * s.part_row * 4);
    uint32_t room = (c.grid > kSms ? 233472 / 2 - 1024 : kSharedMost) - fixed;
    if (part > room) room = kSharedMost - fixed;
    s.stages = (int)(room / stage < (uint32_t)kMaxStages ? room / stage : kMaxStages);
    c.smem = fixed + (s.stages * stage > part ? s.stages * stage : part);
    return c;
}

}  // namespace product
}  // namespace mhcpb
