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

// Blocks of clusters of 1 to 8 that the GPU holds at once, with one and with two
// blocks to an SM (its processing clusters do not all have the same number of SMs).
constexpr int kPlaces[2][9] = {{0, 152, 152, 138, 144, 140, 138, 105, 120}, {0, 304, 304, 291, 296, 290, 276, 266, 288}};

// What a single block of `columns` of B holds: stages, and shared memory in all.
struct Layout {
    int stages;
    uint32_t smem;
};
Layout layout(const Shape& s, int columns, uint32_t b_bytes, int per_sm) {
    // (twice: the last stage is followed by what 128 rows from the middle of A's place on would reach, so that
    // a descriptor may begin at either half)
    const uint32_t after = s.twice && b_bytes < kBoxBytes ? kBoxBytes - b_bytes : 0;
    const uint32_t fixed = 2048 + after, stage = 2 * kBoxBytes + b_bytes;
    const uint32_t rows = (s.twice ? 64 : 0) + (s.M < 128 ? (uint32_t)over(s.M, 32) * 32 : 128);
    const uint32_t part = rows * ((uint32_t)over(columns, 32) * 32 + 4) * 4;
    const uint32_t room = (per_sm == 2 ? 233472 / 2 - 1024 : kSharedMost) - fixed;
    if (part > room || room / stage < 2) return {0, 0};
    const uint32_t n = room / stage, stages = n < (uint32_t)kMaxStages ? n : kMaxStages;
    return {(int)stages, fixed + (stages * stage > part ? stages * stage : part)};
}

// Clocks that a product takes, roughly, from what was seen: a step of 64 k takes a
// block 500 to issue, and its bytes 1500 from L2 (2200 from HBM) with as many in
// flight as it has stages; per SM and clock there are 46 bytes from L2, 24 from HBM
// and 4096 products.
constexpr double kFromL2 = 46, kFromHbm = 24, kIssue = 500, kStart = 8000, kAgain = 4000, kPairStart = 12000,
                 kPairAgain = 3000;

double single_cost(const Shape& s, int64_t steps, int64_t blocks, int split, int columns, uint32_t b_bytes, int stages,
                   int per_sm) {
    const double a_bytes = (s.M < 128 ? s.M : 128) * 128.0;
    const bool once = s.M <= 128;   // B is read once and comes from HBM
    const double turns = (double)over(blocks, kPlaces[per_sm - 1][split]);
    const double sharing = blocks < kPlaces[per_sm - 1][split] ? (double)over(blocks, kSms) : per_sm;
    double step = kIssue;
    const double waiting = (once ? 2200.0 : 1500.0) / stages;
    const double rate = sharing * (a_bytes / kFromL2 + b_bytes / (once ? kFromHbm : kFromL2));
    const double products = sharing * 2.0 * columns;
    if (step < waiting) step = waiting;
    if (step < rate) step = rate;
    if (step < products) step = products;
    return turns * ((double)over(steps, split) * step + kAgain) + kStart - kAgain + 500.0 * (split - 1);
}

}  // namespace

Choice choose(Shape& s) {
    Choice c{};
    const bool side = s.mode == kSideBySide;
    const int64_t steps = (int64_t)s.k_steps * (s.mode == kLongK ? 2 : 1);

    const int64_t pair_n = side ? 128 : 256, pairs = tiles_of(s, 256, pair_n), places = kSms / 2;
    // a last turn of less than half of the places is one of half tiles
    const int64_t rest = pairs % places, halves = rest <= places / 2 ? rest : 0;
    const double waves = (double)((pairs - halves) / places) + (pairs % places > places / 2 ? 1 : 0) + (halves > 0 ? 0.6 : 0);
    const double pair_step = 32768 / kFromL2 < 512 ? 512 : 32768 / kFromL2;
    const double pair_cost = waves * steps * pair_step + kPairStart + (waves < 1 ? 0 : waves - 1) * kPairAgain;

    // single blocks: B's rows per tile free where its rows are k and C is not symmetric; tried are those
    // that fill the GPU's places once or twice
    const bool free_n = !s.b_mn && s.mode != kSymmetric;
    const int64_t unit = side ? 8 : 16, fixed = side ? 64 : 128, m_tiles = over(s.M, 128);
    double best = 1e300;
    Layout best_layout{};
    for (int split = 1; split <= 8 && split <= steps; ++split) {
        // (a long sum has its pieces beside it in TMEM: half of the columns, so that two blocks still share an SM's)
        const int64_t most = (side ? 128 : 256) / (over(steps, split) > kPieceSteps ? 2 : 1);
        for (int per_sm = 1; per_sm <= 2; ++per_sm)
            for (int turns = 1; turns <= 2; ++turns) {
                int64_t n = fixed;
                if (free_n) {
                    const int64_t room = (int64_t)kPlaces[per_sm - 1][split] * turns / (split * m_tiles);
                    n = room < 1 ? most : over(over(s.N, room), unit) * unit;
                    if (n > most) n = most;
                } else if (turns == 2) {
                    continue;
                }
                const int columns = (int)(side ? 2 * n : n);
                const uint32_t b_bytes = free_n ? (uint32_t)columns * 128 : 2 * kBoxBytes;
                const Layout l = layout(s, columns, b_bytes, per_sm);
                if (l.stages == 0) continue;
                const int64_t blocks = tiles_of(s, 128, n) * split;
                const double cost = single_cost(s, steps, blocks, split, columns, b_bytes, l.stages, per_sm);
                if (cost < best) {
                    best = cost;
                    best_layout = l;
                    s.tile_n = (int)n;
                    s.split = split;
                }
            }
    }
    if (s.M > 128 && pair_cost <= best) {
        c.pair = true;
        s.tile_n = (int)pair_n;
        s.split = 1;
        c.long_sum = steps > kPieceSteps;
        s.b_box = 0;
        s.m_tiles = (int)over(s.M, 256);
        s.n_tiles = (int)over(s.N, pair_n);
        s.full = (int)(pairs - halves);
        s.tiles = (int)(pairs + halves);
        c.grid = (int)(2 * (s.tiles < places ? s.tiles : places));
        return c;
    }
    const int columns = side ? 2 * s.tile_n : s.tile_n;
    s.m_tiles = (int)over(s.M, 128);
    s.n_tiles = (int)over(s.N, s.tile_n);
    s.tiles = s.full = (int)tiles_of(s, 128, s.tile_n);
    c.grid = s.tiles * s.split;
    s.b_box = free_n ? s.tile_n : 0;
    s.b_bytes = free_n ? (uint32_t)columns * 128 : 2 * kBoxBytes;
    s.tmem_columns = 32;
    while (s.tmem_columns < columns) s.tmem_columns *= 2;
    c.long_sum = over(steps, s.split) > kPieceSteps;
    if (c.long_sum) s.tmem_columns *= 2;
    s.part_row = (columns + 31) / 32 * 32 + 4;   // 4 more: vectors of neighbouring rows in different banks
    s.stages = best_layout.stages;
    c.smem = best_layout.smem;
    return c;
}

}  // namespace product
}  // namespace mhcpb
