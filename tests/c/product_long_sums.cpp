/* Linked with the product's host code (mhcm_product.cu): sums of more than kPieceSteps
 * steps per block are marked as long, and their pieces fit TMEM and shared memory
 * beside the sum.  Exits 0, or with the number of bad choices (at most 100). */
#include <cmath>
#include <cstdio>
#include <random>

#include "mhcm_internal.h"

using namespace mhcpb::product;

namespace mhcpb {
bool encode_16bit_map(CUtensorMap*, bool, const void*, int64_t, int64_t, int64_t, uint32_t) { return true; }
}  // namespace mhcpb

static uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

int main() {
    std::mt19937_64 g(3);
    auto size = [&](double most) {
        return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(most))(g));
    };
    int bad = 0, longs = 0, pairs = 0;
    for (int i = 0; i < 400000; ++i) {
        Shape s{};
        s.M = size(1 << 15), s.N = size(1 << 15), s.k_steps = (int)size(1 << 18), s.mode = (int)(g() % 5);
        s.a_mn = g() % 2, s.b_mn = g() % 2;
        if (s.mode == kSymmetric) s.M = s.N;
        if (s.mode == kSideBySide) s.a_mn = s.b_mn = 0;
        s.twice = s.M <= 64 && (s.mode == kPlain || s.mode == kLongK) && g() % 2;
        const Choice c = choose(s);
        const int64_t steps = (int64_t)s.k_steps * (s.mode == kLongK ? 2 : 1);
        const bool is = (steps + s.split - 1) / s.split > kPieceSteps;
        longs += is, pairs += is && c.pair;
        bool ok = (c.long_sum != 0) == is;
        if (!c.pair) {
            const uint32_t columns = s.mode == kSideBySide ? 2 * s.tile_n : s.tile_n, stage = 2 * kBoxBytes + s.b_bytes;
            const uint32_t read = (columns + 31) / 32 * 32;   // 32 columns at a time
            const uint32_t rows = (s.twice ? 64 : 0) + (s.M < 128 ? (uint32_t)(s.M + 31) / 32 * 32 : 128);
            const uint32_t end = larger(1024 + s.stages * stage, 1024 + rows * s.part_row * 4);
            ok = ok && read * (is ? 2 : 1) <= (uint32_t)s.tmem_columns && s.tmem_columns <= 256 &&
                 (s.tmem_columns & (s.tmem_columns - 1)) == 0 && s.stages >= 2 && end + 1023 <= c.smem &&
                 c.smem <= kSharedMost && s.b_bytes >= columns * 128 && columns % 16 == 0 && c.grid == s.tiles * s.split;
        }
        if (!ok && ++bad <= 5)
            std::printf("M %lld N %lld steps %d mode %d: tile_n %d, split %d, %d columns of TMEM, long %d\n", (long long)s.M,
                        (long long)s.N, s.k_steps, s.mode, s.tile_n, s.split, s.tmem_columns, c.long_sum);
    }
    if (longs < 1000 || pairs < 100) ++bad;
    return bad < 100 ? bad : 100;
}
