/* Linked with the product's host code (mhcm_product.cu): over many shapes, every byte
 * of shared memory that a single block's copies, MMAs and partial sums touch lies
 * inside what the launch asks for, and the launch's limits hold.  Exits 0, or with
 * the number of bad choices (at most 100). */
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
    std::mt19937_64 g(1);
    auto size = [&](double most) {
        return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(most))(g));
    };
    int bad = 0;
    for (int i = 0; i < 400000; ++i) {
        Shape s{};
        s.M = size(20000), s.N = size(20000), s.k_steps = (int)size(400), s.mode = (int)(g() % 5);
        s.a_mn = g() % 2, s.b_mn = g() % 2;
        if (s.mode == kSymmetric) s.M = s.N;
        if (s.mode == kSideBySide) s.a_mn = s.b_mn = 0;
        s.twice = s.M <= 64 && (s.mode == kPlain || s.mode == kLongK) && g() % 2;
        const Choice c = choose(s);
        if (c.pair) {
            bad += s.M <= 128 || s.twice || c.grid > 152 || s.tiles < s.full;
            continue;
        }
        const uint32_t columns = s.mode == kSideBySide ? 2 * s.tile_n : s.tile_n, stage = 2 * kBoxBytes + s.b_bytes;
        const uint32_t last = 1024 + (s.stages - 1) * stage;   // from the aligned base: barriers, then the stages
        // A's boxes, or 128 rows from its second half on; B's rows, or its two boxes
        uint32_t end = last + 2 * kBoxBytes + (s.twice ? kBoxBytes : 0);
        end = larger(end, last + 2 * kBoxBytes + (s.b_box != 0 ? columns * 128 : 2 * kBoxBytes));
        const uint32_t rows = s.M < 128 ? (uint32_t)(s.M + 31) / 32 * 32 : 128;
        end = larger(end, 1024 + rows * s.part_row * 4);
        const bool ok = end + 1023 <= c.smem && c.smem <= kSharedMost && s.stages >= 2 && s.stages <= kMaxStages &&
                        s.b_bytes >= columns * 128 && (s.b_box == 0 || s.b_box == s.tile_n) && s.b_box <= 256 &&
                        columns % 16 == 0 && columns <= 256 && s.tmem_columns >= (int)columns && s.tmem_columns <= 256 &&
                        (uint32_t)s.part_row >= (columns + 31) / 32 * 32 && stage % 1024 == 0 && s.split >= 1 &&
                        s.split <= 8 && c.grid == s.tiles * s.split && s.full == s.tiles;
        if (!ok && ++bad <= 5)
            std::printf("M %lld N %lld steps %d mode %d twice %d: tile_n %d stages %d, %u bytes of %u\n", (long long)s.M,
                        (long long)s.N, s.k_steps, s.mode, s.twice, s.tile_n, s.stages, end + 1023, c.smem);
    }
    return bad < 100 ? bad : 100;
}
