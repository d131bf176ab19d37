/* Linked with the product's host code (mhcm_product.cu): where A's rows are followed by
 * what their rounding lost, the sums of both, 64 rows apart, lie inside the shared
 * memory that the launch asks for.  Exits 0, or with the number of bad choices (at
 * most 100). */
#include <cmath>
#include <cstdio>
#include <random>

#include "mhcm_internal.h"

using namespace mhcpb::product;

namespace mhcpb {
bool encode_16bit_map(CUtensorMap*, bool, const void*, int64_t, int64_t, int64_t, uint32_t) { return true; }
}  // namespace mhcpb

int main() {
    std::mt19937_64 g(2);
    auto size = [&](double most) {
        return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(most))(g));
    };
    int bad = 0;
    for (int i = 0; i < 400000; ++i) {
        Shape s{};
        s.M = 1 + (int64_t)(g() % 64), s.N = size(1 << 20), s.k_steps = (int)size(1 << 14);
        s.mode = g() % 2 ? kPlain : kLongK;
        s.b_mn = s.mode == kLongK, s.twice = 1;
        const Choice c = choose(s);
        // barriers, then one row of sums for every row of the MMA that is read: 32 at a time, from rows 0 and 64 on
        const uint32_t rows = 64 + (uint32_t)(s.M + 31) / 32 * 32;
        const uint32_t end = 1024 + rows * s.part_row * 4;
        const bool ok = !c.pair && s.m_tiles == 1 && end + 1023 <= c.smem && c.smem <= kSharedMost;
        if (!ok && ++bad <= 5)
            std::printf("M %lld N %lld steps %d mode %d: tile_n %d, %u bytes of %u\n", (long long)s.M, (long long)s.N,
                        s.k_steps, s.mode, s.tile_n, end + 1023, c.smem);
    }
    return bad < 100 ? bad : 100;
}
