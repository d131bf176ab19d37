// The matrix product that the feed-forward block and the orthogonalised update
// are made of (sm_103a): C = sum_k A[m, k] B[n, k] on the tensor cores, 16-bit
// operands, FP32 accumulators, and an epilogue that takes eight neighbouring
// elements of C at a time.
//
// Either operand may be stored with k or with its other index innermost: one
// tensor map per matrix, boxes of 64 x 64 elements (8 KiB, 128-byte swizzle),
// serves both, as the MMA's descriptors say which it is.  What lies outside a
// matrix is read as zero, so no size has to be a multiple of anything; only the
// distance between rows is a multiple of 16 bytes (the tensor map's rule).
//
// Two shapes of one kernel:
//  * PAIR: pairs of blocks (cta_group::2), 256 x 256 tiles, one block per SM,
//    persistent; the tiles that would fill less than half of the last turn are
//    taken as halves of 128 columns.  Each block holds half of A's and of B's rows: 32 KiB of
//    operands per 64 k and block, 64 bytes per clock and SM at the full MMA rate.
//    Two accumulators in TMEM (all 512 columns), so the epilogue of one tile runs
//    under the products of the next.
//  * single blocks, tiles of 128 rows and up to 256 columns, one or two blocks per
//    SM, and clusters of `split` blocks that share the sum over k of one tile and
//    add their parts, in rank order, through distributed shared memory: for outputs
//    of few tiles (few tokens, few rows).  Where B's rows are k its rows per tile
//    are chosen (with the split) to give every SM the same share of B.
//
// Measured alone (GB300, BF16): x Wg^T and x Wu^T with their epilogue at 4096 x 5120 x
// 12800 574 us (1.87 PFLOP/s), dWg and dWu 549 us (1.96), the sum of two products for
// dx 608 us (1.77); one after another the power limit brings them to 1.6.  Pairs are
// bound by the MMA (512 clocks per 64 k; 500 are issue), single blocks by what a block
// costs before and after its products (some 8,000 clocks).  5 stages of 64 k leave
// room for the epilogue's scratch; the epilogue's eight warps read TMEM 32 columns at
// a time and go through that scratch so that a warp's stores are whole 64-byte pieces
// of rows.
//
// Warp roles: 0 copies (TMA), 1 MMA issue, 2 TMEM, 4.. epilogue (eight, or four).  Every wait is
// bounded; a wait that runs out records a status word, and the block drains its
// copies and MMAs and leaves.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "mhcm_internal.h"
#include "mhcm_ptx.cuh"
#include "mhcpb.h"
#include "mhcpb_check.cuh"

namespace mhcpb {
namespace product {

static __device__ uint32_t g_status;   // kDevOk or kDevTimeout, of this translation unit's kernels

constexpr uint32_t kPairStage = 4 * kBoxBytes;     // 128 rows of A, 128 of B, 64 k
constexpr int kEpilogueWarp = 4;                   // the first one
constexpr uint64_t kWaitNs = 1000000000ull;        // 1 s

// PAIR: compile-time layout.  Single blocks: the number of stages and a tile's columns are the launch's.
template <bool PAIR>
struct Cfg {
    static constexpr int blocks = PAIR ? 2 : 1;
    static constexpr int threads = PAIR ? 384 : 256;
    static constexpr int tile_m = 128 * blocks;
    static constexpr int stages = PAIR ? 5 : kMaxStages;
    static constexpr int accumulators = PAIR ? 2 : 1;
    // PAIR: 32 rows of 32 FP32 per epilogue warp, 36 apart (vectors without bank conflicts), behind the stages.
    static constexpr int row = 36;
    static constexpr uint32_t scratch = PAIR ? 8 * 32 * row * 4 : 0;
    // barriers (at the front): full[stages] empty[stages] done[2] free[2] last; then TMEM's address and the abort flag
    static constexpr int b_full = 0, b_empty = stages, b_done = 2 * stages, b_free = 2 * stages + 2,
                         b_last = 2 * stages + 4, bars = 2 * stages + 5;
    static constexpr uint32_t off_misc = bars * 8, off_stages = 1024;
    static_assert(off_misc + 8 <= off_stages, "the barriers' part");
    static constexpr uint32_t smem = PAIR ? 1024 + off_stages + stages * kPairStage + scratch : 0;   // 1 KiB to align
    static_assert(smem <= kSharedMost, "shared memory budget");
};

// Which rows and columns of C a tile has.
struct Tile {
    int group, m, n;   // first row and column; of each of the two products where two are formed side by side
    bool mirror;       // symmetric C: the tile is also written transposed
    bool half;         // half of the columns
};
template <int TILE_M>
__device__ __forceinline__ Tile tile_at(const Shape& s, int t) {
    Tile r;
    r.group = 0;
    r.mirror = r.half = false;
    int right = 0;                         // columns to the right of the tile's first
    if (t >= s.full) {                     // the last tiles are taken in halves
        const int h = t - s.full;
        t = s.full + (h >> 1);
        r.half = true;
        right = (h & 1) * (s.tile_n / 2);
    }
    if (s.mode == kSymmetric) {            // tiles on and above the diagonal, row by row
        int i = 0, left = s.n_tiles;
        while (t >= left) {
            t -= left;
            --left;
            ++i;
        }
        r.m = i * TILE_M;
        r.n = (i + t) * s.tile_n + right;
        r.mirror = t > 0;
        return r;
    }
    const int per_group = s.m_tiles * s.n_tiles;
    if (s.mode == kGroups && t >= per_group) {
        t -= per_group;
        r.group = 1;
    }
    // eight rows of tiles at a time, so that the tiles in flight share rows of both operands
    const int band = t / (8 * s.n_tiles), first = band * 8;
    const int rows = min(8, s.m_tiles - first);
    t -= band * 8 * s.n_tiles;
    r.m = (first + t % rows) * TILE_M;
    r.n = (t / rows) * s.tile_n + right;
    return r;
}

// Bounded wait, as wait_bar (mhcpb_wait.cuh); `cluster`: for arrivals from other blocks.
template <bool CLUSTER>
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, bool honor) {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
        if ((i & 31u) == 0) {
            if (honor && *abort_flag) return false;
            if (ptx::globaltimer() - t0 > kWaitNs) {
                *abort_flag = 1u;
                atomicCAS(&g_status, kDevOk, kDevTimeout);
                return false;
            }
        }
    }
}
template <bool CLUSTER>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, bool honor = true) {
    if (CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
    return wait_slow<CLUSTER>(bar, parity, abort_flag, honor);
}

// wait by a whole warp: true where every lane's was
template <bool CLUSTER>
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
    return __all_sync(0xFFFFFFFFu, wait<CLUSTER>(bar, parity, abort_flag));
}

__device__ __forceinline__ void add8(float (&v)[8], const float4& x, const float4& y) {
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
}

// A long sum's pieces, as the MMAs finish them at `from` (TMEM), added up at `to`: `columns` of them (a multiple
// of 32), and as many `apart` further where that is not 0.  `done` and `free` are the pieces' barriers, `turn`
// counts their uses.  False where a wait ran out.  (Out of line: a call that few launches make.)
template <bool PAIR>
static __device__ __noinline__ bool join_pieces(uint32_t done, uint32_t free, uint32_t from, uint32_t to, int columns, int apart,
                                                int pieces, uint32_t turn, volatile uint32_t* abort_flag) {
    for (int p = 0; p < pieces; ++p, ++turn) {
        if (!wait_all<PAIR>(done, turn & 1u, abort_flag)) return false;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < (apart != 0 ? 2 : 1) * columns; c += 32) {
            const uint32_t at = (uint32_t)(c < columns ? c : c - columns + apart);
            uint32_t u[32], v[32];
            ptx::tmem_ld_32x32b_x32(from + at, u);
            ptx::tc_wait_ld_regs(u);
            if (p > 0) {
                ptx::tmem_ld_32x32b_x32(to + at, v);
                ptx::tc_wait_ld_regs(v);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(v[i]));
            }
            ptx::tmem_st_32x32b_x32(to + at, u);
            ptx::tc_wait_st();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive_cluster(free);
    }
    return true;
}

// The products of two numbers' first and of their second, where those of the first are finite.
template <int N>
__device__ __forceinline__ void add_second(float (&v)[N], const float (&w)[N], float unit) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = isfinite(v[i]) ? fmaf(w[i], unit, v[i]) : v[i];
}

// The elements of one row of C that an epilogue takes at a time: eight neighbours, where the epilogue's
// matrices have rows that start at 16 bytes and end at them or in a workspace's padding (which may be
// written), else one (a warp then has 32 neighbours).
struct Eight {
    static constexpr int n = 8;
    int64_t row, col;
    bool is;             // elements of C
    __device__ __forceinline__ int64_t column(int i) const { return col + i; }
};
struct One {
    static constexpr int n = 1;
    int64_t row, col;
    bool is;
    __device__ __forceinline__ int64_t column(int) const { return col; }
};

// Epilogue: struct with
//   static constexpr bool kDual                    two products side by side
//   static constexpr bool kMirror                  C is symmetric; its matrices are a workspace's (Eight always)
//   static constexpr bool kTwice                   A may be two numbers (Shape::twice)
//   template <class Span> struct Read              what elements' results need from memory
//   void ahead(int group, int64_t row, int64_t col, int cols) const   what read() will read of a row, towards L2
//   Read<Span> read(int group, const Span&) const
//   void write(int group, const Span&, const float (&v)[Span::n], const float (&w)[Span::n], const Read<Span>&) const
// (Span: Eight or One; w: the second product's, where kDual).  Several reads are under way before the first write.
// LONG: a block's sum has more than kPieceSteps steps.  (A kernel of its own: as a branch of the others it
// cost 1285 x 3427 orthogonalised 368 us for 363, its gradients 181 for 177.)
template <bool PAIR, bool LONG, class Epilogue>
__global__ void __launch_bounds__(Cfg<PAIR>::threads, PAIR ? 1 : 2)
    product_kernel(const Shape s, const Epilogue epi, const __grid_constant__ CUtensorMap a0,
                   const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b0,
                   const __grid_constant__ CUtensorMap b1) {
    using C = Cfg<PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t base = ptx::smem_u32(smem), stage0 = base + C::off_stages;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::off_misc);
    volatile uint32_t* abort_flag = holder + 1;
    auto bar = [&](int i) { return base + 8u * (uint32_t)i; };
    // columns of the accumulator (of both products side by side), stages and what one holds
    const uint32_t width = PAIR ? 256 : (uint32_t)(s.mode == kSideBySide ? 2 * s.tile_n : s.tile_n);
    const uint32_t stages = PAIR ? C::stages : (uint32_t)s.stages;
    const uint32_t stage_bytes = PAIR ? kPairStage : 2 * kBoxBytes + s.b_bytes;
    const uint32_t tmem_columns = PAIR ? 512 : (uint32_t)s.tmem_columns;

    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        for (int i = 0; i < C::stages; ++i) {
            ptx::mbar_init(bar(C::b_full + i), 1);
            ptx::mbar_init(bar(C::b_empty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(C::b_done + i), 1);
            ptx::mbar_init(bar(C::b_free + i), PAIR ? 16 : 4);   // the epilogue's warps
        }
        ptx::mbar_init(bar(C::b_last), 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&a0);
        ptx::prefetch_tensormap(&b0);
    }
    if (warp == 2) ptx::tmem_get<PAIR>(ptx::smem_u32(holder), tmem_columns);
    ptx::tc_fence_before();
    ptx::cluster_arrive();   // the pair's barriers are there before either block uses them
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem = *holder;
    // (every launch: only its own wait makes visible what an earlier one wrote, of the launch before the last one too)
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    // Tiles: every gridDim.x / cluster blocks-th one.  k steps of this block: all, or its share of a split sum.
    const int cluster = PAIR ? 2 : s.split;
    const int first_tile = blockIdx.x / cluster, step_tile = gridDim.x / cluster;
    const int steps = s.k_steps * (s.mode == kLongK ? 2 : 1);
    const int k_begin = PAIR ? 0 : (int)((int64_t)rank * steps / s.split);
    const int k_end = PAIR ? steps : (int)((int64_t)(rank + 1) * steps / s.split);
    const bool leader = !PAIR || rank == 0;
    // A long sum is taken in pieces: each is formed in the second half of TMEM's columns and added, rounded, to
    // what is in the first.
    const int pieces = LONG ? (k_end - k_begin + kPieceSteps - 1) / kPieceSteps : 1;
    const uint32_t second_half = PAIR ? width : tmem_columns / 2;

    if (warp == 0) {
        const uint32_t half = PAIR ? rank : 0;
        uint32_t st = 0, ph = 0, n = 0;                      // stage, its turn's parity, steps so far
        bool ok = true;
        for (int t = first_tile; ok && t < s.tiles; t += step_tile) {
            const Tile tile = tile_at<C::tile_m>(s, t);
            const int m0 = tile.m + (int)half * 128;
            const int n0 = tile.n + (s.mode == kSideBySide ? 0 : (int)half * (tile.half ? 64 : 128));
            // (a single block leaves out the half of A's rows that no token has: their results are not read)
            const int a_boxes = !PAIR && s.M - tile.m <= kBox && !s.twice ? 1 : 2;
            const uint32_t bytes = PAIR ? 2 * kPairStage - (tile.half ? 2 * kBoxBytes : 0) : a_boxes * kBoxBytes + s.b_bytes;
            for (int k = k_begin; k < k_end; ++k, ++n) {
                if (!wait_all<PAIR>(bar(C::b_empty + st), ph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t full = PAIR ? ptx::map_rank(bar(C::b_full + st), 0) : bar(C::b_full + st);
                if (leader) ptx::mbar_expect_one(bar(C::b_full + st), bytes);
                const bool second = s.mode == kLongK && k >= s.k_steps;
                const int k0 = (second ? k - s.k_steps : k) * kBox;
                const CUtensorMap* am = second || tile.group ? &a1 : &a0;
                const CUtensorMap* bm = second || tile.group ? &b1 : &b0;
                const uint32_t dst = stage0 + st * stage_bytes, dst_b = dst + 2 * kBoxBytes;
                ptx::tma_load_one<PAIR>(dst, am, s.a_mn ? m0 : k0, s.a_mn ? k0 : m0, full);
                if (a_boxes == 2)
                    ptx::tma_load_one<PAIR>(dst + kBoxBytes, am, s.a_mn ? m0 + kBox : k0, s.a_mn ? k0 : m0 + kBox, full);
                if (!PAIR && s.b_box != 0) {   // all of a product's rows in one box
                    ptx::tma_load_one<PAIR>(dst_b, bm, k0, n0, full);
                    if (s.mode == kSideBySide)
                        ptx::tma_load_one<PAIR>(dst_b + (uint32_t)s.tile_n * (kBox * 2), &b1, k0, n0, full);
                } else {
                    // side by side: a block of a pair has one product's rows, a single block 64 of each
                    const bool side = s.mode == kSideBySide;
                    const int n1 = side && !PAIR ? n0 : n0 + kBox;
                    const CUtensorMap* b_first = side && PAIR && half == 1 ? &b1 : bm;
                    const CUtensorMap* b_second = side && (!PAIR || half == 1) ? &b1 : bm;
                    ptx::tma_load_one<PAIR>(dst_b, b_first, s.b_mn ? n0 : k0, s.b_mn ? k0 : n0, full);
                    if (!PAIR || !tile.half)
                        ptx::tma_load_one<PAIR>(dst_b + kBoxBytes, b_second, s.b_mn ? n1 : k0, s.b_mn ? k0 : n1, full);
                }
                if (++st == stages) st = 0, ph ^= 1u;
            }
        }
        if (!ok && leader)   // the copies that were started end before the block does
            for (uint32_t i = n > stages ? n - stages : 0; i < n; ++i)
                wait<PAIR>(bar(C::b_full + i % stages), (i / stages) & 1u, abort_flag, false);
    } else if (warp == 1 && leader) {
        const uint32_t idesc_whole = ptx::idesc_16bit(C::tile_m, width, s.bf16, s.a_mn, s.b_mn);
        const uint32_t idesc_half = ptx::idesc_16bit(C::tile_m, width / 2, s.bf16, s.a_mn, s.b_mn);
        // 16 k further: 32 bytes along a row, or 16 rows of 128 bytes (in descriptors' units of 16)
        const uint64_t a_step = s.a_mn ? 128 : 2, b_step = s.b_mn ? 128 : 2;
        const uint64_t first = ptx::smem_desc(stage0, kBoxBytes, 1024, ptx::kLayoutSwizzle128B);
        uint32_t st = 0, ph = 0, done = 0;
        bool ok = true;
        for (int t = first_tile, from = k_begin; ok && t < s.tiles; ++done) {
            const uint32_t acc = LONG ? 1 : done % C::accumulators, turn = LONG ? done : done / C::accumulators;
            if (!wait_all<PAIR>(bar(C::b_free + acc), (turn & 1u) ^ 1u, abort_flag)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t d = tmem + acc * second_half, idesc = PAIR && t >= s.full ? idesc_half : idesc_whole;
            const int to = LONG ? min(from + kPieceSteps, k_end) : k_end;
            if (s.stall && !wait_all<PAIR>(bar(C::b_last), 0u, abort_flag)) {   // a test's wait that nothing ends
                ok = false;
                break;
            }
            for (int k = from; k < to; ++k) {
                if (!wait_all<PAIR>(bar(C::b_full + st), ph, abort_flag)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint64_t a = first + ((st * stage_bytes) >> 4);
                ptx::mma64_one<PAIR>(d, a, a + (2 * kBoxBytes >> 4), idesc, a_step, b_step, k > from);
                ptx::mma_commit_one<PAIR>(bar(C::b_empty + st), 3);
                if (++st == stages) st = 0, ph ^= 1u;
            }
            if (ok) ptx::mma_commit_one<PAIR>(bar(C::b_done + acc), 3);
            from = to == k_end ? k_begin : to;
            if (to == k_end) t += step_tile;
        }
        if (!ok) {           // the MMAs that were issued end before the block does
            ptx::mma_commit_one<PAIR>(bar(C::b_last), 1);
            wait<PAIR>(bar(C::b_last), 0u, abort_flag, false);
        }
    } else if (warp >= kEpilogueWarp) {
        const int quad = warp & 3, half = (warp - kEpilogueWarp) >> 2;   // half: 0 where there are four warps
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        if constexpr (PAIR) {
            float* scratch = 
                reinterpret_cast<float*>(smem + C::off_stages + C::stages * kPairStage) + (warp - kEpilogueWarp) * 32 * C::row;
            // 32 columns of this warp's 32 rows into its scratch
            auto stage = [&](uint32_t column) {
                uint32_t u[32];
                ptx::tmem_ld_32x32b_x32(lanes + column, u);
                ptx::tc_wait_ld_regs(u);
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    *reinterpret_cast<uint4*>(scratch + lane * C::row + c) = make_uint4(u[c], u[c + 1], u[c + 2], u[c + 3]);
                __syncwarp();
            };
            // What is added to is sent for a tile earlier: where a tile has few k steps, the reads of one chunk at a
            // time are all that is under way (gradients of 1,000 tokens, 1285 x 3427, added: 147 us for 152).
            auto ahead = [&](const Tile& tile) {
                const int columns = (Epilogue::kDual ? 64 : 128) >> (tile.half ? 1 : 0);
                const int64_t row = tile.m + (int64_t)rank * 128 + quad * 32 + lane, col = tile.n + half * columns;
                if (row < s.M && col < s.N) epi.ahead(tile.group, row, col, (int)min((int64_t)columns, s.N - col));
            };
            uint32_t done = 0;
            Tile tile, next = tile_at<C::tile_m>(s, first_tile);
            ahead(next);
            for (int t = first_tile; t < s.tiles; t += step_tile, ++done) {
                const uint32_t acc = LONG ? 0 : done & 1u;
                tile = next;
                if (t + step_tile < s.tiles) ahead(next = tile_at<C::tile_m>(s, t + step_tile));
                const int64_t row0 = tile.m + (int64_t)rank * 128 + quad * 32;
                const uint32_t d = acc * width;
                const int chunks = (Epilogue::kDual ? 2 : 4) >> (tile.half ? 1 : 0);   // of 32 columns per warp
                const int up = tile.half ? 64 : 128;                                   // the second product's columns
                bool ok = true;
                if constexpr (LONG) {
                    const uint32_t at = lanes + half * chunks * 32;
                    ok = join_pieces<PAIR>(bar(C::b_done + 1), ptx::map_rank(bar(C::b_free + 1), 0), at + second_half, at,
                                           chunks * 32, Epilogue::kDual ? up : 0, pieces, done * pieces, abort_flag);
                    if (!ok) break;
                }
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    const int column = half * chunks * 32 + c * 32;
                    const int64_t col0 = tile.n + column;
                    auto ready = [&] {   // the first chunk's reads are under way: now the accumulator
                        if (c == 0 && !LONG) {
                            ok = wait_all<PAIR>(bar(C::b_done + acc), (done >> 1) & 1u, abort_flag);
                            if (ok) ptx::tc_fence_after();
                        }
                        return ok;
                    };
                    auto drained = [&] {   // the last chunk has left TMEM
                        if (c == chunks - 1 && !LONG) {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_rank(bar(C::b_free + acc), 0));
                        }
                    };
                    if (!Epilogue::kMirror && s.narrow) {
                        // column `lane` of each row, sixteen rows' reads at a time (1,000 tokens, 1285 x 3427, gradients
                        // added: 139 us; eight 146, all 32 before the wait for the products 146)
                        auto at = [&](int row) {
                            return One{row0 + row, col0 + lane, col0 + lane < s.N && row0 + row < s.M};
                        };
                        if (!ready()) break;
                        float w[Epilogue::kDual ? 32 : 1];
                        if constexpr (Epilogue::kDual) {
                            stage(d + up + column);
#pragma unroll
                            for (int q = 0; q < 32; ++q) w[q] = scratch[q * C::row + lane];
                        }
                        stage(d + column);
                        drained();
#pragma unroll(Epilogue::kDual ? 4 : 1)
                        for (int first = 0; first < 32; first += 16) {
                            typename Epilogue::template Read<One> read[16];
#pragma unroll
                            for (int q = 0; q < 16; ++q) read[q] = epi.read(tile.group, at(first + q));
#pragma unroll
                            for (int q = 0; q < 16; ++q) {
                                const float v[1] = {scratch[(first + q) * C::row + lane]};
                                const float u[1] = {w[Epilogue::kDual ? first + q : 0]};
                                epi.write(tile.group, at(first + q), v, u, read[q]);
                            }
                        }
                        continue;
                    }
                    // eight columns of rows 8 q + lane / 4; transposed: of row `lane` of the chunk's columns
                    Eight at[4], mat[4];
                    typename Epilogue::template Read<Eight> read[4], mread[4];
                    const int64_t col = col0 + 8 * (lane & 3);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        at[q] = {row0 + 8 * q + lane / 4, col, col < s.N && row0 + 8 * q + lane / 4 < s.M};
                        if (at[q].is) read[q] = epi.read(tile.group, at[q]);
                    }
                    if (Epilogue::kMirror && tile.mirror) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            mat[q] = {col0 + lane, row0 + 8 * q, col0 + lane < s.N && row0 + 8 * q < s.M};
                            if (mat[q].is) mread[q] = epi.read(0, mat[q]);
                        }
                    }
                    if (!ready()) break;
                    float v[4][8], w[Epilogue::kDual ? 4 : 1][8];
                    auto vectors = [&](float (&x)[4][8]) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4* p =
                                reinterpret_cast<const float4*>(scratch + (8 * q + lane / 4) * C::row + 8 * (lane & 3));
                            const float4 f = p[0], g = p[1];
                            x[q][0] = f.x, x[q][1] = f.y, x[q][2] = f.z, x[q][3] = f.w;
                            x[q][4] = g.x, x[q][5] = g.y, x[q][6] = g.z, x[q][7] = g.w;
                        }
                    };
                    stage(d + column);
                    vectors(v);
                    if constexpr (Epilogue::kDual) {
                        stage(d + up + column);
                        vectors(w);
                    }
                    drained();
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (at[q].is) epi.write(tile.group, at[q], v[q], w[Epilogue::kDual ? q : 0], read[q]);
                    if (Epilogue::kMirror && tile.mirror) {   // the scratch still has the chunk
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = scratch[(8 * q + i) * C::row + lane];
                            if (mat[q].is) epi.write(0, mat[q], x, x, mread[q]);
                        }
                    }
                }
                if (!ok) break;
            }
        } else {
            const Tile tile = tile_at<C::tile_m>(s, first_tile);
            const int own = quad * 32 + lane;
            if (tile.m + own < s.M && own % s.split == (int)rank)
                epi.ahead(tile.group, tile.m + own, tile.n, (int)min((int64_t)s.tile_n, s.N - tile.n));
            const bool ok = LONG ? join_pieces<PAIR>(bar(C::b_done + 1), bar(C::b_free + 1), lanes + second_half, lanes,
                                                     ((int)width + 31) / 32 * 32, 0, pieces, 0u, abort_flag)
                                 : wait_all<PAIR>(bar(C::b_done), 0u, abort_flag);
            ptx::tc_fence_after();
            float* part = reinterpret_cast<float*>(smem + C::off_stages);   // over the (now idle) stages
            const int row = quad * 32 + lane;
            if (ok && (Epilogue::kTwice && s.twice ? quad & 1 : quad) * 32 < s.M - tile.m)
                for (int c = 0; c < (int)width; c += 32) {
                    uint32_t u[32];
                    ptx::tmem_ld_32x32b_x32(lanes + c, u);
                    ptx::tc_wait_ld_regs(u);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(part + row * s.part_row + c + i) =
                            make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                }
        }
    }

    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_arrive();   // pair: no block leaves while the other's MMAs or arrivals may reach it
    ptx::cluster_wait();
    ptx::tc_fence_after();
    __syncwarp();
    if (warp == 2) ptx::tmem_free<PAIR>(tmem, tmem_columns);

    if constexpr (!PAIR) {
        // Every block has its part of the tile in shared memory; each adds up its share of the vectors.
        const Tile tile = tile_at<C::tile_m>(s, first_tile);
        const int rows = (int)min((int64_t)128, s.M - tile.m), cols = (int)min((int64_t)s.tile_n, s.N - tile.n);
        auto part_at = [&](uint32_t i, int z) { return ptx::map_rank(stage0 + 4 * i, z); };
        // One vector per thread at a time, in loops that are not unrolled: these launches are short, and
        // what they cost is the way of their instructions from memory (with four vectors at a time, their
        // loads side by side, 512 x 512 orthogonalised took 223 us for 155).
        // Of an A of two numbers, the second's products are 64 rows further.  They are added where the first's are finite:
        // an infinite weight makes the first's infinite, and the second's, of what rounding left of the same
        // number, of any sign, or NaN where that is zero.
        const bool twice = Epilogue::kTwice && s.twice;
        const uint32_t further = 4u * 64u * (uint32_t)s.part_row;
        const int threads = s.split * C::threads, me = (int)rank * C::threads + threadIdx.x;
        if (!Epilogue::kMirror && s.narrow) {
            // a warp per row, four times 32 columns at a time (a lane has one element of each: their reads side by side)
            constexpr int kTimes = 4;
            for (int r = (int)rank * (C::threads / 32) + warp; r < rows; r += s.split * (C::threads / 32))
#pragma unroll 1
                for (int first = lane; first < cols; first += 32 * kTimes) {
                    typename Epilogue::template Read<One> read[kTimes];
                    float v[kTimes][1] = {}, w[kTimes][1] = {};
                    auto at = [&](int q) {
                        return One{(int64_t)tile.m + r, (int64_t)tile.n + first + 32 * q, first + 32 * q < cols};
                    };
#pragma unroll
                    for (int q = 0; q < kTimes; ++q) read[q] = epi.read(tile.group, at(q));
#pragma unroll 1
                    for (int z = 0; z < s.split; ++z) {
                        const uint32_t p = part_at((uint32_t)(r * s.part_row + first), z);
                        float x[kTimes], y[kTimes];
#pragma unroll
                        for (int q = 0; q < kTimes; ++q) {
                            x[q] = first + 32 * q < cols ? ptx::ld_cluster_f32(p + 128 * q) : 0.f;
                            y[q] = (Epilogue::kDual || twice) && first + 32 * q < cols
                                       ? ptx::ld_cluster_f32(p + 128 * q + (Epilogue::kDual ? 4 * s.tile_n : further)) : 0.f;
                        }
#pragma unroll
                        for (int q = 0; q < kTimes; ++q) v[q][0] += x[q], w[q][0] += y[q];
                    }
#pragma unroll
                    for (int q = 0; q < kTimes; ++q) {
                        if (twice) add_second(v[q], w[q], s.second);
                        epi.write(tile.group, at(q), v[q], w[q], read[q]);
                    }
                }
        } else {
            const int across = (cols + 7) / 8, units = rows * across;
#pragma unroll 1
            for (int u = me; u < units; u += threads) {
                const int r = u / across, c = (u - r * across) * 8;
                const Eight at{(int64_t)tile.m + r, (int64_t)tile.n + c, true};
                const auto read = epi.read(tile.group, at);
                float v[8] = {}, w[8] = {};
#pragma unroll 1
                for (int z = 0; z < s.split; ++z) {
                    const uint32_t p = part_at((uint32_t)(r * s.part_row + c), z);
                    add8(v, ptx::ld_cluster_f32x4(p), ptx::ld_cluster_f32x4(p + 16));
                    if constexpr (Epilogue::kDual)
                        add8(w, ptx::ld_cluster_f32x4(p + 4 * s.tile_n), ptx::ld_cluster_f32x4(p + 4 * s.tile_n + 16));
                    else if (twice)
                        add8(w, ptx::ld_cluster_f32x4(p + further), ptx::ld_cluster_f32x4(p + further + 16));
                }
                if (twice) add_second(v, w, s.second);
                epi.write(tile.group, at, v, w, read);
            }
        }
        if (Epilogue::kMirror && tile.mirror) {   // transposed: eight rows of one column
            const int down = (rows + 7) / 8, flipped = cols * down;
#pragma unroll 1
            for (int u = me; u < flipped; u += threads) {
                const int g = u / cols, c = u - g * cols;
                const Eight at{(int64_t)tile.n + c, (int64_t)tile.m + 8 * g, true};
                const auto read = epi.read(0, at);
                float v[8] = {};
#pragma unroll 1
                for (int z = 0; z < s.split; ++z) {
                    const uint32_t p = part_at((uint32_t)(8 * g * s.part_row + c), z);
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = ptx::ld_cluster_f32(p + 4 * i * s.part_row);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += x[i];
                }
                epi.write(0, at, v, v, read);
            }
        }
        ptx::cluster_arrive();   // the parts stay until every block has read them
        ptx::cluster_wait();
    }
}

// ---------------------------------------------------------------- host
template <class Epilogue>
cudaError_t allow() {
    static std::atomic<uint64_t> done[4] = {};
    cudaError_t e = ops::allow_shared(product_kernel<true, false, Epilogue>, (int)Cfg<true>::smem, done[0]);
    if (e == cudaSuccess) e = ops::allow_shared(product_kernel<false, false, Epilogue>, (int)kSharedMost, done[1]);
    if (e == cudaSuccess) e = ops::allow_shared(product_kernel<true, true, Epilogue>, (int)Cfg<true>::smem, done[2]);
    if (e == cudaSuccess) e = ops::allow_shared(product_kernel<false, true, Epilogue>, (int)kSharedMost, done[3]);
    return e;
}

// a1 and b1 may be null where the mode has one A or B.
template <class Epilogue>
cudaError_t launch(Shape s, const Epilogue& epi, const Factor* a0, const Factor* a1, const Factor* b0, const Factor* b1,
                   cudaStream_t stream) {
    cudaError_t e = allow<Epilogue>();
    if (e != cudaSuccess) return e;
    const Choice c = choose(s);
    const CUtensorMap *mb0 = &b0->map, *mb1 = b1 ? &b1->map : mb0, *ma0 = &a0->map, *ma1 = a1 ? &a1->map : ma0;
    CUtensorMap own[2];
    if (s.b_box != 0) {   // boxes of as many rows as a tile takes
        if (!b0->encode(&own[0], s.b_box) || (b1 && !b1->encode(&own[1], s.b_box))) return cudaErrorInvalidValue;
        mb0 = &own[0], mb1 = b1 ? &own[1] : &own[0];
    }
    cudaLaunchConfig_t config{};
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c.pair ? 2 : (unsigned)s.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    config.attrs = attr;
    config.numAttrs = 2;
    config.blockDim = c.pair ? Cfg<true>::threads : Cfg<false>::threads;
    config.gridDim = (unsigned)c.grid;
    config.dynamicSmemBytes = c.pair ? Cfg<true>::smem : c.smem;
    config.stream = stream;
    auto* kernel = c.pair ? (c.long_sum ? product_kernel<true, true, Epilogue> : product_kernel<true, false, Epilogue>)
                          : (c.long_sum ? product_kernel<false, true, Epilogue> : product_kernel<false, false, Epilogue>);
    return cudaLaunchKernelEx(&config, kernel, s, epi, *ma0, *ma1, *mb0, *mb1);
}

// This translation unit's status word, then cleared if asked (current device).
static inline cudaError_t read_status(uint32_t* status, bool clear) {
    const uint32_t zero = kDevOk;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(uint32_t));
    if (e == cudaSuccess && clear && *status != kDevOk) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(uint32_t));
    return e;
}

// ---------------------------------------------------------------- eight neighbours in memory
template <class T>
struct Pair16;
template <>
struct Pair16<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    }
};
template <>
struct Pair16<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 p = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
};

// Elements as they are stored.
template <class T, class Span>
struct Raw {
    static constexpr int words = (Span::n * (int)sizeof(T) + 3) / 4;
    uint32_t u[words];
    __device__ __forceinline__ void to(float (&v)[Span::n]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < words; ++i) {
                const float2 f = Pair16<T>::unpack(u[i]);
                v[2 * i] = f.x;
                if (2 * i + 1 < Span::n) v[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < words; ++i) v[i] = __uint_as_float(u[i]);
        }
    }
};

// A matrix in memory; `elements` (of the whole matrix) bounds the accesses of a checked build.
template <class T>
struct Matrix {
    using Value = std::remove_const_t<T>;
    T* ptr;
    int64_t ld;
    size_t elements;

    __device__ __forceinline__ bool ok(const T* p, int count, uint32_t site) const {
        return check::in(p, (size_t)count * sizeof(T), ptr, elements * sizeof(T), site);
    }
    __device__ __forceinline__ static uint32_t bits(const T* p) {
        if constexpr (sizeof(T) == 2)
            return *reinterpret_cast<const uint16_t*>(p);
        else
            return *reinterpret_cast<const uint32_t*>(p);
    }
    __device__ __forceinline__ Raw<Value, Eight> raw(const Eight& at, uint32_t site) const {
        const T* p = ptr + at.row * ld + at.col;
        Raw<Value, Eight> r{};
        if (!ok(p, 8, site)) return r;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            r.u[4 * i] = q.x, r.u[4 * i + 1] = q.y, r.u[4 * i + 2] = q.z, r.u[4 * i + 3] = q.w;
        }
        return r;
    }
    __device__ __forceinline__ Raw<Value, One> raw(const One& at, uint32_t site) const {
        const T* p = ptr + at.row * ld + at.col;
        Raw<Value, One> r{};
        if (at.is && ok(p, 1, site)) r.u[0] = bits(p);
        return r;
    }
    __device__ __forceinline__ void store(const Eight& at, const float (&v)[8], uint32_t site) const {
        T* p = ptr + at.row * ld + at.col;
        if (!ok(p, 8, site)) return;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p) = make_uint4(Pair16<T>::pack(v[0], v[1]), Pair16<T>::pack(v[2], v[3]),
                                                      Pair16<T>::pack(v[4], v[5]), Pair16<T>::pack(v[6], v[7]));
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    __device__ __forceinline__ void store(const One& at, const float (&v)[1], uint32_t site) const {
        T* p = ptr + at.row * ld + at.col;
        if (at.is && ok(p, 1, site)) *p = (T)v[0];
    }
    __device__ __forceinline__ void ahead(int64_t row, int64_t col, int cols) const {
        const T* p = ptr + row * ld + col;
        ptx::prefetch_l2(p, p + cols);
    }
    // whether a caller's matrix of `cols` columns can be read and written by Eight (its first row starts at 16 bytes)
    bool by_eight(int64_t cols) const { return ptr == nullptr || (cols % 8 == 0 && ld * (int64_t)sizeof(T) % 16 == 0); }
};

}  // namespace product
}  // namespace mhcpb
