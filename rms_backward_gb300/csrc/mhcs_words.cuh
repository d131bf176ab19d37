// Rows whose addresses are not multiples of 16 bytes.
//
// Loads: a warp's part of a row (32 vectors of kPack columns) is copied to
// shared memory in whole aligned 16-byte chunks.  A vector that starts m
// elements into a chunk lies in that chunk and the next; each lane puts its own
// together from both with selects and funnel shifts, once, and it is used as an
// aligned vector from then on.  A chunk may hold elements of neighbouring rows
// (copied, never used); parts whose chunks stick out of the operand, at its
// beginning or end, are copied as single elements instead.  (4-byte
// copies need no putting together but four times the copies: the collapse
// gradient at T=4096, D=1285 took 93 us instead of 66.)
// Stores: a warp's vectors go through shared memory and leave in 4-byte words,
// or 2-byte elements where the row starts in the middle of a word, consecutive
// lanes on consecutive words.
#pragma once
#include "mhcs_common.cuh"
#include "mhcs_ring.cuh"

namespace mhcpb {
namespace ops {

constexpr int kWarpSlots = 33;   // 16-byte slots of a warp's part of a row: 32 vectors can touch 33 chunks

// Elements between the 16-byte boundary below p and p.
template <typename E>
__device__ __forceinline__ int misaligned(const E* p) {
    return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(E)) & (Elem<E>::kPack - 1);
}
// Whether chunks of row r of `rows`, which are `width` elements and more apart,
// can stick out of the operand: a chunk reaches up to kPack - 1 elements past
// its row on either side.
template <typename E>
__device__ __forceinline__ bool edge_row(int64_t r, int64_t rows, int64_t width) {
    constexpr int64_t kReach = Elem<E>::kPack - 1;
    const int64_t reach = width >= kReach ? 1 : (kReach - 1 + width) / width;   // rows
    return r < reach || r >= rows - reach;
}
// 1 if p lies in the middle of a 4-byte word (16-bit types), else 0.
template <typename E>
__device__ __forceinline__ int half_word(const E* p) {
    return sizeof(E) == 2 ? (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1) : 0;
}

// Starts copying a warp's part of a row, `width` elements (cut to its 32
// vectors; none if <= 0) from element `at` on, into its slots.  Not for
// edge_row()s.  The whole warp.
template <typename E>
__device__ __forceinline__ void copy_chunks(uint4* slots, const Span<const E>& in, size_t at, int width, uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    const int lane = threadIdx.x & 31, m = misaligned(in.p + at);
    const size_t first = at - m + (size_t)lane * kPack;
    if (lane * kPack - m < width && in.has(first, kPack, site)) copy16(slots + lane, in.p + first);
    if (lane == 31 && m > 0 && 32 * kPack - m < width && in.has(first + kPack, kPack, site))
        copy16(slots + 32, in.p + first + kPack);
}
// The same for any row: a part whose chunks stick out of the operand is copied
// element by element, at once.  A call, in a loop over
// the arrays: inlined beside every copy it cost the rows' kernels registers.
template <typename E>
__device__ __noinline__ void copy_edge(uint4* slots, const E* p, size_t count, size_t at, int width, uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    const int lane = threadIdx.x & 31, m = misaligned(p + at);
    if (width <= 0) return;
    if (width > 32 * kPack) width = 32 * kPack;
    const size_t end = at + (width + m + kPack - 1) / kPack * kPack - m;   // of the last chunk
    if (at >= (size_t)m && end <= count) {
        copy_chunks(slots, Span<const E>{p, count}, at, width, site);
        return;
    }
    E v[kPack];
#pragma unroll
    for (int k = 0; k < kPack; ++k) {
        const int i = lane + 32 * k;
        if (i < width && check::in(p + at + i, sizeof(E), p, count * sizeof(E), site)) v[k] = p[at + i];
    }
    E* const dst = reinterpret_cast<E*>(slots) + m;
#pragma unroll
    for (int k = 0; k < kPack; ++k)
        if (lane + 32 * k < width) dst[lane + 32 * k] = v[k];
}
// After the copies have arrived and a __syncwarp: each lane's slot becomes its
// vector, elements past `valid` 0.  m: misaligned() of the part's first
// element.  The whole warp.
template <typename E>
__device__ __forceinline__ void align_chunks(uint4* slots, int m, int valid) {
    constexpr int kPack = Elem<E>::kPack, per_word = 4 / (int)sizeof(E);
    const int lane = threadIdx.x & 31;
    if (m > 0) {   // the same in every lane
        const uint4 a = slots[lane], b = slots[lane + 1];
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const int words = m / per_word;
        if (words & 2)
#pragma unroll
            for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
        if (words & 1)
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
        if constexpr (sizeof(E) == 2)
            if (m & 1)
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        __syncwarp();
        slots[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (valid < kPack) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(slots + lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int left = valid - k * per_word;
            w[k] = left <= 0 ? 0u : left >= per_word ? w[k] : w[k] & 0xffffu;
        }
    }
}

// Stores each lane's vector: `width` elements (cut to the warp's part) from
// element `at` of the warp's first column on.  slots: 32 free ones of the
// warp, which may be used again afterwards.  The whole warp.
template <typename E>
__device__ __forceinline__ void store_words(uint4* slots, const Span<E>& out, size_t at, int width, const uint4& own,
                                            uint32_t site) {
    constexpr int per_word = 4 / (int)sizeof(E);
    const int lane = threadIdx.x & 31;
    slots[lane] = own;
    __syncwarp();
    E* const p = out.p + at;
    if (half_word(p) == 0) {
        const uint32_t* const words = reinterpret_cast<const uint32_t*>(slots);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = lane + 32 * k;
            if ((i + 1) * per_word <= width) {
                if (out.has(at + i * per_word, per_word, site)) reinterpret_cast<uint32_t*>(p)[i] = words[i];
            } else if (sizeof(E) == 2 && i * per_word < width) {
                if (out.has(at + i * per_word, 1, site)) p[i * per_word] = reinterpret_cast<const E*>(slots)[i * per_word];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < Elem<E>::kPack; ++k) {
            const int i = lane + 32 * k;
            if (i < width && out.has(at + i, 1, site)) p[i] = reinterpret_cast<const E*>(slots)[i];
        }
    }
    __syncwarp();
}

}  // namespace ops
}  // namespace mhcpb
