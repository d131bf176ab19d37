// Rows whose addresses are not multiples of 16 bytes.
//
// A row is still read and written in whole aligned 16-byte chunks: a vector of
// kPack columns that starts m elements into a chunk lies in that chunk and the
// next, and is put together from both with selects and funnel shifts.  A chunk
// may hold elements of the neighbouring rows (read, never used); the chunks
// that stick out of the operand itself, in its first and last row, are read
// element by element.
#pragma once
#include "mhcs_common.cuh"
#include "mhcs_ring.cuh"

namespace mhcpb {
namespace ops {

// Elements between the 16-byte boundary below p and p.
template <typename E>
__device__ __forceinline__ int misaligned(const E* p) {
    return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(E)) & (Elem<E>::kPack - 1);
}

// Elements m .. m + kPack - 1 of a followed by b, 0 <= m <= kPack.
template <typename E>
__device__ __forceinline__ uint4 shift_take(const uint4& a, const uint4& b, int m) {
    uint32_t w[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0u};
    const int words = sizeof(E) == 4 ? m : m >> 1;
    if (words & 4)
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 4];
    if (words & 2)
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    if (words & 1)
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    if constexpr (sizeof(E) == 2) {
        const uint32_t bits = (m & 1) * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first `valid` elements of v, the others 0.
template <typename E>
__device__ __forceinline__ uint4 keep_first(const uint4& v, int valid) {
    constexpr int per_word = 4 / (int)sizeof(E);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int left = valid - k * per_word;
        w[k] = left <= 0 ? 0u : left >= per_word ? w[k] : w[k] & 0xffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A chunk that is not wholly inside the operand, element by element.
template <typename E>
__device__ __noinline__ uint4 edge_chunk(const E* p, size_t count, ptrdiff_t first, uint32_t site) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    E* const e = reinterpret_cast<E*>(&v);
    for (int k = 0; k < Elem<E>::kPack; ++k) {
        const ptrdiff_t at = first + k;
        if (at >= 0 && at < (ptrdiff_t)count && check::in(p + at, sizeof(E), p, count * sizeof(E), site)) e[k] = p[at];
    }
    return v;
}
template <typename E>
__device__ __forceinline__ bool whole_chunk(const Span<const E>& in, ptrdiff_t first) {
    return first >= 0 && first + Elem<E>::kPack <= (ptrdiff_t)in.count;
}

// A lane's share of a row of `width` columns for vectors of which the lane's
// starts at element `at`, column c: its chunk, and lane 31's next one too.  The
// warp's slots are 33 in a row.  Only the operand's first and last row can
// have chunks that stick out of it: `edge` says that this is one of them.
template <typename E>
__device__ __forceinline__ void copy_shifted(uint4* slot, const Span<const E>& in, size_t at, int c, int width,
                                             uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    const int m = misaligned(in.p + at);
    const size_t first = at - m;
    if (c - m < width && in.has(first, kPack, site)) copy16(slot, in.p + first);
    if ((threadIdx.x & 31) == 31 && m > 0 && c + kPack - m < width && in.has(first + kPack, kPack, site))
        copy16(slot + 1, in.p + first + kPack);
}
template <typename E>
__device__ __noinline__ void copy_shifted_edge(uint4* slot, const E* p, size_t count, size_t at, int c, int width,
                                               uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    const int m = misaligned(p + at);
    if (c - m < width) slot[0] = edge_chunk(p, count, (ptrdiff_t)at - m, site);
    if ((threadIdx.x & 31) == 31 && m > 0 && c + kPack - m < width)
        slot[1] = edge_chunk(p, count, (ptrdiff_t)at - m + kPack, site);
}
// The lane's vector in place of its chunk, columns past the row 0.  The whole
// warp, after its copies have arrived and a __syncwarp.
template <typename E>
__device__ __forceinline__ void realign(uint4* slot, int m, int valid) {
    uint4 v = slot[0];
    if (m > 0) v = shift_take<E>(v, slot[1], m);   // m is the same in every lane
    if (valid < Elem<E>::kPack) v = keep_first<E>(v, valid);
    __syncwarp();
    slot[0] = v;
}

// The vector at element `at` of which `valid` columns belong to the row (the
// others come back as 0).  CHECKED: it may lie in the operand's first or last
// chunk; otherwise its chunks are known to be inside.
template <bool CHECKED, typename E>
__device__ __forceinline__ uint4 load_shifted(const Span<const E>& in, size_t at, int valid, uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    const int m = misaligned(in.p + at);
    const auto chunk = [&](ptrdiff_t f) {
        if (!CHECKED || whole_chunk(in, f))
            return in.has((size_t)f, kPack, site) ? *reinterpret_cast<const uint4*>(in.p + f) : make_uint4(0u, 0u, 0u, 0u);
        return edge_chunk(in.p, in.count, f, site);
    };
    const ptrdiff_t first = (ptrdiff_t)at - m;
    uint4 a = chunk(first), b = make_uint4(0u, 0u, 0u, 0u);
    if (m > 0 && valid > kPack - m) b = chunk(first + kPack);
    a = shift_take<E>(a, b, m);
    return valid < kPack ? keep_first<E>(a, valid) : a;
}

// Stores the lane's vector at element `at`, `valid` columns of it (all lanes of
// the warp).  `before`: the lane below holds the vector of the columns before;
// `after`: the lane above the one after.  A lane writes the whole chunk its
// vector starts in, with the lower lane's last elements; what no whole chunk
// covers is written element by element.
template <typename E>
__device__ __forceinline__ void store_shifted(const Span<E>& out, size_t at, int valid, bool before, bool after,
                                              const uint4& own, uint32_t site) {
    constexpr int kPack = Elem<E>::kPack;
    uint4 low;
    low.x = __shfl_up_sync(kFullMask, own.x, 1);
    low.y = __shfl_up_sync(kFullMask, own.y, 1);
    low.z = __shfl_up_sync(kFullMask, own.z, 1);
    low.w = __shfl_up_sync(kFullMask, own.w, 1);
    if (valid <= 0) return;
    const int m = misaligned(out.p + at), head = kPack - m;   // own elements of the first chunk
    int from = 0, to = valid < kPack ? valid : kPack;         // elements left for single stores
    if (m == 0) {
        if (valid >= kPack) {
            if (out.has(at, kPack, site)) *reinterpret_cast<uint4*>(out.p + at) = own;
            return;
        }
    } else {
        if (before && valid >= head) {
            if (out.has(at - m, kPack, site)) *reinterpret_cast<uint4*>(out.p + at - m) = shift_take<E>(low, own, head);
            from = head;
        }
        if (after && valid - kPack >= head) to = head;   // the lane above writes the rest
    }
    if (from >= to) return;
    const E* const e = reinterpret_cast<const E*>(&own);
#pragma unroll
    for (int k = 0; k < kPack; ++k)
        if (k >= from && k < to && out.has(at + k, 1, site)) out.p[at + k] = e[k];
}

}  // namespace ops
}  // namespace mhcpb
