// Shared device code of the operators around the projection stage (embedding,
// layer norm, dropout, stream collapse and update): element types, packed
// loads and stores, the counter-based generator and block reductions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "mhcpb_check.cuh"

namespace mhcpb {
namespace ops {

constexpr unsigned kFullMask = 0xffffffffu;

// ------------------------------------------------------------ element types
template <typename E>
struct Elem;   // kPack elements make one 16-byte access
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kPack = 8;
    static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static constexpr int kPack = 8;
    static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
    static constexpr int kPack = 4;
    static __device__ __forceinline__ float to_float(float v) { return v; }
    static __device__ __forceinline__ float from_float(float v) { return v; }
};

// N consecutive elements as FP32.  N > 1: one or two 16-byte accesses, so the
// address is 16-byte aligned; N == 1: an element access.
template <typename E, int N>
__device__ __forceinline__ void load(const E* p, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = Elem<E>::to_float(*p);
    } else {
        constexpr int kPack = Elem<E>::kPack;
        static_assert(N % kPack == 0, "whole 16-byte accesses");
#pragma unroll
        for (int i = 0; i < N / kPack; ++i) {
            const uint4 raw = reinterpret_cast<const uint4*>(p)[i];
            const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
            for (int j = 0; j < kPack; ++j) v[i * kPack + j] = Elem<E>::to_float(e[j]);
        }
    }
}
template <typename E, int N>
__device__ __forceinline__ void store(E* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = Elem<E>::from_float(v[0]);
    } else {
        constexpr int kPack = Elem<E>::kPack;
        static_assert(N % kPack == 0, "whole 16-byte accesses");
#pragma unroll
        for (int i = 0; i < N / kPack; ++i) {
            uint4 raw;
            E* e = reinterpret_cast<E*>(&raw);
#pragma unroll
            for (int j = 0; j < kPack; ++j) e[j] = Elem<E>::from_float(v[i * kPack + j]);
            reinterpret_cast<uint4*>(p)[i] = raw;
        }
    }
}

// ------------------------------------------------------------ pairs
// The kernels that hold 16-byte vectors compute on pairs: one packed FP32
// instruction (fma.rn.f32x2 and the like) per two elements, each rounded as
// its scalar form.
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

template <typename E>
__device__ __forceinline__ void unpack(const uint4& raw, float2 (&v)[Elem<E>::kPack / 2]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(E) == 4) {
        v[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        v[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            } else {
                __half2 h;
                memcpy(&h, &w[i], 4);
                v[i] = __half22float2(h);
            }
        }
    }
}
template <typename E>
__device__ __forceinline__ uint4 pack(const float2 (&v)[Elem<E>::kPack / 2]) {
    uint32_t w[4];
    if constexpr (sizeof(E) == 4) {
        w[0] = __float_as_uint(v[0].x);
        w[1] = __float_as_uint(v[0].y);
        w[2] = __float_as_uint(v[1].x);
        w[3] = __float_as_uint(v[1].y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                const __nv_bfloat162 b = __float22bfloat162_rn(v[i]);
                memcpy(&w[i], &b, 4);
            } else {
                const __half2 h = __float22half2_rn(v[i]);
                memcpy(&w[i], &h, 4);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four elements: half a vector of a 16-bit type, a whole one of FP32.
template <typename E>
__device__ __forceinline__ void unpack_half(const uint2& raw, float2 (&v)[2]) {
    const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (std::is_same<E, __nv_bfloat16>::value) {
            v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            __half2 h;
            memcpy(&h, &w[i], 4);
            v[i] = __half22float2(h);
        }
    }
}
template <typename E>
__device__ __forceinline__ void pack_half(const float2 (&v)[2], uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (sizeof(E) == 4) {
            w[2 * i] = __float_as_uint(v[i].x);
            w[2 * i + 1] = __float_as_uint(v[i].y);
        } else if constexpr (std::is_same<E, __nv_bfloat16>::value) {
            const __nv_bfloat162 b = __float22bfloat162_rn(v[i]);
            memcpy(&w[i], &b, 4);
        } else {
            const __half2 h = __float22half2_rn(v[i]);
            memcpy(&w[i], &h, 4);
        }
    }
}

// [base, base + count) of one operand: what a checked build holds accesses to.
template <typename E>
struct Span {
    E* p;
    size_t count;
    // whether N elements at index i lie inside (always true in a normal build)
    __device__ __forceinline__ bool has(size_t i, int n, uint32_t site) const {
        return check::in(p + i, (size_t)n * sizeof(E), p, count * sizeof(E), site);
    }
    __device__ __forceinline__ bool holds(const E* at, int n, uint32_t site) const {
        return check::in(at, (size_t)n * sizeof(E), p, count * sizeof(E), site);
    }
};
template <int N, typename E, typename F>
__device__ __forceinline__ void load_at(const Span<E>& s, size_t i, F (&v)[N], uint32_t site) {
    if (s.has(i, N, site)) {
        load<typename std::remove_const<E>::type, N>(s.p + i, v);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.f;
    }
}
template <int N, typename E>
__device__ __forceinline__ void store_at(const Span<E>& s, size_t i, const float (&v)[N], uint32_t site) {
    if (s.has(i, N, site)) store<E, N>(s.p + i, v);
}

// One thread per vector of a row, without loops: a block holds several whole
// rows, or one of the tiles of a longer one, whichever leaves few threads idle.
// whole_warps: every warp's vectors are of one row (its last ones may lie past
// the row's end).
struct VectorPlace {
    int64_t token;
    int vector;
    bool valid;   // the thread has a vector of a token below T
};
struct VectorGrid {
    int vectors, threads, tokens, tiles;
    VectorGrid(int64_t per_row, int most, bool whole_warps) : threads(most), tokens(1), tiles(1) {
        if (whole_warps) per_row = (per_row + 31) / 32 * 32;
        vectors = (int)per_row;
        if (per_row <= most / 2) {
            tokens = most / vectors;
            return;
        }
        int64_t least = INT64_MAX;
        for (int w = 128; w <= most; w += 32) {
            const int64_t used = (per_row + w - 1) / w * w;
            if (used <= least) {
                least = used;
                threads = w;
            }
        }
        tiles = (int)((per_row + threads - 1) / threads);
    }
    unsigned blocks(int64_t T) const { return (unsigned)(tiles > 1 ? T * tiles : (T + tokens - 1) / tokens); }
    __device__ __forceinline__ VectorPlace place(int64_t T) const {
        VectorPlace p;
        if (tiles == 1) {
            p.token = (int64_t)blockIdx.x * tokens + threadIdx.x / vectors;
            p.vector = (int)(threadIdx.x % vectors);
            p.valid = threadIdx.x < tokens * vectors && p.token < T;
            if (threadIdx.x >= tokens * vectors) p.token = T;   // no row
        } else {
            p.token = blockIdx.x / tiles;
            p.vector = (int)(blockIdx.x % tiles) * (int)blockDim.x + (int)threadIdx.x;
            p.valid = p.vector < vectors;
        }
        return p;
    }
};

// ------------------------------------------------------------ generator
// Philox4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): a 128-bit counter and a 64-bit key
// give four 32-bit words, with no state between calls.
struct Words {
    uint32_t w[4];
};
__device__ __forceinline__ Words philox(uint64_t counter_lo, uint64_t counter_hi, uint64_t key) {
    uint32_t c0 = (uint32_t)counter_lo, c1 = (uint32_t)(counter_lo >> 32);
    uint32_t c2 = (uint32_t)counter_hi, c3 = (uint32_t)(counter_hi >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Words{{c0, c1, c2, c3}};
}

// Dropout of one tensor: element e (row-major index) is kept when word e % 4
// of counter (e / 4, rng[1] + sequence) under key rng[0] is >= threshold, and
// then multiplied by `scale`.
struct Drop {
    const uint64_t* rng;   // device: {key, step}; null when nothing is dropped
    uint64_t sequence;
    uint32_t threshold;    // round(p 2^32)
    float scale;           // 1 / (1 - p)
};
struct DropKey {
    uint64_t key, step;
};
__device__ __forceinline__ DropKey drop_key(const Drop& d) {
    if (d.rng == nullptr) return DropKey{0, 0};
    return DropKey{d.rng[0], d.rng[1] + d.sequence};
}
// v[k] <- dropout of element e + k; N > 1 needs e % 4 == 0.  Dropped elements
// become 0 whatever they hold (a product with 0 would keep NaN and infinity).
template <int N>
__device__ __forceinline__ void drop(const Drop& d, const DropKey& key, uint64_t e, float (&v)[N]) {
    if (d.rng == nullptr) return;
    if constexpr (N == 1) {
        const Words w = philox(e >> 2, key.step, key.key);
        const int k = (int)(e & 3);
        const uint32_t r = k == 0 ? w.w[0] : k == 1 ? w.w[1] : k == 2 ? w.w[2] : w.w[3];
        v[0] = r >= d.threshold ? v[0] * d.scale : 0.f;
    } else {
        static_assert(N % 4 == 0, "whole counters");
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const Words w = philox((e >> 2) + i, key.step, key.key);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[i * 4 + j] = w.w[j] >= d.threshold ? v[i * 4 + j] * d.scale : 0.f;
        }
    }
}

// The same words where the counter's low half fits 32 bits (fewer than 2^34
// elements): the first two rounds' products that do not depend on the element
// are formed once per thread, 18 multiplications a counter instead of 20.
struct ShortPhilox {
    uint32_t k0, k1;      // key
    uint32_t c3;          // high word of the step
    uint32_t r1_lo;       // round 1: low word of the step's product
    uint32_t r2_hi, r2_lo;// round 2: product of round 1's first word, which no element enters
    __device__ __forceinline__ explicit ShortPhilox(const DropKey& d) {
        // The key is the same in every lane; a warp reduction says so to the
        // compiler, which then keeps the key schedule off the vector units.
        k0 = __reduce_or_sync(__activemask(), (uint32_t)d.key);
        k1 = __reduce_or_sync(__activemask(), (uint32_t)(d.key >> 32));
        c3 = __reduce_or_sync(__activemask(), (uint32_t)(d.step >> 32));
        const uint64_t b = (uint64_t)__reduce_or_sync(__activemask(), (uint32_t)d.step) * 0xCD9E8D57u;
        r1_lo = (uint32_t)b;
        const uint64_t a = (uint64_t)((uint32_t)(b >> 32) ^ k0) * 0xD2511F53u;
        r2_hi = (uint32_t)(a >> 32);
        r2_lo = (uint32_t)a;
    }
    // words of counters i[g], i[g] + 1, ... (COUNT each), all together, so that they share the key schedule
    template <int GROUPS, int COUNT>
    __device__ __forceinline__ void words(const uint32_t (&i)[GROUPS], uint32_t (&w)[GROUPS][COUNT][4]) const {
        uint32_t a0 = k0 + 0x9E3779B9u, a1 = k1 + 0xBB67AE85u;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int n = 0; n < COUNT; ++n) {
                const uint64_t a = (uint64_t)(i[g] + n) * 0xD2511F53u;
                const uint64_t b = (uint64_t)((uint32_t)(a >> 32) ^ c3 ^ k1) * 0xCD9E8D57u;
                w[g][n][0] = (uint32_t)(b >> 32) ^ r1_lo ^ a0;
                w[g][n][1] = (uint32_t)b;
                w[g][n][2] = r2_hi ^ (uint32_t)a ^ a1;
                w[g][n][3] = r2_lo;
            }
#pragma unroll
        for (int r = 2; r < 10; ++r) {
            a0 += 0x9E3779B9u;
            a1 += 0xBB67AE85u;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int n = 0; n < COUNT; ++n) {
                    const uint64_t a = (uint64_t)w[g][n][0] * 0xD2511F53u, b = (uint64_t)w[g][n][2] * 0xCD9E8D57u;
                    w[g][n][0] = (uint32_t)(b >> 32) ^ w[g][n][1] ^ a0;
                    w[g][n][1] = (uint32_t)b;
                    w[g][n][2] = (uint32_t)(a >> 32) ^ w[g][n][3] ^ a1;
                    w[g][n][3] = (uint32_t)a;
                }
        }
    }
};

// ------------------------------------------------------------ reductions
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
// Two values at once: lanes below 16 end with the sum of a, the others with b's.
__device__ __forceinline__ float warp_sum_two(float a, float b) {
    const bool high = threadIdx.x & 16;
    float v = (high ? b : a) + __shfl_xor_sync(kFullMask, high ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
// Four values: lanes 8 j .. 8 j + 7 end with the sum of v[j].  The first steps
// halve what a lane carries, so 6 shuffles do instead of 20.
__device__ __forceinline__ float warp_sum_four(const float (&v)[4]) {
    const bool high = threadIdx.x & 16, mid = threadIdx.x & 8;
    const float a = (high ? v[2] : v[0]) + __shfl_xor_sync(kFullMask, high ? v[0] : v[2], 16);
    const float b = (high ? v[3] : v[1]) + __shfl_xor_sync(kFullMask, high ? v[1] : v[3], 16);
    float s = (mid ? b : a) + __shfl_xor_sync(kFullMask, mid ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    return s;
}
// Sixteen values: lanes 2 k and 2 k + 1 end with the sum of v[k] (16 shuffles).
__device__ __forceinline__ float warp_sum_sixteen(float (&v)[16]) {
#pragma unroll
    for (int half = 8, o = 16; half > 0; half >>= 1, o >>= 1) {
        const bool high = threadIdx.x & o;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float keep = high ? v[half + k] : v[k], give = high ? v[k] : v[half + k];
            v[k] = keep + __shfl_xor_sync(kFullMask, give, o);
        }
    }
    return v[0] + __shfl_xor_sync(kFullMask, v[0], 1);
}
// Sums N values over the block in a fixed order; every thread gets them.
// scratch: N * 32 floats of shared memory, free again after the call.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) scratch[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? scratch[i * 32 + lane] : 0.f);
    __syncthreads();
}

}  // namespace ops
}  // namespace mhcpb
