// Dropout, and the residual streams' update with its gradient.
//
//   dropout          y_e = kept_e ? x_e / (1 - p) : 0
//   update           X'_i = sum_j H_res[i][j] X_j + H_post[i] drop(y)        i, j < 4
//   its gradient     dy = drop(sum_i H_post[i] dX'_i)
//                    dH_post[i] = <dX'_i, drop(y)>,  dH_res[i][j] = <dX'_i, X_j>
//
// FP32 arithmetic, one rounding to BF16 at each store.  The mask is drawn
// again from the counter wherever it is needed, so it takes no memory.  4, 18
// and 20 bytes per BF16 element of y: the update and its gradient are bound by
// HBM, dropout of a 16-bit type by the generator.  Fractions are of the 6.77
// TB/s that a plain copy reaches; "replayed" times are calls captured in a
// graph, without the host's share.
#include "mhcs_common.cuh"
#include "mhcs_internal.h"
#include "mhcs_ring.cuh"
#include "mhcs_words.cuh"
#include "ptx.cuh"

namespace mhcpb {
namespace ops {
namespace streams {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr int64_t kShortCounters = (int64_t)1 << 34;   // elements below which ShortPhilox serves
constexpr int kMaxShared = 227 * 1024;   // shared memory of a block

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tensors that do not begin on a 16-byte boundary, and of 2^34 elements and more:
// the four elements of a counter per thread and step.  4096 x 5120 BF16, one
// element off: 35 us; on the boundary, below: 18.
template <typename E>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(int64_t n, Span<const E> x, Span<E> y, Drop d) {
    ptx::grid_dependency_wait();
    const DropKey key = drop_key(d);
    const int64_t step = (int64_t)gridDim.x * kThreads * 4;
    for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; e < n; e += step) {
        const int here = n - e < 4 ? (int)(n - e) : 4;
        float v[4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < here && x.has(e + k, 1, 0)) v[k] = Elem<E>::to_float(x.p[e + k]);
        drop<4>(d, key, e, v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < here && y.has(e + k, 1, 1)) y.p[e + k] = Elem<E>::from_float(v[k]);
    }
}

// kDropPacks vectors of 16 bytes per thread, a block's width apart; needs
// n < kShortCounters and aligned pointers.  The last, partial vector is one thread's.
// T=16384, D=5120 BF16: 68.4 us (72%), T=4096 18.3 (68%).  FP32, with twice the bytes
// per counter, runs at HBM's rate (T=8192: 48.6 us), so it is the generator's
// arithmetic that the 16-bit types wait for, but no one unit is full: in a
// capture at T=4096 the pipe that multiplies is busy 57% of the time, the other
// integer pipe 49%, the issue slots 50%, DRAM 27%, with 24 warps on an SM (80
// registers a thread).  The BF16 kernel spills 20 bytes a thread (28 loaded).
// A thread's vectors share the key schedule; 1, 2, 4, 8 vectors: 77.3,
// 70.9, 68.6, 83.4 us.
constexpr int kDropPacks = 4;
template <typename E>
__global__ void __launch_bounds__(kThreads) dropout_kernel(int64_t n, Span<const E> x, Span<E> y, Drop d) {
    ptx::grid_dependency_wait();
    constexpr int N = Elem<E>::kPack;
    const DropKey key = drop_key(d);
    const int64_t first = ((int64_t)blockIdx.x * kDropPacks * kThreads + threadIdx.x) * N;
    uint4 raw[kDropPacks];
#pragma unroll
    for (int v = 0; v < kDropPacks; ++v) {
        const int64_t e = first + (int64_t)v * kThreads * N;
        if (e + N <= n && x.has(e, N, 0)) raw[v] = *reinterpret_cast<const uint4*>(x.p + e);
    }
    const ShortPhilox random(key);
    const float2 scale = pair(d.scale);
    uint32_t w[kDropPacks][N / 4][4];
    if (d.rng != nullptr) {
        uint32_t counters[kDropPacks];
#pragma unroll
        for (int v = 0; v < kDropPacks; ++v) counters[v] = (uint32_t)((first + (int64_t)v * kThreads * N) >> 2);
        random.words<kDropPacks, N / 4>(counters, w);
    }
#pragma unroll
    for (int v = 0; v < kDropPacks; ++v) {
        const int64_t e = first + (int64_t)v * kThreads * N;
        if (e + N <= n) {
            float2 f[N / 2];
            unpack<E>(raw[v], f);
            if (d.rng != nullptr) {
#pragma unroll
                for (int k = 0; k < N / 2; ++k) {
                    f[k] = mul2(f[k], scale);
                    f[k].x = w[v][k / 2][k % 2 * 2] >= d.threshold ? f[k].x : 0.f;
                    f[k].y = w[v][k / 2][k % 2 * 2 + 1] >= d.threshold ? f[k].y : 0.f;
                }
            }
            if (y.has(e, N, 1)) *reinterpret_cast<uint4*>(y.p + e) = pack<E>(f);
        } else {
            for (int64_t i = e; i < n; ++i) {
                float one[1];
                load_at<1>(x, i, one, 0);
                drop<1>(d, key, i, one);
                store_at<1>(y, i, one, 1);
            }
        }
    }
}

// The gates of token t: 4 of H_post and 16 of H_res.
__device__ __forceinline__ void gates_at(const Span<const float>& h, int64_t t, bool aligned, float (&g)[20]) {
    if (aligned) {
#pragma unroll
        for (int q = 0; q < 5; ++q) {
            const size_t at = (size_t)t * kGates + 4 + 4 * q;
            const float4 v = h.has(at, 4, 2) ? *reinterpret_cast<const float4*>(h.p + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            g[4 * q] = v.x;
            g[4 * q + 1] = v.y;
            g[4 * q + 2] = v.z;
            g[4 * q + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 20; ++q) {
            const size_t at = (size_t)t * kGates + 4 + q;
            g[q] = h.has(at, 1, 2) ? h.p[at] : 0.f;
        }
    }
}
// One column of a token; gate: H_post and H_res.
__device__ __forceinline__ void update_column(int64_t t, int64_t c, int64_t D, const float* gate, const Span<const bf16>& x,
                                              const Span<const bf16>& y, const Drop& d, const DropKey& key,
                                              const Span<bf16>& x_out) {
    float xs[kStreams][1], yv[1];
    load_at<1>(y, t * D + c, yv, 3);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) load_at<1>(x, (t * kStreams + j) * D + c, xs[j], 4);
    drop<1>(d, key, (uint64_t)(t * D + c), yv);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
        float o[1] = {gate[i] * yv[0]};
#pragma unroll
        for (int j = 0; j < kStreams; ++j) o[0] = fmaf(gate[4 + 4 * i + j], xs[j][0], o[0]);
        store_at<1>(x_out, (t * kStreams + i) * D + c, o, 5);
    }
}

// Rows at any address and of any size, one block per token, a column of every
// stream per thread and step.  For short odd rows, where putting vectors
// together costs more than it saves: D=63 (T=32768) 30.0 us here and 48.5 with
// vectors, D=127 (T=16384) 21.7 and 26.4, D=129 25.2 and 24.7, D=255 35.6 and
// 26.4.
__global__ void __launch_bounds__(kThreads) update_forward_any_kernel(int64_t D, Span<const bf16> x,
                                                                      Span<const bf16> y, Span<const float> h,
                                                                      Drop d, Span<bf16> x_out) {
    ptx::grid_dependency_wait();
    const int64_t t = blockIdx.x;
    float gate[20];
    gates_at(h, t, false, gate);
    const DropKey key = drop_key(d);
    for (int64_t c = threadIdx.x; c < D; c += kThreads) update_column(t, c, D, gate, x, y, d, key, x_out);
}

// Tokens of more columns than update_backward_tokens_kernel takes (10,240; not
// aligned: 8,192).  T=2048, D=10240 takes 296 us here, 84 there.
__global__ void __launch_bounds__(kThreads) update_backward_any_kernel(int64_t D, Span<const bf16> x,
                                                                   Span<const bf16> y, Span<const float> h,
                                                                   Drop d, Span<const bf16> gout,
                                                                   Span<bf16> gy, Span<float> gh) {
    ptx::grid_dependency_wait();
    constexpr int N = 1;
    __shared__ float post[kStreams];
    __shared__ float scratch[20 * 32];
    const int64_t t = blockIdx.x;
    if (threadIdx.x < kStreams) {
        float v[1];
        load_at<1>(h, t * kGates + 4 + threadIdx.x, v, 2);
        post[threadIdx.x] = v[0];
    }
    __syncthreads();
    const DropKey key = drop_key(d);
    const int64_t row = t * kStreams * D;
    float dot[20];   // 4 of dH_post, 16 of dH_res
#pragma unroll
    for (int i = 0; i < 20; ++i) dot[i] = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * N; c < D; c += kThreads * N) {
        float xs[kStreams][N], go[kStreams][N], yv[N], o[N];
        load_at<N>(y, t * D + c, yv, 3);
#pragma unroll
        for (int j = 0; j < kStreams; ++j) {
            load_at<N>(x, row + j * D + c, xs[j], 4);
            load_at<N>(gout, row + j * D + c, go[j], 6);
        }
        drop<N>(d, key, (uint64_t)(t * D + c), yv);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            o[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kStreams; ++i) {
                o[k] = fmaf(post[i], go[i][k], o[k]);
                dot[i] = fmaf(go[i][k], yv[k], dot[i]);
#pragma unroll
                for (int j = 0; j < kStreams; ++j)
                    dot[4 + 4 * i + j] = fmaf(go[i][k], xs[j][k], dot[4 + 4 * i + j]);
            }
        }
        drop<N>(d, key, (uint64_t)(t * D + c), o);
        store_at<N>(gy, t * D + c, o, 7);
    }
    block_sum<20>(dot, scratch);
    if (threadIdx.x < 20) {
        float v[1] = {0.f};
#pragma unroll
        for (int i = 0; i < 20; ++i)
            if (threadIdx.x == i) v[0] = dot[i];
        store_at<1>(gh, t * kGates + 4 + threadIdx.x, v, 8);
    }
}

// ------------------------------------------------------------ update, 16-byte vectors
// f <- dropout of the eight elements from e on; *keep: which are kept.  ANY: e
// need not be a multiple of 4, so the eight words come from three counters.
template <bool ANY>
__device__ __forceinline__ void drop_eight(const Drop& d, const ShortPhilox& random, uint64_t e, float2 (&f)[4],
                                           uint32_t* keep) {
    *keep = 0xffu;
    if (d.rng == nullptr) return;
    constexpr int kCounters = ANY ? 3 : 2;
    uint32_t w[1][kCounters][4];
    const uint32_t counter[1] = {(uint32_t)(e >> 2)};
    random.words<1, kCounters>(counter, w);
    uint32_t bits = 0u;
#pragma unroll
    for (int k = 0; k < 4 * kCounters; ++k) bits |= (w[0][k / 4][k % 4] >= d.threshold ? 1u : 0u) << k;
    if (ANY) bits >>= (uint32_t)e & 3u;
    *keep = bits & 0xffu;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k] = mul2(f[k], pair(d.scale));
        f[k].x = bits >> (2 * k) & 1u ? f[k].x : 0.f;
        f[k].y = bits >> (2 * k + 1) & 1u ? f[k].y : 0.f;
    }
}

// One vector of every stream per thread, everything loaded before anything is
// used: five loads per thread keep enough on their way, and nothing is shared
// between threads.  T=4096, D=5120 with dropout: 60.8 us (92%), T=16384 233
// (96%); one token 1.6 us replayed, an empty launch's time.  WORDS: rows at any
// address (mhcs_words.cuh), D of any size (T=4096, D=1285: 33 us).
template <bool WORDS>
__global__ void __launch_bounds__(kThreads) update_forward_vectors_kernel(
    int64_t T, int64_t D, VectorGrid grid, bool gates_aligned, Span<const bf16> x, Span<const bf16> y,
    Span<const float> h, Drop d, Span<bf16> x_out) {
    constexpr int N = 8, H = 4;
    __shared__ uint4 parts[WORDS ? kThreads / 32 * (kStreams + 1) * kWarpSlots : 1];
    ptx::grid_dependency_wait();
    const VectorPlace place = grid.place(T);
    const int64_t t = place.token;
    const int c = place.vector * N, lane = threadIdx.x & 31;
    const size_t row = (size_t)t * (kStreams * D) + c, flat = (size_t)t * D + c;
    uint4 xs[kStreams], yr;
    float g[20];
    if constexpr (!WORDS) {
        if (!place.valid) return;
        yr = y.has(flat, N, 3) ? *reinterpret_cast<const uint4*>(y.p + flat) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < kStreams; ++j)
            xs[j] = x.has(row + j * D, N, 4) ? *reinterpret_cast<const uint4*>(x.p + row + j * D) : make_uint4(0u, 0u, 0u, 0u);
        gates_at(h, t, gates_aligned, g);
    } else {
        // a warp's vectors are all of one token (VectorGrid's whole warps)
        if (t >= T) return;
        uint4* const mine = parts + (threadIdx.x >> 5) * ((kStreams + 1) * kWarpSlots);
        const int width = (int)D - c + lane * N;
        const size_t row0 = row - lane * N, flat0 = flat - lane * N;
        if (edge_row<bf16>(t, T, D)) {
#pragma unroll 1
            for (int j = 0; j <= kStreams; ++j)
                copy_edge(mine + j * kWarpSlots, j < kStreams ? x.p : y.p, j < kStreams ? x.count : y.count,
                              j < kStreams ? row0 + j * D : flat0, width, 4);
        } else {
            copy_chunks(mine + kStreams * kWarpSlots, y, flat0, width, 3);
#pragma unroll
            for (int j = 0; j < kStreams; ++j) copy_chunks(mine + j * kWarpSlots, x, row0 + j * D, width, 4);
        }
        copies_commit();
        gates_at(h, t, gates_aligned, g);
        copies_wait<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kStreams; ++j) {
            align_chunks<bf16>(mine + j * kWarpSlots, misaligned(x.p + row0 + j * D), (int)D - c);
            xs[j] = mine[j * kWarpSlots + lane];
        }
        align_chunks<bf16>(mine + kStreams * kWarpSlots, misaligned(y.p + flat0), (int)D - c);
        yr = mine[kStreams * kWarpSlots + lane];
        __syncwarp();
    }
    const DropKey key = drop_key(d);
    float2 yv[H], o[kStreams][H];
    uint32_t keep;
    unpack<bf16>(yr, yv);
    drop_eight<WORDS>(d, ShortPhilox(key), flat, yv, &keep);
#pragma unroll
    for (int i = 0; i < kStreams; ++i)
#pragma unroll
        for (int k = 0; k < H; ++k) o[i][k] = mul2(pair(g[i]), yv[k]);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) {
        float2 v[H];
        unpack<bf16>(xs[j], v);
#pragma unroll
        for (int i = 0; i < kStreams; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) o[i][k] = fma2(pair(g[4 + 4 * i + j]), v[k], o[i][k]);
    }
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
        if constexpr (WORDS) {
            store_words(parts + (threadIdx.x >> 5) * ((kStreams + 1) * kWarpSlots), x_out, row - lane * N + i * D,
                        (int)D - c + lane * N, pack<bf16>(o[i]), 5);
        } else {
            if (x_out.has(row + i * D, N, 5)) *reinterpret_cast<uint4*>(x_out.p + row + i * D) = pack<bf16>(o[i]);
        }
    }
}

// A group of G threads takes a token at a time (thread i owns vectors i, i + G,
// ... of it, VPT of them), its inputs copied S tokens ahead into per-thread
// slots.  The token's 20 dot products are left in shared memory by each warp
// and added up after the group's barrier, which the outputs do not wait for.
// T=4096, D=5120 with dropout: 67.8 us (91%), T=16384 255 (97%): HBM's rate.  The
// products are packed over pairs of the gradient's streams, so that 20 sums
// take 10 register pairs and half the instructions (one sum at a time: 73.0 and
// 276 us; pairs of columns would take 20 registers more).  Shapes, measured
// before that, T=4096: 1 vector, 2 tokens ahead, 640 threads: D=5120 73.5 us,
// T=16384 277; 2 vectors, 1 ahead, 512 threads: 77.6 and 294, D=8192 100.9 (now
// 99.5, 100%); 2 vectors by 640 threads: D=8192 131 (it spills 20 bytes a
// thread, 28 loaded), kept for up to 10,240 columns.  Two unaligned vectors spill 8 / 12.  Short odd rows stay here: T=65536, D=7 takes 134 us, element
// by element 454.
template <bool WORDS, int VPT, int S, int MAX>
struct TokenShape {
    static constexpr int kMaxThreads = MAX;            // 640: 96 registers a thread; 512: 128
    static constexpr int kArrays = 2 * kStreams + 1;   // x, grad_x_out, y
    static constexpr int kStage = VPT * kArrays;
    static constexpr int kPitch = WORDS ? MAX / 32 * kWarpSlots : MAX;
    static constexpr int kDots = 20;
    static size_t bytes(int G, int R) {
        return (size_t)kPitch * S * kStage * 16 + (size_t)R * ((G / 32 * S * 4 + 2 * kDots * (G / 32 | 1)) * 4) +
               (WORDS ? 16 + (size_t)R * G * 16 : 0);   // what a warp stores
    }
};
template <bool WORDS, int VPT, int S, int MAX>
__global__ void __launch_bounds__(MAX, 1)
    update_backward_tokens_kernel(int T, int D, int G, int R, Span<const bf16> x, Span<const bf16> y,
                                  Span<const float> h, Drop d, Span<const bf16> gout, Span<bf16> gy, Span<float> gh) {
    using Shape = TokenShape<WORDS, VPT, S, MAX>;
    constexpr int N = 8, P = Shape::kPitch, A = Shape::kArrays;
    extern __shared__ uint4 slots[];
    const int NT = G * R, tid = threadIdx.x, group = tid / G, i = tid - group * G, lane = tid & 31;
    const int warp = i >> 5, warps = G >> 5;
    uint4* const mine = slots + (WORDS ? (tid >> 5) * kWarpSlots + lane : tid);
    float* const floats = reinterpret_cast<float*>(slots + P * S * Shape::kStage);
    float* const posts = floats + (tid >> 5) * (S * 4);                                   // [S][4] per warp
    float* const dots = floats + (NT >> 5) * (S * 4) + group * (2 * Shape::kDots * (warps | 1));
    uint4* buffer = nullptr;   // WORDS: what the warp stores, on the next 16-byte boundary
    if (WORDS)
        buffer = slots + P * S * Shape::kStage + (((NT >> 5) * (S * 4) + R * (2 * Shape::kDots * (warps | 1))) + 3) / 4 +
                 (tid >> 5) * 32;
    const int dot_pitch = warps | 1;   // odd: the 20 lanes that read a column meet 20 banks
    const int groups = (int)gridDim.x * R, first = (int)blockIdx.x * R + group;
    const int c0 = i * N, step = G * N;
    // columns past D: never copied, they stay 0 and add nothing
#pragma unroll
    for (int k = 0; k < S * Shape::kStage; ++k)
        if (!WORDS && c0 + k % Shape::kStage / A * step >= D) mine[k * P] = make_uint4(0u, 0u, 0u, 0u);
    ptx::grid_dependency_wait();

    const auto fetch_vector = [&](uint4* dst, int t, int v) {
        const int c = c0 + v * step;
        const size_t flat = (size_t)((uint64_t)(uint32_t)t * (uint32_t)D + (uint32_t)c);
        const size_t row = (size_t)((uint64_t)(uint32_t)t * (uint32_t)(kStreams * D) + (uint32_t)c);
        if constexpr (WORDS) {
            const int width = D - c + lane * N;   // from the warp's first column on
            uint4* const warps_dst = dst - lane;
            if (edge_row<bf16>(t, T, D)) {
#pragma unroll 1
                for (int s = 0; s < A; ++s) {
                    const Span<const bf16>& in = s < kStreams ? x : s < 2 * kStreams ? gout : y;
                    const size_t at = s < 2 * kStreams ? row + (s % kStreams) * D : flat;
                    copy_edge(warps_dst + (v * A + s) * P, in.p, in.count, at - lane * N, width, 4);
                }
                return;
            }
#pragma unroll
            for (int s = 0; s < kStreams; ++s) {
                copy_chunks(warps_dst + (v * A + s) * P, x, row - lane * N + s * D, width, 4);
                copy_chunks(warps_dst + (v * A + kStreams + s) * P, gout, row - lane * N + s * D, width, 6);
            }
            copy_chunks(warps_dst + (v * A + 2 * kStreams) * P, y, flat - lane * N, width, 3);
        } else if (c < D) {
#pragma unroll
            for (int s = 0; s < kStreams; ++s) {
                if (x.has(row + s * D, N, 4)) copy16(dst + (v * A + s) * P, x.p + row + s * D);
                if (gout.has(row + s * D, N, 6)) copy16(dst + (v * A + kStreams + s) * P, gout.p + row + s * D);
            }
            if (y.has(flat, N, 3)) copy16(dst + (v * A + 2 * kStreams) * P, y.p + flat);
        }
    };
    const auto fetch_post = [&](int t, int stage) {
        if (lane < kStreams && h.has((size_t)t * kGates + 4 + lane, 1, 2))
            copy4(posts + stage * 4 + lane, h.p + (size_t)t * kGates + 4 + lane);
    };
    const auto write_dots = [&](int t, int parity) {
        if (warp == 0 && lane < Shape::kDots) {
            const float* const p = dots + (parity * Shape::kDots + lane) * dot_pitch;
            float v[1] = {0.f};
            for (int w = 0; w < warps; ++w) v[0] += p[w];
            store_at<1>(gh, (size_t)t * kGates + 4 + lane, v, 8);
        }
    };
#pragma unroll
    for (int q = 0; q < S; ++q) {
        if (first + q * groups < T) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) fetch_vector(mine + q * (Shape::kStage * P), first + q * groups, v);
            fetch_post(first + q * groups, q);
        }
        copies_commit();
    }
    const DropKey key = drop_key(d);   // after the first copies are on their way
    const ShortPhilox random(key);
    int stage = 0, parity = 0;
    for (int t = first; t < T; t += groups) {
        copies_wait<S - 1>();
        __syncwarp();
        uint4* const row = mine + stage * (Shape::kStage * P);
        if constexpr (WORDS)
#pragma unroll
            for (int k = 0; k < Shape::kStage; ++k) {
                const int s = k % A;   // x, grad_x_out or y
                const bf16* const p = s < kStreams ? x.p + (size_t)t * (kStreams * D) + s * D
                                      : s < 2 * kStreams ? gout.p + (size_t)t * (kStreams * D) + (s - kStreams) * D
                                                         : y.p + (size_t)t * D;
                align_chunks<bf16>(row - lane + k * P, misaligned(p), D - (c0 + k / A * step));
            }
        const float4 post = *reinterpret_cast<const float4*>(posts + stage * 4);
        const float p4[kStreams] = {post.x, post.y, post.z, post.w};
        const bool more = t + S * groups < T;
        // pairs of streams i: the dot products of dX'_2q and dX'_2q+1 with X_j and y
        float2 d16p[2][kStreams], d4p[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            d4p[q] = pair(0.f);
#pragma unroll
            for (int j = 0; j < kStreams; ++j) d16p[q][j] = pair(0.f);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = c0 + v * step;
            const size_t flat = (size_t)((uint64_t)(uint32_t)t * (uint32_t)D + (uint32_t)c);
            float2 yv[4];
            uint32_t keep, out[4];
            unpack<bf16>(row[(v * A + 2 * kStreams) * P], yv);
            drop_eight<WORDS>(d, random, flat, yv, &keep);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float2 xs[kStreams][2], g[kStreams][2], o[2];
#pragma unroll
                for (int j = 0; j < kStreams; ++j) {
                    unpack_half<bf16>(reinterpret_cast<const uint2*>(row + (v * A + j) * P)[half], xs[j]);
                    unpack_half<bf16>(reinterpret_cast<const uint2*>(row + (v * A + kStreams + j) * P)[half], g[j]);
                }
                const auto column = [&](const float2 (&f)[2], int k) { return k & 1 ? f[k >> 1].y : f[k >> 1].x; };
                float oc[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 sum = pair(0.f);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 gq = make_float2(column(g[2 * q], k), column(g[2 * q + 1], k));
                        sum = fma2(make_float2(p4[2 * q], p4[2 * q + 1]), gq, sum);
                        d4p[q] = fma2(gq, pair(k & 1 ? yv[half * 2 + (k >> 1)].y : yv[half * 2 + (k >> 1)].x), d4p[q]);
#pragma unroll
                        for (int j = 0; j < kStreams; ++j) d16p[q][j] = fma2(gq, pair(column(xs[j], k)), d16p[q][j]);
                    }
                    oc[k] = sum.x + sum.y;
                }
                o[0] = make_float2(oc[0], oc[1]);
                o[1] = make_float2(oc[2], oc[3]);
                if (d.rng != nullptr)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        o[k] = mul2(o[k], pair(d.scale));
                        o[k].x = keep >> (half * 4 + 2 * k) & 1u ? o[k].x : 0.f;
                        o[k].y = keep >> (half * 4 + 2 * k + 1) & 1u ? o[k].y : 0.f;
                    }
                pack_half<bf16>(o, out + half * 2);
            }
            const uint4 packed = make_uint4(out[0], out[1], out[2], out[3]);
            if constexpr (WORDS) {
                store_words(buffer, gy, flat - lane * N, D - c + lane * N, packed, 7);
            } else {
                if (c < D && gy.has(flat, N, 7)) *reinterpret_cast<uint4*>(gy.p + flat) = packed;
            }
            if (more) fetch_vector(row, t + S * groups, v);
        }
        float d16[16];
        const float d4[4] = {d4p[0].x, d4p[0].y, d4p[1].x, d4p[1].y};
#pragma unroll
        for (int j = 0; j < kStreams; ++j) {
            d16[j] = d16p[0][j].x;
            d16[4 + j] = d16p[0][j].y;
            d16[8 + j] = d16p[1][j].x;
            d16[12 + j] = d16p[1][j].y;
        }
        const float res = warp_sum_sixteen(d16), pos = warp_sum_four(d4);
        float* const mine_dots = dots + parity * (Shape::kDots * dot_pitch) + warp;
        if ((lane & 1) == 0) mine_dots[(4 + (lane >> 1)) * dot_pitch] = res;
        if ((lane & 7) == 0) mine_dots[(lane >> 3) * dot_pitch] = pos;
        __syncwarp();   // every lane has read the token's gates
        if (more) fetch_post(t + S * groups, stage);
        copies_commit();
        // The other parity's sums are read after the barrier two tokens later at
        // the earliest, so one barrier per token orders both buffers.
        group_sync(group, G);
        write_dots(t, parity);
        stage = stage + 1 == S ? 0 : stage + 1;
        parity ^= 1;
    }
    copies_wait<0>();
}

// Launches update_backward_tokens_kernel where a token fits its shape.
template <bool WORDS, int VPT, int S, int MAX>
bool update_backward_tokens(int64_t T, int64_t D, const Span<const bf16>& x, const Span<const bf16>& y,
                            const Span<const float>& h, const Drop& d, const Span<const bf16>& gout,
                            const Span<bf16>& gy, const Span<float>& gh, cudaError_t* e, cudaStream_t stream) {
    using Shape = TokenShape<WORDS, VPT, S, MAX>;
    const int64_t threads = ((D + 7) / 8 + VPT - 1) / VPT;
    if (threads > Shape::kMaxThreads) return false;
    const int G = (int)((threads + 31) / 32 * 32);
    int R = Shape::kMaxThreads / G;
    if (R > 15) R = 15;                                // named barriers of a block
    const int64_t spread = (T + kSms - 1) / kSms;      // no more groups than tokens to spread over the blocks
    if (R > spread) R = (int)spread;
    while (R > 1 && Shape::bytes(G, R) > kMaxShared) --R;
    if (Shape::bytes(G, R) > kMaxShared) return false;
    const int64_t grid = (T + R - 1) / R < kSms ? (T + R - 1) / R : kSms;
    auto kernel = update_backward_tokens_kernel<WORDS, VPT, S, MAX>;
    static std::atomic<uint64_t> done{0};
    *e = allow_shared(kernel, kMaxShared, done);
    if (*e != cudaSuccess) return true;
    *e = launch_early(kernel, dim3((unsigned)grid), dim3((unsigned)(G * R)), Shape::bytes(G, R), stream, (int)T, (int)D, G,
                      R, x, y, h, d, gout, gy, gh);
    return true;
}

template <typename E>
cudaError_t dropout_typed(int64_t n, const void* x, void* y, const Drop& d, cudaStream_t stream) {
    const Span<const E> xs{static_cast<const E*>(x), (size_t)n};
    const Span<E> ys{static_cast<E*>(y), (size_t)n};
    if (aligned16(x) && aligned16(y) && n < kShortCounters) {
        const int64_t block = (int64_t)kThreads * Elem<E>::kPack * kDropPacks;
        return launch_early(dropout_kernel<E>, dim3((unsigned)((n + block - 1) / block)), dim3(kThreads), 0, stream, n, xs,
                            ys, d);
    }
    const int64_t blocks = ((n + 3) / 4 + kThreads - 1) / kThreads;
    return launch_early(dropout_any_kernel<E>, dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(kThreads), 0,
                        stream, n, xs, ys, d);
}

}  // namespace

cudaError_t dropout(int64_t n, int type, const void* x, void* y, const DropArgs& a, cudaStream_t stream) {
    const Drop d{a.rng, a.sequence, a.threshold, a.scale};
    if (type == 0) return dropout_typed<bf16>(n, x, y, d, stream);
    if (type == 1) return dropout_typed<__half>(n, x, y, d, stream);
    return dropout_typed<float>(n, x, y, d, stream);
}

cudaError_t update_forward(int64_t T, int64_t D, const void* x, const void* y, const float* h,
                           const DropArgs& a, void* x_out, cudaStream_t stream) {
    const Drop d{a.rng, a.sequence, a.threshold, a.scale};
    const Span<const bf16> xs{static_cast<const bf16*>(x), (size_t)(T * kStreams * D)};
    const Span<const bf16> ys{static_cast<const bf16*>(y), (size_t)(T * D)};
    const Span<const float> hs{h, (size_t)(T * kGates)};
    const Span<bf16> os{static_cast<bf16*>(x_out), (size_t)(T * kStreams * D)};
    // 32-bit vector numbers and counters
    if ((D % 8 == 0 || D >= 128) && T * D < kShortCounters && (D + 7) / 8 * T <= INT32_MAX) {
        const VectorGrid grid((D + 7) / 8, kThreads, D % 8 != 0);
        return launch_early(D % 8 == 0 ? update_forward_vectors_kernel<false> : update_forward_vectors_kernel<true>,
                            dim3(grid.blocks(T)), dim3(grid.threads), 0, stream, T, D, grid, aligned16(h), xs, ys, hs, d,
                            os);
    }
    return launch_early(update_forward_any_kernel, dim3((unsigned)T), dim3(kThreads), 0, stream, D, xs, ys, hs, d, os);
}

cudaError_t update_backward(int64_t T, int64_t D, const void* x, const void* y, const float* h,
                            const DropArgs& a, const void* grad_x_out, void* grad_y, float* grad_h,
                            cudaStream_t stream) {
    const Drop d{a.rng, a.sequence, a.threshold, a.scale};
    const Span<const bf16> xs{static_cast<const bf16*>(x), (size_t)(T * kStreams * D)};
    const Span<const bf16> ys{static_cast<const bf16*>(y), (size_t)(T * D)};
    const Span<const float> hs{h, (size_t)(T * kGates)};
    const Span<const bf16> gs{static_cast<const bf16*>(grad_x_out), (size_t)(T * kStreams * D)};
    const Span<bf16> gys{static_cast<bf16*>(grad_y), (size_t)(T * D)};
    const Span<float> ghs{grad_h, (size_t)(T * kGates)};
    cudaError_t e = cudaSuccess;
    if (T * D < kShortCounters &&
        (D % 8 == 0 ? update_backward_tokens<false, 1, 2, 640>(T, D, xs, ys, hs, d, gs, gys, ghs, &e, stream) ||
                          update_backward_tokens<false, 2, 1, 512>(T, D, xs, ys, hs, d, gs, gys, ghs, &e, stream) ||
                          update_backward_tokens<false, 2, 1, 640>(T, D, xs, ys, hs, d, gs, gys, ghs, &e, stream)
                    : update_backward_tokens<true, 1, 2, 512>(T, D, xs, ys, hs, d, gs, gys, ghs, &e, stream) ||
                          update_backward_tokens<true, 2, 1, 512>(T, D, xs, ys, hs, d, gs, gys, ghs, &e, stream)))
        return e;
    return launch_early(update_backward_any_kernel, dim3((unsigned)T), dim3(kThreads), 0, stream, D, xs, ys, hs, d, gs, gys,
                        ghs);
}

cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace streams
}  // namespace ops
}  // namespace mhcpb
