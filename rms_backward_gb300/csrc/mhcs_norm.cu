// Layer norm, plain and of the collapsed residual streams, with its gradient.
//
//   u       the row: x[t, :], or sum_s H_pre[s] X_s of the four streams
//   forward mu = mean u, var = mean (u - mu)^2, rs = 1 / sqrt(var + eps),
//           y = (u - mu) rs gamma + beta
//   backward, with z = (u - mu) rs and w = dy gamma:
//           du = rs (w - mean w - z mean(w z))
//           dgamma = sum_t dy z, dbeta = sum_t dy
//           plain: dx = du;  streams: dX_s = H_pre[s] du + sum_i H_res[i][s] dX'_i,
//           dH_pre[s] = <X_s, du>
// with dX' the gradient of the streams after the sublayer, so that the
// residual path's share is added in FP32 and rounded once.
//
// Bound by HBM in long batches: 4 bytes per BF16 element forward and 6 for the
// gradient; collapsed rows 10 and 26 per column, so the streams are read once
// and neither u nor du ever goes to memory.  The fractions below are of the
// 6.77 TB/s that a plain copy reaches; "replayed" times are calls captured in
// a graph, without the host's share.
//
// FP32 statistics and sums; the variance is of centred values, not a difference
// of squares.  z is (u - mu) rs, the subtraction first: u rs - mu rs would save a
// product, but the rounding of mu rs, 2^-24 |mu| rs, enters every column of a
// row, 300 times z's own rounding where a row lies 300 deviations from zero.  The
// parameter gradients are summed over row groups whose number depends on T, D
// and the type alone, then over the groups in order: the same bits on every
// call and GPU.
#include "mhcs_common.cuh"
#include "mhcs_internal.h"
#include "mhcs_ring.cuh"
#include "mhcs_words.cuh"
#include "ptx.cuh"

namespace mhcpb {
namespace ops {
namespace norm {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kSms = 152;            // persistent grids: a constant, so that results do not depend on the GPU
constexpr int kMaxParts = 2 * kSms;  // most row groups of the parameter gradients
constexpr int kMaxShared = 227 * 1024;   // shared memory of a block

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t part_count(int64_t T) { return T < kMaxParts ? T : kMaxParts; }

template <typename E>
struct Params {
    int64_t T, D, parts;
    int64_t x_stride, y_stride, gy_stride, gx_stride;
    float eps;
    bool accumulate;
    Span<const E> x;         // rows, or the streams (row stride 4 D)
    Span<const float> h;     // gates when MIX
    Span<const float> gamma, beta;   // p may be null
    Span<E> y;
    Span<float> mean, rstd;          // p may be null in the forward
    Span<const E> grad_y, grad_x_out;
    Span<E> grad_x;
    Span<float> grad_h;
    Span<float> partial;     // [parts][2][D]
    Span<float> grad_gamma, grad_beta;   // p may be null
};

// u at columns c .. c + N - 1 of row t
template <typename E, bool MIX, int N>
__device__ __forceinline__ void row_at(const Params<E>& a, const float* gate, int64_t t, int64_t c,
                                       float (&u)[N]) {
    load_at<N>(a.x, (size_t)(t * a.x_stride + c), u, 0);
    if constexpr (MIX) {
#pragma unroll
        for (int k = 0; k < N; ++k) u[k] *= gate[0];
#pragma unroll
        for (int s = 1; s < kStreams; ++s) {
            float v[N];
            load_at<N>(a.x, (size_t)(t * a.x_stride + s * a.D + c), v, 0);
#pragma unroll
            for (int k = 0; k < N; ++k) u[k] = fmaf(gate[s], v[k], u[k]);
        }
    }
}
template <int N>
__device__ __forceinline__ void vector_at(const Span<const float>& s, int64_t c, float other, float (&v)[N],
                                          uint32_t site) {
    if (s.p != nullptr) {
        load_at<N>(s, (size_t)c, v, site);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = other;
    }
}
// columns c .. c + 3 of a parameter (other where there is none, 0 past D);
// ANY: of any alignment, and D of any size
template <bool ANY>
__device__ __forceinline__ void four_at(const Span<const float>& s, int c, int D, float other, float (&v)[4]) {
    if constexpr (!ANY) {
        if (c < D) vector_at<4>(s, c, other, v, 2);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float one[1] = {0.f};
            if (c + k < D) vector_at<1>(s, c + k, other, one, 2);
            v[k] = one[0];
        }
    }
}
template <typename F>
__device__ __forceinline__ float scalar_at(const Span<F>& s, int64_t i, uint32_t site) {
    float v[1];
    load_at<1>(s, (size_t)i, v, site);
    return v[0];
}

// Rows too long for the kernels below (16-bit types above 18,432 columns, not
// aligned 16,384; FP32 20,480 and 10,240; collapsed 10,240): a block reads its
// row again for each pass, from L1 or L2.  T=2048, D=16384 takes 36.5 us here,
// 29.7 through shared memory.
template <typename E, bool MIX, int N>
__global__ void __launch_bounds__(kThreads) forward_any_kernel(Params<E> a) {
    ptx::grid_dependency_wait();
    __shared__ float gate[kGates], scratch[32];
    const int64_t t = blockIdx.x;
    if constexpr (MIX) {
        if (threadIdx.x < kStreams) gate[threadIdx.x] = scalar_at(a.h, t * kGates + threadIdx.x, 1);
        __syncthreads();
    }
    const int64_t first = (int64_t)threadIdx.x * N, step = kThreads * N;
    float s[1] = {0.f}, u[N];
    for (int64_t c = first; c < a.D; c += step) {
        row_at<E, MIX, N>(a, gate, t, c, u);
#pragma unroll
        for (int k = 0; k < N; ++k) s[0] += u[k];
    }
    block_sum<1>(s, scratch);
    const float mean = s[0] / (float)a.D;
    s[0] = 0.f;
    for (int64_t c = first; c < a.D; c += step) {
        row_at<E, MIX, N>(a, gate, t, c, u);
#pragma unroll
        for (int k = 0; k < N; ++k) s[0] = fmaf(u[k] - mean, u[k] - mean, s[0]);
    }
    block_sum<1>(s, scratch);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.D + a.eps);
    for (int64_t c = first; c < a.D; c += step) {
        float g[N], b[N];
        row_at<E, MIX, N>(a, gate, t, c, u);
        vector_at<N>(a.gamma, c, 1.f, g, 2);
        vector_at<N>(a.beta, c, 0.f, b, 2);
#pragma unroll
        for (int k = 0; k < N; ++k) u[k] = fmaf((u[k] - mean) * rstd, g[k], b[k]);
        store_at<N>(a.y, (size_t)(t * a.y_stride + c), u, 3);
    }
    if (threadIdx.x == 0 && a.mean.p != nullptr) {
        const float m[1] = {mean}, r[1] = {rstd};
        store_at<1>(a.mean, (size_t)t, m, 4);
        store_at<1>(a.rstd, (size_t)t, r, 4);
    }
}

// ------------------------------------------------------------ forward, rows in registers
// A group of G threads holds one row, VPT pieces of N columns per thread (N is
// a 16-byte vector, or 1 for rows that are not aligned), everything loaded
// before anything is used.  For few rows, where a launch and one trip to
// memory are all there is: one vector per thread, so that a row has many.
// T=1, D=5120: 2.3 us replayed, of which an empty launch is about 1.6.
// Also FP32 rows of 10,241 to 20,480 columns, eight vectors per thread
// (T=2048, D=16384: 48.2 us, 82%; the kernel above 71.9).
template <typename E, bool MIX, int N, int VPT>
__global__ void __launch_bounds__(640) forward_rows_kernel(Params<E> a, int G, int R) {
    ptx::grid_dependency_wait();
    __shared__ float sums[2][32];   // by warp of the block
    const int tid = threadIdx.x, group = tid / G, i = tid - group * G, lane = tid & 31;
    const int warp = tid >> 5, warp0 = group * (G >> 5), warps = G >> 5;
    const int64_t t = (int64_t)blockIdx.x * R + group;
    const bool valid = t < a.T;     // the last block's other groups still meet their barriers
    const int D = (int)a.D, c0 = i * N, step = G * N;
    float gate[kStreams] = {};
    if constexpr (MIX)
        if (valid)
#pragma unroll
            for (int s = 0; s < kStreams; ++s) gate[s] = scalar_at(a.h, t * kGates + s, 1);
    float u[VPT][N];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (valid && c0 + v * step < D) {
            row_at<E, MIX, N>(a, gate, t, c0 + v * step, u[v]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) u[v][k] = 0.f;
        }
    }
    const float inv_d = 1.f / (float)D;
    const auto total = [&](float s, int which) {
        s = warp_sum(s);
        if (lane == 0) sums[which][warp] = s;
        group_sync(group, G);
        return warp_sum(lane < warps ? sums[which][warp0 + lane] : 0.f);
    };
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < N; ++k) s += u[v][k];
    const float mean = total(s, 0) * inv_d;
    s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (c0 + v * step < D)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                u[v][k] -= mean;
                s = fmaf(u[v][k], u[v][k], s);
            }
    const float rstd = 1.f / sqrtf(total(s, 1) * inv_d + a.eps);
    if (!valid) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = c0 + v * step;
        if (c < D) {
            float g[N], b[N];
            vector_at<N>(a.gamma, c, 1.f, g, 2);
            vector_at<N>(a.beta, c, 0.f, b, 2);
#pragma unroll
            for (int k = 0; k < N; ++k) u[v][k] = fmaf(u[v][k] * rstd, g[k], b[k]);
            store_at<N>(a.y, (size_t)(t * a.y_stride + c), u[v], 3);
        }
    }
    if (i == 0 && a.mean.p != nullptr) {
        const float m[1] = {mean}, r[1] = {rstd};
        store_at<1>(a.mean, (size_t)t, m, 4);
        store_at<1>(a.rstd, (size_t)t, r, 4);
    }
}

// ------------------------------------------------------------ forward, rows through shared memory
// Groups, per-thread copies S rows ahead and columns as in backward_rows_kernel
// below.  Each warp centres its own columns (their mean m_w, then the squares
// q_w about it) and publishes both, so that one barrier gives the row's
// statistics.  With d_w = m_w - m_0:
//   mean = m_0 + sum n_w d_w / D,
//   var = (sum q_w + sum n_w d_w^2) / D - (mean - m_0)^2.
// m_0 is the mean of n_0 of the row's own columns, so the difference cancels at
// most a factor D / n_0, the number of warps, however far the row is from zero.
// T=16384, D=5120: 55.7 us (89%); collapsed 133 (93%).  T=4096: 20.5 (61%) and
// 35.5 (87%): about 8 and 4 us are the first rows' way in and the last ones'
// out.  In between it is the SM's own work that binds, 37% of the issue slots
// and 46% of the shared-memory pipe in use by 20 warps.  Taken because, for
// T=4096 / 16384: rows in registers 30.7 / 113 us; two vectors and four rows
// ahead 21.7 / 68.5; two rows at a time, for gamma's and beta's loads, 22.4 /
// 65.8.  The 16-bit types' unaligned shapes spill 36 to 40 bytes a thread.  One row
// ahead less where that makes longer rows fit: collapsed above
// 8,192 columns (not aligned 6,656), plain above 13,312 (12,288).
template <typename E, bool MIX, bool WORDS, int VPT, int S>
struct ForwardShape {
    static constexpr int N = Elem<E>::kPack;
    static constexpr int kMaxThreads = 640;
    static constexpr int kArrays = MIX ? kStreams : 1;
    static constexpr int kStage = VPT * kArrays;
    static constexpr int kPitch = WORDS ? kMaxThreads / 32 * kWarpSlots : kMaxThreads;
    static constexpr int kSlots = S * kStage;
    static constexpr int kVectorSlots = 2 * VPT * N / 4;   // gamma and beta of a thread's columns
    static size_t bytes(int G, int R) {
        return (size_t)kPitch * kSlots * 16 + (size_t)G * kVectorSlots * 16 + (size_t)R * (G / 32 * S * 16 + 2 * 2 * 32 * 4) +
               (WORDS ? (size_t)R * G * 16 : 0);   // what a warp stores
    }
};

template <typename E, bool MIX, bool WORDS, int VPT, int S>
__global__ void __launch_bounds__((ForwardShape<E, MIX, WORDS, VPT, S>::kMaxThreads), 1)
    forward_ring_kernel(Params<E> a, int G, int R) {
    using Shape = ForwardShape<E, MIX, WORDS, VPT, S>;
    constexpr int N = Shape::N, H = N / 2, P = Shape::kPitch, A = Shape::kArrays;
    extern __shared__ uint4 slots[];
    const int NT = G * R, tid = threadIdx.x, group = tid / G, i = tid - group * G, lane = tid & 31;
    const int warp = i >> 5, warps = G >> 5;
    uint4* const mine = slots + (WORDS ? (tid >> 5) * kWarpSlots + lane : tid);
    float4* const vectors = reinterpret_cast<float4*>(slots + P * Shape::kSlots);   // [2][VPT N / 4][G]
    float* const floats = reinterpret_cast<float*>(vectors + Shape::kVectorSlots * G);
    float* const gates = floats + (tid >> 5) * (S * 4);                             // [S][4] per warp
    float* const sums = floats + (NT >> 5) * (S * 4) + group * (2 * 2 * 32);        // [2][2][32]
    uint4* const buffer = reinterpret_cast<uint4*>(floats + (NT >> 5) * (S * 4) + R * (2 * 2 * 32)) + (tid >> 5) * 32;
    const int groups = (int)gridDim.x * R, first = (int)blockIdx.x * R + group, T = (int)a.T;
    const int c0 = i * N, step = G * N, D = (int)a.D;

    // columns past D: never copied, they stay 0 and add nothing
#pragma unroll
    for (int k = 0; k < Shape::kSlots; ++k)
        if (!WORDS && c0 + k % Shape::kStage / A * step >= D) mine[k * P] = make_uint4(0u, 0u, 0u, 0u);
    ptx::grid_dependency_wait();
    const auto fetch = [&](int t, int stage) {
        if (t < T) {
            const size_t at = (size_t)((uint64_t)(uint32_t)t * (uint32_t)a.x_stride + (uint32_t)c0);
            if (WORDS && edge_row<E>(t, T, D)) {
#pragma unroll 1
                for (int k = 0; k < Shape::kStage; ++k)
                    copy_edge(mine - lane + (stage * Shape::kStage + k) * P, a.x.p, a.x.count,
                                  at + k / A * step + k % A * D - lane * N, D - (c0 + k / A * step) + lane * N, 0);
            } else {
#pragma unroll
                for (int k = 0; k < Shape::kStage; ++k) {
                    uint4* const slot = mine + (stage * Shape::kStage + k) * P;
                    const size_t from = at + k / A * step + k % A * D;
                    if constexpr (WORDS) {
                        copy_chunks(slot - lane, a.x, from - lane * N, D - (c0 + k / A * step) + lane * N, 0);
                    } else if (c0 + k / A * step < D) {
                        if (a.x.has(from, N, 0)) copy16(slot, a.x.p + from);
                    }
                }
            }
            if (MIX && lane < kStreams && a.h.has((size_t)t * kGates + lane, 1, 1))
                copy4(gates + stage * 4 + lane, a.h.p + (size_t)t * kGates + lane);
        }
        copies_commit();
    };
#pragma unroll
    for (int q = 0; q < S; ++q) fetch(first + q * groups, q);
    if (group == 0)
#pragma unroll
        for (int k = 0; k < Shape::kVectorSlots / 2; ++k) {
            const int c = c0 + k / (N / 4) * step + k % (N / 4) * 4;
            float g[4] = {}, b[4] = {};
            four_at<WORDS>(a.gamma, c, D, 1.f, g);
            four_at<WORDS>(a.beta, c, D, 0.f, b);
            vectors[k * G + i] = make_float4(g[0], g[1], g[2], g[3]);
            vectors[(Shape::kVectorSlots / 2 + k) * G + i] = make_float4(b[0], b[1], b[2], b[3]);
        }
    __syncthreads();

    // this warp's share of the columns, and lane w's: warp w's
    const auto share = [&](int w) {
        int n = 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int left = D - (w * 32 * N + v * step);
            n += left < 0 ? 0 : left < 32 * N ? left : 32 * N;
        }
        return (float)n;
    };
    const float n_mine = share(warp), inv_mine = n_mine > 0.f ? 1.f / n_mine : 0.f;
    const float n_lane = lane < warps ? share(lane) : 0.f, inv_d = 1.f / (float)D;
    int stage = 0, parity = 0;
    for (int t = first; t < T; t += groups) {
        copies_wait<S - 1>();
        __syncwarp();
        uint4* const row = mine + stage * (Shape::kStage * P);
        if constexpr (WORDS)
#pragma unroll
            for (int k = 0; k < Shape::kStage; ++k)
                align_chunks<E>(row - lane + k * P, misaligned(a.x.p + (size_t)t * a.x_stride + k % A * D), D - (c0 + k / A * step));
        float2 u[VPT][H], s2 = pair(0.f);
        float p4[kStreams] = {};
        if constexpr (MIX) {
            const float4 pre = *reinterpret_cast<const float4*>(gates + stage * 4);
            p4[0] = pre.x;
            p4[1] = pre.y;
            p4[2] = pre.z;
            p4[3] = pre.w;
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack<E>(row[v * A * P], u[v]);
            if constexpr (MIX) {
#pragma unroll
                for (int k = 0; k < H; ++k) u[v][k] = mul2(u[v][k], pair(p4[0]));
#pragma unroll
                for (int s = 1; s < A; ++s) {
                    float2 x[H];
                    unpack<E>(row[(v * A + s) * P], x);
#pragma unroll
                    for (int k = 0; k < H; ++k) u[v][k] = fma2(pair(p4[s]), x[k], u[v][k]);
                }
            }
#pragma unroll
            for (int k = 0; k < H; ++k) s2 = add2(s2, u[v][k]);
        }
        __syncwarp();   // every lane has read the gates
        fetch(t + S * groups, stage);
        stage = stage + 1 == S ? 0 : stage + 1;
        const float m_mine = warp_sum(s2.x + s2.y) * inv_mine;
        float2 q2 = pair(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (c0 + v * step < D)
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    float2 d = add2(u[v][k], pair(-m_mine));
                    if (WORDS) {   // a row may end inside the vector
                        if (c0 + v * step + 2 * k >= D) d.x = 0.f;
                        if (c0 + v * step + 2 * k + 1 >= D) d.y = 0.f;
                    }
                    q2 = fma2(d, d, q2);
                }
        const float q_mine = warp_sum(q2.x + q2.y);
        float mean = m_mine, var = q_mine * inv_d;
        if (warps > 1) {
            float* const s0 = sums + parity * (2 * 32);
            if (lane == 0) {
                s0[warp] = m_mine;
                s0[32 + warp] = q_mine;
            }
            group_sync(group, G);
            // about warp 0's mean, so that both sums are formed at once
            const float shift = s0[0], d = lane < warps ? s0[lane] - shift : 0.f, nd = n_lane * d;
            const float both = warp_sum_two(nd, fmaf(nd, d, lane < warps ? s0[32 + lane] : 0.f));
            const float off = __shfl_sync(kFullMask, both, 0) * inv_d;   // mean - shift
            mean = shift + off;
            var = fmaf(__shfl_sync(kFullMask, both, 16), inv_d, -off * off);
        }
        const float rstd = 1.f / sqrtf(var + a.eps);
        const float2 mean2 = pair(-mean), rstd2 = pair(rstd);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float2 o[H];
#pragma unroll
            for (int k = 0; k < H / 2; ++k) {
                const float4 g = vectors[(v * (N / 4) + k) * G + i];
                const float4 b = vectors[(Shape::kVectorSlots / 2 + v * (N / 4) + k) * G + i];
                o[2 * k] = fma2(mul2(add2(u[v][2 * k], mean2), rstd2), make_float2(g.x, g.y), make_float2(b.x, b.y));
                o[2 * k + 1] = fma2(mul2(add2(u[v][2 * k + 1], mean2), rstd2), make_float2(g.z, g.w), make_float2(b.z, b.w));
            }
            const size_t at = (size_t)((uint64_t)(uint32_t)t * (uint32_t)a.y_stride + (uint32_t)(c0 + v * step));
            if constexpr (WORDS) {
                store_words(buffer, a.y, at - lane * N, D - (c0 + v * step) + lane * N, pack<E>(o), 3);
            } else {
                if (c0 + v * step < D && a.y.has(at, N, 3)) *reinterpret_cast<uint4*>(a.y.p + at) = pack<E>(o);
            }
        }
        if (i == 0 && a.mean.p != nullptr) {
            const float o1[1] = {mean}, o2[1] = {rstd};
            store_at<1>(a.mean, (size_t)t, o1, 4);
            store_at<1>(a.rstd, (size_t)t, o2, 4);
        }
        parity ^= 1;
    }
    copies_wait<0>();
}

// Rows too long for the kernel below (above 16,384 columns; collapsed 10,240, not
// aligned 8,192), one per block, read twice; the parameter gradients read
// everything once more.  T=2048, D=10240 collapsed takes 326 us
// here, 148 below.
template <typename E, bool MIX, int N>
__global__ void __launch_bounds__(kThreads) backward_rows_any_kernel(Params<E> a) {
    ptx::grid_dependency_wait();
    __shared__ float gate[kGates], scratch[4 * 32];
    const int64_t t = blockIdx.x;
    if constexpr (MIX) {
        if (threadIdx.x < kGates) gate[threadIdx.x] = scalar_at(a.h, t * kGates + threadIdx.x, 1);
        __syncthreads();
    }
    const float mean = scalar_at(a.mean, t, 4);
    const float rstd = scalar_at(a.rstd, t, 4);
    const int64_t first = (int64_t)threadIdx.x * N, step = kThreads * N;
    float s[2] = {0.f, 0.f};
    for (int64_t c = first; c < a.D; c += step) {
        float u[N], w[N], g[N];
        row_at<E, MIX, N>(a, gate, t, c, u);
        load_at<N>(a.grad_y, (size_t)(t * a.gy_stride + c), w, 5);
        vector_at<N>(a.gamma, c, 1.f, g, 2);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            w[k] *= g[k];
            s[0] += w[k];
            s[1] = fmaf(w[k], (u[k] - mean) * rstd, s[1]);
        }
    }
    block_sum<2>(s, scratch);
    const float mw = s[0] / (float)a.D, mwz = s[1] / (float)a.D;
    float dot[kStreams] = {};
    for (int64_t c = first; c < a.D; c += step) {
        float u[N], w[N], g[N];
        row_at<E, MIX, N>(a, gate, t, c, u);
        load_at<N>(a.grad_y, (size_t)(t * a.gy_stride + c), w, 5);
        vector_at<N>(a.gamma, c, 1.f, g, 2);
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = rstd * (w[k] * g[k] - mw - (u[k] - mean) * rstd * mwz);
        if constexpr (!MIX) {
            store_at<N>(a.grad_x, (size_t)(t * a.gx_stride + c), w, 6);
        } else {
            float go[kStreams][N];
            if (a.grad_x_out.p != nullptr)
#pragma unroll
                for (int i = 0; i < kStreams; ++i)
                    load_at<N>(a.grad_x_out, (size_t)((t * kStreams + i) * a.D + c), go[i], 7);
#pragma unroll
            for (int j = 0; j < kStreams; ++j) {
                float v[N], o[N];
                load_at<N>(a.x, (size_t)((t * kStreams + j) * a.D + c), v, 0);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    dot[j] = fmaf(v[k], w[k], dot[j]);
                    o[k] = gate[j] * w[k];
                    if (a.grad_x_out.p != nullptr)
#pragma unroll
                        for (int i = 0; i < kStreams; ++i) o[k] = fmaf(gate[8 + 4 * i + j], go[i][k], o[k]);
                }
                store_at<N>(a.grad_x, (size_t)((t * kStreams + j) * a.D + c), o, 6);
            }
        }
    }
    if constexpr (MIX) {
        block_sum<kStreams>(dot, scratch);
        if (threadIdx.x < kStreams) {
            float v[1] = {0.f};
#pragma unroll
            for (int j = 0; j < kStreams; ++j)
                if (threadIdx.x == j) v[0] = dot[j];
            store_at<1>(a.grad_h, (size_t)(t * kGates + threadIdx.x), v, 8);
        }
    }
}

// Partial parameter gradients: block (column block, part), a thread per column.
template <typename E, bool MIX>
__global__ void __launch_bounds__(kThreads) backward_columns_any_kernel(Params<E> a) {
    ptx::grid_dependency_wait();
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t part = blockIdx.y;
    if (c >= a.D) return;
    const int64_t begin = a.T * part / a.parts, end = a.T * (part + 1) / a.parts;
    float gg = 0.f, gb = 0.f;
    for (int64_t t = begin; t < end; ++t) {
        float gate[kStreams], u[1], w[1];
        if constexpr (MIX)
#pragma unroll
            for (int s = 0; s < kStreams; ++s) gate[s] = scalar_at(a.h, t * kGates + s, 1);
        row_at<E, MIX, 1>(a, gate, t, c, u);
        load_at<1>(a.grad_y, (size_t)(t * a.gy_stride + c), w, 5);
        const float mean = scalar_at(a.mean, t, 4);
        const float rstd = scalar_at(a.rstd, t, 4);
        gg = fmaf(w[0], (u[0] - mean) * rstd, gg);
        gb += w[0];
    }
    const float g1[1] = {gg}, b1[1] = {gb};
    store_at<1>(a.partial, (size_t)((part * 2 + 0) * a.D + c), g1, 9);
    store_at<1>(a.partial, (size_t)((part * 2 + 1) * a.D + c), b1, 9);
}

// ------------------------------------------------------------ backward, rows in shared memory
// A group of G threads takes a row at a time; thread i owns the same vectors
// i, i + G, ... (VPT of 16 bytes) of every row, so the parameter gradients of
// its columns stay in registers until the end.  The row's inputs come through
// per-thread copies, S rows ahead.  The first half of a row forms its two sums,
// sum w and sum w z; after the group's one barrier, the second half reads the
// slots again (cheaper than holding u and w in registers), writes the
// gradients and refills each slot as it leaves it.  The other groups of the
// block compute while one waits.
//
// T=16384, D=5120: 87.3 us (85%); collapsed 334 (96%, a copy of nine arrays to
// four through the same slots takes 325).  T=4096: 29.2 (64%) and 92.4 (87%).
// Register spills cost more than anything else here (the collapsed gradient
// fell from 480 us to 337 when the last 88 bytes went), so what a row needs is
// formed when it is needed and the shapes are as wide as registers allow.
// Collapsed, T=4096:
//   1 vector, 2 rows ahead, 640 threads   D=5120:  92.4 us   (up to D=5120)
//   2 vectors, 1 ahead, 512 threads       D=5120: 114        (up to D=8192: 175 us, 73%)
//   2 vectors, 1 ahead, 640 threads       D=8192: 237        (up to D=10240: T=2048 148 us, 54%)
// Plain rows: two 16-bit vectors or four of FP32, 2 rows ahead (FP32 T=4096 /
// 16384: 45.8 / 171 us; 1 ahead 48.5 / 158; 3 ahead slower), and up to D=16384
// twice as many with 512 threads, 1 ahead (T=2048, D=16384: 58 us; the kernels
// above 102).
// The shapes for long rows still spill, bytes a thread stores / loads: two
// vectors collapsed by 640 threads 112 / 236, by 512 unaligned 44 / 48; the
// 16-bit types' four vectors 36 / 60 unaligned, BF16's 8 / 12 aligned; eight of
// FP32 44 / 100 aligned.  They are kept because the kernels above take longer.
// Rows at any address take 2 to 3 times as long (T=4096, D=1285: 19.4 us,
// collapsed 66.9): bound by the instructions that put vectors together.
template <typename E, bool MIX, bool WORDS, int VPT, int S, int MAX>
struct RowsShape {
    static constexpr int N = Elem<E>::kPack;
    static constexpr int kMaxThreads = MAX;   // 640: 96 registers a thread; 512: 128
    static constexpr int kArrays = MIX ? 2 * kStreams + 1 : 2;      // x, grad_y, residual gradient
    static constexpr int kStage = VPT * kArrays;                    // 16-byte slots of a row
    // Slot k of every thread of the block lies together, so that a warp's copy
    // writes whole 128-byte lines; the pitch is a constant, for immediate
    // offsets.  WORDS: rows at any address (mhcs_words.cuh).
    static constexpr int kPitch = WORDS ? kMaxThreads / 32 * kWarpSlots : kMaxThreads;
    static constexpr int kSlots = S * kStage;
    static constexpr int kGammaSlots = VPT * N / 4;                 // per thread of a group, FP32
    static constexpr int kWarpFloats = S * 32;                      // per row: 24 gates, mean, rstd
    static constexpr int kSums = 2 + (MIX ? kStreams : 0);
    static constexpr int kGroupFloats = 2 * kSums * 32;
    // slots and gamma; at the end, two FP32 sums for each column of each group's threads
    static size_t rows_bytes(int G) { return (size_t)kPitch * kSlots * 16 + (size_t)G * kGammaSlots * 16; }
    static size_t sums_bytes(int G, int R) { return (size_t)R * G * VPT * N * 2 * 4; }
    static size_t bytes(int G, int R) {
        return rows_bytes(G) + (size_t)R * (G / 32 * kWarpFloats * 4 + kGroupFloats * 4) + (WORDS ? (size_t)R * G * 16 : 0);
    }
};

template <typename E, bool MIX, bool WORDS, int VPT, int S, int MAX, bool MANY>
__global__ void __launch_bounds__(MAX, 1) backward_rows_kernel(Params<E> a, int G, int R) {
    using Shape = RowsShape<E, MIX, WORDS, VPT, S, MAX>;
    constexpr int N = Shape::N, H = N / 2, P = Shape::kPitch, A = Shape::kArrays;
    constexpr int XA = MIX ? kStreams : 1;   // slots of a vector: x (XA), grad_y, residual gradient
    extern __shared__ uint4 slots[];
    const int NT = G * R, tid = threadIdx.x, group = tid / G, i = tid - group * G, lane = tid & 31;
    const int warp = i >> 5, warps = G >> 5;
    uint4* const mine = slots + (WORDS ? (tid >> 5) * kWarpSlots + lane : tid);
    float4* const gammas = reinterpret_cast<float4*>(slots + P * Shape::kSlots);   // [kGammaSlots][G]
    float* const floats = reinterpret_cast<float*>(gammas + Shape::kGammaSlots * G);
    float* const scalars = floats + (tid >> 5) * Shape::kWarpFloats;
    float* const sums = floats + (NT >> 5) * Shape::kWarpFloats + group * Shape::kGroupFloats;   // [2][kSums][32]
    uint4* const buffer =   // WORDS: what the warp stores
        reinterpret_cast<uint4*>(floats + (NT >> 5) * Shape::kWarpFloats + R * Shape::kGroupFloats) + (tid >> 5) * 32;
    const int groups = (int)gridDim.x * R, first = (int)blockIdx.x * R + group, T = (int)a.T;
    const bool residual = MIX && a.grad_x_out.p != nullptr;
    const int c0 = i * N, step = G * N, D = (int)a.D;   // this thread's columns: c0 + v * step

    // columns past D: never copied, they stay 0 and add nothing
#pragma unroll
    for (int k = 0; k < Shape::kSlots; ++k)
        if (!WORDS && c0 + k % Shape::kStage / A * step >= D) mine[k * P] = make_uint4(0u, 0u, 0u, 0u);
    ptx::grid_dependency_wait();

    // Element offset of row t of an array at this thread's first column, formed
    // where it is needed: cheaper than a 64-bit pointer per array kept and moved.
    const auto at_row = [&](int t, int64_t stride) {
        return (size_t)((uint64_t)(uint32_t)t * (uint32_t)stride + (uint32_t)c0);
    };
    const auto fetch_vector = [&](uint4* dst, int t, int v) {
        if constexpr (WORDS) {
            const int width = D - (c0 + v * step) + lane * N;   // from the warp's first column on
            const size_t xo = at_row(t, a.x_stride) + v * step - lane * N, go = at_row(t, a.gy_stride) + v * step - lane * N;
            dst -= lane;
            if (edge_row<E>(t, T, D)) {
#pragma unroll 1
                for (int s = 0; s < A; ++s) {
                    const Span<const E>& in = s < XA ? a.x : s == XA ? a.grad_y : a.grad_x_out;
                    const size_t at = s < XA ? xo + s * D : s == XA ? go : xo + (s - XA - 1) * D;
                    if (s <= XA || residual) copy_edge(dst + (v * A + s) * P, in.p, in.count, at, width, 0);
                }
                return;
            }
#pragma unroll
            for (int s = 0; s < XA; ++s) copy_chunks(dst + (v * A + s) * P, a.x, xo + s * D, width, 0);
            copy_chunks(dst + (v * A + XA) * P, a.grad_y, go, width, 5);
            if (MIX && residual)
#pragma unroll
                for (int s = 0; s < kStreams; ++s)
                    copy_chunks(dst + (v * A + XA + 1 + s) * P, a.grad_x_out, xo + s * D, width, 7);
        } else if (c0 + v * step < D) {
            const size_t xo = at_row(t, a.x_stride) + v * step, go = at_row(t, a.gy_stride) + v * step;
#pragma unroll
            for (int s = 0; s < XA; ++s)
                if (a.x.has(xo + s * D, N, 0)) copy16(dst + (v * A + s) * P, a.x.p + xo + s * D);
            if (a.grad_y.has(go, N, 5)) copy16(dst + (v * A + XA) * P, a.grad_y.p + go);
            if (MIX && residual)
#pragma unroll
                for (int s = 0; s < kStreams; ++s)
                    if (a.grad_x_out.has(xo + s * D, N, 7))   // the streams' layout, as x
                        copy16(dst + (v * A + XA + 1 + s) * P, a.grad_x_out.p + xo + s * D);
        }
    };
    const auto fetch_scalars = [&](int t, int stage) {
        float* const dst = scalars + stage * 32 + lane;
        if (lane < kGates) {
            if (MIX && a.h.has((size_t)t * kGates + lane, 1, 1)) copy4(dst, a.h.p + (size_t)t * kGates + lane);
        } else if (lane == kGates) {
            if (a.mean.has((size_t)t, 1, 4)) copy4(dst, a.mean.p + t);
        } else if (lane == kGates + 1) {
            if (a.rstd.has((size_t)t, 1, 4)) copy4(dst, a.rstd.p + t);
        }
    };
    // the dot products <X_j, du> of row t, left in sums[parity] by its warps
    const auto write_dots = [&](int t, int parity) {
        if (warp == 0) {
            const float* d = sums + (parity * Shape::kSums + 2 + (lane >> 3)) * 32;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if ((lane & 7) + 8 * k < warps) v += d[(lane & 7) + 8 * k];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
            const float o[1] = {v};
            if ((lane & 7) == 0) store_at<1>(a.grad_h, (size_t)t * kGates + (lane >> 3), o, 8);
        }
    };

#pragma unroll
    for (int q = 0; q < S; ++q) {
        if (first + q * groups < T) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) fetch_vector(mine + q * (Shape::kStage * P), first + q * groups, v);
            fetch_scalars(first + q * groups, q);
        }
        copies_commit();
    }

    if (group == 0)
#pragma unroll
        for (int k = 0; k < Shape::kGammaSlots; ++k) {
            const int c = c0 + k / (N / 4) * step + k % (N / 4) * 4;
            float g[4] = {0.f, 0.f, 0.f, 0.f};
            four_at<WORDS>(a.gamma, c, D, 1.f, g);
            gammas[k * G + i] = make_float4(g[0], g[1], g[2], g[3]);
        }
    __syncthreads();

    float2 gg[VPT][H], gb[VPT][H];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < H; ++k) gg[v][k] = gb[v][k] = pair(0.f);
    const float inv_d = 1.f / (float)D;
    int stage = 0, parity = 0, before = -1;
    for (int t = first; t < T; t += groups) {
        copies_wait<S - 1>();
        __syncwarp();
        const float4* const gates = reinterpret_cast<const float4*>(scalars + stage * 32);
        uint4* const row = mine + stage * (Shape::kStage * P);
        if constexpr (WORDS)
#pragma unroll
            for (int k = 0; k < Shape::kStage; ++k) {
                const int s = k % A;   // x, grad_y or the residual path's gradient
                const E* const p = s < XA ? a.x.p + (size_t)t * a.x_stride + s * D
                                   : s == XA ? a.grad_y.p + (size_t)t * a.gy_stride
                                             : a.grad_x_out.p + (size_t)t * a.x_stride + (s - XA - 1) * D;
                if (s <= XA || residual) align_chunks<E>(row - lane + k * P, misaligned(p), D - (c0 + k / A * step));
            }
        const float2 stat = reinterpret_cast<const float2*>(gates)[kGates / 2];
        const float2 rstd2 = pair(stat.y), mean2 = pair(-stat.x);
        // minus the mean at columns c, c + 1 of a vector from column `first` on; past D
        // 0, so that z is 0 there too: 0 - mean could overflow when multiplied by rstd
        const auto centre = [&](int first, int c) {
            if constexpr (!WORDS) return pair(first < D ? mean2.x : 0.f);
            return make_float2(first + c < D ? mean2.x : 0.f, first + c + 1 < D ? mean2.x : 0.f);
        };
        const float4 pre = MIX ? gates[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        const float p4[kStreams] = {pre.x, pre.y, pre.z, pre.w};
        float2 sw = pair(0.f), swz = pair(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float2 z[H], w[H];
            unpack<E>(row[v * A * P], z);
            if constexpr (MIX) {
#pragma unroll
                for (int k = 0; k < H; ++k) z[k] = mul2(z[k], pair(p4[0]));
#pragma unroll
                for (int s = 1; s < XA; ++s) {
                    float2 x[H];
                    unpack<E>(row[(v * A + s) * P], x);
#pragma unroll
                    for (int k = 0; k < H; ++k) z[k] = fma2(pair(p4[s]), x[k], z[k]);
                }
            }
            unpack<E>(row[(v * A + XA) * P], w);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                if ((k & 1) == 0) {
                    const float4 g = gammas[(v * (N / 4) + k / 2) * G + i];
                    z[k] = mul2(add2(z[k], centre(c0 + v * step, 2 * k)), rstd2);
                    z[k + 1] = mul2(add2(z[k + 1], centre(c0 + v * step, 2 * k + 2)), rstd2);
                    gg[v][k] = fma2(w[k], z[k], gg[v][k]);
                    gg[v][k + 1] = fma2(w[k + 1], z[k + 1], gg[v][k + 1]);
                    gb[v][k] = add2(gb[v][k], w[k]);
                    gb[v][k + 1] = add2(gb[v][k + 1], w[k + 1]);
                    w[k] = mul2(w[k], make_float2(g.x, g.y));
                    w[k + 1] = mul2(w[k + 1], make_float2(g.z, g.w));
                    sw = add2(sw, add2(w[k], w[k + 1]));
                    swz = fma2(w[k], z[k], fma2(w[k + 1], z[k + 1], swz));
                }
            }
        }
        float* const s0 = sums + parity * (Shape::kSums * 32);
        const float both = warp_sum_two(sw.x + sw.y, swz.x + swz.y);
        if ((lane & 15) == 0) s0[(lane >> 4) * 32 + warp] = both;
        group_sync(group, G);
        if constexpr (MIX)
            if (before >= 0) write_dots(before, parity ^ 1);
        float q = 0.f;   // lanes 0..7 add up the first sum, 8..15 the second
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if ((lane & 7) + 8 * k < warps) q += s0[(lane >> 3 & 1) * 32 + (lane & 7) + 8 * k];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) q += __shfl_xor_sync(kFullMask, q, o);
        const float mw = __shfl_sync(kFullMask, q, 0) * inv_d, mwz = __shfl_sync(kFullMask, q, 8) * inv_d;
        // du = rstd (w - mw - z mwz)
        const float2 a2 = pair(-stat.y * mw), b2 = pair(-stat.y * mwz);
        float2 dot[kStreams];
#pragma unroll
        for (int j = 0; j < kStreams; ++j) dot[j] = pair(0.f);
        const bool more = t + S * groups < T;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            uint32_t out[XA][4];   // packed results
#pragma unroll
            for (int half = 0; half < N / 4; ++half) {
                // four columns of every array at a time, to bound the registers
                const auto four = [&](int slot, float2 (&f)[2]) {
                    if constexpr (sizeof(E) == 4) {
                        const float4 raw = *reinterpret_cast<const float4*>(row + (v * A + slot) * P);
                        f[0] = make_float2(raw.x, raw.y);
                        f[1] = make_float2(raw.z, raw.w);
                    } else {
                        unpack_half<E>(reinterpret_cast<const uint2*>(row + (v * A + slot) * P)[half], f);
                    }
                };
                const float4 g = gammas[(v * (N / 4) + half) * G + i];
                float2 x[XA][2], z[2], w[2];
#pragma unroll
                for (int s = 0; s < XA; ++s) four(s, x[s]);
                four(XA, w);
                w[0] = mul2(w[0], make_float2(g.x, g.y));
                w[1] = mul2(w[1], make_float2(g.z, g.w));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    z[k] = x[0][k];
                    if constexpr (MIX) {
                        z[k] = mul2(z[k], pair(p4[0]));
#pragma unroll
                        for (int s = 1; s < XA; ++s) z[k] = fma2(pair(p4[s]), x[s][k], z[k]);
                    }
                    z[k] = mul2(add2(z[k], MIX ? centre(c0 + v * step, half * 4 + 2 * k) : mean2), rstd2);
                    w[k] = fma2(z[k], b2, fma2(w[k], rstd2, a2));
                }
                if constexpr (!MIX) {
                    pack_half<E>(w, &out[0][half * 2]);
                } else {
                    float2 o[kStreams][2];
#pragma unroll
                    for (int j = 0; j < kStreams; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            dot[j] = fma2(x[j][k], w[k], dot[j]);
                            o[j][k] = mul2(pair(p4[j]), w[k]);
                        }
                    if (residual)
#pragma unroll
                        for (int s = 0; s < kStreams; ++s) {
                            const float4 r = gates[2 + s];   // H_res[s][0..3]
                            const float r4[kStreams] = {r.x, r.y, r.z, r.w};
                            float2 f[2];
                            four(XA + 1 + s, f);
#pragma unroll
                            for (int j = 0; j < kStreams; ++j)
#pragma unroll
                                for (int k = 0; k < 2; ++k) o[j][k] = fma2(pair(r4[j]), f[k], o[j][k]);
                        }
#pragma unroll
                    for (int j = 0; j < kStreams; ++j) pack_half<E>(o[j], &out[j][half * 2]);
                }
            }
            if constexpr (WORDS) {
                const size_t o = at_row(t, a.gx_stride) + v * step;
#pragma unroll
                for (int j = 0; j < XA; ++j)
                    store_words(buffer, a.grad_x, o + j * D - lane * N, D - (c0 + v * step) + lane * N,
                                make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]), 6);
            } else if (c0 + v * step < D) {
                const size_t o = at_row(t, a.gx_stride) + v * step;
#pragma unroll
                for (int j = 0; j < XA; ++j)
                    if (a.grad_x.has(o + j * D, N, 6))
                        *reinterpret_cast<uint4*>(a.grad_x.p + o + j * D) =
                            make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]);
            }
            if (more) fetch_vector(row, t + S * groups, v);
        }
        if constexpr (MIX) {
            float d4[4] = {dot[0].x + dot[0].y, dot[1].x + dot[1].y, dot[2].x + dot[2].y, dot[3].x + dot[3].y};
            const float d = warp_sum_four(d4);
            if ((lane & 7) == 0) s0[(2 + (lane >> 3)) * 32 + warp] = d;
        }
        __syncwarp();   // every lane has read the row's scalars
        if (more) fetch_scalars(t + S * groups, stage);
        copies_commit();
        stage = stage + 1 == S ? 0 : stage + 1;
        parity ^= 1;
        before = t;
    }
    copies_wait<0>();
    if constexpr (MIX) {
        group_sync(group, G);
        if (before >= 0) write_dots(before, parity ^ 1);
    }
    if (a.grad_gamma.p == nullptr && a.grad_beta.p == nullptr) return;
    // The block's parameter gradients, its groups added in order (the slots are
    // free now).  MANY: all of their sums at once and a thread per column; else
    // one group after another, each on the sums before it, which leaves the last
    // one vectors to store.
    if constexpr (MANY) {
        float* const sum = reinterpret_cast<float*>(slots);   // [R][2][VPT * step]
        const int width = VPT * step;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int k = 0; k < H; k += 2) {
                float4* const at = reinterpret_cast<float4*>(sum + group * 2 * width + v * step + c0 + 2 * k);
                at[0] = make_float4(gg[v][k].x, gg[v][k].y, gg[v][k + 1].x, gg[v][k + 1].y);
                at[width / 4] = make_float4(gb[v][k].x, gb[v][k].y, gb[v][k + 1].x, gb[v][k + 1].y);
            }
        __syncthreads();
        for (int part = 0; part < 2; ++part)
            for (int c = tid; c < D; c += NT) {
                float o[1] = {sum[part * width + c]};
                for (int g = 1; g < R; ++g) o[0] += sum[(g * 2 + part) * width + c];
                store_at<1>(a.partial, ((size_t)blockIdx.x * 2 + part) * D + c, o, 9);
            }
        return;
    }
    float2* const acc = reinterpret_cast<float2*>(slots);   // [2][VPT][H][G]
    for (int g = 0; g < R; ++g) {
        __syncthreads();
        if (g != group) continue;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                float2* const p = acc + (v * H + k) * G + i;
                float2* const q = p + VPT * H * G;
                if (g > 0) {
                    gg[v][k] = add2(gg[v][k], *p);
                    gb[v][k] = add2(gb[v][k], *q);
                }
                if (g + 1 < R) {
                    *p = gg[v][k];
                    *q = gb[v][k];
                }
            }
    }
    if (group + 1 < R) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = c0 + v * step;
        if (c < D) {
            float o[N];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    const float2 q = part == 0 ? gg[v][k] : gb[v][k];
                    o[2 * k] = q.x;
                    o[2 * k + 1] = q.y;
                }
                const size_t at = ((size_t)blockIdx.x * 2 + part) * D + c;
                if constexpr (WORDS) {
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const float one[1] = {o[k]};
                        if (c + k < D) store_at<1>(a.partial, at + k, one, 9);
                    }
                } else {
                    store_at<N>(a.partial, at, o, 9);
                }
            }
        }
    }
}

// Parameter gradients: the partials of a column in a fixed order (16 threads
// each add every 16th part, then their sums are added in order).
// blockIdx.y: 0 gamma, 1 beta.  A thread's loads are all under way at once: the
// kernel is little but their latency.
constexpr int kReduceBatch = (kSms + 15) / 16;   // parts of the rows' kernels in one batch
__global__ void __launch_bounds__(512) reduce_parts_kernel(int64_t D, int64_t parts, bool accumulate,
                                                           Span<float> partial, Span<float> gamma, Span<float> beta) {
    __shared__ float s[16][33];
    ptx::grid_dependency_wait();
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const Span<float> out = blockIdx.y == 0 ? gamma : beta;
    if (out.p == nullptr) return;
    float sum = 0.f, o[1] = {0.f};
    if (c < D) {
        if (threadIdx.y == 0 && accumulate) o[0] = scalar_at(out, c, 11);
        for (int64_t first = threadIdx.y; first < parts; first += 16 * kReduceBatch) {
            float v[kReduceBatch];
#pragma unroll
            for (int k = 0; k < kReduceBatch; ++k) {
                const int64_t q = first + 16 * k;
                v[k] = q < parts ? scalar_at(partial, (q * 2 + blockIdx.y) * D + c, 10) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kReduceBatch; ++k) sum += v[k];
        }
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y != 0 || c >= D) return;
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) sum += s[q][threadIdx.x];
    o[0] += sum;
    store_at<1>(out, (size_t)c, o, 11);
}

template <typename E, bool MIX>
Params<E> params_of(const Args& a) {
    Params<E> p{};
    const auto extent = [&](int64_t stride, int64_t width) {
        return a.T == 0 ? (size_t)0 : (size_t)((a.T - 1) * stride + width);
    };
    const int64_t width = MIX ? kStreams * a.D : a.D;
    p.T = a.T;
    p.D = a.D;
    p.parts = part_count(a.T);
    p.x_stride = a.x_stride;
    p.y_stride = a.y_stride;
    p.gy_stride = a.gy_stride;
    p.gx_stride = a.gx_stride;
    p.eps = a.eps;
    p.accumulate = a.accumulate;
    p.x = {static_cast<const E*>(a.x), extent(a.x_stride, width)};
    p.h = {a.h, (size_t)(a.T * kGates)};
    p.gamma = {a.gamma, (size_t)a.D};
    p.beta = {a.beta, (size_t)a.D};
    p.y = {static_cast<E*>(a.y), extent(a.y_stride, a.D)};
    p.mean = {a.mean, (size_t)a.T};
    p.rstd = {a.rstd, (size_t)a.T};
    p.grad_y = {static_cast<const E*>(a.grad_y), extent(a.gy_stride, a.D)};
    p.grad_x_out = {static_cast<const E*>(a.grad_x_out), (size_t)(a.T * kStreams * a.D)};
    p.grad_x = {static_cast<E*>(a.grad_x), extent(a.gx_stride, width)};
    p.grad_h = {a.grad_h, (size_t)(a.T * kGates)};
    p.partial = {a.workspace, (size_t)(p.parts * 2 * a.D)};
    p.grad_gamma = {a.grad_gamma, (size_t)a.D};
    p.grad_beta = {a.grad_beta, (size_t)a.D};
    return p;
}

bool rows_packed(const void* p, int64_t stride, int pack) { return aligned16(p) && stride % pack == 0; }

// Launches forward_rows_kernel where the row fits its registers; false otherwise.
template <typename E, bool MIX, int N, int VPT>
bool forward_rows(const Params<E>& p, cudaError_t* e, cudaStream_t stream) {
    const int64_t threads = ((p.D + N - 1) / N + VPT - 1) / VPT;
    if (threads > 640) return false;
    const int G = (int)((threads + 31) / 32 * 32);
    int R = 256 / G < 1 ? 1 : 256 / G;             // blocks of about 256 threads
    while (R > 1 && (p.T + R - 1) / R < kSms) --R; // but first a block per SM
    *e = launch_early(forward_rows_kernel<E, MIX, N, VPT>, dim3((unsigned)((p.T + R - 1) / R)), dim3((unsigned)(G * R)), 0,
                      stream, p, G, R);
    return true;
}

// Likewise forward_ring_kernel.
template <typename E, bool MIX, bool WORDS, int VPT, int S>
bool forward_ring(const Params<E>& p, cudaError_t* e, cudaStream_t stream) {
    using Shape = ForwardShape<E, MIX, WORDS, VPT, S>;
    const int64_t threads = ((p.D + Shape::N - 1) / Shape::N + VPT - 1) / VPT;
    if (threads > Shape::kMaxThreads) return false;
    const int G = (int)((threads + 31) / 32 * 32);
    int R = Shape::kMaxThreads / G > 15 ? 15 : Shape::kMaxThreads / G;
    const int64_t spread = (p.T + kSms - 1) / kSms;
    if (R > spread) R = (int)spread;
    const size_t shared = Shape::bytes(G, R);
    if (shared > kMaxShared) return false;
    const int64_t grid = (p.T + R - 1) / R < kSms ? (p.T + R - 1) / R : kSms;
    auto kernel = forward_ring_kernel<E, MIX, WORDS, VPT, S>;
    static std::atomic<uint64_t> done{0};
    *e = allow_shared(kernel, kMaxShared, done);
    if (*e != cudaSuccess) return true;
    *e = launch_early(kernel, dim3((unsigned)grid), dim3((unsigned)(G * R)), shared, stream, p, G, R);
    return true;
}

template <typename E, bool MIX>
cudaError_t forward_typed(const Args& a, cudaStream_t stream) {
    const Params<E> p = params_of<E, MIX>(a);
    constexpr int N = Elem<E>::kPack;
    const bool packed = a.D % N == 0 && rows_packed(a.x, a.x_stride, N) && rows_packed(a.y, a.y_stride, N) &&
                        aligned16(a.gamma) && aligned16(a.beta);
    cudaError_t e = cudaSuccess;
    // Few rows: in registers.  A ring's start (its slots, gamma and beta in
    // shared memory) pays from more than one wave of blocks on: T=1, D=5120
    // takes 2.3 us in registers, 3.0 in the ring; T=304 3.2 and 3.7, T=608 5.9
    // and 4.6; D=1280: T=608 2.5 and 3.2, T=912 3.7 and 3.5.  Unaligned: D=1285:
    // T=1216 5.9 and 6.4, T=2432 10.4 and 10.5.
    const int64_t per_sm = a.T * a.D / kSms;
    const bool few = a.T <= 2 * kSms || per_sm <= (packed ? 5120 : 10240);
    if (packed) {
        if ((few && forward_rows<E, MIX, N, 1>(p, &e, stream)) ||
            forward_ring<E, MIX, false, MIX ? 2 : 4, MIX ? 2 : 3>(p, &e, stream))
            return e;
        if constexpr (sizeof(E) == 2) {
            if (forward_ring<E, MIX, false, MIX ? 2 : 4, MIX ? 1 : 2>(p, &e, stream)) return e;
        } else {
            if (forward_rows<E, MIX, N, 8>(p, &e, stream)) return e;
        }
    } else {
        if ((few && forward_rows<E, MIX, 1, 4>(p, &e, stream)) ||
            forward_ring<E, MIX, true, MIX ? 2 : 4, MIX ? 2 : 3>(p, &e, stream))
            return e;
        if constexpr (sizeof(E) == 2)
            if (forward_ring<E, MIX, true, MIX ? 2 : 4, MIX ? 1 : 2>(p, &e, stream)) return e;
    }
    return launch_early(packed && a.D % 8 == 0 ? forward_any_kernel<E, MIX, 8> : forward_any_kernel<E, MIX, 1>,
                        dim3((unsigned)a.T), dim3(kThreads), 0, stream, p);
}

// Launches backward_rows_kernel where the row fits its shape; false otherwise.
// *parts: the row groups it writes partial parameter gradients for.
template <typename E, bool MIX, bool WORDS, int VPT, int S, int MAX>
bool backward_rows(const Params<E>& p, int64_t* parts, cudaError_t* e, cudaStream_t stream) {
    using Shape = RowsShape<E, MIX, WORDS, VPT, S, MAX>;
    const int64_t vectors = (p.D + Shape::N - 1) / Shape::N, threads = (vectors + VPT - 1) / VPT;
    if (threads > Shape::kMaxThreads) return false;
    const int G = (int)((threads + 31) / 32 * 32);
    const int64_t blocks = kSms;
    int R = Shape::kMaxThreads / G;
    if (R > 15) R = 15;                                        // named barriers of a block
    const int64_t spread = (p.T + blocks - 1) / blocks;        // no more groups than rows to spread over the blocks
    if (R > spread) R = (int)spread;
    while (R > 1 && (Shape::bytes(G, R) > kMaxShared || Shape::sums_bytes(G, R) > Shape::rows_bytes(G))) --R;
    const size_t shared = Shape::bytes(G, R);
    if (shared > kMaxShared) return false;
    const int64_t grid = (p.T + R - 1) / R < blocks ? (p.T + R - 1) / R : blocks;
    *parts = grid;
    const auto launch = [&](auto kernel, std::atomic<uint64_t>& done) {
        *e = allow_shared(kernel, kMaxShared, done);
        if (*e == cudaSuccess)
            *e = launch_early(kernel, dim3((unsigned)grid), dim3((unsigned)(G * R)), shared, stream, p, G, R);
        return true;
    };
    // Six groups and more join their parameter gradients at once: T=16384, D=320
    // (15 groups) 13.7 us instead of 16.1, T=4096, D=64 6.1 instead of 8.4; with two,
    // T=1000, D=5120 FP32, 19.9 instead of 18.8.  (Collapsed rows would spill
    // registers; the wide shape has one group.)
    if constexpr (!MIX && S == 2) {
        static std::atomic<uint64_t> many{0};
        if (R > 5) return launch(backward_rows_kernel<E, MIX, WORDS, VPT, S, MAX, true>, many);
    }
    static std::atomic<uint64_t> few{0};
    return launch(backward_rows_kernel<E, MIX, WORDS, VPT, S, MAX, false>, few);
}

template <typename E, bool MIX>
cudaError_t backward_typed(const Args& a, cudaStream_t stream) {
    Params<E> p = params_of<E, MIX>(a);
    constexpr int N = Elem<E>::kPack;
    const bool packed = a.D % N == 0 && rows_packed(a.x, a.x_stride, N) && rows_packed(a.grad_y, a.gy_stride, N) &&
                        rows_packed(a.grad_x, a.gx_stride, N) && aligned16(a.gamma) && aligned16(a.grad_x_out);
    const bool params = a.grad_gamma != nullptr || a.grad_beta != nullptr;
    cudaError_t e = cudaSuccess;
    if (a.T > 0) {
        bool done = false;
        if constexpr (MIX) {
            if (packed)
                done = backward_rows<E, true, false, 1, 2, 640>(p, &p.parts, &e, stream) ||
                       backward_rows<E, true, false, 2, 1, 512>(p, &p.parts, &e, stream) ||
                       backward_rows<E, true, false, 2, 1, 640>(p, &p.parts, &e, stream);
            else
                done = backward_rows<E, true, true, 1, 2, 512>(p, &p.parts, &e, stream) ||
                       backward_rows<E, true, true, 2, 1, 512>(p, &p.parts, &e, stream);
        } else {
            done = packed ? backward_rows<E, false, false, 16 / N, 2, 640>(p, &p.parts, &e, stream) ||
                                backward_rows<E, false, false, 32 / N, 1, 512>(p, &p.parts, &e, stream)
                          : backward_rows<E, false, true, 16 / N, 2, 640>(p, &p.parts, &e, stream) ||
                                backward_rows<E, false, true, 32 / N, 1, 512>(p, &p.parts, &e, stream);
        }
        if (!done) {
            e = launch_early(packed && a.D % 8 == 0 ? backward_rows_any_kernel<E, MIX, 8> : backward_rows_any_kernel<E, MIX, 1>,
                             dim3((unsigned)a.T), dim3(kThreads), 0, stream, p);
            if (e == cudaSuccess && params)
                e = launch_early(backward_columns_any_kernel<E, MIX>,
                                 dim3((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)p.parts), dim3(kThreads), 0, stream, p);
        }
        if (e != cudaSuccess) return e;
    }
    if (!params) return cudaSuccess;
    return launch_early(reduce_parts_kernel, dim3((unsigned)((a.D + 31) / 32), 2), dim3(32, 16), 0, stream, a.D, p.parts,
                        a.accumulate, p.partial, p.grad_gamma, p.grad_beta);
}

}  // namespace

size_t workspace_bytes(int64_t T, int64_t D) { return (size_t)part_count(T) * 2 * (size_t)D * sizeof(float); }

cudaError_t forward(const Args& a, cudaStream_t stream) {
    if (a.h != nullptr) return forward_typed<bf16, true>(a, stream);
    if (a.type == 0) return forward_typed<bf16, false>(a, stream);
    if (a.type == 1) return forward_typed<__half, false>(a, stream);
    return forward_typed<float, false>(a, stream);
}

cudaError_t backward(const Args& a, cudaStream_t stream) {
    if (a.h != nullptr) return backward_typed<bf16, true>(a, stream);
    if (a.type == 0) return backward_typed<bf16, false>(a, stream);
    if (a.type == 1) return backward_typed<__half, false>(a, stream);
    return backward_typed<float, false>(a, stream);
}

cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace norm
}  // namespace ops
}  // namespace mhcpb
