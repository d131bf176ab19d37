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
// FP32 statistics and sums; the variance is centred (two passes over the row),
// not a difference of squares.  The parameter gradients are summed over a
// number of row groups that depends on T alone, then over the groups in order:
// the same bits on every call and GPU.
#include "mhcs_common.cuh"
#include "mhcs_internal.h"

namespace mhcpb {
namespace ops {
namespace norm {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kMaxParts = 304;   // row groups of the parameter gradients

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
template <typename F>
__device__ __forceinline__ float scalar_at(const Span<F>& s, int64_t i, uint32_t site) {
    float v[1];
    load_at<1>(s, (size_t)i, v, site);
    return v[0];
}

// Any row length: the row is read again for each pass (from L1 or L2).
template <typename E, bool MIX, int N>
__global__ void __launch_bounds__(kThreads) forward_any_kernel(Params<E> a) {
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

// One row per block: its input gradient (and the gates').
template <typename E, bool MIX, int N>
__global__ void __launch_bounds__(kThreads) backward_rows_any_kernel(Params<E> a) {
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

// Parameter gradients: the partials of a column in order.  blockIdx.y: 0 gamma, 1 beta.
__global__ void __launch_bounds__(kThreads) reduce_parts_kernel(int64_t D, int64_t parts, bool accumulate,
                                                                Span<float> partial, Span<float> gamma,
                                                                Span<float> beta) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const Span<float> out = blockIdx.y == 0 ? gamma : beta;
    if (c >= D || out.p == nullptr) return;
    float s = 0.f;
    for (int64_t q = 0; q < parts; ++q) {
        float v[1];
        load_at<1>(partial, (size_t)((q * 2 + blockIdx.y) * D + c), v, 10);
        s += v[0];
    }
    float o[1] = {0.f};
    if (accumulate) load_at<1>(out, (size_t)c, o, 11);
    o[0] += s;
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

template <typename E, bool MIX>
cudaError_t forward_typed(const Args& a, cudaStream_t stream) {
    const Params<E> p = params_of<E, MIX>(a);
    constexpr int N = 8;
    const bool packed = a.D % N == 0 && rows_packed(a.x, a.x_stride, N) && rows_packed(a.y, a.y_stride, N) &&
                        aligned16(a.gamma) && aligned16(a.beta);
    if (packed)
        forward_any_kernel<E, MIX, N><<<(unsigned)a.T, kThreads, 0, stream>>>(p);
    else
        forward_any_kernel<E, MIX, 1><<<(unsigned)a.T, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename E, bool MIX>
cudaError_t backward_typed(const Args& a, cudaStream_t stream) {
    const Params<E> p = params_of<E, MIX>(a);
    constexpr int N = 8;
    const bool packed = a.D % N == 0 && rows_packed(a.x, a.x_stride, N) && rows_packed(a.grad_y, a.gy_stride, N) &&
                        rows_packed(a.grad_x, a.gx_stride, N) && aligned16(a.gamma) && aligned16(a.grad_x_out);
    const unsigned column_blocks = (unsigned)((a.D + kThreads - 1) / kThreads);
    if (a.T > 0) {
        if (packed)
            backward_rows_any_kernel<E, MIX, N><<<(unsigned)a.T, kThreads, 0, stream>>>(p);
        else
            backward_rows_any_kernel<E, MIX, 1><<<(unsigned)a.T, kThreads, 0, stream>>>(p);
        if (a.grad_gamma != nullptr || a.grad_beta != nullptr)
            backward_columns_any_kernel<E, MIX><<<dim3(column_blocks, (unsigned)p.parts), kThreads, 0, stream>>>(p);
    }
    if (a.grad_gamma != nullptr || a.grad_beta != nullptr)
        reduce_parts_kernel<<<dim3(column_blocks, 2), kThreads, 0, stream>>>(a.D, p.parts, a.accumulate, p.partial,
                                                                            p.grad_gamma, p.grad_beta);
    return cudaGetLastError();
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
