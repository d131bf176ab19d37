// Dropout, and the residual streams' update with its gradient.
//
//   dropout          y_e = kept_e ? x_e / (1 - p) : 0
//   update           X'_i = sum_j H_res[i][j] X_j + H_post[i] drop(y)        i, j < 4
//   its gradient     dy = drop(sum_i H_post[i] dX'_i)
//                    dH_post[i] = <dX'_i, drop(y)>,  dH_res[i][j] = <dX'_i, X_j>
//
// FP32 arithmetic, one rounding to BF16 at each store.  The mask is drawn
// again from the counter wherever it is needed, so it takes no memory.  All
// three are bound by HBM: 4, 18 and 20 bytes per BF16 element of y.
#include "mhcs_common.cuh"
#include "mhcs_internal.h"

namespace mhcpb {
namespace ops {
namespace streams {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename E, int N>
__global__ void __launch_bounds__(kThreads) dropout_kernel(int64_t n, Span<const E> x, Span<E> y, Drop d) {
    const DropKey key = drop_key(d);
    const int64_t step = (int64_t)gridDim.x * kThreads * N;
    for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * N; e < n; e += step) {
        if (e + N <= n) {
            float v[N];
            load_at<N>(x, e, v, 0);
            drop<N>(d, key, e, v);
            store_at<N>(y, e, v, 1);
        } else {
            for (int64_t i = e; i < n; ++i) {
                float v[1];
                load_at<1>(x, i, v, 0);
                drop<1>(d, key, i, v);
                store_at<1>(y, i, v, 1);
            }
        }
    }
}

// One block per token; N columns of every stream per thread and step.
template <int N>
__global__ void __launch_bounds__(kThreads) update_forward_kernel(int64_t D, Span<const bf16> x,
                                                                  Span<const bf16> y, Span<const float> h,
                                                                  Drop d, Span<bf16> x_out) {
    __shared__ float gate[kGates];
    const int64_t t = blockIdx.x;
    if (threadIdx.x < kGates) {
        float v[1];
        load_at<1>(h, t * kGates + threadIdx.x, v, 2);
        gate[threadIdx.x] = v[0];
    }
    __syncthreads();
    const DropKey key = drop_key(d);
    const int64_t row = t * kStreams * D;
    for (int64_t c = (int64_t)threadIdx.x * N; c < D; c += kThreads * N) {
        float xs[kStreams][N], yv[N];
        load_at<N>(y, t * D + c, yv, 3);
#pragma unroll
        for (int j = 0; j < kStreams; ++j) load_at<N>(x, row + j * D + c, xs[j], 4);
        drop<N>(d, key, (uint64_t)(t * D + c), yv);
#pragma unroll
        for (int i = 0; i < kStreams; ++i) {
            float o[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                o[k] = gate[4 + i] * yv[k];
#pragma unroll
                for (int j = 0; j < kStreams; ++j) o[k] = fmaf(gate[8 + 4 * i + j], xs[j][k], o[k]);
            }
            store_at<N>(x_out, row + i * D + c, o, 5);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads) update_backward_kernel(int64_t D, Span<const bf16> x,
                                                                   Span<const bf16> y, Span<const float> h,
                                                                   Drop d, Span<const bf16> gout,
                                                                   Span<bf16> gy, Span<float> gh) {
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

template <typename E>
cudaError_t dropout_typed(int64_t n, const void* x, void* y, const Drop& d, cudaStream_t stream) {
    constexpr int N = 8;
    const Span<const E> xs{static_cast<const E*>(x), (size_t)n};
    const Span<E> ys{static_cast<E*>(y), (size_t)n};
    if (aligned16(x) && aligned16(y)) {
        const int64_t blocks = (n + kThreads * N - 1) / (kThreads * N);
        dropout_kernel<E, N><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), kThreads, 0, stream>>>(n, xs, ys, d);
    } else {
        const int64_t blocks = (n + kThreads - 1) / kThreads;
        dropout_kernel<E, 1><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), kThreads, 0, stream>>>(n, xs, ys, d);
    }
    return cudaGetLastError();
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
    if (D % 8 == 0)
        update_forward_kernel<8><<<(unsigned)T, kThreads, 0, stream>>>(D, xs, ys, hs, d, os);
    else
        update_forward_kernel<1><<<(unsigned)T, kThreads, 0, stream>>>(D, xs, ys, hs, d, os);
    return cudaGetLastError();
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
    if (D % 8 == 0)
        update_backward_kernel<8><<<(unsigned)T, kThreads, 0, stream>>>(D, xs, ys, hs, d, gs, gys, ghs);
    else
        update_backward_kernel<1><<<(unsigned)T, kThreads, 0, stream>>>(D, xs, ys, hs, d, gs, gys, ghs);
    return cudaGetLastError();
}

cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace streams
}  // namespace ops
}  // namespace mhcpb
