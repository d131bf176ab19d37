// Host side of the operators around the projection stage (include/mhcpb.h):
// shape, pointer, alignment and overlap checks, then the launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "mhcpb.h"
#include "mhcpb_check.cuh"
#include "mhcpb_internal.h"
#include "mhcs_internal.h"

using namespace mhcpb;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 24;

struct Operand {
    const void* ptr;
    size_t bytes;       // 0: no elements, the pointer is not looked at
    unsigned align;     // bytes, a power of two
    bool output;
    int in_place = -1;  // which of the call's operands, an input, this output may be (all of it, element for element)
    size_t pitch = 0;   // bytes from row to row and in a row of a strided operand; 0: compact
    size_t row = 0;
};

mhcpb_status_t cuda_failed(cudaError_t e, const char* what) {
    return (mhcpb_status_t)record_cuda_error(e, what);
}

// One-time set-up of the current device's kernels.  Only success is kept: after
// an error the next call tries again.  (Two first calls at once may both set up;
// what they set is the same.)
mhcpb_status_t device_ready(int device) {
    constexpr int kMaxDevices = 64;
    static std::atomic<uint64_t> ready{0};
    if (device < 0 || device >= kMaxDevices) return MHCPB_ERR_INVALID_ARG;
    const uint64_t bit = (uint64_t)1 << device;
    if ((ready.load(std::memory_order_acquire) & bit) != 0) return MHCPB_OK;
    int major = 0, minor = 0;
    cudaError_t e;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device)) != cudaSuccess)
        return cuda_failed(e, "cudaDeviceGetAttribute");
    if (major != 10 || minor != 3) return MHCPB_ERR_UNSUPPORTED_DEVICE;
    if ((e = ops::embed::setup()) != cudaSuccess || (e = ops::norm::setup()) != cudaSuccess ||
        (e = ops::streams::setup()) != cudaSuccess)
        return cuda_failed(e, "setup (operators)");
    ready.fetch_or(bit, std::memory_order_release);
    return MHCPB_OK;
}

// Whether two operands share a byte.  Of two with one distance between rows, the
// rows of one may lie between the other's, such as column slices of one buffer.
// (The kernels copy whole 16-byte chunks, whose bytes of other columns they do
// not use, and store nothing outside a row's columns.)  Otherwise the gaps
// between rows count as the operand's.
bool share_bytes(const Operand& a, const Operand& b) {
    const uintptr_t la = reinterpret_cast<uintptr_t>(a.ptr), lb = reinterpret_cast<uintptr_t>(b.ptr);
    if (la >= lb + b.bytes || lb >= la + a.bytes) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    const size_t ahead = lb >= la ? (lb - la) % a.pitch : (a.pitch - (la - lb) % a.pitch) % a.pitch;
    return ahead < a.row || ahead + b.row > a.pitch;   // from a row of a to the next row of b
}

// An operand with elements needs a pointer, aligned, in memory of the current
// device; an output overlaps no other operand (but may be its in_place input).
template <int N>
mhcpb_status_t check_operands(const Operand (&o)[N]) {
    for (const Operand& a : o)
        if (a.bytes > 0 && a.ptr == nullptr) return MHCPB_ERR_INVALID_ARG;
    for (const Operand& a : o)
        if (a.bytes > 0 && (reinterpret_cast<uintptr_t>(a.ptr) & (a.align - 1u)) != 0) return MHCPB_ERR_MISALIGNED;
    for (int i = 0; i < N; ++i) {
        if (!o[i].output || o[i].bytes == 0) continue;
        for (int j = 0; j < N; ++j) {
            if (j == i || o[j].bytes == 0) continue;
            if (j == o[i].in_place && o[j].ptr == o[i].ptr) continue;
            if (share_bytes(o[i], o[j])) return MHCPB_ERR_ALIASING;
        }
    }
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return cuda_failed(e, "cudaGetDevice");
    for (const Operand& a : o) {
        if (a.bytes == 0) continue;
        const int s = check_device_pointer(a.ptr, device);
        if (s != MHCPB_OK) return (mhcpb_status_t)s;
    }
    return device_ready(device);
}

int type_bytes(int type) { return type == MHCPB_FP32 ? 4 : 2; }
bool type_known(int type) { return type == MHCPB_BF16 || type == MHCPB_FP16 || type == MHCPB_FP32; }
bool tokens_ok(int64_t T) { return T >= 0 && T <= MHCPB_MAX_T; }
bool hidden_ok(int64_t D, int64_t n) { return D >= 1 && D <= MHCPB_MAX_K / n; }
// rows of `width` elements, `stride` apart
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= kMaxStride; }
Operand rows_of(const void* p, int64_t T, int64_t stride, int64_t width, int es, bool output) {
    const size_t bytes = T == 0 ? 0 : (size_t)((T - 1) * stride + width) * (size_t)es;
    return {p, bytes, (unsigned)es, output, -1, (size_t)stride * es, (size_t)width * es};
}

bool drop_args(float p, const void* rng, uint64_t sequence, ops::DropArgs* d) {
    if (!(p >= 0.f) || !(p < 1.f)) return false;
    d->rng = p > 0.f ? static_cast<const uint64_t*>(rng) : nullptr;
    d->sequence = sequence;
    // p < 1 in FP32 is at most 1 - 2^-24, so the threshold stays below 2^32
    d->threshold = (uint32_t)std::floor((double)p * 4294967296.0 + 0.5);
    d->scale = 1.f / (1.f - p);
    return true;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- embedding
mhcpb_status_t mhcpb_embed_forward(int64_t T, int64_t V, int64_t D, int n_streams, int type, const void* table,
                                   const void* ids, int id_bytes, float scale, void* x, void* stream) {
    if (!type_known(type) || (id_bytes != 4 && id_bytes != 8)) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || V < 1 || V > MHCPB_MAX_VOCAB || n_streams < 1 || n_streams > MHCPB_MAX_STREAMS ||
        !hidden_ok(D, n_streams))
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const int es = type_bytes(type);
    const Operand o[3] = {{table, T == 0 ? 0 : (size_t)(V * D) * es, (unsigned)es, false},
                          {ids, (size_t)T * id_bytes, (unsigned)id_bytes, false},
                          {x, (size_t)(T * n_streams * D) * 2, 2, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || T == 0) return s;
    ops::embed::Args a{};
    a.T = T;
    a.V = V;
    a.D = D;
    a.n_streams = n_streams;
    a.type = type;
    a.table = table;
    a.x = x;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.scale = scale;
    const cudaError_t e = ops::embed::forward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (embedding lookup)");
}

mhcpb_status_t mhcpb_embed_workspace_bytes(int64_t T, int64_t V, int64_t D, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || V < 1 || V > MHCPB_MAX_VOCAB || !hidden_ok(D, 1)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = ops::embed::workspace_bytes(T, V, D);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_embed_backward(int64_t T, int64_t V, int64_t D, int n_streams, const void* grad_x,
                                    const void* ids, int id_bytes, float scale, uint32_t flags, float* grad_table,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    if ((id_bytes != 4 && id_bytes != 8) || (flags & ~(uint32_t)MHCPB_ACCUMULATE_DW) != 0)
        return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || V < 1 || V > MHCPB_MAX_VOCAB || n_streams < 1 || n_streams > MHCPB_MAX_STREAMS ||
        !hidden_ok(D, n_streams))
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t need = ops::embed::workspace_bytes(T, V, D);
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const Operand o[4] = {{grad_x, (size_t)(T * n_streams * D) * 2, 2, false},
                          {ids, (size_t)T * id_bytes, (unsigned)id_bytes, false},
                          {grad_table, (size_t)(V * D) * 4, 4, true},
                          {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK) return s;
    ops::embed::Args a{};
    a.T = T;
    a.V = V;
    a.D = D;
    a.n_streams = n_streams;
    a.grad_x = grad_x;
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.scale = scale;
    a.grad_table = grad_table;
    a.accumulate = (flags & MHCPB_ACCUMULATE_DW) != 0;
    a.workspace = workspace;
    const cudaError_t e = ops::embed::backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (embedding gradient)");
}

// ---------------------------------------------------------------- layer norm
mhcpb_status_t mhcpb_layernorm_forward(int64_t T, int64_t D, int type, const void* x, int64_t x_stride,
                                       const float* gamma, const float* beta, float eps, void* y, int64_t y_stride,
                                       float* mean, float* rstd, void* stream) {
    if (!type_known(type) || !(eps >= 0.f) || !(eps < INFINITY) || (mean == nullptr) != (rstd == nullptr))
        return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, 1) || !stride_ok(x_stride, D) || !stride_ok(y_stride, D))
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const int es = type_bytes(type);
    const size_t t4 = (size_t)T * 4, d4 = (size_t)D * 4;
    const Operand o[6] = {rows_of(x, T, x_stride, D, es, false),
                          {gamma, gamma ? d4 : 0, 4, false},
                          {beta, beta ? d4 : 0, 4, false},
                          rows_of(y, T, y_stride, D, es, true),
                          {mean, mean ? t4 : 0, 4, true},
                          {rstd, rstd ? t4 : 0, 4, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || T == 0) return s;
    ops::norm::Args a{};
    a.T = T;
    a.D = D;
    a.type = type;
    a.x = x;
    a.x_stride = x_stride;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.y = y;
    a.y_stride = y_stride;
    a.mean = mean;
    a.rstd = rstd;
    const cudaError_t e = ops::norm::forward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (layer norm)");
}

mhcpb_status_t mhcpb_layernorm_workspace_bytes(int64_t T, int64_t D, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, 1)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = ops::norm::workspace_bytes(T, D);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_layernorm_backward(int64_t T, int64_t D, int type, const void* x, int64_t x_stride,
                                        const void* grad_y, int64_t grad_y_stride, const float* gamma,
                                        const float* mean, const float* rstd, void* grad_x, int64_t grad_x_stride,
                                        float* grad_gamma, float* grad_beta, uint32_t flags, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    if (!type_known(type) || (flags & ~(uint32_t)MHCPB_ACCUMULATE_DW) != 0) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, 1) || !stride_ok(x_stride, D) || !stride_ok(grad_y_stride, D) ||
        !stride_ok(grad_x_stride, D))
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const bool params = grad_gamma != nullptr || grad_beta != nullptr;
    const size_t need = params ? ops::norm::workspace_bytes(T, D) : 0;
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const int es = type_bytes(type);
    const size_t t4 = (size_t)T * 4, d4 = (size_t)D * 4;
    const Operand o[9] = {rows_of(x, T, x_stride, D, es, false),
                          rows_of(grad_y, T, grad_y_stride, D, es, false),
                          {gamma, gamma ? d4 : 0, 4, false},
                          {mean, t4, 4, false},
                          {rstd, t4, 4, false},
                          rows_of(grad_x, T, grad_x_stride, D, es, true),
                          {grad_gamma, grad_gamma ? d4 : 0, 4, true},
                          {grad_beta, grad_beta ? d4 : 0, 4, true},
                          {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || (T == 0 && !params)) return s;
    ops::norm::Args a{};
    a.T = T;
    a.D = D;
    a.type = type;
    a.x = x;
    a.x_stride = x_stride;
    a.gamma = gamma;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.grad_y = grad_y;
    a.gy_stride = grad_y_stride;
    a.grad_x = grad_x;
    a.gx_stride = grad_x_stride;
    a.grad_gamma = grad_gamma;
    a.grad_beta = grad_beta;
    a.accumulate = (flags & MHCPB_ACCUMULATE_DW) != 0;
    a.workspace = static_cast<float*>(workspace);
    const cudaError_t e = ops::norm::backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (layer norm gradient)");
}

// ---------------------------------------------------------------- dropout
mhcpb_status_t mhcpb_dropout(int64_t n, int type, const void* x, float p, const void* rng, uint64_t sequence,
                             void* y, void* stream) {
    ops::DropArgs d{};
    if (!type_known(type) || !drop_args(p, rng, sequence, &d)) return MHCPB_ERR_INVALID_ARG;
    if (n < 0 || n > (int64_t)MHCPB_MAX_T * MHCPB_MAX_K) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const int es = type_bytes(type);
    const Operand o[3] = {{x, (size_t)n * es, (unsigned)es, false},
                          {rng, p > 0.f ? (size_t)16 : 0, 8, false},
                          {y, (size_t)n * es, (unsigned)es, true, 0}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || n == 0) return s;
    const cudaError_t e = ops::streams::dropout(n, type, x, y, d, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (dropout)");
}

// ---------------------------------------------------------------- collapse and norm
mhcpb_status_t mhcpb_collapse_norm_forward(int64_t T, int64_t D, const void* x, const float* h, const float* gamma,
                                           const float* beta, float eps, void* y, float* mean, float* rstd,
                                           void* stream) {
    if (!(eps >= 0.f) || !(eps < INFINITY) || (mean == nullptr) != (rstd == nullptr)) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, ops::kStreams)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t t4 = (size_t)T * 4, d4 = (size_t)D * 4, td = (size_t)(T * D);
    const Operand o[7] = {{x, td * ops::kStreams * 2, 16, false},
                          {h, t4 * ops::kGates, 4, false},
                          {gamma, gamma ? d4 : 0, 4, false},
                          {beta, beta ? d4 : 0, 4, false},
                          {y, td * 2, 16, true},
                          {mean, mean ? t4 : 0, 4, true},
                          {rstd, rstd ? t4 : 0, 4, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || T == 0) return s;
    ops::norm::Args a{};
    a.T = T;
    a.D = D;
    a.x = x;
    a.x_stride = ops::kStreams * D;
    a.h = h;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.y = y;
    a.y_stride = D;
    a.mean = mean;
    a.rstd = rstd;
    const cudaError_t e = ops::norm::forward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (collapse and norm)");
}

mhcpb_status_t mhcpb_collapse_norm_workspace_bytes(int64_t T, int64_t D, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, ops::kStreams)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = ops::norm::workspace_bytes(T, D);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_collapse_norm_backward(int64_t T, int64_t D, const void* x, const float* h, const void* grad_y,
                                            const float* gamma, const float* mean, const float* rstd,
                                            const void* grad_x_out, void* grad_x, float* grad_h, float* grad_gamma,
                                            float* grad_beta, uint32_t flags, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    if ((flags & ~(uint32_t)MHCPB_ACCUMULATE_DW) != 0) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, ops::kStreams)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const bool params = grad_gamma != nullptr || grad_beta != nullptr;
    const size_t need = params ? ops::norm::workspace_bytes(T, D) : 0;
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const size_t t4 = (size_t)T * 4, d4 = (size_t)D * 4, td = (size_t)(T * D);
    const Operand o[12] = {{x, td * ops::kStreams * 2, 16, false},
                           {h, t4 * ops::kGates, 4, false},
                           {grad_y, td * 2, 16, false},
                           {gamma, gamma ? d4 : 0, 4, false},
                           {mean, t4, 4, false},
                           {rstd, t4, 4, false},
                           {grad_x_out, grad_x_out ? td * ops::kStreams * 2 : 0, 16, false},
                           {grad_x, td * ops::kStreams * 2, 16, true},
                           {grad_h, t4 * ops::kGates, 4, true},
                           {grad_gamma, grad_gamma ? d4 : 0, 4, true},
                           {grad_beta, grad_beta ? d4 : 0, 4, true},
                           {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || (T == 0 && !params)) return s;
    ops::norm::Args a{};
    a.T = T;
    a.D = D;
    a.x = x;
    a.x_stride = ops::kStreams * D;
    a.h = h;
    a.gamma = gamma;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.grad_y = grad_y;
    a.gy_stride = D;
    a.grad_x_out = grad_x_out;
    a.grad_x = grad_x;
    a.gx_stride = ops::kStreams * D;
    a.grad_h = grad_h;
    a.grad_gamma = grad_gamma;
    a.grad_beta = grad_beta;
    a.accumulate = (flags & MHCPB_ACCUMULATE_DW) != 0;
    a.workspace = static_cast<float*>(workspace);
    const cudaError_t e = ops::norm::backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (collapse and norm gradient)");
}

// ---------------------------------------------------------------- stream update
mhcpb_status_t mhcpb_update_forward(int64_t T, int64_t D, const void* x, const void* y, const float* h, float p,
                                    const void* rng, uint64_t sequence, void* x_out, void* stream) {
    ops::DropArgs d{};
    if (!drop_args(p, rng, sequence, &d)) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, ops::kStreams)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t td = (size_t)(T * D);
    const Operand o[5] = {{x, td * ops::kStreams * 2, 16, false},
                          {y, td * 2, 16, false},
                          {h, (size_t)(T * ops::kGates) * 4, 4, false},
                          {rng, p > 0.f && T > 0 ? (size_t)16 : 0, 8, false},
                          {x_out, td * ops::kStreams * 2, 16, true, 0}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || T == 0) return s;
    const cudaError_t e = ops::streams::update_forward(T, D, x, y, h, d, x_out, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (stream update)");
}

mhcpb_status_t mhcpb_update_backward(int64_t T, int64_t D, const void* x, const void* y, const float* h, float p,
                                     const void* rng, uint64_t sequence, const void* grad_x_out, void* grad_y,
                                     float* grad_h, void* stream) {
    ops::DropArgs d{};
    if (!drop_args(p, rng, sequence, &d)) return MHCPB_ERR_INVALID_ARG;
    if (!tokens_ok(T) || !hidden_ok(D, ops::kStreams)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t td = (size_t)(T * D);
    const Operand o[7] = {{x, td * ops::kStreams * 2, 16, false},
                          {y, td * 2, 16, false},
                          {h, (size_t)(T * ops::kGates) * 4, 4, false},
                          {rng, p > 0.f && T > 0 ? (size_t)16 : 0, 8, false},
                          {grad_x_out, td * ops::kStreams * 2, 16, false},
                          {grad_y, td * 2, 16, true},
                          {grad_h, (size_t)(T * ops::kGates) * 4, 4, true}};
    const mhcpb_status_t s = check_operands(o);
    if (s != MHCPB_OK || T == 0) return s;
    const cudaError_t e = ops::streams::update_backward(T, D, x, y, h, d, grad_x_out, grad_y, grad_h,
                                                        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (stream update gradient)");
}

mhcpb_status_t mhcpb_debug_checked_operator_sites(uint32_t* sites, int* checked) {
    if (sites == nullptr || checked == nullptr) return MHCPB_ERR_INVALID_ARG;
    *checked = check::kEnabled ? 1 : 0;
    cudaError_t e;
    if ((e = ops::embed::checked_site(&sites[0])) != cudaSuccess ||
        (e = ops::norm::checked_site(&sites[1])) != cudaSuccess ||
        (e = ops::streams::checked_site(&sites[2])) != cudaSuccess)
        return cuda_failed(e, "checked-build site words");
    return MHCPB_OK;
}

}  // extern "C"
