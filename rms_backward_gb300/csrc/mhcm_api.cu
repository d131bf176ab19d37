// Host side of the feed-forward block and of the orthogonalised update
// (include/mhcpb.h): shape, pointer, alignment and overlap checks, then the launches.
#include <cmath>

#include "mhcm_internal.h"
#include "mhcpb_check.cuh"
#include "mhcs_operands.h"

using namespace mhcpb;
using namespace mhcpb::ops;

namespace {

mhcpb_status_t ready(int device) {
    static std::atomic<uint64_t> done{0};
    return device_ready(device, done, [] {
        const cudaError_t e = ffn::setup();
        return e != cudaSuccess ? e : orth::setup();
    });
}

bool size_ok(int64_t n) { return n >= 1 && n <= MHCPB_MAX_K; }
// rows of `width`, or a multiple of 8 elements apart
bool pitch_ok(int64_t stride, int64_t width) { return stride == width || (stride_ok(stride, width) && stride % 8 == 0); }
Operand compact(const void* p, int64_t elements, int bytes, bool output) {
    return {p, p == nullptr ? 0 : (size_t)elements * (size_t)bytes, 16, output};
}
// as rows_of, aligned to 16 bytes
Operand pitched(const void* p, int64_t rows, int64_t stride, int64_t width, int bytes, bool output) {
    Operand o = rows_of(p, rows, stride, width, bytes, output);
    o.align = 16;
    return o;
}
Operand needed(Operand o, int64_t elements, int bytes) {   // an operand that may not be NULL
    o.bytes = (size_t)elements * (size_t)bytes;
    return o;
}

bool ffn_shape_ok(int64_t T, int64_t D, int64_t F) { return tokens_ok(T) && size_ok(D) && size_ok(F); }
bool ffn_types_ok(int type, int activation) {
    return (type == MHCPB_BF16 || type == MHCPB_FP16) && (activation == MHCPB_SILU || activation == MHCPB_GELU);
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- feed-forward
mhcpb_status_t mhcpb_ffn_forward_workspace_bytes(int64_t T, int64_t D, int64_t F, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!ffn_shape_ok(T, D, F)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = T == 0 ? 0 : ffn::forward_workspace_bytes(T, D, F);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_ffn_forward(int64_t T, int64_t D, int64_t F, int type, int activation, const void* x,
                                 int64_t x_stride, const void* w_gate, const void* w_up, const void* w_down, void* y,
                                 int64_t y_stride, void* gate, void* up, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    if (!ffn_types_ok(type, activation) || (gate == nullptr) != (up == nullptr)) return MHCPB_ERR_INVALID_ARG;
    if (!ffn_shape_ok(T, D, F) || !pitch_ok(x_stride, D) || !pitch_ok(y_stride, D)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t need = T == 0 ? 0 : ffn::forward_workspace_bytes(T, D, F);
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const int64_t weights = T == 0 ? 0 : D * F;
    const Operand o[8] = {pitched(x, T, x_stride, D, 2, false),
                          needed(compact(w_gate, 0, 2, false), weights, 2),
                          needed(compact(w_up, 0, 2, false), weights, 2),
                          needed(compact(w_down, 0, 2, false), weights, 2),
                          pitched(y, T, y_stride, D, 2, true),
                          compact(gate, T * F, 2, true),
                          compact(up, T * F, 2, true),
                          {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o, ready);
    if (s != MHCPB_OK || T == 0) return s;
    ffn::Args a{};
    a.T = T;
    a.D = D;
    a.F = F;
    a.type = type;
    a.activation = activation;
    a.x = x;
    a.x_stride = x_stride;
    a.w_gate = w_gate;
    a.w_up = w_up;
    a.w_down = w_down;
    a.y = y;
    a.y_stride = y_stride;
    a.gate = gate;
    a.up = up;
    a.workspace = workspace;
    const cudaError_t e = ffn::forward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (feed-forward)");
}

mhcpb_status_t mhcpb_ffn_backward_workspace_bytes(int64_t T, int64_t D, int64_t F, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!ffn_shape_ok(T, D, F)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = T == 0 ? 0 : ffn::backward_workspace_bytes(T, D, F);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_ffn_backward(int64_t T, int64_t D, int64_t F, int type, int activation, const void* x,
                                  int64_t x_stride, const void* w_gate, const void* w_up, const void* w_down,
                                  const void* gate, const void* up, const void* grad_y, int64_t grad_y_stride,
                                  void* grad_x, int64_t grad_x_stride, int grad_type, void* grad_w_gate,
                                  void* grad_w_up, void* grad_w_down, uint32_t flags, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (!ffn_types_ok(type, activation) || (grad_type != type && grad_type != MHCPB_FP32) ||
        (flags & ~(uint32_t)(MHCPB_ACCUMULATE_DW | MHCPB_TEST_INJECT_STALL)) != 0)
        return MHCPB_ERR_INVALID_ARG;
    if (!ffn_shape_ok(T, D, F) || !pitch_ok(x_stride, D) || !pitch_ok(grad_y_stride, D) ||
        !pitch_ok(grad_x_stride, D))
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    if (grad_x == nullptr && grad_w_gate == nullptr && grad_w_up == nullptr && grad_w_down == nullptr) return MHCPB_OK;
    const size_t need = T == 0 ? 0 : ffn::backward_workspace_bytes(T, D, F);
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const int64_t weights = T == 0 ? 0 : D * F, tf = T * F;
    const int gs = type_bytes(grad_type);
    Operand dx = pitched(grad_x, T, grad_x_stride, D, 2, true);
    if (grad_x == nullptr) dx.bytes = 0;
    const Operand o[12] = {pitched(x, T, x_stride, D, 2, false),
                           needed(compact(w_gate, 0, 2, false), weights, 2),
                           needed(compact(w_up, 0, 2, false), weights, 2),
                           needed(compact(w_down, 0, 2, false), weights, 2),
                           needed(compact(gate, 0, 2, false), tf, 2),
                           needed(compact(up, 0, 2, false), tf, 2),
                           pitched(grad_y, T, grad_y_stride, D, 2, false),
                           dx,
                           compact(grad_w_gate, D * F, gs, true),
                           compact(grad_w_up, D * F, gs, true),
                           compact(grad_w_down, D * F, gs, true),
                           {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o, ready);
    if (s != MHCPB_OK) return s;
    ffn::Args a{};
    a.T = T;
    a.D = D;
    a.F = F;
    a.type = type;
    a.activation = activation;
    a.x = x;
    a.x_stride = x_stride;
    a.w_gate = w_gate;
    a.w_up = w_up;
    a.w_down = w_down;
    a.gate = const_cast<void*>(gate);
    a.up = const_cast<void*>(up);
    a.grad_y = grad_y;
    a.gy_stride = grad_y_stride;
    a.grad_x = grad_x;
    a.gx_stride = grad_x_stride;
    a.grad_w[0] = grad_w_gate;
    a.grad_w[1] = grad_w_up;
    a.grad_w[2] = grad_w_down;
    a.grad_type = grad_type;
    a.accumulate = (flags & MHCPB_ACCUMULATE_DW) != 0;
    a.stall = (flags & MHCPB_TEST_INJECT_STALL) != 0;
    a.workspace = workspace;
    const cudaError_t e = ffn::backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (feed-forward gradient)");
}

// ---------------------------------------------------------------- orthogonalised update
mhcpb_status_t mhcpb_orthogonalize_workspace_bytes(int64_t m, int64_t n, size_t* bytes) {
    if (bytes == nullptr) return MHCPB_ERR_INVALID_ARG;
    if (!size_ok(m) || !size_ok(n)) return MHCPB_ERR_UNSUPPORTED_SHAPE;
    *bytes = orth::workspace_bytes(m, n);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_orthogonalize(int64_t m, int64_t n, int type, const void* g, int64_t g_stride, int steps,
                                   float eps, float scale, void* out, int64_t out_stride, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    if (!type_known(type) || !(eps >= 0.f) || !(eps < INFINITY) || !std::isfinite(scale)) return MHCPB_ERR_INVALID_ARG;
    if (!size_ok(m) || !size_ok(n) || !pitch_ok(g_stride, n) || !pitch_ok(out_stride, n) || steps < 1 ||
        steps > MHCPB_ORTH_MAX_STEPS)
        return MHCPB_ERR_UNSUPPORTED_SHAPE;
    const size_t need = orth::workspace_bytes(m, n);
    if (workspace_bytes < need) return MHCPB_ERR_WORKSPACE_TOO_SMALL;
    const Operand o[3] = {pitched(g, m, g_stride, n, type_bytes(type), false),
                          pitched(out, m, out_stride, n, 2, true),
                          {workspace, need, 16, true}};
    const mhcpb_status_t s = check_operands(o, ready);
    if (s != MHCPB_OK) return s;
    orth::Args a{};
    a.m = m;
    a.n = n;
    a.type = type;
    a.g = g;
    a.g_stride = g_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.steps = steps;
    a.eps = eps;
    a.scale = scale;
    a.workspace = workspace;
    const cudaError_t e = orth::orthogonalize(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHCPB_OK : cuda_failed(e, "launch (orthogonalised update)");
}

// ---------------------------------------------------------------- status
mhcpb_status_t mhcpb_operators_device_status(mhcpb_status_t* status, int clear) {
    if (status == nullptr) return MHCPB_ERR_INVALID_ARG;
    uint32_t words[2] = {kDevOk, kDevOk};
    cudaError_t e;
    if ((e = cudaDeviceSynchronize()) != cudaSuccess || (e = ffn::device_status(&words[0], clear != 0)) != cudaSuccess ||
        (e = orth::device_status(&words[1], clear != 0)) != cudaSuccess)
        return cuda_failed(e, "status words");
    *status = (mhcpb_status_t)(words[0] != kDevOk ? words[0] : words[1]);
    return MHCPB_OK;
}

mhcpb_status_t mhcpb_debug_checked_matrix_sites(uint32_t* sites, int* checked) {
    if (sites == nullptr || checked == nullptr) return MHCPB_ERR_INVALID_ARG;
    *checked = check::kEnabled ? 1 : 0;
    cudaError_t e;
    if ((e = ffn::checked_site(&sites[0])) != cudaSuccess || (e = orth::checked_site(&sites[1])) != cudaSuccess)
        return cuda_failed(e, "checked-build site words");
    return MHCPB_OK;
}

}  // extern "C"
