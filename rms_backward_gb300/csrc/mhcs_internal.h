// Internal interface of the operators around the projection stage: launches
// (mhcs_embed.cu, mhcs_norm.cu, mhcs_streams.cu) and their host checks
// (mhcs_api.cu).
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "mhcpb_internal.h"

namespace mhcpb {

// MHCPB_OK when ptr is device memory of `device`, else MHCPB_ERR_WRONG_DEVICE
// (defined in mhcpb_api.cu).
int check_device_pointer(const void* ptr, int device);

namespace ops {

constexpr int kStreams = 4;      // residual streams (the gate step's n)
constexpr int kGates = 24;       // gates per token: 4 pre, 4 post, 16 residual

struct DropArgs {                // see Drop in mhcs_common.cuh
    const uint64_t* rng;
    uint64_t sequence;
    uint32_t threshold;
    float scale;
};

// Lets a kernel's blocks have `bytes` of dynamic shared memory, once per device
// (`done` is the kernel's own; devices above 63 are set each time).
template <typename Kernel>
cudaError_t allow_shared(Kernel* kernel, int bytes, std::atomic<uint64_t>& done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
    if (e != cudaSuccess || (done.load(std::memory_order_acquire) & bit) != 0) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Launches a kernel whose blocks may start before the kernel ahead of it in the
// stream has ended; each of these kernels waits for that one by itself
// (griddepcontrol.wait) before its first global access.
template <typename... Params, typename... Values>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t shared, cudaStream_t stream,
                         Values... values) {
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = block;
    config.dynamicSmemBytes = shared;
    config.stream = stream;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(values)...);
}

namespace embed {
struct Args {
    int64_t T, V, D;
    int n_streams;
    int type;            // of the table (forward)
    const void* table;   // [V, D]
    void* x;             // BF16 [T, n_streams * D]
    const void* grad_x;  // BF16 [T, n_streams * D]
    const void* ids;     // [T] int32 or int64
    int id_bytes;
    float scale;
    float* grad_table;   // [V, D]
    bool accumulate;
    void* workspace;
};
size_t workspace_bytes(int64_t T, int64_t V, int64_t D);
cudaError_t forward(const Args& a, cudaStream_t stream);
cudaError_t backward(const Args& a, cudaStream_t stream);
cudaError_t setup();
cudaError_t checked_site(uint32_t* site);
}  // namespace embed

namespace norm {
struct Args {
    int64_t T, D;
    int type;
    const void* x;       // [T, D], or the streams [T, 4 D] BF16 when h is given
    const float* h;      // [T, 24] or null: the plain norm
    int64_t x_stride;
    const float* gamma;  // [D] or null (ones)
    const float* beta;   // [D] or null (zeros)
    float eps;
    void* y;
    int64_t y_stride;
    float* mean;         // [T]; null allowed in the forward
    float* rstd;
    // backward
    const void* grad_y;
    int64_t gy_stride;
    const void* grad_x_out;  // [T, 4 D] or null: the residual path's upstream gradient
    void* grad_x;
    int64_t gx_stride;
    float* grad_h;       // [T, 24], columns 0..3 written
    float* grad_gamma;   // [D] or null
    float* grad_beta;
    bool accumulate;
    float* workspace;
};
size_t workspace_bytes(int64_t T, int64_t D);
cudaError_t forward(const Args& a, cudaStream_t stream);
cudaError_t backward(const Args& a, cudaStream_t stream);
cudaError_t setup();
cudaError_t checked_site(uint32_t* site);
}  // namespace norm

namespace streams {
cudaError_t dropout(int64_t n, int type, const void* x, void* y, const DropArgs& d, cudaStream_t stream);
cudaError_t update_forward(int64_t T, int64_t D, const void* x, const void* y, const float* h,
                           const DropArgs& d, void* x_out, cudaStream_t stream);
cudaError_t update_backward(int64_t T, int64_t D, const void* x, const void* y, const float* h,
                            const DropArgs& d, const void* grad_x_out, void* grad_y, float* grad_h,
                            cudaStream_t stream);
cudaError_t setup();
cudaError_t checked_site(uint32_t* site);
}  // namespace streams

}  // namespace ops
}  // namespace mhcpb
