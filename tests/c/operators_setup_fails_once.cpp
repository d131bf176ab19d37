/* Linked with the operators' host code (mhcs_api.cu) in the place of the CUDA
 * runtime and of the kernels: a set-up that fails on the first call of a
 * device must be tried again by the next one, and be done once when it has
 * succeeded.  Exits 0, or with the line of the first wrong answer. */
#include <cuda_runtime.h>

#include "mhcpb.h"
#include "mhcs_internal.h"

static int attribute_failures = 0, setup_failures = 0, setups = 0, launches = 0, device = 0, minor_version = 3;

extern "C" cudaError_t cudaGetDevice(int* d) {
    *d = device;
    return cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    if (attribute_failures > 0) {
        --attribute_failures;
        return cudaErrorUnknown;
    }
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : minor_version;
    return cudaSuccess;
}

namespace mhcpb {
int record_cuda_error(cudaError_t, const char*) { return MHCPB_ERR_CUDA; }
int check_device_pointer(const void*, int) { return MHCPB_OK; }
namespace ops {
static cudaError_t done() { return ++launches, cudaSuccess; }
namespace embed {
size_t workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
cudaError_t forward(const Args&, cudaStream_t) { return done(); }
cudaError_t backward(const Args&, cudaStream_t) { return done(); }
cudaError_t setup() {
    ++setups;
    if (setup_failures == 0) return cudaSuccess;
    --setup_failures;
    return cudaErrorMemoryAllocation;
}
cudaError_t checked_site(uint32_t*) { return cudaSuccess; }
}  // namespace embed
namespace norm {
size_t workspace_bytes(int64_t, int64_t) { return 0; }
cudaError_t forward(const Args&, cudaStream_t) { return done(); }
cudaError_t backward(const Args&, cudaStream_t) { return done(); }
cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t*) { return cudaSuccess; }
}  // namespace norm
namespace streams {
cudaError_t dropout(int64_t, int, const void*, void*, const DropArgs&, cudaStream_t) { return done(); }
cudaError_t update_forward(int64_t, int64_t, const void*, const void*, const float*, const DropArgs&, void*,
                           cudaStream_t) {
    return done();
}
cudaError_t update_backward(int64_t, int64_t, const void*, const void*, const float*, const DropArgs&, const void*,
                            void*, float*, cudaStream_t) {
    return done();
}
cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t*) { return cudaSuccess; }
}  // namespace streams
}  // namespace ops
}  // namespace mhcpb

static float x[8], y[8];
static mhcpb_status_t call() { return mhcpb_dropout(8, MHCPB_FP32, x, 0.f, nullptr, 0, y, nullptr); }

#define EXPECT(condition) \
    if (!(condition)) return __LINE__

int main() {
    setup_failures = 1;
    EXPECT(call() == MHCPB_ERR_CUDA && launches == 0);
    EXPECT(call() == MHCPB_OK && launches == 1 && setups == 2);
    EXPECT(call() == MHCPB_OK && launches == 2 && setups == 2);   // done once when it has succeeded
    device = 1;                                                   // another device has its own set-up
    attribute_failures = 1;
    EXPECT(call() == MHCPB_ERR_CUDA && setups == 2);
    EXPECT(call() == MHCPB_OK && setups == 3);
    device = 2;
    minor_version = 0;
    EXPECT(call() == MHCPB_ERR_UNSUPPORTED_DEVICE && call() == MHCPB_ERR_UNSUPPORTED_DEVICE && setups == 3);
    device = 64;
    EXPECT(call() == MHCPB_ERR_INVALID_ARG);
    return launches == 3 ? 0 : __LINE__;
}
