// Host checks that the operators' entry points share: an operand's pointer,
// alignment, device and overlap, the limits of sizes and strides, a device's
// one-time set-up.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mhcpb.h"
#include "mhcs_internal.h"

namespace mhcpb {
namespace ops {

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

inline mhcpb_status_t cuda_failed(cudaError_t e, const char* what) {
    return (mhcpb_status_t)record_cuda_error(e, what);
}

// One-time set-up of the current device's kernels by `setup`, kept in `ready`.  Only
// success is kept: after an error the next call tries again.  (Two first calls at
// once may both set up; what they set is the same.)
template <class Setup>
mhcpb_status_t device_ready(int device, std::atomic<uint64_t>& ready, Setup setup) {
    constexpr int kMaxDevices = 64;
    if (device < 0 || device >= kMaxDevices) return MHCPB_ERR_INVALID_ARG;
    const uint64_t bit = (uint64_t)1 << device;
    if ((ready.load(std::memory_order_acquire) & bit) != 0) return MHCPB_OK;
    int major = 0, minor = 0;
    cudaError_t e;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device)) != cudaSuccess)
        return cuda_failed(e, "cudaDeviceGetAttribute");
    if (major != 10 || minor != 3) return MHCPB_ERR_UNSUPPORTED_DEVICE;
    if ((e = setup()) != cudaSuccess) return cuda_failed(e, "setup (operators)");
    ready.fetch_or(bit, std::memory_order_release);
    return MHCPB_OK;
}

// Whether two operands share a byte.  Of two with one distance between rows, the
// rows of one may lie between the other's, such as column slices of one buffer.
// (The kernels copy whole 16-byte chunks, whose bytes of other columns they do
// not use, and store nothing outside a row's columns.)  Otherwise the gaps
// between rows count as the operand's.
inline bool share_bytes(const Operand& a, const Operand& b) {
    const uintptr_t la = reinterpret_cast<uintptr_t>(a.ptr), lb = reinterpret_cast<uintptr_t>(b.ptr);
    if (la >= lb + b.bytes || lb >= la + a.bytes) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    const size_t ahead = lb >= la ? (lb - la) % a.pitch : (a.pitch - (la - lb) % a.pitch) % a.pitch;
    return ahead < a.row || ahead + b.row > a.pitch;   // from a row of a to the next row of b
}

// An operand with elements needs a pointer, aligned, in memory of the current
// device; an output overlaps no other operand (but may be its in_place input).
// ready: the device's set-up.
template <int N, class Ready>
mhcpb_status_t check_operands(const Operand (&o)[N], Ready ready) {
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
    return ready(device);
}

inline int type_bytes(int type) { return type == MHCPB_FP32 ? 4 : 2; }
inline bool type_known(int type) { return type == MHCPB_BF16 || type == MHCPB_FP16 || type == MHCPB_FP32; }
inline bool tokens_ok(int64_t T) { return T >= 0 && T <= MHCPB_MAX_T; }
inline bool hidden_ok(int64_t D, int64_t n) { return D >= 1 && D <= MHCPB_MAX_K / n; }
// rows of `width` elements, `stride` apart
inline bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= kMaxStride; }
inline Operand rows_of(const void* p, int64_t T, int64_t stride, int64_t width, int es, bool output) {
    const size_t bytes = T == 0 ? 0 : (size_t)((T - 1) * stride + width) * (size_t)es;
    return {p, bytes, (unsigned)es, output, -1, (size_t)stride * es, (size_t)width * es};
}

}  // namespace ops
}  // namespace mhcpb
