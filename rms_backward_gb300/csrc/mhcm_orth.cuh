// What the kernels of the orthogonalised update share: the polynomial, G's elements,
// its norm and the division by it.
#pragma once
#include "mhcm_product.cuh"

namespace mhcpb {
namespace orth {

using product::Matrix;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

// 1 / (|G|_F + eps) as a product that neither overflows nor loses bits: three factors.
struct Inverse {
    float p, q, r;
};
__device__ __forceinline__ float scaled(float g, const Inverse& f) { return g * f.p * f.q * f.r; }

// G's elements by its type
struct Input {
    const void* ptr;
    int type;
    int64_t rows, ld, cols;
    // elements as they are stored (a 16-bit type's in the first half of the words), and as FP32
    bool by_eight() const { return cols % 8 == 0 && ld * (type == MHCPB_FP32 ? 4 : 2) % 16 == 0; }
    template <class Span>
    __device__ __forceinline__ product::Raw<float, Span> raw(const Span& at, uint32_t site) const {
        const size_t n = (size_t)((rows - 1) * ld + cols);
        if (type == MHCPB_FP32) return Matrix<const float>{static_cast<const float*>(ptr), ld, n}.raw(at, site);
        const auto h = Matrix<const __half>{static_cast<const __half*>(ptr), ld, n}.raw(at, site);
        product::Raw<float, Span> r{};
#pragma unroll
        for (int i = 0; i < h.words; ++i) r.u[i] = h.u[i];
        return r;
    }
    template <class Span>
    __device__ __forceinline__ void to(const product::Raw<float, Span>& r, float (&v)[Span::n]) const {
        if (type == MHCPB_FP32) return r.to(v);
        if (type == MHCPB_BF16) {
            product::Raw<__nv_bfloat16, Span> h;
#pragma unroll
            for (int i = 0; i < h.words; ++i) h.u[i] = r.u[i];
            return h.to(v);
        }
        product::Raw<__half, Span> h;
#pragma unroll
        for (int i = 0; i < h.words; ++i) h.u[i] = r.u[i];
        h.to(v);
    }
};

// Sums of squares of the small, middling and large elements apart, the outer two
// scaled, so that none overflows or vanishes (Blue, ACM TOMS 4, 1978).
struct Squares {
    float low = 0.f, mid = 0.f, high = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float m = fabsf(v);
        if (m > 0x1p50f) {
            const float t = v * 0x1p-80f;
            high = fmaf(t, t, high);
        } else if (m < 0x1p-50f) {
            const float t = v * 0x1p80f;
            low = fmaf(t, t, low);
        } else {
            mid = fmaf(v, v, mid);   // NaN too
        }
    }
    __device__ __forceinline__ double sum() const { return (double)mid + (double)high * 0x1p160 + (double)low * 0x1p-160; }
};

// From |G| + eps.
__device__ __forceinline__ Inverse inverse_of(double total) {
    int e;
    const double f = frexp(total, &e);   // total = f 2^e, f in [1/2, 1)
    e = min(max(e, -240), 240);
    Inverse inv;
    inv.r = (float)(1.0 / f);
    inv.p = exp2f((float)(-e / 2));
    inv.q = exp2f((float)(-(e - e / 2)));
    return inv;
}

}  // namespace orth
}  // namespace mhcpb
