// What the feed-forward block's kernels share: the activation.
#pragma once
#include "mhcpb.h"

namespace mhcpb {
namespace ffn {

// The normal distribution function at -|g|, from e = exp(-g^2 / 2): e / 2 times the scaled
// complementary error function of z = |g| / sqrt 2, which is t times a polynomial in
// t = 1 / (1 + 0.4 z) in [0, 1]: degree 8, fitted by reweighted least squares to the function
// in FP64; with the constants as rounded here off by 2e-7 of it at most (in FP32 arithmetic 4.6e-7), in the
// tail too.
__device__ __forceinline__ float normal_tail(float g, float e) {
    const float t = __fdividef(1.f, 1.f + 0.28284271f * fabsf(g));
    float p = 0.05026213f;
    p = fmaf(p, t, -0.18290149f);
    p = fmaf(p, t, 0.16908546f);
    p = fmaf(p, t, -0.0056075598f);
    p = fmaf(p, t, 0.14143145f);
    p = fmaf(p, t, 0.16854198f);
    p = fmaf(p, t, 0.20784270f);
    p = fmaf(p, t, 0.22566959f);
    p = fmaf(p, t, 0.22567587f);
    return 0.5f * e * (p * t);
}
// act(g) and act'(g)
__device__ __forceinline__ float2 activate(float g, int kind) {
    if (kind == MHCPB_GELU) {
        const float e = __expf(-0.5f * g * g), tail = normal_tail(g, e), p = g < 0.f ? tail : 1.f - tail;
        return make_float2(g * p, p + g * (0.39894228f * e));
    }
    const float e = __expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), q = g < 0.f ? e * r : r;   // 1 / (1 + exp(-g))
    return make_float2(g * q, q * (1.f + g * (1.f - q)));
}

}  // namespace ffn
}  // namespace mhcpb
