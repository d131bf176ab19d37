// What the feed-forward block's kernels share: the activation.
#pragma once
#include "mhcpb.h"

namespace mhcpb {
namespace ffn {

// act(g) and act'(g).  (gelu out of line: inlined for every element of an epilogue it is 100 KB of code.)
static __device__ __noinline__ float2 gelu(float g) {
    const float p = 0.5f * erfcf(g * -0.70710678f);   // the normal distribution function, accurate in its tail
    return make_float2(g * p, p + g * (0.39894228f * __expf(-0.5f * g * g)));
}
__device__ __forceinline__ float2 activate(float g, int kind) {
    if (kind == MHCPB_GELU) return gelu(g);
    const float e = __expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), q = g < 0.f ? e * r : r;   // 1 / (1 + exp(-g))
    return make_float2(g * q, q * (1.f + g * (1.f - q)));
}

}  // namespace ffn
}  // namespace mhcpb
