// What the feed-forward block's kernels share: the activation.
#pragma once
#include "mhcpb.h"

namespace mhcpb {
namespace ffn {

// act(g) and act'(g)
__device__ __forceinline__ float2 activate(float g, int kind) {
    if (kind == MHCPB_SILU) {
        const float q = __frcp_rn(1.f + __expf(-g));   // (__fdividef gives 0 beyond 2^126)
        return make_float2(g * q, q * (1.f + g * (1.f - q)));
    }
    const float p = 0.5f * erfcf(g * -0.70710678f);   // the normal distribution function, accurate in its tail
    return make_float2(g * p, p + g * (0.39894228f * __expf(-0.5f * g * g)));
}

}  // namespace ffn
}  // namespace mhcpb
