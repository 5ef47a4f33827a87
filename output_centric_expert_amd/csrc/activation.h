// Activations of the dense product and gates of the norm behind a block, in float32, on the hardware's base-2 exponential
// and reciprocal (one unit in the last place each). A sigmoid is off by (1.23 |v| + 5) 2^-24 of itself at most: the constant
// log2(e) by 0.23, its product with v by one, both of them |v| times in the exponential; exponential and reciprocal by two
// each, the sum by one. The epilogue of a product is bound by these instructions: five for a SiLU. Where the reciprocal is
// below 2^-126 (v < -87.3) it is 0, also where the exponential passes float32's range.
#pragma once

#include "block.h"

namespace moed {

namespace {

__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.442695041f * v));
}

// tanh(v): an odd polynomial (Taylor's) next to zero, where 1 - exp(-2|v|) would lose digits.
__device__ __forceinline__ float tanh_of(float v)
{
    const float a = __builtin_fabsf(v), e = __builtin_amdgcn_exp2f(-2.885390082f * a), q = v * v;
    float p = __builtin_fmaf(q, 0x1.664f48p-6f, -0x1.ba1ba2p-5f);
    p = __builtin_fmaf(q, p, 0x1.111112p-3f);
    p = __builtin_fmaf(q, p, -0x1.555556p-2f);
    const float near = __builtin_fmaf(v * q, p, v);
    const float far = __builtin_copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), v);
    return a < 0.25f ? near : far;
}

template <int V>
__device__ __forceinline__ void activate(float (&v)[V], int act)
{
    switch (act) {
    case kActSilu:
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = v[i] * sigmoid(v[i]);
        break;
    case kActGelu:                                            // 1 + erf(z) = erfc(-z), without cancellation
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = 0.5f * v[i] * erfcf(-0.70710678f * v[i]);
        break;
    case kActGeluTanh:                                        // (1 + tanh(u)) / 2 = sigmoid(2u)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = 1.5957691f * __builtin_fmaf(0.044715f * v[i] * v[i], v[i], v[i]);
            v[i] = v[i] * sigmoid(u);
        }
        break;
    case kActRelu:
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = v[i] < 0.0f ? 0.0f : v[i];
        break;
    case kActSigmoid:
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = sigmoid(v[i]);
        break;
    case kActTanh:
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = tanh_of(v[i]);
        break;
    default:
        break;
    }
}

}  // namespace

}  // namespace moed
