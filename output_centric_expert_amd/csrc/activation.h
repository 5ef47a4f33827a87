// Activations of the dense product and gates of the norm behind a block, in float32.
//
// exp(-x) is the hardware's base-2 exponential of -x log2(e), whose product is taken with its rounding error, so that the
// error stays at two units in the last place over the whole range (the bare exponential of a rounded product is off by
// |x| 2^-24); sigmoids are its reciprocal. Arguments below -87 count as -87: the results there are 0 to 1e-36.
#pragma once

#include "block.h"

namespace moed {

namespace {

// exp(-x) for -88 < x; x up to infinity.
__device__ __forceinline__ float exp_neg(float x)
{
    x = x > 200.0f ? 200.0f : x;
    const float t = -x * 0x1.715476p+0f;
    const float low = __builtin_fmaf(-x, 0x1.4ae0bep-26f, __builtin_fmaf(-x, 0x1.715476p+0f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, low * 0x1.62e43p-1f, e);
}

__device__ __forceinline__ float at_least_m87(float v) { return v < -87.0f ? -87.0f : v; }      // a NaN stays

__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + exp_neg(at_least_m87(v)));
}

// tanh(v): an odd polynomial (Taylor's) next to zero, where 1 - exp(-2|v|) would lose digits.
__device__ __forceinline__ float tanh_of(float v)
{
    const float a = __builtin_fabsf(v), e = exp_neg(2.0f * a), q = v * v;
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
            v[i] = at_least_m87(v[i]) * sigmoid(v[i]);
        break;
    case kActGelu:                                            // 1 + erf(z) = erfc(-z), without cancellation
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = 0.5f * at_least_m87(v[i]) * erfcf(-0.70710678f * at_least_m87(v[i]));
        break;
    case kActGeluTanh:                                        // (1 + tanh(u)) / 2 = sigmoid(2u)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = 1.5957691f * __builtin_fmaf(0.044715f * v[i] * v[i], v[i], v[i]);
            v[i] = at_least_m87(v[i]) * sigmoid(u);
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
