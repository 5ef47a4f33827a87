// What the kernels of the dense product share: loads of rows that begin at any element, and the epilogue
//   out[b][n] = act(v + bias[n]) + residual[b][n], rounded once.
#pragma once

#include "block.h"
#include "row_values.h"

namespace moed {

namespace {

__device__ __forceinline__ float activate(float v, int act)
{
    switch (act) {
    case kActSilu:
        return v / (1.0f + expf(-v));
    case kActGelu:
        return 0.5f * v * erfcf(-0.70710678f * v);            // 1 + erf(z) = erfc(-z), without cancellation
    case kActGeluTanh:                                        // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u))
        return v / (1.0f + expf(-1.5957691f * (v + 0.044715f * v * v * v)));
    case kActRelu:
        return v != v ? v : v > 0.0f ? v : 0.0f;
    case kActSigmoid:
        return 1.0f / (1.0f + expf(-v));
    case kActTanh:
        return tanhf(v);
    default:
        return v;
    }
}

__device__ __forceinline__ float value_at(bool bf16, const void* p, size_t at)
{
    return bf16 ? bf16_val(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// One output.
__device__ __forceinline__ void linear_store(const LinearArgs& p, float v, size_t b, int n)
{
    if (p.bias)
        v += value_at(p.bias_bf16, p.bias, (size_t)n);
    v = activate(v, p.act);
    const size_t at = b * (size_t)p.N + (size_t)n;
    if (p.residual)
        v += value_at(p.residual_bf16, p.residual, at);
    if (p.out_bf16)
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rne(v);
    else
        static_cast<float*>(p.out)[at] = v;
}

}  // namespace

}  // namespace moed
