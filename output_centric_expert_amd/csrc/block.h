// Internal interface of the operators around the MoE block: C ABI (block.hip) to kernels.
#pragma once

#include "prompt.h"

namespace moed {

// Activations (moed_activation of the C ABI).
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4, kActSigmoid = 5, kActTanh = 6;

// Dense product with an epilogue (linear.hip).
struct LinearArgs {
    const void* x;          // [B][K] bf16 or f32
    const void* w;          // [N][K] bf16 or f32
    const void* bias;       // [N] or null
    const void* residual;   // [B][N] or null
    void* out;              // [B][N]
    int B, K, N;
    int act;
    bool bias_bf16, residual_bf16, out_bf16;
};
size_t linear_workspace(int B, int K, int N, bool x_bf16, bool w_bf16);
hipError_t launch_linear(const LinearArgs& p, bool x_bf16, bool w_bf16, void* workspace, hipStream_t s);
// What launch_linear takes: see moed_selftest_linear.
void linear_path(int B, int K, int N, bool x_bf16, bool w_bf16, int32_t* path);

// The router's choice by scores and groups (route_scored.hip).
constexpr int kRouteMaxGroups = 64;
struct RouteArgs {
    const void* logits;     // [B][E]
    const float* bias;      // [E] or null
    int32_t* ids;           // [B][k + n_shared]
    float* w;
    int B, E, k, n_shared, n_group, topk_group;
    float routed_scale;
    bool logits_bf16, sigmoid, top2, renormalize;
};
hipError_t launch_route_scored(const RouteArgs& p, hipStream_t s);

// Norm behind a block, gate, residual, norm in front of the next (post_norm.hip).
constexpr int kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateFull = 3;
struct PostNormArgs {
    const void* y;          // [B][H], or [R][H] with position
    const int32_t* position;// [B][k] or null
    const float* topk_w;    // [B][k]
    const void* post_gain;  // [H] or null
    const void* gate;
    const void* residual;   // [B][H]
    void* residual_out;     // or null
    const void* gain;       // [H] or null
    void* out;              // or null
    uint8_t* q;             // [B][H] codes or null
    uint8_t* q_s;           // [B][H/32]
    int B, H, R, k;
    int gate_shape, gate_act;
    float post_eps, eps, scale, residual_scale;
    bool post_gain_bf16, gate_bf16, gain_bf16, out_bf16;
};
hipError_t launch_post_norm(const PostNormArgs& p, bool y_bf16, bool residual_bf16, hipStream_t s);

}  // namespace moed
