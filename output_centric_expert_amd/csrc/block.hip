// C ABI of the operators around the MoE block (moe_linear, moe_route_scored,
// moe_post_norm): argument checks and launches. All arithmetic runs in the
// kernels; no call keeps state between calls.
#include "moedecode.h"
#include "block.h"

namespace {

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bool dtype_ok(int d) { return d == MOED_BF16 || d == MOED_F32; }

// A buffer of `count` elements of a dtype, or of bytes.
struct Range {
    const void* p;
    unsigned long long bytes;
    int dtype;
};
inline Range range(const void* p, int dtype, unsigned long long count) { return {p, count * (dtype == MOED_BF16 ? 2 : 4), dtype}; }
inline Range bytes(const void* p, unsigned long long count) { return {p, count, -1}; }
inline bool overlap(const Range& a, const Range& b)
{
    const uintptr_t s = (uintptr_t)a.p, t = (uintptr_t)b.p;
    return s && t && s < t + b.bytes && t < s + a.bytes;
}
// out over an operand that is read once, by the thread that writes the same element: one buffer of one type.
inline bool in_place(const Range& out, const Range& in) { return out.p == in.p && out.dtype == in.dtype; }

static_assert(moed::kActNone == MOED_ACT_NONE && moed::kActSilu == MOED_ACT_SILU && moed::kActGelu == MOED_ACT_GELU &&
                  moed::kActGeluTanh == MOED_ACT_GELU_TANH && moed::kActRelu == MOED_ACT_RELU &&
                  moed::kActSigmoid == MOED_ACT_SIGMOID && moed::kActTanh == MOED_ACT_TANH,
              "activations are the ABI's");
static_assert(moed::kGateNone == MOED_GATE_NONE && moed::kGateToken == MOED_GATE_TOKEN &&
                  moed::kGateChannel == MOED_GATE_CHANNEL && moed::kGateFull == MOED_GATE_FULL,
              "gate shapes are the ABI's");

constexpr int kMaxRows = 1 << 28;
constexpr int kMaxRowLength = 1 << 20;

bool linear_ok(int B, int K, int N)
{
    return B >= 0 && B < moed::kMaxTokens && K >= 1 && N >= 1 && K < kMaxRowLength && N < kMaxRowLength &&
           (long long)K * N < (1LL << 32) && (long long)B * K < (1LL << 40) && (long long)B * N < (1LL << 38);
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int B, int K, int N, int x_dtype, int w_dtype)
{
    if (!linear_ok(B, K, N) || B == 0 || !dtype_ok(x_dtype) || !dtype_ok(w_dtype))
        return 0;
    return moed::linear_workspace(B, K, N, x_dtype == MOED_BF16, w_dtype == MOED_BF16);
}

int moed_selftest_linear(int B, int K, int N, int x_dtype, int w_dtype, int32_t* path)
{
    if (!linear_ok(B, K, N) || B == 0)
        return MOED_ERR_SHAPE;
    if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype))
        return MOED_ERR_DTYPE;
    if (!path)
        return MOED_ERR_NULL;
    moed::linear_path(B, K, N, x_dtype == MOED_BF16, w_dtype == MOED_BF16, path);
    return MOED_OK;
}

int moe_linear(const void* x, int x_dtype, const void* w, int w_dtype, const void* bias, int bias_dtype, int activation,
               const void* residual, int residual_dtype, void* out, int out_dtype, int B, int K, int N, void* workspace,
               size_t workspace_bytes, void* stream)
{
    if (!linear_ok(B, K, N))
        return MOED_ERR_SHAPE;
    if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || (bias && !dtype_ok(bias_dtype)) ||
        (residual && !dtype_ok(residual_dtype)) || !dtype_ok(out_dtype) || activation < MOED_ACT_NONE ||
        activation > MOED_ACT_TANH)
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    if (!x || !w || !out)
        return MOED_ERR_NULL;
    const size_t need = moed::linear_workspace(B, K, N, x_dtype == MOED_BF16, w_dtype == MOED_BF16);
    if (need && !workspace)
        return MOED_ERR_NULL;
    if (workspace_bytes < need)
        return MOED_ERR_WORKSPACE;
    if (!aligned16(x) || !aligned16(w) || !aligned16(residual) || !aligned16(out) || (need && !aligned16(workspace)) ||
        (bias && !aligned(bias, bias_dtype == MOED_BF16 ? 2 : 4)))
        return MOED_ERR_ALIGN;
    const unsigned long long rows = (unsigned long long)B, outputs = rows * (unsigned)N;
    const Range o = range(out, out_dtype, outputs), r = range(residual, residual_dtype, outputs);
    const Range ws = bytes(need ? workspace : nullptr, need);
    const Range in[] = {range(x, x_dtype, rows * (unsigned)K), range(w, w_dtype, (unsigned long long)N * (unsigned)K),
                        range(bias, bias_dtype, (unsigned)N)};
    for (const Range& i : in)                                 // read after the first outputs and sums are written
        if (overlap(o, i) || overlap(ws, i))
            return MOED_ERR_SHAPE;
    if ((overlap(o, r) && !in_place(o, r)) || overlap(ws, r) || overlap(ws, o))
        return MOED_ERR_SHAPE;
    moed::LinearArgs p;
    p.x = x; p.w = w; p.bias = bias; p.residual = residual; p.out = out;
    p.B = B; p.K = K; p.N = N; p.act = activation;
    p.bias_bf16 = bias_dtype == MOED_BF16;
    p.residual_bf16 = residual_dtype == MOED_BF16;
    p.out_bf16 = out_dtype == MOED_BF16;
    return moed::abi_status(moed::launch_linear(p, x_dtype == MOED_BF16, w_dtype == MOED_BF16, workspace,
                                                static_cast<hipStream_t>(stream)));
}

int moe_route_scored(const void* logits, int logits_dtype, const float* bias, int score, int n_group, int topk_group,
                     int group_score, int renormalize, int B, int E, int k, int n_shared, float routed_scale,
                     int32_t* topk_ids, float* topk_w, void* stream)
{
    if (B < 0 || B >= moed::kMaxTokens || E < 1 || E > moed::kRouteMaxE || n_group < 1 || n_group > moed::kRouteMaxGroups ||
        E % n_group != 0 || topk_group < 1 || topk_group > n_group || k < 1 || k > moed::kRouteMaxK ||
        k > topk_group * (E / n_group) || n_shared < 0)
        return MOED_ERR_SHAPE;
    if ((long long)B * ((long long)k + n_shared) >= (1LL << 31) || (long long)B * E >= (1LL << 31) ||
        (long long)E + n_shared >= (1LL << 31))
        return MOED_ERR_SHAPE;
    if (!dtype_ok(logits_dtype) || (score != MOED_SCORE_SOFTMAX && score != MOED_SCORE_SIGMOID) ||
        (group_score != MOED_GROUP_MAX && group_score != MOED_GROUP_TOP2))
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    if (!logits || !topk_ids || !topk_w)
        return MOED_ERR_NULL;
    if (!aligned(logits, logits_dtype == MOED_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return MOED_ERR_ALIGN;
    const unsigned long long rows = (unsigned long long)B, slots = rows * ((unsigned long long)k + (unsigned)n_shared);
    const Range ids = bytes(topk_ids, slots * 4), w = bytes(topk_w, slots * 4);
    const Range in[] = {range(logits, logits_dtype, rows * (unsigned)E), bytes(bias, (unsigned long long)E * 4)};
    for (const Range& i : in)                                 // other tokens read them
        if (overlap(ids, i) || overlap(w, i))
            return MOED_ERR_SHAPE;
    if (overlap(ids, w))
        return MOED_ERR_SHAPE;
    moed::RouteArgs p;
    p.logits = logits; p.bias = bias; p.ids = topk_ids; p.w = topk_w;
    p.B = B; p.E = E; p.k = k; p.n_shared = n_shared;
    p.n_group = n_group; p.topk_group = topk_group;
    p.routed_scale = routed_scale;
    p.logits_bf16 = logits_dtype == MOED_BF16;
    p.sigmoid = score == MOED_SCORE_SIGMOID;
    p.top2 = group_score == MOED_GROUP_TOP2;
    p.renormalize = renormalize != 0;
    return moed::abi_status(moed::launch_route_scored(p, static_cast<hipStream_t>(stream)));
}

int moe_post_norm(const void* y, int y_dtype, int R, const int32_t* position, const float* topk_w, int k,
                  const void* post_gain, int post_gain_dtype, float post_eps, const void* gate, int gate_dtype,
                  int gate_shape, int gate_act, float scale, const void* residual, int residual_dtype,
                  float residual_scale, void* residual_out, const void* gain, int gain_dtype, float eps, void* out,
                  int out_dtype, uint8_t* out_q, uint8_t* out_s, int B, int H, void* stream)
{
    if (B < 0 || B >= moed::kMaxTokens || H < 1 || H > moed::kNormMaxH || !(eps >= 0.0f) || !(post_eps >= 0.0f))
        return MOED_ERR_SHAPE;
    if (out_q && H % 32 != 0)
        return MOED_ERR_SHAPE;
    if (position && (k < 1 || k > moed::kRouteMaxK || R < 0 || R >= kMaxRows))
        return MOED_ERR_SHAPE;
    if (!dtype_ok(y_dtype) || !dtype_ok(residual_dtype) || (post_gain && !dtype_ok(post_gain_dtype)) ||
        (gain && !dtype_ok(gain_dtype)) || (out && !dtype_ok(out_dtype)) || gate_shape < MOED_GATE_NONE ||
        gate_shape > MOED_GATE_FULL || (gate && !dtype_ok(gate_dtype)) ||
        (gate_act != MOED_ACT_NONE && gate_act != MOED_ACT_SIGMOID && gate_act != MOED_ACT_TANH))
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    if ((!y && !(position && R == 0)) || !residual || (position == nullptr) != (topk_w == nullptr) ||
        (gate_shape != MOED_GATE_NONE) != (gate != nullptr) || (out_q == nullptr) != (out_s == nullptr) ||
        (!residual_out && !out && !out_q) || (gain != nullptr) != (out != nullptr || out_q != nullptr))
        return MOED_ERR_NULL;
    if (!aligned16(y) || !aligned16(post_gain) || !aligned16(gate) || !aligned16(residual) || !aligned16(residual_out) ||
        !aligned16(gain) || !aligned16(out) || !aligned16(out_q) || !aligned(position, 4) || !aligned(topk_w, 4))
        return MOED_ERR_ALIGN;
    const unsigned long long rows = (unsigned long long)B, n = rows * (unsigned)H, h = (unsigned)H;
    const unsigned long long slots = position ? rows * (unsigned)k : 0;
    const unsigned long long gates = gate_shape == MOED_GATE_TOKEN ? rows : gate_shape == MOED_GATE_CHANNEL ? h : n;
    const Range outs[] = {range(residual_out, residual_dtype, n), range(out, out_dtype, n), bytes(out_q, n), bytes(out_s, n / 32)};
    const Range in[] = {range(y, y_dtype, position ? (unsigned)R * h : n), range(residual, residual_dtype, n),
                        range(gate, gate_dtype, gates), range(post_gain, post_gain_dtype, h), range(gain, gain_dtype, h),
                        bytes(position, slots * 4), bytes(topk_w, slots * 4)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j]))
                return MOED_ERR_SHAPE;
        for (int j = 0; j < 7; ++j) {
            // with a position other tokens read the rows of y
            const bool may = i < 2 && (j == 1 || (j == 0 && !position)) && in_place(outs[i], in[j]);
            if (overlap(outs[i], in[j]) && !may)
                return MOED_ERR_SHAPE;
        }
    }
    moed::PostNormArgs p;
    p.y = y; p.position = position; p.topk_w = topk_w; p.post_gain = post_gain; p.gate = gate; p.residual = residual;
    p.residual_out = residual_out; p.gain = gain; p.out = out; p.q = out_q; p.q_s = out_s;
    p.B = B; p.H = H; p.R = R; p.k = k;
    p.gate_shape = gate_shape; p.gate_act = gate_act;
    p.post_eps = post_eps; p.eps = eps; p.scale = scale; p.residual_scale = residual_scale;
    p.post_gain_bf16 = post_gain_dtype == MOED_BF16;
    p.gate_bf16 = gate_dtype == MOED_BF16;
    p.gain_bf16 = gain_dtype == MOED_BF16;
    p.out_bf16 = out_dtype == MOED_BF16;
    return moed::abi_status(moed::launch_post_norm(p, y_dtype == MOED_BF16, residual_dtype == MOED_BF16,
                                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"
