// C ABI of the prompt-side calls (moe_norm, moe_group, moe_grouped_gate_up,
// moe_grouped_matmul, moe_combine, moe_prefill): argument checks and launches.
// All arithmetic runs in the kernels; no call keeps state between calls.
#include "moedecode.h"
#include "prompt.h"

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline bool dtype_ok(int d) { return d == MOED_BF16 || d == MOED_F32; }
inline bool rows_ok(int r) { return r == MOED_ROWS_BF16 || r == MOED_ROWS_MXFP8 || r == MOED_ROWS_MXFP8_FAST; }
inline bool wformat_ok(int f) { return f == MOED_MXFP8 || f == MOED_MXFP4; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int kMaxRows = 1 << 28;            // sorted rows of a prompt-side call
constexpr int kMaxRowLength = 1 << 20;

bool group_ok(int B, int k, int E)
{
    return B >= 0 && B < moed::kMaxTokens && k >= 1 && k <= moed::kRouteMaxK && E >= 1 && E <= moed::kGroupMaxE &&
           (long long)B * k < kMaxRows;
}

// The kernels number their tiles (of 16 rows and 32 outputs or more) with 31 bits.
bool too_many_tiles(long long R, int E, int N)
{
    return (R / 16 + (R < E ? R : E)) * ((N + 31) / 32) >= (1LL << 31);
}

int check_product(int a_rows, int wfmt, int n_a, int k, bool ordered, int R, int E, int K, int N)
{
    if (R < 0 || R >= kMaxRows || n_a < 0 || n_a >= kMaxRows || E < 1 || E > moed::kGroupMaxE || k < 1 ||
        (!ordered && n_a < R) || (R > 0 && n_a == 0))
        return MOED_ERR_SHAPE;
    if (K < 32 || N < 32 || K % 32 != 0 || N % 32 != 0 || K >= kMaxRowLength || N >= kMaxRowLength)
        return MOED_ERR_SHAPE;
    if (too_many_tiles(R, E, N))
        return MOED_ERR_SHAPE;
    // the kernels address one expert's matrix, and gathered rows, with 32-bit offsets
    if ((long long)K * N >= (1LL << 32) || (ordered && (long long)n_a * K * (a_rows == MOED_ROWS_BF16 ? 2 : 1) >= (1LL << 32)))
        return MOED_ERR_SHAPE;
    if (!rows_ok(a_rows) || !wformat_ok(wfmt))
        return MOED_ERR_DTYPE;
    return MOED_OK;
}

// Workspace of a product call, where its scales need one.
int check_scales(size_t need, const void* workspace, size_t bytes)
{
    if (need == 0)
        return MOED_OK;
    if (!workspace)
        return MOED_ERR_NULL;
    if (bytes < need)
        return MOED_ERR_WORKSPACE;
    return aligned16(workspace) ? MOED_OK : MOED_ERR_ALIGN;
}

moed::ProductArgs product_args(const void* a, const uint8_t* a_s, bool fast, int n_a, const int32_t* order, int k,
                               const int32_t* offsets, const uint8_t* w_q, const uint8_t* w_s, const uint8_t* u_q,
                               const uint8_t* u_s, int wfmt, void* out, uint8_t* out_s, int out_rows, int R, int E,
                               int K, int N)
{
    static_assert(moed::kOutBF16 == MOED_ROWS_BF16 && moed::kOutF32 == MOED_ROWS_F32 && moed::kOutMX8 == MOED_ROWS_MXFP8,
                  "output kinds are the ABI's");
    moed::ProductArgs p;
    p.a = a; p.a_s = a_s; p.order = order; p.offsets = offsets;
    p.w_q = w_q; p.w_s = w_s; p.u_q = u_q; p.u_s = u_s;
    p.out = out; p.out_s = out_s;
    p.n_a = n_a; p.k = k; p.R = R; p.E = E; p.K = K; p.N = N;
    p.inv_k = (uint32_t)(k == 1 ? 0xFFFFFFFFu : (1ull << 32) / (unsigned)k);
    p.fp4 = wfmt == MOED_MXFP4;
    p.fast = fast;
    p.out_kind = out_rows;
    return p;
}

moed::CombineArgs combine_args(const void* y, int R, const int32_t* position, const float* w, void* out, int out_dtype,
                               int B, int k, int H)
{
    moed::CombineArgs p;
    p.y = y; p.position = position; p.w = w; p.out = out;
    p.B = B; p.k = k; p.H = H; p.R = R;
    p.out_bf16 = out_dtype == MOED_BF16;
    return p;
}

// Workspace of moe_prefill: byte offsets of its parts, each 256-byte aligned.
struct PrefillLayout {
    size_t counts, order, position, offsets, scales, a, a_s, y, bytes;
};

int prefill_layout(int B, int E, int k, int H, int I, int x_rows, int out_dtype, PrefillLayout* l)
{
    if (!group_ok(B, k, E) || k > E)
        return MOED_ERR_SHAPE;
    if (H < 32 || I < 32 || H % 32 != 0 || I % 32 != 0 || H >= kMaxRowLength || I >= kMaxRowLength)
        return MOED_ERR_SHAPE;
    if (!rows_ok(x_rows) || !dtype_ok(out_dtype))
        return MOED_ERR_DTYPE;
    const bool mx = x_rows != MOED_ROWS_BF16;
    if (too_many_tiles((long long)B * k, E, H > I ? H : I) || (long long)H * I >= (1LL << 32) ||
        (long long)B * H * (mx ? 1 : 2) >= (1LL << 32))
        return MOED_ERR_SHAPE;
    const size_t R = (size_t)B * (size_t)k;
    size_t at = 0;
    auto part = [&at](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    l->counts = part(moed::group_workspace((int)R, E));
    l->order = part(R * 4);
    l->position = part(R * 4);
    l->offsets = part(((size_t)E + 1) * 4);
    const size_t up = moed::product_scales_bytes(E, H, I, B, mx, true);
    const size_t down = moed::product_scales_bytes(E, I, H, (int)R, mx, false);
    l->scales = part(up > down ? up : down);                  // one product at a time
    l->a = part(R * (size_t)I * (mx ? 1 : 2));
    l->a_s = part(mx ? R * (size_t)I / 32 : 0);
    l->y = part(R * (size_t)H * (out_dtype == MOED_F32 ? 4 : 2));
    l->bytes = at;
    return MOED_OK;
}

}  // namespace

extern "C" {

int moe_norm(const void* x, int x_dtype, const void* residual, int residual_dtype, const void* gain, int gain_dtype,
             float eps, void* residual_out, void* out, int out_dtype, uint8_t* out_q, uint8_t* out_s, int B, int H,
             void* stream)
{
    if (B < 0 || B >= moed::kMaxTokens || H < 1 || H > moed::kNormMaxH || !(eps >= 0.0f))
        return MOED_ERR_SHAPE;
    if (out_q && H % 32 != 0)
        return MOED_ERR_SHAPE;
    if (!dtype_ok(x_dtype) || !dtype_ok(gain_dtype) || (residual && !dtype_ok(residual_dtype)) ||
        (out && !dtype_ok(out_dtype)))
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    if (!x || !gain || (!out && !out_q) || (out_q == nullptr) != (out_s == nullptr) || (residual_out && !residual))
        return MOED_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(gain) || !aligned16(residual_out) || !aligned16(out) ||
        !aligned16(out_q))
        return MOED_ERR_ALIGN;
    if (out && out == residual_out)                           // the sum would be lost
        return MOED_ERR_SHAPE;
    moed::NormArgs p;
    p.x = x; p.residual = residual; p.gain = gain; p.residual_out = residual_out; p.out = out;
    p.q = out_q; p.q_s = out_s;
    p.B = B; p.H = H; p.eps = eps;
    p.gain_bf16 = gain_dtype == MOED_BF16;
    p.out_bf16 = out_dtype == MOED_BF16;
    return moed::abi_status(moed::launch_norm(p, x_dtype == MOED_BF16, !residual ? 0 : residual_dtype == MOED_BF16 ? 1 : 2,
                                        static_cast<hipStream_t>(stream)));
}

size_t moe_group_workspace_bytes(int B, int k, int E)
{
    return group_ok(B, k, E) ? moed::group_workspace(B * k, E) : 0;
}

int moe_group(const int32_t* topk_ids, int B, int k, int E, int32_t* order, int32_t* position, int32_t* offsets,
              void* workspace, size_t workspace_bytes, void* stream)
{
    if (!group_ok(B, k, E))
        return MOED_ERR_SHAPE;
    if (!offsets || (B > 0 && (!topk_ids || !order || !position)))
        return MOED_ERR_NULL;
    const size_t need = moed::group_workspace(B * k, E);
    if (need && !workspace)
        return MOED_ERR_NULL;
    if (workspace_bytes < need)
        return MOED_ERR_WORKSPACE;
    if (need && ((uintptr_t)workspace & 3u) != 0)
        return MOED_ERR_ALIGN;
    return moed::abi_status(moed::launch_group(topk_ids, B * k, E, static_cast<int32_t*>(workspace), order, position, offsets,
                                         static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_workspace_bytes(int E, int K, int N, int n_a, int a_rows, int matrices)
{
    // sizes as without an order, whose limits are the wider ones
    if (check_product(a_rows, MOED_MXFP8, n_a, 1, false, 0, E, K, N) || (matrices != 1 && matrices != 2))
        return 0;
    return moed::product_scales_bytes(E, K, N, n_a, a_rows != MOED_ROWS_BF16, matrices == 2);
}

int moe_grouped_gate_up(const void* a, const uint8_t* a_s, int a_rows, int n_a, const int32_t* order, int k,
                        const int32_t* offsets, const uint8_t* wg_q, const uint8_t* wg_s, const uint8_t* wu_q,
                        const uint8_t* wu_s, int weight_format, void* out, uint8_t* out_s, int out_rows, int R, int E,
                        int K, int N, void* workspace, size_t workspace_bytes, void* stream)
{
    if (out_rows != MOED_ROWS_BF16 && out_rows != MOED_ROWS_F32 && out_rows != MOED_ROWS_MXFP8)
        return MOED_ERR_DTYPE;
    if (int st = check_product(a_rows, weight_format, n_a, k, order != nullptr, R, E, K, N))
        return st;
    if (R == 0)
        return MOED_OK;
    if (!a || !offsets || !wg_q || !wg_s || !wu_q || !wu_s || !out || (a_rows != MOED_ROWS_BF16) != (a_s != nullptr) ||
        (out_rows == MOED_ROWS_MXFP8) != (out_s != nullptr))
        return MOED_ERR_NULL;
    if (!aligned16(a) || !aligned16(wg_q) || !aligned16(wu_q) || !aligned16(out) || !aligned4(wg_s) || !aligned4(wu_s) ||
        !aligned4(a_s))
        return MOED_ERR_ALIGN;
    if (int st = check_scales(moed::product_scales_bytes(E, K, N, n_a, a_s != nullptr, true), workspace, workspace_bytes))
        return st;
    return moed::abi_status(moed::launch_product(
        product_args(a, a_s, a_rows == MOED_ROWS_MXFP8_FAST, n_a, order, k, offsets, wg_q, wg_s, wu_q, wu_s, weight_format,
                     out, out_s, out_rows, R, E, K, N),
        workspace, static_cast<hipStream_t>(stream)));
}

int moe_grouped_matmul(const void* a, const uint8_t* a_s, int a_rows, int n_a, const int32_t* order, int k,
                       const int32_t* offsets, const uint8_t* w_q, const uint8_t* w_s, int weight_format, void* out,
                       int out_rows, int R, int E, int K, int N, void* workspace, size_t workspace_bytes, void* stream)
{
    if (out_rows != MOED_ROWS_BF16 && out_rows != MOED_ROWS_F32)
        return MOED_ERR_DTYPE;
    if (int st = check_product(a_rows, weight_format, n_a, k, order != nullptr, R, E, K, N))
        return st;
    if (R == 0)
        return MOED_OK;
    if (!a || !offsets || !w_q || !w_s || !out || (a_rows != MOED_ROWS_BF16) != (a_s != nullptr))
        return MOED_ERR_NULL;
    if (!aligned16(a) || !aligned16(w_q) || !aligned16(out) || !aligned4(w_s) || !aligned4(a_s))
        return MOED_ERR_ALIGN;
    if (int st = check_scales(moed::product_scales_bytes(E, K, N, n_a, a_s != nullptr, false), workspace, workspace_bytes))
        return st;
    return moed::abi_status(moed::launch_product(
        product_args(a, a_s, a_rows == MOED_ROWS_MXFP8_FAST, n_a, order, k, offsets, w_q, w_s, nullptr, nullptr,
                     weight_format, out, nullptr, out_rows, R, E, K, N),
        workspace, static_cast<hipStream_t>(stream)));
}

int moe_combine(const void* y, int y_dtype, int R, const int32_t* position, const float* topk_w, void* out,
                int out_dtype, int B, int k, int H, void* stream)
{
    if (B < 0 || B >= moed::kMaxTokens || k < 1 || k > moed::kRouteMaxK || H < 1 || H >= kMaxRowLength || R < 0 ||
        R >= kMaxRows)
        return MOED_ERR_SHAPE;
    if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype))
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    if ((!y && R > 0) || !position || !topk_w || !out)
        return MOED_ERR_NULL;
    if (!aligned16(y) || !aligned16(out))
        return MOED_ERR_ALIGN;
    return moed::abi_status(moed::launch_combine(combine_args(y, R, position, topk_w, out, out_dtype, B, k, H),
                                           y_dtype == MOED_BF16, static_cast<hipStream_t>(stream)));
}

size_t moe_prefill_workspace_bytes(int B, int E, int k, int H, int I, int x_rows, int out_dtype)
{
    PrefillLayout l;
    return prefill_layout(B, E, k, H, I, x_rows, out_dtype, &l) == MOED_OK && B > 0 ? l.bytes : 0;
}

int moe_prefill(const void* x, const uint8_t* x_s, int x_rows, const int32_t* topk_ids, const float* topk_w,
                const uint8_t* wg_q, const uint8_t* wg_s, const uint8_t* wu_q, const uint8_t* wu_s, const uint8_t* wd_q,
                const uint8_t* wd_s, int weight_format, void* out, int out_dtype, int B, int E, int k, int H, int I,
                void* workspace, size_t workspace_bytes, void* stream)
{
    PrefillLayout l;
    if (int st = prefill_layout(B, E, k, H, I, x_rows, out_dtype, &l))
        return st;
    if (!wformat_ok(weight_format))
        return MOED_ERR_DTYPE;
    if (B == 0)
        return MOED_OK;
    const bool mx = x_rows != MOED_ROWS_BF16, fast = x_rows == MOED_ROWS_MXFP8_FAST;
    if (!x || mx != (x_s != nullptr) || !topk_ids || !topk_w || !wg_q || !wg_s || !wu_q || !wu_s || !wd_q || !wd_s ||
        !out || !workspace)
        return MOED_ERR_NULL;
    if (workspace_bytes < l.bytes)
        return MOED_ERR_WORKSPACE;
    if (!aligned16(x) || !aligned16(wg_q) || !aligned16(wu_q) || !aligned16(wd_q) || !aligned16(out) ||
        !aligned16(workspace) || !aligned4(x_s) || !aligned4(wg_s) || !aligned4(wu_s) || !aligned4(wd_s))
        return MOED_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // where weights are decoded to bfloat16 the block scales are folded into the conversion, as in the large-batch
    // kernels: both steps with bfloat16 rows, the down step with float32 outputs (MXFP8 rows with rounded outputs take
    // any scale)
    moed::CheckArgs c;
    c.ids = topk_ids;
    c.wg_q = wg_q; c.wg_s = wg_s; c.wu_q = wu_q; c.wu_s = wu_s; c.wd_q = wd_q; c.wd_s = wd_s;
    c.B = B; c.E = E; c.k = k; c.H = H; c.I = I; c.wfmt = weight_format;
    if (int st = moed::abi_check(c, !mx, !mx || out_dtype == MOED_F32, s))
        return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int32_t* order = reinterpret_cast<int32_t*>(ws + l.order);
    int32_t* position = reinterpret_cast<int32_t*>(ws + l.position);
    int32_t* offsets = reinterpret_cast<int32_t*>(ws + l.offsets);
    const int R = B * k;
    if (int st = moed::abi_status(moed::launch_group(topk_ids, R, E, reinterpret_cast<int32_t*>(ws + l.counts), order, position,
                                               offsets, s)))
        return st;
    if (int st = moed::abi_status(moed::launch_product(
            product_args(x, x_s, fast, B, order, k, offsets, wg_q, wg_s, wu_q, wu_s, weight_format, ws + l.a,
                         mx ? ws + l.a_s : nullptr, mx ? MOED_ROWS_MXFP8 : MOED_ROWS_BF16, R, E, H, I),
            ws + l.scales, s)))
        return st;
    // Rows in out_dtype: float32 rows under a bfloat16 output would spare each term of the sum one rounding (2^-8 of it at
    // most, as much as the output's own) for twice the bytes between the product and the sum: with bfloat16 rows 901
    // instead of 790 us at 8192 tokens (8 of 128 experts, H = 2048, I = 768, MXFP8).
    if (int st = moed::abi_status(moed::launch_product(
            product_args(ws + l.a, mx ? ws + l.a_s : nullptr, fast, R, nullptr, 1, offsets, wd_q, wd_s, nullptr, nullptr,
                         weight_format, ws + l.y, nullptr, out_dtype, R, E, I, H),
            ws + l.scales, s)))
        return st;
    return moed::abi_status(moed::launch_combine(combine_args(ws + l.y, R, position, topk_w, out, out_dtype, B, k, H),
                                           out_dtype == MOED_BF16, s));
}

}  // extern "C"
