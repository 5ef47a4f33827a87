// The end of a block and the norm in front of the next one:
//   t = y * rsqrt(mean(y^2) + post_eps) * post_gain        (y without post_gain)
//   s = residual_scale * residual + scale * act(gate) * t;  residual_out = s, rounded
//   out = s * rsqrt(mean(s^2) + eps) * gain, rounded once, and in MXFP8 by the rule of norm.hip
// y is given, or is the weighted sum of a token's expert rows (combine.hip), which then is never stored: each of its
// k rows is read, the sum goes on in registers. Everything between loads and stores is float32.
//
// A row stays in the registers of its threads (8 values a piece, NV pieces a thread, TPR threads a row) from the
// loads to the last store; two sums over the row stand between them. Residual and gate are asked for with y, in front
// of the first sum, so that a row waits for memory once. Memory bound.
// Rows whose length is no multiple of 8 begin at any element; their pieces are loaded as they lie, and the last one
// value by value.
#include "activation.h"
#include "mx_encode.h"
#include "row_values.h"

namespace moed {

namespace {

constexpr int kRowsAhead = 4;                     // expert rows asked for before the first is added

// Piece of 8 values, of which n exist (WHOLE: 8).
template <bool BF16, bool NT, bool WHOLE>
__device__ __forceinline__ void load_piece(const void* p, size_t at, int n, float (&v)[8])
{
    if constexpr (WHOLE)
        load_vals<BF16, NT>(p, at, v);
    else
        load_any<BF16, NT>(p, at, n, v);
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store_piece(void* p, size_t at, int n, const float (&v)[8])
{
    if constexpr (WHOLE)
        store_vals<BF16>(p, at, v);
    else
        store_any<BF16>(p, at, n, v);
}

template <bool WHOLE>
__device__ __forceinline__ void load_piece(bool bf16, const void* p, size_t at, int n, float (&v)[8])
{
    if (bf16)
        load_piece<true, false, WHOLE>(p, at, n, v);
    else
        load_piece<false, false, WHOLE>(p, at, n, v);
}

__device__ __forceinline__ float gate_value(float g, int act)
{
    return act == kActSigmoid ? sigmoid(g) : act == kActTanh ? tanh_of(g) : g;
}

// 1 / sqrt(mean of squares + eps) of a row as mul * scale: mul is 1 but for rows whose squares would underflow
// (kSmall), which are taken times kLift.
struct Root {
    float mul, scale;
};

template <int NV, int WAVES>
__device__ __forceinline__ Root row_root(const float (&s)[NV][8], int H, float eps, float* part)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < 8; ++v)
            ss = __builtin_fmaf(s[i][v], s[i][v], ss);
    ss = row_sum<WAVES>(ss, part);
    float mul = 1.0f;
    if (eps < kSmall && ss < kSmall) {            // the same for all threads of a row
        mul = kLift;
        eps = eps * kLift * kLift;
        ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < 8; ++v)
                ss = __builtin_fmaf(s[i][v] * kLift, s[i][v] * kLift, ss);
        if constexpr (WAVES > 1)
            __syncthreads();                      // everybody has the first sum
        ss = row_sum<WAVES>(ss, part);
    }
    return {mul, rsqrtf(ss / (float)H + eps)};
}

}  // namespace

template <int NV, int TPR, bool YBF16, bool RBF16, bool ROWS, bool WHOLE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
moe_post_norm_kernel(PostNormArgs p)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;          // rows per workgroup
    constexpr int kWaves = TPR / kWave;
    __shared__ float part[2][kWaves];
    const int t = threadIdx.x % TPR;
    const long long b = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    if (b >= p.B)
        return;                                               // whole wavefronts; no barrier follows for kRows > 1
    const size_t row = (size_t)b * (size_t)p.H;
    float s[NV][8], r[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = (t + i * TPR) * 8;
#pragma unroll
        for (int v = 0; v < 8; ++v)
            s[i][v] = r[i][v] = 0.0f;
        if (h < p.H) {
            load_piece<RBF16, true, WHOLE>(p.residual, row + h, p.H - h, r[i]);
            if constexpr (!ROWS)
                load_piece<YBF16, true, WHOLE>(p.y, row + h, p.H - h, s[i]);
        }
    }
    if constexpr (ROWS) {
        const int32_t* pos = p.position + (size_t)b * p.k;
        const float* w = p.topk_w + (size_t)b * p.k;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int h = (t + i * TPR) * 8;
            if (h >= p.H)
                continue;
            for (int j0 = 0; j0 < p.k; j0 += kRowsAhead) {
                float piece[kRowsAhead][8];
#pragma unroll
                for (int j = 0; j < kRowsAhead; ++j)
                    if (j0 + j < p.k) {                       // uniform over the row
                        const int at = pos[j0 + j];
                        const bool ok = (unsigned)at < (unsigned)p.R;
                        bad |= !ok;
                        if (ok)
                            load_piece<YBF16, true, WHOLE>(p.y, (size_t)at * (size_t)p.H + h, p.H - h, piece[j]);
                    }
#pragma unroll
                for (int j = 0; j < kRowsAhead; ++j)
                    if (j0 + j < p.k && (unsigned)pos[j0 + j] < (unsigned)p.R)
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            s[i][v] = __builtin_fmaf(w[j0 + j], piece[j][v], s[i][v]);
            }
            if (bad)
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s[i][v] = __builtin_nanf("");
        }
    }
    Root post = {1.0f, 1.0f};
    if (p.post_gain)
        post = row_root<NV, kWaves>(s, p.H, p.post_eps, part[0]);
    float token_gate = p.scale;
    if (p.gate_shape == kGateToken) {
        const float g = p.gate_bf16 ? bf16_val(static_cast<const uint16_t*>(p.gate)[b]) : static_cast<const float*>(p.gate)[b];
        token_gate *= gate_value(g, p.gate_act);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = (t + i * TPR) * 8, n = p.H - h;
        if (n <= 0)
            continue;
        if (p.post_gain) {
            float g[8];
            load_piece<WHOLE>(p.post_gain_bf16, p.post_gain, (size_t)h, n, g);
#pragma unroll
            for (int v = 0; v < 8; ++v)
                s[i][v] = s[i][v] * post.mul * post.scale * g[v];
        }
        float g[8];
#pragma unroll
        for (int v = 0; v < 8; ++v)
            g[v] = token_gate;
        if (p.gate_shape >= kGateChannel) {
            load_piece<WHOLE>(p.gate_bf16, p.gate, p.gate_shape == kGateFull ? row + h : (size_t)h, n, g);
#pragma unroll
            for (int v = 0; v < 8; ++v)
                g[v] = p.scale * gate_value(g[v], p.gate_act);
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
            s[i][v] = WHOLE || v < n ? __builtin_fmaf(p.residual_scale, r[i][v], g[v] * s[i][v]) : 0.0f;
        if (p.residual_out)
            store_piece<RBF16, WHOLE>(p.residual_out, row + h, n, s[i]);
    }
    if (!p.gain)
        return;
    const Root pre = row_root<NV, kWaves>(s, p.H, p.eps, part[1]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = (t + i * TPR) * 8, n = p.H - h;
        if (n <= 0)
            continue;
        float g[8];
        load_piece<WHOLE>(p.gain_bf16, p.gain, (size_t)h, n, g);
        float y[8];
#pragma unroll
        for (int v = 0; v < 8; ++v)
            y[v] = s[i][v] * pre.mul * pre.scale * g[v];
        if (p.out) {
            if (p.out_bf16)
                store_piece<true, WHOLE>(p.out, row + h, n, y);
            else
                store_piece<false, WHOLE>(p.out, row + h, n, y);
        }
        if constexpr (WHOLE) {
            if (p.q) {                                        // H is a multiple of 32: four whole lanes per block
                uint32_t m = 0;
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const uint32_t a = __float_as_uint(y[v]) & 0x7FFFFFFFu;
                    m = a > m ? a : m;
                }
                m = quad_max(m);
                u32x2 codes;
                const uint32_t c = mx8_scale_code(m);
                codes.x = mx8_codes4(y[0], y[1], y[2], y[3], c);
                codes.y = mx8_codes4(y[4], y[5], y[6], y[7], c);
                __builtin_nontemporal_store(codes, reinterpret_cast<u32x2*>(p.q + row + h));
                if ((t & 3) == 0)
                    p.q_s[(row + h) / 32] = (uint8_t)c;
            }
        }
    }
}

namespace {

template <int NV, int TPR, bool WHOLE>
hipError_t launch_shape(const PostNormArgs& p, bool y_bf16, bool r_bf16, hipStream_t s)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((p.B + kRows - 1) / kRows)), block(TPR < 256 ? 256 : TPR);
#define MOED_POST(Y, R) \
    do { \
        if (p.position) hipLaunchKernelGGL((moe_post_norm_kernel<NV, TPR, Y, R, true, WHOLE>), grid, block, 0, s, p); \
        else hipLaunchKernelGGL((moe_post_norm_kernel<NV, TPR, Y, R, false, WHOLE>), grid, block, 0, s, p); \
    } while (0)
    if (y_bf16) {
        if (r_bf16) MOED_POST(true, true);
        else MOED_POST(true, false);
    } else {
        if (r_bf16) MOED_POST(false, true);
        else MOED_POST(false, false);
    }
#undef MOED_POST
    return hipGetLastError();
}

template <bool WHOLE>
hipError_t launch_rows(const PostNormArgs& p, bool y_bf16, bool r_bf16, hipStream_t s)
{
    if (p.H <= 2048)
        return launch_shape<1, 256, WHOLE>(p, y_bf16, r_bf16, s);
    if (p.H <= 4096)
        return launch_shape<2, 256, WHOLE>(p, y_bf16, r_bf16, s);
    if (p.H <= 8192)
        return launch_shape<4, 256, WHOLE>(p, y_bf16, r_bf16, s);
    return launch_shape<4, 1024, WHOLE>(p, y_bf16, r_bf16, s);
}

}  // namespace

hipError_t launch_post_norm(const PostNormArgs& p, bool y_bf16, bool residual_bf16, hipStream_t s)
{
    return p.H % 8 == 0 ? launch_rows<true>(p, y_bf16, residual_bf16, s) : launch_rows<false>(p, y_bf16, residual_bf16, s);
}

}  // namespace moed
