// Residual addition and root-mean-square norm in front of the router and the
// experts, with the result in bfloat16 or float32 and, beside it, in MXFP8.
//
//   s = x + residual (float32);  residual_out = s, rounded to the residual's type
//   y = s * rsqrt(mean(s^2) + eps) * gain;  out = y rounded once
//   MXFP8 of y: blocks of 32 values share 2^(c-127), c = max(exponent field of
//   the block's largest |y| - 8, 0) (the OCP rule floor(log2 amax) - 8; an
//   all-zero block gives c = 0), codes = E4M3(clamp(y * 2^(127-c), +-448)),
//   round to nearest even. A block that holds an infinity or a NaN gets the
//   NaN scale 255 and NaN codes.
//
// The norm is taken of the float32 sum, not of its rounded copy, so the only
// roundings are the ones on store. Sums are float32.
//
// A row is read once and stays in registers between the two passes of the
// formula (V values per load, NV loads per thread, TPR threads per row), so the
// kernel moves each input and output byte once. It is bound by memory: 8192
// tokens of 4096 values, residual and MXFP8 included, take 49-54 us from box to
// box (303 MB at 5.6-6.1 TB/s; a 2 GiB copy reaches 6.2-6.35). Loads and stores
// are streaming (cached: 58 us). A single token is bound by one load and one
// reduction (2 us in a graph). Rows that are no multiple of 8 go by single
// values: 8192 tokens of 2049 bf16 110 us, of 1111 25 us (1.2 and 2.9 TB/s).
// With 8 values per thread an MX block is four neighbouring lanes, whose
// largest value is found with two DPP steps.
#include "mx_encode.h"
#include "prompt.h"
#include "row_values.h"

namespace moed {

namespace {

// RES: 0 no residual, 1 bfloat16, 2 float32. TINY: eps < kSmall.
template <int V, int NV, int TPR, bool XBF16, int RES, bool TINY>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
moe_norm_kernel(NormArgs p)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;          // rows per workgroup
    constexpr int kWaves = TPR / kWave;
    const int t = threadIdx.x % TPR;
    const long long b = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    if (b >= p.B)
        return;                                               // whole wavefronts; no barrier follows for kRows > 1
    const size_t row = (size_t)b * (size_t)p.H;
    float s[NV][V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = (t + i * TPR) * V;
        if (h < p.H) {
            load_vals<XBF16, true>(p.x, row + h, s[i]);
            if constexpr (RES != 0) {
                float r[V];
                load_vals<RES == 1, true>(p.residual, row + h, r);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s[i][v] += r[v];
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[i][v] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
            ss = __builtin_fmaf(s[i][v], s[i][v], ss);
    __shared__ float part[kWaves];
    ss = row_sum<kWaves>(ss, part);
    float eps = p.eps, mul = 1.0f;
    if constexpr (TINY) {
        if (ss < kSmall) {                                    // the same for all threads of a row
            mul = kLift;
            eps = eps * kLift * kLift;
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    ss = __builtin_fmaf(s[i][v] * kLift, s[i][v] * kLift, ss);
            if constexpr (kWaves > 1)
                __syncthreads();                              // everybody has the first sum
            ss = row_sum<kWaves>(ss, part);
        }
    }
    const float scale = rsqrtf(ss / (float)p.H + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = (t + i * TPR) * V;
        if (h >= p.H)
            continue;
        if constexpr (RES != 0)
            if (p.residual_out)
                store_vals<RES == 1>(p.residual_out, row + h, s[i]);
        float g[V];
        if (p.gain_bf16)
            load_vals<true, false>(p.gain, (size_t)h, g);
        else
            load_vals<false, false>(p.gain, (size_t)h, g);
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            y[v] = (TINY ? s[i][v] * mul : s[i][v]) * scale * g[v];
        if (p.out) {
            if (p.out_bf16)
                store_vals<true>(p.out, row + h, y);
            else
                store_vals<false>(p.out, row + h, y);
        }
        if constexpr (V == 8) {
            if (p.q) {                                        // H is a multiple of 32: four whole lanes per block
                uint32_t m = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
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

template <int V, int NV, int TPR, bool TINY>
hipError_t launch_kind(const NormArgs& p, bool x_bf16, int res, hipStream_t s)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((p.B + kRows - 1) / kRows)), block(TPR < 256 ? 256 : TPR);
#define MOED_NORM(X, R) hipLaunchKernelGGL((moe_norm_kernel<V, NV, TPR, X, R, TINY>), grid, block, 0, s, p)
    if (x_bf16) {
        if (res == 0) MOED_NORM(true, 0);
        else if (res == 1) MOED_NORM(true, 1);
        else MOED_NORM(true, 2);
    } else {
        if (res == 0) MOED_NORM(false, 0);
        else if (res == 1) MOED_NORM(false, 1);
        else MOED_NORM(false, 2);
    }
#undef MOED_NORM
    return hipGetLastError();
}

template <int V, int NV, int TPR>
hipError_t launch_shape(const NormArgs& p, bool x_bf16, int res, hipStream_t s)
{
    return p.eps < kSmall ? launch_kind<V, NV, TPR, true>(p, x_bf16, res, s) : launch_kind<V, NV, TPR, false>(p, x_bf16, res, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& p, bool x_bf16, int res, hipStream_t s)
{
    const int H = p.H;
    // rows of a multiple of 8 values are whole 16-byte pieces; others go by single values
    if (H % 8 == 0) {
        if (H <= 2048 && p.B >= 2048)
            return launch_shape<8, 4, 64>(p, x_bf16, res, s);
        if (H <= 2048)
            return launch_shape<8, 1, 256>(p, x_bf16, res, s);
        if (H <= 4096)
            return launch_shape<8, 2, 256>(p, x_bf16, res, s);
        if (H <= 8192)
            return launch_shape<8, 4, 256>(p, x_bf16, res, s);
        return launch_shape<8, 4, 1024>(p, x_bf16, res, s);
    }
    if (H <= 2048)
        return launch_shape<1, 8, 256>(p, x_bf16, res, s);
    return launch_shape<1, 32, 1024>(p, x_bf16, res, s);
}

}  // namespace moed
