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

namespace moed {

namespace {

__device__ __forceinline__ float bf16_val(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// V consecutive values of a bf16 or float32 array as float32.
template <bool BF16, bool NT, int V>
__device__ __forceinline__ void load_vals(const void* p, size_t at, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = BF16 ? bf16_val(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
    } else if constexpr (BF16) {
        const u32x4 u = ld<NT>(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    } else {
        const f32x4 a = ld<NT>(reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at));
        const f32x4 b = ld<NT>(reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at + 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}

template <bool BF16, int V>
__device__ __forceinline__ void store_vals(void* p, size_t at, const float (&v)[V])
{
    if constexpr (V == 1) {
        if constexpr (BF16)
            static_cast<uint16_t*>(p)[at] = f32_to_bf16_rne(v[0]);
        else
            static_cast<float*>(p)[at] = v[0];
    } else if constexpr (BF16) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at));
    } else {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(static_cast<float*>(p) + at));
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(static_cast<float*>(p) + at + 4));
    }
}

// Squares of a row whose sum is below 2^-80 (all |s| < 2^-40) may underflow, and its reciprocal root may pass
// float32's range. With an eps as small (TINY) the row is then taken times 2^100, and eps times 2^200, which changes
// nothing else: values from the smallest subnormal number to 2^60, their squares from 2^-98 to 2^120. Above, what is
// lost to underflow is at most 2^15 squares below 2^-126 each: 2^-31 of the sum, or of eps. A kernel of its own, because
// the test costs the others: a token of 2048 2.19 instead of 2.10 us, 8192 tokens of 2049 112.7 instead of 110.1.
constexpr float kSmall = 0x1p-80f, kLift = 0x1p100f;

// Sum over the threads of a row (one wavefront, or all of the workgroup), in every one of them.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part)
{
    v = wave_sum(v);
    if constexpr (W > 1) {
        if (threadIdx.x % kWave == 0)
            part[threadIdx.x / kWave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += part[w];
    }
    return v;
}

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
