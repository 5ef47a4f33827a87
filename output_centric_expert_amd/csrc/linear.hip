// Dense product with bias, activation and residual: out[b][n] = act(x[b] . w[n] + bias[n]) + residual[b][n].
//
// A wavefront owns NW weight rows and RB rows of x. Its lanes take pieces of 8 neighbouring k, so that a load of a row
// is contiguous over the wavefront; products are summed in float32 per lane and then over the lanes. KS wavefronts of
// a workgroup share a row's k where there are too few rows to fill the chip.
#include "linear_common.h"

namespace moed {

namespace {

constexpr int kDotWaves = 4;

}  // namespace

template <bool XBF16, bool WBF16, int RB, int NW, int KS>
__global__ void __launch_bounds__(kDotWaves * kWave)
moe_linear_dot_kernel(LinearArgs p, int n_blocks)
{
    constexpr int kParts = kDotWaves / KS;        // wavefronts with weight rows of their own
    __shared__ float part[kDotWaves][RB * NW];
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave, ks = w % KS;
    const size_t b0 = (size_t)(blockIdx.x / (unsigned)n_blocks) * RB;
    const int block_n = (int)(blockIdx.x % (unsigned)n_blocks) * (NW * kParts);
    const int n0 = block_n + w / KS * NW;
    float acc[RB][NW];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NW; ++n)
            acc[r][n] = 0.0f;
    // rows behind the last repeat it
    size_t wrow[NW], xrow[RB];
#pragma unroll
    for (int n = 0; n < NW; ++n)
        wrow[n] = (size_t)(n0 + n < p.N ? n0 + n : p.N - 1) * (size_t)p.K;
#pragma unroll
    for (int r = 0; r < RB; ++r)
        xrow[r] = (b0 + r < (size_t)p.B ? b0 + r : (size_t)p.B - 1) * (size_t)p.K;
    for (int k = (ks * kWave + lane) * 8; k < p.K; k += KS * kWave * 8) {
        float wv[NW][8];
#pragma unroll
        for (int n = 0; n < NW; ++n)
            load_any<WBF16, false>(p.w, wrow[n] + k, p.K - k, wv[n]);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            float xv[8];
            load_any<XBF16, false>(p.x, xrow[r] + k, p.K - k, xv);
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[r][n] = __builtin_fmaf(xv[i], wv[n][i], acc[r][n]);
        }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            const float v = wave_sum(acc[r][n]);
            if (lane == 0)
                part[w][r * NW + n] = v;
        }
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= kParts * RB * NW)
        return;
    const int at = i % (RB * NW), from = i / (RB * NW);
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < KS; ++q)
        v += part[from * KS + q][at];
    const size_t b = b0 + at / NW;
    const int n = block_n + from * NW + at % NW;
    if (b < (size_t)p.B && n < p.N)
        linear_store(p, v, b, n);
}

size_t linear_workspace(int, int, int, bool, bool) { return 0; }

namespace {

template <bool X, bool W>
hipError_t launch_dot(const LinearArgs& p, hipStream_t s)
{
    constexpr int RB = 4, NW = 1, KS = 4;
    const int nb = (p.N + NW * (kDotWaves / KS) - 1) / (NW * (kDotWaves / KS));
    const unsigned grid = (unsigned)((long long)nb * ((p.B + RB - 1) / RB));
    hipLaunchKernelGGL((moe_linear_dot_kernel<X, W, RB, NW, KS>), dim3(grid), dim3(kDotWaves * kWave), 0, s, p, nb);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& p, bool x_bf16, bool w_bf16, void* workspace, hipStream_t s)
{
    (void)workspace;
    if (x_bf16)
        return w_bf16 ? launch_dot<true, true>(p, s) : launch_dot<true, false>(p, s);
    return w_bf16 ? launch_dot<false, true>(p, s) : launch_dot<false, false>(p, s);
}

}  // namespace moed
