// Dense product with bias, activation and residual: out[b][n] = act(x[b] . w[n] + bias[n]) + residual[b][n].
//
// A wavefront owns NW weight rows and RB rows of x. Its lanes take pieces of 8 neighbouring k, so that a load of a row
// is contiguous over the wavefront; products are summed in float32 per lane and then over the lanes. KS wavefronts of
// a workgroup share a row's k where there are too few rows to fill the chip.
#include "linear_skinny.h"
#include "linear_tiled.h"

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

// The sums of a product whose k was split, added in the order of the splits, and the epilogue.
__global__ void __launch_bounds__(256)
moe_linear_join_kernel(LinearArgs p, const float* partial, int splits)
{
    const size_t count = (size_t)p.B * (size_t)p.N;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    float v = 0.0f;
#pragma unroll 4
    for (int q = 0; q < splits; ++q)
        v += partial[q * count + i];
    const size_t b = i / (unsigned)p.N;
    linear_store(p, v, b, (int)(i - b * (unsigned)p.N));
}

namespace {

constexpr int kDotRows = 1;                       // up to here the rows are multiplied without matrix instructions
constexpr int kSkinnyRows = 64;                   // rows of the smaller side up to which it is a skinny product

TileSize tile_of(bool x_bf16, bool w_bf16, int tile)
{
    return x_bf16 ? (w_bf16 ? linear_tile_bf16(tile) : linear_tile_mixed_w(tile))
                  : (w_bf16 ? linear_tile_mixed_x(tile) : linear_tile_f32(tile));
}

enum class Kind { dot, skinny, tiled };
struct Choice {
    Kind kind;
    int tile, rt;
    bool swapped;
    LinearPlan plan;
    SkinnyPlan skinny;
};

Choice choose(int B, int K, int N, bool x_bf16, bool w_bf16)
{
    Choice c;
    if (B <= kDotRows) {
        c.kind = Kind::dot;
        return c;
    }
    if (B <= kSkinnyRows || N <= kSkinnyRows) {
        c.kind = Kind::skinny;
        c.swapped = N < B;
        const int few = c.swapped ? N : B, many = c.swapped ? B : N;
        c.rt = few <= 16 ? 1 : 2;
        c.skinny.few_blocks = (few + 16 * c.rt - 1) / (16 * c.rt);
        c.skinny.many_blocks = (many + 15) / 16;
        const int steps = (K + (!x_bf16 && !w_bf16 ? 31 : 63)) / (!x_bf16 && !w_bf16 ? 32 : 64);
        const long long tiles = (long long)c.skinny.few_blocks * c.skinny.many_blocks;
        long long splits = 256 / tiles, most = steps / (2 * kSkinnyWaves);
        splits = splits < most ? splits : most;
        c.skinny.splits = (int)(splits < 1 ? 1 : splits > 16 ? 16 : splits);
        return c;
    }
    c.kind = Kind::tiled;
    c.tile = kTileMiddle;
    TileSize t = tile_of(x_bf16, w_bf16, kTileLarge);
    const long long large = ((B + t.rows - 1LL) / t.rows) * ((N + t.outputs - 1LL) / t.outputs);
    if (large >= 256)
        c.tile = kTileLarge;
    t = tile_of(x_bf16, w_bf16, c.tile);
    c.plan.m_blocks = (B + t.rows - 1) / t.rows;
    c.plan.n_blocks = (N + t.outputs - 1) / t.outputs;
    c.plan.group = c.plan.n_blocks < 8 ? c.plan.n_blocks : 8;
    const int steps = (K + t.k - 1) / t.k;
    const long long tiles = (long long)c.plan.m_blocks * c.plan.n_blocks;
    long long splits = tiles >= 256 ? 1 : 512 / tiles;
    splits = splits < steps / 4 ? splits : steps / 4;
    splits = splits < 1 ? 1 : splits > 32 ? 32 : splits;
    c.plan.split_steps = (int)((steps + splits - 1) / splits);
    c.plan.splits = (steps + c.plan.split_steps - 1) / c.plan.split_steps;
    c.plan.partial = nullptr;
    return c;
}

}  // namespace

size_t linear_workspace(int B, int K, int N, bool x_bf16, bool w_bf16)
{
    const Choice c = choose(B, K, N, x_bf16, w_bf16);
    const int splits = c.kind == Kind::tiled ? c.plan.splits : c.kind == Kind::skinny ? c.skinny.splits : 1;
    return splits > 1 ? (size_t)splits * (size_t)B * (size_t)N * 4 : 0;
}

namespace {

template <bool X, bool W, int RB, int NW, int KS>
hipError_t launch_dot_shape(const LinearArgs& p, hipStream_t s)
{
    const int per = NW * (kDotWaves / KS), nb = (p.N + per - 1) / per;
    const unsigned grid = (unsigned)((long long)nb * ((p.B + RB - 1) / RB));
    hipLaunchKernelGGL((moe_linear_dot_kernel<X, W, RB, NW, KS>), dim3(grid), dim3(kDotWaves * kWave), 0, s, p, nb);
    return hipGetLastError();
}

template <bool X, bool W>
hipError_t launch_dot(const LinearArgs& p, hipStream_t s)
{
    return launch_dot_shape<X, W, 1, 1, 4>(p, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& p, bool x_bf16, bool w_bf16, void* workspace, hipStream_t s)
{
    Choice c = choose(p.B, p.K, p.N, x_bf16, w_bf16);
    if (c.kind == Kind::dot) {
        if (x_bf16)
            return w_bf16 ? launch_dot<true, true>(p, s) : launch_dot<true, false>(p, s);
        return w_bf16 ? launch_dot<false, true>(p, s) : launch_dot<false, false>(p, s);
    }
    c.plan.partial = c.skinny.partial = static_cast<float*>(workspace);
    hipError_t e;
    int splits;
    if (c.kind == Kind::skinny) {
        auto launch = x_bf16 ? (w_bf16 ? launch_skinny_bf16 : launch_skinny_mixed_w) : (w_bf16 ? launch_skinny_mixed_x : launch_skinny_f32);
        e = launch(c.swapped, c.rt, p, c.skinny, s);
        splits = c.skinny.splits;
    } else {
        auto launch = x_bf16 ? (w_bf16 ? launch_linear_bf16 : launch_linear_mixed_w) : (w_bf16 ? launch_linear_mixed_x : launch_linear_f32);
        e = launch(c.tile, p, c.plan, s);
        splits = c.plan.splits;
    }
    if (e != hipSuccess || splits == 1)
        return e;
    const size_t count = (size_t)p.B * (size_t)p.N;
    hipLaunchKernelGGL(moe_linear_join_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, s, p,
                       static_cast<const float*>(workspace), splits);
    return hipGetLastError();
}

}  // namespace moed
