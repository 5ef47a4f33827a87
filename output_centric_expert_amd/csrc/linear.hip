// Dense product with bias, activation and residual: out[b][n] = act(x[b] . w[n] + bias[n]) + residual[b][n].
// The choice of a kernel, the kernel of a single row of x, and the sum of a product whose k was split.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

constexpr int kDotWaves = 4;

}  // namespace

// One row of x. A workgroup's four wavefronts share an output's k; their lanes take pieces of 8 neighbouring values, so that
// a load of a row is contiguous over the wavefront. Bound by the weights' way from memory (4096 x 4096 bfloat16 in a graph
// 8.4 us from the Infinity Cache, 4.0 TB/s, 9.8-10.2 from HBM; a row's second piece is asked for behind the first one's
// sum, and the kernel of few rows takes 8.1 where this one takes 8.6) and, with few outputs, by one round trip (2048 -> 128
// float32: 2.6 us, the kernel of few rows 5.1: it has 8 workgroups for it, this one 128).
template <bool XBF16, bool WBF16>
__global__ void __launch_bounds__(kDotWaves * kWave)
moe_linear_dot_kernel(LinearArgs p)
{
    __shared__ float part[kDotWaves];
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave, n = blockIdx.x;
    const size_t row = (size_t)n * (size_t)p.K;
    float sum = 0.0f;
    for (int k = threadIdx.x * 8; k < p.K; k += kDotWaves * kWave * 8) {
        float wv[8], xv[8];
        load_any<WBF16, false>(p.w, row + k, p.K - k, wv);
        load_any<XBF16, false>(p.x, (size_t)k, p.K - k, xv);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fmaf(xv[i], wv[i], sum);
    }
    sum = wave_sum(sum);
    if (lane == 0)
        part[w] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        linear_store(p, (part[0] + part[1]) + (part[2] + part[3]), 0, n);
}

// The sums of a product whose k was split, added in the order of the splits, and the epilogue. V neighbouring outputs of a
// row a thread (fewer at its end).
template <int V>
__global__ void __launch_bounds__(256)
moe_linear_join_kernel(LinearArgs p, const float* partial, int splits, unsigned threads)
{
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= threads)
        return;
    const unsigned pieces = ((unsigned)p.N + V - 1) / V, b = i / pieces;
    const int n = (int)(i - b * pieces) * V, have = p.N - n;
    const size_t at = (size_t)b * (size_t)p.N + (size_t)n, count = (size_t)p.B * (size_t)p.N;
    if constexpr (V == 1) {
        float v = 0.0f;
#pragma unroll 4
        for (int q = 0; q < splits; ++q)
            v += partial[q * count + at];
        linear_store(p, v, b, n);
    } else {
        float v[8] = {}, bias[8] = {}, residual[8] = {};
#pragma unroll 2
        for (int q = 0; q < splits; ++q) {
            float o[8];
            load_any<false, true>(partial, q * count + at, have, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] += o[e];
        }
        if (p.bias)
            load_some(p.bias_bf16, p.bias, (size_t)n, have, bias);
        if (p.residual)
            load_some(p.residual_bf16, p.residual, at, have, residual);
        linear_finish(p, bias, residual, v);
        store_some(p.out_bf16, p.out, at, have, v);
    }
}

namespace {

// Tiles up to which a product of more than 16 rows is a skinny one: beyond, the chip is full of workgroups that load the same
// rows. 256 x 7168 -> 256, w float32, 128 tiles: 12.8 us, with the other kernel 14.3; 64 x 4096 -> 4096 bfloat16, 512
// tiles: 15.4 and 14.7.
constexpr int kSkinnyTiles = 400;
// A wavefront's us a step of the skinny kernel, by the number of float32 operands (two: steps of 32 values, else of 64).
constexpr float kSkinnyStep[3] = {0.26f, 0.50f, 0.40f};
constexpr float kSkinnySplitPays = 4.5f;          // us of steps from which a second launch pays

struct Choice {
    enum Kind { dot, skinny, tiled } kind;
    int tile, rt, splits;
    bool swapped;
    LinearPlan plan;
    SkinnyPlan skinny_plan;
};

// Values of k in a step of the skinny kernel.
int skinny_step(bool x_bf16, bool w_bf16) { return !x_bf16 && !w_bf16 ? 32 : 64; }

bool tile_cost(bool x_bf16, bool w_bf16, int tile, TileCost* t)
{
    return x_bf16 ? (w_bf16 ? linear_cost_bf16(tile, t) : linear_cost_mixed_w(tile, t))
                  : (w_bf16 ? linear_cost_mixed_x(tile, t) : linear_cost_f32(tile, t));
}

// The kernel by the sizes.
Choice choose(int B, int K, int N, bool x_bf16, bool w_bf16)
{
    Choice c;
    c.tile = c.rt = 0;
    c.splits = 1;
    c.swapped = false;
    if (B == 1) {
        c.kind = Choice::dot;
        return c;
    }
    const int step = skinny_step(x_bf16, w_bf16);
    {
        c.swapped = N < B;
        const int few = c.swapped ? N : B, many = c.swapped ? B : N;
        // 16 x 16 outputs a workgroup where each has a CU of its own then: 32 x 1024 -> 1024 float32 5.5 us (32 x 16: 6.8),
        // 64 x 4096 -> 1024 bfloat16 6.1 (7.5). Beyond, 32 x 16, which read the side with many half as often.
        c.rt = few <= 16 || (long long)((few + 15) / 16) * ((many + 15) / 16) <= 256 ? 1 : 2;
        SkinnyPlan& s = c.skinny_plan;
        s.few_blocks = (few + 16 * c.rt - 1) / (16 * c.rt);
        s.many_blocks = (many + 15) / 16;
        const long long tiles = (long long)s.few_blocks * s.many_blocks;
        if (few <= 16 || tiles <= kSkinnyTiles) {
            c.kind = Choice::skinny;
            // k is split where that saves more than a second launch costs, which the host feels more than the GPU: workgroups
            // for the whole chip then, but a step and a half at least for a wavefront. us of the GPU, 16 rows, 256 outputs,
            // bfloat16: K = 4096 4.7 whole and 6.1 split, 7168 8.0 and 6.8, 8192 8.3 and 7.1; 64 rows, float32 w: K = 4096
            // 8.2 and 7.5, 7168 11.4 and 8.9; float32: K = 2048 7.5 and 6.1, 7168 17.2 and 9.9.
            const int steps = (K + step - 1) / step;
            const float whole = (float)steps / kSkinnyWaves * kSkinnyStep[(x_bf16 ? 0 : 1) + (w_bf16 ? 0 : 1)];
            long long splits = 256 / tiles;
            const long long most = (long long)steps * 2 / (3 * kSkinnyWaves);
            splits = splits < most ? splits : most;
            c.splits = s.splits = whole < kSkinnySplitPays || splits < 1 ? 1 : (int)splits;
            return c;
        }
    }
    c.kind = Choice::tiled;
    // Of the tiles and ways to split k the one that should take least: some us to begin and end, a step's time for each
    // round of the chip's workgroups, and for split k a second launch and its bytes.
    const float outputs = (float)B * (float)N;
    float best = 0.0f;
    TileCost t;
    for (int i = 0; tile_cost(x_bf16, w_bf16, i, &t); ++i) {
        const int m_blocks = (B + t.rows - 1) / t.rows, n_blocks = (N + t.outputs - 1) / t.outputs, steps = (K + t.k - 1) / t.k;
        const long long tiles = (long long)m_blocks * n_blocks;
        for (int splits = 1; splits <= 16 && (splits == 1 || (tiles * splits <= 512 && steps >= 7 * splits)); ++splits) {
            const int each = (steps + splits - 1) / splits;
            const long long groups = tiles * splits;
            const float rounds = t.paired > 0.0f && groups > 256 ? (float)((groups + 511) / 512) * t.paired
                                                                  : (float)((groups + 255) / 256) * t.alone;
            const float us = 4.0f + (float)each * rounds + (splits > 1 ? 3.0f + outputs * (float)splits * 1.6e-6f : 0.0f);
            if ((i == 0 && splits == 1) || us < best) {
                best = us;
                c.tile = i;
                c.plan.m_blocks = m_blocks;
                c.plan.n_blocks = n_blocks;
                c.plan.split_steps = each;
                c.splits = c.plan.splits = (steps + each - 1) / each;
            }
        }
    }
    c.plan.group = c.plan.n_blocks < 8 ? c.plan.n_blocks : 8;
    return c;
}

}  // namespace

size_t linear_workspace(int B, int K, int N, bool x_bf16, bool w_bf16)
{
    const Choice c = choose(B, K, N, x_bf16, w_bf16);
    return c.splits > 1 ? (size_t)c.splits * (size_t)B * (size_t)N * 4 : 0;
}

void linear_path(int B, int K, int N, bool x_bf16, bool w_bf16, int32_t* path)
{
    const Choice c = choose(B, K, N, x_bf16, w_bf16);
    const bool tiled = c.kind == Choice::tiled, skinny = c.kind == Choice::skinny;
    TileCost t = {};
    if (tiled)
        tile_cost(x_bf16, w_bf16, c.tile, &t);
    path[0] = skinny ? 1 : tiled ? 2 : 0;
    path[1] = skinny ? c.rt : tiled ? c.tile : 0;
    path[2] = skinny && c.swapped;
    path[3] = c.splits;
    path[4] = skinny ? skinny_step(x_bf16, w_bf16) : t.k;
    path[5] = tiled ? c.plan.split_steps : 0;
}

namespace {

hipError_t launch_join(const LinearArgs& p, const float* partial, int splits, hipStream_t s)
{
    // The whole product in us with 8 a thread and with one: 256 x 4096 -> 4096 bfloat16 (2^20 outputs) 24.5 and 25.1,
    // 256 x 7168 -> 8192 (2^21) 63.5 and 64.5, 8192 x 7168 -> 256 with float32 w (2^21) 91 either way; 128 x 4096 -> 4096
    // (2^19) 17.8 and 17.5, 64 x 7168 -> 256 with float32 w (2^14) 9.2 and 8.7.
    if ((size_t)p.B * (size_t)p.N >= 1u << 20) {
        const unsigned threads = (unsigned)p.B * (((unsigned)p.N + 7) / 8);
        hipLaunchKernelGGL(moe_linear_join_kernel<8>, dim3((threads + 255) / 256), dim3(256), 0, s, p, partial, splits, threads);
    } else {
        const unsigned threads = (unsigned)p.B * (unsigned)p.N;
        hipLaunchKernelGGL(moe_linear_join_kernel<1>, dim3((threads + 255) / 256), dim3(256), 0, s, p, partial, splits, threads);
    }
    return hipGetLastError();
}

template <bool X, bool W>
hipError_t launch_dot(const LinearArgs& p, hipStream_t s)
{
    hipLaunchKernelGGL((moe_linear_dot_kernel<X, W>), dim3((unsigned)p.N), dim3(kDotWaves * kWave), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& p, bool x_bf16, bool w_bf16, void* workspace, hipStream_t s)
{
    Choice c = choose(p.B, p.K, p.N, x_bf16, w_bf16);
    if (c.kind == Choice::dot) {
        if (x_bf16)
            return w_bf16 ? launch_dot<true, true>(p, s) : launch_dot<true, false>(p, s);
        return w_bf16 ? launch_dot<false, true>(p, s) : launch_dot<false, false>(p, s);
    }
    c.plan.partial = c.skinny_plan.partial = static_cast<float*>(workspace);
    hipError_t e;
    if (c.kind == Choice::skinny) {
        auto launch = x_bf16 ? (w_bf16 ? launch_skinny_bf16 : launch_skinny_mixed_w)
                             : (w_bf16 ? launch_skinny_mixed_x : launch_skinny_f32);
        e = launch(c.swapped, c.rt, p, c.skinny_plan, s);
    } else {
        auto launch = x_bf16 ? (w_bf16 ? launch_linear_bf16 : launch_linear_mixed_w)
                             : (w_bf16 ? launch_linear_mixed_x : launch_linear_f32);
        e = launch(c.tile, p, c.plan, s);
    }
    if (e != hipSuccess || c.splits == 1)
        return e;
    return launch_join(p, static_cast<const float*>(workspace), c.splits, s);
}

}  // namespace moed
