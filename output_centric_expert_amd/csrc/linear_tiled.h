// The kernel of the dense product for more than a few rows: tiles of rows of x times rows of w, through LDS, on the
// matrix instructions. Included by one source file per pair of types.
//
// A step is kBK values of k, in two buffers: while a step is multiplied the next one goes from memory straight to LDS.
// A float32 operand stays as it is in LDS and is split as its fragments are read, into three bfloat16 whose sum is the
// value (each the rounded rest of the ones before: 8 + 8 + 8 bits of a float32's 24). A bfloat16 times a float32 value
// is then three exact products, two float32 values take the six of the nine that reach 2^-23 of the product. That is
// float32's precision at a third (a sixth) of the bfloat16 rate; the float32 matrix instructions have a sixteenth.
#pragma once

#include <type_traits>

#include "lds_loads.h"
#include "linear_common.h"

namespace moed {

// Where a call's tiles lie. splits > 1: each split's sums go to partial [splits][B][N] instead of the epilogue.
struct LinearPlan {
    float* partial;
    int n_blocks, m_blocks, splits, split_steps;
    int group;              // blocks of w's rows that are taken together
};

namespace {

template <bool XF32, bool WF32, int RT, int NT, int WR, int WN>
struct LinearShape {
    static constexpr int kWaves = WR * WN, kThreads = kWaves * kWave;
    static constexpr int kBM = 16 * RT * WR, kBN = 16 * NT * WN;          // rows of x and of w in a tile
    static constexpr int kBK = XF32 && WF32 ? 32 : 64;
    static constexpr int kXU = kBK * (XF32 ? 4 : 2) / 16, kWU = kBK * (WF32 ? 4 : 2) / 16;     // units of a row and step
    static constexpr int kXBytes = kBM * kXU * 16, kWBytes = kBN * kWU * 16;
    static constexpr int kXLoads = kBM * kXU / kThreads, kWLoads = kBN * kWU / kThreads;
    static constexpr int kBuffer = kXBytes + kWBytes;
    // outputs of a wavefront on their way out: strips of 16 rows, as many as fit
    static constexpr int kOutRow = 16 * NT + 4;                           // float32 values, padded
    static constexpr int kStrip = kWaves * 16 * kOutRow * 4;
    static constexpr int kStrips = RT * kStrip <= 2 * kBuffer ? RT : RT / 2 * kStrip <= 2 * kBuffer ? RT / 2 : RT / 4;
    static constexpr int kLds = 2 * kBuffer;
    static_assert(kBM * kXU % kThreads == 0 && kBN * kWU % kThreads == 0, "whole loads");
    static_assert((kThreads / kXU) % 16 == 0 && (kThreads / kWU) % 16 == 0, "a thread's loads share their place in the row");
    static_assert(kStrips >= 1 && kStrips * kStrip <= kLds, "room for the outputs");
};

}  // namespace

// DIRECT: rows begin at 16-byte borders (any K % 8 = 0, or % 4 with float32), so that whole steps go straight to LDS.
template <bool XF32, bool WF32, bool DIRECT, int RT, int NT, int WR, int WN>
__global__ void __launch_bounds__(WR * WN * kWave)
moe_linear_tiled_kernel(LinearArgs p, LinearPlan plan)
{
    using S = LinearShape<XF32, WF32, RT, NT, WR, WN>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int g = lane / 16, col = lane % 16;
    const int wr = w / WN, wn = w % WN;
    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)lds;

    // neighbouring workgroups of an XCD share rows of x and of w
    const int tiles = plan.n_blocks * plan.m_blocks;
    const int item = xcd_contiguous(blockIdx.x, gridDim.x);
    const int split = item / tiles, tile = item - split * tiles;
    const int first = tile / (plan.group * plan.m_blocks) * plan.group;       // of this group's blocks
    const int rest = tile - first * plan.m_blocks;
    const int width = plan.n_blocks - first < plan.group ? plan.n_blocks - first : plan.group;
    const int mb = rest / width, nb = first + rest - mb * width;
    const size_t m0 = (size_t)mb * S::kBM;
    const int n0 = nb * S::kBN;
    const int all = (p.K + S::kBK - 1) / S::kBK;
    const int st0 = split * plan.split_steps, st1 = st0 + plan.split_steps < all ? st0 + plan.split_steps : all;
    const int full = DIRECT ? p.K / S::kBK : 0;               // steps that go straight to LDS

    // sources: a uniform base and 32-bit offsets of this thread's rows; those behind the last repeat it
    const int xc = (tid % S::kXU) ^ linear_swizzle<XF32, S::kXU>(tid / S::kXU);
    const int wc = (tid % S::kWU) ^ linear_swizzle<WF32, S::kWU>(tid / S::kWU);
    const size_t x_row = (size_t)p.K * (XF32 ? 4 : 2), w_row = (size_t)p.K * (WF32 ? 4 : 2);
    const uint8_t* const xbase = static_cast<const uint8_t*>(p.x) + m0 * x_row;
    const uint8_t* const wbase = static_cast<const uint8_t*>(p.w) + (size_t)n0 * w_row;
    uint32_t xoff[S::kXLoads], woff[S::kWLoads];
    {
        const int xlast = (size_t)p.B - m0 < (size_t)S::kBM ? (int)((size_t)p.B - m0) - 1 : S::kBM - 1;
        const int wlast = p.N - n0 < S::kBN ? p.N - n0 - 1 : S::kBN - 1;
#pragma unroll
        for (int i = 0; i < S::kXLoads; ++i) {
            const int r = i * (S::kThreads / S::kXU) + tid / S::kXU;
            xoff[i] = (uint32_t)(r < xlast ? r : xlast) * (uint32_t)x_row;
        }
#pragma unroll
        for (int i = 0; i < S::kWLoads; ++i) {
            const int r = i * (S::kThreads / S::kWU) + tid / S::kWU;
            woff[i] = (uint32_t)(r < wlast ? r : wlast) * (uint32_t)w_row;
        }
    }
    auto stage = [&](int st) {
        const int to = (st & 1) * S::kBuffer;
        if (st < full) {
            const uint32_t at = lds0 + (uint32_t)(to + w * 1024);
            const uint8_t* xs = xbase + (size_t)st * (S::kXU * 16);
            const uint8_t* ws = wbase + (size_t)st * (S::kWU * 16);
#pragma unroll
            for (int i = 0; i < S::kXLoads; ++i)
                load_to_lds16(xs, xoff[i] + 16u * xc, at + i * S::kThreads * 16);
#pragma unroll
            for (int i = 0; i < S::kWLoads; ++i)
                load_to_lds16(ws, woff[i] + 16u * wc, at + S::kXBytes + i * S::kThreads * 16);
        } else {
            u32x4* const x16 = reinterpret_cast<u32x4*>(lds + to) + tid;
            u32x4* const w16 = reinterpret_cast<u32x4*>(lds + to + S::kXBytes) + tid;
#pragma unroll
            for (int i = 0; i < S::kXLoads; ++i)
                x16[i * S::kThreads] = row_unit<XF32>(xbase + xoff[i], st * S::kBK + xc * (S::kBK / S::kXU), p.K);
#pragma unroll
            for (int i = 0; i < S::kWLoads; ++i)
                w16[i * S::kThreads] = row_unit<WF32>(wbase + woff[i], st * S::kBK + wc * (S::kBK / S::kWU), p.K);
        }
    };

    f32x4 acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int f = 0; f < NT; ++f)
            acc[r][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int XP = XF32 ? 3 : 1, WP = WF32 ? 3 : 1;
    auto compute = [&](int st) {
        const uint8_t* xb = lds + (st & 1) * S::kBuffer + wr * RT * 16 * S::kXU * 16;
        const uint8_t* wb = lds + (st & 1) * S::kBuffer + S::kXBytes + wn * NT * 16 * S::kWU * 16;
#pragma unroll
        for (int s = 0; s < S::kBK / 32; ++s) {
            bf16x8 wv[NT][WP];
#pragma unroll
            for (int f = 0; f < NT; ++f)
                linear_fragment<WF32, S::kWU>(wb + f * 16 * S::kWU * 16, s, g, col, wv[f]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                bf16x8 xv[XP];
                linear_fragment<XF32, S::kXU>(xb + r * 16 * S::kXU * 16, s, g, col, xv);
                // small parts first, and the same accumulator not twice in a row
#pragma unroll
                for (int q = (XF32 || WF32) ? 2 : 0; q >= 0; --q)
#pragma unroll
                    for (int i = 0; i < XP; ++i)
                        if (q - i >= 0 && q - i < WP)
#pragma unroll
                            for (int f = 0; f < NT; ++f)
                                acc[r][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f][q - i], xv[i], acc[r][f], 0, 0, 0);
            }
        }
    };
    stage(st0);
    for (int st = st0; st < st1; ++st) {
        wait_loads<0>();
        __syncthreads();                                      // step st is in LDS, and nobody reads the other buffer
        if (st + 1 < st1)
            stage(st + 1);
        compute(st);
    }
    __syncthreads();

    // A lane holds outputs 4 g .. 4 g + 3 of row col: through LDS, some strips of 16 rows at a time, so that a lane has 8
    // neighbouring outputs and a row's leave together.
    float* const mine = reinterpret_cast<float*>(lds) + w * (S::kStrips * 16 * S::kOutRow);
    constexpr int kCols = 16 * NT, kRowsAtOnce = kWave * 8 / kCols;
    const bool eights = p.N % 8 == 0;                         // a row's eights are whole, and begin at 16-byte borders
    const bool partial = plan.splits > 1;
    const int i8 = lane / (kCols / 8), c8 = lane % (kCols / 8) * 8, n8 = n0 + wn * kCols + c8;
    Eight bias = {};
    if (p.bias && eights && n8 < p.N) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = value_at(p.bias_bf16, p.bias, (size_t)n8 + i);
        bias.a = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        bias.b = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    }
#pragma unroll
    for (int part = 0; part < RT / S::kStrips; ++part) {
        const size_t b0 = m0 + (size_t)(wr * RT + part * S::kStrips) * 16;
        const int live = b0 >= (size_t)p.B ? 0 : (size_t)p.B - b0 < (size_t)S::kStrips * 16 ? (int)((size_t)p.B - b0) : S::kStrips * 16;
        const size_t at0 = b0 * (size_t)p.N + (size_t)n8;
        Eight next = {};                                      // of the residual, asked for one turn ahead
        if (eights && p.residual && !partial && i8 < live && n8 < p.N)
            next = load_eight(p.residual_bf16, p.residual, at0 + (size_t)i8 * (size_t)p.N);
#pragma unroll
        for (int r = 0; r < S::kStrips; ++r)
#pragma unroll
            for (int f = 0; f < NT; ++f)
                *reinterpret_cast<f32x4*>(mine + (r * 16 + col) * S::kOutRow + f * 16 + 4 * g) = acc[part * S::kStrips + r][f];
        wave_lds_fence();
        if (eights) {
#pragma unroll 1
            for (int i = i8; i < live; i += kRowsAtOnce) {
                if (n8 >= p.N)
                    break;
                const f32x4 lo = *reinterpret_cast<const f32x4*>(mine + i * S::kOutRow + c8);
                const f32x4 hi = *reinterpret_cast<const f32x4*>(mine + i * S::kOutRow + c8 + 4);
                if (partial) {
                    float* to = plan.partial + ((size_t)split * (size_t)p.B) * (size_t)p.N + at0 + (size_t)i * (size_t)p.N;
                    *reinterpret_cast<f32x4*>(to) = lo;
                    *reinterpret_cast<f32x4*>(to + 4) = hi;
                    continue;
                }
                const Eight residual = next;
                if (p.residual && i + kRowsAtOnce < live)
                    next = load_eight(p.residual_bf16, p.residual, at0 + (size_t)(i + kRowsAtOnce) * (size_t)p.N);
                float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                if (p.bias)
                    add_eight(false, bias, v);
                activate(v, p.act);
                if (p.residual)
                    add_eight(p.residual_bf16, residual, v);
                if (p.out_bf16)
                    store_vals<true>(p.out, at0 + (size_t)i * (size_t)p.N, v);
                else
                    store_vals<false>(p.out, at0 + (size_t)i * (size_t)p.N, v);
            }
        } else {
            constexpr int kPer = kWave / kCols;               // rows that a wavefront stores at once, value by value
            const int n = n0 + wn * kCols + lane % kCols;
            if (n < p.N)
#pragma unroll 1
                for (int i = lane / kCols; i < live; i += kPer) {
                    const float v = mine[i * S::kOutRow + lane % kCols];
                    if (partial)
                        plan.partial[((size_t)split * (size_t)p.B + b0 + i) * (size_t)p.N + n] = v;
                    else
                        linear_store(p, v, b0 + i, n);
                }
        }
        wave_lds_fence();
    }
}

// Tiles of the shapes that a pair of types has (linear.hip chooses one).
constexpr int kTileSmall = 0, kTileMiddle = 1, kTileLarge = 2, kTiles = 3;
struct TileSize {
    int rows, outputs, k;   // of x, of w, of a step
};

template <bool XF32, bool WF32, bool DIRECT, int RT, int NT, int WR, int WN>
hipError_t launch_linear_shape(const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    using S = LinearShape<XF32, WF32, RT, NT, WR, WN>;
    static_assert(16 * NT <= kWave, "a wavefront stores whole rows of its outputs");
    const void* f = reinterpret_cast<const void*>(&moe_linear_tiled_kernel<XF32, WF32, DIRECT, RT, NT, WR, WN>);
    if (S::kLds > 49152)
        if (hipError_t e = set_max_dynamic_lds(f, S::kLds))
            return e;
    const unsigned grid = (unsigned)((long long)plan.n_blocks * plan.m_blocks * plan.splits);
    hipLaunchKernelGGL((moe_linear_tiled_kernel<XF32, WF32, DIRECT, RT, NT, WR, WN>), dim3(grid), dim3(S::kThreads), S::kLds, s, p,
                       plan);
    return hipGetLastError();
}

template <bool XF32, bool WF32, int RT, int NT, int WR, int WN>
hipError_t launch_linear_tile(const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    if (p.K % (XF32 ? 4 : 8) == 0 && p.K % (WF32 ? 4 : 8) == 0)
        return launch_linear_shape<XF32, WF32, true, RT, NT, WR, WN>(p, plan, s);
    return launch_linear_shape<XF32, WF32, false, RT, NT, WR, WN>(p, plan, s);
}

// f(RT, NT, WR, WN) with the shape of a tile, as constants.
template <bool XF32, bool WF32, typename F>
auto with_tile(int tile, F&& f)
{
    auto shape = [&](auto rt, auto nt, auto wr, auto wn) { return f(rt, nt, wr, wn); };
#define MOED_TILE(RT, NT, WR, WN) \
    shape(std::integral_constant<int, RT>{}, std::integral_constant<int, NT>{}, std::integral_constant<int, WR>{}, \
          std::integral_constant<int, WN>{})
    if (tile == kTileSmall)
        return MOED_TILE(2, 2, 1, 4);
    if constexpr (XF32 && WF32)
        return MOED_TILE(4, 4, 2, 2);
    else if constexpr (XF32)
        return tile == kTileMiddle ? MOED_TILE(4, 2, 2, 4) : MOED_TILE(4, 4, 2, 4);
    else if constexpr (WF32)
        return tile == kTileMiddle ? MOED_TILE(4, 2, 2, 4) : MOED_TILE(8, 2, 2, 4);
    else
        return tile == kTileMiddle ? MOED_TILE(4, 4, 2, 2) : MOED_TILE(8, 4, 2, 4);
#undef MOED_TILE
}

template <bool XF32, bool WF32>
TileSize tile_size(int tile)
{
    return with_tile<XF32, WF32>(tile, [](auto rt, auto nt, auto wr, auto wn) {
        using S = LinearShape<XF32, WF32, rt, nt, wr, wn>;
        return TileSize{S::kBM, S::kBN, S::kBK};
    });
}

template <bool XF32, bool WF32>
hipError_t launch_tile(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    return with_tile<XF32, WF32>(tile, [&](auto rt, auto nt, auto wr, auto wn) {
        return launch_linear_tile<XF32, WF32, rt, nt, wr, wn>(p, plan, s);
    });
}

// One source file per pair of types.
TileSize linear_tile_bf16(int tile);
TileSize linear_tile_mixed_w(int tile);       // bfloat16 x, float32 w
TileSize linear_tile_mixed_x(int tile);       // float32 x, bfloat16 w
TileSize linear_tile_f32(int tile);
hipError_t launch_linear_bf16(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_mixed_w(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_mixed_x(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_f32(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);

}  // namespace moed
