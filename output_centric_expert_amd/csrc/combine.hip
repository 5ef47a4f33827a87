// out[b][h] = sum_j w[b][j] * y[position[b][j]][h], j in increasing order, one
// float32 accumulator, one store. A position outside [0, R) makes the token's
// outputs NaN (no read is made for it).
//
// Memory bound: k rows in, one row out (8192 tokens, 8 rows of 2048 bfloat16
// values each: 302 MB in 50 us, 6.0 TB/s; 60 us without streaming loads and
// stores). A thread owns V neighbouring outputs of one token and asks for up to
// kAhead rows' values before it adds the first; the positions and weights are
// uniform over the workgroup and load as scalars.
#include "mx_device.h"
#include "prompt.h"

namespace moed {

namespace {

constexpr int kAhead = 8;

template <bool BF16, int V>
struct Piece {
    u32x4 a, b;                                    // b: float32 rows only
};

template <bool BF16, int V>
__device__ __forceinline__ void fetch(const void* y, size_t at, Piece<BF16, V>& p)
{
    if constexpr (V == 1) {
        p.a.x = BF16 ? (uint32_t)static_cast<const uint16_t*>(y)[at] << 16 : static_cast<const uint32_t*>(y)[at];
    } else if constexpr (BF16) {
        p.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(y) + at));
    } else {
        p.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const float*>(y) + at));
        p.b = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const float*>(y) + at + 4));
    }
}

template <bool BF16, int V>
__device__ __forceinline__ void add(const Piece<BF16, V>& p, float w, float (&acc)[V])
{
    if constexpr (V == 1) {
        acc[0] = __builtin_fmaf(w, __uint_as_float(p.a.x), acc[0]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                acc[2 * i] = __builtin_fmaf(w, bf16_lo(p.a[i]), acc[2 * i]);
                acc[2 * i + 1] = __builtin_fmaf(w, bf16_hi(p.a[i]), acc[2 * i + 1]);
            } else {
                acc[i] = __builtin_fmaf(w, __uint_as_float(p.a[i]), acc[i]);
                acc[4 + i] = __builtin_fmaf(w, __uint_as_float(p.b[i]), acc[4 + i]);
            }
        }
    }
}

}  // namespace

template <bool YBF16, int V>
__global__ void __launch_bounds__(256)
moe_combine_kernel(CombineArgs p)
{
    const int b = blockIdx.x;
    const int h = (int)(blockIdx.y * 256 + threadIdx.x) * V;
    if (h >= p.H)
        return;
    const int32_t* pos = p.position + (size_t)b * p.k;
    const float* w = p.w + (size_t)b * p.k;
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.0f;
    bool bad = false;
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
        Piece<YBF16, V> r[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j0 + j < p.k) {                    // uniform
                const int at = pos[j0 + j];
                const bool ok = (unsigned)at < (unsigned)p.R;
                bad |= !ok;
                if (ok)
                    fetch<YBF16, V>(p.y, (size_t)at * (size_t)p.H + h, r[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j0 + j < p.k && (unsigned)pos[j0 + j] < (unsigned)p.R)
                add<YBF16, V>(r[j], w[j0 + j], acc);
    }
    if (bad) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            acc[v] = __builtin_nanf("");
    }
    const size_t at = (size_t)b * (size_t)p.H + h;
    if constexpr (V == 1) {
        if (p.out_bf16)
            static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rne(acc[0]);
        else
            static_cast<float*>(p.out)[at] = acc[0];
    } else if (p.out_bf16) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = f32x2_to_bf16x2_rne(acc[2 * i], acc[2 * i + 1]);
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + at));
    } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at) = f32x4{acc[0], acc[1], acc[2], acc[3]};
        *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at + 4) = f32x4{acc[4], acc[5], acc[6], acc[7]};
    }
}

hipError_t launch_combine(const CombineArgs& p, bool y_bf16, hipStream_t s)
{
    const int v = p.H % 8 == 0 ? 8 : 1;
    const dim3 grid((unsigned)p.B, (unsigned)((p.H + 256 * v - 1) / (256 * v))), block(256);
#define MOED_CB(Y, V) hipLaunchKernelGGL((moe_combine_kernel<Y, V>), grid, block, 0, s, p)
    if (v == 8) {
        if (y_bf16) MOED_CB(true, 8);
        else MOED_CB(false, 8);
    } else {
        if (y_bf16) MOED_CB(true, 1);
        else MOED_CB(false, 1);
    }
#undef MOED_CB
    return hipGetLastError();
}

}  // namespace moed
