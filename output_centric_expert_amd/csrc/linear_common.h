// What the kernels of the dense product share: loads of rows that begin at any element, and the epilogue
//   out[b][n] = act(v + bias[n]) + residual[b][n], rounded once.
#pragma once

#include "activation.h"
#include "lds_loads.h"
#include "row_values.h"

namespace moed {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace {

__device__ __forceinline__ float value_at(bool bf16, const void* p, size_t at)
{
    return bf16 ? bf16_val(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// One output.
__device__ __forceinline__ void linear_store(const LinearArgs& p, float sum, size_t b, int n)
{
    float v[1] = {p.bias ? sum + value_at(p.bias_bf16, p.bias, (size_t)n) : sum};
    activate(v, p.act);
    const size_t at = b * (size_t)p.N + (size_t)n;
    if (p.residual)
        v[0] += value_at(p.residual_bf16, p.residual, at);
    if (p.out_bf16)
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rne(v[0]);
    else
        static_cast<float*>(p.out)[at] = v[0];
}

// Eight neighbouring values as they lie in memory: bfloat16 (b unused) or float32.
struct Eight {
    u32x4 a, b;
};

__device__ __forceinline__ Eight load_eight(bool bf16, const void* p, size_t at)
{
    Eight e;
    if (bf16) {
        e.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at));
        e.b = e.a;
    } else {
        e.a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at));
        e.b = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at + 4));
    }
    return e;
}

__device__ __forceinline__ void add_eight(bool bf16, const Eight& e, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            v[2 * i] += bf16_lo(e.a[i]);
            v[2 * i + 1] += bf16_hi(e.a[i]);
        } else {
            v[i] += __uint_as_float(e.a[i]);
            v[4 + i] += __uint_as_float(e.b[i]);
        }
    }
}

// Units of 16 bytes of a row are stored at u ^ linear_swizzle(row). One of the four passes of a 16-byte LDS read serves 16
// lanes of two lane groups: units u of 8 rows of a fragment and u + 1 (bfloat16) or u + 2 (float32) of the other 8, rows
// 0-3 and 12-15 apart from 4-11. These are the patterns for which they meet all 64 banks, two rows of 8 units or one of 16
// in a line of them.
template <bool F32, int UNITS>
__device__ __forceinline__ int linear_swizzle(int row)
{
    return UNITS == 16 ? row & 15 : F32 ? (row >> 1) & 5 : row & 7;
}

// Byte offset of unit u of row `col` (below 16) of a fragment.
template <bool F32, int UNITS>
__device__ __forceinline__ int linear_unit(int col, int u)
{
    return (col * UNITS + (u ^ linear_swizzle<F32, UNITS>(col))) * 16;
}

// 8 float32 values as the sum of three bfloat16 each.
__device__ __forceinline__ void split3(u32x4 lo, u32x4 hi, bf16x8 (&part)[3])
{
    u32x4 p0, p1, p2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(i < 2 ? lo[2 * i] : hi[2 * i - 4]);
        const float b = __uint_as_float(i < 2 ? lo[2 * i + 1] : hi[2 * i - 3]);
        p0[i] = f32x2_to_bf16x2_rne(a, b);
        const float a1 = a - bf16_lo(p0[i]), b1 = b - bf16_hi(p0[i]);
        p1[i] = f32x2_to_bf16x2_rne(a1, b1);
        p2[i] = f32x2_to_bf16x2_rne(a1 - bf16_lo(p1[i]), b1 - bf16_hi(p1[i]));
    }
    part[0] = __builtin_bit_cast(bf16x8, p0);
    part[1] = __builtin_bit_cast(bf16x8, p1);
    part[2] = __builtin_bit_cast(bf16x8, p2);
}

// 16 bytes of a row from any element, zeros behind its end.
template <bool F32>
__device__ __forceinline__ u32x4 row_unit(const void* row, int k, int K)
{
    u32x4 v = {0, 0, 0, 0};
    if constexpr (F32) {
        const float* p = static_cast<const float*>(row) + k;
        if (k + 4 <= K) {
            v = __builtin_bit_cast(u32x4, ld_at4<false>(p));
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (k + i < K)
                    v[i] = __float_as_uint(p[i]);
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(row) + k;
        if (k + 8 <= K) {
            v = ld_at2<false>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (k + i < K)
                    v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        }
    }
    return v;
}

// The fragment whose 16 rows of UNITS units begin at `at`, for k 32 s .. 32 s + 31 of the step: lane group g has 8 of
// them, in three parts with float32.
template <bool F32, int UNITS>
__device__ __forceinline__ void linear_fragment(const uint8_t* at, int s, int g, int col, bf16x8 (&part)[F32 ? 3 : 1])
{
    if constexpr (F32)
        split3(lds16(at + linear_unit<true, UNITS>(col, 8 * s + 2 * g)), lds16(at + linear_unit<true, UNITS>(col, 8 * s + 2 * g + 1)), part);
    else
        part[0] = __builtin_bit_cast(bf16x8, lds16(at + linear_unit<false, UNITS>(col, 4 * s + g)));
}

// The parts' products, small ones first: all of one side's three, or the six of nine that count. a: its rows become the
// sums' four registers, b: their lanes.
template <bool B32, bool A32>
__device__ __forceinline__ void linear_products(const bf16x8 (&a)[A32 ? 3 : 1], const bf16x8 (&b)[B32 ? 3 : 1], f32x4& acc)
{
    constexpr int NA = A32 ? 3 : 1, NB = B32 ? 3 : 1;
#pragma unroll
    for (int q = (A32 || B32) ? 2 : 0; q >= 0; --q)
#pragma unroll
        for (int i = 0; i < NB; ++i)
            if (q - i >= 0 && q - i < NA)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q - i], b[i], acc, 0, 0, 0);
}

// What this wavefront wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace

}  // namespace moed
