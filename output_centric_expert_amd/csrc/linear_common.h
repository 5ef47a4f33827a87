// What the kernels of the dense product share: loads of rows that begin at any element, and the epilogue
//   out[b][n] = act(v + bias[n]) + residual[b][n], rounded once.
#pragma once

#include "activation.h"
#include "lds_loads.h"
#include "mx_encode.h"
#include "row_values.h"

namespace moed {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace {

__device__ __forceinline__ float value_at(bool bf16, const void* p, size_t at)
{
    return bf16 ? bf16_val(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// Sums to outputs.
template <int V>
__device__ __forceinline__ void linear_finish(const LinearArgs& p, const float (&bias)[V], const float (&residual)[V], float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] += bias[i];
    activate(v, p.act);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] += residual[i];
}

// One output.
__device__ __forceinline__ void linear_store(const LinearArgs& p, float sum, size_t b, int n)
{
    const size_t at = b * (size_t)p.N + (size_t)n;
    float v[1] = {sum};
    const float bias[1] = {p.bias ? value_at(p.bias_bf16, p.bias, (size_t)n) : 0.0f};
    const float residual[1] = {p.residual ? value_at(p.residual_bf16, p.residual, at) : 0.0f};
    linear_finish(p, bias, residual, v);
    if (p.out_bf16)
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rne(v[0]);
    else
        static_cast<float*>(p.out)[at] = v[0];
}

// Up to 8 neighbouring values from any element on.
__device__ __forceinline__ void load_some(bool bf16, const void* p, size_t at, int n, float (&v)[8])
{
    if (bf16)
        load_any<true, true>(p, at, n, v);
    else
        load_any<false, true>(p, at, n, v);
}

__device__ __forceinline__ void store_some(bool bf16, void* p, size_t at, int n, const float (&v)[8])
{
    if (bf16)
        store_any<true>(p, at, n, v);
    else
        store_any<false>(p, at, n, v);
}

// Units of 16 bytes of a row are stored at u ^ linear_swizzle(row). One of the four passes of a 16-byte LDS read serves 16
// lanes of two lane groups: units u of 8 rows of a fragment and u + 1 (u + 2 where a unit is half of a lane's values) of
// the other 8, rows 0-3 and 12-15 apart from 4-11. With these patterns they meet all 64 banks, whose line holds four rows
// of 4 units, two of 8 or one of 16.
template <int UNITS, bool TWO = false>
__device__ __forceinline__ int linear_swizzle(int row)
{
    if constexpr (UNITS == 4) {
        const int i = (row >> 2) & 3;
        return ((i ^ (i >> 1)) & 1) * 2 + (i >> 1);
    }
    return UNITS == 16 ? row & 15 : TWO ? (row >> 1) & 5 : row & 7;
}

// Byte offset of unit u of row `col` (below 16) of a fragment.
template <int UNITS, bool TWO = false>
__device__ __forceinline__ int linear_unit(int col, int u)
{
    return (col * UNITS + (u ^ linear_swizzle<UNITS, TWO>(col))) * 16;
}

// 4 float32 values as the sum of three bfloat16 each.
__device__ __forceinline__ void split3(u32x4 v, u32x2 (&part)[3])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = __uint_as_float(v[2 * i]), b = __uint_as_float(v[2 * i + 1]);
        part[0][i] = f32x2_to_bf16x2_rne(a, b);
        const float a1 = a - bf16_lo(part[0][i]), b1 = b - bf16_hi(part[0][i]);
        part[1][i] = f32x2_to_bf16x2_rne(a1, b1);
        part[2][i] = f32x2_to_bf16x2_rne(a1 - bf16_lo(part[1][i]), b1 - bf16_hi(part[1][i]));
    }
}

// 16 bytes of a row from any element.
template <bool F32>
__device__ __forceinline__ u32x4 row_unit_at(const void* row, int k)
{
    if constexpr (F32)
        return __builtin_bit_cast(u32x4, ld_at4<false>(static_cast<const float*>(row) + k));
    else
        return ld_at2<false>(static_cast<const uint16_t*>(row) + k);
}

// The same with zeros behind the row's end.
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
    if constexpr (F32) {
        u32x2 lo[3], hi[3];
        split3(lds16(at + linear_unit<UNITS, true>(col, 8 * s + 2 * g)), lo);
        split3(lds16(at + linear_unit<UNITS, true>(col, 8 * s + 2 * g + 1)), hi);
#pragma unroll
        for (int q = 0; q < 3; ++q)
            part[q] = __builtin_bit_cast(bf16x8, u32x4{lo[q].x, lo[q].y, hi[q].x, hi[q].y});
    } else
        part[0] = __builtin_bit_cast(bf16x8, lds16(at + linear_unit<UNITS>(col, 4 * s + g)));
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

}  // namespace

}  // namespace moed
