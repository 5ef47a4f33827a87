// Rows of bfloat16 or float32 values in the registers of one wavefront or
// workgroup: loads, stores and sums (moe_norm, moe_post_norm).
#pragma once

#include "mx_device.h"

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
// lost to underflow is at most 2^15 squares below 2^-126 each: 2^-31 of the sum, or of eps. moe_norm has a kernel of its own
// for such an eps, because the test costs the others: a token of 2048 2.19 instead of 2.10 us, 8192 tokens of 2049 112.7
// instead of 110.1. moe_post_norm, with two norms and an eps of each, tests at run time.
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

// Up to 8 consecutive values from any element's address: n >= 8 goes by loads that ask for the alignment of an element
// only, fewer (a row's end) value by value.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

template <bool NT>
__device__ __forceinline__ u32x4 ld_at2(const uint16_t* p)
{
    const u32x4_at2* q = reinterpret_cast<const u32x4_at2*>(p);
    if constexpr (NT)
        return __builtin_nontemporal_load(q);
    else
        return *q;
}

template <bool NT>
__device__ __forceinline__ f32x4 ld_at4(const float* p)
{
    const f32x4_at4* q = reinterpret_cast<const f32x4_at4*>(p);
    if constexpr (NT)
        return __builtin_nontemporal_load(q);
    else
        return *q;
}

template <bool BF16, bool NT>
__device__ __forceinline__ void load_any(const void* p, size_t at, int n, float (&v)[8])
{
    if (n >= 8) {
        if constexpr (BF16) {
            const u32x4 u = ld_at2<NT>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(u[i]);
                v[2 * i + 1] = bf16_hi(u[i]);
            }
        } else {
            const f32x4 a = ld_at4<NT>(static_cast<const float*>(p) + at);
            const f32x4 b = ld_at4<NT>(static_cast<const float*>(p) + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.0f;
            if (i < n)
                v[i] = BF16 ? bf16_val(static_cast<const uint16_t*>(p)[at + i]) : static_cast<const float*>(p)[at + i];
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store_any(void* p, size_t at, int n, const float (&v)[8])
{
    if (n >= 8) {
        if constexpr (BF16) {
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4_at2*>(static_cast<uint16_t*>(p) + at) = u;
        } else {
            *reinterpret_cast<f32x4_at4*>(static_cast<float*>(p) + at) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_at4*>(static_cast<float*>(p) + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                if constexpr (BF16)
                    static_cast<uint16_t*>(p)[at + i] = f32_to_bf16_rne(v[i]);
                else
                    static_cast<float*>(p)[at + i] = v[i];
            }
    }
}

// Eight values as they lie in memory, from any element on: bfloat16 (b unused) or float32. What is loaded well ahead of its
// use stays raw: a conversion behind a load waits for it.
struct Raw {
    u32x4 a, b;
};

template <bool NT>
__device__ __forceinline__ Raw load_raw(bool bf16, const void* p, size_t at)
{
    Raw r;
    if (bf16) {
        r.a = ld_at2<NT>(static_cast<const uint16_t*>(p) + at);
        r.b = u32x4{0, 0, 0, 0};
    } else {
        r.a = __builtin_bit_cast(u32x4, ld_at4<NT>(static_cast<const float*>(p) + at));
        r.b = __builtin_bit_cast(u32x4, ld_at4<NT>(static_cast<const float*>(p) + at + 4));
    }
    return r;
}

__device__ __forceinline__ void raw_values(bool bf16, const Raw& r, float (&v)[8])
{
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(r.a[i]);
            v[2 * i + 1] = bf16_hi(r.a[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(r.a[i]);
            v[4 + i] = __uint_as_float(r.b[i]);
        }
    }
}

// Fewer than eight, value by value; zeros behind.
__device__ __forceinline__ Raw load_short(bool bf16, const void* p, size_t at, int n)
{
    Raw r = {};
#pragma unroll
    for (int v = 0; v < 7; ++v)
        if (v < n) {
            if (bf16)
                r.a[v / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[at + v] << (16 * (v & 1));
            else if (v < 4)
                r.a[v & 3] = static_cast<const uint32_t*>(p)[at + v];
            else
                r.b[v & 3] = static_cast<const uint32_t*>(p)[at + v];
        }
    return r;
}

}  // namespace

}  // namespace moed
