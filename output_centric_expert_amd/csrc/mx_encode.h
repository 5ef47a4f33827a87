// MXFP8 encoding on the device (the prompt-side kernels): block scale from the
// largest magnitude, E4M3 codes.
#pragma once

#include "mx_device.h"

namespace moed {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Largest of v over the four lanes of a quad (DPP quad_perm xor 1, xor 2).
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);
    v = a > v ? a : v;
    const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
    return b > v ? b : v;
}

// UE8M0 scale code of an MXFP8 block from the float32 bits of its largest
// magnitude: floor(log2 amax) - 8 + 127 = exponent field - 8, at least 0 (a
// block of zeros, or one below 2^-118, whose values then underflow); 255 (NaN)
// where the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx8_scale_code(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 8u ? e - 8u : 0u);
}

// Four values -> four E4M3 codes of a block with scale code c: times 2^(127-c)
// (a power of two; exact), saturated to +-448, round to nearest even. NaN
// codes for c = 255.
__device__ __forceinline__ uint32_t mx8_codes4(float v0, float v1, float v2, float v3, uint32_t c)
{
    const float inv = __uint_as_float((254u - (c == 255u ? 0u : c)) << 23);
    v0 = __builtin_amdgcn_fmed3f(v0 * inv, -448.0f, 448.0f);
    v1 = __builtin_amdgcn_fmed3f(v1 * inv, -448.0f, 448.0f);
    v2 = __builtin_amdgcn_fmed3f(v2 * inv, -448.0f, 448.0f);
    v3 = __builtin_amdgcn_fmed3f(v3 * inv, -448.0f, 448.0f);
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v2, v3, r, true);
    return c == 255u ? 0x7F7F7F7Fu : (uint32_t)r;
}

}  // namespace moed
