// Products grouped by expert: the layout of the block scales and the choice of
// the kernel.
#include "product_common.h"

namespace moed {

namespace {

// Copies rows of n bytes to rows of `padded` bytes (a multiple of 16, the rest
// zero: scale codes of values that do not exist), 16 bytes a thread. Bound by
// memory: 1/32 of the codes' bytes once in and once out.
__global__ void __launch_bounds__(256)
moe_pad_scales_kernel(const uint8_t* f0, const uint8_t* f1, const uint8_t* f2, uint8_t* t0, uint8_t* t1, uint8_t* t2,
                      long long r0, long long r1, long long r2, int n, int padded)
{
    const int per = padded / 16;
    const long long all = (r0 + r1 + r2) * per;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        long long row = i / per;
        const int c = (int)(i - row * per) * 16;
        const uint8_t* from = f0;
        uint8_t* to = t0;
        if (row >= r0 + r1) {
            row -= r0 + r1;
            from = f2;
            to = t2;
        } else if (row >= r0) {
            row -= r0;
            from = f1;
            to = t1;
        }
        from += (size_t)row * n + c;
        u32x4 v{0, 0, 0, 0};
        if (c + 16 <= n) {
            __builtin_memcpy(&v, from, 16);
        } else {
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (c + b < n)
                    v[b / 4] |= (uint32_t)from[b] << (8 * (b % 4));
        }
        *reinterpret_cast<u32x4*>(to + (size_t)row * padded + c) = v;
    }
}

bool fits(int K) { return K % 128 == 0 && K >= 512; }
int padded_row(int K) { return (K / 32 + 15) / 16 * 16; }

}  // namespace

size_t product_scales_bytes(int E, int K, int N, int n_a, bool mx_rows, bool two)
{
    if (fits(K))
        return 0;
    return ((size_t)E * (size_t)N * (two ? 2 : 1) + (mx_rows ? (size_t)n_a : 0)) * (size_t)padded_row(K);
}

hipError_t launch_product(ProductArgs p, void* scales, hipStream_t s)
{
    if (fits(p.K)) {
        p.s_row = p.K / 32;
    } else {
        p.s_row = padded_row(p.K);
        const long long w = (long long)p.E * p.N, u = p.u_s ? w : 0, a = p.a_s ? p.n_a : 0;
        uint8_t* to = static_cast<uint8_t*>(scales);
        uint8_t* tu = to + (size_t)w * p.s_row;
        uint8_t* ta = tu + (size_t)u * p.s_row;
        const long long all = (w + u + a) * (p.s_row / 16);
        const unsigned grid = (unsigned)((all + 255) / 256 < 4096 ? (all + 255) / 256 : 4096);
        hipLaunchKernelGGL(moe_pad_scales_kernel, dim3(grid), dim3(256), 0, s, p.w_s, p.u_s, p.a_s, to, tu, ta, w, u, a,
                           p.K / 32, p.s_row);
        if (hipError_t e = hipGetLastError())
            return e;
        p.w_s = to;
        p.u_s = p.u_s ? tu : nullptr;
        p.a_s = p.a_s ? ta : nullptr;
    }
    const int experts = p.R < p.E ? p.R : p.E;
    const long long avg = ((long long)p.R + experts - 1) / experts;
    if (!p.a_s)
        return launch_product_bf16(p, (int)avg, s);
    return p.out_kind == kOutF32 ? launch_product_exact(p, (int)avg, s) : launch_product_mx(p, (int)avg, s);
}

}  // namespace moed
