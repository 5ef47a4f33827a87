// Products grouped by expert: the layout of the block scales and the choice of
// the kernel.
#include "product_common.h"

namespace moed {

namespace {

// Copies rows of n bytes to rows of `padded` bytes (a multiple of 16, the rest
// zero: scale codes of values that do not exist), 16 bytes a thread: the scales
// of all experts' weight rows (N an expert in each matrix), then of the
// activations' rows. K/32 bytes a row in and up to 16 times that out (K = 32).
// With offsets, experts without rows are left out. An expert has rows only if
// its offsets rise, whatever they are (build_tiles clamps them and takes the
// largest so far), so what the others' places hold is never read.
__global__ void __launch_bounds__(256)
moe_pad_scales_kernel(const uint8_t* f0, const uint8_t* f1, const uint8_t* f2, uint8_t* t0, uint8_t* t1, uint8_t* t2,
                      long long r0, long long r1, long long r2, int n, int padded, const int32_t* offsets, int N)
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
        } else {
            if (row >= r0) {
                row -= r0;
                from = f1;
                to = t1;
            }
            if (offsets) {
                const int e = (int)(row / N);
                if (offsets[e + 1] <= offsets[e])
                    continue;
            }
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
        // Where many experts may be without rows (fewer than four an expert on average) those are left out; where few
        // are, asking costs more. E = 128, 8 of them a token, K = 2880, N = 1120, gate and up in MXFP8: 8 tokens 88.8
        // instead of 98.2 us, 1000 tokens 261.7 instead of 258.1; one token of one of 256 experts, K = 1056, N = 2048:
        // 15.2 instead of 20.7.
        const int32_t* offsets = p.R < 4LL * p.E ? p.offsets : nullptr;
        hipLaunchKernelGGL(moe_pad_scales_kernel, dim3(grid), dim3(256), 0, s, p.w_s, p.u_s, p.a_s, to, tu, ta, w, u, a,
                           p.K / 32, p.s_row, offsets, p.N);
        if (hipError_t e = hipGetLastError())
            return e;
        p.w_s = to;
        p.u_s = p.u_s ? tu : nullptr;
        p.a_s = p.a_s ? ta : nullptr;
    }
    // The kinds of rows choose their tile by the average of rows an expert; their tables are of gate_up, K = 2048, N =
    // 768. The product of K = 768, N = 2048 was timed with every bound halved and doubled: within 10 % at most sizes, but
    // tiles of 16 rows would take 23 instead of 32 us at 4 rows an expert, bfloat16 x MXFP4, and the next larger ones 29
    // instead of 36 at 16, MXFP8 x MXFP4 with float32 outputs.
    const int experts = p.R < p.E ? p.R : p.E;
    const long long avg = ((long long)p.R + experts - 1) / experts;
    if (!p.a_s)
        return launch_product_bf16(p, (int)avg, s);
    if (p.out_kind == kOutF32)
        return launch_product_exact(p, (int)avg, s);
    return p.fast ? launch_product_mx(p, (int)avg, s) : launch_product_rounded(p, (int)avg, s);
}

}  // namespace moed
