// Products of MXFP8 rows with float32 outputs: rows and weights are both decoded to bfloat16 with their block scales
// folded in, because the scaled matrix instructions drop more than float32 does (product_mx.hip). Products are exact and
// the sums as good as any order of float32 additions (about 1e-7 of the result's norm).
#include "product_tiled.h"

namespace moed {

namespace {

// The tile by the average of rows an expert (all the host knows). gate_up, K = 2048, N = 768, 8 of 128 experts, us of
// the choices next to each other (MXFP8 / MXFP4 weights):
//   rows an expert              1         4         16        32        64         128        256
//   16 x 128, 4 wavefronts    37 / 27   77 / 56   90 / 71  118 / 86  178 / 144  316 / 251  585 / 458
//   16 x 256, 4 wavefronts    41 / 26   91 / 48  104 / 72  119 / 89  176 / 141  307 / 230  572 / 406
//   32 x 256, 8 wavefronts    47 / 30   78 / 53   81 / 56  108 / 90  158 / 126  270 / 202  497 / 348
//   64 x 128, 4 wavefronts    45 / 29   77 / 63   81 / 64   88 / 76  126 / 112  193 / 151  333 / 259
//   128 x 128, 4 wavefronts   47 / 35   80 / 59   85 / 60   93 / 77  119 / 113  182 / 168  297 / 266
template <bool FP4, bool GLU>
hipError_t by_rows(const ProductArgs& p, int avg, hipStream_t s)
{
    if constexpr (FP4) {
        // up to 32 rows in all: few tiles, so a short one is done sooner (two fragments of weights 13.5 us, four 18.0, at
        // 8 rows; 32 rows 16.8 and 18.7, 128 rows 30.5 and 29.7)
        if (avg < 4 && p.R < 32)
            return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 1, 2, 1, 4>(p, avg, s);
        if (avg < 8)
            return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 1, 4, 1, 4>(p, avg, s);
        if (avg < 24)
            return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 2, 2, 1, 8>(p, avg, s);
        return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 4, 2, 1, 4>(p, avg, s);
    } else {
        if (avg < 4)
            return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 1, 2, 1, 4>(p, avg, s);
        if (avg < 48)
            return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 4, 2, 1, 4>(p, avg, s);
        return launch_shape<kRowsMXExact, FP4, GLU, kOutF32, 8, 2, 1, 4>(p, avg, s);
    }
}

}  // namespace

hipError_t launch_product_exact(const ProductArgs& p, int avg, hipStream_t s)
{
    if (p.u_q)
        return p.fp4 ? by_rows<true, true>(p, avg, s) : by_rows<false, true>(p, avg, s);
    return p.fp4 ? by_rows<true, false>(p, avg, s) : by_rows<false, false>(p, avg, s);
}

}  // namespace moed
