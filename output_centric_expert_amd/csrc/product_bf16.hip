// Products of bfloat16 rows: weights decoded to bfloat16 with their block scale folded in.
#include "product_tiled.h"

namespace moed {

namespace {

// The tile by the average of rows an expert (all the host knows). gate_up, K = 2048, N = 768, 8 of 128 experts, us of
// the choices next to each other (8 wavefronts where not said; MXFP8 / MXFP4 weights):
//   rows an expert              1         4         16        32        64         128        256
//   16 x 128, 4 wavefronts    37 / 27   77 / 57   90 / 72  120 / 84  178 / 133  297 / 232  548 / 430
//   64 x 128, 4 wavefronts    45 / 32   77 / 55   85 / 57   89 / 64  122 / 101  184 / 156  318 / 254
//   64 x 256                  44 / 27   76 / 58   79 / 60   83 / 69  122 /  99  185 / 127  316 / 216
//   128 x 256                 47 / 37   78 / 58   82 / 60   86 / 70  112 /  96  174 / 158  277 / 244
// MXFP8 outputs need whole blocks of 32 in a wavefront (four fragments):
//   16 x 128, 2 wavefronts    38 / 27   77 / 58   88 / 73  117 / 84  181 / 130  322 / 224  609 / 418
//   64 x 256, 4 wavefronts    48 / 28   78 / 61   80 / 63   89 / 72  136 / 103  205 / 130  351 / 228
//   128 x 256                 59 / 48   92 / 74   93 / 76  104 / 86  113 /  92  197 / 163  308 / 263
template <bool FP4, bool GLU, int OUT>
hipError_t by_rows(const ProductArgs& p, int avg, hipStream_t s)
{
    if constexpr (OUT == kOutMX8) {
        if (avg < 4)
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 1, 4, 1, 2>(p, avg, s);
        if (FP4 || avg < 48)
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 4, 4, 1, 4>(p, avg, s);
        if constexpr (!FP4)
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 4, 4, 2, 4>(p, avg, s);
    } else {
        if (avg < 4)
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 1, 2, 1, 4>(p, avg, s);
        if constexpr (FP4) {
            if (avg < 48)
                return launch_shape<kRowsBF16, FP4, GLU, OUT, 4, 2, 1, 4>(p, avg, s);
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 4, 2, 1, 8>(p, avg, s);
        } else {
            if (avg < 32)
                return launch_shape<kRowsBF16, FP4, GLU, OUT, 4, 2, 1, 8>(p, avg, s);
            return launch_shape<kRowsBF16, FP4, GLU, OUT, 8, 2, 1, 8>(p, avg, s);
        }
    }
    return hipErrorInvalidValue;
}

template <bool FP4>
hipError_t by_out(const ProductArgs& p, int avg, hipStream_t s)
{
    if (p.u_q) {
        if (p.out_kind == kOutBF16)
            return by_rows<FP4, true, kOutBF16>(p, avg, s);
        if (p.out_kind == kOutF32)
            return by_rows<FP4, true, kOutF32>(p, avg, s);
        return by_rows<FP4, true, kOutMX8>(p, avg, s);
    }
    return p.out_kind == kOutBF16 ? by_rows<FP4, false, kOutBF16>(p, avg, s) : by_rows<FP4, false, kOutF32>(p, avg, s);
}

}  // namespace

hipError_t launch_product_bf16(const ProductArgs& p, int avg, hipStream_t s)
{
    return p.fp4 ? by_out<true>(p, avg, s) : by_out<false>(p, avg, s);
}

}  // namespace moed
