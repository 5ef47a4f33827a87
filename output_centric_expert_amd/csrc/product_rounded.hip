// Products of MXFP8 rows with bfloat16 or MXFP8 outputs: as for float32 outputs (product_exact.hip) rows and weights are
// both decoded to bfloat16 with their block scales folded in, so that sums are as good as any order of float32 additions
// and an output is the rounding of such a sum. The scaled matrix instructions (product_mx.hip) take about half the time
// for long prompts, but drop what lies 2^-14 below the largest of eight neighbouring products; a caller asks for them.
//
// A block scale outside the range that the decode holds exactly (10..245 of MXFP8, 2..252 of MXFP4; 255 is NaN either
// way), of a block that is not all zeros, makes its tile be computed once more with the scaled instructions, which take
// any scale. Steps that hold such a scale look at the block's codes: 8192 tokens, half of them zeros with scale 0, take 664
// us instead of 551 (gate_up below); with such a block in every second row, all tiles twice, 773.
#include "product_tiled.h"

namespace moed {

namespace {

// The tile by the average of rows an expert (all the host knows). 8 of 128 experts, us of the choices next to each other
// (rows x weight rows; 4 wavefronts where not said; MXFP8 / MXFP4 weights). gate_up, K = 2048, N = 768:
//   rows an expert              1         4         16        32        64         128        256        512
//   16 x 128                  37 / 22   78 / 48  107 / 63  119 / 90  186 / 151  338 / 268  640 / 499  1250 / 965
//   64 x 128                  43 / 26   79 / 56   81 / 57   90 / 69  129 / 114  201 / 162  350 / 283   637 / 516
//   64 x 256                  53 / 30   81 / 53   84 / 55   95 / 63  151 /  93  234 / 145  399 / 240   736 / 436
//   128 x 128                           95 / 77   94 / 78  116 / 97  118 / 102  179 / 150  296 / 268   517 / 471
// the product, K = 768, N = 2048:
//   16 x 128                  21 / 15   44 / 25   54 / 35   71 / 51  114 /  87  209 / 161  389 / 299   756 / 580
//   64 x 128                  22 / 17   44 / 28   46 / 30   51 / 36   76 /  57  117 /  85  205 / 151   377 / 272
//   64 x 256                  25 / 17   49 / 29   51 / 31   56 / 35   91 /  57  130 /  83  227 / 143   426 / 265
//   128 x 128                           55 / 45   56 / 46   64 / 55   71 /  62  105 /  94  168 / 152   300 / 274
// and gate_up with MXFP8 outputs, which need whole blocks of 32 in a wavefront (four fragments):
//   16 x 128, 2 wavefronts    39 / 26   80 / 55  102 / 69  126 / 88  213 / 145  392 / 262  746 / 491  1457 / 949
//   32 x 256                  53 / 31   81 / 52   84 / 55  126 / 78  192 / 110  330 / 171  609 / 299  1163 / 537
//   64 x 256                  53 / 31   82 / 53   85 / 56   95 / 64  153 /  95  234 / 144  403 / 244   741 / 445
//   128 x 128                           92 / 79   97 / 82  118 / 99  122 / 105  183 / 156  313 / 275   540 / 471
// (256 x 256 does not fit in the registers: 915 at 512 rows.)
template <bool FP4, bool GLU, int OUT>
hipError_t by_rows(const ProductArgs& p, int avg, hipStream_t s)
{
    if constexpr (OUT == kOutMX8) {
        if (avg < 4)
            return launch_shape<kRowsMXExact, FP4, GLU, OUT, 1, 4, 1, 2>(p, avg, s);
        if (avg < 24)
            return launch_shape<kRowsMXExact, FP4, GLU, OUT, 2, 4, 1, 4>(p, avg, s);
    } else {
        if (avg < (FP4 ? 8 : 4))
            return launch_shape<kRowsMXExact, FP4, GLU, OUT, 1, 2, 1, 4>(p, avg, s);
    }
    if constexpr (FP4) {
        return launch_shape<kRowsMXExact, FP4, GLU, OUT, 4, 4, 1, 4>(p, avg, s);
    } else {
        if (avg < 48)
            return launch_shape<kRowsMXExact, FP4, GLU, OUT, 4, OUT == kOutMX8 ? 4 : 2, 1, 4>(p, avg, s);
        return launch_shape<kRowsMXExact, FP4, GLU, OUT, 4, 4, 2, 2>(p, avg, s);
    }
}

template <bool FP4>
hipError_t by_out(const ProductArgs& p, int avg, hipStream_t s)
{
    if (!p.u_q)
        return by_rows<FP4, false, kOutBF16>(p, avg, s);
    return p.out_kind == kOutBF16 ? by_rows<FP4, true, kOutBF16>(p, avg, s) : by_rows<FP4, true, kOutMX8>(p, avg, s);
}

}  // namespace

hipError_t launch_product_rounded(const ProductArgs& p, int avg, hipStream_t s)
{
    return p.fp4 ? by_out<true>(p, avg, s) : by_out<false>(p, avg, s);
}

}  // namespace moed
