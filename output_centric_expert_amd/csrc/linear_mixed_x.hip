// Dense products of float32 x and bfloat16 w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

// us with either (float32 out): 8192 x 4096 -> 4096 636 and 781, 8192 x 7168 -> 256 97 and 108, 2048 x 2048 -> 1024 38.3 and
// 35.2, 1024 x 1024 -> 1024 29.9 and 18.7. x's rows are split once for 256 rows of w in the first; the second fills the chip.
constexpr TileCost kTiles[] = {
    {128, 256, 64, 2.60f, 0.00f},
    {64, 128, 64, 0.95f, 1.50f}};

}  // namespace

bool linear_cost_mixed_x(int tile, TileCost* cost)
{
    if (tile >= (int)(sizeof kTiles / sizeof kTiles[0]))
        return false;
    *cost = kTiles[tile];
    return true;
}

hipError_t launch_linear_mixed_x(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    switch (tile) {
    case 0: return launch_linear_tile<true, false, 4, 4, 2, 4, 2>(p, plan, s);
    case 1: return launch_linear_tile<true, false, 1, 4, 4, 2, 2>(p, plan, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_skinny_mixed_x(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<true, false>(swapped, rt, p, plan, s);
}

}  // namespace moed
