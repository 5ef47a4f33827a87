// Dense products of bfloat16 x and float32 w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

// us with either (float32 out): 8192 x 4096 -> 4096 611 and 1050, 8192 x 7168 -> 256 89 and 132, 2048 x 2048 -> 1024 39.9 and
// 37.8, 1024 x 1024 -> 1024 28.3 and 16.4. w's rows are split once for 256 rows of x in the first; the second fills the chip.
constexpr TileCost kTiles[] = {
    {256, 128, 64, 2.45f, 0.00f},
    {64, 64, 64, 0.80f, 1.05f}};

}  // namespace

bool linear_cost_mixed_w(int tile, TileCost* cost)
{
    if (tile >= (int)(sizeof kTiles / sizeof kTiles[0]))
        return false;
    *cost = kTiles[tile];
    return true;
}

hipError_t launch_linear_mixed_w(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    switch (tile) {
    case 0: return launch_linear_tile<false, true, 8, 2, 2, 4, 2>(p, plan, s);
    case 1: return launch_linear_tile<false, true, 2, 1, 2, 4, 2>(p, plan, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_skinny_mixed_w(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<false, true>(swapped, rt, p, plan, s);
}

}  // namespace moed
