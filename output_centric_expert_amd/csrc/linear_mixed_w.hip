// Dense products of bfloat16 x and float32 w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

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
