// Dense products of bfloat16 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

constexpr TileCost kTiles[] = {
    {256, 256, 64, 1.67f, 0.00f},
    {128, 256, 64, 1.00f, 0.00f},
    {64, 128, 64, 0.46f, 0.60f},
    {64, 128, 64, 0.44f, 0.00f}};

}  // namespace

bool linear_cost_bf16(int tile, TileCost* cost)
{
    if (tile >= (int)(sizeof kTiles / sizeof kTiles[0]))
        return false;
    *cost = kTiles[tile];
    return true;
}

hipError_t launch_linear_bf16(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    switch (tile) {
    case 0: return launch_linear_tile<false, false, 8, 4, 2, 4, kDeep>(p, plan, s);
    case 1: return launch_linear_tile<false, false, 4, 4, 2, 4, 3>(p, plan, s);
    case 2: return launch_linear_tile<false, false, 2, 4, 2, 2, 3>(p, plan, s);
    case 3: return launch_linear_tile<false, false, 2, 2, 2, 4, 4>(p, plan, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_skinny_bf16(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<false, false>(swapped, rt, p, plan, s);
}

}  // namespace moed
