// Dense products of float32 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

constexpr TileCost kTiles[] = {
    {256, 128, 32, 2.40f, 0.00f},
    {64, 64, 32, 0.78f, 1.05f},
    {64, 64, 64, 1.14f, 0.00f}};

}  // namespace

bool linear_cost_f32(int tile, TileCost* cost)
{
    if (tile >= (int)(sizeof kTiles / sizeof kTiles[0]))
        return false;
    *cost = kTiles[tile];
    return true;
}

hipError_t launch_linear_f32(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    switch (tile) {
    case 0: return launch_linear_tile<true, true, 4, 4, 4, 2, 2, 32>(p, plan, s);
    case 1: return launch_linear_tile<true, true, 2, 2, 2, 2, 2, 32>(p, plan, s);
    case 2: return launch_linear_tile<true, true, 2, 1, 2, 4, 2>(p, plan, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_skinny_f32(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<true, true>(swapped, rt, p, plan, s);
}

}  // namespace moed
