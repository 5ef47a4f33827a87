// Dense products of float32 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

// us with each of the three: 4096 x 4096 -> 4096 579, 876, 1039 (both sides split once for 256 and 128 rows of the other);
// 2000 x 300 -> 1000 28.2, 16.4, 20.8 (two of the second to a CU); 1024 x 1024 -> 1024 32.6, 25.7, 20.9 (one to a CU: half as
// many barriers).
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
