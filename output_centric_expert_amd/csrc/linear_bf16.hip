// Dense products of bfloat16 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

namespace {

// us with each of the four, k split as suits it best (float32 out; rows x K -> outputs):
//   8192 x 4096 -> 4096   226  275  373  448     the larger the tile, the fewer bytes through LDS for a product
//   2048 x 4096 -> 4096    84   75   99  115     256 of the second
//   1024 x 1024 -> 4096  32.7 23.2 16.7 20.0     512 of the third, two to a CU
//   1024 x 1024 -> 1024  25.4 20.0 11.3 10.4     the last: the third's with more wavefronts and a fourth buffer
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
