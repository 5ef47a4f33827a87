// Dense products of float32 x and bfloat16 w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

TileSize linear_tile_mixed_x(int tile) { return tile_size<true, false>(tile); }

hipError_t launch_linear_mixed_x(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    return launch_tile<true, false>(tile, p, plan, s);
}

hipError_t launch_skinny_mixed_x(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<true, false>(swapped, rt, p, plan, s);
}

}  // namespace moed
