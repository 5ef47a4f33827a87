// Dense products of bfloat16 x and float32 w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

TileSize linear_tile_mixed_w(int tile) { return tile_size<false, true>(tile); }

hipError_t launch_linear_mixed_w(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    return launch_tile<false, true>(tile, p, plan, s);
}

hipError_t launch_skinny_mixed_w(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<false, true>(swapped, rt, p, plan, s);
}

}  // namespace moed
