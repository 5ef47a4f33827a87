// Dense products of bfloat16 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

TileSize linear_tile_bf16(int tile) { return tile_size<false, false>(tile); }

hipError_t launch_linear_bf16(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    return launch_tile<false, false>(tile, p, plan, s);
}

hipError_t launch_skinny_bf16(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<false, false>(swapped, rt, p, plan, s);
}

}  // namespace moed
