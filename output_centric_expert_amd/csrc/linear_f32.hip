// Dense products of float32 x and w on the matrix instructions.
#include "linear_skinny.h"
#include "linear_tiled.h"

namespace moed {

TileSize linear_tile_f32(int tile) { return tile_size<true, true>(tile); }

hipError_t launch_linear_f32(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    return launch_tile<true, true>(tile, p, plan, s);
}

hipError_t launch_skinny_f32(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    return launch_skinny<true, true>(swapped, rt, p, plan, s);
}

}  // namespace moed
