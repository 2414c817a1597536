#include "grouped_tile.hpp"

namespace moe {

int launch_tile_glu_f32(const GroupArgs& a, int op, TileShape t, hipStream_t s) {
  if (op == kOpGlu)
    return t == kStaged ? tile_launch_one<kOpGlu, kF32, 4, 4, false, true>(a, s)
                        : tile_launch_one<kOpGlu, kF32, 4, 4, false, false>(a, s);
  return t == kStaged ? tile_launch_one<kOpGluDx, kF32, 4, 4, false, true>(a, s)
                      : tile_launch_one<kOpGluDx, kF32, 4, 4, false, false>(a, s);
}

}  // namespace moe
