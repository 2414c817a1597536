#include "grouped_tile.hpp"

namespace moe {

int launch_tile_f32(const GroupArgs& a, int op, TileShape t, hipStream_t s) {
  if (op == kOpY)
    return t == kStaged ? tile_launch_one<kOpY, kF32, 4, 4, false, true>(a, s)
                        : tile_launch_one<kOpY, kF32, 4, 4, false, false>(a, s);
  if (op == kOpDx)
    return t == kStaged ? tile_launch_one<kOpDx, kF32, 4, 4, false, true>(a, s)
                        : tile_launch_one<kOpDx, kF32, 4, 4, false, false>(a, s);
  if (t == kStaged)
    return a.perm_src ? tile_launch_one<kOpDw, kF32, 4, 4, true, true>(a, s)
                      : tile_launch_one<kOpDw, kF32, 4, 4, false, true>(a, s);
  return a.perm_src ? tile_launch_one<kOpDw, kF32, 4, 4, true, false>(a, s)
                    : tile_launch_one<kOpDw, kF32, 4, 4, false, false>(a, s);
}

}  // namespace moe
