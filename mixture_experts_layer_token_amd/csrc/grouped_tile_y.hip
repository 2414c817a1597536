#include "grouped_tile.hpp"

namespace moe {

int launch_tile_y(const GroupArgs& a, int type, int wi, hipStream_t s) {
  if (type == kI8) return tile_launch_one<kOpY, kI8, 8, 8, false>(a, s);
  return tile_launch_one<kOpY, kBf16, 8, 8, false>(a, s);
}

}  // namespace moe
