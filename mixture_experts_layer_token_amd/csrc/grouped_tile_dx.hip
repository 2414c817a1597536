#include "grouped_tile.hpp"

namespace moe {

int launch_tile_dx(const GroupArgs& a, int wi, hipStream_t s) {
  return tile_launch_one<kOpDx, kBf16, 8, 8, false>(a, s);
}

}  // namespace moe
