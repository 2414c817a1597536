#include "grouped_tile.hpp"

namespace moe {

int launch_tile_dw(const GroupArgs& a, int wi, hipStream_t s) {
  if (a.perm_src) return tile_launch_one<kOpDw, kBf16, 8, 8, true>(a, s);
  return tile_launch_one<kOpDw, kBf16, 8, 8, false>(a, s);
}

}  // namespace moe
