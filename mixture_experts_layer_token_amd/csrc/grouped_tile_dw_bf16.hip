#include "grouped_tile.hpp"

namespace moe {

int launch_tile_dw_bf16(const GroupArgs& a, TileShape t, hipStream_t s) {
  if (a.perm_src) return launch_tile_dw_bf16_gather(a, t, s);
  if (t == kStaged) return tile_launch_one<kOpDw, kBf16, 4, 4, false, true>(a, s);
  if (t == kSmall) return tile_launch_one<kOpDw, kBf16, 4, 4, false, false>(a, s);
  if (t == kDeep) return tile_launch_one<kOpDw, kBf16, 4, 4, false, false, 4>(a, s);
  return tile_launch_one<kOpDw, kBf16, 8, 8, false, false>(a, s);
}

}  // namespace moe
