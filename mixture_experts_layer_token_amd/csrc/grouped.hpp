// Shared pieces of the products grouped by expert over plain weights (moe_grouped_gemm*).
#pragma once

#include "ffn_common.hpp"

namespace moe {

enum GroupOp { kOpY = 0, kOpDx = 1, kOpDw = 2 };

// One call.  x, w, y name the matrices of the forward product: for the gradient of the rows x is dx
// (written) and y is dy, for that of the weights w is dw (written) and y is dy.
struct GroupArgs {
  const void* x;
  const void* w;
  const void* y;
  const int32_t* offsets;
  const int32_t* perm_src;  // or null: x rows are grouped rows
  int k, x_rows;            // x row of grouped row p: perm_src[p] / k, a row of zeros unless in [0, x_rows)
  int rows, E, N, K;
  long long ldx, ldy, ldw, w_stride;  // elements
  const float* x_scale;  // 8-bit operands: scale of every x row and of every w row ([E][N])
  const float* w_scale;
  int out_bf16;
};

// Rows of expert e, clamped so that no offsets, however wrong, lead outside [0, rows).
__device__ __forceinline__ int2 group_range(const int32_t* __restrict__ offsets, int e, int rows) {
  const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], 0), rows);
  return make_int2(lo, max(hi - lo, 0));
}

// x row of grouped row p (p < rows), or -1 where perm_src names none
__device__ __forceinline__ int x_row(const GroupArgs& a, int p) {
  if (!a.perm_src) return p;
  const int s = a.perm_src[p];
  const int r = s / a.k;
  return s >= 0 && r < a.x_rows ? r : -1;
}

// Row tiles of mr rows over the groups in expert order; at most this many exist for any offsets whose
// groups do not overlap (launch bound: overlapping groups are cut off there).
inline long long group_tiles_max(int rows, int E, int mr) {
  return (long long)rows / mr + (rows < E ? rows : E);
}

// Tile `slot` of the groups' row tiles.  Every wave of the workgroup computes it on its own (lane l
// scans experts [l * per, (l + 1) * per)), so that it needs no LDS and no barrier; the result is uniform.
// Returns e = -1 past the last tile; total = the number of tiles.
struct GroupTile {
  int e, p0, rows, total;
};
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* __restrict__ offsets, int E, int rows, int mr,
                                                     int slot) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
  int local = 0;
  for (int e = e0; e < e1; ++e) local += (group_range(offsets, e, rows).y + mr - 1) / mr;
  int incl = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int t = __shfl_up(incl, off, 64);
    if (lane >= off) incl += t;
  }
  int acc = incl - local, fe = -1, fp = 0, fr = 0;
  const bool mine = slot >= acc && slot < incl;
  if (mine)
    for (int e = e0; e < e1; ++e) {
      const int2 r = group_range(offsets, e, rows);
      const int nt = (r.y + mr - 1) / mr;
      if (fe < 0 && slot < acc + nt) {
        fe = e;
        fp = r.x + (slot - acc) * mr;
        fr = min(mr, r.y - (slot - acc) * mr);
      }
      acc += nt;
    }
  const unsigned long long b = __ballot(mine);
  const int owner = b ? __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(b)) : 0;
  GroupTile t;
  t.e = __builtin_amdgcn_readlane(fe, owner);
  t.p0 = __builtin_amdgcn_readlane(fp, owner);
  t.rows = __builtin_amdgcn_readlane(fr, owner);
  t.total = __builtin_amdgcn_readlane(incl, 63);
  return t;
}

__device__ __forceinline__ void store_out(void* out, size_t i, float v, int bf16) {
  if (bf16)
    ((unsigned short*)out)[i] = f32_to_bf16_rne(v);
  else
    ((float*)out)[i] = v;
}

constexpr long long kMaxThreads = 0xFFFFFFFFLL;  // of one launch

enum GroupType { kBf16 = 0, kF32 = 1, kI8 = 2 };

// the kernel that suits the call; ws holds grouped_workspace bytes
int launch_grouped(const GroupArgs& a, int op, int type, void* ws, hipStream_t s);
size_t grouped_workspace(int type, int rows, int N, int K, int E);

}  // namespace moe
