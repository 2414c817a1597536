// Shared pieces of the products grouped by expert over plain weights (moe_grouped_gemm*).
#pragma once

#include "ffn_common.hpp"

namespace moe {

// kOpGlu: the gated block, y = SiLU(x wg^T) (x wu^T) with w = [wg; wu] of 2N rows; kOpGluDx: the gradient of rows, on to
// the gate's operands
enum GroupOp { kOpY = 0, kOpDx = 1, kOpDw = 2, kOpGlu = 3, kOpGluDx = 4 };

// One call.  x, w, y name the matrices of the forward product: for the gradient of the rows x is dx
// (written) and y is dy, for that of the weights w is dw (written) and y is dy.
struct GroupArgs {
  const void* x;
  const void* w;
  const void* y;
  const int32_t* offsets;
  const int32_t* perm_src;  // or null: x rows are grouped rows
  int k, x_rows;            // x row of grouped row p: perm_src[p] / k, a row of zeros unless in [0, x_rows)
  unsigned k_inv;           // ceil(2^32 / k)
  int rows, E, N, K;
  long long ldx, ldy, ldw, w_stride;  // elements
  const float* x_scale;  // 8-bit operands: scale of every x row and of every w row ([E][N])
  const float* w_scale;
  int out_bf16;
  // weights' gradient: parts each group's rows are cut into; with more than one, w is fp32 partial sums
  // [split][E][N][K]
  int split;
  int each_xcd;  // tile kernel: every group's tiles are shared out over the XCDs (else a range of all tiles to each)
  // gated block: rows [g | u], contiguous.  kOpGlu: written with y unless null; kOpGluDx: read, and dgu written, and h = SiLU(g) u
  // again unless null (x is not: there is no dh in memory)
  void* gu;
  void* dgu;
  void* h;
};

// Rows of expert e, clamped so that no offsets, however wrong, lead outside [0, rows).
__device__ __forceinline__ int2 group_range(const int32_t* __restrict__ offsets, int e, int rows) {
  const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], 0), rows);
  return make_int2(lo, max(hi - lo, 0));
}

// s / k for the flat index of a pair, s < x_rows * k <= 2^28: the product with ceil(2^32 / k) is off by less than 2^-4 <= 1 / k
// there.  (Of larger s, which names no row, only "at least x_rows" is needed, and the product keeps that.)
__device__ __forceinline__ int div_k(const GroupArgs& a, int s) {
  return a.k == 1 ? s : (int)__umulhi((unsigned)s, a.k_inv);
}
// x row that an entry of perm_src names, or -1 for none
__device__ __forceinline__ int named_row(const GroupArgs& a, int s) {
  const int r = div_k(a, s);
  return s >= 0 && r < a.x_rows ? r : -1;
}
// x row of grouped row p (p < rows), or -1
__device__ __forceinline__ int x_row(const GroupArgs& a, int p) { return a.perm_src ? named_row(a, a.perm_src[p]) : p; }

// Most row tiles of mr rows that groups which do not overlap can have (the bound of the launch).
inline long long group_tiles_max(int rows, int E, int mr) {
  return (long long)rows / mr + (rows < E ? rows : E);
}

// Tiles of a grouped product, shared out in `parts` (the XCDs, or 1: everything in one list).  A group of n rows has
// ceil(n / mr) * ncol tiles, and part x takes a contiguous share of every group's, so that groups of unequal cost weigh
// on all parts alike; the shares rotate from group to group.  A part's list is in group order.  Every wave scans the groups on its own (lane l takes groups [l * per, (l + 1) *
// per)), so no LDS and no barrier is needed; totals and found tiles are uniform.
__host__ __device__ __forceinline__ int2 part_range(int n, int e, int x, int parts) {  // {first, count} of the n tiles of group e
  const int p = (x + e) % parts;
  const int lo = (int)((long long)n * p / parts), hi = (int)((long long)n * (p + 1) / parts);
  int2 r;
  r.x = lo, r.y = hi - lo;
  return r;
}
struct GroupSpan {
  int e, p0, n, tile;  // expert, its first grouped row, its rows, and which of its tiles
};
struct GroupScan {
  int acc, incl, total;  // this lane's tiles are [acc, incl) of the part's list; its length
  int mr, ncol, x, parts;
  // tile `slot` (< total) of the list
  __device__ __forceinline__ GroupSpan find(const int32_t* __restrict__ offsets, int E, int rows, int slot) const {
    const int per = (E + 63) / 64, lane = threadIdx.x & 63;
    GroupSpan f = {0, 0, 0, 0};
    const bool mine = slot >= acc && slot < incl;
    if (mine) {
      int t = acc;
      for (int e = lane * per; e < min(E, (lane + 1) * per); ++e) {
        const int2 r = group_range(offsets, e, rows);
        const int2 p = part_range((r.y + mr - 1) / mr * ncol, e, x, parts);
        if (slot >= t && slot < t + p.y) f = GroupSpan{e, r.x, r.y, p.x + slot - t};
        t += p.y;
      }
    }
    const unsigned long long b = __ballot(mine);
    const int owner = b ? __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(b)) : 0;
    return GroupSpan{__builtin_amdgcn_readlane(f.e, owner), __builtin_amdgcn_readlane(f.p0, owner),
                     __builtin_amdgcn_readlane(f.n, owner), __builtin_amdgcn_readlane(f.tile, owner)};
  }
};
__device__ __forceinline__ GroupScan scan_groups(const int32_t* __restrict__ offsets, int E, int rows, int mr, int ncol,
                                                 int x, int parts) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  int local = 0;
  for (int e = lane * per; e < min(E, (lane + 1) * per); ++e)
    local += part_range((group_range(offsets, e, rows).y + mr - 1) / mr * ncol, e, x, parts).y;
  int incl = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int t = __shfl_up(incl, off, 64);
    if (lane >= off) incl += t;
  }
  return GroupScan{incl - local, incl, __builtin_amdgcn_readlane(incl, 63), mr, ncol, x, parts};
}

__device__ __forceinline__ void store_out(void* out, size_t i, float v, int bf16) {
  if (bf16)
    ((unsigned short*)out)[i] = f32_to_bf16_rne(v);
  else
    ((float*)out)[i] = v;
}

constexpr long long kMaxThreads = 0xFFFFFFFFLL;  // of one launch

enum GroupType { kBf16 = 0, kF32 = 1, kI8 = 2 };

constexpr long long kMaxSpan = 0xFFFF0000LL;  // bytes a buffer descriptor of the tile kernel may cover
// Whether every descriptor of the kernel covers its operand: rows of a tile, or all of x where it is gathered, within
// 32-bit offsets.
inline bool tile_spans_fit(const GroupArgs& a, int op, int eb) {
  if (op == kOpGluDx) op = kOpDx;
  auto rows = [&](long long n, long long ld) { return (n - 1) * ld * eb + ld * eb <= kMaxSpan && ld * eb < kMaxSpan / 512; };
  const bool x = a.perm_src ? a.x_rows == 0 || rows(a.x_rows, a.ldx) : rows(256, a.ldx);
  if (op == kOpGlu) return x && rows((long long)a.N + 128, a.ldw);  // a tile's gate and up rows lie N rows apart
  return (op == kOpDx || x) && (op == kOpDw || rows(256, a.ldw)) && (op == kOpY || rows(256, a.ldy));
}

// grouped_tile_*.hip: the MFMA tile kernel.  kLarge: 256 x 256 results per workgroup (bf16, int8), kSmall: 128 x 128;
// kDeep: 128 x 128 with four stages in LDS instead of two; these for rows on 16-byte boundaries and spans that fit;
// kStaged: 128 x 128 for any others.
enum TileShape { kLarge, kSmall, kDeep, kStaged };
int launch_tile_y_bf16(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_y_i8(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_dx_bf16(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_dw_bf16(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_dw_bf16_gather(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_f32(const GroupArgs& a, int op, TileShape t, hipStream_t s);
int launch_tile_glu_bf16(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_gludx_bf16(const GroupArgs& a, TileShape t, hipStream_t s);
int launch_tile_glu_f32(const GroupArgs& a, int op, TileShape t, hipStream_t s);
constexpr int kDecodeRows = 64;  // rows of a workgroup there
// grouped_decode.hip: forward for few rows; direct: rows on 16-byte boundaries and spans that fit
int launch_grouped_decode(const GroupArgs& a, int type, bool direct, hipStream_t s);
int launch_glu_decode(const GroupArgs& a, int type, bool direct, hipStream_t s);
// the gradient through the gate for few rows: kGluDxRows rows and kGluDxBytes of columns to a workgroup; K of at least 16 bytes, rows of
// w under 2 GiB, and at most kMaxThreads
constexpr int kGluDxRows = 16, kGluDxBytes = 256, kGluDxThreads = 512;
int launch_gludx_few(const GroupArgs& a, int type, hipStream_t s);
// the kernel that suits the call; ws holds grouped_workspace bytes
int launch_grouped(const GroupArgs& a, int op, int type, void* ws, hipStream_t s);
size_t grouped_workspace(int type, int rows, int N, int K, int E);

}  // namespace moe
