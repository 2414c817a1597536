// Products grouped by expert over plain weights: choice of the kernel, and the sum of split weight gradients.
#include <algorithm>
#include <cmath>

#include "grouped.hpp"

namespace moe {
namespace {

// How many parts the rows of each group are cut into for a weight gradient: its tiles of 128 x 128 alone would leave
// compute units idle.  A part keeps at least 256 rows.
//  - bf16, direct loads: one workgroup to a compute unit (four stages in LDS), 0.5 us per stage of 64 rows and 8 to begin and
//    end; the parts' sum takes 5 us and its bytes at 4.5 TB/s.  The count that takes the least, measured: 640 x 640 over
//    8 groups of 1024 rows (200 tiles) whole 15 us, in 2 parts 32; over 4 groups 13 and 22; 1024 x 1024 over 8192 rows (64
//    tiles) whole 57, in 4 parts 29, in 8 38; 1280 x 1280 (100 tiles) whole 58, in 2 parts 41, in 5 48.
//  - bf16 through registers (staged): two workgroups to a unit, waiting on memory: all that fit.  1023 x 1023 over 8192 rows
//    whole 229 us, in 4 parts 74, in 8 58; 2047 x 1535 (192 tiles) whole 229, in 2 parts 143.
//  - fp32 is bound by the matrix cores, so two parts on one unit take twice as long as one and the units with one wait: of the
//    counts that keep the busiest unit's share of the rows smallest, the least.  128 x 2880 over 4096 rows, 23 tiles: in 16
//    parts each 48 us, in 11 41; 384 x 7168, 168 tiles: whole 248 us, in 3 parts 187.
int dw_split(int type, bool staged, int rows, int N, int K, int E) {
  const long long tiles = (long long)E * ((N + 127) / 128) * ((K + 127) / 128);
  if (tiles >= 256) return 1;
  const long long by_rows = (long long)rows / E / 256, by_tiles = 512 / tiles;
  const int most = (int)std::min({by_rows, by_tiles, 32LL});
  if (type != kF32 && staged) return std::max(most, 1);
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= most || s == 1; s++) {
    const double turns = (double)((tiles * s + 255) / 256), stages = (double)rows / E / 64 / s;  // of the busiest unit
    const double sum = s > 1 ? 5 + 8.0 * s * E * N * K / 4.5e6 : 0;
    const double cost = type == kF32 ? turns / s : turns * (0.5 * stages + 8) + sum;
    if (cost < least) best = s, least = cost;
  }
  return best;
}

// dw = sum over the parts, in order: one thread per element (the partial sums are at most 32 MiB: 512 tiles)
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ part, int split, int N, int K,
                                                        long long n, void* __restrict__ dw, long long ldw,
                                                        long long w_stride, int bf16) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int s = 0; s < split; ++s) v += part[s * n + i];
  const long long row = i / K, e = row / N;
  store_out(dw, (size_t)(e * w_stride + (row - e * N) * ldw + (i - row * K)), v, bf16);
}

// Whether a forward product runs on the kernel that spreads every expert's features over N / 16 workgroups.  It wins while
// the tile kernel would have too few tiles of 128 x 128 to fill the card, but reads all rows of x again for every 16 features,
// so fewer tiles are allowed the more rows there are.  Measured, this kernel against the tile kernel (us, weights not in a
// cache; "rows" per touched expert):
//   bf16   5760 x 2880, 1 expert (45 tiles): 1 row 15 : 23, 32 rows 24 : 25, 48 rows 30 : 26
//          2880 x 2880, 1 row: 8 experts (184 tiles) 31 : 45, 16 experts (368) 56 : 53;  4 experts (92): 4 rows 24 : 24, 16 28 : 25
//          4096 x 7168, 8 experts (256): 1 row 85 : 115;  4096 x 14336, 8 experts (256): 4 rows 173 : 163, 32 rows 364 : 168
//          4096 x 4096, 1 expert (32): 64 rows 25 : 34
//   int8   5760 x 2880, 45 tiles: 32 rows 15 : 19, 64 rows 21.5 : 20.8;  4096 x 14336, 256 tiles: 1 row 81 : 81, 32 rows 184 : 83
//   rows through registers (staged), bf16   5759 x 2881 (45): 32 rows 86 : 86, 48 rows 102 : 89;  2879 x 2881, 4 experts (92):
//          1 row 71 : 83, 8 rows 91 : 84;  4095 x 4097, 8 experts (256): 1 row 159 : 119, 32 rows 386 : 124
//   fp32 (bound by the matrix cores, of which its many workgroups use more at a time)   4096 x 14336, 8 experts (256):
//          8 rows 387 : 466, 16 rows 490 : 466;  14336 x 4096, 1 expert (112): 48 rows 138 : 145, 64 rows 166 : 146
// The gated block counts its 2N rows of weights and fits the same rule.  bf16   2 x 2880 x 2880, 1 expert (45): 16 rows 12 : 19, 64 rows
//          20 : 20;  4 experts of 2 x 1440 x 2880 (92): 8 rows 20 : 20, 32 rows 27 : 21;  8 experts of 2 x 2048 x 4096 (256): 1 row 54 : 65, 16
//          rows 59 : 65, 32 rows 79 : 65;  64 experts of 2 x 512 x 1024 (512): 1 row 34 : 28;  staged 2 x 1441 x 2881 (23): 48 rows 46 : 68, 64
//          68 : 67;  fp32   2 x 2880 x 2880 (45): 64 rows 49 : 98;  8 experts of 2 x 2048 x 4096 (256): 16 rows 126 : 149, 32 rows 164 : 150
bool few_rows_kernel(int type, bool staged, int rows, int N, int E) {
  const long long tiles = (long long)std::min(rows, E) * ((N + 127) / 128), mean = ((long long)rows + E - 1) / E;
  if (mean > kDecodeRows) return false;
  if (type == kF32) return tiles * (mean + 16) <= 7500;
  return tiles * (mean + (staged ? 16 : 4)) <= 2200;
}

// Whether the gradient through the gate runs on the kernel of small workgroups that split its sum.  How many those and the tile
// kernel's tiles of 128 x 128 are is an estimate, as row counts are known on average only; of E experts, as many count as rows that
// choose at random touch.  Measured at some 800 sizes, this kernel against the tile kernel (us; weights not in a cache; rows x H x I,
// workgroups):
//   bf16   while they fit the card at once: then a compute unit's reading bounds each of them.  40 x 4096 x 4096 (96) 21 : 28, 400 x 4096 x
//          768 (150) 21 : 35, 200 x 4096 x 2048 (208) 20 : 34, 100 x 4096 x 4096 (224) 21 : 35;  200 x 2880 x 2880 (299) 36 : 28.  Weights of
//          many strips (kGluDxBytes wide) bound both kernels, the tile kernel a little less: 64 rows to 8 experts of 2880 x 2880 (184 strips)
//          32 : 31, to 32 of 2048 x 768 (168) 25 : 23, but 8 to 128 of 2880 x 2880 (179) 25 : 34, as the tiles' shape is that for more
//          experts than have rows.  Sums over fewer than 512 rows of the matrix leave waves without work: 9 rows to 9 experts of 64 x 1696 (82)
//          7.6 : 6.1.  Experts of 64 rows and more make up for it: 1791 x 192 x 160 (224) 8.2 : 10.8
//   rows through registers (staged), whose tiles wait longer for their loads, and longer in more than one round:  40 x 4095 x 4095 (96) 41 :
//          113, 1000 x 4099 x 519 (315) 71 : 124, 400 rows to 16 experts of 4095 x 2047 (528) 96 : 128, 8510 to 46 of 2874 x 33 (555) 58 : 82;  64
//          to 32 of 2880 x 2881 (640, as many tiles) 117 : 143, 64 to 64 of 4095 x 2047 (650) 161 : 268;  400 to 16 of 2880 x 2881 (759,
//          half as many tiles) 112 : 80, 1767 to 45 of 63 x 625 (665) 29 : 14
//   fp32   (bound by the matrix cores, which a tile of few rows keeps as busy as a full one)   40 x 2880 x 2880 (135) 22 : 101, 300 x 4096 x
//          4096 (1216, 96 tiles) 126 : 259, 700 x 2880 x 2880 (1980, 138 tiles) 207 : 182.  Weights of more strips than compute units
//          bound this kernel, and the rounds of tiles the other:  64 rows to 16 experts of 2048 x 4096 (1008, 504 tiles) 102 : 92, of
//          2048 x 4128 (1023, 520 tiles) 99 : 145, 708 to 42 of 1776 x 3656 (3784, 1218 tiles) 315 : 237, 256 to 32 of 2880 x 2880 (1440,
//          736 tiles) 192 : 220.  Short sums:  400 to 8 of 64 x 4096 (1856) 19 : 15, but 40 x 64 x 4096 (192) 5.8 : 11
bool few_rows_gradient(const GroupArgs& a, int type, bool staged) {
  const int eb = type == kF32 ? 4 : 2;
  const long long width = ((long long)a.K * eb + kGluDxBytes - 1) / kGluDxBytes;
  if (a.K * eb < 16 || a.ldw * eb >= 1LL << 31) return false;  // (its loads and addresses)
  if (group_tiles_max(a.rows, a.E, kGluDxRows) * width > kMaxThreads / kGluDxThreads) return false;
  const double touched = a.E == 1 ? 1 : -a.E * std::expm1(a.rows * std::log1p(-1.0 / a.E)), avg = a.rows / touched;
  auto count = [&](int mr) { return a.E == 1 ? std::ceil(avg / mr) : touched * std::max(1.0, avg / mr + 0.5); };
  const double groups = count(kGluDxRows) * width, tiles = count(128) * ((a.K + 127) / 128);
  const double strips = touched * a.K * eb / kGluDxBytes, cus = cu_count();
  if (type == kF32) {
    if (a.N <= 128) return groups <= 3 * cus;
    if (staged || strips <= cus) return groups <= 4.8 * std::max(tiles, cus);
    return groups <= 3 * cus * std::ceil(tiles / (2 * cus));
  }
  if (avg >= 64) return groups <= (staged ? 3 : 1) * cus;
  const double busy = std::min(1.0, a.N / 512.0);
  if (staged) return groups <= 2.25 * busy * std::max(tiles / 2, cus);
  return groups <= busy * cus && (a.rows < a.E || strips <= 0.45 * cus);
}

// The tile shape that takes the least time, from rounds of tiles and stages of 128 bytes (us; fitted to measured calls).
// A 256 x 256 tile has a compute unit to itself: 1.46 per stage of full tiles, 10 to begin and end; 128 x 128 ones go two
// to a compute unit, 0.94 and 7; where they leave units idle anyway, four stages in LDS instead of two hide the loads
// better: 0.5 and 8.  Rows that do not fill a tile save matrix instructions but not loads.  Measured, large against small:
// 8192 rows x 4096 x 4096 210 : 252 us, 2048 rows 93 : 64; 16384 rows over 16 experts of 1024 x 1024 66 : 50; 16384 rows over
// 32 experts of 5760 x 2880 594 : 681, 4096 rows 264 : 302, 2036 rows over 128 experts of 2880 x 2880 473 : 393; weight gradient of 8192 rows, 4096 x
// 4096, 197 : 250.  Small against deep: 1024 rows x 4096 x 4096 48 : 38.
TileShape cheapest_shape(const GroupArgs& a, int op, int eb, double large, double small, double rows) {
  const double c = op == kOpY || op == kOpGlu ? a.K : op == kOpDx || op == kOpGluDx ? a.N : (double)a.rows / a.E;
  const double ns = std::max(1.0, std::ceil(c * eb / 128));
  const double fl = std::max(0.6, rows / 256), fs = std::max(0.6, std::min(1.0, rows / 128));
  const double cus = cu_count();
  const double cost_large = std::ceil(large / cus) * (1.46 * fl * ns + 10);
  const double cost_small = std::ceil(small / (2 * cus)) * (0.94 * fs * ns + 7);
  const double cost_deep = small <= cus ? 0.5 * fs * ns + 8 : 1e30;
  return cost_large <= std::min(cost_small, cost_deep) ? kLarge : cost_deep < cost_small ? kDeep : kSmall;
}

}  // namespace

size_t grouped_workspace(int type, int rows, int N, int K, int E) {
  // (whether operands start on 16 bytes is not known here: the more parts of the two)
  const int s = std::max(dw_split(type, true, rows, N, K, E), dw_split(type, false, rows, N, K, E));
  return s > 1 ? ((size_t)s * E * N * K * 4 + 255) / 256 * 256 : 0;
}

int launch_grouped(const GroupArgs& a0, int op, int type, void* ws, hipStream_t s) {
  GroupArgs a = a0;
  a.split = 1;
  a.each_xcd = 0;
  // direct loads: operand rows on 16-byte boundaries
  const int eb = type == kI8 ? 1 : type == kBf16 ? 2 : 4;
  auto al = [&](const void* p, long long ld) { return (uintptr_t)p % 16 == 0 && ld * eb % 16 == 0; };
  const bool forward = op == kOpY || op == kOpGlu, to_rows = op == kOpDx || op == kOpGluDx;
  const bool ax = to_rows || (al(a.x, a.ldx) && a.K * eb % 16 == 0);
  const bool aw = op == kOpDw || (al(a.w, a.ldw) && a.w_stride * eb % 16 == 0 && a.K * eb % 16 == 0);
  const bool ay = forward || (al(a.y, a.ldy) && a.N * eb % 16 == 0);
  TileShape t = ax && aw && ay && tile_spans_fit(a, op, eb) ? kLarge : kStaged;
  if (forward && few_rows_kernel(type, t == kStaged, a.rows, op == kOpGlu ? 2 * a.N : a.N, a.E))
    return op == kOpGlu ? launch_glu_decode(a, type, t == kLarge, s) : launch_grouped_decode(a, type, t == kLarge, s);
  if (op == kOpDw) {
    const int split = dw_split(type, t == kStaged, a.rows, a.N, a.K, a.E);
    if (split > 1) {
      if (t == kLarge) t = kDeep;
      GroupArgs p = a;
      p.split = split;
      p.w = ws, p.ldw = a.K, p.w_stride = (long long)a.N * a.K, p.out_bf16 = 0;
      const int rc = type == kF32 ? launch_tile_f32(p, op, t, s) : launch_tile_dw_bf16(p, t, s);
      if (rc != MOE_OK) return rc;
      const long long n = (long long)a.E * a.N * a.K;
      hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, (const float*)ws, split,
                         a.N, a.K, n, (void*)a.w, a.ldw, a.w_stride, a.out_bf16);
      MOE_CHECK_LAUNCH("moe_grouped_gemm_dw launch");
      return MOE_OK;
    }
  }
  // tiles of b x b (row counts are known on average only: half a tile more per group)
  const double avg = (double)a.rows / a.E;
  const long long nj = op == kOpGlu ? 2LL * a.N : forward ? a.N : a.K;
  auto tiles = [&](int b) {
    const double ni = op == kOpDw ? (double)((a.N + b - 1) / b) : a.E == 1 ? (double)((a.rows + b - 1) / b) : std::max(1.0, avg / b + 0.5);
    return ni * a.E * ((nj + b - 1) / b);
  };
  if (op == kOpGluDx && few_rows_gradient(a, type, t == kStaged)) return launch_gludx_few(a, type, s);
  // (fp32 has tiles of 128 x 128 only, with two stages, whatever shape is chosen: the order below by the chosen shape's tiles or
  // by its own took the same time to 1%)
  if (t == kLarge) t = cheapest_shape(a, op, eb, tiles(256), tiles(128), op == kOpDw ? 256 : std::min(avg, 256.0));
  // Groups of many tiles are shared out over the XCDs one by one, as they may differ in cost (weight gradients of 8
  // experts with 540 to 1000 rows 1228 -> 906 us); small ones stay on one XCD, whose L2 then holds their rows (16384 rows over 16
  // experts of 1024 x 1024: 50 against 61 us).
  a.each_xcd = tiles(t == kLarge ? 256 : 128) >= 128.0 * a.E;
  if (op == kOpGlu || op == kOpGluDx) {
    if (type == kF32) return launch_tile_glu_f32(a, op, t, s);
    return op == kOpGlu ? launch_tile_glu_bf16(a, t, s) : launch_tile_gludx_bf16(a, t, s);
  }
  if (type == kF32) return launch_tile_f32(a, op, t, s);
  if (type == kI8) return launch_tile_y_i8(a, t, s);
  return op == kOpY ? launch_tile_y_bf16(a, t, s) : op == kOpDx ? launch_tile_dx_bf16(a, t, s) : launch_tile_dw_bf16(a, t, s);
}

}  // namespace moe
