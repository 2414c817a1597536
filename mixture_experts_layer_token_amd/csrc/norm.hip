// Layer norm and RMS norm of rows, and their gradients.  Bound by memory: every row is read once, held in registers through
// its sums, and written once.
//
//   mean = sum x / H (RMS: 0),  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),  xh = (x - mean) rstd,  y = xh w + b
//   dx = rstd (v - m1 - xh m2) (+ add),  v = w dy,  m1 = sum v / H (RMS: 0),  m2 = sum v xh / H
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// The variance is taken from the deviations (a second pass over registers), not from a difference of squares.  The sums over
// rows stay in registers while a workgroup walks over its rows, one partial sum per workgroup goes to memory, and a second
// kernel adds those up in order: no atomics, results are bitwise reproducible.
//
// Measured, bf16, inputs in no cache: 8192 rows of 7168 forward 52 us (4.6 TB/s), gradient with the residual's 87 + 5 us (5.2 TB/s;
// the parts are 15 MB of it); 517 rows of 2880, gradient, 7.5 + 3.4 us; one row of 7168, forward, 3.0 us.  fp32: 8192 rows of 7168 forward
// 89 us (5.2 TB/s), gradient 173 + 5 us.
#include <algorithm>
#include <type_traits>

#include "ffn_common.hpp"
#include "norm.hpp"
#include "operand.hpp"

namespace moe {
namespace {

// ------------------------------------------------------------------ 8 elements of a row

// as they are in memory
template <bool BF16>
struct Raw {
  u32x4 v[BF16 ? 1 : 2];
};

// Elements j .. j+7 of a row of n, zeros past its end, at any element-aligned address.  Without conditions, behind which
// the loads of a row would wait for one another: a chunk that ends past the row reads the row's last 8 elements, and unpack()
// moves them down.  Rows of less than 8 are read one by one.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* row, int j, int n) {
  constexpr int EB = BF16 ? 2 : 4;
  Raw<BF16> r;
  if (n < 8) {  // (uniform)
    if constexpr (BF16) {
      r.v[0] = load_part<2>((gptr)row + (size_t)j * 2, (n - j) * 2);
    } else {
      r.v[0] = load_part<4>((gptr)row + (size_t)j * 4, (n - j) * 4);
      r.v[1] = load_part<4>((gptr)row + (size_t)j * 4 + 16, (n - j - 4) * 4);
    }
    return r;
  }
  const gptr p = (gptr)row + (size_t)min(j, n - 8) * EB;
  r.v[0] = load_any(p);
  if constexpr (!BF16) r.v[1] = load_any(p + 16);
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& r, int j, int n, float (&v)[8]) {
  const int s = n < 8 ? 0 : max(j - (n - 8), 0);  // elements to move down; 8 and more: zeros
  if constexpr (BF16) {
    u32x4 b = r.v[0];
    if (n % 8) b = shift_bytes(b, min(s, 8) * 2);
    else if (s) b = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(b[i] << 16), v[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.v[i / 4][i % 4]);
    if (n % 8) {
#pragma unroll
      for (int d = 1; d < 8; d *= 2) {
        if (!(s & d)) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i + d < 8 ? v[(i + d) % 8] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s >= 8 ? 0.f : v[i];
  }
}

// two fp32 to bf16, nearest-even (one instruction)
__device__ __forceinline__ unsigned pair_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 b2;
  return __builtin_bit_cast(unsigned, b2{(__bf16)lo, (__bf16)hi});
}
template <bool BF16>
__device__ __forceinline__ void store_chunk(void* row, int j, int n, const float (&v)[8]) {
  typedef u32x4 __attribute__((aligned(1))) any4;
  typedef __attribute__((address_space(1))) any4* anyp;
  if (j + 8 <= n) {
    if constexpr (BF16) {
      *(anyp)((__attribute__((address_space(1))) char*)row + (size_t)j * 2) =
          u32x4{pair_bf16(v[0], v[1]), pair_bf16(v[2], v[3]), pair_bf16(v[4], v[5]), pair_bf16(v[6], v[7])};
    } else {
      const anyp p = (anyp)((__attribute__((address_space(1))) char*)row + (size_t)j * 4);
      p[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
      p[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < n) {
        if constexpr (BF16) ((unsigned short*)row)[j + i] = f32_to_bf16_rne(v[i]);
        else ((float*)row)[j + i] = v[i];
      }
  }
}

// elements j .. j+7 of weight or bias (null: `none`), zeros past the end
__device__ __forceinline__ void load_param(const void* p, int bf16, int j, int n, float none, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j + i < n ? none : 0.f;
  } else if (bf16) {
    unpack<true>(load_raw<true>(p, j, n), j, n, v);
  } else {
    unpack<false>(load_raw<false>(p, j, n), j, n, v);
  }
}

// ------------------------------------------------------------------ sums over a row

// over the wave, in a fixed order; every lane gets it.  (Row shifts and broadcasts cost an instruction each; the butterfly of
// lane permutes goes through LDS.)
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);  // lanes 1, 2, 4 and 8 below, in rows of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // the last lane of a row to the next row (rows 1 and 3)
  v = dpp_add<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
// over the WPR waves of a row; part: WPR floats that no other sum uses until two barriers later
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (WPR == 1) return v;
  const int wave = threadIdx.x / 64 % WPR;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  barrier_keep_loads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) t += part[i];
  return t;
}
// Two such sums at once, in place.  A lane reads one of the 2 WPR floats, and they are added up across lanes: read by every lane they
// take 2 WPR registers, which the gradient does not have (4000 rows of 16384 in bf16 136 -> 84 us, most of it spills); the forward
// pass has them, and is 8% faster that way.
template <int WPR>
__device__ __forceinline__ void row_sums(float& s1, float& s2, float (&part)[2][WPR]) {
  s1 = wave_sum(s1), s2 = wave_sum(s2);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x / 64 % WPR, lane = threadIdx.x & 63;
    if (lane == 0) part[0][wave] = s1, part[1][wave] = s2;
    barrier_keep_loads();
    float v = lane < 2 * WPR ? (&part[0][0])[lane] : 0.f;
    v = dpp_add<0x111, 0xF>(v);  // (the last lane of each WPR ends up with their sum)
    if constexpr (WPR > 2) v = dpp_add<0x112, 0xF>(v);
    if constexpr (WPR > 4) v = dpp_add<0x114, 0xF>(v);
    if constexpr (WPR > 8) v = dpp_add<0x118, 0xF>(v);
    s1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), WPR - 1));
    s2 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 2 * WPR - 1));
  }
}

// ------------------------------------------------------------------ forward

// Finite rows can leave fp32's range: sums of elements from 2^108 on and squares of deviations from 2^54 on may overflow, squares below
// 2^-126 lose bits and then vanish.  The sums of such a row are taken again, of its elements times a power of two, which is exact where
// it counts.  var_eps is the row's variance plus eps; the result is 1 where that is right.
//   Not finite: an element is 2^54 or more.  Times 2^-80 neither sums (2^20 elements below 2^48) nor squares overflow, and squares that
//   vanish are nothing to the row's.  (Rows that hold a NaN or an infinity are taken again too, and stay what they were.)
//   Below 2^-100: no deviation is more than 2^-40.  Times 2^90 the square of the smallest element is 2^-118.  Where the mean is far
//   from that, deviations are zeros, and the variance is as it was.
// In between, lost bits are 2^-149 to a sum of 2^-100 or more.

// How far var_eps is past 2^-100, counted in floats: kOut and more if it is out of range (below it as well)
constexpr unsigned kOut = 0x7F800000u - 0x0D800000u;
__device__ __forceinline__ unsigned past_low(float var_eps) { return __float_as_uint(var_eps) - 0x0D800000u; }
__device__ __forceinline__ float other_scale(float var_eps, float mean) {
  if (past_low(var_eps) < kOut) return 1.f;
  if (!(var_eps < 0x1p-100f)) return 0x1p-80f;
  return fabsf(mean) < 0x1p10f ? 0x1p90f : 1.f;
}

// mean of a row times `scale` and the sum of its squared deviations, read from memory by WPR waves
struct RowSums {
  float mean, sq;
};
template <bool BF16, int WPR>
__device__ __forceinline__ RowSums row_again(const NormArgs& a, long long r, int lane, float scale, float (&part)[2][WPR], int& parity) {
  constexpr int LPR = 64 * WPR, EB = BF16 ? 2 : 4;
  const char* xr = (const char*)a.x + (size_t)r * a.ldx * EB;
  const float inv = 1.f / (float)a.H;
  float v[8], mean = 0.f, sum = 0.f, sq = 0.f;
  if (!a.rms) {
    for (int j = lane * 8; j < a.H; j += LPR * 8) {
      unpack<BF16>(load_raw<BF16>(xr, j, a.H), j, a.H, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i] * scale;
    }
    mean = row_sum<WPR>(sum, part[parity]) * inv, parity ^= 1;
  }
  for (int j = lane * 8; j < a.H; j += LPR * 8) {
    unpack<BF16>(load_raw<BF16>(xr, j, a.H), j, a.H, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = j + i < a.H ? v[i] * scale - mean : 0.f;
      sq = fmaf(d, d, sq);
    }
  }
  sq = row_sum<WPR>(sq, part[parity]);
  parity ^= 1;
  return RowSums{mean, sq};
}
// its results
template <bool BF16, int WPR>
__device__ __forceinline__ void write_again(const NormArgs& a, long long r, int lane, float scale, RowSums s) {
  constexpr int LPR = 64 * WPR, EB = BF16 ? 2 : 4;
  const char* xr = (const char*)a.x + (size_t)r * a.ldx * EB;
  char* yr = (char*)a.y + (size_t)r * a.ldy * EB;
  // 1 / sqrt(variance + eps) of the row times `scale`, and of the row.  (Without deviations eps is all there is, and any factor of
  // theirs will do.)
  const float inv = 1.f / (float)a.H, e = s.sq == 0.f ? 1.f : scale;
  const float scaled = 1.f / sqrtf(fmaf(s.sq, inv, a.eps * e * e)), rstd = scaled * e;
  float v[8], w[8], b[8];
  for (int j = lane * 8; j < a.H; j += LPR * 8) {
    unpack<BF16>(load_raw<BF16>(xr, j, a.H), j, a.H, v);
    load_param(a.weight, a.par_bf16, j, a.H, 1.f, w);
    load_param(a.bias, a.par_bf16, j, a.H, 0.f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] * scale - s.mean) * scaled, w[i], b[i]);
    store_chunk<BF16>(yr, j, a.H, v);
  }
  if (a.stats && lane == 0) a.stats[2 * r] = s.mean / scale, a.stats[2 * r + 1] = rstd;
}

// WPR waves to a row, CH chunks of 8 elements per lane; workgroups walk over the rows, with the next row's loads under
// way while one is worked on (a row's two sums each wait for all of its waves).
template <bool BF16, int WPR, int CH>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void norm_kernel(NormArgs a) {
  constexpr int LPR = 64 * WPR, EB = BF16 ? 2 : 4, RPB = WPR > 4 ? 1 : 4 / WPR;
  static_assert(WPR == 1 || RPB == 1, "a row that is taken again meets no other row's waves at its barriers");
  __shared__ float part[RPB][2][WPR];
  const int lane = threadIdx.x % LPR, team = __builtin_amdgcn_readfirstlane(threadIdx.x / LPR);
  const long long step = (long long)gridDim.x * RPB;
  long long r0 = (long long)blockIdx.x * RPB;
  Raw<BF16> raw[CH];
  auto fetch = [&](long long first) {
    const long long r = first + team;
    if (r >= a.rows) return;  // (uniform over a wave)
    const char* xr = (const char*)a.x + (size_t)r * a.ldx * EB;
#pragma unroll
    for (int c = 0; c < CH; ++c) raw[c] = load_raw<BF16>(xr, (c * LPR + lane) * 8, a.H);
  };
  fetch(r0);
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_param(a.weight, a.par_bf16, (c * LPR + lane) * 8, a.H, 1.f, w[c]);
    load_param(a.bias, a.par_bf16, (c * LPR + lane) * 8, a.H, 0.f, b[c]);
  }
  const float inv = 1.f / (float)a.H;
  int parity = 0;
  unsigned past = 0;
  // (the workgroup's waves stay together for the barriers, whether or not their team has a row)
  for (; r0 < a.rows; r0 += step) {
    // (Which elements exist is found out again for every row: as masks held over the loop it takes more scalar registers than
    // there are, and reading them back costs more: with them, and the rows taken again below, 517 rows of 2880 took 5.2 us, now 4.2,
    // 8192 of 7168 48.6, now 47.)
    int H = a.H;
    asm volatile("" : "+s"(H));
    const int n = H - lane * 8;
    float v[CH][8];
    float mean = 0.f, sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      unpack<BF16>(raw[c], (c * LPR + lane) * 8, H, v[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[c][i];
    }
    fetch(r0 + step);
    if (!a.rms) mean = row_sum<WPR>(sum, part[team][parity]) * inv, parity ^= 1;
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = c * LPR * 8 + i < n ? v[c][i] - mean : 0.f;
        sq = fmaf(v[c][i], v[c][i], sq);
      }
    }
    const float var_eps = fmaf(row_sum<WPR>(sq, part[team][parity]), inv, a.eps), rstd = 1.f / sqrtf(var_eps);
    parity ^= 1;
    const long long r = r0 + team;
    if (r >= a.rows) continue;
    past = max(past, past_low(var_eps));
    char* yr = (char*)a.y + (size_t)r * a.ldy * EB;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i] * rstd, w[c][i], b[c][i]);
      store_chunk<BF16>(yr, (c * LPR + lane) * 8, H, v[c]);
    }
    if (a.stats && lane == 0) a.stats[2 * r] = mean, a.stats[2 * r + 1] = rstd;
  }
  if ((unsigned)__builtin_amdgcn_readfirstlane(past) < kOut) return;  // (the same for all waves of a row)
  // The rare rows out of fp32's range are found by the same sums and written again, behind the loop: inside it, registers kept for them
  // cost 8192 rows of 7168 20%.
#pragma unroll 1
  for (long long r = (long long)blockIdx.x * RPB + team; r < a.rows; r += step) {
    const RowSums s = row_again<BF16, WPR>(a, r, lane, 1.f, part[team], parity);
    const float scale = other_scale(fmaf(s.sq, inv, a.eps), s.mean);
    if (scale != 1.f) write_again<BF16, WPR>(a, r, lane, scale, row_again<BF16, WPR>(a, r, lane, scale, part[team], parity));
  }
}

// Rows too long for the registers: the row is read again for every sum and for the result (from L2, as it was just read).
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
  __shared__ float part[2][16];
  const float inv = 1.f / (float)a.H;
  int parity = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    RowSums s = row_again<BF16, 16>(a, r, threadIdx.x, 1.f, part, parity);
    const float scale = other_scale(fmaf(s.sq, inv, a.eps), s.mean);
    if (scale != 1.f) s = row_again<BF16, 16>(a, r, threadIdx.x, scale, part, parity);
    write_again<BF16, 16>(a, r, threadIdx.x, scale, s);
  }
}

// ------------------------------------------------------------------ gradient

// dx of 8 elements, from the row's sums m1 and m2 (divided by H)
template <bool BF16>
__device__ __forceinline__ void write_dx(const NormArgs& a, long long r, int j, const float (&v)[8], const float (&xh)[8],
                                         float m1, float m2, float rstd) {
  constexpr int EB = BF16 ? 2 : 4;
  const size_t at = (size_t)r * a.H * EB;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = rstd * (v[i] - m1 - xh[i] * m2);
  if (a.add) {
    float d[8];
    unpack<BF16>(load_raw<BF16>((const char*)a.add + at, j, a.H), j, a.H, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += d[i];
  }
  store_chunk<BF16>((char*)a.dx + at, j, a.H, o);
}

// 1024 threads: 16 / WPR teams of WPR waves, a row to a team at a time, the next row's loads under way (one chunk per lane; two
// leave no registers for that: spilled, it takes 136 us instead of 84 for 4000 rows of 16384; two are spilled as it is).
template <bool BF16, int WPR, int CH>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormArgs a) {
  constexpr int LPR = 64 * WPR, EB = BF16 ? 2 : 4, TEAMS = 16 / WPR;
  constexpr bool AHEAD = CH == 1;
  __shared__ __align__(16) float lds[TEAMS > 1 ? 8192 : 1];
  __shared__ float part[TEAMS][2][2][WPR];
  const int lane = threadIdx.x % LPR, team = __builtin_amdgcn_readfirstlane(threadIdx.x / LPR);
  const long long step = (long long)gridDim.x * TEAMS;
  long long r0 = (long long)blockIdx.x * TEAMS;
  struct Row {
    Raw<BF16> x[CH], d[CH], a[AHEAD ? CH : 1];
    float mean, rstd;
  } row;
  auto fetch = [&](long long first) {
    const long long r = first + team;
    if (r >= a.rows) return;  // (uniform over a wave)
    const char* xr = (const char*)a.x + (size_t)r * a.ldx * EB;
    const char* dr = (const char*)a.dy + (size_t)r * a.ldy * EB;
    row.mean = a.stats[2 * r], row.rstd = a.stats[2 * r + 1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      row.x[c] = load_raw<BF16>(xr, (c * LPR + lane) * 8, a.H);
      row.d[c] = load_raw<BF16>(dr, (c * LPR + lane) * 8, a.H);
      if constexpr (AHEAD)
        if (a.add) row.a[c] = load_raw<BF16>((const char*)a.add + (size_t)r * a.H * EB, (c * LPR + lane) * 8, a.H);
    }
  };
  if constexpr (AHEAD) fetch(r0);
  float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_param(a.weight, a.par_bf16, (c * LPR + lane) * 8, a.H, 1.f, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.f;
  }
  const float inv = 1.f / (float)a.H;
  int parity = 0;
  for (; r0 < a.rows; r0 += step) {
    const bool mine = r0 + team < a.rows;
    if constexpr (!AHEAD) fetch(r0);
    float v[CH][8], xh[CH][8], o[8];
    float s1 = 0.f, s2 = 0.f;
    const float mean = a.rms ? 0.f : row.mean, rstd = row.rstd;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * LPR + lane) * 8;
      float d[8];
      unpack<BF16>(row.x[c], j, a.H, xh[c]);
      unpack<BF16>(row.d[c], j, a.H, d);
      if constexpr (AHEAD)
        if (a.add) unpack<BF16>(row.a[c], j, a.H, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[c][i] = (xh[c][i] - mean) * rstd;  // (past the row's end d and w are zeros)
        v[c][i] = d[i] * w[c][i];
        s1 += v[c][i];
        s2 = fmaf(v[c][i], xh[c][i], s2);
        if (mine) dw[c][i] = fmaf(d[i], xh[c][i], dw[c][i]), db[c][i] += d[i];
      }
    }
    if constexpr (AHEAD) fetch(r0 + step);
    row_sums<WPR>(s1, s2, part[team][parity]);
    parity ^= 1;
    const float m1 = a.rms ? 0.f : s1 * inv, m2 = s2 * inv;
    if (!mine) continue;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * LPR + lane) * 8;
      if (j >= a.H) continue;
      char* dr = (char*)a.dx + (size_t)(r0 + team) * a.H * EB;
      if constexpr (!AHEAD)
        if (a.add) unpack<BF16>(load_raw<BF16>((const char*)a.add + (size_t)(r0 + team) * a.H * EB, j, a.H), j, a.H, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = rstd * (v[c][i] - m1 - xh[c][i] * m2);
        o[i] = a.add ? g + o[i] : g;
      }
      store_chunk<BF16>(dr, j, a.H, o);
    }
  }
  if (!a.part) return;
  float* out = a.part + (size_t)blockIdx.x * 2 * a.H;
  if constexpr (TEAMS == 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.dweight) store_chunk<false>(out, (c * LPR + lane) * 8, a.H, dw[c]);
      if (a.dbias) store_chunk<false>(out + a.H, (c * LPR + lane) * 8, a.H, db[c]);
    }
  } else {
    // the teams' sums side by side in LDS (TEAMS * H <= 8192), added up column by column in team order; dw, then db
    auto add_up = [&](const float(&v)[CH][8], float* to) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((c * LPR + lane) * 8 + i < a.H) lds[team * a.H + (c * LPR + lane) * 8 + i] = v[c][i];
      __syncthreads();
      for (int j = threadIdx.x; j < a.H; j += 1024) {
        float t = lds[j];
#pragma unroll
        for (int i = 1; i < TEAMS; ++i) t += lds[i * a.H + j];
        to[j] = t;
      }
    };
    if (a.dweight) add_up(dw, out);
    if (a.dweight && a.dbias) __syncthreads();
    if (a.dbias) add_up(db, out + a.H);
  }
}

// Rows too long for the registers: a kernel for the rows' sums, and one over columns for dx and the sums over rows.
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_grad_sums_kernel(NormArgs a) {
  constexpr int LPR = 1024, EB = BF16 ? 2 : 4;
  __shared__ float part[2][2][16];
  const int lane = threadIdx.x;
  int parity = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const char* xr = (const char*)a.x + (size_t)r * a.ldx * EB;
    const char* dr = (const char*)a.dy + (size_t)r * a.ldy * EB;
    const float mean = a.rms ? 0.f : a.stats[2 * r], rstd = a.stats[2 * r + 1];
    float x[8], d[8], w[8], s1 = 0.f, s2 = 0.f;
    for (int j = lane * 8; j < a.H; j += LPR * 8) {
      unpack<BF16>(load_raw<BF16>(xr, j, a.H), j, a.H, x);
      unpack<BF16>(load_raw<BF16>(dr, j, a.H), j, a.H, d);
      load_param(a.weight, a.par_bf16, j, a.H, 1.f, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = d[i] * w[i];
        s1 += v;
        s2 = fmaf(v, (x[i] - mean) * rstd, s2);
      }
    }
    s1 = row_sum<16>(s1, part[parity][0]);
    s2 = row_sum<16>(s2, part[parity][1]);
    parity ^= 1;
    if (lane == 0) a.sums[2 * r] = a.rms ? 0.f : s1 / (float)a.H, a.sums[2 * r + 1] = s2 / (float)a.H;
  }
}
template <bool BF16>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(NormArgs a) {
  constexpr int EB = BF16 ? 2 : 4;
  const int j = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (j >= a.H) return;
  float w[8], dw[8] = {}, db[8] = {};
  load_param(a.weight, a.par_bf16, j, a.H, 1.f, w);
  for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float mean = a.rms ? 0.f : a.stats[2 * r], rstd = a.stats[2 * r + 1];
    float x[8], d[8], v[8];
    unpack<BF16>(load_raw<BF16>((const char*)a.x + (size_t)r * a.ldx * EB, j, a.H), j, a.H, x);
    unpack<BF16>(load_raw<BF16>((const char*)a.dy + (size_t)r * a.ldy * EB, j, a.H), j, a.H, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = (x[i] - mean) * rstd;
      v[i] = d[i] * w[i];
      dw[i] = fmaf(d[i], x[i], dw[i]), db[i] += d[i];
    }
    write_dx<BF16>(a, r, j, v, x, a.sums[2 * r], a.sums[2 * r + 1], rstd);
  }
  if (!a.part) return;
  float* out = a.part + (size_t)blockIdx.y * 2 * a.H;
  if (a.dweight) store_chunk<false>(out, j, a.H, dw);
  if (a.dbias) store_chunk<false>(out + a.H, j, a.H, db);
}

// dweight and dbias from the parts: a workgroup adds up 64 columns, its 16 waves every 16th part each, then the waves' sums
// in order.
__global__ __launch_bounds__(1024) void norm_parts_kernel(const float* __restrict__ part, int parts, int H, int par_bf16,
                                                          void* __restrict__ dweight, void* __restrict__ dbias) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane, which = blockIdx.y;
  void* out = which ? dbias : dweight;
  if (!out) return;
  float v = 0.f;
  // (the loads of 16 parts together: one after the other they are a chain of latencies)
  for (int p0 = wave; p0 < parts; p0 += 16 * 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = part[((size_t)min(p0 + 16 * i, parts - 1) * 2 + which) * H + min(col, H - 1)];
#pragma unroll
    for (int i = 0; i < 16; ++i) v += p0 + 16 * i < parts ? x[i] : 0.f;
  }
  sum[wave][lane] = v;
  __syncthreads();
  if (wave || col >= H) return;
  for (int i = 1; i < 16; ++i) v += sum[i][lane];
  if (par_bf16) ((unsigned short*)out)[col] = f32_to_bf16_rne(v);
  else ((float*)out)[col] = v;
}

template <bool BF16>
int norm_any(const NormArgs& a, hipStream_t s) {
  auto go = [&](auto wpr, auto ch) {
    constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value, RPB = WPR > 4 ? 1 : 4 / WPR;
    const int threads = WPR > 4 ? 64 * WPR : 256;
    const long long blocks = ((long long)a.rows + RPB - 1) / RPB, slots = (long long)cu_count() * (2048 / threads);
    hipLaunchKernelGGL((norm_kernel<BF16, WPR, CH>), dim3((unsigned)std::min(blocks, slots)), dim3(threads), 0, s, a);
  };
  using std::integral_constant;
#define MOE_NORM(W, C) go(integral_constant<int, W>{}, integral_constant<int, C>{})
  // Few rows: as many lanes as possible to each, one chunk per lane (one row of 7168: 16 waves 2.85 us, 8 waves of two chunks
  // 3.2, 4 of four 4.5).  Many: fewer waves to wait for one another (8192 rows of 7168: 53, 40 and 45 us).
  const bool few = a.rows <= 2 * cu_count();
  if (a.H <= 512) MOE_NORM(1, 1);
  else if (a.H <= 1024 && !few) MOE_NORM(1, 2);
  else if (a.H <= 2048) MOE_NORM(4, 1);
  else if (a.H <= 4096 && !few) MOE_NORM(4, 2);
  else if (a.H <= 8192 && few) MOE_NORM(16, 1);
  else if (a.H <= 8192) MOE_NORM(8, 2);
  else if (a.H <= 16384) MOE_NORM(16, 2);
  else
    hipLaunchKernelGGL(norm_long_kernel<BF16>, dim3((unsigned)std::min((long long)a.rows, 2LL * cu_count())), dim3(1024), 0, s,
                       a);
#undef MOE_NORM
  MOE_CHECK_LAUNCH("moe_norm launch");
  return MOE_OK;
}

template <bool BF16>
int norm_grad_any(const NormArgs& a, hipStream_t s) {
  const int parts = norm_parts(a.rows, a.H);  // (none without rows: the sums over them are zeros)
  auto go = [&](auto wpr, auto ch) {
    constexpr int WPR = decltype(wpr)::value, CH = decltype(ch)::value;
    hipLaunchKernelGGL((norm_grad_kernel<BF16, WPR, CH>), dim3(parts), dim3(1024), 0, s, a);
  };
  using std::integral_constant;
#define MOE_NORM(W, C) go(integral_constant<int, W>{}, integral_constant<int, C>{})
  if (a.rows == 0) {}
  else if (a.H <= 512) MOE_NORM(1, 1);
  else if (a.H <= 1024) MOE_NORM(2, 1);
  else if (a.H <= 2048) MOE_NORM(4, 1);
  else if (a.H <= 4096) MOE_NORM(8, 1);
  else if (a.H <= 8192) MOE_NORM(16, 1);
  else if (a.H <= 16384) MOE_NORM(16, 2);
  else {
    hipLaunchKernelGGL(norm_grad_sums_kernel<BF16>, dim3((unsigned)std::min((long long)a.rows, 2LL * cu_count())), dim3(1024),
                       0, s, a);
    hipLaunchKernelGGL(norm_grad_columns_kernel<BF16>, dim3((a.H + 2047) / 2048, parts), dim3(256), 0, s, a);
  }
#undef MOE_NORM
  MOE_CHECK_LAUNCH("moe_norm_grad launch");
  if (a.dweight || a.dbias) {
    hipLaunchKernelGGL(norm_parts_kernel, dim3((a.H + 63) / 64, a.dbias ? 2 : 1), dim3(1024), 0, s, a.part, parts, a.H,
                       a.par_bf16, a.dweight, a.dbias);
    MOE_CHECK_LAUNCH("moe_norm_grad launch");
  }
  return MOE_OK;
}

}  // namespace

bool norm_long(int H) { return H > 16384; }

// One workgroup of 1024 threads to a compute unit, or fewer where there are fewer rows; long rows: as many parts as give the
// columns' kernel 1024 workgroups.
int norm_parts(int rows, int H) {
  if (rows < 1) return 0;
  if (norm_long(H)) return std::min(rows, std::max(1, 1024 / ((H + 2047) / 2048)));
  int teams = 16;
  while (teams > 1 && 8192 / teams < H) teams /= 2;
  return std::min((rows + teams - 1) / teams, cu_count());
}

int launch_norm(const NormArgs& a, int dt, hipStream_t s) { return dt == MOE_BF16 ? norm_any<true>(a, s) : norm_any<false>(a, s); }

int launch_norm_grad(const NormArgs& a, int dt, hipStream_t s) {
  return dt == MOE_BF16 ? norm_grad_any<true>(a, s) : norm_grad_any<false>(a, s);
}

}  // namespace moe
