// Products grouped by expert over plain weights: the plain tile kernel, for every type, size and stride.
//
// C[i][j] = sum_c A[i][c] B[j][c], with (i, j, c) = (row, output feature, input feature) forward,
// (row, input feature, output feature) for the rows' gradient, (output feature, input feature, row) for the
// weights' gradient.  A workgroup computes a 64 x 64 tile, 4 x 4 results per thread, over slices of 16 of c
// staged in LDS as fp32 (int32 for 8-bit operands).
#include "grouped.hpp"

namespace moe {
namespace {

constexpr int kS = 64, kC = 16;

template <int TYPE>
struct Elem;
template <>
struct Elem<kBf16> {
  typedef unsigned short T;
  typedef float Acc;
  static __device__ __forceinline__ float get(unsigned short v) { return bf16_to_f32(v); }
};
template <>
struct Elem<kF32> {
  typedef float T;
  typedef float Acc;
  static __device__ __forceinline__ float get(float v) { return v; }
};
template <>
struct Elem<kI8> {
  typedef signed char T;
  typedef int Acc;
  static __device__ __forceinline__ int get(signed char v) { return v; }
};

template <int OP, int TYPE>
__global__ __launch_bounds__(256) void simple_kernel(GroupArgs a) {
  typedef Elem<TYPE> El;
  typedef typename El::T T;
  typedef typename El::Acc Acc;
  __shared__ Acc sa[kC][kS + 4], sb[kC][kS + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int ncol = ((OP == kOpY ? a.N : a.K) + kS - 1) / kS;
  const int it0 = blockIdx.x / ncol;  // row tile
  const int j0 = (blockIdx.x - it0 * ncol) * kS;
  int e, p0, rows, i0;  // group, its first row of this tile, rows, first output feature (weights' gradient)
  if constexpr (OP == kOpDw) {
    const int it = (a.N + kS - 1) / kS;
    e = it0 / it;
    i0 = (it0 - e * it) * kS;
    const int2 r = group_range(a.offsets, e, a.rows);
    p0 = r.x, rows = r.y;
  } else {
    const GroupScan sc = scan_groups(a.offsets, a.E, a.rows, kS);
    if (it0 >= sc.total) return;
    const GroupSpan g = sc.find(a.offsets, a.E, a.rows, kS, it0);
    e = g.e, p0 = g.p0 + (it0 - g.first) * kS, rows = min(kS, g.n - (it0 - g.first) * kS), i0 = 0;
  }
  const int ni = OP == kOpDw ? a.N - i0 : rows;            // results below and right of these do not exist
  const int nj = (OP == kOpY ? a.N : a.K) - j0;
  const int nc = OP == kOpY ? a.K : OP == kOpDx ? a.N : rows;
  const T* x = (const T*)a.x;
  const T* w = (const T*)a.w + (size_t)e * a.w_stride;
  const T* y = (const T*)a.y;
  Acc acc[4][4] = {};
  for (int c0 = 0; c0 < nc; c0 += kC) {
    // neighbouring threads take neighbouring elements of memory
    for (int t = threadIdx.x; t < kS * kC; t += 256) {
      const int ic = OP == kOpDw ? t % kS : t / kC, ca = OP == kOpDw ? t / kS : t % kC;
      T v = 0;
      if (ic < ni && c0 + ca < nc) {
        if constexpr (OP == kOpY) {
          const int r = x_row(a, p0 + ic);
          if (r >= 0) v = x[(size_t)r * a.ldx + c0 + ca];
        } else if constexpr (OP == kOpDx) {
          v = y[(size_t)(p0 + ic) * a.ldy + c0 + ca];
        } else {
          v = y[(size_t)(p0 + c0 + ca) * a.ldy + i0 + ic];
        }
      }
      sa[ca][ic] = El::get(v);
      const int jc = OP == kOpY ? t / kC : t % kS, cb = OP == kOpY ? t % kC : t / kS;
      T u = 0;
      if (jc < nj && c0 + cb < nc) {
        if constexpr (OP == kOpY) {
          u = w[(size_t)(j0 + jc) * a.ldw + c0 + cb];
        } else if constexpr (OP == kOpDx) {
          u = w[(size_t)(c0 + cb) * a.ldw + j0 + jc];
        } else {
          const int r = x_row(a, p0 + c0 + cb);
          if (r >= 0) u = x[(size_t)r * a.ldx + j0 + jc];
        }
      }
      sb[cb][jc] = El::get(u);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      Acc va[4], vb[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) va[q] = sa[c][ty * 4 + q], vb[q] = sb[c][tx * 4 + q];
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] += va[p] * vb[q];
    }
    __syncthreads();
  }
  for (int p = 0; p < 4; ++p) {
    const int i = ty * 4 + p;
    if (i >= ni) continue;
    float rs = 1.f;
    if constexpr (TYPE == kI8) {
      const int r = x_row(a, p0 + i);
      rs = r >= 0 ? a.x_scale[r] : 0.f;
    }
    for (int q = 0; q < 4; ++q) {
      const int j = tx * 4 + q;
      if (j >= nj) continue;
      float v = (float)acc[p][q];
      if constexpr (TYPE == kI8) v = v * rs * a.w_scale[(size_t)e * a.N + j0 + j];
      if constexpr (OP == kOpY)
        store_out((void*)a.y, (size_t)(p0 + i) * a.ldy + j0 + j, v, a.out_bf16);
      else if constexpr (OP == kOpDx)
        store_out((void*)a.x, (size_t)(p0 + i) * a.ldx + j0 + j, v, a.out_bf16);
      else
        store_out((void*)a.w, (size_t)e * a.w_stride + (size_t)(i0 + i) * a.ldw + j0 + j, v, a.out_bf16);
    }
  }
}

}  // namespace

size_t grouped_workspace(int, int, int, int, int) { return 0; }

int launch_grouped(const GroupArgs& a, int op, int type, void*, hipStream_t s) {
  // rows of the operands on 16-byte boundaries
  const int eb = type == kI8 ? 1 : type == kBf16 ? 2 : 4;
  auto al = [&](const void* p, long long ld) { return (uintptr_t)p % 16 == 0 && ld * eb % 16 == 0; };
  const bool ax = op == kOpDx || (al(a.x, a.ldx) && a.K * eb % 16 == 0);
  const bool aw = op == kOpDw || (al(a.w, a.ldw) && a.w_stride * eb % 16 == 0 && a.K * eb % 16 == 0);
  const bool ay = op == kOpY || (al(a.y, a.ldy) && a.N * eb % 16 == 0);
  if (type != kF32 && ax && aw && ay && tile_spans_fit(a, op, eb)) {
    const int wi = 8;
    return op == kOpY ? launch_tile_y(a, type, wi, s) : op == kOpDx ? launch_tile_dx(a, wi, s) : launch_tile_dw(a, wi, s);
  }
  const int nj = op == kOpY ? a.N : a.K;
  const long long ty = op == kOpDw ? (long long)a.E * ((a.N + kS - 1) / kS) : group_tiles_max(a.rows, a.E, kS);
  if (ty == 0) return MOE_OK;
  const long long nb = ty * ((nj + kS - 1) / kS);
  if (nb > kMaxThreads / 256) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gemm: %lld tiles in one launch", nb);
  const dim3 grid((unsigned)nb);
  if (type == kI8)
    hipLaunchKernelGGL((simple_kernel<kOpY, kI8>), grid, dim3(256), 0, s, a);
  else if (type == kBf16) {
    if (op == kOpY) hipLaunchKernelGGL((simple_kernel<kOpY, kBf16>), grid, dim3(256), 0, s, a);
    if (op == kOpDx) hipLaunchKernelGGL((simple_kernel<kOpDx, kBf16>), grid, dim3(256), 0, s, a);
    if (op == kOpDw) hipLaunchKernelGGL((simple_kernel<kOpDw, kBf16>), grid, dim3(256), 0, s, a);
  } else {
    if (op == kOpY) hipLaunchKernelGGL((simple_kernel<kOpY, kF32>), grid, dim3(256), 0, s, a);
    if (op == kOpDx) hipLaunchKernelGGL((simple_kernel<kOpDx, kF32>), grid, dim3(256), 0, s, a);
    if (op == kOpDw) hipLaunchKernelGGL((simple_kernel<kOpDw, kF32>), grid, dim3(256), 0, s, a);
  }
  MOE_CHECK_LAUNCH("moe_grouped_gemm launch");
  return MOE_OK;
}

}  // namespace moe
