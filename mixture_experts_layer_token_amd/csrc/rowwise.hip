// Row-wise operators beside the grouped products: 8-bit quantization of rows (with the SwiGLU gate on the
// way), the SwiGLU gate and its gradient, and the gradient of the weighted combine.  All of them touch every
// byte once and are bound by memory: 16-byte accesses where rows allow them, one pass over the data.
#include <float.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "rowwise.hpp"

namespace moe {
namespace {

// ------------------------------------------------------------------ 8 elements at a time

typedef __attribute__((__vector_size__(8 * sizeof(unsigned short)))) unsigned short u16x8;

// elements j .. j+7 of a row of n (j < n); V: the row starts on 16 bytes and n is a multiple of 8
template <bool BF16, bool V>
__device__ __forceinline__ void load8(const void* row, int j, int n, float (&v)[8]) {
  if constexpr (BF16) {
    const unsigned short* p = (const unsigned short*)row + j;
    if constexpr (V) {
      const u16x8 u = *(const u16x8*)p;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = j + i < n ? bf16_to_f32(p[i]) : 0.f;
    }
  } else {
    const float* p = (const float*)row + j;
    if constexpr (V) {
      const f32x4 a = ((const f32x4*)p)[0], b = ((const f32x4*)p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = j + i < n ? p[i] : 0.f;
    }
  }
}

template <bool BF16, bool V>
__device__ __forceinline__ void store8(void* row, int j, int n, const float (&v)[8]) {
  if constexpr (BF16) {
    unsigned short* p = (unsigned short*)row + j;
    if constexpr (V) {
      u16x8 u;
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = f32_to_bf16_rne(v[i]);
      *(u16x8*)p = u;
    } else {
      for (int i = 0; i < 8; ++i)
        if (j + i < n) p[i] = f32_to_bf16_rne(v[i]);
    }
  } else {
    float* p = (float*)row + j;
    if constexpr (V) {
      ((f32x4*)p)[0] = f32x4{v[0], v[1], v[2], v[3]};
      ((f32x4*)p)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      for (int i = 0; i < 8; ++i)
        if (j + i < n) p[i] = v[i];
    }
  }
}

__device__ __forceinline__ int row_limit(int rows, const int32_t* n_rows) {
  return n_rows ? min(rows, max(*n_rows, 0)) : rows;
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= FLT_MAX; }

// ------------------------------------------------------------------ 8-bit quantization

// SiLU(g) u with the accurate exponential: the result is rounded to one of 255 integers, and a coarser
// value next to a half would come out as the other one
__device__ __forceinline__ float gate_exact(float g, float u) { return g / (1.f + expf(-g)) * u; }

// q = the integer nearest to 127 v / max, halves to even.  v and max are scaled by 2^e, which puts max into
// [1, 2) (so that neither the product nor the reciprocal leaves the fp32 range; an element this pushes into
// the denormals is 0 anyway).  The quotient by reciprocal is off by less than 2^-15.4 (three roundings of 2^-24 each, at
// values up to 127): only within 2^-15 of a half is it taken again, in 64 bits, where 127 v is exact and the quotient is off
// by 2^-45 -- closer to a half than that without meeting it no two fp32 numbers' ratio comes.
__device__ __forceinline__ int quantize(float v, int e, float top, float inv) {
  const float x = 127.f * ldexpf(v, e);
  const float t = x * inv;
  float q = rintf(t);
  if (fabsf(fabsf(t - q) - 0.5f) < 0x1p-15f)
    q = (float)rint(127.0 * (double)ldexpf(v, e) / (double)top);
  return (int)q;
}

// One row per 64 * WPR lanes (WPR = 1: a wave; 4: the workgroup).  The row's values stay in registers
// between the maximum and the rounding when it fits CH chunks of 8 per lane; else (CH = 0) they are read
// (and gated) a second time.
template <bool BF16, bool GATE, bool V, int WPR, int CH>
__global__ __launch_bounds__(256) void quant_kernel(const void* __restrict__ x, int row0, int rows, int K,
                                                    const int32_t* __restrict__ n_rows, int8_t* __restrict__ q,
                                                    float* __restrict__ scale) {
  constexpr int LPR = 64 * WPR, C = CH > 0 ? CH : 1;
  __shared__ float s_max[4];
  __shared__ int s_bad[4];
  const int lane = threadIdx.x % LPR;
  const int r = row0 + blockIdx.x * (4 / WPR) + threadIdx.x / LPR;
  if (r >= row_limit(rows, n_rows)) return;  // uniform over the lanes of a row (WPR = 4: over the workgroup)
  const char* xr = (const char*)x + (size_t)r * K * (GATE ? 2 : 1) * (BF16 ? 2 : 4);
  const char* xu = xr + (size_t)K * (BF16 ? 2 : 4);
  auto value = [&](int j, float (&v)[8]) {
    load8<BF16, V>(xr, j, K, v);
    if constexpr (GATE) {
      float u[8];
      load8<BF16, V>(xu, j, K, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = gate_exact(v[i], u[i]);
    }
  };
  float keep[C][8];
  float top = 0.f;
  int bad = 0;
  auto scan = [&](const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(v[i]));
      bad |= !finite(v[i]);
    }
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * LPR + lane) * 8;
      if (j < K) {
        value(j, keep[c]);
        scan(keep[c]);
      }
    }
  } else {
    for (int j = lane * 8; j < K; j += LPR * 8) {
      value(j, keep[0]);
      scan(keep[0]);
    }
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  bad = __ballot(bad) != 0;
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x / 64;
    if ((threadIdx.x & 63) == 0) s_max[wave] = top, s_bad[wave] = bad;
    __syncthreads();
    top = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
  }
  if (lane == 0) scale[r] = bad ? __uint_as_float(0x7FC00000u) : top / 127.f;
  const bool zero = bad || top == 0.f;
  const int e = zero ? 0 : -ilogbf(top);
  const float tops = ldexpf(top, e), inv = 1.f / tops;
  int8_t* qr = q + (size_t)r * K;
  auto emit = [&](int j, const float (&v)[8]) {
    int8_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = zero ? 0 : (int8_t)quantize(v[i], e, tops, inv);
    if constexpr (V) {
      *(u32x2*)(qr + j) = __builtin_bit_cast(u32x2, o);
    } else {
      for (int i = 0; i < 8; ++i)
        if (j + i < K) qr[j + i] = o[i];
    }
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = (c * LPR + lane) * 8;
      if (j < K) emit(j, keep[c]);
    }
  } else {
    for (int j = lane * 8; j < K; j += LPR * 8) {
      value(j, keep[0]);
      emit(j, keep[0]);
    }
  }
}

template <bool BF16, bool GATE, bool V>
void quant_some(const void* x, int row0, int count, int rows, int K, const int32_t* n_rows, int8_t* q, float* scale,
                hipStream_t s) {
  const dim3 one((count + 3) / 4), all(count), b(256);
  if (K <= 512)
    hipLaunchKernelGGL((quant_kernel<BF16, GATE, V, 1, 1>), one, b, 0, s, x, row0, rows, K, n_rows, q, scale);
  else if (K <= 2048)
    hipLaunchKernelGGL((quant_kernel<BF16, GATE, V, 4, 1>), all, b, 0, s, x, row0, rows, K, n_rows, q, scale);
  else if (K <= 4096)
    hipLaunchKernelGGL((quant_kernel<BF16, GATE, V, 4, 2>), all, b, 0, s, x, row0, rows, K, n_rows, q, scale);
  else if (K <= 16384)
    hipLaunchKernelGGL((quant_kernel<BF16, GATE, V, 4, 8>), all, b, 0, s, x, row0, rows, K, n_rows, q, scale);
  else
    hipLaunchKernelGGL((quant_kernel<BF16, GATE, V, 4, 0>), all, b, 0, s, x, row0, rows, K, n_rows, q, scale);
}

// (a launch holds 2^32 threads, the rows of all experts' weights may be more than 2^24)
template <bool BF16, bool GATE, bool V>
void quant_any(const void* x, int rows, int K, const int32_t* n_rows, int8_t* q, float* scale, hipStream_t s) {
  constexpr int kRows = 1 << 23;
  for (int r = 0; r < rows; r += std::min(kRows, rows - r))
    quant_some<BF16, GATE, V>(x, r, std::min(kRows, rows - r), rows, K, n_rows, q, scale, s);
}

// ------------------------------------------------------------------ SwiGLU gate

// h = SiLU(g) u, or with dh: dg = dh u s (1 + g (1 - s)), du = dh g s, s = 1 / (1 + e^-g), and h if asked
// for.  A workgroup is bx x by lanes (bx a power of two), 8 columns per lane.
template <bool BF16, bool V, bool GRAD, bool H>
__global__ __launch_bounds__(256) void swiglu_kernel(const void* __restrict__ gu, const void* __restrict__ dh,
                                                     int rows, int I, const int32_t* __restrict__ n_rows,
                                                     void* __restrict__ dgu, void* __restrict__ h, int log_bx) {
  constexpr size_t B = BF16 ? 2 : 4;
  const int j = ((int)blockIdx.x * (1 << log_bx) + (threadIdx.x & ((1 << log_bx) - 1))) * 8;
  if (j >= I) return;
  const int by = 256 >> log_bx, limit = row_limit(rows, n_rows);
  for (long long r = (long long)blockIdx.y * by + (threadIdx.x >> log_bx); r < limit; r += (long long)gridDim.y * by) {
    const char* gr = (const char*)gu + (size_t)r * 2 * I * B;
    float g[8], u[8], d[8], o[8];
    load8<BF16, V>(gr, j, I, g);
    load8<BF16, V>(gr + (size_t)I * B, j, I, u);
    if constexpr (GRAD) load8<BF16, V>((const char*)dh + (size_t)r * I * B, j, I, d);
    float sg[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = 1.f / (1.f + expf(-g[i]));
    if constexpr (H) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = g[i] * sg[i] * u[i];
      store8<BF16, V>((char*)h + (size_t)r * I * B, j, I, o);
    }
    if constexpr (GRAD) {
      char* dr = (char*)dgu + (size_t)r * 2 * I * B;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = d[i] * u[i] * sg[i] * (1.f + g[i] * (1.f - sg[i]));
      store8<BF16, V>(dr, j, I, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = d[i] * g[i] * sg[i];
      store8<BF16, V>(dr + (size_t)I * B, j, I, o);
    }
  }
}

template <bool BF16, bool V>
void swiglu_any(const void* gu, const void* dh, int rows, int I, const int32_t* n_rows, void* dgu, void* h,
                hipStream_t s) {
  const int chunks = (I + 7) / 8;
  int log_bx = 0;
  while (log_bx < 8 && (1 << log_bx) < chunks) ++log_bx;
  const int by = 256 >> log_bx;
  const dim3 grid((chunks + (1 << log_bx) - 1) >> log_bx, (unsigned)std::min(65535LL, ((long long)rows + by - 1) / by));
  if (!dh)
    hipLaunchKernelGGL((swiglu_kernel<BF16, V, false, true>), grid, dim3(256), 0, s, gu, dh, rows, I, n_rows, dgu, h,
                       log_bx);
  else if (h)
    hipLaunchKernelGGL((swiglu_kernel<BF16, V, true, true>), grid, dim3(256), 0, s, gu, dh, rows, I, n_rows, dgu, h,
                       log_bx);
  else
    hipLaunchKernelGGL((swiglu_kernel<BF16, V, true, false>), grid, dim3(256), 0, s, gu, dh, rows, I, n_rows, dgu, h,
                       log_bx);
}

// ------------------------------------------------------------------ gradient of the combine

// One workgroup per token: its row of dout is read once, its k rows of y_perm once; every lane writes the k
// products of its columns and keeps k partial dot products, which are summed over the workgroup in a fixed
// order.  The gates' softmax gradient needs all k of them and follows in the same workgroup.
template <bool OB, bool YB, bool V, int K>
__global__ __launch_bounds__(1024) void combine_grad_kernel(const void* __restrict__ dout, const float* __restrict__ y,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ inv, int T, int H,
                                                           void* __restrict__ dy, float* __restrict__ dw,
                                                           const int32_t* __restrict__ ids, int E,
                                                           float* __restrict__ dlogits) {
  __shared__ float part[16][K], total[K];
  const int t = blockIdx.x;
  int rows[K];
  float gate[K], dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int p = __builtin_amdgcn_readfirstlane(inv[(size_t)t * K + j]);
    rows[j] = (unsigned)p < (unsigned)(T * K) ? p : -1;
    gate[j] = w[(size_t)t * K + j];
    dot[j] = 0.f;
  }
  const char* dr = (const char*)dout + (size_t)t * H * (OB ? 2 : 4);
  // the loads of up to 8 of the rows are issued together: one after the other, a row's load behind the last row's
  // products, the latencies of a small batch add up (16 tokens, top-8: 10 us)
  constexpr int G = K < 8 ? K : 8;
  for (int c = threadIdx.x * 8; c < H; c += blockDim.x * 8) {
    float d[8];
    load8<OB, V>(dr, c, H, d);
#pragma unroll
    for (int j0 = 0; j0 < K; j0 += G) {
      float v[G][8];
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (j0 + g < K) load8<false, V>(y + (size_t)max(rows[(j0 + g) % K], 0) * H, c, H, v[g]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int j = (j0 + g) % K;
        if (j0 + g >= K || rows[j] < 0) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[j] = fmaf(d[i], v[g][i], dot[j]);
          o[i] = gate[j] * d[i];
        }
        store8<YB, V>((char*)dy + (size_t)rows[j] * H * (YB ? 2 : 4), c, H, o);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int off = 32; off; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64][j] = dot[j];
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float v = 0.f;
    for (int i = 0; i < (int)blockDim.x / 64; ++i) v += part[i][threadIdx.x];
    total[threadIdx.x] = v;
    dw[(size_t)t * K + threadIdx.x] = v;
  }
  if (!dlogits) return;
  __syncthreads();
  float mean = 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (rows[j] >= 0) mean = fmaf(gate[j], total[j], mean);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (rows[j] >= 0 && ids[(size_t)t * K + j] == e) v += gate[j] * (total[j] - mean);
    dlogits[(size_t)t * E + e] = v;
  }
}

template <bool OB, bool YB, bool V, int... Ks>
void combine_grad_any(int k, unsigned T, int threads, const void* dout, const float* y, const float* w,
                      const int32_t* inv, int H, void* dy, float* dw, const int32_t* ids, int E, float* dlogits,
                      hipStream_t s, std::integer_sequence<int, Ks...>) {
  auto go = [&](auto kk) {
    constexpr int K = decltype(kk)::value;
    hipLaunchKernelGGL((combine_grad_kernel<OB, YB, V, K>), dim3(T), dim3(threads), 0, s, dout, y, w, inv, (int)T, H,
                       dy, dw, ids, E, dlogits);
  };
  ((k == Ks + 1 ? go(std::integral_constant<int, Ks + 1>{}) : void()), ...);
}

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace

int launch_quant_rows(const void* x, int xdt, int rows, int K, int act, const int32_t* n_rows, int8_t* q,
                      float* scale, hipStream_t s) {
  const bool v = K % 8 == 0 && al16(x) && (uintptr_t)q % 8 == 0, bf = xdt == MOE_BF16, gate = act == MOE_ACT_SWIGLU;
  auto go = [&](auto b, auto g) {
    if (v)
      quant_any<decltype(b)::value, decltype(g)::value, true>(x, rows, K, n_rows, q, scale, s);
    else
      quant_any<decltype(b)::value, decltype(g)::value, false>(x, rows, K, n_rows, q, scale, s);
  };
  if (bf)
    gate ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  else
    gate ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  MOE_CHECK_LAUNCH("moe_quant_rows launch");
  return MOE_OK;
}

int launch_swiglu(const void* gu, const void* dh, int dt, int rows, int I, const int32_t* n_rows, void* dgu, void* h,
                  hipStream_t s) {
  const bool v = I % 8 == 0 && al16(gu) && al16(dh) && al16(dgu) && al16(h);
  if (dt == MOE_BF16)
    v ? swiglu_any<true, true>(gu, dh, rows, I, n_rows, dgu, h, s)
      : swiglu_any<true, false>(gu, dh, rows, I, n_rows, dgu, h, s);
  else
    v ? swiglu_any<false, true>(gu, dh, rows, I, n_rows, dgu, h, s)
      : swiglu_any<false, false>(gu, dh, rows, I, n_rows, dgu, h, s);
  MOE_CHECK_LAUNCH("moe_swiglu launch");
  return MOE_OK;
}

int launch_combine_grad(const void* dout, int odt, const float* y, const float* w, const int32_t* inv, int T, int k,
                        int H, void* dy, int ydt, float* dw, const int32_t* ids, int E, float* dlogits,
                        hipStream_t s) {
  const bool v = H % 8 == 0 && al16(dout) && al16(y) && al16(dy);
  // fewer tokens than compute units: more lanes for each, so that a row takes one pass (16 tokens, top-8, H = 7168:
  // 10.7 -> 9.9 us)
  int threads = T < 256 ? 1024 : 512;
  while (threads > 64 && threads * 8 > H) threads >>= 1;
  while (threads < 1024 && threads * 8 < H && T < 256) threads <<= 1;
  if ((long long)T * threads > 0xFFFFFFFFLL) return fail(MOE_ERR_UNSUPPORTED, "moe_combine_grad: T=%d in one launch", T);
  auto go = [&](auto ob, auto yb) {
    constexpr bool OB = decltype(ob)::value, YB = decltype(yb)::value;
    if (v)
      combine_grad_any<OB, YB, true>(k, (unsigned)T, threads, dout, y, w, inv, H, dy, dw, ids, E, dlogits, s,
                                     std::make_integer_sequence<int, 16>{});
    else
      combine_grad_any<OB, YB, false>(k, (unsigned)T, threads, dout, y, w, inv, H, dy, dw, ids, E, dlogits, s,
                                      std::make_integer_sequence<int, 16>{});
  };
  if (odt == MOE_BF16)
    ydt == MOE_BF16 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  else
    ydt == MOE_BF16 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  MOE_CHECK_LAUNCH("moe_combine_grad launch");
  return MOE_OK;
}

}  // namespace moe
