// The global norm of many gradients, and clipping: norm = sqrt(sum of g^2 over all tensors), out = g min(1, max / norm).
// Bound by memory: the gradients are read for the sum, and read again and written for the result.
//
// The table of tensors travels as a kernel argument (nothing is copied to the device, so a call can be captured), kTensors to
// a launch.  Tensors are cut into chunks; a workgroup of the first kernel adds up the squares of every
// G-th chunk in 64 bits (they cost less than the bytes, the sum is as good as exact, and no square overflows) and leaves one
// partial sum; every workgroup of the second adds those up in the same order, so all of them scale by the same number and
// results are bitwise reproducible.  A small list is one workgroup's, in one launch.
//
// Measured: 2^30 bf16 elements in 3 tensors 370 + 815 us (6.4 GB at 5.4 TB/s); 131,072 fp32 elements in 5 tensors 3.5 + 5.0 us.
#include <algorithm>

#include "ffn_common.hpp"
#include "norm.hpp"
#include "operand.hpp"

namespace moe {
namespace {

constexpr int kTensors = 140, kThreads = 256;
constexpr int kStep = kThreads * 8;      // elements of one pass of a workgroup
constexpr int kUnroll = 4;               // passes whose loads are in flight together
constexpr int kBlocks = 2048;            // 8 to a compute unit
constexpr int kMaxChunk = kStep * 16;

struct TensorTable {
  int n, chunks;
  int chunk;                  // elements
  int end[kTensors];          // chunks of the tensors up to this one
  long long numel[kTensors];  // complemented for bf16
  const void* src[kTensors];
  void* dst[kTensors];        // null: not written
};
static_assert(sizeof(TensorTable) + 32 <= 4096, "kernel arguments");

struct Chunk {
  int t, len;       // tensor, elements
  bool bf16;
  long long first;  // its first element
};
__device__ __forceinline__ Chunk find_chunk(const TensorTable& tab, int c) {
  int lo = 0, hi = tab.n - 1;  // the first tensor with end > c
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (tab.end[mid] > c) hi = mid;
    else lo = mid + 1;
  }
  const long long first = (long long)(c - (lo ? tab.end[lo - 1] : 0)) * tab.chunk, n = tab.numel[lo];
  return Chunk{lo, (int)min((long long)tab.chunk, (n < 0 ? ~n : n) - first), n < 0, first};
}

// Elements i .. i+7 of a chunk, at any element-aligned address.
template <bool BF16>
struct Eight {
  u32x4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(gptr p, int i) {
    v[0] = load_any(p + (size_t)i * (BF16 ? 2 : 4));
    if constexpr (!BF16) v[1] = load_any(p + (size_t)i * 4 + 16);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (BF16) return __uint_as_float(e % 2 ? v[0][e / 2] & 0xFFFF0000u : v[0][e / 2] << 16);
    return __uint_as_float(v[e / 4][e % 4]);
  }
};
template <bool BF16>
__device__ __forceinline__ float element(gptr p, int i) {
  if constexpr (BF16) return bf16_to_f32(((const __attribute__((address_space(1))) unsigned short*)p)[i]);
  return ((const __attribute__((address_space(1))) float*)p)[i];
}
// PAST: without keeping the lines in the caches
template <bool BF16, bool PAST>
__device__ __forceinline__ void store_eight(char* p, int i, const float (&v)[8]) {
  typedef u32x4 __attribute__((aligned(1))) any4;
  typedef __attribute__((address_space(1))) any4* anyp;
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 b2;
  const anyp o = (anyp)((__attribute__((address_space(1))) char*)p + (size_t)i * (BF16 ? 2 : 4));
  auto put = [&](anyp to, u32x4 w) {
    if constexpr (PAST) __builtin_nontemporal_store((any4)w, to);
    else *to = w;
  };
  if constexpr (BF16) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __builtin_bit_cast(unsigned, b2{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]});
    put(o, w);
  } else {
    put(o, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    put(o + 1, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
  }
}
// f(i, eight) for the groups of 8 elements that thread `tid` of STEP / 8 has of a chunk, kUnroll passes' loads together, then g(i)
// for the elements behind the last whole group
template <bool BF16, int STEP, typename F, typename G>
__device__ __forceinline__ void walk(gptr p, int len, int tid, F&& f, G&& g) {
  int i = tid * 8;
  for (; i + (kUnroll - 1) * STEP + 8 <= len; i += kUnroll * STEP) {
    Eight<BF16> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u].load(p, i + u * STEP);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) f(i + u * STEP, x[u]);
  }
  for (; i + 8 <= len; i += STEP) {
    Eight<BF16> x;
    x.load(p, i);
    f(i, x);
  }
  for (; i < len; ++i) g(i);  // (at most one thread, at most 7 elements: the chunk's end)
}

// squares of a chunk, onto v
template <bool BF16, int STEP>
__device__ __forceinline__ void add_squares(gptr p, int len, int tid, double (&v)[4]) {
  walk<BF16, STEP>(p, len, tid, [&](int, const Eight<BF16>& x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double g = x.get(e);
      v[e % 4] = fma(g, g, v[e % 4]);
    }
  }, [&](int i) {
    const double g = element<BF16>(p, i);
    v[0] = fma(g, g, v[0]);
  });
}
// The factor of a norm n: `scale`, then `post`.  A factor that fp32 holds with fewer bits is applied in two: gradients near the end
// of the fp32 range have a norm past it.  A norm that is not finite in 64 bits is one of a NaN or an infinity, and scales nothing.
// Factor and products are rounded to fp32, 2^-24 of the value each, where a factor in 64 bits would cost the store loop two conversions
// per element; bf16 results are rounded by 2^-8.
struct Factor {
  float scale, post;
  bool one;
};
__device__ __forceinline__ Factor factor_of(double n, float max_norm) {
  const double f = n > (double)max_norm && n <= 1.7976931348623157e308 ? (double)max_norm / n : 1.0;
  return Factor{(float)(f < 0x1p-100 ? f * 0x1p80 : f), f < 0x1p-100 ? 0x1p-80f : 1.f, f == 1.0};
}
template <bool BF16, int STEP, bool PAST>
__device__ __forceinline__ void scale_chunk(gptr p, char* o, int len, int tid, Factor f) {
  walk<BF16, STEP>(p, len, tid, [&](int i, const Eight<BF16>& x) {
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = x.get(e) * f.scale * f.post;
    store_eight<BF16, PAST>(o, i, g);
  }, [&](int i) {
    const float g = element<BF16>(p, i) * f.scale * f.post;
    if constexpr (BF16) ((unsigned short*)o)[i] = f32_to_bf16_rne(g);
    else ((float*)o)[i] = g;
  });
}

// the workgroup's sum, to every thread
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < THREADS / 64; ++i) t += lds[i];
  return t;
}

__global__ __launch_bounds__(kThreads) void square_sums_kernel(TensorTable tab, double* __restrict__ part) {
  __shared__ double lds[kThreads / 64];
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(tab, c);
    const gptr p = (gptr)tab.src[k.t] + k.first * (k.bf16 ? 2 : 4);
    if (k.bf16) add_squares<true, kStep>(p, k.len, threadIdx.x, v);
    else add_squares<false, kStep>(p, k.len, threadIdx.x, v);
  }
  const double sum = block_sum<kThreads>((v[0] + v[1]) + (v[2] + v[3]), lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// parts: of all tables of the call
template <bool PAST>
__global__ __launch_bounds__(kThreads) void clip_kernel(TensorTable tab, const double* __restrict__ part, int parts, int clip,
                                                        float max_norm, float* __restrict__ norm) {
  __shared__ double lds[kThreads / 64];
  double total = 0.0;
  for (int i = threadIdx.x; i < parts; i += 8 * kThreads) {  // (loads together)
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = part[min(i + u * kThreads, parts - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u) total += i + u * kThreads < parts ? v[u] : 0.0;
  }
  const double n = sqrt(block_sum<kThreads>(total, lds));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  if (!clip) return;
  const Factor f = factor_of(n, max_norm);
  // from the end: what the first kernel read last is still in the last-level cache
  for (int c = tab.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const Chunk k = find_chunk(tab, c);
    if (!tab.dst[k.t] || (tab.dst[k.t] == tab.src[k.t] && f.one)) continue;
    const gptr p = (gptr)tab.src[k.t] + k.first * (k.bf16 ? 2 : 4);
    char* o = (char*)tab.dst[k.t] + k.first * (k.bf16 ? 2 : 4);
    if (k.bf16) scale_chunk<true, kStep, PAST>(p, o, k.len, threadIdx.x, f);
    else scale_chunk<false, kStep, PAST>(p, o, k.len, threadIdx.x, f);
  }
}

// Small lists: one workgroup for everything, in one launch, a chunk of a tensor to each of its waves (with its address in the
// table).  While that is one chunk per wave it is no slower than two launches of many workgroups: on the GPU, us, one against two:
// 5 tensors of 1000 elements 3.4 : 5.9, 16 of 2048 6.4 : 6.3, 32 of 2048 10.5 : 6.4; from the host 12.1 : 17.1, 17.6 : 20.2, 25.8 : 27.8.
constexpr int kSmallWaves = 16, kSmallStep = 64 * 8, kSmallChunk = kUnroll * kSmallStep;
constexpr int kSmallChunks = kSmallWaves;
struct SmallTable {
  int chunks, clip;
  float max_norm;
  struct {
    const void* src;
    void* dst;
    int len, bf16;
  } chunk[kSmallChunks];
};
static_assert(sizeof(SmallTable) + 32 <= 4096, "kernel arguments");
__global__ __launch_bounds__(64 * kSmallWaves) void small_clip_kernel(SmallTable tab, float* __restrict__ norm) {
  __shared__ double lds[kSmallWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  const bool mine = wave < tab.chunks;
  const auto& k = tab.chunk[mine ? wave : 0];
  if (mine) {
    if (k.bf16) add_squares<true, kSmallStep>((gptr)k.src, k.len, lane, v);
    else add_squares<false, kSmallStep>((gptr)k.src, k.len, lane, v);
  }
  const double n = sqrt(block_sum<64 * kSmallWaves>((v[0] + v[1]) + (v[2] + v[3]), lds));
  if (threadIdx.x == 0) *norm = (float)n;
  if (!tab.clip || !mine) return;
  const Factor f = factor_of(n, tab.max_norm);
  if (!k.dst || (k.dst == k.src && f.one)) return;
  if (k.bf16) scale_chunk<true, kSmallStep, false>((gptr)k.src, (char*)k.dst, k.len, lane, f);
  else scale_chunk<false, kSmallStep, false>((gptr)k.src, (char*)k.dst, k.len, lane, f);
}

// What the size of the call decides.
struct Plan {
  int chunk;  // elements: long chunks cost less to find, short ones fill the card when there is little to do
  // Results past the caches where the gradients are more than a quarter of the last-level cache: the results would drive out
  // gradients that are still to be read (193 tensors of 345 MB in all 240 -> 204 us), while smaller ones stay for the optimizer.
  bool past;
};
Plan plan_of(const moe_tensor* t, int n) {
  long long total = 0, bytes = 0;
  for (int i = 0; i < n; ++i) total += t[i].numel, bytes += t[i].numel * (t[i].dt == MOE_BF16 ? 2 : 4);
  int chunk = kStep;
  while (chunk < kMaxChunk && total / chunk > 4 * kBlocks) chunk *= 2;
  return Plan{chunk, bytes > (64 << 20)};
}

// Tables of the call: as few as hold it, of about equal length.
int tables_of(int n) { return (n + kTensors - 1) / kTensors; }
// the next table of tensors from `at` on (empty ones left out); at moves past them
void next_table(const moe_tensor* t, int n, const Plan& p, int& at, TensorTable& tab) {
  const int chunk = p.chunk;
  tab.n = tab.chunks = 0, tab.chunk = chunk;
  const int each = (n + std::max(tables_of(n), 1) - 1) / std::max(tables_of(n), 1);
  for (const int end = std::min(n, at + each); at < end; ++at) {
    if (t[at].numel == 0) continue;
    tab.chunks += (int)((t[at].numel + chunk - 1) / chunk);
    tab.end[tab.n] = tab.chunks;
    tab.numel[tab.n] = t[at].dt == MOE_BF16 ? ~(long long)t[at].numel : t[at].numel;
    tab.src[tab.n] = t[at].src;
    tab.dst[tab.n] = t[at].dst;
    ++tab.n;
  }
}
int blocks_of(const TensorTable& tab) { return std::min(tab.chunks, kBlocks); }

}  // namespace

size_t grad_norm_workspace(int n) { return ((size_t)std::max(tables_of(n), 1) * kBlocks * sizeof(double) + 255) / 256 * 256; }

// the table of a small list, or false
bool small_table(const moe_tensor* t, int n, SmallTable& tab) {
  tab = {};
  for (int i = 0; i < n; ++i) {
    const size_t b = t[i].dt == MOE_BF16 ? 2 : 4;
    if (t[i].numel > (long long)kSmallChunks * kSmallChunk) return false;
    for (int at = 0; at < t[i].numel; at += kSmallChunk) {
      if (tab.chunks == kSmallChunks) return false;
      auto& c = tab.chunk[tab.chunks++];
      c.src = (const char*)t[i].src + at * b;
      c.dst = t[i].dst ? (char*)t[i].dst + at * b : nullptr;
      c.len = (int)std::min<long long>(kSmallChunk, t[i].numel - at);
      c.bf16 = t[i].dt == MOE_BF16;
    }
  }
  return true;
}

int launch_grad_norm(const moe_tensor* t, int n, int clip, float max_norm, float* norm, double* part, hipStream_t s) {
  SmallTable small;
  if (small_table(t, n, small)) {
    small.clip = clip, small.max_norm = max_norm;
    hipLaunchKernelGGL(small_clip_kernel, dim3(1), dim3(64 * kSmallWaves), 0, s, small, norm);
    MOE_CHECK_LAUNCH("moe_clip_grad_norm launch");
    return MOE_OK;
  }
  int parts = 0;
  const Plan plan = plan_of(t, n);
  TensorTable tab;
  tab.n = tab.chunks = 0;
  for (int at = 0; at < n;) {
    next_table(t, n, plan, at, tab);
    if (!tab.n) continue;
    hipLaunchKernelGGL(square_sums_kernel, dim3(blocks_of(tab)), dim3(kThreads), 0, s, tab, part + parts);
    parts += blocks_of(tab);
  }
  // The norm comes with the first table that is scaled; the tables go backwards, for what the caches still hold.  (One table: it
  // is there from above.)
  const int tables = std::max(tables_of(n), 1), each = (n + tables - 1) / tables;
  for (int i = tables - 1; i >= 0; --i) {
    int at = i * each;
    if (tables > 1) next_table(t, n, plan, at, tab);
    if (i < tables - 1 && (!clip || !tab.n)) continue;
    const dim3 grid(clip ? std::max(blocks_of(tab), 1) : 1);
    float* to = i == tables - 1 ? norm : nullptr;
    if (plan.past) hipLaunchKernelGGL(clip_kernel<true>, grid, dim3(kThreads), 0, s, tab, part, parts, clip, max_norm, to);
    else hipLaunchKernelGGL(clip_kernel<false>, grid, dim3(kThreads), 0, s, tab, part, parts, clip, max_norm, to);
  }
  MOE_CHECK_LAUNCH("moe_clip_grad_norm launch");
  return MOE_OK;
}

}  // namespace moe
