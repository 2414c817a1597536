// The global norm of many gradients, and clipping: norm = sqrt(sum of g^2 over all tensors), out = g min(1, max / norm).
// Bound by memory: the gradients are read for the sum, and read again and written for the result.
//
// The table of tensors travels as a kernel argument (nothing is copied to the device, so a call can be captured), kTensors to
// a launch.  Tensors are cut into chunks of kChunk elements; a workgroup of the first kernel adds up the squares of every
// G-th chunk in 64 bits (they cost less than the bytes, the sum is as good as exact, and no square overflows) and leaves one
// partial sum; every workgroup of the second adds those up in the same order, so all of them scale by the same number and
// results are bitwise reproducible.
#include <algorithm>

#include "ffn_common.hpp"
#include "norm.hpp"
#include "operand.hpp"

namespace moe {
namespace {

constexpr int kTensors = 96, kChunk = 8192, kThreads = 256;
constexpr int kBlocks = 2048;  // 8 to a compute unit

struct TensorTable {
  int n, chunks;
  int end[kTensors];  // chunks of the tensors up to this one
  int bf16[kTensors];
  long long numel[kTensors];
  const void* src[kTensors];
  void* dst[kTensors];  // null: not written
};
static_assert(sizeof(TensorTable) <= 3500, "kernel argument");

struct Chunk {
  int t, len;       // tensor, elements
  long long first;  // its first element
};
__device__ __forceinline__ Chunk find_chunk(const TensorTable& tab, int c) {
  int lo = 0, hi = tab.n - 1;  // the first tensor with end > c
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (tab.end[mid] > c) hi = mid;
    else lo = mid + 1;
  }
  const long long first = (long long)(c - (lo ? tab.end[lo - 1] : 0)) * kChunk;
  return Chunk{lo, (int)min((long long)kChunk, tab.numel[lo] - first), first};
}

template <bool BF16>
__device__ __forceinline__ float element(const void* p, long long i) {
  if constexpr (BF16) return bf16_to_f32(((const unsigned short*)p)[i]);
  return ((const float*)p)[i];
}

// the workgroup's sum, to every thread
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < kThreads / 64; ++i) t += lds[i];
  return t;
}

__global__ __launch_bounds__(kThreads) void square_sums_kernel(TensorTable tab, double* __restrict__ part) {
  __shared__ double lds[kThreads / 64];
  double v = 0.0;
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(tab, c);
    auto add = [&](auto bf) {
      constexpr bool BF = decltype(bf)::value;
      for (int i = threadIdx.x; i < k.len; i += kThreads) {
        const double g = element<BF>(tab.src[k.t], k.first + i);
        v = fma(g, g, v);
      }
    };
    if (tab.bf16[k.t]) add(std::true_type{});
    else add(std::false_type{});
  }
  v = block_sum(v, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// parts: of all tables of the call.  A norm that is not finite scales nothing.
__global__ __launch_bounds__(kThreads) void clip_kernel(TensorTable tab, const double* __restrict__ part, int parts, int clip,
                                                        float max_norm, float* __restrict__ norm) {
  __shared__ double lds[kThreads / 64];
  double total = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) total += part[i];
  const double n = sqrt(block_sum(total, lds));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  if (!clip) return;
  const double f = n > (double)max_norm && n <= 1.7976931348623157e308 ? (double)max_norm / n : 1.0;
  // (a factor that fp32 holds with fewer bits is applied in two: gradients near the end of the fp32 range have a norm past it)
  const float post = f < 0x1p-100 ? 0x1p-80f : 1.f;
  const float scale = (float)(f < 0x1p-100 ? f * 0x1p80 : f);
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const Chunk k = find_chunk(tab, c);
    const void* src = tab.src[k.t];
    void* dst = tab.dst[k.t];
    if (!dst || (dst == src && f == 1.0)) continue;
    auto apply = [&](auto bf) {
      constexpr bool BF = decltype(bf)::value;
      for (int i = threadIdx.x; i < k.len; i += kThreads) {
        const float g = element<BF>(src, k.first + i) * scale * post;
        if constexpr (BF) ((unsigned short*)dst)[k.first + i] = f32_to_bf16_rne(g);
        else ((float*)dst)[k.first + i] = g;
      }
    };
    if (tab.bf16[k.t]) apply(std::true_type{});
    else apply(std::false_type{});
  }
}

long long chunks_of(const moe_tensor& t) { return (t.numel + kChunk - 1) / kChunk; }

// the next table's worth of tensors from `at` on (empty ones left out); at moves past them
TensorTable next_table(const moe_tensor* t, int n, int& at) {
  TensorTable tab = {};
  for (; at < n && tab.n < kTensors; ++at) {
    if (t[at].numel == 0) continue;
    const long long c = chunks_of(t[at]);
    if (tab.chunks + c > 0x7FFFFFFFLL) break;  // (one tensor alone always fits: numel is limited)
    tab.chunks += (int)c;
    tab.end[tab.n] = tab.chunks;
    tab.bf16[tab.n] = t[at].dt == MOE_BF16;
    tab.numel[tab.n] = t[at].numel;
    tab.src[tab.n] = t[at].src;
    tab.dst[tab.n] = t[at].dst;
    ++tab.n;
  }
  return tab;
}
int blocks_of(const TensorTable& tab) { return std::min(tab.chunks, kBlocks); }

}  // namespace

size_t grad_norm_workspace(const moe_tensor* t, int n) {
  long long parts = 0;
  for (int at = 0; at < n;) parts += blocks_of(next_table(t, n, at));
  return ((size_t)parts * sizeof(double) + 255) / 256 * 256 + 256;
}

int launch_grad_norm(const moe_tensor* t, int n, int clip, float max_norm, float* norm, double* part, hipStream_t s) {
  int parts = 0;
  for (int at = 0; at < n;) {
    const TensorTable tab = next_table(t, n, at);
    if (!tab.n) continue;
    hipLaunchKernelGGL(square_sums_kernel, dim3(blocks_of(tab)), dim3(kThreads), 0, s, tab, part + parts);
    parts += blocks_of(tab);
  }
  bool first = true;
  for (int at = 0; first || (clip && at < n);) {
    const TensorTable tab = next_table(t, n, at);
    if (first || tab.n)
      hipLaunchKernelGGL(clip_kernel, dim3(clip ? std::max(blocks_of(tab), 1) : 1), dim3(kThreads), 0, s, tab, part, parts, clip,
                         max_norm, first ? norm : nullptr);
    first = false;
  }
  MOE_CHECK_LAUNCH("moe_clip_grad_norm launch");
  return MOE_OK;
}

}  // namespace moe
