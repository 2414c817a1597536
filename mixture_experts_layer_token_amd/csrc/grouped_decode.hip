// Forward product grouped by expert for few rows: every touched weight is read once and nothing is reused, so
// the kernel is bound by the weights' bytes and, for the smallest calls, by latency.
//
// A workgroup computes 16 output features of up to 64 rows of one expert: many small workgroups (N / 16 per expert)
// keep enough loads in flight where whole tiles would leave compute units idle.  Its waves split the input
// features among them, 128 bytes of every weight row at a time; a lane's 16 bytes of a weight row are an MFMA
// operand as they come from memory (so are those of the rows of x, which come from L2), so nothing passes
// through LDS until the waves' partial sums are added up in a fixed order.  D groups of loads are in flight per wave.
#include "grouped.hpp"
#include "mfma_pipe.hpp"
#include "operand.hpp"

namespace moe {
namespace {

__device__ __forceinline__ f32x4 mma(const bf16x8& b, const bf16x8& a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mma(const i32x4& b, const i32x4& a, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const f32x4& b, const f32x4& a, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(b[e], a[e], c, 0, 0, 0);
  return c;
}

constexpr int kDecodeCols = 16;

// Rows of 16 bytes per lane, at byte c of the row: through a buffer descriptor (DIRECT), whose end turns everything
// outside into zeros, or by ordinary loads at any address.
template <int EB, bool DIRECT>
struct Rows {
  __amdgpu_buffer_rsrc_t desc;
  unsigned voff;
  gptr row;
  int len;  // bytes of the lane's row (0: a row of zeros)
  __device__ __forceinline__ void init(gptr base, unsigned span, long long off, int bytes) {
    len = bytes;
    if constexpr (DIRECT) {
      desc = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)span, 0x00027000);
      voff = (unsigned)off;
    } else {
      row = base + off;
    }
  }
  // whole: every lane's 16 bytes end inside the row, whose length is `total`
  __device__ __forceinline__ u32x4 load(int c, bool whole, int total) const {
    if constexpr (DIRECT)
      return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(desc, c < len ? (int)(voff + c) : (int)kOutside, 0, 0));
    if (total < 16) return load_part<EB>(row + c, len - c);
    // (unconditional, as behind a condition the loads would wait for one another)
    const u32x4 v = load_any(len ? row + min(c, len - 16) : (gptr)g_zero_page);
    return whole ? v : shift_bytes(v, max(c - (len - 16), 0));
  }
};

template <int TYPE, bool DIRECT, int MT>
__device__ __forceinline__ void decode_body(const GroupArgs& a, int e, int p0, int rows, int n0, char* smem) {
  typedef TileT<TYPE> TT;
  typedef typename TT::Frag Frag;
  typedef typename TT::Acc Acc;
  constexpr int EB = TT::EB, D = MT == 1 ? 4 : MT == 2 ? 3 : 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int len = a.K * EB, nj = min(kDecodeCols, a.N - n0);
  Rows<EB, DIRECT> W, X[MT];
  const gptr w = (gptr)a.w + ((size_t)e * a.w_stride + (size_t)n0 * a.ldw) * EB;
  W.init(w, (unsigned)((nj - 1) * a.ldw * EB) + len, (long long)min(lane & 15, nj - 1) * a.ldw * EB, len);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = p0 + min(16 * m + (lane & 15), rows - 1);
    if (a.perm_src) {
      const int xr = x_row(a, r);
      X[m].init((gptr)a.x, a.x_rows > 0 ? (unsigned)((a.x_rows - 1) * a.ldx * EB) + len : 0, (long long)max(xr, 0) * a.ldx * EB, xr >= 0 ? len : 0);
    } else {
      X[m].init((gptr)a.x + (size_t)p0 * a.ldx * EB, (unsigned)((rows - 1) * a.ldx * EB) + len,
                (long long)(r - p0) * a.ldx * EB, len);
    }
  }
  // group g: bytes 128 g .. 128 g + 127 of every row, as two MFMA operands per lane
  struct Group {
    u32x4 w[2], x[2][MT];
  };
  const int c0 = (lane >> 4) * 16;
  auto load = [&](Group& G, int g) {
    const bool whole = g * 128 + 128 <= len;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = g * 128 + h * 64 + c0;
      G.w[h] = W.load(c, whole, len);
#pragma unroll
      for (int m = 0; m < MT; ++m) G.x[h][m] = X[m].load(c, whole, len);
    }
  };
  Acc acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = Acc{};
  const int ng = (len + 127) / 128;
  Group ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], wave + d * nw);  // (past the end: zeros)
  for (int g = wave; g < ng; g += D * nw) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m] = mma(__builtin_bit_cast(Frag, ring[d].w[h]), __builtin_bit_cast(Frag, ring[d].x[h][m]), acc[m]);
      load(ring[d], g + (d + D) * nw);
    }
  }
  // the waves' sums, in wave order
  Acc* part = (Acc*)smem;
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = acc[m];
  __syncthreads();
  for (int t = threadIdx.x; t < MT * 64; t += blockDim.x) {
    const int m = t >> 6, i = 16 * m + (t & 15), jj = ((t & 63) >> 4) * 4;
    if (i >= rows) continue;
    Acc v = part[t];
    for (int o = 1; o < nw; ++o) v += part[o * MT * 64 + t];
    float rs = 1.f;
    if constexpr (TYPE == kI8) {
      const int xr = x_row(a, p0 + i);
      rs = xr >= 0 ? a.x_scale[xr] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (jj + r >= nj) break;
      const int j = n0 + jj + r;
      float f = (float)v[r];
      if constexpr (TYPE == kI8) f = f * rs * a.w_scale[(size_t)e * a.N + j];
      store_out((void*)a.y, (size_t)(p0 + i) * a.ldy + j, f, a.out_bf16);
    }
  }
}

template <int TYPE, bool DIRECT>
__global__ __launch_bounds__(512) void grouped_decode_kernel(GroupArgs a) {
  __shared__ __align__(16) char smem[8 * 4 * 64 * 16];
  const int ncol = (a.N + kDecodeCols - 1) / kDecodeCols;
  const GroupScan sc = scan_groups(a.offsets, a.E, a.rows, kDecodeRows, ncol, 0, 1);
  if ((int)blockIdx.x >= sc.total) return;
  const GroupSpan g = sc.find(a.offsets, a.E, a.rows, blockIdx.x);
  const int tile = g.tile / ncol, col = g.tile - tile * ncol;
  const int r0 = tile * kDecodeRows, rows = min(kDecodeRows, g.n - r0), mt = (rows + 15) / 16;
  static_for<kDecodeRows / 16>([&](auto mc) {
    constexpr int MT = mc + 1;
    if (mt == MT) decode_body<TYPE, DIRECT, MT>(a, g.e, g.p0 + r0, rows, col * kDecodeCols, smem);
  });
}

template <int TYPE>
int decode_launch(const GroupArgs& a, bool direct, hipStream_t s) {
  const long long nb = group_tiles_max(a.rows, a.E, kDecodeRows) * ((a.N + kDecodeCols - 1) / kDecodeCols);
  if (nb == 0) return MOE_OK;
  // 8 waves where there are few workgroups: each then has half the groups to walk
  const int threads = nb < 1024 ? 512 : 256;
  if (nb > kMaxThreads / threads) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gemm: %lld tiles in one launch", nb);
  if (direct)
    hipLaunchKernelGGL((grouped_decode_kernel<TYPE, true>), dim3((unsigned)nb), dim3(threads), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_decode_kernel<TYPE, false>), dim3((unsigned)nb), dim3(threads), 0, s, a);
  MOE_CHECK_LAUNCH("moe_grouped_gemm launch");
  return MOE_OK;
}

}  // namespace

int launch_grouped_decode(const GroupArgs& a, int type, bool direct, hipStream_t s) {
  return type == kI8 ? decode_launch<kI8>(a, direct, s)
                     : type == kF32 ? decode_launch<kF32>(a, direct, s) : decode_launch<kBf16>(a, direct, s);
}

}  // namespace moe
