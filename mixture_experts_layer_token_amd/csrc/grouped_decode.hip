// Forward product grouped by expert, gated block and its gradient, for few rows: every touched weight is read once and nothing is reused, so
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
constexpr int kGluDxWaves = kGluDxThreads / 64;

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

// GLU: the gated block.  kStrips: a strip of 16 gate rows and one of 16 up rows to a workgroup, so that the rows of x are read
// once for both; the sums of the gate's strip pass through LDS first, then those of the up strip.  kHalves: one strip of 8 gate
// rows and 8 up rows, for twice as many workgroups where there are few.
enum GluForm { kNoGlu, kStrips, kHalves };
template <int TYPE, bool DIRECT, int MT, int GLU>
__device__ __forceinline__ void decode_body(const GroupArgs& a, int e, int p0, int rows, int n0, char* smem) {
  typedef TileT<TYPE> TT;
  typedef typename TT::Frag Frag;
  typedef typename TT::Acc Acc;
  constexpr int EB = TT::EB, D = MT == 1 ? 4 : MT == 2 ? 3 : 2, S = GLU == kStrips ? 2 : 1;  // S: strips of 16 weight rows
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int len = a.K * EB, nj = min(GLU == kHalves ? kDecodeCols / 2 : kDecodeCols, a.N - n0);
  Rows<EB, DIRECT> W[S], X[MT];
  const gptr w = (gptr)a.w + ((size_t)e * a.w_stride + (size_t)n0 * a.ldw) * EB;
  if constexpr (GLU == kHalves) {
    const long long r = min(lane & 7, nj - 1) + (lane & 8 ? a.N : 0);
    W[0].init(w, (unsigned)((a.N + nj - 1) * a.ldw * EB) + len, r * a.ldw * EB, len);
  } else {
#pragma unroll
    for (int z = 0; z < S; ++z)
      W[z].init(w + (z ? (size_t)a.N * a.ldw * EB : 0), (unsigned)((nj - 1) * a.ldw * EB) + len,
                (long long)min(lane & 15, nj - 1) * a.ldw * EB, len);
  }
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
    u32x4 w[2][S], x[2][MT];
  };
  const int c0 = (lane >> 4) * 16;
  auto load = [&](Group& G, int g) {
    const bool whole = g * 128 + 128 <= len;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = g * 128 + h * 64 + c0;
#pragma unroll
      for (int z = 0; z < S; ++z) G.w[h][z] = W[z].load(c, whole, len);
#pragma unroll
      for (int m = 0; m < MT; ++m) G.x[h][m] = X[m].load(c, whole, len);
    }
  };
  Acc acc[S][MT];
#pragma unroll
  for (int z = 0; z < S; ++z)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[z][m] = Acc{};
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
#pragma unroll
          for (int z = 0; z < S; ++z)
            acc[z][m] = mma(__builtin_bit_cast(Frag, ring[d].w[h][z]), __builtin_bit_cast(Frag, ring[d].x[h][m]), acc[z][m]);
      load(ring[d], g + (d + D) * nw);
    }
  }
  // the waves' sums, in wave order
  Acc* part = (Acc*)smem;
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = acc[0][m];
  __syncthreads();
  if constexpr (GLU != kNoGlu) {
    const int t = threadIdx.x, m = t >> 6, i = 16 * m + (t & 15), jj = ((t & 63) >> 4) * 4;
    // (MT * 64 <= blockDim.x.  Halves: rows 0..7 of the strip, in lanes 0..31, are the gate's, their up rows 32 lanes on)
    const bool mine = t < MT * 64 && i < rows && (GLU == kStrips || (t & 32) == 0);
    Acc g = Acc{}, u = Acc{};
    if (mine)
      for (int o = 0; o < nw; ++o) g += part[o * MT * 64 + t];
    if constexpr (GLU == kStrips) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < MT; ++q) part[(wave * MT + q) * 64 + lane] = acc[S - 1][q];
      __syncthreads();
    }
    if (!mine) return;
    for (int o = 0; o < nw; ++o) u += part[o * MT * 64 + t + (GLU == kHalves ? 32 : 0)];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (jj + r >= nj) break;
      const size_t p = (size_t)(p0 + i);
      const int j = n0 + jj + r;
      store_out((void*)a.y, p * a.ldy + j, g[r] / (1.f + expf(-g[r])) * u[r], EB == 2);
      if (!a.gu) continue;
      store_out(a.gu, p * 2 * a.N + j, g[r], EB == 2);
      store_out(a.gu, p * 2 * a.N + a.N + j, u[r], EB == 2);
    }
    return;
  }
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

template <int TYPE, bool DIRECT, int GLU>
__global__ __launch_bounds__(GLU ? 256 : 512) void grouped_decode_kernel(GroupArgs a) {
  __shared__ __align__(16) char smem[(GLU ? 4 : 8) * 4 * 64 * 16];
  constexpr int COLS = GLU == kHalves ? kDecodeCols / 2 : kDecodeCols;
  const int ncol = (a.N + COLS - 1) / COLS;
  const GroupScan sc = scan_groups(a.offsets, a.E, a.rows, kDecodeRows, ncol, 0, 1);
  if ((int)blockIdx.x >= sc.total) return;
  const GroupSpan g = sc.find(a.offsets, a.E, a.rows, blockIdx.x);
  const int tile = g.tile / ncol, col = g.tile - tile * ncol;
  const int r0 = tile * kDecodeRows, rows = min(kDecodeRows, g.n - r0), mt = (rows + 15) / 16;
  static_for<kDecodeRows / 16>([&](auto mc) {
    constexpr int MT = mc + 1;
    if (mt == MT) decode_body<TYPE, DIRECT, MT, GLU>(a, g.e, g.p0 + r0, rows, col * COLS, smem);
  });
}

template <int TYPE, int GLU = kNoGlu>
int decode_launch(const GroupArgs& a, bool direct, hipStream_t s) {
  constexpr int COLS = GLU == kHalves ? kDecodeCols / 2 : kDecodeCols;
  const long long nb = group_tiles_max(a.rows, a.E, kDecodeRows) * ((a.N + COLS - 1) / COLS);
  if (nb == 0) return MOE_OK;
  // 8 waves where there are few workgroups: each then has half the groups to walk.  (The gated block has twice the loads per
  // workgroup, and 4 waves are enough: one row to 4 experts of 5760 x 2880 30 us, with 8 waves 38.)
  const int threads = GLU || nb >= 1024 ? 256 : 512;
  if (nb > kMaxThreads / threads) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gemm: %lld tiles in one launch", nb);
  if (direct)
    hipLaunchKernelGGL((grouped_decode_kernel<TYPE, true, GLU>), dim3((unsigned)nb), dim3(threads), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_decode_kernel<TYPE, false, GLU>), dim3((unsigned)nb), dim3(threads), 0, s, a);
  MOE_CHECK_LAUNCH("moe_grouped_gemm launch");
  return MOE_OK;
}

// Halves while strips would leave half of the compute units idle.  Measured, halves against strips (us, weights not in a cache):
// 32 workgroups of strips (512 x 7168, 1 row) 13.5 : 18.9, 90 (1440 x 2880) 9.2 : 11.3, 128 (2048 x 7168) 13.8 : 19.1, 180 (1440 x 2880,
// 2 experts) 12.2 : 11.3, 256 (4096 x 4096) 15.8 : 16.7 and (2048 x 7168, 2 experts) 27.0 : 25.4, 720 (2880 x 2880, 4 experts) 33.5 : 30.6.
template <int TYPE>
int glu_launch(const GroupArgs& a, bool direct, hipStream_t s) {
  const long long strips = group_tiles_max(a.rows, a.E, kDecodeRows) * ((a.N + kDecodeCols - 1) / kDecodeCols);
  return 2 * strips <= cu_count() ? decode_launch<TYPE, kHalves>(a, direct, s) : decode_launch<TYPE, kStrips>(a, direct, s);
}

// The gradient through the gate where the tile kernel would have few tiles, or tiles of few rows: a workgroup computes 16 rows of one
// expert by 256 bytes of columns, and its 8 waves split the long sum over the matrix rows among them, 64 bytes of every row of dy at
// a time.  A lane loads 16 bytes of as many neighbouring matrix rows as an MFMA operand has elements per lane and turns that square
// by itself: element c of them all is the operand whose column is the lane's own c-th.  So a wave reads the matrix in rows of 256
// bytes, nothing passes through LDS but the waves' sums, and a lane ends with neighbouring columns.  Bound by what one compute unit
// can read (65 GB/s) where workgroups are few, else by the matrix's bytes: 2 rows to each of 32 experts of 6524 x 896, bf16, 61 us
// (5.3 TB/s), 16 rows x 5216 x 275, 14 experts, fp32, 40 us (the tile kernel: 132 and 259).  Deeper pipelines (3 or 4 groups of
// loads under way instead of 2), 16 waves, or 32 rows to a workgroup took the same time or more.
template <int TYPE>
__device__ __forceinline__ void gludx_few_body(const GroupArgs& a, int e, int p0, int rows, int j0, float (*part)[4][64][16 / TileT<TYPE>::EB]) {
  typedef TileT<TYPE> TT;
  typedef typename TT::Frag Frag;
  constexpr int EB = TT::EB, C = 16 / EB, KS = 4 * C, D = 2;  // C: columns of a lane, and matrix rows of its operand
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
  const int len = a.N * EB, ng = (a.N + KS - 1) / KS;
  const unsigned step = (unsigned)(a.ldw * EB);
  // (the columns of a lane past the row's end are the row's last ones, which the lane before computes and stores alike)
  const gptr w = (gptr)a.w + ((size_t)e * a.w_stride + min(j0 + C * (lane & 15), a.K - C)) * EB;
  Rows<EB, false> Y;
  Y.init((gptr)a.y, 0, (long long)(p0 + min(lane & 15, rows - 1)) * a.ldy * EB, len);
  struct Group {
    u32x4 w[C], y;
  };
  auto load = [&](Group& G, int g) {
#pragma unroll
    for (int r = 0; r < C; ++r) G.w[r] = load_any(w + (size_t)(unsigned)min(g * KS + q * C + r, a.N - 1) * step);
    G.y = Y.load(g * 64 + q * 16, g * 64 + 64 <= len, len);
  };
  f32x4 acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = f32x4{};
  Group ring[D];
  constexpr int nw = kGluDxWaves;
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], wave + d * nw);
  for (int g = wave; g < ng; g += D * nw) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Group& G = ring[d];
      const int at = g + d * nw;
      // (dy is zeros there already, but zero times a matrix row that is not finite is not)
      if (at * KS + KS > a.N) {
#pragma unroll
        for (int r = 0; r < C; ++r)
          if (at * KS + q * C + r >= a.N) G.w[r] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (EB == 2)
            f[i] = __builtin_amdgcn_perm(G.w[(2 * i + 1) % C][c / 2 % 4], G.w[2 * i % C][c / 2 % 4], c % 2 ? 0x07060302 : 0x05040100);
          else
            f[i] = G.w[i][c % 4];
        }
        acc[c] = mma(__builtin_bit_cast(Frag, G.y), __builtin_bit_cast(Frag, f), acc[c]);
      }
      load(ring[d], at + D * nw);
    }
  }
  // the waves' sums in wave order, then the gate: a thread takes a lane's C columns of one row
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) part[wave][r][lane][c] = acc[c][r];
  __syncthreads();
  const int r = threadIdx.x >> 6, row = 4 * q + r, col = j0 + C * (lane & 15);
  if (r >= 4 || row >= rows || col >= a.K) return;
  float dh[C] = {};
  for (int o = 0; o < nw; ++o)
#pragma unroll
    for (int c = 0; c < C; ++c) dh[c] += part[o][r][lane][c];
  const size_t p = (size_t)(p0 + row), at = (p * 2 * a.K + min(col, a.K - C)) * EB, up = (size_t)a.K * EB;
  const u32x4 gv = load_any((gptr)a.gu + at), uv = load_any((gptr)a.gu + at + up);
  u32x4 dg = {}, du = {}, h = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    auto get = [&](const u32x4& v) {
      if constexpr (EB == 2) return __uint_as_float(c % 2 ? v[c / 2 % 4] & 0xFFFF0000u : v[c / 2 % 4] << 16);
      return __uint_as_float(v[c % 4]);
    };
    auto put = [&](u32x4& v, float f) {
      if constexpr (EB == 2) v[c / 2 % 4] |= (unsigned)f32_to_bf16_rne(f) << (c % 2 * 16);
      else v[c % 4] = __float_as_uint(f);
    };
    const float g = get(gv), u = get(uv), s = 1.f / (1.f + expf(-g)), gs = g * s;
    put(dg, dh[c] * u * (s * (1.f + g * (1.f - s))));
    put(du, dh[c] * gs);
    put(h, gs * u);
  }
  auto store = [](void* base, size_t off, const u32x4& v) {
    typedef u32x4 __attribute__((aligned(1))) any4;
    *(__attribute__((address_space(1))) any4*)((__attribute__((address_space(1))) char*)base + off) = v;
  };
  store(a.dgu, at, dg);
  store(a.dgu, at + up, du);
  if (a.h) store(a.h, (p * a.K + min(col, a.K - C)) * EB, h);
}

// (128 registers, of which bf16 spills two, and two workgroups to a unit: 644 rows, 74 experts of 95 x 5784, bf16, 77 -> 64 us)
template <int TYPE>
__global__ __launch_bounds__(kGluDxThreads, 4) void gludx_few_kernel(GroupArgs a) {
  constexpr int COLS = kGluDxBytes / TileT<TYPE>::EB;
  __shared__ __align__(16) float part[kGluDxWaves][4][64][COLS / 16];
  const int ncol = (a.K + COLS - 1) / COLS;
  const GroupScan sc = scan_groups(a.offsets, a.E, a.rows, kGluDxRows, ncol, 0, 1);
  if ((int)blockIdx.x >= sc.total) return;
  const GroupSpan g = sc.find(a.offsets, a.E, a.rows, blockIdx.x);
  const int tile = g.tile / ncol, r0 = tile * kGluDxRows;
  gludx_few_body<TYPE>(a, g.e, g.p0 + r0, min(kGluDxRows, g.n - r0), (g.tile - tile * ncol) * COLS, part);
}

template <int TYPE>
int gludx_few_launch(const GroupArgs& a, hipStream_t s) {
  constexpr int COLS = kGluDxBytes / TileT<TYPE>::EB;
  const long long nb = group_tiles_max(a.rows, a.E, kGluDxRows) * ((a.K + COLS - 1) / COLS);  // (the caller checked it)
  hipLaunchKernelGGL(gludx_few_kernel<TYPE>, dim3((unsigned)nb), dim3(kGluDxThreads), 0, s, a);
  MOE_CHECK_LAUNCH("moe_grouped_swiglu_dx launch");
  return MOE_OK;
}

}  // namespace

int launch_gludx_few(const GroupArgs& a, int type, hipStream_t s) {
  return type == kF32 ? gludx_few_launch<kF32>(a, s) : gludx_few_launch<kBf16>(a, s);
}
int launch_grouped_decode(const GroupArgs& a, int type, bool direct, hipStream_t s) {
  return type == kI8 ? decode_launch<kI8>(a, direct, s)
                     : type == kF32 ? decode_launch<kF32>(a, direct, s) : decode_launch<kBf16>(a, direct, s);
}
int launch_glu_decode(const GroupArgs& a, int type, bool direct, hipStream_t s) {
  return type == kF32 ? glu_launch<kF32>(a, direct, s) : glu_launch<kBf16>(a, direct, s);
}

}  // namespace moe
