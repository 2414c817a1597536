// MFMA operands of the products over plain weights: their element types, and how 16 bytes of a row are read.
#pragma once

#include <type_traits>

#include "grouped.hpp"
#include "mfma_pipe.hpp"

namespace moe {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

template <int TYPE>
struct TileT;
template <>
struct TileT<kBf16> {
  typedef bf16x8 Frag;
  typedef f32x4 Acc;
  static constexpr int EB = 2, MPF = 1;  // bytes of an element, MFMAs per pair of fragments
};
template <>
struct TileT<kI8> {
  typedef i32x4 Frag;
  typedef i32x4 Acc;
  static constexpr int EB = 1, MPF = 1;
};
// An fp32 fragment is 16 bytes of c per lane as well: lane group g (lane / 16) holds c = 4 g .. 4 g + 3, and MFMA e takes
// element e of every lane, that is c = e, 4 + e, 8 + e, 12 + e.
template <>
struct TileT<kF32> {
  typedef f32x4 Frag;
  typedef f32x4 Acc;
  static constexpr int EB = 4, MPF = 4;
};

// Offset past the end of every buffer descriptor (they cover at most kMaxSpan bytes), also with the bytes of a row's
// chunk added: a lane with this offset reads zeros.
constexpr unsigned kOutside = 0xFFFFFC00u;

// 16 bytes at any address
__device__ __forceinline__ u32x4 load_any(gptr p) {
  typedef u32x4 __attribute__((aligned(1))) any4;
  return *(const __attribute__((address_space(1))) any4*)p;
}
// 16 bytes at any element-aligned address, of which the first n exist (the others are zeros)
template <int EB>
__device__ __forceinline__ u32x4 load_part(gptr p, int n) {
  typedef typename std::conditional<EB == 1, unsigned char, typename std::conditional<EB == 2, unsigned short, unsigned>::type>::type El;
  u32x4 v = {0, 0, 0, 0};
  if (n >= 16) {
    v = load_any(p);
  } else {
#pragma unroll
    for (int i = 0; i < 16 / EB; ++i)
      if (i * EB < n) v[i * EB / 4] |= (unsigned)((const __attribute__((address_space(1))) El*)p)[i] << (i * EB % 4 * 8);
  }
  return v;
}

// v moved down by s bytes, zeros from above (s >= 16: zeros)
__device__ __forceinline__ u32x4 shift_bytes(u32x4 v, int s) {
  const unsigned long long lo = (unsigned long long)v[1] << 32 | v[0], hi = (unsigned long long)v[3] << 32 | v[2];
  const int b = (s & 7) * 8;
  const unsigned long long carry = b ? hi << (64 - b) : 0;
  unsigned long long a = lo >> b | carry, c = hi >> b;
  if (s >= 8) a = c, c = 0;
  if (s >= 16) a = 0;
  return u32x4{(unsigned)a, (unsigned)(a >> 32), (unsigned)c, (unsigned)(c >> 32)};
}

}  // namespace
}  // namespace moe
