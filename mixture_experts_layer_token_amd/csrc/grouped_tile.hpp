// Tile kernel of the products grouped by expert over plain weights: C[i][j] = sum_c A[i][c] B[j][c] with both
// operands in their row-major form, the output tile stationary in accumulation registers.
//
//   forward             i = grouped row,    j = output feature, c = input feature:  A, B contiguous along c
//   gradient of rows    i = grouped row,    j = input feature,  c = output feature: B strided along c
//   gradient of weights i = output feature, j = input feature,  c = grouped row:    A and B strided along c
//
// A workgroup of 4 waves (2 x 2) computes up to 32 WI x 32 WJ results of one expert; a wave owns 16 WI x 16 WJ of
// them.  Bound by the matrix cores for many rows per expert, by the weights' bytes for few.
//  - two stages of 128 bytes of c per row (64 bf16 or 128 int8, two MFMA steps) in LDS, written by direct
//    global->LDS loads of 16 bytes per lane.  The fragments of the next step are read into registers while the
//    current one is multiplied; a stage's buffer is therefore free when its second step begins, the loads of
//    the stage after next are issued then and have a step and a half to land.  One barrier per stage.
//  - whole 128-byte lines: with stages of half a line (four of 64 bytes in the same LDS) every line came from L2
//    twice, as the second half was asked for when the L1 had long dropped it -- 16.9 GB of operands as 30 GB of
//    L2 hits on the Mixtral-shaped gate/up product, the whole of an L1's fill rate.
//  - an operand contiguous along c sits in LDS as rows of 128 bytes and is read as MFMA fragments directly
//    (ds_read_b128); one that is strided along c sits there as it is in memory, c rows of up to 512 bytes, and is
//    transposed on the way to the registers by ds_read_b64_tr_b16 (16 lanes read 4 rows of 16 elements,
//    lane i receives column i), so neither needs a transposed copy in memory.  16-byte chunks (32-byte
//    ones for the strided form) are XOR-swizzled by row against bank conflicts: the loads write LDS
//    linearly, so the lanes fetch the chunks in swizzled order instead.
//  - the B operand is the MFMA's first one: a lane's four results are four neighbouring columns j of one row i,
//    stored as 8 or 16 bytes.
//  - ragged rows: a group of n rows is cut into ceil(n / (32 WI)) tiles of even size, and a tile of r rows runs
//    with NI = ceil(r / 32) row fragments per wave (the two wave rows take every other fragment).
//  - chunks past the end of c are zeros on both sides (what lies behind a row may hold anything); rows and
//    columns past the edge repeat valid ones and are not stored.
#pragma once

#include <algorithm>

#include "grouped.hpp"
#include "mfma_pipe.hpp"
#include "operand.hpp"

namespace moe {
namespace {

// Waits until at most N of this wave's loads are in flight (the compiler does not know the ones in inline assembly)
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// In-place MFMA on an accumulator held in AGPRs; b is the first operand (see the head of the file).  Its operands
// come straight from LDS reads, which the compiler waits for; no vector instruction writes them.
template <int E>
__device__ __forceinline__ void tile_mfma(f32x4& acc, const bf16x8& b, const bf16x8& a) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
template <int E>
__device__ __forceinline__ void tile_mfma(i32x4& acc, const i32x4& b, const i32x4& a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
template <int E>
__device__ __forceinline__ void tile_mfma(f32x4& acc, const f32x4& b, const f32x4& a) {
  asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+a"(acc) : "v"(b[E]), "v"(a[E]));
}

// The four values of an accumulator, read by assembly as well: the compiler then has no use of accumulators of its
// own and never moves one (its copies next to an MFMA would miss the wait states, and do not fit beside 256 of
// them).  Volatile: not before acc_hazard_guard().
__device__ __forceinline__ float acc_get(const f32x4& acc, int r) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(acc[r]));
  return v;
}
__device__ __forceinline__ float acc_get(const i32x4& acc, int r) {
  int v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(acc[r]));
  return (float)v;
}

typedef __attribute__((address_space(3))) char* lptr;
constexpr int kStageC = 128;  // bytes of c per row and stage
constexpr int kWaves = 4;

// ------------------------------------------------------------------ operands
// Operands are read through buffer descriptors with an exact length: a lane whose offset lies past the end
// gets zeros, which is how everything outside an operand (the end of c, rows of zeros) enters the LDS as
// zeros with no work per load.  The base advances by scalar arithmetic, the lanes' 32-bit offsets stay.

// The loads are inline assembly (they have no result register: the data goes to LDS): after the compiler's own
// LDS-direct loads, every transposing LDS read would wait for all loads in flight.  `Load` is one of them, kept
// until it is written out, on its own or around an MFMA, which then separates the write of m0 from its use.
// Where scalar registers are short a descriptor word waits in a vector register, and the v_readfirstlane that brings it
// back may stand right before the assembly, in which the compiler inserts nothing; a buffer instruction may read a scalar
// register 5 wait states after a vector instruction wrote it.  So the assembly of the first load of an operand and stage (a
// descriptor is made once for all of them) and of every load on its own waits by itself.  (On every load around an
// MFMA: forward product of 8192 rows over 8 experts of 28672 x 4096 1.62 -> 1.65 ms, in turn on one card.)  The generated code is checked.
struct Load {
  u32x4 desc;
  unsigned voff, lds;
};
__device__ __forceinline__ Load make_load(gptr base, unsigned bytes, unsigned voff, lptr l) {
  const unsigned long long p = (unsigned long long)base;
  // (uniform: assembly operands have to be scalar registers, wherever the compiler has kept the values)
  auto u = [](unsigned v) { return (unsigned)__builtin_amdgcn_readfirstlane((int)v); };
  return Load{u32x4{u((unsigned)p), u((unsigned)(p >> 32)) & 0xFFFFu, u(bytes), 0x00027000u}, voff,
              u((unsigned)(size_t)l)};
}
__device__ __forceinline__ void load_now(const Load& d) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               : : "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
}
template <int E, bool FIRST>
__device__ __forceinline__ void tile_mfma(f32x4& acc, const bf16x8& b, const bf16x8& a, const Load& d) {
  if constexpr (FIRST)
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\ts_nop 2\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b), "v"(a), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b), "v"(a), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
}
template <int E, bool FIRST>
__device__ __forceinline__ void tile_mfma(i32x4& acc, const i32x4& b, const i32x4& a, const Load& d) {
  if constexpr (FIRST)
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0\n\ts_nop 2\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b), "v"(a), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b), "v"(a), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
}
template <int E, bool FIRST>
__device__ __forceinline__ void tile_mfma(f32x4& acc, const f32x4& b, const f32x4& a, const Load& d) {
  if constexpr (FIRST)
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x4_f32 %0, %1, %2, %0\n\ts_nop 2\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b[E]), "v"(a[E]), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x4_f32 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 : "+a"(acc) : "v"(b[E]), "v"(a[E]), "s"(d.lds), "v"(d.voff), "s"(d.desc) : "memory", "m0");
}

// One operand of one tile: BM rows of i (or j).  Wave w issues its loads q = 0 .. LQ-1 of every stage; fragments
// of 16 rows are read.  Two forms: `load` gives a direct load to LDS (16-byte rows, spans within 32 bits), `fetch`
// the same 16 bytes in registers by ordinary loads at any address, for `put` to write to the same place.
template <int BM, int EB>
struct Contig {
  static constexpr int LQ = BM / 32;
  static constexpr int BYTES = BM * kStageC;
  gptr base;          // first byte of the stage to be loaded next, row 0
  unsigned span;      // bytes of the operand; the lanes that are not kOutside never pass its end
  int left;           // bytes of c from there to the end of a row
  unsigned voff[LQ];  // this lane's bytes
  unsigned tail;      // its part of the next stage lies past the end of c: kOutside, else 0
  int c_byte;         // its byte of c within a stage
  gptr row[LQ];       // (fetch) its rows; null: zeros

  // off(r, q): byte offset of row r (load q) from p, or kOutside for a row of zeros; all < bytes
  template <typename F>
  __device__ __forceinline__ void init(int wave, int lane, gptr p, unsigned bytes, int c_bytes, F&& off) {
    base = p, span = bytes, left = c_bytes;
    c_byte = ((lane & 7) ^ (lane >> 3)) * 16;  // 8 rows per load: chunk c of row r goes to slot c ^ (r & 7)
#pragma unroll
    for (int q = 0; q < LQ; ++q) {
      const unsigned o = off((q * kWaves + wave) * 8 + lane / 8, q);
      voff[q] = o == kOutside ? o : o + c_byte;
    }
  }
  // rowp(r): address of row r, or null for a row of zeros
  template <typename F>
  __device__ __forceinline__ void init_fetch(int wave, int lane, int c_bytes, F&& rowp) {
    left = c_bytes;
    c_byte = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int q = 0; q < LQ; ++q) row[q] = rowp((q * kWaves + wave) * 8 + lane / 8);
  }
  // Behind conditions the loads of a stage would wait for one another, so they are unconditional: a chunk that ends past
  // the row reads the row's last 16 bytes, moved down afterwards (`adjust`), and a row of zeros reads a page of zeros.
  // Rows of less than 16 bytes (TINY) are read element by element.
  template <bool TINY>
  __device__ __forceinline__ u32x4 fetch(int q) const {
    if constexpr (TINY) return load_part<EB>(row[q] + c_byte, row[q] ? left - c_byte : 0);
    return load_any(row[q] ? row[q] + min(c_byte, left - 16) : (gptr)g_zero_page);
  }
  __device__ __forceinline__ bool whole() const { return left >= kStageC; }
  __device__ __forceinline__ u32x4 adjust(u32x4 v, int) const { return shift_bytes(v, max(c_byte - (left - 16), 0)); }
  __device__ __forceinline__ void end_fetch() {
#pragma unroll
    for (int q = 0; q < LQ; ++q) row[q] += row[q] ? kStageC : 0;
    left -= kStageC;
  }
  __device__ __forceinline__ void begin_stage() { tail = c_byte >= left ? kOutside : 0; }
  __device__ __forceinline__ Load load(int q, lptr lds, int wave) {
    return make_load(base, span, voff[q] | tail, lds + (q * kWaves + wave) * 1024);
  }
  __device__ __forceinline__ void end_stage() {
    base += kStageC;
    left -= kStageC;
  }
  // fragment address of this lane, step 0: first row r0 (a multiple of 16)
  static __device__ __forceinline__ int lane_addr(int r0, int lane) {
    return (r0 + (lane & 15)) * kStageC + ((lane >> 4) ^ (lane & 7)) * 16;
  }
  // rows 16 f from there, MFMA step h of the stage
  template <typename Frag>
  static __device__ __forceinline__ Frag read(lptr base, int addr, int f, int h) {
    return *(const __attribute__((address_space(3))) Frag*)(base + (addr ^ (h * 64)) + f * 16 * kStageC);
  }
};

// BM columns of memory rows that are c, swizzled in units of 16 columns.
template <int BM, int EB>
struct Strided {
  static constexpr int LQ = BM / 32;
  static constexpr int BYTES = BM * kStageC;
  static constexpr int ROWS = kStageC / EB;  // c rows of a stage
  static constexpr int RB = BM * EB;         // bytes per c row
  static constexpr int RPL = 1024 / RB;      // c rows per wave-wide load
  static constexpr int CPR = RB / 16;        // chunks per c row
  static constexpr int US = EB == 2 ? 1 : 2; // log2 of the chunks of a unit
  static_assert(EB == 2 ? BM >= 64 : BM == 128, "bank layout");
  gptr base;      // first byte of the stage to be loaded next
  unsigned ld;    // bytes between c rows
  int stages;     // full stages left
  unsigned tail;  // bytes of the rows of the last, partial one
  unsigned span;
  unsigned voff[LQ];
  long long ld64;  // (fetch)
  int left, ncol;  // (fetch) c rows and bytes of a row that exist

  // The rows that one read touches -- bf16: c = 8 g + 0..3, fp32: c = 4 g + e, for lane groups g = 0..3 -- get
  // different units in the same place, so that they fall into different banks.
  static __device__ __forceinline__ int swz(int c) {
    if constexpr (EB == 4) return (c >> 2) & 3;
    return BM >= 128 ? (c & 3) | ((c >> 3) & 1) << 2 : ((c >> 1) & 1) | ((c >> 3) & 1) << 1;
  }
  static __device__ __forceinline__ int c_row(int q, int wave, int lane) {
    return (q * kWaves + wave) * RPL + lane / CPR;
  }
  // this lane's byte within the row in load q
  static __device__ __forceinline__ unsigned col_of(int q, int wave, int lane) {
    const int slot = lane % CPR;
    return (unsigned)((((slot >> US) ^ swz(c_row(q, wave, lane))) << US) | (slot & ((1 << US) - 1))) * 16;
  }
  // the same where `cols` bytes exist: past them, the first ones again
  static __device__ __forceinline__ unsigned col(int q, int wave, int lane, unsigned cols) {
    const unsigned c = col_of(q, wave, lane);
    return c < cols ? c : 0u;
  }
  __device__ __forceinline__ void init(int wave, int lane, gptr p, unsigned ld_bytes, int c_rows, unsigned col_bytes) {
    base = p, ld = ld_bytes, stages = c_rows / ROWS, tail = (unsigned)(c_rows % ROWS) * ld_bytes;
#pragma unroll
    for (int q = 0; q < LQ; ++q) voff[q] = (unsigned)c_row(q, wave, lane) * ld + col(q, wave, lane, col_bytes);
  }
  // the rows that exist of the next stage: the others lie past the end
  __device__ __forceinline__ void begin_stage() { span = stages > 0 ? ld * ROWS : stages == 0 ? tail : 0; }
  __device__ __forceinline__ Load load(int q, lptr lds, int wave) {
    return make_load(base, span, voff[q], lds + (q * kWaves + wave) * 1024);
  }
  __device__ __forceinline__ void end_stage() {
    base += (size_t)ld * ROWS;
    --stages;
  }
  __device__ __forceinline__ void init_fetch(gptr p, long long ld_bytes, int c_rows, int col_bytes) {
    base = p, ld64 = ld_bytes, left = c_rows, ncol = col_bytes;
  }
  // (as in Contig: columns past the edge from the row's last 16 bytes, rows past the end from the last row)
  template <bool TINY>
  __device__ __forceinline__ u32x4 fetch(int q, int wave, int lane) const {
    const int c = c_row(q, wave, lane), o = (int)col_of(q, wave, lane);
    if constexpr (TINY) return load_part<EB>(base + c * ld64 + o, c < left ? ncol - o : 0);
    return load_any(base + min(c, left - 1) * ld64 + min(o, ncol - 16));
  }
  __device__ __forceinline__ bool whole() const { return left >= ROWS && ncol >= RB; }
  __device__ __forceinline__ u32x4 adjust(u32x4 v, int q, int wave, int lane) const {
    return shift_bytes(v, c_row(q, wave, lane) < left ? max((int)col_of(q, wave, lane) - (ncol - 16), 0) : 16);
  }
  __device__ __forceinline__ void end_fetch() {
    base += ld64 * ROWS;
    left -= ROWS;
  }
  // bf16: lane i of each 16 reads c row 8 (lane / 16) + i / 4, four columns from 4 (i % 4); the second read takes the c
  // rows 4 below.  fp32: lane i of group g reads column i of the c rows 4 g .. 4 g + 3.  m: index of the 16-column
  // fragment.
  static __device__ __forceinline__ int lane_addr(int m, int lane) {
    if constexpr (EB == 4) return 4 * (lane >> 4) * RB + ((m ^ (lane >> 4)) << 6) + 4 * (lane & 15);
    const int c = 8 * (lane >> 4) + ((lane & 15) >> 2);
    return c * RB + ((m ^ swz(c)) << 5) + 8 * (lane & 3);
  }
  // fragment m ^ x (x: the bits by which it differs from lane_addr's), MFMA step h of the stage
  template <typename Frag>
  static __device__ __forceinline__ Frag read(lptr base, int addr, int x, int h) {
    if constexpr (EB == 4) {
      const __attribute__((address_space(3))) float* p =
          (const __attribute__((address_space(3))) float*)(base + (addr ^ (x << 6)) + h * 16 * RB);
      return Frag{p[0], p[RB / 4], p[2 * RB / 4], p[3 * RB / 4]};
    } else {
      typedef __attribute__((address_space(3))) s16x4* p4;
      const lptr p = base + (addr ^ (x << 5)) + h * 32 * RB;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)(p + 4 * RB));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// ------------------------------------------------------------------ results
// two fp32 to bf16, nearest-even (one instruction)
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 b2;
  return __builtin_bit_cast(unsigned, b2{(__bf16)lo, (__bf16)hi});
}

// 16 rows of w columns from a wave's LDS region, of which ni rows and nj columns exist; they start at row i0, column
// j0 of the tile.  Element by element: the rare layouts take it.
__device__ __forceinline__ void store_rows(const __attribute__((address_space(3))) float* reg, char* out, long long ldc,
                                           int ni, int nj, int i0, int j0, int w, const float* sw, int bf16) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int r = 0; r < min(ni, 16); ++r)
#pragma unroll 1
    for (int c = lane; c < min(nj, w); c += 64) {
      const float v = reg[r * w + c];
      store_out(out, (size_t)(i0 + r) * ldc + j0 + c, sw ? v * sw[j0 + c] : v, bf16);
    }
}

// ------------------------------------------------------------------ tiles
struct TileItem {
  int e, i0, ni, j0, nj, p0, nc;  // expert; first i and j and how many exist; first grouped row; length of c
  int part;                       // weights' gradient: part of the group's rows
};

// STAGED: operands pass through registers (any alignment, stride and extent).  NB: stages in LDS.
template <int OP, int TYPE, int WI, int WJ, bool GATHER, bool STAGED, int NB>
struct TileKernel {
  typedef TileT<TYPE> TT;
  typedef typename TT::Frag Frag;
  typedef typename TT::Acc Acc;
  static constexpr int EB = TT::EB, KE = kStageC / EB;  // elements of c per stage
  static constexpr int BI = 32 * WI, BJ = 32 * WJ;
  static constexpr bool SA = OP == kOpDw, SB = OP != kOpY;  // strided operands
  typedef typename std::conditional<SA, Strided<BI, EB>, Contig<BI, EB>>::type OpA;
  typedef typename std::conditional<SB, Strided<BJ, EB>, Contig<BJ, EB>>::type OpB;
  static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  static constexpr int NL = OpA::LQ + OpB::LQ;           // loads per stage and wave
  static constexpr int REGION = 16 * 16 * WJ * 4;        // per wave, behind the stages: see store_rows
  static constexpr size_t LDS = (size_t)NB * STAGE + kWaves * REGION;
  static constexpr bool IDX = GATHER && OP == kOpDw && !STAGED;  // x rows of c through perm_src
  static constexpr int RPL = IDX ? 1024 / (BJ * EB) : 1;  // c rows per load of B
  static constexpr int NX = IDX ? OpB::LQ * RPL : 1;
  static_assert(NB == 2 || (NB == 4 && !STAGED), "stages");

  // The operands of one tile on their way to LDS.
  struct Feed {
    const GroupArgs& a;
    const int lane, wave;
    const lptr lds;
    TileItem t;
    OpA A;
    OpB B;
    // IDX: perm_src of this wave's c rows of a stage, by scalar loads one stage ahead, and the offsets of the x rows
    // they name for the stage to be loaded next (kOutside: zeros)
    int idx_next[NX];
    unsigned idx[NX], bcol[OpB::LQ];
    // offsets of the gathered x rows of the tile to come
    static constexpr bool AHEAD = OP == kOpY && !STAGED;
    unsigned ahead[AHEAD ? OpA::LQ : 1];
    // STAGED: a stage in registers
    u32x4 held[STAGED ? NL : 1];
    int fetched;  // stages

    __device__ __forceinline__ Feed(const GroupArgs& args, lptr smem)
        : a(args), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lds(smem) {}

    // looks up what init(item) needs from memory
    __device__ __forceinline__ void look_ahead(const TileItem& item) {
      if constexpr (AHEAD) {
        if (!a.perm_src) return;
#pragma unroll
        for (int q = 0; q < OpA::LQ; ++q) {
          const int xr = x_row(a, item.p0 + min((q * kWaves + wave) * 8 + lane / 8, item.ni - 1));
          ahead[q] = xr >= 0 ? (unsigned)xr * (unsigned)a.ldx * EB : kOutside;
        }
      }
    }
    __device__ __forceinline__ void init(const TileItem& item) {
      t = item;
      const gptr x = (gptr)a.x, w = (gptr)a.w + (size_t)t.e * a.w_stride * EB, y = (gptr)a.y;
      const unsigned ldx = (unsigned)a.ldx * EB, ldw = (unsigned)a.ldw * EB, ldy = (unsigned)a.ldy * EB;
      if constexpr (STAGED) {
        fetched = 0;
        if constexpr (OP == kOpY) {
          A.init_fetch(wave, lane, a.K * EB, [&](int r) -> gptr {
            const int xr = x_row(a, t.p0 + min(r, t.ni - 1));
            return xr >= 0 ? x + (size_t)xr * a.ldx * EB : (gptr) nullptr;
          });
          B.init_fetch(wave, lane, a.K * EB, [&](int r) -> gptr { return w + (size_t)(t.j0 + min(r, t.nj - 1)) * a.ldw * EB; });
        } else if constexpr (OP == kOpDx) {
          A.init_fetch(wave, lane, a.N * EB, [&](int r) -> gptr { return y + (size_t)(t.p0 + min(r, t.ni - 1)) * a.ldy * EB; });
          B.init_fetch(w + (size_t)t.j0 * EB, a.ldw * EB, t.nc, t.nj * EB);
        } else {
          A.init_fetch(y + ((size_t)t.p0 * a.ldy + t.i0) * EB, a.ldy * EB, t.nc, t.ni * EB);
          B.init_fetch(x + ((size_t)(GATHER ? 0 : t.p0) * a.ldx + t.j0) * EB, a.ldx * EB, t.nc, t.nj * EB);
        }
      } else if constexpr (OP == kOpY) {
        const unsigned cb = (unsigned)a.K * EB;
        if (a.perm_src)
          A.init(wave, lane, x, a.x_rows > 0 ? (unsigned)(a.x_rows - 1) * ldx + cb : 0, cb,
                 [&](int, int q) -> unsigned { return ahead[AHEAD ? q : 0]; });
        else
          A.init(wave, lane, x + (size_t)t.p0 * a.ldx * EB, (unsigned)(t.ni - 1) * ldx + cb, cb,
                 [&](int r, int) -> unsigned { return (unsigned)min(r, t.ni - 1) * ldx; });
        B.init(wave, lane, w + (size_t)t.j0 * a.ldw * EB, (unsigned)(t.nj - 1) * ldw + cb, cb,
               [&](int r, int) -> unsigned { return (unsigned)min(r, t.nj - 1) * ldw; });
      } else if constexpr (OP == kOpDx) {
        const unsigned cb = (unsigned)a.N * EB;
        A.init(wave, lane, y + (size_t)t.p0 * a.ldy * EB, (unsigned)(t.ni - 1) * ldy + cb, cb,
               [&](int r, int) -> unsigned { return (unsigned)min(r, t.ni - 1) * ldy; });
        B.init(wave, lane, w + (size_t)t.j0 * EB, ldw, t.nc, t.nj * EB);
      } else {
        A.init(wave, lane, y + ((size_t)t.p0 * a.ldy + t.i0) * EB, ldy, t.nc, t.ni * EB);
        if constexpr (!IDX) B.init(wave, lane, x + ((size_t)t.p0 * a.ldx + t.j0) * EB, ldx, t.nc, t.nj * EB);
      }
      if constexpr (IDX) {
#pragma unroll
        for (int q = 0; q < OpB::LQ; ++q) bcol[q] = OpB::col(q, wave, lane, t.nj * EB);
      }
    }
    __device__ __forceinline__ void idx_load(int s) {
      if constexpr (IDX) {
        const __attribute__((address_space(4))) int* p = (const __attribute__((address_space(4))) int*)a.perm_src + t.p0;
#pragma unroll
        for (int n = 0; n < NX; ++n) idx_next[n] = p[min(s * KE + (n / RPL * kWaves + wave) * RPL + n % RPL, t.nc - 1)];
      }
    }
    __device__ __forceinline__ void idx_rows(int s) {
      if constexpr (IDX) {
#pragma unroll
        for (int n = 0; n < NX; ++n) {
          const int v = idx_next[n], r = div_k(a, v);
          const bool ok = v >= 0 && r < a.x_rows && s * KE + (n / RPL * kWaves + wave) * RPL + n % RPL < t.nc;
          idx[n] = ok ? (unsigned)r * (unsigned)a.ldx * EB : kOutside;
        }
      }
    }
    // the loads of the stage to be loaded next, into buffer buf: begin, load L = 0 .. NL-1, end
    __device__ __forceinline__ void begin_stage() {
      A.begin_stage();
      if constexpr (!IDX) B.begin_stage();
    }
    template <int L>
    __device__ __forceinline__ Load load(int buf) {
      const lptr la = lds + buf * STAGE, lb = la + OpA::BYTES;
      if constexpr (L < OpA::LQ) {
        return A.load(L, la, wave);
      } else if constexpr (IDX) {
        constexpr int q = L - OpA::LQ;
        unsigned o = idx[(q * RPL) % NX];
        static_for<RPL - 1>([&](auto ic) { o = lane / (64 / RPL) == ic + 1 ? idx[(q * RPL + ic + 1) % NX] : o; });
        const unsigned span = a.x_rows > 0 ? (unsigned)(a.x_rows - 1) * (unsigned)a.ldx * EB + (unsigned)t.nj * EB : 0;
        return make_load((gptr)a.x + (size_t)t.j0 * EB, span, o + bcol[q], lb + (q * kWaves + wave) * 1024);
      } else {
        return B.load(L - OpA::LQ, lb, wave);
      }
    }
    __device__ __forceinline__ void end_stage() {
      A.end_stage();
      if constexpr (!IDX) B.end_stage();
    }
    // the first NB stages
    __device__ __forceinline__ void prologue() {
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        idx_load(s);
        idx_rows(s);
        begin_stage();
        static_for<NL>([&](auto Lc) { load_now(load<Lc>(s)); });
        end_stage();
      }
      idx_load(NB);
    }

    // a stage into registers
    __device__ __forceinline__ void fetch() {
      const bool tiny_a = (OP == kOpY ? a.K : a.N) * EB < 16, tiny_b = a.K * EB < 16;  // bytes of the operands' rows
      if (tiny_a || tiny_b) fetch_stage<true>();
      else fetch_stage<false>();
      A.end_fetch();
      B.end_fetch();
      ++fetched;
    }
    template <bool TINY>
    __device__ __forceinline__ void fetch_stage() {
      constexpr bool GB = GATHER && OP == kOpDw;
      int xr[GB ? OpB::LQ : 1];
#pragma unroll
      for (int q = 0; q < OpA::LQ; ++q) {
        if constexpr (SA) held[q] = A.template fetch<TINY>(q, wave, lane);
        else held[q] = A.template fetch<TINY>(q);
      }
#pragma unroll
      for (int q = 0; q < OpB::LQ; ++q) {
        if constexpr (GB) {
          const int c = fetched * KE + OpB::c_row(q, wave, lane), p = a.perm_src[t.p0 + min(c, t.nc - 1)];
          xr[q] = c < t.nc ? named_row(a, p) : -1;
        } else if constexpr (SB) {
          held[OpA::LQ + q] = B.template fetch<TINY>(q, wave, lane);
        } else {
          held[OpA::LQ + q] = B.template fetch<TINY>(q);
        }
      }
      if constexpr (GB) {
#pragma unroll
        for (int q = 0; q < OpB::LQ; ++q) {
          const int o = (int)OpB::col_of(q, wave, lane), ncol = t.nj * EB;
          const gptr r = (gptr)a.x + ((size_t)max(xr[q], 0) * a.ldx + t.j0) * EB;
          if constexpr (TINY) held[OpA::LQ + q] = load_part<EB>(r + o, xr[q] >= 0 ? ncol - o : 0);
          else held[OpA::LQ + q] = load_any(xr[q] >= 0 ? r + min(o, ncol - 16) : (gptr)g_zero_page);
        }
      }
      bool ok = A.whole() && B.whole();
      if constexpr (GB) {
        ok = ok && fetched * KE + KE <= t.nc;
      }
      if (TINY || ok) return;  // (uniform)
#pragma unroll
      for (int q = 0; q < OpA::LQ; ++q) {
        if constexpr (SA) held[q] = A.adjust(held[q], q, wave, lane);
        else held[q] = A.adjust(held[q], q);
      }
#pragma unroll
      for (int q = 0; q < OpB::LQ; ++q) {
        u32x4& h = held[OpA::LQ + q];
        if constexpr (GB) h = shift_bytes(h, xr[q] >= 0 ? max((int)OpB::col_of(q, wave, lane) - (t.nj * EB - 16), 0) : 16);
        else if constexpr (SB) h = B.adjust(h, q, wave, lane);
        else h = B.adjust(h, q);
      }
    }
    __device__ __forceinline__ void put(int buf) {
#pragma unroll
      for (int L = 0; L < NL; ++L) {
        const lptr l =
            lds + buf * STAGE + (L < OpA::LQ ? 0 : OpA::BYTES) + ((L < OpA::LQ ? L : L - OpA::LQ) * kWaves + wave) * 1024;
        *(__attribute__((address_space(3))) u32x4*)(l + lane * 16) = held[L];
      }
    }
  };

  // One tile with NI row fragments per wave.  Its first NB stages have landed for this wave (STAGED: feed is
  // initialised).  advance() is called when the tile's last operands have been read: it starts the loads of the
  // workgroup's next tile, which land while this tile's results are written.
  template <int NI, typename F>
  static __device__ __forceinline__ void body(const GroupArgs& a, const TileItem& t, Feed& feed, F&& advance) {
    const int lane = feed.lane, wave = feed.wave, wi = wave >> 1, wj = wave & 1;
    const lptr lds = feed.lds;
    // ---- fragments.  Row fragments of wave row wi: 2 f + wi; column fragments of wave column wj: WJ wj + f
    int addr_a, addr_b;
    if constexpr (SA) addr_a = OpA::lane_addr(wi, lane);
    else addr_a = OpA::lane_addr(16 * wi, lane);
    if constexpr (SB) addr_b = OpB::lane_addr(WJ * wj, lane);
    else addr_b = OpB::lane_addr(16 * WJ * wj, lane);
    auto read_a = [&](int f, int buf, int h) { return OpA::template read<Frag>(lds + buf * STAGE, addr_a, 2 * f, h); };
    auto read_b = [&](int f, int buf, int h) {
      return OpB::template read<Frag>(lds + buf * STAGE + OpA::BYTES, addr_b, f, h);
    };

    Acc acc[WJ][NI];
#pragma unroll
    for (int j = 0; j < WJ; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        acc[j][i] = Acc{};
        asm volatile("" : "+a"(acc[j][i]));  // (written here, two wait states before the first MFMA at least)
      }

    const int ns = (t.nc + KE - 1) / KE;  // >= 1
    if constexpr (STAGED) {
      feed.fetch();
      barrier_keep_loads();  // every wave is done with the buffers of the tile before
      feed.put(0);
      feed.fetch();
    }
    Frag fa[2][NI], fb[2][WJ];
    barrier_keep_loads();
#pragma unroll
    for (int i = 0; i < NI; ++i) fa[0][i] = read_a(i, 0, 0);
#pragma unroll
    for (int j = 0; j < WJ; ++j) fb[0][j] = read_b(j, 0, 0);

    // ---- one MFMA step: step h of stage s is multiplied, the next one's fragments are read.  With h = 1 the
    // barrier comes first: it publishes stage s+1 (every wave has waited for its own loads of it) and frees the
    // buffer of stage s (its last fragments are in registers), into which stage s+NB is then loaded.
    auto step = [&](auto hc, int s) {
      constexpr int h = hc;
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      if constexpr (h == 1) {
        // (stage 1 landed before the tile began; a wait there would be one for the last tile's stores)
        if constexpr (!STAGED)
          if (s > 0) wait_loads<(NB - 2) * NL>();
        barrier_keep_loads();
        if constexpr (STAGED) feed.fetch();
        feed.idx_rows(s + NB);
        feed.idx_load(s + NB + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      const int cbuf = s & (NB - 1), nbuf = (s + 1) & (NB - 1), rbuf = h == 0 ? cbuf : nbuf;
      // slots: reads over the first three quarters of the MFMAs, loads over all of them (over half: 2% slower)
      constexpr int R = WJ * NI * TT::MPF, NR = NI + WJ, T = 3 * R / 4 > 0 ? 3 * R / 4 : 1;
      constexpr int NQ = h == 1 && !STAGED ? NL : 0;
      static_for<R>([&](auto rc) {
        constexpr int r = rc, e = r / (WJ * NI), j = r % (WJ * NI) / NI, i = r % NI;
        constexpr int l0 = spread_lo(r, NQ, R), l1 = spread_hi(r, NQ, R);
        if constexpr (l0 == 0 && l1 > 0) feed.begin_stage();
        constexpr bool first = l0 == 0 || l0 == OpA::LQ;
        if constexpr (l1 > l0) tile_mfma<e, first>(acc[j][i], fb[h][j], fa[h][i], feed.template load<l0>(cbuf));
        else tile_mfma<e>(acc[j][i], fb[h][j], fa[h][i]);
        static_for<(l1 > l0 ? l1 - l0 - 1 : 0)>([&](auto Lc) { load_now(feed.template load<l0 + 1 + Lc>(cbuf)); });
        if constexpr (l1 > l0 && l1 == NQ) feed.end_stage();
        constexpr int lo = spread_lo(r, NR, T), hi = r < T ? spread_hi(r, NR, T) : lo;
        static_for<hi - lo>([&](auto mc) {
          constexpr int m = lo + mc;
          if constexpr (m < NI) fa[h ^ 1][m] = read_a(m, rbuf, h ^ 1);
          else fb[h ^ 1][m - NI] = read_b(m - NI, rbuf, h ^ 1);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (STAGED && h == 0) feed.put(nbuf);  // free since the barrier of the stage before
    };
    int s = 0;
    do {
      step(std::integral_constant<int, 0>{}, s);
      step(std::integral_constant<int, 1>{}, s);
    } while (++s < ns);
    acc_hazard_guard();
    // the stages past the end (zeros) have landed, and every wave is done reading: the buffers are free
    if constexpr (!STAGED) wait_loads<0>();
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier_keep_loads();
    advance();

    // ---- results
    // A lane's four results are neighbouring columns of one row: 8 or 16 bytes per store, straight from the
    // accumulators.  The code is kept short on purpose: with every address and rounding spelled out it took 28 us
    // per tile, most of it waiting for instructions.
    const int rlane = wi * 16 + (lane & 15);  // row of fragment 0; the others follow 32 rows apart
    const int clane = WJ * wj * 16 + (lane >> 4) * 4;  // column of fragment 0; the others follow 16 apart
    const long long ldc = OP == kOpY ? a.ldy : OP == kOpDx ? a.ldx : a.ldw;
    const int ob = a.out_bf16 ? 2 : 4;
    char* out = (char*)(OP == kOpY ? a.y : OP == kOpDx ? a.x : a.w);
    out += ((OP == kOpDw ? ((size_t)t.part * a.E + t.e) * a.w_stride + (size_t)t.i0 * ldc : (size_t)t.p0 * ldc) + t.j0) * ob;
    const float* sw = TYPE == kI8 ? a.w_scale + (size_t)t.e * a.N + t.j0 : nullptr;
    float rs[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      rs[i] = 1.f;
      if constexpr (TYPE == kI8) {
        const int xr = x_row(a, t.p0 + min(32 * i + rlane, t.ni - 1));
        rs[i] = xr >= 0 ? a.x_scale[xr] : 0.f;
      }
    }
    // rows that start on a store's width and end on four columns
    if (((size_t)out | (size_t)(ldc * ob)) % (4 * ob) == 0 && t.nj % 4 == 0) {
      f32x4 cs[TYPE == kI8 ? WJ : 1];
      if constexpr (TYPE == kI8) {
#pragma unroll
        for (int j = 0; j < WJ; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) cs[j][r] = sw[min(clane + 16 * j + r, t.nj - 1)];
      }
      // the next tile's first stages have landed before the first store: its loop need not wait for stores
      if constexpr (!STAGED) wait_loads<0>();
      auto rows = [&](auto bf) {
        constexpr bool BF = decltype(bf)::value;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (32 * i + rlane >= t.ni) continue;
          char* p = out + ((size_t)(32 * i + rlane) * ldc + clane) * (BF ? 2 : 4);
#pragma unroll
          for (int j = 0; j < WJ; ++j) {
            if (clane + 16 * j >= t.nj) continue;
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = acc_get(acc[j][i], r);
              if constexpr (TYPE == kI8) v[r] = v[r] * rs[i] * cs[j][r];
            }
            if constexpr (BF) *(u32x2*)(p + 32 * j) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            else *(f32x4*)(p + 64 * j) = v;
          }
        }
      };
      if (a.out_bf16) rows(std::true_type{});
      else rows(std::false_type{});
    } else {
      // any other: 16 rows at a time through the wave's own LDS region, element by element
      if constexpr (!STAGED) wait_loads<0>();
      typedef __attribute__((address_space(3))) float* lfloat;
      const lfloat reg = (lfloat)(lds + NB * STAGE + wave * REGION);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
          f32x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc_get(acc[j][i], r) * rs[i];
          *(__attribute__((address_space(3))) f32x4*)(reg + (lane & 15) * 16 * WJ + 16 * j + (lane >> 4) * 4) = v;
        }
        store_rows(reg, out, ldc, t.ni - (32 * i + wi * 16), t.nj - WJ * wj * 16, 32 * i + wi * 16, WJ * wj * 16, 16 * WJ, sw,
                   a.out_bf16);
      }
    }
  }
};

// Workgroup b runs on XCD b % 8.  Tiles of an expert go in bands of up to 8 row tiles, column by column: the 32 tiles an
// XCD works on at a time span few row and column panels.
constexpr int kBand = 8;
__device__ __forceinline__ void band_order(int u, int nt, int ncol, int& row, int& col) {
  const int band = u / (kBand * ncol), r = u - band * kBand * ncol, h = min(kBand, nt - band * kBand);
  col = r / h;
  row = band * kBand + r - col * h;
}

// Persistent: each XCD's workgroups walk its tiles (part_range) side by side.
template <int OP, int TYPE, int WI, int WJ, bool GATHER, bool STAGED, int NB>
__global__ __launch_bounds__(256, (WI * WJ > 16 || NB > 2 ? 1 : 2)) void grouped_tile_kernel(GroupArgs a) {
  typedef TileKernel<OP, TYPE, WI, WJ, GATHER, STAGED, NB> Tk;
  extern __shared__ __align__(1024) char smem[];
  const int nj = OP == kOpY ? a.N : a.K, ncol = (nj + Tk::BJ - 1) / Tk::BJ;
  const int ntw = (a.N + Tk::BI - 1) / Tk::BI;  // row tiles of a weight gradient
  const int xcd = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
  // This XCD's tiles: its part of every group, or (few tiles per group) a contiguous range of all of them
  const int parts = a.each_xcd ? kXcds : 1, px = a.each_xcd ? xcd : 0;
  GroupScan sc;
  int end;
  if constexpr (OP == kOpDw) {
    const int n = a.split * a.E;  // parts of groups, all of ntw * ncol tiles: each 8 of them give an XCD that many
    if (a.each_xcd) {
      end = n / kXcds * ntw * ncol;
      for (int e = n / kXcds * kXcds; e < n; ++e) end += part_range(ntw * ncol, e, xcd, kXcds).y;
    } else {
      end = n * ntw * ncol;
    }
  } else {
    sc = scan_groups(a.offsets, a.E, a.rows, Tk::BI, ncol, px, parts);
    end = sc.total;
  }
  int u = blockIdx.x / kXcds;
  if (!a.each_xcd) {
    const int2 r = part_range(end, 0, xcd, kXcds);
    u += r.x;
    end = r.x + r.y;
  }
  auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };

  // tile u, or the next one of this workgroup with anything to add up; false: none left
  auto next_tile = [&](TileItem& t) __attribute__((always_inline)) {
    for (; u < end; u += stride) {
      int row, col;
      t.part = 0;
      if constexpr (OP == kOpDw) {
        const int tiles = ntw * ncol;
        int e = u / tiles * parts, v = u % tiles;
        int2 p = part_range(tiles, e, px, parts);
        while (v >= p.y) {
          v -= p.y;
          p = part_range(tiles, ++e, px, parts);
        }
        t.part = uni(e / a.E);
        t.e = uni(e - t.part * a.E);
        band_order(uni(p.x + v), ntw, ncol, row, col);
        const int2 g = group_range(a.offsets, t.e, a.rows);
        t.p0 = g.x, t.nc = g.y;
        if (a.split > 1) {  // this part of the group's rows, in whole stages
          const int len = (g.y + a.split * Tk::KE - 1) / (a.split * Tk::KE) * Tk::KE;
          const int from = min(t.part * len, g.y);
          t.p0 += from, t.nc = min(len, g.y - from);
        }
        t.i0 = row * Tk::BI;
        t.ni = min(Tk::BI, a.N - t.i0);
      } else {
        const GroupSpan g = sc.find(a.offsets, a.E, a.rows, u);
        if (g.n <= 0) return false;  // (only groups that overlap, more tiles than an int counts, can lead here)
        t.e = g.e;
        const int nt = (g.n + Tk::BI - 1) / Tk::BI;
        band_order(g.tile, nt, ncol, row, col);
        const int each = g.n / nt, longer = g.n - each * nt;  // the first `longer` tiles have one row more
        t.p0 = g.p0 + row * each + min(row, longer), t.ni = each + (row < longer), t.i0 = 0;
        t.nc = OP == kOpY ? a.K : a.N;
      }
      t.j0 = col * Tk::BJ;
      t.nj = min(Tk::BJ, nj - t.j0);
      // everything about the tile is uniform
      t.i0 = uni(t.i0), t.ni = uni(t.ni), t.j0 = uni(t.j0), t.nj = uni(t.nj), t.p0 = uni(t.p0), t.nc = uni(t.nc);
      if (OP != kOpDw || t.nc > 0) {
        u += stride;
        return true;
      }
      // an expert (or part) without rows
      const size_t o = ((size_t)t.part * a.E + t.e) * a.w_stride + (size_t)t.i0 * a.ldw + t.j0;
      for (int i = threadIdx.x / 64; i < t.ni; i += kWaves)
        for (int j = threadIdx.x % 64; j < t.nj; j += 64) store_out((void*)a.w, o + (size_t)i * a.ldw + j, 0.f, a.out_bf16);
    }
    return false;
  };

  TileItem cur, next;
  if (!next_tile(cur)) return;
  typename Tk::Feed feed(a, (lptr)smem);
  feed.look_ahead(cur);
  feed.init(cur);
  if constexpr (!STAGED) feed.prologue();
  bool more = next_tile(next);
  if (more) feed.look_ahead(next);
  if constexpr (!STAGED) wait_loads<0>();
  for (;;) {
    TileItem after;
    bool any_after = false;
    auto advance = [&]() __attribute__((always_inline)) {
      if (!more) return;
      feed.init(next);
      if constexpr (!STAGED) feed.prologue();
      any_after = next_tile(after);  // while the loads are under way
      if (any_after) feed.look_ahead(after);
    };
    const int n = (cur.ni + 31) / 32;
    static_for<WI>([&](auto ic) {
      constexpr int NI = ic + 1;
      if (n == NI) Tk::template body<NI>(a, cur, feed, advance);
    });
    if (!more) break;
    cur = next, next = after, more = any_after;
  }
}

template <int OP, int TYPE, int WI, int WJ, bool GATHER, bool STAGED, int NB = 2>
int tile_launch_one(const GroupArgs& a, hipStream_t s) {
  typedef TileKernel<OP, TYPE, WI, WJ, GATHER, STAGED, NB> Tk;
  const int nj = OP == kOpY ? a.N : a.K;
  const long long nt = OP == kOpDw ? (long long)a.E * ((a.N + Tk::BI - 1) / Tk::BI) * a.split
                                   : group_tiles_max(a.rows, a.E, Tk::BI);
  long long nb = nt * ((nj + Tk::BJ - 1) / Tk::BJ);
  if (nb == 0) return MOE_OK;
  if (nb > 0x7FFFFF00LL) return fail(MOE_ERR_UNSUPPORTED, "moe_grouped_gemm: %lld tiles", nb);
  static bool attr_set[64];  // per device
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!attr_set[dev]) {
    hipError_t e = hipFuncSetAttribute((const void*)grouped_tile_kernel<OP, TYPE, WI, WJ, GATHER, STAGED, NB>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)Tk::LDS);
    if (e != hipSuccess) return hip_fail(e, "moe_grouped_gemm: LDS attribute");
    attr_set[dev] = true;
  }
  // a multiple of the XCDs, as many as are resident at a time (two per compute unit where LDS allows)
  const long long slots = (long long)cu_count() * (2 * Tk::LDS <= 160 * 1024 ? 2 : 1) / kXcds * kXcds;
  nb = (std::min(nb, std::max(slots, (long long)kXcds)) + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((grouped_tile_kernel<OP, TYPE, WI, WJ, GATHER, STAGED, NB>), dim3((unsigned)nb), dim3(256), Tk::LDS, s,
                     a);
  MOE_CHECK_LAUNCH("moe_grouped_gemm launch");
  return MOE_OK;
}

}  // namespace
}  // namespace moe
