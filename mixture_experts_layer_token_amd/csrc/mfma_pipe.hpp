// Pieces of hand-scheduled MFMA loops: compile-time loops, spreading of work over MFMA slots, and the wait
// states of MFMAs written as inline assembly.
#pragma once

#include <utility>

#include "common.hpp"

namespace moe {
namespace {

typedef const __attribute__((address_space(1))) char* gptr;

// The wait states between the last inline-assembly MFMA and the first other use of its result.
__device__ __forceinline__ void acc_hazard_guard() { asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory"); }

// Compile-time loop: f(std::integral_constant<int, i>) for i = 0 .. N-1, so that every index is
// a constant expression in the body (the K loop's schedule is decided while the code is written
// out, not left to the unroller, which gives up on bodies this large).
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// n items spread over T slots, item i in slot i*T/n: the items of slot s are [spread_lo, spread_hi)
constexpr int spread_lo(int s, int n, int T) { return (s * n + T - 1) / T; }
constexpr int spread_hi(int s, int n, int T) { return ((s + 1) * n + T - 1) / T; }

}  // namespace
}  // namespace moe
