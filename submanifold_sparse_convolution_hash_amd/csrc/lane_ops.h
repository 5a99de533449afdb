// Exchanges between the lanes of a wave that the dense layers use.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace submconv {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// v_permlane16_swap: exchanges lanes 16..31 and 48..63 of a with lanes 0..15
// and 32..47 of b; v_permlane32_swap: lanes 32..63 of a with lanes 0..31 of b.
__device__ __forceinline__ u32x2 lane_rows_swap(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  return u32x2{r[0], r[1]};
}
__device__ __forceinline__ u32x2 lane_halves_swap(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return u32x2{r[0], r[1]};
}
// both results of a swap of x with itself, added
__device__ __forceinline__ float swap_sum(u32x2 p) {
  const uint32_t a = p[0], b = p[1];  // (a bit cast of a vector's element takes element 0)
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sum over each G neighbouring lanes (a power of two from 4 to 64), the same
// value in all of them.
template <int G>
__device__ __forceinline__ float lanes_sum(float x) {
  static_assert(G >= 4 && G <= 64, "lanes");
  x += dpp<0xB1>(x);                          // lanes 1 0 3 2 of each four
  x += dpp<0x4E>(x);                          // lanes 2 3 0 1
  if constexpr (G >= 8) x += dpp<0x141>(x);   // each eight mirrored
  if constexpr (G >= 16) x += dpp<0x140>(x);  // each sixteen mirrored
  if constexpr (G >= 32) {
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    x = swap_sum(lane_rows_swap(v, v));
  }
  if constexpr (G >= 64) {
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    x = swap_sum(lane_halves_swap(v, v));
  }
  return x;
}

// Sum over the lanes that are equal modulo L (2, 4 or 8), in all of them.
template <int L>
__device__ __forceinline__ float lanes_sum_over(float x) {
  static_assert(L == 2 || L == 4 || L == 8, "lanes");
  if constexpr (L <= 2) x += dpp<0x4E>(x);   // lanes 2 3 0 1 of each four
  if constexpr (L <= 4) x += dpp<0x124>(x);  // each sixteen turned by four
  x += dpp<0x128>(x);                        // and by eight
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  x = swap_sum(lane_rows_swap(v, v));
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return swap_sum(lane_halves_swap(u, u));
}

}  // namespace
}  // namespace submconv
