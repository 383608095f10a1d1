// Quotients rounded to nearest, two at a time, without a division.
#pragma once

#include "common.cuh"

namespace pkv {

// Two fp32 in one register pair, and their products and sums (each rounded as by
// itself) in one instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 of_pair(uint64_t a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// a / b from r = 1/b and minus_b = -b, by STEPS corrections with the exact remainder
// (Markstein, IBM J. Res. Dev. 34, 1990). With r rounded to nearest the first leaves
// less than a unit in the last place and the second nothing: the quotient is
// rounded to nearest. Holds while b, r, the quotient and the remainder's last bit
// are normal numbers.
template <int STEPS>
__device__ __forceinline__ uint64_t quotients(uint64_t a, uint64_t minus_b, uint64_t r) {
  uint64_t q = mul_pair(a, r);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) q = fma_pair(fma_pair(minus_b, q, a), r, q);
  return q;
}

}  // namespace pkv
