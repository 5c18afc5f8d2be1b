// fp32 arithmetic two values at a time: one instruction for the two on sm_103a,
// each rounded as the single form rounds it.
#pragma once

#include <cstdint>

namespace mt {
namespace row {

__device__ __forceinline__ uint64_t bits_of(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 pair_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(a)), "l"(bits_of(b)));
  return pair_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(a)), "l"(bits_of(b)));
  return pair_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
  return pair_of(r);
}
__device__ __forceinline__ float2 get2(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void put2(float* v, float2 p) {
  v[0] = p.x;
  v[1] = p.y;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace row
}  // namespace mt
