// pairs.cuh -- two fp32 operations by one instruction.
#pragma once

#include "device_common.cuh"

namespace ccl {

// ------------------------------------------------------- pairs of fp32 numbers
// One instruction, two operations, each rounded to nearest as the single ones
// are.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// a + b; a product before it may come out fused with it.
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float total2(F2 a) {
  const float2 t = parts(a);
  return t.x + t.y;
}
// The two elements of a raw word, or of two (fp32), widened.
template <int DT>
__device__ __forceinline__ F2 widen2(const uint32_t* w, int i) {
  return pair(widen<DT>(w, 2 * i), widen<DT>(w, 2 * i + 1));
}
// 2 N elements, rounded to DT.
template <int DT, int N>
__device__ __forceinline__ void pack2(const F2* f, uint32_t* w) {
  float v[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 t = parts(f[i]);
    v[2 * i] = t.x;
    v[2 * i + 1] = t.y;
  }
  pack_out<DT, 2 * N>(v, w);
}

}  // namespace ccl
