// packed.cuh -- two fp32 values in one operand of the packed instructions, each
// rounded as the scalar instruction rounds it.
#pragma once

#include "vec16.cuh"

namespace dsa {

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void pair_split(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float pair_sum(uint64_t r) {
  float a, b;
  pair_split(r, a, b);
  return a + b;
}

// A 16-byte slice of a layer-dtype row as pairs (vec16.cuh).
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& u, uint64_t* p) {
  float f[Vec16<T>::N];
  unpack16<T>(u, f);
#pragma unroll
  for (int i = 0; i < Vec16<T>::N / 2; ++i) p[i] = pair_of(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const uint64_t* p) {
  float f[Vec16<T>::N];
#pragma unroll
  for (int i = 0; i < Vec16<T>::N / 2; ++i) pair_split(p[i], f[2 * i], f[2 * i + 1]);
  return pack16<T>(f);
}

}  // namespace dsa
