// rotate.cuh -- rotation of a lane's pairs of channels.
//
// A lane holds two 16-byte chunks of a head: the two halves of its pairs, or,
// interleaved, two neighbouring chunks, whose pairs are its N in order.
#pragma once

#include "packed.cuh"

namespace dsa {

// (cos, sin) of the angle of position p at a frequency of `turns` 2^-64ths of a
// turn: p * turns modulo 2^64 is exact; its top 32 bits go to sincospi as a
// signed fraction of half a turn.
__device__ __forceinline__ void rotation_at(int64_t pos, uint64_t turns, float& cs, float& sn) {
  const uint64_t w = (uint64_t)pos * turns;
  sincospif((float)(int32_t)(w >> 32) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31 half turns
}

// The same of N values of each chunk, in fp32.
template <int N>
__device__ __forceinline__ void rotate_values(float* a, float* b, const float* cs, const float* sn, bool interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * cs[e] - y * sn[e];
      b[e] = x * sn[e] + y * cs[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], w = b[2 * e + 1];
      a[2 * e] = x * cs[e] - y * sn[e];
      a[2 * e + 1] = x * sn[e] + y * cs[e];
      b[2 * e] = z * cs[N / 2 + e] - w * sn[N / 2 + e];
      b[2 * e + 1] = z * sn[N / 2 + e] + w * cs[N / 2 + e];
    }
  }
}
// The same of pairs of neighbouring values.
template <int N>
__device__ __forceinline__ void rotate_pairs(uint64_t* a, uint64_t* b, const uint64_t* cs, const uint64_t* sn, bool interleaved) {
  if (!interleaved) {
    const uint64_t minus1 = pair_of(-1.f, -1.f);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const uint64_t x = a[e], y = b[e];
      a[e] = fma2(x, cs[e], mul2(mul2(y, minus1), sn[e]));
      b[e] = fma2(y, cs[e], mul2(x, sn[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      float c[2], s[2], x, y;
      pair_split(cs[e], c[0], c[1]);   // of values 2 e and 2 e + 1 of the lane's N pairs
      pair_split(sn[e], s[0], s[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint64_t& p = 2 * e + h < N / 2 ? a[2 * e + h] : b[2 * e + h - N / 2];
        pair_split(p, x, y);
        p = pair_of(x * c[h] - y * s[h], x * s[h] + y * c[h]);
      }
    }
  }
}
template <typename T>
__device__ __forceinline__ void rotate_unit(uint4& u0, uint4& u1, const float* cs, const float* sn, bool interleaved) {
  constexpr int N = Vec16<T>::N;
  float a[N], b[N];
  unpack16<T>(u0, a);
  unpack16<T>(u1, b);
  rotate_values<N>(a, b, cs, sn, interleaved);
  u0 = pack16<T>(a);
  u1 = pack16<T>(b);
}

}  // namespace dsa
