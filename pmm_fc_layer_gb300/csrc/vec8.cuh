// Eight columns of a row: what a thread of the kernels without tiles works
// on.
#pragma once
#include "epilogue_math.cuh"

namespace axonn {

// Eight consecutive elements of a row, kept as loaded: 4 words of bf16 or 8
// of fp32.  n of them exist (the others are neither read nor written).  Full
// vectors are 16-byte aligned: base pointers and leading dimensions are
// checked by the host and columns are multiples of 8.  Every element is
// touched once, so loads and stores are marked streaming (not kept in the
// caches at the expense of others); load<false> is for those that are read
// again.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint32_t w[4];
  template <bool kOnce = true>
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 8) {
      const uint4* q = reinterpret_cast<const uint4*>(p);
      const uint4 a = kOnce ? __ldcs(q) : *q;
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (2 * j < n ? p[2 * j] : 0u) | ((2 * j + 1 < n ? p[2 * j + 1] : 0u) << 16);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float w[8];
  template <bool kOnce = true>
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 8) {
      const float4* q = reinterpret_cast<const float4*>(p);
      const float4 a = kOnce ? __ldcs(q) : q[0], b = kOnce ? __ldcs(q + 1) : q[1];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < n ? p[j] : 0.0f;
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = w[j];
  }
};
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&x)[8]) {
  const uint32_t w[4] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                         pack_bf16(x[6], x[7])};
  if (n >= 8) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&x)[8]) {
  if (n >= 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = x[j];
  }
}

}  // namespace axonn
