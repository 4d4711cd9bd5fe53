// Device arithmetic shared by the fused epilogues and the elementwise
// kernels: the activations with their derivatives, the counter-based
// generator behind dropout, and 32-column row segments in bf16 and fp32.
// Everything is fp32 between the loads and the one rounding at the store.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "epilogue.h"
#include "ptx.cuh"

namespace axonn {

constexpr float kEpiLog2e = 1.4426950408889634f;

// 2^x and 1/x by the SFU (PTX ex2.approx and rcp.approx: relative errors
// near 2^-22 and 1 ulp; results below 2^-126 flush to zero), far inside the
// rounding of a bf16 output and of the order of an fp32 sum's own error.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x); NaN stays NaN, and the ends are 0 and 1.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.0f + ex2_approx(-kEpiLog2e * x)); }

// The tanh form of GELU, 0.5 z (1 + tanh(u)) with u = c0 (z + c1 z^3), is
// z sigmoid(2u).
constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2/pi)
constexpr float kGeluC1 = 0.044715f;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float gelu_tanh_gate(float z) {
  return sigmoid(2.0f * kGeluC0 * z * fmaf(kGeluC1 * z, z, 1.0f));
}

// The normal distribution's tail beyond |z| and its density at z.  The tail
// is half of erfc(|z| / sqrt 2) by formula 7.1.26 of Abramowitz and Stegun
// (C. Hastings' rational approximation): t (a1 + .. + a5 t^4) e^(-z^2 / 2),
// t = 1 / (1 + p |z| / sqrt 2), within 1.5e-7 of erfc, which leaves 1e-7 of z
// in GELU.  It costs two SFU steps, half of what erfcf costs, and the slope
// uses the exponential again.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  e = ex2_approx(-0.5f * kEpiLog2e * z * z);
  const float t = rcp_approx(fmaf(0.3275911f * kRsqrt2, fabsf(z), 1.0f));
  float h = fmaf(t, 1.061405429f, -1.453152027f);
  h = fmaf(t, h, 1.421413741f);
  h = fmaf(t, h, -0.284496736f);
  h = fmaf(t, h, 0.254829592f);
  return 0.5f * h * t * e;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // NaN stays
  if constexpr (ACT == kActGelu) {
    float e;
    const float h = normal_tail(z, e);
    return z * (z >= 0.0f ? 1.0f - h : h);
  }
  if constexpr (ACT == kActGeluTanh) return z * gelu_tanh_gate(z);
  if constexpr (ACT == kActSilu) return z * sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == kActGelu) {
    float e;
    const float h = normal_tail(z, e);
    return fmaf(z * kRsqrt2Pi, e, z >= 0.0f ? 1.0f - h : h);
  }
  if constexpr (ACT == kActGeluTanh) {
    // with s = sigmoid(2u): s + z s (1 - s) 2 u'(z).  z is clamped where the
    // gate has long saturated, so that its square cannot overflow.
    const float s = gelu_tanh_gate(z);
    const float c = fminf(fmaxf(z, -64.0f), 64.0f);
    return fmaf(c * s * (1.0f - s), 2.0f * kGeluC0 * fmaf(3.0f * kGeluC1 * c, c, 1.0f), s);
  }
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    const float c = fminf(fmaxf(z, -1e4f), 1e4f);
    return fmaf(c * s, 1.0f - s, s);
  }
  return 1.0f;
}

// v[j] = act(v[j]), and v[j] *= act'(z_j) for z in bf16 pairs, over 16 values;
// the switch is outside the loop.
__device__ __forceinline__ void apply_act16(int act, float* v) {
#define AXONN_EACH(A)                        \
  case A:                                    \
    _Pragma("unroll") for (int j = 0; j < 16; ++j) v[j] = act_value<A>(v[j]); \
    break
  switch (act) {
    AXONN_EACH(kActRelu);
    AXONN_EACH(kActGelu);
    AXONN_EACH(kActGeluTanh);
    AXONN_EACH(kActSilu);
    default: break;
  }
#undef AXONN_EACH
}
__device__ __forceinline__ void apply_slope16(int act, float* v, const uint32_t* z) {
#define AXONN_EACH(A)                                                                     \
  case A:                                                                                 \
    _Pragma("unroll") for (int j = 0; j < 16; ++j) v[j] *=                                \
        act_slope<A>(__uint_as_float((j & 1) ? z[j >> 1] & 0xFFFF0000u : z[j >> 1] << 16)); \
    break
  switch (act) {
    AXONN_EACH(kActRelu);
    AXONN_EACH(kActGelu);
    AXONN_EACH(kActGeluTanh);
    AXONN_EACH(kActSilu);
    default: break;
  }
#undef AXONN_EACH
}

// ------------------------------------------------------------------ dropout
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC'11): ten rounds of two 32 x 32 -> 64 bit products.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// One call's generator: the two words the caller keeps on the device.
struct DropRng {
  uint64_t seed, offset;
};
__device__ __forceinline__ DropRng load_rng(const DropoutArgs& d) {
  DropRng r{0, 0};
  if (d.thr != 0) {
    r.seed = d.rng[0];
    r.offset = d.rng[1];
  }
  return r;
}

// The generator's four words for the eight consecutive columns 8 * col8 ..
// of one row.
__device__ __forceinline__ uint4 drop_words(const DropRng& g, uint32_t row, uint32_t col8) {
  return philox4x32_10(make_uint4(col8, row, static_cast<uint32_t>(g.offset),
                                  static_cast<uint32_t>(g.offset >> 32)),
                       static_cast<uint32_t>(g.seed), static_cast<uint32_t>(g.seed >> 32));
}

// v[j] = base[j] + D(v[j]) over those columns, in one rounding.  A half word
// u is at least thr exactly when u 2^16 is above `above` = thr 2^16 - 1, the
// upper half whatever lies below it.  A dropped element becomes 0 whatever it
// was (an infinity or NaN there does not survive), hence a select.
__device__ __forceinline__ void drop8_add(const DropoutArgs& d, const uint4& r, float* v, const float* base) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = fmaf(v[2 * j], d.scale, base[2 * j]);
    const float hi = fmaf(v[2 * j + 1], d.scale, base[2 * j + 1]);
    v[2 * j] = (w[j] << 16) > d.above ? lo : base[2 * j];
    v[2 * j + 1] = w[j] > d.above ? hi : base[2 * j + 1];
  }
}
__device__ __forceinline__ void drop8(const DropoutArgs& d, const DropRng& g, uint32_t row, uint32_t col8,
                                      float* v) {
  const uint4 r = drop_words(g, row, col8);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (w[j] << 16) > d.above ? v[2 * j] * d.scale : 0.0f;
    v[2 * j + 1] = w[j] > d.above ? v[2 * j + 1] * d.scale : 0.0f;
  }
}

// ------------------------------------------------------------------ rows
__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// 16 consecutive elements of a row, as loaded: bf16 in 8 words or fp32 in
// 16.  `n` of them exist; a full segment is 16-byte aligned (base pointers
// and leading dimensions are checked by the host, columns are multiples of
// 16), a short one is read element by element so that nothing past the row's
// end is touched.
template <bool kF32>
struct Row16 {
  uint32_t w[kF32 ? 16 : 8];
  __device__ __forceinline__ void load(const void* base, int64_t at, int n) {
    if constexpr (kF32) {
      const float* p = reinterpret_cast<const float*>(base) + at;
      if (n >= 16) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint4 a = reinterpret_cast<const uint4*>(p)[v];
          w[4 * v] = a.x;
          w[4 * v + 1] = a.y;
          w[4 * v + 2] = a.z;
          w[4 * v + 3] = a.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = j < n ? __float_as_uint(p[j]) : 0u;
      }
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
      if (n >= 16) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint4 a = reinterpret_cast<const uint4*>(p)[v];
          w[4 * v] = a.x;
          w[4 * v + 1] = a.y;
          w[4 * v + 2] = a.z;
          w[4 * v + 3] = a.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t lo = 2 * j < n ? p[2 * j] : 0u;
          const uint32_t hi = 2 * j + 1 < n ? p[2 * j + 1] : 0u;
          w[j] = lo | (hi << 16);
        }
      }
    }
  }
  __device__ __forceinline__ float value(int j) const {  // j known at compile time
    if constexpr (kF32) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  }
};

// Asks for a line to be brought into L2.
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The linear cross entropy keeps a logit z of a piece as its distance below
// its group's maximum m, (m - z) log2 e, in steps of 2^-11 up to 2^5: half a
// step changes e^(z - m) by 2^-12 ln 2, a twentieth of the bf16 rounding that
// the probability gets afterwards (an exponential kept in bf16 would be
// rounded twice: the gradients' error against 64 bits was 1.6 times that of
// one rounding).  kCeFar stands for anything from 2^-32 of the maximum down,
// whose probability is taken as 0.
constexpr float kCeStep = 2048.0f;
constexpr uint32_t kCeFar = 65535;

}  // namespace axonn
