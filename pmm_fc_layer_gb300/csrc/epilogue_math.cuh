// Device arithmetic shared by the fused epilogues and the elementwise
// kernels: the activations with their derivatives, the counter-based
// generator behind dropout, and 16-column row segments in bf16 and fp32.
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

// Two fp32 numbers in a register pair: one instruction for both (the f32x2
// forms of sm_100 and later; each half rounds as its scalar form does).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 min2(F2 a, float b) {
  float x, y;
  split(a, x, y);
  return f2(fminf(x, b), fminf(y, b));
}
// Each half's magnitude at most b > 0, its sign kept; NaN stays.
__device__ __forceinline__ F2 clamp2(F2 a, float b) {
  float x, y;
  split(a, x, y);
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(x) : "f"(b));
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(y) : "f"(b));
  return f2(x, y);
}
__device__ __forceinline__ F2 ex2_2(F2 a) {
  float x, y;
  split(a, x, y);
  return f2(ex2_approx(x), ex2_approx(y));
}
__device__ __forceinline__ F2 rcp_2(F2 a) {
  float x, y;
  split(a, x, y);
  return f2(rcp_approx(x), rcp_approx(y));
}

// 1 / (1 + 2^-a): with a = x log2 e the logistic function; NaN stays NaN, and
// the ends are 0 and 1.  `neg` is -a.
__device__ __forceinline__ F2 logistic2(F2 neg) { return rcp_2(add2(ex2_2(neg), f2(1.0f))); }

// The tanh form of GELU, 0.5 z (1 + tanh(u)) with u = c0 (z + c1 z^3), is
// z s, s = sigmoid(2u) = 1 / (1 + e), e = 2^(-2u log2 e); -2u log2 e = z
// (kTanhA + kTanhB z^2).
constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2/pi)
constexpr float kGeluC1 = 0.044715f;
constexpr float kTanhA = -2.0f * kGeluC0 * kEpiLog2e;
constexpr float kTanhB = kTanhA * kGeluC1;
constexpr float kRsqrt2 = 0.7071067811865476f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;
__device__ __forceinline__ F2 gelu_tanh_exponent2(F2 z, F2 zz) {
  return mul2(z, fma2(zz, f2(kTanhB), f2(kTanhA)));
}

// The normal distribution function at z, and e = e^(-z^2 / 2).  Its tail
// beyond |z| is erfc(x) / 2 at x = |z| / sqrt 2, which is
//   t (b0 + b1 t + .. + b7 t^7) e,   t = 1 / (1 + p x), p = 0.43:
// a minimax fit of e^(x^2) erfc(x) / 2 over 0 <= x <= 9.4 (where e has left
// the fp32 range), relatively within 1e-7 in exact arithmetic and 4e-7 in fp32,
// 1/2 at 0.  Relatively, since GELU's negative tail is nothing but this number:
// a form bound absolutely by 1.5e-7 was 0.16 % off at z = -5 and 1 % at -8.
// With the exponential's argument (three roundings of z^2/2) the tail is within
// 1.5 z^2 2^-24 + 2^-19 of itself.  It costs two SFU steps, half of what erfcf
// costs, and the slope uses the exponential again.
constexpr float kTailP = 0.43f * kRsqrt2;
__device__ __forceinline__ F2 normal_cdf2(F2 z, F2& e) {
  float z0, z1;
  split(z, z0, z1);
  e = ex2_2(mul2(mul2(z, f2(-0.5f * kEpiLog2e)), z));
  const F2 t = rcp_2(fma2(f2(fabsf(z0), fabsf(z1)), f2(kTailP), f2(1.0f)));
  F2 h = fma2(t, f2(0.036614003f), f2(-0.154214349f));
  h = fma2(t, h, f2(0.190222684f));
  h = fma2(t, h, f2(-0.041401893f));
  h = fma2(t, h, f2(0.122668828f));
  h = fma2(t, h, f2(0.102698375f));
  h = fma2(t, h, f2(0.122152819f));
  h = fma2(t, h, f2(0.121259533f));
  h = mul2(mul2(h, t), e);
  float h0, h1;
  split(h, h0, h1);
  return f2(z0 >= 0.0f ? 1.0f - h0 : h0, z1 >= 0.0f ? 1.0f - h1 : h1);
}

// act and its slope at two points.
template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 z) {
  if constexpr (ACT == kActRelu) {
    float x, y;
    split(z, x, y);
    return f2(x < 0.0f ? 0.0f : x, y < 0.0f ? 0.0f : y);  // NaN stays
  }
  if constexpr (ACT == kActGelu) {
    F2 e;
    return mul2(z, normal_cdf2(z, e));
  }
  if constexpr (ACT == kActGeluTanh) {
    // z^2 stops where the gate has long saturated, so that nothing overflows
    return mul2(z, logistic2(gelu_tanh_exponent2(z, min2(mul2(z, z), 4096.0f))));
  }
  if constexpr (ACT == kActSilu) return mul2(z, logistic2(mul2(z, f2(-kEpiLog2e))));
  return z;
}

template <int ACT>
__device__ __forceinline__ F2 act_slope2(F2 z) {
  if constexpr (ACT == kActRelu) {
    float x, y;
    split(z, x, y);
    return f2(x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x), y > 0.0f ? 1.0f : (y <= 0.0f ? 0.0f : y));
  }
  if constexpr (ACT == kActGelu) {
    F2 e;
    const F2 cdf = normal_cdf2(z, e);
    return fma2(mul2(z, f2(kRsqrt2Pi)), e, cdf);
  }
  if constexpr (ACT == kActGeluTanh) {
    // s + z s (1 - s) 2 u'(z).  1 - s = e s: as a difference it would keep
    // s's rounding, which z 2 u'(z) makes 2^-19 of at z = 5.  At z = 10 the slope
    // is 1 and at -10 it is 0 in fp32, with e at 2^-126 and 2^126: there z stops.
    z = clamp2(z, 10.0f);
    const F2 zz = mul2(z, z);
    const F2 e = ex2_2(gelu_tanh_exponent2(z, zz)), s = rcp_2(add2(e, f2(1.0f)));
    const F2 w = mul2(z, mul2(mul2(e, s), s));
    return fma2(w, fma2(zz, f2(6.0f * kGeluC0 * kGeluC1), f2(2.0f * kGeluC0)), s);
  }
  if constexpr (ACT == kActSilu) {
    const F2 s = logistic2(mul2(z, f2(-kEpiLog2e)));
    return fma2(z, fma2(mul2(s, f2(-1.0f)), s, s), s);
  }
  return f2(1.0f);
}

// v[j] = act(v[j]), and v[j] *= act'(z_j) for z in bf16 pairs, over 16 values;
// the switch is outside the loop.
template <int ACT, int N>
__device__ __forceinline__ void act_values(float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 2) split(act_value2<ACT>(f2(v[j], v[j + 1])), v[j], v[j + 1]);
}
template <int ACT, int N>
__device__ __forceinline__ void act_slopes(float* v, const uint32_t* z) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const uint32_t w = z[j >> 1];
    const F2 s = act_slope2<ACT>(f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)));
    split(mul2(f2(v[j], v[j + 1]), s), v[j], v[j + 1]);
  }
}
__device__ __forceinline__ void apply_act16(int act, float* v) {
  switch (act) {
    case kActRelu: act_values<kActRelu, 16>(v); break;
    case kActGelu: act_values<kActGelu, 16>(v); break;
    case kActGeluTanh: act_values<kActGeluTanh, 16>(v); break;
    case kActSilu: act_values<kActSilu, 16>(v); break;
    default: break;
  }
}
__device__ __forceinline__ void apply_slope16(int act, float* v, const uint32_t* z) {
  switch (act) {
    case kActRelu: act_slopes<kActRelu, 16>(v, z); break;
    case kActGelu: act_slopes<kActGelu, 16>(v, z); break;
    case kActGeluTanh: act_slopes<kActGeluTanh, 16>(v, z); break;
    case kActSilu: act_slopes<kActSilu, 16>(v, z); break;
    default: break;
  }
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
