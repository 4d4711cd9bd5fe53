// Arithmetic shared by the kernels over rows of vocabulary logits: the running
// sums of a softmax, their joins, and a row's cut into shares.
//
// With z = logits / tau, m the row's largest logit and c = log2(e) / tau,
//   S = sum_v 2^((x_v - m) c),   A = sum_v 2^((x_v - m) c) (x_v - m) c,
//   ln p_v = (x_v - m) / tau - ln S,   H = ln S - ln 2 A / S.
// The difference is taken before the product, so that a row of finite logits
// of any size (a mask of the type's lowest value throughout, too) gives its
// own distribution.  (m, S, A) are running fp32 numbers of each thread, joined
// in a fixed order.  A row without a finite logit (all -inf) has S = 0: its
// probabilities are taken as 0.  A NaN or +inf makes S a NaN, and with it
// everything that the row gives but the order of its list.
#pragma once
#include <algorithm>

#include "vec8.cuh"
#include "vocab_rows.h"

namespace axonn {

constexpr float kRowLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xFFFFFFFFu;

template <typename T>
__device__ __forceinline__ float logit_at(const T* p) {
  if constexpr (sizeof(T) == 2) return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  else return *p;
}

__device__ __forceinline__ void put_logit(uint16_t* p, float x) { *p = static_cast<uint16_t>(pack_bf16(x, 0.0f)); }
__device__ __forceinline__ void put_logit(float* p, float x) { *p = x; }

// A row's (m, S, A), or a part's.
struct RowSums {
  float m = -INFINITY, s = 0.0f, a = 0.0f;
};

// Adds N logits; returns the largest of them.
template <bool kEntropy, int N>
__device__ __forceinline__ float add(RowSums& r, const float (&x)[N], float c) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < N; ++j) top = fmaxf(top, x[j]);
  if (top > r.m) {
    if (r.m > -INFINITY) {
      const float d = (r.m - top) * c, f = ex2_approx(d);
      if (kEntropy) r.a = f * fmaf(r.s, fmaxf(d, -256.0f), r.a);
      r.s *= f;
    }
    r.m = top;
  }
  const F2 m = f2(r.m > -INFINITY ? -r.m : 0.0f), c2 = f2(c);
  F2 s = f2(0.0f), a = f2(0.0f);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const F2 d = mul2(add2(f2(x[2 * j], x[2 * j + 1]), m), c2);
    const F2 e = ex2_2(d);
    s = add2(s, e);
    if (kEntropy) {
      // 2^d is 0 below -126; the product must be too where d is -inf
      float d0, d1;
      split(d, d0, d1);
      a = fma2(e, f2(fmaxf(d0, -256.0f), fmaxf(d1, -256.0f)), a);
    }
  }
  float s0, s1;
  split(s, s0, s1);
  r.s += s0 + s1;
  if (kEntropy) {
    split(a, s0, s1);
    r.a += s0 + s1;
  }
  return top;
}

// A part's sums from another maximum, m >= r.m.  A part without a finite logit
// has S = 0, or NaN, which stays.
template <bool kEntropy>
__device__ __forceinline__ void shift_to(RowSums& r, float m, float c) {
  const float d = r.m > -INFINITY ? (r.m - m) * c : 0.0f, f = ex2_approx(d);
  if (kEntropy) r.a = f * fmaf(r.s, fmaxf(d, -256.0f), r.a);
  r.s *= f;
  r.m = m;
}

// The sum of kParts parts in order, or of the first n.
template <bool kEntropy, int kParts>
__device__ __forceinline__ RowSums join_parts(const RowSums* parts, int n, float c) {
  RowSums r;
#pragma unroll
  for (int w = 0; w < kParts; ++w)
    if (w < n) r.m = fmaxf(r.m, parts[w].m);
#pragma unroll
  for (int w = 0; w < kParts; ++w)
    if (w < n) {
      RowSums o = parts[w];
      shift_to<kEntropy>(o, r.m, c);
      r.s += o.s;
      if (kEntropy) r.a += o.a;
    }
  return r;
}

// A warp's sum of its threads' parts, known to every lane: the maximum first,
// so that the additions need no exponentials between them.
template <bool kEntropy>
__device__ __forceinline__ RowSums join_warp(RowSums r, float c) {
  float m = r.m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  shift_to<kEntropy>(r, m, c);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    r.s += __shfl_xor_sync(kAll, r.s, o);
    if (kEntropy) r.a += __shfl_xor_sync(kAll, r.a, o);
  }
  return r;
}

// The sum of kParts parts that every lane of a warp can read (a power of two),
// known to every lane: a lane takes one, and they join as a tree.
template <bool kEntropy, int kParts>
__device__ __forceinline__ RowSums join_parts_warp(const RowSums* parts, float c) {
  RowSums r = parts[threadIdx.x % kParts];
  float m = r.m;
#pragma unroll
  for (int o = 1; o < kParts; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  shift_to<kEntropy>(r, m, c);
#pragma unroll
  for (int o = 1; o < kParts; o <<= 1) {
    r.s += __shfl_xor_sync(kAll, r.s, o);
    if (kEntropy) r.a += __shfl_xor_sync(kAll, r.a, o);
  }
  return r;
}

// The block's sum of the threads' parts, known to every thread.
template <bool kEntropy, int kWarps>
__device__ __forceinline__ RowSums join_block(RowSums r, float c, RowSums* parts) {
  r = join_warp<kEntropy>(r, c);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = r;
  __syncthreads();
  return join_parts_warp<kEntropy, kWarps>(parts, c);
}

// ------------------------------------------------------------------ shares of a row
// A row is cut over the CTAs of a cluster, whole vectors of eight to each; the
// last one has the row's last V mod 8 logits too.
struct Share {
  int first, end;  // its vectors
  int tail;        // logits behind the last whole vector, or 0
  int64_t tail_at;
};
__device__ __forceinline__ Share share_of(int64_t V) {
  const int whole = static_cast<int>(V >> 3), ctas = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank()), each = (whole + ctas - 1) / ctas;
  Share s;
  s.first = min(whole, rank * each);
  s.end = min(whole, s.first + each);
  s.tail = rank == ctas - 1 ? static_cast<int>(V & 7) : 0;
  s.tail_at = V & ~static_cast<int64_t>(7);
  return s;
}

// The halves of a cluster's barrier: CTAs must have begun before their shared
// memory is written to, which the first pair makes sure of at no cost.  A warp's
// lanes take an aligned barrier together, whatever branch they come from.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Writes into the shared memory of a CTA of the cluster.
__device__ __forceinline__ void put_remote(const RowSums* at, int rank, const RowSums& r) {
  const uint32_t a = mapa_shared(smem_addr(at), static_cast<uint32_t>(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(r.m) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(r.s) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(r.a) : "memory");
}
__device__ __forceinline__ void put_remote(const uint64_t* at, int rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_addr(at), static_cast<uint32_t>(rank))),
               "l"(v)
               : "memory");
}

constexpr int kMaxCluster = 8;
// Vectors a thread loads at a time, the next ones on their way meanwhile: two,
// a power of two where segments are counted in them; three where registers
// allow (8192 x 128256 with entropy 314 us against 322; fp32 spills, 1003 x
// 50257 49 against 40).
constexpr int kUnroll = 2;
template <typename T>
constexpr int kUnrollSums = sizeof(T) == 2 ? 3 : 2;

// Streams a share: f(logits, vector) for every whole vector, a thread every
// kThreads-th, ascending; next(batch) before each batch of kVectors of them.  kOnce: not read again.
template <int kThreads, int kVectors, bool kOnce, typename T, class Next, class F>
__device__ __forceinline__ void stream_share(const T* row, const Share& sh, Next&& next, F&& f) {
  constexpr int kStep = kThreads * kVectors;
  auto load = [&](Vec8<T>(&v)[kVectors], int i0) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
      if (i0 + kThreads * u < sh.end) v[u].template load<kOnce>(row + static_cast<int64_t>(i0 + kThreads * u) * 8, 8);
  };
  auto use = [&](const Vec8<T>(&v)[kVectors], int i0) {
    next(i0);
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
      if (i0 + kThreads * u < sh.end) {
        float x[8];
        v[u].values(x);
        f(x, i0 + kThreads * u);
      }
  };
  Vec8<T> v[kVectors], w[kVectors];
  int i = sh.first + static_cast<int>(threadIdx.x);
  load(v, i);
  while (i < sh.end) {
    load(w, i + kStep);
    use(v, i);
    i += kStep;
    if (i >= sh.end) break;
    load(v, i + kStep);
    use(w, i);
    i += kStep;
  }
}

// The eight places of a share's tail; -inf where there is none.
template <typename T>
__device__ __forceinline__ void tail_values(const T* row, const Share& sh, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = j < sh.tail ? logit_at(row + sh.tail_at + j) : -INFINITY;
}

// 16 bytes of a row: 8 bf16 or 4 fp32 logits.
template <typename T>
constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
template <typename T>
__device__ __forceinline__ void unit_values(const uint4& v, float (&x)[kUnit<T>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < kUnit<T>; ++j)
    x[j] = __uint_as_float(sizeof(T) == 4 ? w[j] : (j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
}
template <typename T>
__device__ __forceinline__ uint4 no_unit() {  // of -inf
  const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
  return make_uint4(w, w, w, w);
}
// Their largest logit, two bf16 at a time (a NaN is passed over).
__device__ __forceinline__ __nv_bfloat162 pair_max(uint32_t a, uint32_t b) {
  return __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
}
template <typename T, int U>
__device__ __forceinline__ float units_max(const uint4 (&v)[U]) {
  float top = -INFINITY;
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 m = __hmax2(pair_max(v[0].x, v[0].y), pair_max(v[0].z, v[0].w));
#pragma unroll
    for (int u = 1; u < U; ++u) m = __hmax2(m, __hmax2(pair_max(v[u].x, v[u].y), pair_max(v[u].z, v[u].w)));
    top = fmaxf(__low2float(m), __high2float(m));
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[4];
      unit_values<T>(v[u], x);
      top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
    }
  }
  return top;
}
__device__ __forceinline__ uint4 unit_of(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint4 unit_of(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Adds units, without A.
template <typename T, int U>
__device__ __forceinline__ void add_units(RowSums& r, const uint4 (&v)[U], float c) {
  const float top = units_max<T>(v);
  if (top > r.m) {
    if (r.m > -INFINITY) r.s *= ex2_approx((r.m - top) * c);
    r.m = top;
  }
  const F2 m = f2(r.m > -INFINITY ? -r.m : 0.0f), c2 = f2(c);
  F2 s[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[kUnit<T>];
    unit_values<T>(v[u], x);
#pragma unroll
    for (int j = 0; j < kUnit<T>; j += 2) {
      F2& to = s[(j / 2) & 1];
      to = add2(to, ex2_2(mul2(add2(f2(x[j], x[j + 1]), m), c2)));
    }
  }
  float s0, s1;
  split(add2(s[0], s[1]), s0, s1);
  r.s += s0 + s1;
}

// CTAs a row: up to four on each SM in all, each with some thousands of logits.
// More only add to what a CTA costs whatever its share, and rows in shares of
// which some wait for a place take longer than whole rows (sums of 128256 words
// with a cold L2: 100 rows 14.0 us by 4 CTAs a row, 16.0 by 2 or 8; 200 rows
// 18.7 by 2, 20.8 by 4; 400 rows 26.3 whole, 32.4 by 2; lists of 20 alike).
inline int row_cluster(int64_t rows, int64_t vocab, int sms) {
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster * 2 <= int64_t{4} * sms && vocab / (2 * cluster) >= 4096) cluster *= 2;
  return cluster;
}

}  // namespace axonn
