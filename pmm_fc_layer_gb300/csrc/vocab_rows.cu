// Kernels over rows of vocabulary logits: log probabilities of given tokens
// with entropy and top alternatives, their way back, and distillation from a
// teacher's lists of logits.
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
#include <algorithm>

#include "launch.h"
#include "vec8.cuh"
#include "vocab_rows.h"

namespace axonn {
namespace {

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

// Adds eight logits.
template <bool kEntropy>
__device__ __forceinline__ void add8(RowSums& r, const float (&x)[8], float c) {
  const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
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
  for (int j = 0; j < 4; ++j) {
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
}

// Joins two parts.  A part without a finite logit has S = 0, or NaN, which stays.
template <bool kEntropy>
__device__ __forceinline__ void join(RowSums& r, const RowSums& o, float c) {
  const float m = fmaxf(r.m, o.m);
  const float d0 = r.m > -INFINITY ? (r.m - m) * c : 0.0f, d1 = o.m > -INFINITY ? (o.m - m) * c : 0.0f;
  const float f0 = ex2_approx(d0), f1 = ex2_approx(d1);
  if (kEntropy) r.a = f0 * fmaf(r.s, fmaxf(d0, -256.0f), r.a) + f1 * fmaf(o.s, fmaxf(d1, -256.0f), o.a);
  r.s = r.s * f0 + o.s * f1;
  r.m = m;
}

// The block's sum of the threads' parts, known to every thread.
template <bool kEntropy, int kWarps>
__device__ __forceinline__ RowSums join_block(RowSums r, float c, RowSums* parts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    RowSums other;
    other.m = __shfl_xor_sync(kAll, r.m, o);
    other.s = __shfl_xor_sync(kAll, r.s, o);
    if (kEntropy) other.a = __shfl_xor_sync(kAll, r.a, o);
    join<kEntropy>(r, other, c);
  }
  if (lane == 0) parts[warp] = r;
  __syncthreads();
  r = parts[0];
#pragma unroll 4
  for (int w = 1; w < kWarps; ++w) join<kEntropy>(r, parts[w], c);
  return r;
}

// ------------------------------------------------------------------ logprobs
constexpr int kStatThreads = 512;
constexpr int kBatch = 4;  // vectors of eight a thread loads before it uses them

// Adds a row's logits to the threads' parts: a thread every kThreads-th vector.
template <bool kEntropy, int kThreads, typename T>
__device__ __forceinline__ RowSums row_sums(const T* row, int64_t V, float c) {
  RowSums r;
  for (int64_t base = 8 * threadIdx.x; base < V; base += 8 * kThreads * kBatch) {
    Vec8<T> v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = base + 8 * kThreads * u;
      if (i < V) v[u].load(row + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = base + 8 * kThreads * u;
      if (i < V) {
        float x[8];
        v[u].values(x);
        if (V - i < 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j >= V - i) x[j] = -INFINITY;
        }
        add8<kEntropy>(r, x, c);
      }
    }
  }
  return r;
}

// The order of a list as whole numbers: a NaN above every number, -0 as 0,
// and of equal logits the lower index first.  0 is below every entry, and
// 2^64 - 1 above.
constexpr uint32_t kNanKey = 0xFFC00000u;  // an infinity's is 0xFF800000
__device__ __forceinline__ uint64_t rank_of(float x, int64_t index) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t key = x != x ? kNanKey : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int64_t rank_index(uint64_t r) { return 0xFFFFFFFFu - static_cast<uint32_t>(r); }
__device__ __forceinline__ float rank_value(uint64_t r) {
  const uint32_t key = static_cast<uint32_t>(r >> 32);
  if (key == kNanKey) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// The largest entry of the row below `below`, known to every thread.
template <int kThreads, typename T>
__device__ __forceinline__ uint64_t next_entry(const T* row, int64_t V, uint64_t below, uint64_t* parts) {
  uint64_t best = 0;
  for (int64_t i = threadIdx.x; i < V; i += kThreads) {
    const uint64_t r = rank_of(logit_at(row + i), i);
    if (r < below && r > best) best = r;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) best = max(best, __shfl_xor_sync(kAll, best, o));
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = best;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) best = max(best, parts[w]);
  __syncthreads();
  return best;
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kStatThreads) logprobs_kernel(const LogprobArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ RowSums parts[kStatThreads / 32];
  __shared__ uint64_t best[kStatThreads / 32];
  const int64_t V = p.in.vocab;
  const float inv = 1.0f / p.in.temperature, c = kEpiLog2e * inv;
  for (int64_t t = blockIdx.x; t < p.in.rows; t += gridDim.x) {
    if (p.in.keep && p.in.keep[t] == 0) {
      if (threadIdx.x == 0) {
        if (p.logprob) p.logprob[t] = 0.0f;
        if (p.entropy) p.entropy[t] = 0.0f;
        if (p.lse) p.lse[t] = 0.0f;
      }
      for (int j = threadIdx.x; j < p.k; j += kStatThreads) {
        if (p.top_index) p.top_index[t * p.ld_top + j] = -1;
        if (p.top_logprob) p.top_logprob[t * p.ld_top + j] = 0.0f;
      }
      continue;
    }
    const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
    const RowSums r = join_block<kEntropy, kStatThreads / 32>(row_sums<kEntropy, kStatThreads>(row, V, c), c, parts);
    const float log2s = log2f(r.s), lns = log2s * kRowLn2;  // -inf for a row of -inf
    // ln p of a logit x, which may be as far below the maximum as fp32 reaches
    auto lnp = [&](float x) {
      return r.s == 0.0f ? -INFINITY : fmaf(x - r.m, inv, -lns);
    };
    if (threadIdx.x == 0) {
      if (p.logprob) {
        const int32_t y = p.tokens[t];
        p.logprob[t] = y >= 0 && y < V ? lnp(logit_at(row + y)) : 0.0f;
      }
      if (p.lse) p.lse[t] = fmaf(r.m, inv, lns);
      if (kEntropy) p.entropy[t] = r.s == 0.0f ? 0.0f : (log2s - r.a / r.s) * kRowLn2;
    }
    uint64_t at = ~static_cast<uint64_t>(0);
    for (int j = 0; j < p.k; ++j) {
      at = next_entry<kStatThreads>(row, V, at, best);
      if (threadIdx.x == 0) {
        if (p.top_index) p.top_index[t * p.ld_top + j] = static_cast<int32_t>(rank_index(at));
        if (p.top_logprob) p.top_logprob[t * p.ld_top + j] = lnp(rank_value(at));
      }
    }
    __syncthreads();  // parts and best are written again for the next row
  }
}

// ------------------------------------------------------------------ logprobs, backward
constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;
constexpr int kBwdCols = 8 * kBwdThreads * kBwdVecs;

// Blocks over (row, kBwdCols columns).
template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(const LogprobBwdArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t V = p.in.vocab;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBwdCols + 8 * threadIdx.x;
  const float inv = 1.0f / p.in.temperature;
  for (int64_t t = blockIdx.y; t < p.in.rows; t += gridDim.y) {
    const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
    T* out = static_cast<T*>(p.dlogits) + t * p.ld_dlogits;
    const float lse = p.lse[t];
    float g = 0.0f, h = 0.0f, entropy = 0.0f;
    int64_t y = -1;
    if (p.dlogprob) {
      y = p.tokens[t];
      if (y >= 0 && y < V) g = p.dlogprob[t] * inv;
      else y = -1;
    }
    if (kEntropy) {
      h = p.dentropy[t] * inv;
      entropy = p.entropy[t];
    }
    // nothing to say, or a row of -inf: zeros, and nothing is read
    const bool zero = (p.in.keep && p.in.keep[t] == 0) || lse == -INFINITY || (g == 0.0f && h == 0.0f);
    Vec8<T> v[kBwdVecs];
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
      const int64_t i = first + 8 * kBwdThreads * u;
      if (i < V && !zero) v[u].load(row + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)));
    }
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
      const int64_t i = first + 8 * kBwdThreads * u;
      if (i < V) {
        float x[8] = {};
        if (!zero) {
          v[u].values(x);
          const int64_t at = y - i;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float lnp = fmaf(x[j], inv, -lse);
            const float prob = ex2_approx(lnp * kEpiLog2e);
            float w = g;
            if (kEntropy) w = fmaf(h, fmaxf(lnp, -256.0f) + entropy, g);
            x[j] = -w * prob;
            if (at == j) x[j] += g;
          }
        }
        store8(out + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)), x);
      }
    }
  }
}

// ------------------------------------------------------------------ distillation
// A list ends at its first index outside the vocabulary, so a row counts where
// it is kept and its first index is inside.
__device__ __forceinline__ bool row_counts(const DistillArgs& p, int64_t t) {
  if (p.in.keep && p.in.keep[t] == 0) return false;
  const int32_t first = p.top_index[t * p.ld_top];
  return first >= 0 && first < p.in.vocab;
}

__global__ void __launch_bounds__(1024) distill_count_kernel(const DistillArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int counts[32];
  int n = 0;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < p.in.rows; t += 1024) n += row_counts(p, t) ? 1 : 0;
  n = __reduce_add_sync(kAll, n);
  if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    n = __reduce_add_sync(kAll, counts[threadIdx.x]);
    if (threadIdx.x == 0) {
      *p.kept = n;
      *p.loss = 0.0f;  // as a word: no block of the next kernel has finished
    }
  }
}

constexpr int kDistThreads = 512;

// The sums of the row's softmax and of the list's, the row's loss, and (in a
// second pass over the row, which L2 still has) the gradient: p everywhere,
// then the list's entries, p - q, by the threads that have them.  The block
// that finishes last adds up the losses in a fixed order.
template <typename T>
__global__ void __launch_bounds__(kDistThreads) distill_kernel(const DistillArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ RowSums parts[kDistThreads / 32];
  __shared__ float list_q[kMaxList];       // log2 of the list's weights, then q
  __shared__ float list_x[kMaxList];       // the row's logits there
  __shared__ int32_t list_at[kMaxList];
  __shared__ int length;
  __shared__ bool last, teaches;
  const int64_t V = p.in.vocab;
  const float c = kEpiLog2e * (1.0f / p.in.temperature);
  const int n = *p.kept;
  const float scale = n > 0 ? p.grad_scale * p.in.temperature / static_cast<float>(n) : 0.0f;
  for (int64_t t = blockIdx.x; t < p.in.rows; t += gridDim.x) {
    const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
    T* out = p.dlogits ? static_cast<T*>(p.dlogits) + t * p.ld_dlogits : nullptr;
    if (!row_counts(p, t)) {
      if (threadIdx.x == 0) p.token_loss[t] = 0.0f;
      if (out) {
        const float none[8] = {};
        for (int64_t i = 8 * threadIdx.x; i < V; i += 8 * kDistThreads)
          store8(out + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)), none);
      }
      continue;
    }
    if (threadIdx.x == 0) length = p.k;
    __syncthreads();
    for (int j = threadIdx.x; j < p.k; j += kDistThreads) {
      const int32_t at = p.top_index[t * p.ld_top + j];
      list_at[j] = at;
      if (at >= 0 && at < V) {
        list_q[j] = p.top_logit[t * p.ld_top + j];
        list_x[j] = logit_at(row + at);
      } else {
        atomicMin(&length, j);
      }
    }
    const RowSums r = join_block<false, kDistThreads / 32>(row_sums<false, kDistThreads>(row, V, c), c, parts);
    const int len = length;  // at least 1
    const float log2s = log2f(r.s);
    if (threadIdx.x < 32) {
      float top = -INFINITY;
      for (int j = threadIdx.x; j < len; j += 32) top = fmaxf(top, list_q[j]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      const float base = top > -INFINITY ? top : 0.0f;
      float sum = 0.0f;
      for (int j = threadIdx.x; j < len; j += 32) {
        const float d = (list_q[j] - base) * c;
        list_q[j] = d;
        sum += ex2_approx(d);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
      const float log2w = log2f(sum);
      float kl = 0.0f;
      for (int j = threadIdx.x; j < len; j += 32) {
        const float lq = list_q[j] - log2w;
        const float q = sum == 0.0f ? 0.0f : ex2_approx(list_q[j]) / sum;
        const float lp = r.s == 0.0f ? -INFINITY : (list_x[j] - r.m) * c - log2s;
        if (q != 0.0f) kl = fmaf(q, lq - lp, kl);
        list_q[j] = q;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) kl += __shfl_xor_sync(kAll, kl, o);
      if (threadIdx.x == 0) {
        p.token_loss[t] = kl * (kRowLn2 * p.in.temperature * p.in.temperature);
        teaches = sum != 0.0f;
      }
    }
    __syncthreads();
    if (out) {
      const float share = r.s == 0.0f || !teaches ? 0.0f : scale / r.s;
      const float m = r.m > -INFINITY ? r.m : 0.0f;
      for (int64_t i = 8 * threadIdx.x; i < V; i += 8 * kDistThreads) {
        const int w = static_cast<int>(min(static_cast<int64_t>(8), V - i));
        Vec8<T> v;
        v.load(row + i, w);
        float x[8];
        v.values(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ex2_approx((x[j] - m) * c) * share;
        store8(out + i, w, x);
      }
      __syncthreads();
      for (int j = threadIdx.x; j < len; j += kDistThreads) {
        const int32_t at = list_at[j];
        float q = 0.0f;
        for (int i = 0; i < len; ++i)  // an index given twice teaches twice
          if (list_at[i] == at) q += list_q[i];
        put_logit(out + at, fmaf(ex2_approx((list_x[j] - m) * c), share, -scale * q));
      }
    }
    __syncthreads();  // the shared arrays are written again for the next row
  }
  // the mean: token_loss in order, by the block that finishes last
  __shared__ float sums[kDistThreads / 32];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(reinterpret_cast<unsigned*>(p.loss), 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f;
  for (int64_t t = threadIdx.x; t < p.in.rows; t += kDistThreads) sum += __ldcg(p.token_loss + t);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float total = 0.0f;
    for (int w = 0; w < kDistThreads / 32; ++w) total += sums[w];
    *p.loss = n > 0 ? total / static_cast<float>(n) : 0.0f;
  }
}

}  // namespace

cudaError_t logprobs_launch(const LogprobArgs& a, int sms, bool pdl, cudaStream_t stream) {
  (void)sms;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.in.rows, INT32_MAX)));
  auto kernel = a.in.f32 ? (a.entropy ? logprobs_kernel<float, true> : logprobs_kernel<float, false>)
                         : (a.entropy ? logprobs_kernel<uint16_t, true> : logprobs_kernel<uint16_t, false>);
  return launch_after(kernel, grid, kStatThreads, pdl, stream, a);
}

cudaError_t logprobs_bwd_launch(const LogprobBwdArgs& a, bool pdl, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.in.vocab + kBwdCols - 1) / kBwdCols),
                  static_cast<unsigned>(std::min<int64_t>(a.in.rows, 65535)));
  auto kernel = a.in.f32 ? (a.dentropy ? logprobs_bwd_kernel<float, true> : logprobs_bwd_kernel<float, false>)
                         : (a.dentropy ? logprobs_bwd_kernel<uint16_t, true> : logprobs_bwd_kernel<uint16_t, false>);
  return launch_after(kernel, grid, kBwdThreads, pdl, stream, a);
}

cudaError_t distill_launch(const DistillArgs& a, int sms, bool pdl, cudaStream_t stream) {
  (void)sms;
  const cudaError_t e = launch_after(distill_count_kernel, dim3(1), 1024, pdl, stream, a);
  if (e != cudaSuccess || a.in.rows == 0) return e;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.in.rows, INT32_MAX)));
  return launch_after(a.in.f32 ? distill_kernel<float> : distill_kernel<uint16_t>, grid, kDistThreads, pdl, stream, a);
}

}  // namespace axonn
