// Log probabilities of given tokens, with their entropy and the row's top
// alternatives, and the way back through them.  The sums are those of
// vocab_rows.cuh.
#include <algorithm>

#include "launch.h"
#include "vocab_rows.cuh"

namespace axonn {
namespace {

constexpr int kStatThreads = 256;  // the most, and those of blocks in clusters

// ------------------------------------------------------------------ lists
// The order of a list as whole numbers: a NaN above every number, -0 as 0,
// and of equal logits the lower index first.  0 is below every entry, and
// 2^64 - 1 above.
constexpr uint32_t kNanKey = 0xFFC00000u;  // an infinity's is 0xFF800000
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return x != x ? kNanKey : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t rank_of(uint32_t key, uint32_t index) {
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ uint32_t rank_index(uint64_t r) { return 0xFFFFFFFFu - static_cast<uint32_t>(r); }
__device__ __forceinline__ float rank_value(uint64_t r) {
  const uint32_t key = static_cast<uint32_t>(r >> 32);
  if (key == kNanKey) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// How the k largest of a share are found, in work that the logits' values do
// not change but in one case (at the end): while it streams, a thread keeps for each of its kSegments
// segments (vectors that follow each other in its own sequence) the largest
// logit, as the rank of the last index of the first vector that has it.  A
// segment has an entry at least that good, so the k-th best of these numbers
// is a bound that k entries reach.  An entry that reaches it lies in a segment
// that does: only those are read again, and what reaches the bound is the
// candidates.  The bound is sought among the threads' best segments alone,
// between the k-th and a few places (half of k, at most 16, and 4) behind it.
// Where more candidates reach it than kSegments * kThreads, because a few threads'
// segments hold nearly all that is large, the share is read once for each entry of
// the list instead (every row of 4096 x 128256 so, lists of 64: 23.8 ms for 206 us).
constexpr int kSegments = 8;

template <int kThreads>
struct alignas(16) TopShared {
  union {
    uint64_t segment[kSegments][kThreads];
    uint64_t entry[kSegments * kThreads + 2];  // the candidates, after the segments
  };
  uint64_t best[kThreads];  // of each thread's segments
  uint64_t bound;
  uint16_t again[kSegments * kThreads];  // segments that reach the bound
  uint64_t part[kThreads / 32];
  uint64_t list[kThreads];
  int segments, entries, listed;
};

// The largest entry of a share below `below`, known to every thread.
template <int kThreads, typename T>
__device__ __noinline__ uint64_t next_entry(const T* row, const Share sh, uint64_t below, uint64_t* parts) {
  uint64_t best = 0;
  const int64_t end = sh.tail ? sh.tail_at + sh.tail : static_cast<int64_t>(sh.end) * 8;
  for (int64_t i = static_cast<int64_t>(sh.first) * 8 + threadIdx.x; i < end; i += kThreads) {
    const uint64_t r = rank_of(key_of(logit_at(row + i)), static_cast<uint32_t>(i));
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

// A number that at least k numbers reach and at most `most`, where reach(x)
// says how many reach x; all are different and below `hi`, and more than `most`
// reach 1.  Downwards from hi in growing steps, then by halves: n reach lo, fewer
// than k hi.
template <class F>
__device__ __forceinline__ uint64_t seek_bound(int k, int most, uint64_t hi, F&& reach) {
  uint64_t lo = hi, step = static_cast<uint64_t>(1) << 50;
  int n = 0;
  for (; n < k; step <<= 2) {
    hi = lo;
    lo = step < hi && step < (static_cast<uint64_t>(1) << 62) ? hi - step : 1;
    n = reach(lo);
  }
  while (n > most && hi - lo > 1) {
    const uint64_t mid = lo + (hi - lo) / 2;
    const int at = reach(mid);
    if (at >= k) {
      lo = mid;
      n = at;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// That among the block's numbers, or 1 where no more than `most` are not 0.
// One warp's work: it reads them all, and the others wait (every warp counting
// its own, with a barrier for each step, took four times the instructions).
template <int kThreads>
__device__ __forceinline__ uint64_t bound_of(const uint64_t* numbers, int k, int most, uint64_t hi) {
  uint64_t mine[kThreads / 32];
#pragma unroll
  for (int j = 0; j < kThreads / 32; ++j) mine[j] = numbers[(threadIdx.x & 31) + 32 * j];
  auto reach = [&](uint64_t x) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < kThreads / 32; ++j) n += mine[j] >= x ? 1 : 0;
    return __reduce_add_sync(kAll, n);
  };
  return reach(1) <= most ? 1 : seek_bound(k, most, hi, reach);
}

// Of n entries, all different and more than kThreads, leaves at least the k
// largest and at most kThreads as the first ones; returns how many.
template <int kThreads>
__device__ __noinline__ int cut_entries(TopShared<kThreads>& sh, int n, int k, uint64_t hi) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lo = seek_bound(k, kThreads, hi, [&](uint64_t x) {
    int c = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) c += sh.entry[i] >= x ? 1 : 0;
    c = __reduce_add_sync(kAll, c);
    if (lane == 0) sh.part[warp] = static_cast<uint64_t>(c);
    __syncthreads();
    c = 0;
    for (int w = 0; w < kThreads / 32; ++w) c += static_cast<int>(sh.part[w]);
    __syncthreads();
    return c;
  });
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (sh.entry[i] >= lo) sh.list[atomicAdd(&sh.listed, 1)] = sh.entry[i];
  __syncthreads();
  n = sh.listed;
  for (int i = threadIdx.x; i < n; i += kThreads) sh.entry[i] = sh.list[i];
  __syncthreads();
  return n;
}

// The best segments of a share by whole-number order, for rows with a NaN,
// which comparisons of floats pass over.
template <int kThreads, typename T>
__device__ __noinline__ uint64_t segments_of_nan(const T* row, const Share sh, int batches, TopShared<kThreads>& top) {
  uint64_t best = 0;
  for (int j = 0; j < kSegments; ++j) {
    uint64_t seg = 0;
    for (int b = 0; b < batches * kUnroll; ++b) {
      const int i = sh.first + static_cast<int>(threadIdx.x) + kThreads * (j * batches * kUnroll + b);
      if (i >= sh.end) break;
      uint32_t key = 0;
      for (int e = 0; e < 8; ++e) key = max(key, key_of(logit_at(row + static_cast<int64_t>(i) * 8 + e)));
      seg = max(seg, rank_of(key, static_cast<uint32_t>(i) * 8u + 7u));
    }
    top.segment[j][threadIdx.x] = seg;
    best = max(best, seg);
  }
  __syncthreads();
  return best;
}

// ------------------------------------------------------------------ logprobs
// ln p of a logit x from its row's largest: (x - m) / tau - ln S.  Two finite
// logits may be further apart than fp32 reaches, and their z not: the difference is
// that of their halves, which is exact where x - m is (in this order, since x may
// still be on its way: 64 x 128256 fp32 10.1 us, 10.2 by 0.5 x - 0.5 m).
__device__ __forceinline__ float logprob_of(float x, float m, float inv, float ln_s) {
  return fmaf(fmaf(0.5f, x, -0.5f * m), 2.0f * inv, -ln_s);
}

// A cluster takes a row, a CTA a share of it.  Each CTA sums its share and
// finds its own list; they meet in the shared memory of the cluster's first
// CTA, which joins them in order and writes.
// HBM-bound for sums alone: 8192 x 128256 with entropy 305 to 317 us, 6.6 to
// 6.9 TB/s (issue slots 70 % busy; without loads ahead of their use 501).  A
// list of 64 of 128256 costs a quarter more (4096 rows 204 us, 160 without): of
// a block's 70000 cycles the bound takes 2000, the segments that are read again
// 8000, at the latency of a busy memory and with 14 % more traffic, and the
// places 2500.  One row with a list of 20, on 8 CTAs: 6.9 us, 3.4 without.
template <typename T, bool kEntropy, bool kTop, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident) logprobs_kernel(const LogprobArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kWarps = kThreads / 32;
  constexpr bool kClusters = kThreads == kStatThreads;
  __shared__ RowSums parts[kWarps];
  __shared__ RowSums shares[kMaxCluster];                        // the first CTA's: the others' sums
  __shared__ uint64_t lists[kTop && kClusters ? kMaxCluster * kMaxTop : 1];  // and lists, each in order
  __shared__ TopShared<kTop ? kThreads : 32> top;
  const int64_t V = p.in.vocab;
  const int64_t t = cluster_id_x();
  const int rank = kClusters ? static_cast<int>(cluster_ctarank()) : 0;
  const int ctas = kClusters ? static_cast<int>(cluster_nctarank()) : 1;
  const int tid = static_cast<int>(threadIdx.x);
  const float inv = 1.0f / p.in.temperature, c = kEpiLog2e * inv;
  auto put_lse = [&](float m, float log_sum, float lse) {
    if (p.lse_parts) {
      p.lse[2 * t] = m;
      p.lse[2 * t + 1] = log_sum;
    } else {
      p.lse[t] = lse;
    }
  };
  if (p.in.keep && p.in.keep[t] == 0) {
    if (rank != 0) return;
    if (tid == 0) {
      if (p.logprob) p.logprob[t] = 0.0f;
      if (p.entropy) p.entropy[t] = 0.0f;
      if (p.lse) put_lse(0.0f, 0.0f, 0.0f);
    }
    for (int j = tid; j < p.k; j += kThreads) {
      if (p.top_index) p.top_index[t * p.ld_top + j] = -1;
      if (p.top_logprob) p.top_logprob[t * p.ld_top + j] = 0.0f;
    }
    return;
  }
  if (ctas > 1) cluster_arrive();
  const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
  const Share sh = share_of(V);
  float own = -INFINITY;  // the token's logit
  bool inside = false;
  if (rank == 0 && tid == 0 && p.logprob) {
    const int32_t y = p.tokens[t];
    inside = y >= 0 && y < V;
    if (inside) own = logit_at(row + y);
  }

  // the sums, and the largest logit of each segment
  RowSums r;
  uint64_t best = 0;
  int batches = 1;  // of a segment, a power of two
  if constexpr (kTop) {
    const int all = (sh.end - sh.first + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    while (batches * kSegments < all) batches *= 2;
    if (tid == 0) top.segments = top.entries = top.listed = 0;
    float seg_m = -INFINITY;
    int seg_at = 0, j = -1, left = 0;
    auto flush = [&]() {
      const uint64_t seg = rank_of(key_of(seg_m), static_cast<uint32_t>(seg_at) * 8u + 7u);
      top.segment[j][tid] = seg;
      best = max(best, seg);
    };
    stream_share<kThreads, kUnroll, false>(
        row, sh,
        [&](int i) {
          if (left == 0) {
            if (j >= 0) flush();
            ++j;
            left = batches;
            seg_m = -INFINITY;
            seg_at = i;
          }
          --left;
        },
        [&](const float(&x)[8], int i) {
          const float m = add<kEntropy>(r, x, c);
          if (m > seg_m) {
            seg_m = m;
            seg_at = i;
          }
        });
    if (j >= 0) flush();
    for (++j; j < kSegments; ++j) top.segment[j][tid] = 0;
  } else {
    stream_share<kThreads, kUnrollSums<T>, true>(row, sh, [](int) {},
                                                 [&](const float(&x)[8], int) { add<kEntropy>(r, x, c); });
  }
  if (sh.tail && tid == kThreads - 1) {
    float x[8];
    tail_values(row, sh, x);
    add<kEntropy>(r, x, c);
  }
  r = join_block<kEntropy, kWarps>(r, c, parts);

  if (ctas > 1) {
    cluster_wait();  // every CTA has begun
    if (tid == 0) put_remote(&shares[rank], 0, r);
  }
  if constexpr (kTop) {
    const int64_t have = static_cast<int64_t>(sh.end - sh.first) * 8 + sh.tail;
    const int k = static_cast<int>(min(static_cast<int64_t>(p.k), have));  // of this share
    uint64_t hi = rank_of(key_of(r.m), 0) + 1;
    if (r.s != r.s) {
      best = segments_of_nan<kThreads>(row, sh, batches, top);
      hi = ~static_cast<uint64_t>(0);
    }
    top.best[tid] = best;
    __syncthreads();
    if (tid < 32) {
      const uint64_t b = bound_of<kThreads>(top.best, k, k + min(k / 2, 16) + 4, hi);
      if (tid == 0) top.bound = b;
    }
    __syncthreads();
    const uint64_t bound = top.bound;
    unsigned reach = 0;
    if (best >= bound) {
#pragma unroll
      for (int j = 0; j < kSegments; ++j) reach |= top.segment[j][tid] >= bound ? 1u << j : 0u;
    }
    for (; reach; reach &= reach - 1)
      top.again[atomicAdd(&top.segments, 1)] = static_cast<uint16_t>((__ffs(static_cast<int>(reach)) - 1) * kThreads + tid);
    __syncthreads();
    // from here the segments' memory takes the candidates
    constexpr int kRoom = kSegments * kThreads;
    const float least = rank_value(bound);  // a NaN where the bound is one, or none
    auto offer = [&](float x, int64_t at) {
      const uint64_t e = rank_of(key_of(x), static_cast<uint32_t>(at));
      if (e >= bound) {
        const int place = atomicAdd(&top.entries, 1);
        if (place < kRoom) top.entry[place] = e;
      }
    };
    const int each = __ffs(batches * kUnroll) - 1;  // log2 of a segment's vectors
    for (int w = tid; w < top.segments << each; w += kThreads) {
      const int s = top.again[w >> each], j = s / kThreads;
      const int i = sh.first + s % kThreads + kThreads * ((j << each) + (w & ((1 << each) - 1)));
      if (i < sh.end) {
        Vec8<T> v;
        v.load(row + static_cast<int64_t>(i) * 8, 8);
        float x[8];
        v.values(x);
        unsigned large = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) large |= x[e] < least ? 0u : 1u << e;
        for (; large; large &= large - 1) {
          const int64_t at = static_cast<int64_t>(i) * 8 + __ffs(static_cast<int>(large)) - 1;
          offer(logit_at(row + at), at);
        }
      }
    }
    if (tid < sh.tail) offer(logit_at(row + sh.tail_at + tid), sh.tail_at + tid);
    __syncthreads();
    int n = top.entries;
    if (n > kRoom) {
      // more candidates than there is room for (a share of which a few segments
      // hold nearly everything that is large): one by one
      uint64_t at = ~static_cast<uint64_t>(0);
      for (int j = 0; j < k; ++j) {
        at = next_entry<kThreads>(row, sh, at, top.part);
        if (tid == 0) top.entry[j] = at;
      }
      n = k;
      __syncthreads();
    } else if (n > 2 * kThreads) {
      n = cut_entries(top, n, k, hi);
    }
    // each candidate's place is the number of larger ones
    const float lns = log2f(r.s) * kRowLn2;
    auto write = [&](int place, uint64_t e, float m, float s, float ln_s) {
      const int64_t at = t * p.ld_top + place;
      if (p.top_index) p.top_index[at] = static_cast<int32_t>(rank_index(e));
      if (p.top_logprob) p.top_logprob[at] = s == 0.0f ? -INFINITY : logprob_of(rank_value(e), m, inv, ln_s);
    };
    if (tid == 0 && (n & 1)) top.entry[n] = 0;  // two are read at a time
    __syncthreads();
    for (int at = tid; at < n; at += kThreads) {
      const uint64_t e = top.entry[at];
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < n; i += 2) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(top.entry + i);
        place += two.x > e ? 1 : 0;
        place += two.y > e ? 1 : 0;
      }
      if (place < k) {
        if (ctas == 1) write(place, e, r.m, r.s, lns);
        else put_remote(&lists[rank * p.k + place], 0, e);
      }
    }
    if (ctas > 1) {
      for (int j = k + tid; j < p.k; j += kThreads) put_remote(&lists[rank * p.k + j], 0, 0);
      __syncwarp();
      cluster_sync();
      if (rank != 0) return;
      r = join_parts<kEntropy, kMaxCluster>(shares, ctas, c);
      const float ln_s = log2f(r.s) * kRowLn2;
      // an entry's place: its own in its list, and those above it in the others,
      // a prefix of each; the lists are searched side by side
      int half = 1;
      while (2 * half <= p.k) half *= 2;
      for (int i = tid; i < ctas * p.k; i += kThreads) {
        const uint64_t e = lists[i];
        if (e == 0) continue;
        int above[kMaxCluster] = {};
        for (int step = half; step; step /= 2) {
          uint64_t at[kMaxCluster];  // without a branch, so that the loads go together
#pragma unroll
          for (int l = 0; l < kMaxCluster; ++l) at[l] = lists[min(l, ctas - 1) * p.k + min(above[l] + step, p.k) - 1];
#pragma unroll
          for (int l = 0; l < kMaxCluster; ++l) above[l] += above[l] + step <= p.k && at[l] > e ? step : 0;
        }
        int place = 0;
#pragma unroll
        for (int l = 0; l < kMaxCluster; ++l) place += l < ctas ? above[l] : 0;
        if (place < p.k) write(place, e, r.m, r.s, ln_s);
      }
    }
  } else if (ctas > 1) {
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
    r = join_parts<kEntropy, kMaxCluster>(shares, ctas, c);
  }
  if (tid == 0) {
    const float log2s = log2f(r.s), lns = log2s * kRowLn2;  // -inf for a row of -inf
    if (p.logprob) p.logprob[t] = !inside ? 0.0f : r.s == 0.0f ? -INFINITY : logprob_of(own, r.m, inv, lns);
    if (p.lse) put_lse(r.m, lns, fmaf(r.m, inv, lns));
    if (kEntropy) p.entropy[t] = r.s == 0.0f ? 0.0f : (log2s - r.a / r.s) * kRowLn2;
  }
}

// ------------------------------------------------------------------ logprobs, backward
constexpr int kBwdThreads = 64;
constexpr int kBwdVecs = 4;
constexpr int kBwdCols = 8 * kBwdThreads * kBwdVecs;
// The largest |lse| in one number whose p = e^(z - lse) is worth having: half a
// step of it is then 2^-8 of p, bf16's own rounding.  Beyond it ln S goes under in
// lse (in a row of a mask's -1e9 throughout, p would be 1 everywhere).
constexpr float kLseMost = 65536.0f;

// p comes from the forward's sums: with kParts from the row's largest logit m and
// ln S, as e^((x - m) / tau - ln S), which is right for logits of any size, else
// from lse, as e^(x / tau - lse).
// Blocks over (row, kBwdCols columns).  HBM-bound: 8192 x 128256 with entropy
// 638 us, 6.6 TB/s.  What counts is how soon a block has its loads on their
// way: they are issued before the row's scalars are known (after them 24 us
// more), and from small blocks, of which an SM has 21 to 25 (blocks of 256 threads
// 4 us more, of 64 with eight vectors a thread 14).
template <typename T, bool kEntropy, bool kParts>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(const LogprobBwdArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t V = p.in.vocab;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBwdCols + 8 * threadIdx.x;
  const float inv = 1.0f / p.in.temperature;
  for (int64_t t = blockIdx.y; t < p.in.rows; t += gridDim.y) {
    const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
    T* out = static_cast<T*>(p.dlogits) + t * p.ld_dlogits;
    const bool kept = !p.in.keep || p.in.keep[t] != 0;
    Vec8<T> v[kBwdVecs];
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
      const int64_t i = first + 8 * kBwdThreads * u;
      if (i < V && kept) v[u].load(row + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)));
    }
    const float m = kParts ? p.lse[2 * t] : 0.0f;
    float lse = kParts ? p.lse[2 * t + 1] : p.lse[t];
    const bool empty = lse == -INFINITY;
    if (!kParts && fabsf(lse) > kLseMost) lse = NAN;
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
    // nothing to say, or a row of -inf: zeros
    const bool zero = !kept || (kParts && empty) || (g == 0.0f && h == 0.0f);
    if (!kParts && empty && !zero) {
      // a row of -inf, or one whose lse is below fp32's range
#pragma unroll 1
      for (int n = 0; n < 8 * kBwdVecs; ++n) {
        const int64_t i = first + 8 * kBwdThreads * (n / 8) + n % 8;
        if (i < V) put_logit(out + i, logit_at(row + i) == -INFINITY ? 0.0f : NAN);
      }
      continue;
    }
    const F2 inv2 = f2(inv), m2 = f2(-m), lse2 = f2(-lse), g2 = f2(-g), h2 = f2(-h), entropy2 = f2(entropy);
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
      const int64_t i = first + 8 * kBwdThreads * u;
      if (i < V) {
        float x[8] = {};
        if (!zero) {
          v[u].values(x);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            F2 z = f2(x[j], x[j + 1]);
            if (kParts) z = add2(z, m2);
            const F2 lnp = fma2(z, inv2, lse2);
            const F2 prob = ex2_2(mul2(lnp, f2(kEpiLog2e)));
            F2 w = g2;  // -(g + h (ln p + H)), where p is not 0
            if (kEntropy) {
              float a, b;
              split(lnp, a, b);
              w = fma2(h2, add2(f2(fmaxf(a, -256.0f), fmaxf(b, -256.0f)), entropy2), g2);
            }
            split(mul2(w, prob), x[j], x[j + 1]);
          }
          const int64_t at = y - i;
          if (at >= 0 && at < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (at == j) x[j] += g;
          }
        }
        store8(out + i, static_cast<int>(min(static_cast<int64_t>(8), V - i)), x);
      }
    }
  }
}

// Blocks of kThreads, as many on an SM as their registers allow: 1280 or 1024
// threads.
template <int kThreads>
cudaError_t logprobs_launch_blocks(const LogprobArgs& a, int cluster, bool pdl, cudaStream_t stream) {
  constexpr int kAt5 = std::min(32, 1280 / kThreads), kAt4 = 1024 / kThreads;
  using Kernel = void (*)(LogprobArgs);
  static constexpr Kernel kKernels[8] = {
      logprobs_kernel<uint16_t, false, false, kThreads, kAt5>, logprobs_kernel<uint16_t, false, true, kThreads, kAt5>,
      logprobs_kernel<uint16_t, true, false, kThreads, kAt4>,  logprobs_kernel<uint16_t, true, true, kThreads, kAt4>,
      logprobs_kernel<float, false, false, kThreads, kAt4>,    logprobs_kernel<float, false, true, kThreads, kAt4>,
      logprobs_kernel<float, true, false, kThreads, kAt4>,     logprobs_kernel<float, true, true, kThreads, kAt4>};
  const int which = (a.in.f32 ? 4 : 0) + (a.entropy ? 2 : 0) + (a.k > 0 ? 1 : 0);
  const dim3 grid(static_cast<unsigned>(a.in.rows * cluster));
  return launch_clusters(kKernels[which], grid, static_cast<unsigned>(cluster), kThreads, pdl, stream, 0, a);
}
cudaError_t logprobs_launch_with(const LogprobArgs& a, int threads, int cluster, bool pdl, cudaStream_t stream) {
  if (threads == 32) return logprobs_launch_blocks<32>(a, cluster, pdl, stream);
  if (threads == 64) return logprobs_launch_blocks<64>(a, cluster, pdl, stream);
  if (threads == 128) return logprobs_launch_blocks<128>(a, cluster, pdl, stream);
  return logprobs_launch_blocks<kStatThreads>(a, cluster, pdl, stream);
}

// Threads a block: what a block costs whatever its row is the work of its
// warps, so short rows have few (8192 rows of 2000 words, lists of 8: 15.6 us by
// 32 threads, 21.0 by 64, 26.7 by 128, 48.8 by 256; lists of 20 of 32000 words
// 123 by 64, 111 by 128, 134 by 256).  Long rows, and rows that come one to an
// SM, want as many loads on their way as a block can have (4096 x 128256, lists
// of 20: 271 by 64, 196, 189; 64 rows of 128256 words 39, 21, 12; a mask that
// leaves few rows does the same to long ones), and a list of k comes from the
// best of at least 2 k threads, or better 3 k (lists of 16 of 1000 words 28 by
// 32 threads, 20 by 64; of 32 of 2000 words 42 by 64, 33 by 128).  In between it
// is the number of rows (lists of 20 of 4000 words: 2000 rows 12.9 by 64, 11.0
// by 128; 3000 rows 13.3 and 14.3).
int row_threads(const LogprobArgs& a, int cluster, int sms) {
  const int64_t V = a.in.vocab, bytes = V * (a.in.f32 ? 4 : 2);
  if (cluster > 1 || a.k > 64 || bytes >= (96 << 10) || (V > 8192 && a.in.rows < 4 * sms)) return kStatThreads;
  if (V > 8192 || a.k > 24 || a.in.rows < 4 * sms) return 128;
  if (a.k <= 10 && (V <= 2048 || (V <= 6144 && a.in.rows >= 24 * sms))) return 32;
  return a.in.rows >= 16 * sms ? 64 : 128;
}

}  // namespace

cudaError_t logprobs_launch(const LogprobArgs& a, int sms, bool pdl, cudaStream_t stream) {
  const int cluster = row_cluster(a.in.rows, a.in.vocab, sms);
  return logprobs_launch_with(a, row_threads(a, cluster, sms), cluster, pdl, stream);
}

cudaError_t logprobs_bwd_launch(const LogprobBwdArgs& a, bool pdl, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.in.vocab + kBwdCols - 1) / kBwdCols),
                  static_cast<unsigned>(std::min<int64_t>(a.in.rows, 65535)));
  using Kernel = void (*)(LogprobBwdArgs);
  static constexpr Kernel kKernels[8] = {
      logprobs_bwd_kernel<uint16_t, false, false>, logprobs_bwd_kernel<uint16_t, false, true>,
      logprobs_bwd_kernel<uint16_t, true, false>,  logprobs_bwd_kernel<uint16_t, true, true>,
      logprobs_bwd_kernel<float, false, false>,    logprobs_bwd_kernel<float, false, true>,
      logprobs_bwd_kernel<float, true, false>,     logprobs_bwd_kernel<float, true, true>};
  const Kernel kernel = kKernels[(a.in.f32 ? 4 : 0) + (a.dentropy ? 2 : 0) + (a.lse_parts ? 1 : 0)];
  return launch_after(kernel, grid, kBwdThreads, pdl, stream, a);
}

}  // namespace axonn
