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
constexpr int kStatThreads = 256;

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
// memory is written to, which the first pair makes sure of at no cost.
__device__ __forceinline__ void cluster_arrive() {
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
constexpr int kUnroll = 2;  // vectors a thread loads at a time; the next ones are on their way meanwhile

// Streams a share: f(logits, vector) for every whole vector, a thread every
// kThreads-th, ascending; next(batch) before each batch of kUnroll of them.
template <int kThreads, typename T, class Next, class F>
__device__ __forceinline__ void stream_share(const T* row, const Share& sh, Next&& next, F&& f) {
  constexpr int kStep = kThreads * kUnroll;
  auto load = [&](Vec8<T>(&v)[kUnroll], int i0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + kThreads * u < sh.end) v[u].load(row + static_cast<int64_t>(i0 + kThreads * u) * 8, 8);
  };
  auto use = [&](const Vec8<T>(&v)[kUnroll], int i0) {
    next(i0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + kThreads * u < sh.end) {
        float x[8];
        v[u].values(x);
        f(x, i0 + kThreads * u);
      }
  };
  Vec8<T> v[kUnroll], w[kUnroll];
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
// not change: while it streams, a thread keeps for each of its kSegments
// segments (vectors that follow each other in its own sequence) the largest
// logit, as the rank of the last index of the first vector that has it.  A
// segment has an entry at least that good, so the k-th best of these numbers
// is a bound that k entries reach.  An entry that reaches it lies in a segment
// that does: only those are read again, and what reaches the bound is the
// candidates.  The bound is sought among the threads' best segments alone,
// between the k-th and the (1.5 k + 4)-th.
constexpr int kSegments = 8;

template <int kThreads>
struct TopShared {
  union {
    uint64_t segment[kSegments][kThreads];
    uint64_t entry[kSegments * kThreads];  // the candidates, after the segments
  };
  uint16_t again[kSegments * kThreads];  // segments that reach the bound
  uint64_t part[kThreads / 32];
  uint64_t list[kMaxTop];
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

// A number that at least k (or else all) of the threads' numbers reach, and at
// most `most` unless fewer numbers than k are not 0.  All are different, and
// below `hi`.
__device__ __forceinline__ uint64_t bound_of(uint64_t mine, int k, int most, uint64_t hi) {
  int n = __syncthreads_count(mine != 0);
  if (n <= most) return 1;
  // downwards from hi in growing steps, then by halves: n reach lo, fewer than k hi
  uint64_t lo = hi, step = static_cast<uint64_t>(1) << 50;
  for (n = 0; n < k; step <<= 2) {
    hi = lo;
    lo = step < hi && step < (static_cast<uint64_t>(1) << 62) ? hi - step : 1;
    n = __syncthreads_count(mine >= lo);
  }
  while (n > most && hi - lo > 1) {
    const uint64_t mid = lo + (hi - lo) / 2;
    const int at = __syncthreads_count(mine >= mid);
    if (at >= k) {
      lo = mid;
      n = at;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// Leaves the k largest of n > k entries, all different, in sh.list.
template <int kThreads>
__device__ __noinline__ void cut_entries(TopShared<kThreads>& sh, int n, int k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t lo = 1, hi = ~static_cast<uint64_t>(0);
  int reach = n;
  while (reach > k) {
    const uint64_t mid = lo + (hi - lo) / 2;
    int c = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) c += sh.entry[i] >= mid ? 1 : 0;
    c = __reduce_add_sync(kAll, c);
    if (lane == 0) sh.part[warp] = static_cast<uint64_t>(c);
    __syncthreads();
    c = 0;
    for (int w = 0; w < kThreads / 32; ++w) c += static_cast<int>(sh.part[w]);
    __syncthreads();
    if (c >= k) {
      lo = mid;
      reach = c;
    } else {
      hi = mid;
    }
  }
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (sh.entry[i] >= lo) sh.list[atomicAdd(&sh.listed, 1)] = sh.entry[i];
  __syncthreads();
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
// A cluster takes a row, a CTA a share of it.  Each CTA sums its share and
// finds its own list; they meet in the shared memory of the cluster's first
// CTA, which joins them in order and writes.
template <typename T, bool kEntropy, bool kTop, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident) logprobs_kernel(const LogprobArgs p) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kWarps = kThreads / 32;
  __shared__ RowSums parts[kWarps];
  __shared__ RowSums shares[kMaxCluster];                        // the first CTA's: the others' sums
  __shared__ uint64_t lists[kTop ? kMaxCluster * kMaxTop : 1];   // and lists, each in order
  __shared__ TopShared<kTop ? kThreads : 32> top;
  const int64_t V = p.in.vocab;
  const int64_t t = cluster_id_x();
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  const int tid = static_cast<int>(threadIdx.x);
  const float inv = 1.0f / p.in.temperature, c = kEpiLog2e * inv;
  if (p.in.keep && p.in.keep[t] == 0) {
    if (rank != 0) return;
    if (tid == 0) {
      if (p.logprob) p.logprob[t] = 0.0f;
      if (p.entropy) p.entropy[t] = 0.0f;
      if (p.lse) p.lse[t] = 0.0f;
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
    stream_share<kThreads>(
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
    stream_share<kThreads>(row, sh, [](int) {}, [&](const float(&x)[8], int) { add<kEntropy>(r, x, c); });
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
    const uint64_t bound = bound_of(best, k, k + k / 2 + 4, hi);
    unsigned reach = 0;
#pragma unroll
    for (int j = 0; j < kSegments; ++j)
      if (best >= bound && top.segment[j][tid] >= bound) reach |= 1u << j;
    for (; reach; reach &= reach - 1)
      top.again[atomicAdd(&top.segments, 1)] = static_cast<uint16_t>((__ffs(static_cast<int>(reach)) - 1) * kThreads + tid);
    __syncthreads();
    // from here the segments' memory takes the candidates
    constexpr int kRoom = kSegments * kThreads;
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
#pragma unroll
        for (int e = 0; e < 8; ++e) offer(x[e], static_cast<int64_t>(i) * 8 + e);
      }
    }
    if (tid < sh.tail) offer(logit_at(row + sh.tail_at + tid), sh.tail_at + tid);
    __syncthreads();
    int n = top.entries;
    const uint64_t* entry = top.entry;
    if (n > kRoom) {
      // more candidates than there is room for (a share of which a few segments
      // hold nearly everything that is large): one by one
      uint64_t at = ~static_cast<uint64_t>(0);
      for (int j = 0; j < k; ++j) {
        at = next_entry<kThreads>(row, sh, at, top.part);
        if (tid == 0) top.list[j] = at;
      }
      __syncthreads();
      n = k;
      entry = top.list;
    } else if (n > kThreads) {
      cut_entries(top, n, k);
      n = k;
      entry = top.list;
    }
    // each candidate's place is the number of larger ones
    const float lns = log2f(r.s) * kRowLn2;
    auto write = [&](int place, uint64_t e, float m, float s, float ln_s) {
      const int64_t at = t * p.ld_top + place;
      if (p.top_index) p.top_index[at] = static_cast<int32_t>(rank_index(e));
      // as far below the maximum as fp32 reaches
      if (p.top_logprob) p.top_logprob[at] = s == 0.0f ? -INFINITY : fmaf(rank_value(e) - m, inv, -ln_s);
    };
    if (tid < n) {
      const uint64_t e = entry[tid];
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) place += entry[i] > e ? 1 : 0;
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
      r = shares[0];
      for (int i = 1; i < ctas; ++i) join<kEntropy>(r, shares[i], c);
      const float ln_s = log2f(r.s) * kRowLn2;
      // an entry's place: its own in its list, and those before it in the others
      for (int i = tid; i < ctas * p.k; i += kThreads) {
        const uint64_t e = lists[i];
        const int of = i / p.k;
        int place = i - of * p.k;
        if (e == 0) continue;
        for (int l = 0; l < ctas; ++l) {
          if (l == of) continue;
          int before = 0, behind = p.k;  // entries above e: a prefix of the list
          while (before < behind) {
            const int mid = (before + behind) / 2;
            if (lists[l * p.k + mid] > e) before = mid + 1;
            else behind = mid;
          }
          place += before;
        }
        if (place < p.k) write(place, e, r.m, r.s, ln_s);
      }
    }
  } else if (ctas > 1) {
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
    r = shares[0];
    for (int i = 1; i < ctas; ++i) join<kEntropy>(r, shares[i], c);
  }
  if (tid == 0) {
    const float log2s = log2f(r.s), lns = log2s * kRowLn2;  // -inf for a row of -inf
    if (p.logprob) p.logprob[t] = !inside ? 0.0f : r.s == 0.0f ? -INFINITY : fmaf(own - r.m, inv, -lns);
    if (p.lse) p.lse[t] = fmaf(r.m, inv, lns);
    if (kEntropy) p.entropy[t] = r.s == 0.0f ? 0.0f : (log2s - r.a / r.s) * kRowLn2;
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

constexpr int kDistThreads = 256;
constexpr int kHeldBytes = 64 << 10;  // of a row that a CTA holds, where 8 CTAs can hold a row so
constexpr int kMostHeld = 200 << 10;

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
__device__ __forceinline__ uint4 unit_of(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint4 unit_of(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Asynchronous copies of 16 bytes into shared memory, in groups of the thread
// that asks for them.
__device__ __forceinline__ void copy_unit(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A cluster takes a row, a CTA a share of it, which it copies to its shared
// memory (as much of it as there is room for: `room` units; a thread copies
// what it will use itself, so nothing waits for another).  The softmax's sums
// meet in every CTA's shared memory; then the gradient comes from the copy: p
// everywhere, and the list's entries, p - q, by the threads that have them.
// Without a gradient nothing is kept.  The row whose cluster finishes last
// adds up the losses in a fixed order.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDistThreads) distill_kernel(const DistillArgs p, int room) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kWarps = kDistThreads / 32, kPer = kUnit<T>, kGroups = 4;
  extern __shared__ __align__(16) uint4 held[];
  __shared__ RowSums parts[kWarps];
  __shared__ RowSums shares[kMaxCluster];  // of every CTA of the cluster
  __shared__ int length;
  __shared__ bool last, teaches;
  float* list_q = reinterpret_cast<float*>(held + room);  // log2 of the list's weights, then q
  float* list_x = list_q + p.k;                           // the row's logits there
  int32_t* list_at = reinterpret_cast<int32_t*>(list_x + p.k);
  const int64_t V = p.in.vocab;
  const int64_t t = cluster_id_x();
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  const int tid = static_cast<int>(threadIdx.x);
  const float c = kEpiLog2e * (1.0f / p.in.temperature);
  const int n = *p.kept;
  const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
  T* out = kGrad ? static_cast<T*>(p.dlogits) + t * p.ld_dlogits : nullptr;
  const Share sh = share_of(V);
  // the share in units; its logits are those from `lo` to before `hi`
  const int units = (sh.end - sh.first) * (8 / kPer);
  const int64_t lo = static_cast<int64_t>(sh.first) * 8, hi = sh.tail ? V : static_cast<int64_t>(sh.end) * 8;
  const uint4* src = reinterpret_cast<const uint4*>(row + lo);
  const bool counts = row_counts(p, t);
  if (counts) {
    if (ctas > 1) cluster_arrive();
    if (tid == 0) length = p.k;
    const int keep = kGrad ? min(units, room) : 0;
    const int each = (keep + kGroups * kDistThreads - 1) / (kGroups * kDistThreads);  // units of a thread and group
    if (kGrad) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        for (int e = 0; e < each; ++e) {
          const int i = tid + kDistThreads * (g * each + e);
          if (i < keep) copy_unit(held + i, src + i);
        }
        copy_commit();
      }
    }
    __syncthreads();
    // the list; every CTA has all of it, with the logits that it needs: the
    // first CTA all of them, for the loss
    for (int j = tid; j < p.k; j += kDistThreads) {
      const int32_t at = p.top_index[t * p.ld_top + j];
      list_at[j] = at;
      if (at >= 0 && at < V) {
        list_q[j] = p.top_logit[t * p.ld_top + j];
        if (rank == 0 || (at >= lo && at < hi)) list_x[j] = logit_at(row + at);
      } else {
        atomicMin(&length, j);
      }
    }
    // the sums of the share: what is held as it arrives, the rest from memory
    RowSums r;
    auto take = [&](const uint4& v) {
      float x[kPer];
      unit_values<T>(v, x);
      add<false>(r, x, c);
    };
    if (kGrad) {
      auto take_group = [&](int g) {
        for (int e = 0; e < each; ++e) {
          const int i = tid + kDistThreads * (g * each + e);
          if (i < keep) take(held[i]);
        }
      };
      copy_wait<3>();
      take_group(0);
      copy_wait<2>();
      take_group(1);
      copy_wait<1>();
      take_group(2);
      copy_wait<0>();
      take_group(3);
      for (int i = keep + tid; i < units; i += kDistThreads) take(src[i]);
    } else {
      stream_share<kDistThreads>(row, sh, [](int) {}, [&](const float(&x)[8], int) { add<false>(r, x, c); });
    }
    if (sh.tail && tid == kDistThreads - 1) {
      float x[8];
      tail_values(row, sh, x);
      add<false>(r, x, c);
    }
    r = join_block<false, kWarps>(r, c, parts);
    if (ctas > 1) {
      cluster_wait();  // every CTA has begun
      if (tid < ctas) put_remote(&shares[rank], tid, r);
      __syncwarp();
      cluster_sync();
      r = shares[0];
      for (int i = 1; i < ctas; ++i) join<false>(r, shares[i], c);
    }
    const int len = length;  // at least 1
    if (tid < 32) {
      float top = -INFINITY;
      for (int j = tid; j < len; j += 32) top = fmaxf(top, list_q[j]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      const float base = top > -INFINITY ? top : 0.0f;
      float sum = 0.0f;
      for (int j = tid; j < len; j += 32) {
        const float d = (list_q[j] - base) * c;
        list_q[j] = d;
        sum += ex2_approx(d);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
      const float log2w = log2f(sum), log2s = log2f(r.s);
      float kl = 0.0f;
      for (int j = tid; j < len; j += 32) {
        const float lq = list_q[j] - log2w;
        const float q = sum == 0.0f ? 0.0f : ex2_approx(list_q[j]) / sum;
        list_q[j] = q;
        if (rank == 0) {
          const float lp = r.s == 0.0f ? -INFINITY : (list_x[j] - r.m) * c - log2s;
          if (q != 0.0f) kl = fmaf(q, lq - lp, kl);
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) kl += __shfl_xor_sync(kAll, kl, o);
      if (tid == 0) {
        if (rank == 0) p.token_loss[t] = kl * (kRowLn2 * p.in.temperature * p.in.temperature);
        teaches = sum != 0.0f;
      }
    }
    if (kGrad) {
      __syncthreads();
      const float scale = p.grad_scale * p.in.temperature / static_cast<float>(n);
      const float share = r.s == 0.0f || !teaches ? 0.0f : scale / r.s;
      const float m = r.m > -INFINITY ? r.m : 0.0f;
      const F2 m2 = f2(-m), c2 = f2(c), share2 = f2(share);
      uint4* dst = reinterpret_cast<uint4*>(out + lo);
      auto give = [&](int i, const uint4& v) {
        float x[kPer];
        unit_values<T>(v, x);
#pragma unroll
        for (int j = 0; j < kPer; j += 2)
          split(mul2(ex2_2(mul2(add2(f2(x[j], x[j + 1]), m2), c2)), share2), x[j], x[j + 1]);
        __stcs(dst + i, unit_of(x));
      };
#pragma unroll 4
      for (int i = tid; i < keep; i += kDistThreads) give(i, held[i]);
      for (int i = keep + tid; i < units; i += kDistThreads) give(i, src[i]);
      if (tid < sh.tail)
        put_logit(out + sh.tail_at + tid, ex2_approx((logit_at(row + sh.tail_at + tid) - m) * c) * share);
      __syncthreads();
      for (int j = tid; j < len; j += kDistThreads) {
        const int32_t at = list_at[j];
        if (at < lo || at >= hi) continue;
        float q = 0.0f;
        for (int i = 0; i < len; ++i)  // an index given twice teaches twice
          if (list_at[i] == at) q += list_q[i];
        put_logit(out + at, fmaf(ex2_approx((list_x[j] - m) * c), share, -scale * q));
      }
    }
  } else {
    if (rank == 0 && tid == 0) p.token_loss[t] = 0.0f;
    if (kGrad) {
      uint4* dst = reinterpret_cast<uint4*>(out + lo);
      for (int i = tid; i < units; i += kDistThreads) __stcs(dst + i, make_uint4(0, 0, 0, 0));
      if (tid < sh.tail) put_logit(out + sh.tail_at + tid, 0.0f);
    }
  }
  if (rank != 0) return;
  // the mean: token_loss in order, by the row that finishes last
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(reinterpret_cast<unsigned*>(p.loss), 1u) == static_cast<unsigned>(p.in.rows) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f;
  for (int64_t i = tid; i < p.in.rows; i += kDistThreads) sum += __ldcg(p.token_loss + i);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if ((tid & 31) == 0) parts[tid >> 5].s = sum;
  __syncthreads();
  if (tid == 0) {
    float total = 0.0f;
    for (int w = 0; w < kWarps; ++w) total += parts[w].s;
    *p.loss = n > 0 ? total / static_cast<float>(n) : 0.0f;
  }
}

// CTAs a row: as many as fill the GPU's places a few times over, each with
// some thousands of logits.
int row_cluster(int64_t rows, int64_t vocab, int sms) {
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster < int64_t{12} * sms && vocab / (2 * cluster) >= 4096) cluster *= 2;
  return cluster;
}

}  // namespace

cudaError_t logprobs_launch(const LogprobArgs& a, int sms, bool pdl, cudaStream_t stream) {
  const int cluster = row_cluster(a.in.rows, a.in.vocab, sms);
  const dim3 grid(static_cast<unsigned>(a.in.rows * cluster));
  const int which = (a.in.f32 ? 4 : 0) + (a.entropy ? 2 : 0) + (a.k > 0 ? 1 : 0);
  using Kernel = void (*)(LogprobArgs);
  static constexpr Kernel kKernels[8] = {
      logprobs_kernel<uint16_t, false, false, kStatThreads, 6>, logprobs_kernel<uint16_t, false, true, kStatThreads, 5>,
      logprobs_kernel<uint16_t, true, false, kStatThreads, 5>,  logprobs_kernel<uint16_t, true, true, kStatThreads, 4>,
      logprobs_kernel<float, false, false, kStatThreads, 4>,    logprobs_kernel<float, false, true, kStatThreads, 4>,
      logprobs_kernel<float, true, false, kStatThreads, 4>,     logprobs_kernel<float, true, true, kStatThreads, 4>};
  return launch_clusters(kKernels[which], grid, static_cast<unsigned>(cluster), kStatThreads, pdl, stream, 0, a);
}

cudaError_t logprobs_bwd_launch(const LogprobBwdArgs& a, bool pdl, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.in.vocab + kBwdCols - 1) / kBwdCols),
                  static_cast<unsigned>(std::min<int64_t>(a.in.rows, 65535)));
  auto kernel = a.in.f32 ? (a.dentropy ? logprobs_bwd_kernel<float, true> : logprobs_bwd_kernel<float, false>)
                         : (a.dentropy ? logprobs_bwd_kernel<uint16_t, true> : logprobs_bwd_kernel<uint16_t, false>);
  return launch_after(kernel, grid, kBwdThreads, pdl, stream, a);
}

cudaError_t distill_init() {
  for (auto kernel : {distill_kernel<float, true>, distill_kernel<uint16_t, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMostHeld + 12 * kMaxList);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t distill_launch(const DistillArgs& a, int sms, bool pdl, cudaStream_t stream) {
  const cudaError_t e = launch_after(distill_count_kernel, dim3(1), 1024, pdl, stream, a);
  if (e != cudaSuccess || a.in.rows == 0) return e;
  int cluster = row_cluster(a.in.rows, a.in.vocab, sms);
  int held = 0;
  if (a.dlogits) {
    const int64_t vectors = a.in.vocab / 8, bytes = a.in.f32 ? 32 : 16;
    auto share = [&] { return (vectors + cluster - 1) / cluster * bytes; };
    while (cluster < kMaxCluster && share() > kHeldBytes) cluster *= 2;
    held = static_cast<int>(std::min<int64_t>(share(), kMostHeld));
  }
  const dim3 grid(static_cast<unsigned>(a.in.rows * cluster));
  auto kernel = a.in.f32 ? (a.dlogits ? distill_kernel<float, true> : distill_kernel<float, false>)
                         : (a.dlogits ? distill_kernel<uint16_t, true> : distill_kernel<uint16_t, false>);
  return launch_clusters(kernel, grid, static_cast<unsigned>(cluster), kDistThreads, pdl, stream,
                         static_cast<size_t>(held + 12 * a.k), a, held / 16);
}

}  // namespace axonn
