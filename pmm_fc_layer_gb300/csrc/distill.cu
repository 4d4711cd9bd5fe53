// Distillation from a teacher's lists of logits: the loss of each row, their
// mean, and its gradient.  The sums are those of vocab_rows.cuh.
#include <algorithm>

#include "launch.h"
#include "vocab_rows.cuh"

namespace axonn {
namespace {

// A list ends at its first index outside the vocabulary, so a row counts where
// it is kept and its first index is inside.  Both are asked for at once.
__device__ __forceinline__ bool row_counts(const DistillArgs& p, int64_t t) {
  const int32_t first = p.top_index[t * p.ld_top];
  const bool kept = !p.in.keep || p.in.keep[t] != 0;
  return kept && first >= 0 && first < p.in.vocab;
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

constexpr int kHeldBytes = 64 << 10;  // of a row that a CTA holds, where 8 CTAs can hold a row so
constexpr int kMostHeld = 200 << 10;

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

// Counts a row whose loss this thread has written; true for the last of them.
__device__ __forceinline__ bool distill_row_done(const DistillArgs& p) {
  __threadfence();
  return atomicAdd(reinterpret_cast<unsigned*>(p.loss), 1u) == static_cast<unsigned>(p.in.rows) - 1;
}

// The mean of the rows' losses, by the block that knows them all written: a
// thread every kThreads-th row in order, then the warps' sums in order.
template <int kThreads>
__device__ __forceinline__ void mean_of_rows(const DistillArgs& p, RowSums* parts) {
  __threadfence();
  float total = 0.0f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < p.in.rows; i += kThreads) total += __ldcg(p.token_loss + i);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) total += __shfl_xor_sync(kAll, total, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5].s = total;
  __syncthreads();
  if (threadIdx.x != 0) return;
  total = 0.0f;
  for (int w = 0; w < kThreads / 32; ++w) total += parts[w].s;
  const int n = *p.kept;
  *p.loss = n > 0 ? total / static_cast<float>(n) : 0.0f;
}

// A cluster takes a row, a CTA a share of it, which it copies to its shared
// memory (as much of it as there is room for: `room` units; a thread copies
// what it will use itself, so nothing waits for another).  The list's weights
// are worked out while the copies are on their way.  The softmax's sums meet in
// every CTA's shared memory; then the gradient comes from the copy: p
// everywhere, and the list's entries, p - q, by the threads that have them.
// Without a gradient nothing is kept.  The row whose cluster finishes last
// adds up the losses in a fixed order.
// For few rows or short ones, where latencies bound it: 100 x 128256 16.4 us,
// 16 x 1003 7 us with the counting kernel.  A cluster's launch and barriers cost
// an SM about a microsecond a CTA, which is why many long rows go through a
// ring instead (below).
template <typename T, bool kGrad, int kDistThreads>
__global__ void __launch_bounds__(kDistThreads) distill_kernel(const DistillArgs p, int room) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kWarps = kDistThreads / 32, kPer = kUnit<T>, kGroups = 4;
  extern __shared__ __align__(16) uint4 held[];
  __shared__ RowSums parts[kWarps];
  __shared__ RowSums shares[kMaxCluster];  // of every CTA of the cluster
  __shared__ int length;
  __shared__ bool last;
  __shared__ float list_sum;
  float* list_q = reinterpret_cast<float*>(held + room);  // logits, distances (log2), weights, q
  float* list_x = list_q + p.k;                           // the row's logits there
  int32_t* list_at = reinterpret_cast<int32_t*>(list_x + p.k);
  const int64_t V = p.in.vocab;
  const int64_t t = cluster_id_x();
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  const int tid = static_cast<int>(threadIdx.x);
  const float c = kEpiLog2e * (1.0f / p.in.temperature);
  const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
  T* out = kGrad ? static_cast<T*>(p.dlogits) + t * p.ld_dlogits : nullptr;
  const Share sh = share_of(V);
  // the share in units; its logits are those from `lo` to before `hi`
  const int units = (sh.end - sh.first) * (8 / kPer);
  const int64_t lo = static_cast<int64_t>(sh.first) * 8, hi = sh.tail ? V : static_cast<int64_t>(sh.end) * 8;
  const uint4* src = reinterpret_cast<const uint4*>(row + lo);
  // a thread's entry of the list (the first one of it, where k is longer than
  // the block) is asked for beside what says whether the row counts
  int32_t at = -1;
  float value = 0.0f;
  if (tid < p.k) {
    at = p.top_index[t * p.ld_top + tid];
    value = p.top_logit[t * p.ld_top + tid];
  }
  const int n = *p.kept;
  if (!row_counts(p, t)) {
    if (rank == 0 && tid == 0) p.token_loss[t] = 0.0f;
    if (kGrad) {
      uint4* dst = reinterpret_cast<uint4*>(out + lo);
      for (int i = tid; i < units; i += kDistThreads) __stcs(dst + i, make_uint4(0, 0, 0, 0));
      if (tid < sh.tail) put_logit(out + sh.tail_at + tid, 0.0f);
    }
    if (rank != 0) return;
    if (tid == 0) last = distill_row_done(p);
  } else {
    if (ctas > 1) cluster_arrive();
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
    if (tid == 0) length = p.k;
    __syncthreads();
    // the list; every CTA has all of it, with the logits that it needs: the
    // first CTA all of them, for the loss
    for (int j = tid; j < p.k; j += kDistThreads) {
      if (j != tid) {
        at = p.top_index[t * p.ld_top + j];
        value = p.top_logit[t * p.ld_top + j];
      }
      list_at[j] = at;
      list_q[j] = value;
      if (at < 0 || at >= V) atomicMin(&length, j);
      else if (rank == 0 || (at >= lo && at < hi)) list_x[j] = logit_at(row + at);
    }
    __syncthreads();
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
      if (tid == 0) list_sum = sum;
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
      stream_share<kDistThreads, kUnrollSums<T>, true>(row, sh, [](int) {},
                                                       [&](const float(&x)[8], int) { add<false>(r, x, c); });
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
      r = join_parts<false, kMaxCluster>(shares, ctas, c);
    }
    const float sum = list_sum;
    if (rank == 0 && tid < 32) {
      const float log2w = log2f(sum), log2s = log2f(r.s);
      float kl = 0.0f;
      for (int j = tid; j < len; j += 32) {
        const float lq = list_q[j] - log2w;
        const float q = sum == 0.0f ? 0.0f : ex2_approx(list_q[j]) / sum;
        const float lp = r.s == 0.0f ? -INFINITY : (list_x[j] - r.m) * c - log2s;
        if (q != 0.0f) kl = fmaf(q, lq - lp, kl);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) kl += __shfl_xor_sync(kAll, kl, o);
      if (tid == 0) {
        p.token_loss[t] = kl * (kRowLn2 * p.in.temperature * p.in.temperature);
        last = distill_row_done(p);
      }
    }
    if (kGrad) {
      const float scale = p.grad_scale * p.in.temperature / static_cast<float>(n);
      const float share = r.s == 0.0f || sum == 0.0f ? 0.0f : scale / r.s;
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
      // the entries of this share; an index given twice teaches twice
      const float teach = sum == 0.0f ? 0.0f : scale / sum;
      __syncthreads();
      for (int j = tid; j < len; j += kDistThreads) {
        const int32_t v = list_at[j];
        if (v < lo || v >= hi) continue;
        float w = 0.0f;
        for (int i = 0; i < len; ++i)
          if (list_at[i] == v) w += ex2_approx(list_q[i]);
        put_logit(out + v, fmaf(ex2_approx((list_x[j] - m) * c), share, -teach * w));
      }
    }
    if (rank != 0) return;
  }
  __syncthreads();
  if (last) mean_of_rows<kDistThreads>(p, parts);
}

// ------------------------------------------------------------------ many long rows
// One CTA on each SM takes row after row through a ring of kChunk buffers that
// a producer warp fills with bulk copies, so that loads never stop for a row's
// barriers: the next row arrives while this one's gradient is written.  The
// consumer warps take a row's sums, then its gradient: from the buffers, as far
// as the ring holds the row (its last chunks), the rest from L2 through the
// ring again.  Two list warps take the rows in turn, each one row of its own
// ahead: it reads the list, gathers the row's logits there, makes the weights,
// and when the sums are known the loss; when the gradient p is written it
// writes the list's entries, p - q, over it.
// Rows are claimed one by one (the first ones by block), since those that do
// not count cost half.
// HBM-bound: 4096 x 128256 bf16 with lists of 64 takes 332 us, 6.3 TB/s (the
// same in shares 428); fp32 1024 x 128256 182, 5.8 TB/s (6.7 rows an SM).  What
// it took: four units of a thread at once (one: 435), maxima of bf16 in pairs,
// two list warps (4096 x 32000: one 149, two 107).
constexpr int kRowWarps = 16, kRowConsumers = 32 * kRowWarps;
constexpr int kListWarps = 2;
constexpr int kFirstConsumer = 32 * (1 + kListWarps);  // after the producer and the list warps
constexpr int kRowThreads = kRowConsumers + kFirstConsumer;
constexpr int kChunk = 2048;                     // units: 32 KB
constexpr int kTake = kChunk / kRowConsumers;    // of a thread
constexpr int kRing = 6;
constexpr int kSpare = 2;   // buffers that stay free for what comes next
constexpr int kRowSlots = 4;
constexpr int kStreamList = 256;  // longest list

__device__ unsigned long long g_distill_status;

// Bounded wait on an mbarrier phase by polling; false (and an error word) on
// expiry.  Every lane that reads what the barrier guards waits itself.  No
// barrier waited on so can complete its next phase before its waiters have
// gone on.  A warp of which one lane's wait has run out arrives nowhere any more:
// what it waited for may still be on its way into a buffer, which is then never
// filled again, and the waits of those who need its arrival run out in their turn.
__device__ __noinline__ bool row_wait_long(uint32_t bar, uint32_t parity, uint64_t timeout_ns, uint32_t site) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (mbar_test_wait(bar, parity)) return true;
    if (global_timer_ns() - t0 > timeout_ns) {
      atomicCAS(&g_distill_status, 0ULL,
                (0x7DULL << 32) | (static_cast<unsigned long long>(blockIdx.x & 0xFFFFFFu) << 8) | site);
      return false;
    }
  }
}
__device__ __forceinline__ bool row_wait(const uint64_t& bar, uint32_t parity, uint64_t timeout_ns, uint32_t site) {
  return mbar_test_wait(smem_addr(&bar), parity) || row_wait_long(smem_addr(&bar), parity, timeout_ns, site);
}
__device__ __forceinline__ void arrive(uint64_t& bar) { mbar_arrive(smem_addr(&bar)); }
// A wait that ran out for one lane has for all: they go on together.
__device__ __forceinline__ bool all_lanes(bool mine) { return __all_sync(kAll, mine) != 0; }

// The consumers' barrier, which also says whether any of them has `pred`; a warp's
// lanes come to it together.
__device__ __forceinline__ bool consumers_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "n"(kRowConsumers)
      : "memory");
  return r != 0;
}

struct RowSlot {
  int64_t row;  // -1: no more rows
  bool counts;
  int len;      // of its list
  float sum;    // of the list's weights
  float m, s;   // of the row
};

struct alignas(16) RowTail {
  uint64_t full[kRing];
  uint64_t empty[kRing];
  uint64_t row_full[kRowSlots];   // the slot's row is known
  uint64_t list_full[kRowSlots];  // its list is ready
  uint64_t sums_full[kRowSlots];  // its sums are
  uint64_t written[kRowSlots];    // its p are
  uint64_t row_empty[kRowSlots];  // all are done with it
  RowSlot slot[kRowSlots];
  RowSums parts[kRowThreads / 32];
  bool last;
};

// One row's list: [k] each.
struct RowList {
  int32_t* at;
  float* d;  // distance of a teacher's logit from the largest, log2
  float* w;  // its weight, those of a repeated index together
  float* x;  // the row's logit there
};

struct StreamArgs {
  DistillArgs a;
  int units, chunks, held;  // of a row: whole vectors in units, in chunks, chunks kept
  int list;                 // k rounded up to 4
  uint64_t timeout_ns;
  int32_t inject;  // tests of the bounded waits: 1 withholds every copy, 2 delays a CTA's first past the limit
};

// Reads a row's list and prepares it, a warp.
template <typename T>
__device__ __forceinline__ void take_list(const DistillArgs& p, int64_t t, const RowList& l, RowSlot& slot, float c) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const T* row = static_cast<const T*>(p.in.logits) + t * p.in.ld;
  int len = p.k;
  float top = -INFINITY;
#pragma unroll 2
  for (int j = lane; j < p.k; j += 32) {
    const int32_t at = p.top_index[t * p.ld_top + j];
    const float v = p.top_logit[t * p.ld_top + j];
    l.at[j] = at;
    l.d[j] = v;
    if (at >= 0 && at < p.in.vocab) l.x[j] = logit_at(row + at);
    else len = min(len, j);
  }
  len = __reduce_min_sync(kAll, len);
  for (int j = lane; j < len; j += 32) top = fmaxf(top, l.d[j]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  const float base = top > -INFINITY ? top : 0.0f;
  float sum = 0.0f;
  for (int j = lane; j < (len + 3) / 4 * 4; j += 32) {
    const float d = j < len ? (l.d[j] - base) * c : 0.0f, w = j < len ? ex2_approx(d) : 0.0f;
    l.d[j] = d;
    l.w[j] = w;
    if (j >= len) l.at[j] = -1;
    sum += w;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  __syncwarp();
  // an index given twice teaches twice; the sums go to registers before any
  // is written
  float mine[kStreamList / 32];
#pragma unroll
  for (int e = 0; e < kStreamList / 32; ++e) {
    const int j = lane + 32 * e;
    if (32 * e >= len) break;
    const int32_t at = j < len ? l.at[j] : -2;
    float w = 0.0f;
#pragma unroll 4
    for (int i = 0; i < len; i += 4) {
      const int4 a4 = *reinterpret_cast<const int4*>(l.at + i);
      const float4 w4 = *reinterpret_cast<const float4*>(l.w + i);
      if (a4.x == at) w += w4.x;
      if (a4.y == at) w += w4.y;
      if (a4.z == at) w += w4.z;
      if (a4.w == at) w += w4.w;
    }
    mine[e] = w;
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < kStreamList / 32; ++e)
    if (lane + 32 * e < len) l.w[lane + 32 * e] = mine[e];
  if (lane == 0) {
    slot.len = len;
    slot.sum = sum;
  }
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1) distill_rows_kernel(const __grid_constant__ StreamArgs p) {
  constexpr int kPer = kUnit<T>;
  extern __shared__ __align__(128) uint4 ring[];
  RowTail* const tl = reinterpret_cast<RowTail*>(ring + kRing * kChunk);
  const DistillArgs& a = p.a;
  const int64_t V = a.in.vocab, T_ = a.in.rows;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const float c = kEpiLog2e * (1.0f / a.in.temperature);
  const uint64_t tmo = p.timeout_ns;
  unsigned* const counter = reinterpret_cast<unsigned*>(a.loss);
  // the list of a slot
  auto list_of = [&](uint32_t r) {
    float* base = reinterpret_cast<float*>(tl + 1) + static_cast<int64_t>(r % kRowSlots) * 4 * p.list;
    return RowList{reinterpret_cast<int32_t*>(base), base + p.list, base + 2 * p.list, base + 3 * p.list};
  };
  auto parity = [](uint32_t r) { return (r / kRowSlots) & 1u; };

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int b = 0; b < kRing; ++b) {
      mbar_init(smem_addr(&tl->full[b]), 1);
      mbar_init(smem_addr(&tl->empty[b]), kRowWarps);
    }
    for (int q = 0; q < kRowSlots; ++q) {
      mbar_init(smem_addr(&tl->row_full[q]), 1);
      mbar_init(smem_addr(&tl->list_full[q]), 1);
      mbar_init(smem_addr(&tl->sums_full[q]), 1);
      mbar_init(smem_addr(&tl->written[q]), kRowWarps);
      mbar_init(smem_addr(&tl->row_empty[q]), kRowWarps + 1);
    }
    fence_mbarrier_init();
  }
  __syncthreads();
  griddep_wait();

  bool ok = true;  // this thread's waits all completed
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t keep_pol = l2_policy(true, 1.0f), drop_pol = evict_first_policy();
      uint32_t seq = 0;  // copies issued
      // copies one chunk of a row
      auto copy = [&](const T* row, int chunk, uint64_t policy) {
        const int b = static_cast<int>(seq % kRing);
        ok = ok && row_wait(tl->empty[b], ((seq / kRing) & 1u) ^ 1u, tmo, 1);
        if (!ok) return;
        if (p.inject == 2 && seq == 0)
          for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < min(2 * tmo, uint64_t{2'000'000'000});) {}
        const uint32_t bytes = static_cast<uint32_t>(min(kChunk, p.units - chunk * kChunk)) * 16u;
        mbar_arrive_expect_tx(smem_addr(&tl->full[b]), bytes);
        bulk_load(smem_addr(ring + b * kChunk), reinterpret_cast<const uint4*>(row) + static_cast<int64_t>(chunk) * kChunk,
                  bytes, smem_addr(&tl->full[b]), policy);
        ++seq;
      };
      auto post = [&](uint32_t r, int64_t row, bool counts) {
        RowSlot& slot = tl->slot[r % kRowSlots];
        ok = ok && row_wait(tl->row_empty[r % kRowSlots], parity(r) ^ 1u, tmo, 2);
        if (!ok) return;  // the slot is still another row's: the others' waits run out, too
        slot.row = row;
        slot.counts = counts;
        arrive(tl->row_full[r % kRowSlots]);
      };
      int64_t row = blockIdx.x;
      bool counts = row_counts(a, row);
      post(0, row, counts);
      for (uint32_t r = 0; row >= 0 && ok; ++r) {
        const int64_t next = static_cast<int64_t>(gridDim.x) + atomicAdd(counter, 1u);
        const T* at = static_cast<const T*>(a.in.logits) + row * a.in.ld;
        const bool copies = counts && p.inject != 1;
        const int again = p.chunks - p.held;
        if (copies)
          for (int i = 0; i < p.chunks && ok; ++i) copy(at, i, i < again ? keep_pol : drop_pol);
        row = next < T_ ? next : -1;
        counts = row >= 0 && row_counts(a, row);
        post(r + 1, row, counts);
        if (row < 0)  // each list warp is told
          for (uint32_t i = 2; i <= kListWarps; ++i) post(r + i, row, false);
        if (copies)
          for (int i = 0; i < again && ok; ++i) copy(at, i, drop_pol);
      }
      // Copies that nobody took, after an expired wait of anyone's: they land
      // (bounded) before this CTA's shared memory goes away.  Where all were taken
      // these waits are over at once.
      for (uint32_t i = seq > kRing ? seq - kRing : 0; i < seq; ++i)
        row_wait(tl->full[i % kRing], (i / kRing) & 1u, tmo, 3);
    }
    __syncwarp();
  } else if (warp <= kListWarps) {
    // ------------------------------------------------------------ lists
    auto prepare = [&](uint32_t r) {
      RowSlot& slot = tl->slot[r % kRowSlots];
      ok = all_lanes(ok && row_wait(tl->row_full[r % kRowSlots], parity(r), tmo, 4));
      if (!ok || slot.row < 0) return false;
      if (slot.counts) take_list<T>(a, slot.row, list_of(r), slot, c);
      if (lane == 0) arrive(tl->list_full[r % kRowSlots]);
      return true;
    };
    uint32_t r = static_cast<uint32_t>(warp - 1);
    for (bool more = prepare(r); more; r += kListWarps) {
      const RowSlot& slot = tl->slot[r % kRowSlots];
      const RowList l = list_of(r);
      const int64_t t = slot.row;
      const bool counts = slot.counts;
      more = prepare(r + kListWarps);
      ok = all_lanes(ok && row_wait(tl->sums_full[r % kRowSlots], parity(r), tmo, 5));
      if (ok && !counts && lane == 0) a.token_loss[t] = 0.0f;
      if (ok && counts) {
        const float log2w = log2f(slot.sum), log2s = log2f(slot.s);
        float kl = 0.0f;
        for (int j = lane; j < slot.len; j += 32) {
          const float q = slot.sum == 0.0f ? 0.0f : ex2_approx(l.d[j]) / slot.sum;
          const float lp = slot.s == 0.0f ? -INFINITY : (l.x[j] - slot.m) * c - log2s;
          if (q != 0.0f) kl = fmaf(q, l.d[j] - log2w - lp, kl);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) kl += __shfl_xor_sync(kAll, kl, o);
        if (lane == 0) a.token_loss[t] = kl * (kRowLn2 * a.in.temperature * a.in.temperature);
      }
      ok = all_lanes(ok && row_wait(tl->written[r % kRowSlots], parity(r), tmo, 6));
      if (ok && counts) {
        const float scale = a.grad_scale * a.in.temperature / static_cast<float>(*a.kept);
        const float share = slot.s == 0.0f || slot.sum == 0.0f ? 0.0f : scale / slot.s;
        const float teach = slot.sum == 0.0f ? 0.0f : scale / slot.sum;
        const float m = slot.m > -INFINITY ? slot.m : 0.0f;
        T* out = static_cast<T*>(a.dlogits) + t * a.ld_dlogits;
        for (int j = lane; j < slot.len; j += 32)
          put_logit(out + l.at[j], fmaf(ex2_approx((l.x[j] - m) * c), share, -teach * l.w[j]));
      }
      __syncwarp();
      if (ok && lane == 0) arrive(tl->row_empty[r % kRowSlots]);
      more = more && ok;
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int cw = warp - 1 - kListWarps, ct = static_cast<int>(threadIdx.x) - kFirstConsumer;
    const int n = *a.kept;
    const float scale = n > 0 ? a.grad_scale * a.in.temperature / static_cast<float>(n) : 0.0f;
    const int tail = static_cast<int>(V & 7);
    const int64_t tail_at = V & ~static_cast<int64_t>(7);
    uint32_t seq = 0;
    for (uint32_t r = 0;; ++r) {
      RowSlot& slot = tl->slot[r % kRowSlots];
      ok = all_lanes(ok && row_wait(tl->row_full[r % kRowSlots], parity(r), tmo, 7));
      if (consumers_any(!ok || slot.row < 0)) break;
      const int64_t t = slot.row;
      const T* row = static_cast<const T*>(a.in.logits) + t * a.in.ld;
      T* out = static_cast<T*>(a.dlogits) + t * a.ld_dlogits;
      uint4* dst = reinterpret_cast<uint4*>(out);
      if (!slot.counts) {
        for (int i = ct; i < p.units; i += kRowConsumers) __stcs(dst + i, make_uint4(0, 0, 0, 0));
        if (ct < tail) put_logit(out + tail_at + ct, 0.0f);
        if (ct == 0) arrive(tl->sums_full[r % kRowSlots]);
      } else {
        // f(units, first, n) on a thread's units of a chunk that arrived as the
        // s-th: the first of them at `first`, the others kRowConsumers apart, those
        // from n on of -inf
        auto chunk = [&](uint32_t s, int i, bool arrived, bool release, auto&& f) {
          const int b = static_cast<int>(s % kRing);
          if (!arrived) ok = all_lanes(ok && row_wait(tl->full[b], (s / kRing) & 1u, tmo, 8));
          const uint4* buf = ring + b * kChunk;
          const int n = ok ? min(kChunk, p.units - i * kChunk) : 0;
          uint4 v[kTake];
#pragma unroll
          for (int u = 0; u < kTake; ++u)
            v[u] = ct + kRowConsumers * u < n ? buf[ct + kRowConsumers * u] : no_unit<T>();
          f(v, i * kChunk + ct, i * kChunk + n);
          if (release) {
            __syncwarp();
            if (ok && lane == 0) arrive(tl->empty[b]);
          }
        };
        const int again = p.chunks - p.held;
        RowSums sums;
        for (int i = 0; i < p.chunks; ++i)
          chunk(seq + i, i, false, i < again,
                [&](const uint4(&v)[kTake], int, int) { add_units<T>(sums, v, c); });
        float last[8];  // the row's last logits, one thread
        if (ct == kRowConsumers - 1 && tail) {
#pragma unroll
          for (int j = 0; j < 8; ++j) last[j] = j < tail ? logit_at(row + tail_at + j) : -INFINITY;
          add<false>(sums, last, c);
        }
        sums = join_warp<false>(sums, c);
        if (lane == 0) tl->parts[cw] = sums;
        __syncwarp();
        (void)consumers_any(false);
        sums = join_parts_warp<false, kRowWarps>(tl->parts, c);
        if (ok && ct == 0) {
          slot.m = sums.m;
          slot.s = sums.s;
          arrive(tl->sums_full[r % kRowSlots]);
        }
        // in place, a list warp must have read before anything is written
        ok = all_lanes(ok && row_wait(tl->list_full[r % kRowSlots], parity(r), tmo, 9));
        const float share = sums.s == 0.0f || slot.sum == 0.0f ? 0.0f : scale / sums.s;
        const float m = sums.m > -INFINITY ? sums.m : 0.0f;
        const F2 m2 = f2(-m), c2 = f2(c), share2 = f2(share);
        auto give = [&](const uint4(&v)[kTake], int first, int end) {
#pragma unroll
          for (int u = 0; u < kTake; ++u) {
            float x[kPer];
            unit_values<T>(v[u], x);
#pragma unroll
            for (int j = 0; j < kPer; j += 2)
              split(mul2(ex2_2(mul2(add2(f2(x[j], x[j + 1]), m2), c2)), share2), x[j], x[j + 1]);
            if (first + kRowConsumers * u < end) __stcs(dst + first + kRowConsumers * u, unit_of(x));
          }
        };
        for (int i = again; i < p.chunks; ++i) chunk(seq + i, i, true, true, give);
        for (int i = 0; i < again; ++i) chunk(seq + p.chunks + i, i, false, true, give);
        if (ok && ct == kRowConsumers - 1) {
          for (int j = 0; j < tail; ++j) put_logit(out + tail_at + j, ex2_approx((logit_at(row + tail_at + j) - m) * c) * share);
        }
        seq += static_cast<uint32_t>(p.chunks + again);
      }
      __syncwarp();
      if (ok && lane == 0) {
        arrive(tl->written[r % kRowSlots]);
        arrive(tl->row_empty[r % kRowSlots]);
      }
    }
  }
  // the mean, by the CTA that finishes last: each has claimed rows until one
  // claim came back empty, so that T claims and a count for each CTA are all
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    tl->last = atomicAdd(counter, 1u) == static_cast<unsigned>(T_) + gridDim.x - 1;
  }
  __syncthreads();
  if (tl->last) mean_of_rows<kRowThreads>(a, tl->parts);
}

int stream_shared(int k) {
  return kRing * kChunk * 16 + static_cast<int>(sizeof(RowTail)) + kRowSlots * 16 * ((k + 3) / 4 * 4);
}

// Which rows go through the ring: long ones, of which an SM gets several
// (gradients of 4096 rows: 98 us against 90 in shares at 24000 bf16 words, 105
// against 117 at 32000, 323 against 428 at 128256; of 64000 words 30.3 against
// 30.5 for 400 rows, 17.7 against 16.7 for 200), with lists that one warp
// prepares while others take a row.  Each entry looks for its index in the whole
// list, here and in shares: 4096 x 128256 with lists of 64 takes 332 us, of 256 464,
// of 257, in shares, 664, and of 1024 3.8 ms.
bool streams_rows(int64_t rows, int64_t row_bytes, int k, int sms) {
  return k <= kStreamList && rows >= 2 * sms && row_bytes >= (56 << 10);
}

cudaError_t distill_ring_launch(const DistillArgs& a, int sms, uint64_t timeout_ns, int inject, bool pdl,
                                cudaStream_t stream) {
  StreamArgs p{};
  p.a = a;
  p.units = static_cast<int>(a.in.vocab / 8 * (a.in.f32 ? 2 : 1));
  p.chunks = (p.units + kChunk - 1) / kChunk;
  p.held = std::min(p.chunks, kRing - kSpare);
  p.list = (a.k + 3) / 4 * 4;
  p.timeout_ns = timeout_ns;
  p.inject = inject;
  return launch_clusters(a.in.f32 ? distill_rows_kernel<float> : distill_rows_kernel<uint16_t>,
                         dim3(static_cast<unsigned>(std::min<int64_t>(a.in.rows, sms))), 1, kRowThreads, pdl, stream,
                         static_cast<size_t>(stream_shared(a.k)), p);
}

template <int kThreads>
cudaError_t distill_shares_blocks(const DistillArgs& a, int cluster, bool pdl, cudaStream_t stream) {
  int held = 0;
  if (a.dlogits) {
    const int64_t vectors = (a.in.vocab / 8 + cluster - 1) / cluster;
    held = static_cast<int>(std::min<int64_t>(vectors * (a.in.f32 ? 32 : 16), kMostHeld));
  }
  auto kernel = a.in.f32 ? (a.dlogits ? distill_kernel<float, true, kThreads> : distill_kernel<float, false, kThreads>)
                         : (a.dlogits ? distill_kernel<uint16_t, true, kThreads>
                                      : distill_kernel<uint16_t, false, kThreads>);
  return launch_clusters(kernel, dim3(static_cast<unsigned>(a.in.rows * cluster)), static_cast<unsigned>(cluster),
                         kThreads, pdl, stream, static_cast<size_t>(held + 12 * a.k), a, held / 16);
}
cudaError_t distill_shares_launch(const DistillArgs& a, int threads, int cluster, bool pdl, cudaStream_t stream) {
  return threads == 128 ? distill_shares_blocks<128>(a, cluster, pdl, stream)
                        : distill_shares_blocks<256>(a, cluster, pdl, stream);
}

// Threads a block: fewer for many short rows (gradients of 4096 x 4000: 33 us by
// 128, 43 by 256; 4096 x 16000 72 and 69), and for many rows of which only the
// sums are wanted (1024 x 128256 55 us and 63).
int row_threads(const DistillArgs& a, int64_t bytes, int sms) {
  if (!a.dlogits) return a.in.rows >= 4 * sms ? 128 : 256;
  return bytes <= (16 << 10) && a.in.rows >= 12 * sms ? 128 : 256;
}

}  // namespace

cudaError_t distill_init() {
  cudaError_t e = cudaSuccess;
  for (auto kernel : {distill_kernel<float, true, 128>, distill_kernel<uint16_t, true, 128>,
                      distill_kernel<float, true, 256>, distill_kernel<uint16_t, true, 256>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld + 12 * kMaxList);
  for (auto kernel : {distill_rows_kernel<float>, distill_rows_kernel<uint16_t>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, stream_shared(kStreamList));
  return e;
}

cudaError_t distill_launch(const DistillArgs& a, int sms, uint64_t timeout_ns, int inject, bool pdl,
                           cudaStream_t stream) {
  const cudaError_t e = launch_after(distill_count_kernel, dim3(1), 1024, pdl, stream, a);
  if (e != cudaSuccess || a.in.rows == 0) return e;
  const int64_t bytes = a.in.vocab / 8 * (a.in.f32 ? 32 : 16);
  if (a.dlogits && streams_rows(a.in.rows, bytes, a.k, sms))
    return distill_ring_launch(a, sms, timeout_ns, inject, pdl, stream);
  int cluster = row_cluster(a.in.rows, a.in.vocab, sms);
  while (a.dlogits && cluster < kMaxCluster && bytes / cluster > kHeldBytes) cluster *= 2;
  return distill_shares_launch(a, row_threads(a, bytes, sms), cluster, pdl, stream);
}

cudaError_t distill_take_status(unsigned long long* word, cudaStream_t stream) {
  *word = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_distill_status, sizeof(*word), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || *word == 0) return e;
  const unsigned long long zero = 0;
  e = cudaMemcpyToSymbolAsync(g_distill_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace axonn
