// Row kernels of the linear cross entropy, between its products.
//
// Rows whose label does not count (padding, or a label left out by a mask)
// are never read: the others are packed first, so that they cost no
// products, and an infinity or NaN in a row that is masked reaches nothing.
//
// The statistics product leaves (m_g, s_g) for each row and column group g:
// the group's maximum and its sum of e^(z - m_g).  With M = max_g m_g,
//   logsumexp = M + ln sum_g s_g e^(m_g - M),
// and a logit kept as its distance q below m_g (see kCeStep) has the
// probability 2^(m_g log2 e - logsumexp log2 e - q), rounded to bf16 once.  A
// label's own entry, p - 1, is computed from its logit in fp32, so that a
// confident row's small gradient does not come from the difference of two
// rounded numbers.  The factor g / n waits for the fp32 epilogues of dX and
// dW: in P it would shift every label's entry, about -g / n, by the same
// rounding.
#include <algorithm>

#include "launch.h"
#include "linear_ce.h"
#include "vec8.cuh"

namespace axonn {
namespace {

constexpr float kCeLn2 = 0.6931471805599453f;

// 7 us for 4096 labels, one block's latency.  It walks the labels 4096 at a time, a thread four consecutive ones:
// a place is the counted labels before it, by a scan of the threads' counts
// within a warp and the warps' totals across them.
__global__ void __launch_bounds__(1024) ce_index_kernel(CeRowArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int totals[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int64_t base = 0; base < a.rows; base += 4096) {
    const int64_t t0 = base + 4 * threadIdx.x;
    int32_t y[4];
    bool counted[4];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + j;
      y[j] = t < a.rows ? a.labels[t] : -1;
      counted[j] = y[j] >= 0 && y[j] < a.vocab && (!a.keep || a.keep[t] != 0);
      mine += counted[j] ? 1 : 0;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) totals[warp] = upto;
    __syncthreads();
    int at = n + upto - mine;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += totals[w];
      n += totals[w];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + j;
      if (t >= a.rows) break;
      a.place[t] = counted[j] ? at : -1;
      if (counted[j]) {
        a.index[at] = static_cast<int32_t>(t);
        a.packed_labels[at++] = y[j];
      } else {
        a.token_loss[t] = 0.0f;
        if (a.lse) a.lse[t] = 0.0f;
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *a.kept = n;
    *a.coef = n > 0 ? a.grad_scale / static_cast<float>(n) : 0.0f;
    *a.done = 0;
    // As many parts as keep the GPU's units busy with n rows (fewer than the
    // host, which knows only `rows`, could count on), packed n rows apart.
    int parts = 1;
    const int64_t apart = (n + 31) / 32 * 32;
    if (a.part_rows > 0 && n > 0) {
      const int64_t tiles = (n + a.part_tile - 1) / a.part_tile * static_cast<int64_t>(a.part_tiles_n);
      parts = static_cast<int>(max(static_cast<int64_t>(1),
                                   min(min(a.part_rows / apart, static_cast<int64_t>(a.most_parts)),
                                       static_cast<int64_t>(a.part_units) / tiles)));
    }
    *a.parts = make_int2(parts, static_cast<int>(apart));
  }
}

// Copies the counted rows of X to their packed places (zeros up to the next
// multiple of 64 rows, which the weight gradient's reduction reads): blocks
// over rows and 2048 columns, a thread eight of them.  HBM-bound: 4096 x 6144
// takes 17 us, 5.9 TB/s.
__global__ void __launch_bounds__(256) ce_gather_kernel(CeRowArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t n = *a.kept;
  const int64_t pad = min(a.rows, (n + 63) / 64 * 64);
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= a.cols) return;
  const int m = static_cast<int>(min(static_cast<int64_t>(8), a.cols - c));
  for (int64_t i = blockIdx.y; i < pad; i += gridDim.y) {
    uint16_t* dst = a.packed_x + i * a.ld_packed + c;
    const uint16_t* src = i < n ? a.x + a.index[i] * a.ld_x + c : nullptr;
    if (m == 8) {
      *reinterpret_cast<uint4*>(dst) = src ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
    } else {
      for (int j = 0; j < m; ++j) dst[j] = src ? src[j] : 0;
    }
  }
}

// Adds (m2, s2) to a running (m, s).
__device__ __forceinline__ void ce_join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == -INFINITY) {  // no finite logit yet: sums of 0, or NaN
    s += s2;
    return;
  }
  s = s * ex2_approx((m - top) * kEpiLog2e) + s2 * ex2_approx((m2 - top) * kEpiLog2e);
  m = top;
}

// A block takes kRows rows: a warp's lanes are kRows rows x 32 / kRows groups,
// its 32 warps take the groups in turn.  Lanes of the same row are joined by
// shuffles, warps through shared memory, in a fixed order.  The block that
// finishes last adds up the losses, a thread every 1024th row in order, then
// the threads' sums as a tree.  4096 rows x 2004 groups (66 MB, most of it
// still in L2) take 25 us.
template <int kRows>
__global__ void __launch_bounds__(1024) ce_combine_kernel(CeRowArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float pm[32][kRows], ps[32][kRows];
  __shared__ float part[32];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = *a.kept;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + lane % kRows;
  if (static_cast<int64_t>(blockIdx.x) * kRows < n) {
    float m = -INFINITY, s = 0.0f;
    if (i < n) {
#pragma unroll 4
      for (int64_t g = warp * (32 / kRows) + lane / kRows; g < a.groups; g += 1024 / kRows) {
        const float2 v = a.stats[g * a.rows + i];
        ce_join(m, s, v.x, v.y);
      }
    }
#pragma unroll
    for (int o = kRows; o < 32; o <<= 1)
      ce_join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if (lane < kRows) {
      pm[warp][lane] = m;
      ps[warp][lane] = s;
    }
    __syncthreads();
    if (threadIdx.x < kRows && i < n) {
      m = -INFINITY;
      s = 0.0f;
      for (int w = 0; w < 32; ++w) ce_join(m, s, pm[w][lane], ps[w][lane]);
      const float l2 = log2f(s);  // s is at least 1 where the row has a finite logit
      const float lse = fmaf(l2, kCeLn2, m);
      const int32_t t = a.index[i];
      a.lse2[i] = fmaf(m, kEpiLog2e, l2);
      if (a.lse) a.lse[t] = lse;
      a.token_loss[t] = lse - a.label_logit[i];
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f;
  for (int64_t t = threadIdx.x; t < a.rows; t += 1024) sum += __ldcg(a.token_loss + t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float total = 0.0f;
    for (int w = 0; w < 32; ++w) total += part[w];
    *a.loss = n > 0 ? total / static_cast<float>(n) : 0.0f;
  }
}

// Blocks over (row, 4096 columns), a thread two vectors of eight columns,
// both loaded before either is used.  HBM-bound: 4 bytes an element; 4096 x
// 128256 takes 410 to 465 us (4.5 to 5.1 TB/s; one vector a thread 451 where
// two took 411), 490 x 50257, which L2 holds, 26 (3.8 TB/s).
constexpr int kScaleVecs = 2;
constexpr int kScaleCols = 2048 * kScaleVecs;
__global__ void __launch_bounds__(256) ce_scale_kernel(CeRowArgs a, uint16_t* piece, int64_t ld,
                                                       int64_t col0, int64_t cols) {
  griddep_launch_dependents();
  griddep_wait();
  const int kept = *a.kept;
  const int64_t pad = min(a.rows, (static_cast<int64_t>(kept) + 63) / 64 * 64);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kScaleCols + 8 * threadIdx.x;
  for (int64_t row = blockIdx.y; row < pad; row += gridDim.y) {
    Vec8<uint16_t> v[kScaleVecs];
    float top[kScaleVecs];
    const bool in = row < kept;
    const float lse2 = in ? a.lse2[row] : 0.0f;
    const float far = lse2 - lse2;  // 0, or NaN throughout a row whose sum is not a number
#pragma unroll
    for (int u = 0; u < kScaleVecs; ++u) {
      const int64_t c = first + 2048 * u;
      if (in && c < cols) {
        v[u].load(piece + row * ld + c, static_cast<int>(min(static_cast<int64_t>(8), cols - c)));
        top[u] = fmaf(a.stats[(col0 + c) / a.group_cols * a.rows + row].x, kEpiLog2e, -lse2);
      }
    }
    const int64_t label = in ? a.packed_labels[row] - col0 : -1;
#pragma unroll
    for (int u = 0; u < kScaleVecs; ++u) {
      const int64_t c = first + 2048 * u;
      if (c < cols) {
        float x[8] = {};
        if (in) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t q = (j & 1) ? v[u].w[j >> 1] >> 16 : v[u].w[j >> 1] & 0xFFFFu;
            // q as a float: the low bits of 2^23 + q
            const float f = __uint_as_float(0x4B000000u | q) - 8388608.0f;
            x[j] = q == kCeFar ? far : ex2_approx(fmaf(f, -1.0f / kCeStep, top[u]));
          }
          const int64_t d = label - c;
          if (d >= 0 && d < 8) {
            const float py = ex2_approx(fmaf(a.label_logit[row], kEpiLog2e, -lse2)) - 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j == d) x[j] = py;
          }
        }
        store8(piece + row * ld + c, static_cast<int>(min(static_cast<int64_t>(8), cols - c)), x);
      }
    }
  }
}

// A block takes a row of dX at a time, a thread eight columns: the packed
// row, the sum of its fp32 parts in order, or zeros.  4096 x 6144 of five
// parts (0.5 GB, partly in L2) take 23 us.
template <bool kF32>
__global__ void __launch_bounds__(256) ce_unpack_kernel(CeRowArgs a, const void* packed, int64_t ld) {
  griddep_launch_dependents();
  griddep_wait();
  const int splits = kF32 ? a.parts->x : 0;
  const int64_t split_rows = kF32 ? a.parts->y : 0;
  const int64_t vecs = (a.cols + 7) / 8;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const int64_t at = a.place[t];
    for (int64_t v = threadIdx.x; v < vecs; v += 256) {
      uint16_t* dst = a.dx + t * a.ld_dx + 8 * v;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (at >= 0 && kF32) {
        // the row's padding up to 8 columns is the workspace's own
        const float* src = static_cast<const float*>(packed) + at * ld + 8 * v;
        float4 p = reinterpret_cast<const float4*>(src)[0], q = reinterpret_cast<const float4*>(src)[1];
        for (int s = 1; s < splits; ++s) {
          src += split_rows * ld;
          const float4 p2 = reinterpret_cast<const float4*>(src)[0], q2 = reinterpret_cast<const float4*>(src)[1];
          p = make_float4(p.x + p2.x, p.y + p2.y, p.z + p2.z, p.w + p2.w);
          q = make_float4(q.x + q2.x, q.y + q2.y, q.z + q2.z, q.w + q2.w);
        }
        w = make_uint4(pack_bf16(p.x, p.y), pack_bf16(p.z, p.w), pack_bf16(q.x, q.y), pack_bf16(q.z, q.w));
      } else if (at >= 0) {
        w = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(packed) + at * ld)[v];
      }
      const int n = static_cast<int>(min(static_cast<int64_t>(8), a.cols - 8 * v));
      if (n == 8) {
        *reinterpret_cast<uint4*>(dst) = w;
      } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) dst[j] = static_cast<uint16_t>(x[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

}  // namespace

cudaError_t ce_index_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream) {
  return launch_after(ce_index_kernel, dim3(1), 1024, pdl, stream, a);
}

cudaError_t ce_gather_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((a.cols + 2047) / 2048),
                  static_cast<unsigned>(std::min<int64_t>(a.rows, 65535)));
  return launch_after(ce_gather_kernel, grid, 256, pdl, stream, a);
}

cudaError_t ce_combine_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream) {
  // Eight rows read a group's statistics as whole 64 bytes; fewer rows a
  // block where there are not enough of them to fill the GPU (16 rows x 2004
  // groups: 28 us by 32 rows a block, 10 by 2).
  const int rows = a.rows >= 1024 ? 8 : 2;
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (a.rows + rows - 1) / rows)));
  return launch_after(rows == 8 ? ce_combine_kernel<8> : ce_combine_kernel<2>, grid, 1024, pdl, stream, a);
}

cudaError_t ce_scale_launch(const CeRowArgs& a, uint16_t* piece, int64_t ld_piece, int64_t col0,
                            int64_t cols, int sms, bool pdl, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  // About 48 blocks an SM: a block a row leaves one idle for each row that
  // does not count (1003 x 768 x 50257, half masked: 165 us in all, 159 so),
  // and even without a mask takes 3 % more over 4096 x 50304.
  const int64_t across = (cols + kScaleCols - 1) / kScaleCols;
  const dim3 grid(static_cast<unsigned>(across),
                  static_cast<unsigned>(std::min<int64_t>(a.rows, std::max<int64_t>(1, 48 * sms / across))));
  return launch_after(ce_scale_kernel, grid, 256, pdl, stream, a, piece, ld_piece, col0, cols);
}

cudaError_t ce_unpack_launch(const CeRowArgs& a, const void* packed, int64_t ld, bool f32, int sms, bool pdl,
                             cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t{8} * sms)));
  return launch_after(f32 ? ce_unpack_kernel<true> : ce_unpack_kernel<false>, grid, 256, pdl, stream, a, packed, ld);
}

}  // namespace axonn
