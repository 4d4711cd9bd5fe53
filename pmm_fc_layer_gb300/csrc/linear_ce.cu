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

#include "epilogue_math.cuh"
#include "linear_ce.h"

namespace axonn {
namespace {

constexpr float kCeLn2 = 0.6931471805599453f;

// One block walks the labels 1024 at a time: a place is the counted labels
// before it, by a ballot within a warp and the warps' counts across them.
__global__ void __launch_bounds__(1024) ce_index_kernel(CeRowArgs a) {
  __shared__ int counts[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int64_t base = 0; base < a.rows; base += 1024) {
    const int64_t t = base + threadIdx.x;
    int32_t y = -1;
    bool counts_here = false;
    if (t < a.rows) {
      y = a.labels[t];
      counts_here = y >= 0 && y < a.vocab && (!a.keep || a.keep[t] != 0);
    }
    const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, counts_here);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = n, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += counts[w];
      total += counts[w];
    }
    if (counts_here) {
      const int at = before + __popc(ballot & ((1u << lane) - 1u));
      a.index[at] = static_cast<int32_t>(t);
      a.packed_labels[at] = y;
      a.place[t] = at;
    } else if (t < a.rows) {
      a.place[t] = -1;
      a.token_loss[t] = 0.0f;
      if (a.lse) a.lse[t] = 0.0f;
    }
    n += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *a.kept = n;
    *a.coef = n > 0 ? a.grad_scale / static_cast<float>(n) : 0.0f;
  }
}

// Copies the counted rows of X to their packed places (zeros up to the next
// multiple of 64 rows, which the weight gradient's reduction reads).  A warp
// takes a row at a time in 16-byte vectors; the row's last cols % 8 elements
// go one by one.
__global__ void __launch_bounds__(256) ce_gather_kernel(CeRowArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t n = *a.kept;
  const int64_t pad = min(a.rows, (n + 63) / 64 * 64);
  const int64_t vecs = a.cols / 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < pad; i += warps) {
    uint16_t* dst = a.packed_x + i * a.ld_packed;
    const uint16_t* src = i < n ? a.x + a.index[i] * a.ld_x : nullptr;
#pragma unroll 4
    for (int64_t v = lane; v < vecs; v += 32)
      reinterpret_cast<uint4*>(dst)[v] = src ? reinterpret_cast<const uint4*>(src)[v] : make_uint4(0, 0, 0, 0);
    for (int64_t c = 8 * vecs + lane; c < a.cols; c += 32) dst[c] = src ? src[c] : 0;
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

// A block takes 32 rows (a lane each); its 32 warps take every 32nd group,
// and the first warp joins their results in order.
__global__ void __launch_bounds__(1024) ce_combine_kernel(CeRowArgs a) {
  __shared__ float pm[32][33], ps[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = *a.kept;
  if (static_cast<int64_t>(blockIdx.x) * 32 >= n) return;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  if (i < n) {
#pragma unroll 4
    for (int64_t g = warp; g < a.groups; g += 32) {
      const float2 v = a.stats[g * a.rows + i];
      ce_join(m, s, v.x, v.y);
    }
  }
  pm[warp][lane] = m;
  ps[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= n) return;
  for (int w = 1; w < 32; ++w) ce_join(m, s, pm[w][lane], ps[w][lane]);
  const float l2 = log2f(s);  // s is at least 1 where the row has a finite logit
  const float lse = fmaf(l2, kCeLn2, m);
  const int32_t t = a.index[i];
  a.lse2[i] = fmaf(m, kEpiLog2e, l2);
  if (a.lse) a.lse[t] = lse;
  a.token_loss[t] = lse - a.label_logit[i];
}

__global__ void __launch_bounds__(1024) ce_mean_kernel(CeRowArgs a) {
  __shared__ float part[32];
  float s = 0.0f;
  for (int64_t t = threadIdx.x; t < a.rows; t += 1024) s += a.token_loss[t];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.0f;
    for (int w = 0; w < 32; ++w) t += part[w];
    const int n = *a.kept;
    *a.loss = n > 0 ? t / static_cast<float>(n) : 0.0f;
  }
}

// Eight columns a thread, blocks over (row, 2048 columns).  HBM-bound: 4
// bytes an element.
__global__ void __launch_bounds__(256) ce_scale_kernel(CeRowArgs a, uint16_t* piece, int64_t ld,
                                                       int64_t col0, int64_t cols) {
  const int64_t kept = *a.kept;
  const int64_t pad = min(a.rows, (kept + 63) / 64 * 64);
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= cols) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(8), cols - c));
  const int64_t group = (col0 + c) / a.group_cols;
  for (int64_t row = blockIdx.y; row < pad; row += gridDim.y) {
    uint16_t* p = piece + row * ld + c;
    float x[8] = {};
    if (row < kept) {
      const float lse2 = a.lse2[row];
      const float2 st = a.stats[group * a.rows + row];
      const float top = fmaf(st.x, kEpiLog2e, -lse2);
      uint32_t q[8];
      if (n >= 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q[2 * j] = w[j] & 0xFFFFu;
          q[2 * j + 1] = w[j] >> 16;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = j < n ? p[j] : kCeFar;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // q as a float: the low bits of 2^23 + q
        const float f = __uint_as_float(0x4B000000u | q[j]) - 8388608.0f;
        x[j] = q[j] == kCeFar ? 0.0f : ex2_approx(fmaf(f, -1.0f / kCeStep, top));
      }
      const int64_t d = a.packed_labels[row] - col0 - c;
      if (d >= 0 && d < 8) {
        const float py = ex2_approx(fmaf(a.label_logit[row], kEpiLog2e, -lse2)) - 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j == d) x[j] = py;
      }
    }
    const uint32_t w[4] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                           pack_bf16(x[6], x[7])};
    if (n >= 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// A warp takes a row of dX at a time: its packed row, rounded if fp32, or
// zeros.
template <bool kF32>
__global__ void __launch_bounds__(256) ce_unpack_kernel(CeRowArgs a, const void* packed, int64_t ld) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t vecs = a.cols / 8;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < a.rows; t += warps) {
    const int64_t at = a.place[t];
    uint16_t* dst = a.dx + t * a.ld_dx;
    const uint16_t* s16 = static_cast<const uint16_t*>(packed) + at * ld;
    const float* s32 = static_cast<const float*>(packed) + at * ld;
#pragma unroll 4
    for (int64_t v = lane; v < vecs; v += 32) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (at >= 0 && kF32) {
        const float4 p = reinterpret_cast<const float4*>(s32)[2 * v], q = reinterpret_cast<const float4*>(s32)[2 * v + 1];
        w = make_uint4(pack_bf16(p.x, p.y), pack_bf16(p.z, p.w), pack_bf16(q.x, q.y), pack_bf16(q.z, q.w));
      } else if (at >= 0) {
        w = reinterpret_cast<const uint4*>(s16)[v];
      }
      reinterpret_cast<uint4*>(dst)[v] = w;
    }
    for (int64_t c = 8 * vecs + lane; c < a.cols; c += 32)
      dst[c] = at < 0 ? 0 : (kF32 ? static_cast<uint16_t>(pack_bf16(s32[c], 0.0f)) : s16[c]);
  }
}

unsigned row_blocks(int64_t rows, int sms) {
  return static_cast<unsigned>(std::min<int64_t>((rows + 7) / 8, int64_t{8} * sms));
}

}  // namespace

cudaError_t ce_index_launch(const CeRowArgs& a, cudaStream_t stream) {
  ce_index_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t ce_gather_launch(const CeRowArgs& a, int sms, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  ce_gather_kernel<<<row_blocks(a.rows, sms), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t ce_combine_launch(const CeRowArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  ce_combine_kernel<<<static_cast<unsigned>((a.rows + 31) / 32), 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t ce_mean_launch(const CeRowArgs& a, cudaStream_t stream) {
  ce_mean_kernel<<<1, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t ce_scale_launch(const CeRowArgs& a, uint16_t* piece, int64_t ld_piece, int64_t col0,
                            int64_t cols, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((cols + 2047) / 2048),
                  static_cast<unsigned>(std::min<int64_t>(a.rows, 65535)));
  ce_scale_kernel<<<grid, 256, 0, stream>>>(a, piece, ld_piece, col0, cols);
  return cudaGetLastError();
}

cudaError_t ce_unpack_launch(const CeRowArgs& a, const void* packed, int64_t ld, bool f32, int sms,
                             cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  if (f32) ce_unpack_kernel<true><<<row_blocks(a.rows, sms), 256, 0, stream>>>(a, packed, ld);
  else ce_unpack_kernel<false><<<row_blocks(a.rows, sms), 256, 0, stream>>>(a, packed, ld);
  return cudaGetLastError();
}

}  // namespace axonn
