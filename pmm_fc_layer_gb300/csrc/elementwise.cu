// Elementwise kernels beside the fused products, both bound by HBM:
//   dropout   Y = R + D(X)                       (bf16 or fp32)
//   backward  d = act'(Z) D(dY), dZ = d in bf16, column sums of d
// A thread owns eight consecutive columns of a row: one 16-byte vector of
// bf16 and one call of the generator, whose mask is therefore never stored.
// Measured: dropout with a residual, bf16 8192 x 6144, 50 us (6.0 TB/s, 89 % of
// a copy); backward with tanh-GELU' and column sums, bf16 8192 x 24576, 188 us
// (6.4 TB/s, 95 %), with the other GELU's 193.
#include <algorithm>

#include "elementwise.h"
#include "launch.h"
#include "vec8.cuh"

namespace axonn {
namespace {

constexpr int kThreads = 256;

// The vectors of the matrix in row order, dealt out to the grid's threads
// kDropUnroll at a time: all their loads are issued before the first is
// used, which is what keeps enough bytes in flight.  The row and column of a
// thread's next vector follow from the last by one addition and one wrap.
// One vector at a time took 74 us where four take 50 (8192 x 6144).
constexpr int kDropUnroll = 4;
template <typename T, bool kRes>
constexpr int kDropBlocks = sizeof(T) == 2 ? (kRes ? 4 : 5) : (kRes ? 2 : 3);  // resident on an SM
template <typename T, bool kRes>
__global__ void __launch_bounds__(kThreads, kDropBlocks<T, kRes>) dropout_kernel(DropoutKernelArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const T* X = static_cast<const T*>(a.x);
  const T* R = static_cast<const T*>(a.residual);
  T* Y = static_cast<T*>(a.y);
  const int n8 = static_cast<int>((a.cols + 7) / 8);
  const int tail = static_cast<int>(a.cols - 8 * static_cast<int64_t>(n8 - 1));  // of a row's last vector
  const int64_t total = a.rows * n8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= total) return;
  const DropRng g = load_rng(a.drop);
  const int dr = static_cast<int>(stride / n8), dc = static_cast<int>(stride - static_cast<int64_t>(dr) * n8);
  int row = static_cast<int>(i / n8), c8 = static_cast<int>(i - static_cast<int64_t>(row) * n8);
  while (i < total) {
    Vec8<T> x[kDropUnroll], r[kDropUnroll];
    int rows[kDropUnroll], cols[kDropUnroll];
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      rows[u] = row;
      cols[u] = c8;
      if (i + u * stride < total) {
        const int n = c8 + 1 < n8 ? 8 : tail;
        x[u].load(X + row * a.ld_x + 8 * static_cast<int64_t>(c8), n);
        if (kRes) r[u].load(R + row * a.ld_res + 8 * static_cast<int64_t>(c8), n);
      }
      row += dr;
      c8 += dc;
      if (c8 >= n8) {
        c8 -= n8;
        ++row;
      }
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      if (i + u * stride >= total) break;
      float v[8], b[8] = {};
      x[u].values(v);
      if (kRes) r[u].values(b);
      if (a.drop.thr != 0) {
        drop8_add(a.drop, drop_words(g, static_cast<uint32_t>(rows[u]), static_cast<uint32_t>(cols[u])), v, b);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += b[j];
      }
      store8(Y + rows[u] * a.ld_y + 8 * static_cast<int64_t>(cols[u]), cols[u] + 1 < n8 ? 8 : tail, v);
    }
    i += kDropUnroll * stride;
  }
}

// A block covers kBwdRows rows x 256 columns: each of its eight warps takes
// every eighth row, a lane eight columns, kBwdUnroll rows' loads at a time.
// A lane adds its rows' columns in order, the block its warps' sums in
// order: partial sums of kBwdRows rows.  The activation and whether there is
// dropout are compiled in: at 6 bytes an element the arithmetic has about 40
// instructions an element to spend, and the general form took more.
constexpr int kBwdRows = 64;
constexpr int kBwdUnroll = 4;
static_assert(kBwdRows >= 32, "the partial sums' workspace holds one row of them per 32 rows");
static_assert(kBwdRows % (8 * kBwdUnroll) == 0, "whole batches of rows");

// One lane's eight columns over rows r0, r0 + 8, ... below r1; kFull: all
// eight exist.
template <typename T, int ACT, bool kDrop, bool kFull>
__device__ __forceinline__ void act_bwd_rows(const BwdKernelArgs& a, const DropRng& g, int64_t r0, int64_t r1,
                                             int64_t col, int n, float (&sum)[8]) {
  constexpr int U = kFull ? kBwdUnroll * 2 / static_cast<int>(sizeof(T)) : 1;  // the same bytes in flight for fp32
  if (kFull) n = 8;
  const T* dy = static_cast<const T*>(a.dy) + r0 * a.ld_dy + col;
  const uint16_t* pre = a.pre + r0 * a.ld_pre + col;
  uint16_t* dz = a.dz + r0 * a.ld_dz + col;
#pragma unroll 1
  for (int64_t base = r0; base < r1; base += 8 * U) {
    Vec8<T> x[U];
    Vec8<uint16_t> z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + 8 * u < r1) {
        x[u].load(dy, n);
        if (ACT != kActNone) z[u].load(pre, n);
      }
      dy += 8 * a.ld_dy;
      if (ACT != kActNone) pre += 8 * a.ld_pre;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + 8 * u < r1) {
        float v[8];
        x[u].values(v);
        if (kDrop) drop8(a.drop, g, static_cast<uint32_t>(base + 8 * u), static_cast<uint32_t>(col / 8), v);
        if (ACT != kActNone) {
          act_slopes<ACT, 8>(v, z[u].w);
        }
        store8(dz, n, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
      }
      dz += 8 * a.ld_dz;
    }
  }
}

template <typename T, int ACT, bool kDrop>
__global__ void __launch_bounds__(kThreads, 3) act_bwd_kernel(BwdKernelArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float part[8][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + 8 * lane;
  const int n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), a.cols - col)));
  DropRng g{0, 0};
  if (kDrop) g = load_rng(a.drop);
  for (int64_t group = blockIdx.y; group * kBwdRows < a.rows; group += gridDim.y) {
    const int64_t r0 = group * kBwdRows + warp;
    const int64_t r1 = min(a.rows, group * kBwdRows + kBwdRows);
    float sum[8] = {};
    if (n == 8) act_bwd_rows<T, ACT, kDrop, true>(a, g, r0, r1, col, 8, sum);
    else if (n > 0) act_bwd_rows<T, ACT, kDrop, false>(a, g, r0, r1, col, n, sum);
    if (a.colsum) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) part[warp][lane][j] = sum[j];
      __syncthreads();
      const int c = threadIdx.x;  // one of the block's 256 columns
      const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + c;
      if (at < a.cols) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part[w][c >> 3][c & 7];
        a.colsum[group * a.ld_colsum + at] = s;
      }
    }
  }
}

template <typename T, bool kDrop>
cudaError_t act_bwd_start(const BwdKernelArgs& a, dim3 grid, bool pdl, cudaStream_t stream) {
  switch (a.act) {
    case kActRelu: return launch_after(act_bwd_kernel<T, kActRelu, kDrop>, grid, kThreads, pdl, stream, a);
    case kActGelu: return launch_after(act_bwd_kernel<T, kActGelu, kDrop>, grid, kThreads, pdl, stream, a);
    case kActGeluTanh: return launch_after(act_bwd_kernel<T, kActGeluTanh, kDrop>, grid, kThreads, pdl, stream, a);
    case kActSilu: return launch_after(act_bwd_kernel<T, kActSilu, kDrop>, grid, kThreads, pdl, stream, a);
    default: return launch_after(act_bwd_kernel<T, kActNone, kDrop>, grid, kThreads, pdl, stream, a);
  }
}

// out[col] = sum over the groups' partial sums, in a fixed order: a warp's
// lanes take 32 columns, its eight warps every eighth group, then the warps'
// sums in order.
__global__ void __launch_bounds__(kThreads) colsum_kernel(const float* part, int64_t ld, int64_t groups,
                                                          int64_t cols, float* out) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int64_t g = warp; g < groups; g += 8) s += part[g * ld + col];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < cols) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][lane];
    out[col] = t;
  }
}

}  // namespace

namespace {
template <typename T, bool kRes>
cudaError_t dropout_start(const DropoutKernelArgs& a, int sms, bool pdl, cudaStream_t stream) {
  const int64_t vectors = a.rows * ((a.cols + 7) / 8);
  const int64_t blocks =
      std::min<int64_t>((vectors + kThreads - 1) / kThreads, int64_t{kDropBlocks<T, kRes>} * sms);
  if (blocks == 0) return cudaSuccess;
  return launch_after(dropout_kernel<T, kRes>, dim3(static_cast<unsigned>(blocks)), kThreads, pdl, stream, a);
}
}  // namespace

cudaError_t dropout_launch(const DropoutKernelArgs& a, bool f32, int sms, bool pdl, cudaStream_t stream) {
  if (f32)
    return a.residual ? dropout_start<float, true>(a, sms, pdl, stream)
                      : dropout_start<float, false>(a, sms, pdl, stream);
  return a.residual ? dropout_start<uint16_t, true>(a, sms, pdl, stream)
                    : dropout_start<uint16_t, false>(a, sms, pdl, stream);
}

cudaError_t act_bwd_launch(const BwdKernelArgs& a, bool dy_f32, bool pdl, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  const int64_t groups = (a.rows + kBwdRows - 1) / kBwdRows;
  const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256),
                  static_cast<unsigned>(std::min<int64_t>(groups, 65535)));
  const bool drop = a.drop.thr != 0;
  if (dy_f32)
    return drop ? act_bwd_start<float, true>(a, grid, pdl, stream) : act_bwd_start<float, false>(a, grid, pdl, stream);
  return drop ? act_bwd_start<uint16_t, true>(a, grid, pdl, stream)
              : act_bwd_start<uint16_t, false>(a, grid, pdl, stream);
}

int64_t act_bwd_groups(int64_t rows) { return (rows + kBwdRows - 1) / kBwdRows; }

cudaError_t colsum_launch(const float* part, int64_t ld, int64_t groups, int64_t cols, float* out, bool pdl,
                          cudaStream_t stream) {
  if (cols == 0) return cudaSuccess;
  return launch_after(colsum_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), kThreads, pdl, stream, part, ld,
                      groups, cols, out);
}

}  // namespace axonn
