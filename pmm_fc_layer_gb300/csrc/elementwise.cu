// Elementwise kernels beside the fused products, both bound by HBM:
//   dropout   Y = R + D(X)                       (bf16 or fp32)
//   backward  d = act'(Z) D(dY), dZ = d in bf16, column sums of d
// A thread owns eight consecutive columns of a row: one 16-byte vector of
// bf16 and one call of the generator, whose mask is therefore never stored.
#include <algorithm>

#include "elementwise.h"
#include "epilogue_math.cuh"

namespace axonn {
namespace {

constexpr int kThreads = 256;

// Eight elements of a row, n of them existing (the others are neither read
// nor written).  Full vectors are 16-byte aligned: base pointers and leading
// dimensions are checked by the host and columns are multiples of 8.
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&x)[8]) {
  if (n >= 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? bf16_bits_f32(p[j]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int n, float (&x)[8]) {
  if (n >= 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? p[j] : 0.0f;
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&x)[8]) {
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
__device__ __forceinline__ void store8(float* p, int n, const float (&x)[8]) {
  if (n >= 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = x[j];
  }
}

// The vectors of the matrix in row order, dealt out to the grid's threads.
// The row and column of a thread's next vector follow from the last by one
// addition and one wrap.
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutKernelArgs a) {
  const T* X = static_cast<const T*>(a.x);
  const T* R = static_cast<const T*>(a.residual);
  T* Y = static_cast<T*>(a.y);
  const int64_t n8 = (a.cols + 7) / 8;
  const int64_t total = a.rows * n8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= total) return;
  const DropRng g = load_rng(a.drop);
  const int64_t dr = stride / n8, dc = stride - dr * n8;
  int64_t row = i / n8, c8 = i - row * n8;
  for (; i < total; i += stride) {
    const int n = static_cast<int>(min(static_cast<int64_t>(8), a.cols - 8 * c8));
    float x[8], r[8];
    load8(X + row * a.ld_x + 8 * c8, n, x);
    if (R) load8(R + row * a.ld_res + 8 * c8, n, r);
    const uint32_t bits =
        a.drop.thr != 0 ? keep8(a.drop, g, static_cast<uint32_t>(row), static_cast<uint32_t>(c8)) : 0xFFu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // R + scale x in one rounding
      const float base = R ? r[j] : 0.0f;
      x[j] = (bits >> j) & 1u ? fmaf(x[j], a.drop.scale, base) : base;
    }
    store8(Y + row * a.ld_y + 8 * c8, n, x);
    row += dr;
    c8 += dc;
    if (c8 >= n8) {
      c8 -= n8;
      ++row;
    }
  }
}

// A block covers kBwdRows rows x 256 columns: each of its eight warps takes
// every eighth row, a lane eight columns.  A lane adds its rows' columns in
// order, the block its warps' sums in order: partial sums of kBwdRows rows.
constexpr int kBwdRows = 64;
static_assert(kBwdRows >= 32, "the partial sums' workspace holds one row of them per 32 rows");

template <typename T>
__global__ void __launch_bounds__(kThreads) act_bwd_kernel(BwdKernelArgs a) {
  __shared__ float part[8][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* dY = static_cast<const T*>(a.dy);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + 8 * lane;
  const int n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), a.cols - col)));
  const DropRng g = load_rng(a.drop);
  for (int64_t group = blockIdx.y; group * kBwdRows < a.rows; group += gridDim.y) {
    const int64_t r0 = group * kBwdRows;
    const int64_t r1 = min(a.rows, r0 + kBwdRows);
    float sum[8] = {};
    if (n > 0) {
#pragma unroll 4
      for (int64_t row = r0 + warp; row < r1; row += 8) {
        float x[8];
        load8(dY + row * a.ld_dy + col, n, x);
        if (a.act != kActNone) {
          float z[8];
          load8(a.pre + row * a.ld_pre + col, n, z);
          if (a.drop.thr != 0) drop8(a.drop, g, static_cast<uint32_t>(row), static_cast<uint32_t>(col / 8), x);
          apply_slope(a.act, x, z);
        } else if (a.drop.thr != 0) {
          drop8(a.drop, g, static_cast<uint32_t>(row), static_cast<uint32_t>(col / 8), x);
        }
        store8(a.dz + row * a.ld_dz + col, n, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += x[j];
      }
    }
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

// out[col] = sum over the groups' partial sums, in a fixed order: a warp's
// lanes take 32 columns, its eight warps every eighth group, then the warps'
// sums in order.
__global__ void __launch_bounds__(kThreads) colsum_kernel(const float* part, int64_t ld, int64_t groups,
                                                          int64_t cols, float* out) {
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

cudaError_t dropout_launch(const DropoutKernelArgs& a, bool f32, int sms, cudaStream_t stream) {
  const int64_t vectors = a.rows * ((a.cols + 7) / 8);
  const int64_t blocks = std::min<int64_t>((vectors + kThreads - 1) / kThreads, int64_t{8} * sms);
  if (blocks == 0) return cudaSuccess;
  if (f32) dropout_kernel<float><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  else dropout_kernel<uint16_t><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t act_bwd_launch(const BwdKernelArgs& a, bool dy_f32, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  const int64_t groups = (a.rows + kBwdRows - 1) / kBwdRows;
  const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256),
                  static_cast<unsigned>(std::min<int64_t>(groups, 65535)));
  if (dy_f32) act_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else act_bwd_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

int64_t act_bwd_groups(int64_t rows) { return (rows + kBwdRows - 1) / kBwdRows; }

cudaError_t colsum_launch(const float* part, int64_t ld, int64_t groups, int64_t cols, float* out,
                          cudaStream_t stream) {
  if (cols == 0) return cudaSuccess;
  colsum_kernel<<<static_cast<unsigned>((cols + 31) / 32), kThreads, 0, stream>>>(part, ld, groups, cols, out);
  return cudaGetLastError();
}

}  // namespace axonn
