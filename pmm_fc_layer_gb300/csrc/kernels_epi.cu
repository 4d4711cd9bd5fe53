// Products with the training epilogues of an FC layer:
//   forward   Z = acc + b;  Y = R + D(act(Z))      (Z stored in bf16 if asked)
//   backward  d = act'(Z) D(acc);  dZ = d + R;  column sums of d
// Both are bound by the tensor cores wherever the reduction is long; the
// epilogue's arithmetic and its reads of R and Z run beside the next tile's
// mainloop.  A thread owns one row and walks its columns 32 at a time.
#include "fused_gemm.cuh"

namespace axonn {
namespace {

// 32 elements of a row in the output's type, kept as loaded.
struct RowSegment {
  uint32_t w[32];
};
__device__ __forceinline__ void load_segment(RowSegment& s, const void* base, int64_t ld, bool f32, int row,
                                             int col, int n) {
  if (!f32) {
    uint32_t h[16];
    load_row32_bf16(reinterpret_cast<const uint16_t*>(base) + row * ld + col, n, h);
#pragma unroll
    for (int j = 0; j < 16; ++j) s.w[j] = h[j];
    return;
  }
  const float* p = reinterpret_cast<const float*>(base) + row * ld + col;
  if (n >= 32) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[v];
      s.w[4 * v] = a.x;
      s.w[4 * v + 1] = a.y;
      s.w[4 * v + 2] = a.z;
      s.w[4 * v + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) s.w[j] = j < n ? __float_as_uint(p[j]) : 0u;
  }
}
__device__ __forceinline__ void add_segment(const RowSegment& s, bool f32, float (&x)[32]) {
  if (f32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] += __uint_as_float(s.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x[2 * j] += __uint_as_float(s.w[j] << 16);
      x[2 * j + 1] += __uint_as_float(s.w[j] & 0xFFFF0000u);
    }
  }
}

// The bias of 32 columns (n exist): every lane reads the same addresses.
__device__ __forceinline__ void add_bias(const EpilogueArgs& a, int col, int n, float (&x)[32]) {
  if (a.bias_f32) {
    const float* b = reinterpret_cast<const float*>(a.bias) + col;
    if (n >= 32) {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float4 f = reinterpret_cast<const float4*>(b)[v];
        x[4 * v] += f.x;
        x[4 * v + 1] += f.y;
        x[4 * v + 2] += f.z;
        x[4 * v + 3] += f.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) x[j] += b[j];
    }
    return;
  }
  uint32_t w[16];
  load_row32_bf16(reinterpret_cast<const uint16_t*>(a.bias) + col, n, w);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    x[2 * j] += __uint_as_float(w[j] << 16);
    x[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store_out(const EpilogueArgs& a, int row, int col, int n, const float (&x)[32]) {
  if (a.out_f32) store_row32_f32(reinterpret_cast<float*>(a.out) + row * a.ld_out + col, n, x);
  else store_row32_bf16(reinterpret_cast<uint16_t*>(a.out) + row * a.ld_out + col, n, x);
}

__device__ __forceinline__ void drop32(const DropoutArgs& d, const DropRng& g, int row, int col, float (&x)[32]) {
#pragma unroll
  for (int o = 0; o < 4; ++o) drop8(d, g, static_cast<uint32_t>(row), static_cast<uint32_t>(col) / 8 + o, x + 8 * o);
}

struct FwdEpilogue {
  using Args = EpilogueArgs;
  using State = DropRng;
  static __device__ __forceinline__ State begin(const Args& a) { return load_rng(a.drop); }

  template <int kCols, class Ready>
  static __device__ __forceinline__ bool run(const Args& a, const State& g, const EpiTile& t, Ready&& ready) {
    const bool in = t.row < t.M;
    const bool res = a.residual != nullptr && in;
    RowSegment r;
    if (res && t.col < t.N) load_segment(r, a.residual, a.ld_res, a.out_f32, t.row, t.col, t.N - t.col);
    if (!ready()) return false;
#pragma unroll 1
    for (int c = 0; c < kCols / 32; ++c) {
      const int col = t.col + 32 * c, n = t.N - col;
      if (n <= 0) break;
      float x[32];
      load_acc32(t, c, x);
      if (a.bias) add_bias(a, col, n, x);
      if (a.pre_out && in) store_row32_bf16(a.pre_out + t.row * a.ld_pre + col, n, x);
      apply_act(a.act, x);
      if (a.drop.thr != 0) drop32(a.drop, g, t.row, col, x);
      if (res) {
        add_segment(r, a.out_f32, x);
        // the next columns' residual, before these are stored
        if (c + 1 < kCols / 32 && n > 32)
          load_segment(r, a.residual, a.ld_res, a.out_f32, t.row, col + 32, n - 32);
      }
      if (in) store_out(a, t.row, col, n, x);
    }
    return true;
  }
};

// Column sums over the 32 rows of a warp: at each step a lane keeps half of
// its columns and hands the other half to the lane across, so that 31
// shuffles (rather than 32 x 5) leave lane j with the sum of column j.  The
// order of the additions is fixed.
__device__ __forceinline__ float column_sum32(const float (&x)[32]) {
  const int lane = threadIdx.x & 31;
  float v[16];
  {
    const bool up = lane & 16;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      v[j] = (up ? x[j + 16] : x[j]) + __shfl_xor_sync(0xFFFFFFFFu, up ? x[j] : x[j + 16], 16);
  }
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int j = 0; j < w; ++j)
      v[j] = (up ? v[j + w] : v[j]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[j + w], w);
  }
  return v[0];
}

struct BwdEpilogue {
  using Args = EpilogueArgs;
  using State = DropRng;
  static __device__ __forceinline__ State begin(const Args& a) { return load_rng(a.drop); }

  template <int kCols, class Ready>
  static __device__ __forceinline__ bool run(const Args& a, const State& g, const EpiTile& t, Ready&& ready) {
    const bool in = t.row < t.M;
    const bool res = a.residual != nullptr && in;
    const bool slope = a.act != kActNone && in;
    const int lane = threadIdx.x & 31;
    RowSegment r;
    uint32_t zw[16] = {};
    if (t.col < t.N) {
      if (slope) load_row32_bf16(a.pre_in + t.row * a.ld_pre + t.col, t.N - t.col, zw);
      if (res) load_segment(r, a.residual, a.ld_res, a.out_f32, t.row, t.col, t.N - t.col);
    }
    if (!ready()) return false;
#pragma unroll 1
    for (int c = 0; c < kCols / 32; ++c) {
      const int col = t.col + 32 * c, n = t.N - col;
      if (n <= 0) break;
      const bool more = c + 1 < kCols / 32 && n > 32;
      float x[32];
      load_acc32(t, c, x);
      if (a.drop.thr != 0) drop32(a.drop, g, t.row, col, x);
      if (slope) {
        float z[32];
        unpack32(zw, z);
        if (more) load_row32_bf16(a.pre_in + t.row * a.ld_pre + col + 32, n - 32, zw);
        apply_slope(a.act, x, z);
      }
      if (a.colsum) {
        // Rows past the end hold zero-filled operands' products, which are
        // 0; they are set so here in any case (a NaN weight would not be).
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = in ? x[j] : 0.0f;
        const float s = column_sum32(y);
        const int64_t group = t.row >> 5;  // the same for the warp: rows are 32-aligned
        if (lane < n && (t.row & ~31) < t.M) a.colsum[group * a.ld_colsum + col + lane] = s;
      }
      if (res) {
        add_segment(r, a.out_f32, x);
        if (more) load_segment(r, a.residual, a.ld_res, a.out_f32, t.row, col + 32, n - 32);
      }
      if (in) store_out(a, t.row, col, n, x);
    }
    return true;
  }
};

}  // namespace

cudaError_t fused_init() {
  const cudaError_t e = fused_init_all<FwdEpilogue>();
  return e == cudaSuccess ? fused_init_all<BwdEpilogue>() : e;
}

cudaError_t fused_launch(FusedKind kind, int config, const FusedParams<EpilogueArgs>& p, int units,
                         bool pdl, cudaStream_t stream) {
  return kind == kFusedFwd ? fused_launch_config<FwdEpilogue>(config, p, units, pdl, stream)
                           : fused_launch_config<BwdEpilogue>(config, p, units, pdl, stream);
}

cudaError_t fused_take_status(unsigned long long* word, cudaStream_t stream) {
  return fused_read_status(word, stream);
}

}  // namespace axonn
