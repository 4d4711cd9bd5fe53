// Products of the linear cross entropy, z = X . W over a range of the
// vocabulary, whose epilogues keep no logits:
//   statistics     (max, sum of exp) of each row over the columns of one
//                  epilogue warp, the label's logit, and (for the piece of
//                  the vocabulary that stays) how far each logit lies below
//                  that maximum, in 16 bits (see kCeStep)
//   probabilities  P = e^(z - lse) - [v = label] in bf16, for columns
//                  that did not stay
// All in fp32 up to that one rounding.  A thread owns a row, so neither the
// maximum nor the sum needs another lane.
#include "fused_gemm.cuh"

namespace axonn {
namespace {

struct NoState {};

// 32 distances of one row (n exist) in steps of 1 / kCeStep, up to kCeFar.
__device__ __forceinline__ void store_distance32(uint16_t* p, int n, const float (&x)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t lo = __float2uint_rn(fminf(x[2 * j] * kCeStep, static_cast<float>(kCeFar)));
    const uint32_t hi = __float2uint_rn(fminf(x[2 * j + 1] * kCeStep, static_cast<float>(kCeFar)));
    w[j] = __byte_perm(lo, hi, 0x5410);
  }
  store_row32_u16(p, n, w);
}

struct StatsEpilogue {
  using Args = CeArgs;
  using State = NoState;
  static __device__ __forceinline__ State begin(const Args&) { return {}; }

  template <int kCols, class Ready>
  static __device__ __forceinline__ bool run(const Args& a, const State&, const EpiTile& t, Ready&& ready) {
    const bool in = t.row < t.M;
    const int width = min(kCols, t.N - t.col);
    // the label's place among this warp's columns (outside: another warp's)
    const int64_t y = in ? a.labels[t.row] - a.col0 - t.col : -1;
    if (!ready()) return false;
    if (width <= 0) return true;
    float m = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kCols / 32 && 32 * c < width; ++c) {
      float x[32];
      load_acc32(t, c, x);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (32 * c + j < width) m = fmaxf(m, x[j]);  // skips NaN, which the sum then shows
    }
    // A row whose every logit is -inf sums to 0 (not to e^(-inf + inf)).
    const float mb = m == -INFINITY ? 0.0f : m * kEpiLog2e;
    float s = 0.0f;
#pragma unroll 1
    for (int c = 0; c < kCols / 32 && 32 * c < width; ++c) {
      float x[32];
      load_acc32(t, c, x);
      const int64_t d = y - 32 * c;
      if (d >= 0 && d < 32 && d < width - 32 * c) {
        float zy = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == d) zy = x[j];
        a.label_logit[t.row] = zy;
      }
      // distance below the maximum, in powers of two
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = 32 * c + j < width ? fmaf(x[j], -kEpiLog2e, mb) : INFINITY;
      if (a.piece && in) store_distance32(a.piece + t.row * a.ld_piece + t.col + 32 * c, width - 32 * c, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = ex2_approx(-x[j]);
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        s0 += x[j];
        s1 += x[j + 1];
      }
      s += s0 + s1;
    }
    if (in) a.stats[((a.col0 + t.col) / kCols) * a.ld_stats + t.row] = make_float2(m, s);
    return true;
  }
};

struct ProbEpilogue {
  using Args = CeArgs;
  using State = NoState;
  static __device__ __forceinline__ State begin(const Args&) { return {}; }

  template <int kCols, class Ready>
  static __device__ __forceinline__ bool run(const Args& a, const State&, const EpiTile& t, Ready&& ready) {
    const bool in = t.row < t.M;
    // Rows up to the next multiple of 64 are zeros: the weight gradient's
    // reduction runs over them.
    const bool pad = !in && t.row < ((t.M + 63) & ~63) && t.row < a.rows;
    const int64_t y = in ? a.labels[t.row] - a.col0 - t.col : -1;
    const float lse2 = in ? a.lse2[t.row] : 0.0f;
    if (!ready()) return false;
#pragma unroll 1
    for (int c = 0; c < kCols / 32; ++c) {
      const int col = t.col + 32 * c, n = t.N - col;
      if (n <= 0) break;
      float x[32];
      load_acc32(t, c, x);
      const int64_t d = y - 32 * c;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float p = ex2_approx(fmaf(x[j], kEpiLog2e, -lse2));
        if (j == d) p -= 1.0f;
        x[j] = in ? p : 0.0f;
      }
      if (in || pad) store_row32_bf16(a.piece + t.row * a.ld_piece + col, n, x);
    }
    return true;
  }
};

// The products that follow: a tile as it is, rows possibly scattered.
struct StoreEpilogue {
  using Args = StoreArgs;
  using State = NoState;
  static __device__ __forceinline__ State begin(const Args&) { return {}; }

  static __device__ __forceinline__ void store(const Args& a, int64_t row, int col, int n, bool has,
                                               const float (&x)[32]) {
    if (a.mode == kOutBF16) {
      store_row32_bf16(reinterpret_cast<uint16_t*>(a.out) + row * a.ld_out + col, n, x);
      return;
    }
    float* o = reinterpret_cast<float*>(a.out) + row * a.ld_out + col;
    if (a.mode == kOutF32) {
      store_row32_f32(o, n, x);
    } else if (has) {  // one writer an element: the reduction rounds as a load-add-store would
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        if (j + 4 <= n) {
          red_add_v4_f32(o + j, __float_as_uint(x[j]), __float_as_uint(x[j + 1]), __float_as_uint(x[j + 2]),
                         __float_as_uint(x[j + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j + i < n) red_add_f32(o + j + i, __float_as_uint(x[j + i]));
        }
      }
    }
  }

  template <int kCols, class Ready>
  static __device__ __forceinline__ bool run(const Args& a, const State&, const EpiTile& t, Ready&& ready) {
    const bool in = t.row < t.M;
    const int64_t row = in && a.row_map ? a.row_map[t.row] : t.row;
    const float scale = a.scale ? *a.scale : 1.0f;
    if (!ready()) return false;
#pragma unroll 1
    for (int c = 0; c < kCols / 32; ++c) {
      const int col = t.col + 32 * c, n = t.N - col;
      if (n <= 0) break;
      float x[32];
      load_acc32(t, c, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] *= scale;
      if (in) store(a, row, col, n, t.has, x);
    }
    return true;
  }
};

}  // namespace

cudaError_t ce_init() {
  cudaError_t e = fused_init_all<StatsEpilogue>();
  if (e == cudaSuccess) e = fused_init_all<ProbEpilogue>();
  return e == cudaSuccess ? fused_init_all<StoreEpilogue>() : e;
}

cudaError_t store_launch(int config, const FusedParams<StoreArgs>& p, int units, bool pdl,
                         cudaStream_t stream) {
  return fused_launch_config<StoreEpilogue>(config, p, units, pdl, stream);
}

cudaError_t ce_launch(CeKind kind, int config, const FusedParams<CeArgs>& p, int units, bool pdl,
                      cudaStream_t stream) {
  return kind == kCeStats ? fused_launch_config<StatsEpilogue>(config, p, units, pdl, stream)
                          : fused_launch_config<ProbEpilogue>(config, p, units, pdl, stream);
}

cudaError_t ce_take_status(unsigned long long* word, cudaStream_t stream) {
  return fused_read_status(word, stream);
}

}  // namespace axonn
