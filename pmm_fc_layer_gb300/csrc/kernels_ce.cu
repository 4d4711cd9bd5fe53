// Products of the linear cross entropy, z = X . W over a range of the
// vocabulary, whose epilogues keep no logits:
//   statistics     (max, sum of exp) of each row over the columns of one
//                  epilogue warp, the label's logit, and (for the piece of
//                  the vocabulary that stays) how far each logit lies below
//                  that maximum, in 16 bits (see kCeStep)
//   probabilities  P = e^(z - lse) - [v = label] in bf16, for columns
//                  that did not stay
// All in fp32 up to that one rounding.  A thread owns a row, so neither the
// maximum nor the sum needs another lane.  Tensor-bound at long reductions:
// the statistics of 4096 x 6144 x 128256 take 3.4 to 3.5 ms (1.85 to 1.9
// PFLOP/s).  490 x 768 x 50257 takes 52 us with cold caches, two and a half
// times its flops: a short reduction leaves its epilogue to be seen (a plain
// product there takes 42).
#include "fused_gemm.cuh"

namespace axonn {
namespace {

struct NoState {};

// The distances -x of 32 logits below their maximum, x <= 0 in powers of two,
// in steps of 1 / kCeStep up to kCeFar: a saturating product (also of the
// rounding that leaves x above 0), then the low bits of 2^23 + q.
__device__ __forceinline__ void store_distances(const EpiTile& t, int col, const float (&x)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float lo = __saturatef(x[2 * j] * (-kCeStep / static_cast<float>(kCeFar)));
    float hi = __saturatef(x[2 * j + 1] * (-kCeStep / static_cast<float>(kCeFar)));
    split(fma2(f2(lo, hi), f2(static_cast<float>(kCeFar)), f2(8388608.0f)), lo, hi);
    w[j] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
  }
  store_segment<uint16_t>(t, t.out, col, w);
}

// Columns past the vocabulary's end become -inf: no maximum, nothing in the
// sum, far in the piece.
__device__ __forceinline__ void drop_columns(float (&x)[32], int width) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j >= width) x[j] = -INFINITY;
}

struct StatsEpilogue {
  using Args = CeArgs;
  using State = NoState;
  static constexpr int kEachStages = 16;
  static __device__ __forceinline__ State begin(const Args&) { return {}; }

  template <int kCols, bool kHold, class Ready, class Release>
  static __device__ __forceinline__ bool run(const Args& a, const State&, const EpiTile& t, Ready&& ready,
                                             Release&& release) {
    const bool in = t.row < t.M;
    const int width = min(kCols, t.N - t.col);
    // the label's place among this warp's columns (outside: another warp's)
    const int64_t y = in ? a.labels[t.row] - a.col0 - t.col : -1;
    if (!ready()) return false;
    float m = -INFINITY, s = 0.0f, mb = 0.0f;
    auto take_max = [&](int c, float(&x)[32]) {
      if (32 * c + 32 > width) drop_columns(x, width - 32 * c);
#pragma unroll
      for (int j = 0; j < 32; ++j) m = fmaxf(m, x[j]);  // skips NaN, which the sum then shows
    };
    auto take_sum = [&](int c, float(&x)[32]) {
      const int64_t d = y - 32 * c;
      if (d >= 0 && d < 32 && d < width - 32 * c) {
        float zy = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == d) zy = x[j];
        a.label_logit[t.row] = zy;
      }
      // minus the distance below the maximum, in powers of two
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        split(fma2(f2(x[j], x[j + 1]), f2(kEpiLog2e), f2(-mb)), x[j], x[j + 1]);
      if (a.keep_piece) store_distances(t, t.col + 32 * c, x);
      F2 sum = f2(0.0f);
#pragma unroll
      for (int j = 0; j < 32; j += 2) sum = add2(sum, f2(ex2_approx(x[j]), ex2_approx(x[j + 1])));
      float s0, s1;
      split(sum, s0, s1);
      s += s0 + s1;
    };
    // A row whose every logit is -inf sums to 0 (not to e^(-inf + inf)).
    auto set_base = [&]() { mb = m == -INFINITY ? 0.0f : m * kEpiLog2e; };
    if constexpr (kHold) {  // the columns stay in registers
      float x[kCols / 32][32];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        if (32 * c < width) {
          load_acc32(t, c, x[c]);
          take_max(c, x[c]);
        }
      }
      release();
      set_base();
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c)
        if (32 * c < width) take_sum(c, x[c]);
    } else {  // they are read twice
      float x[32];
#pragma unroll 1
      for (int c = 0; c < kCols / 32 && 32 * c < width; ++c) {
        load_acc32(t, c, x);
        take_max(c, x);
      }
      set_base();
#pragma unroll 1
      for (int c = 0; c < kCols / 32 && 32 * c < width; ++c) {
        load_acc32(t, c, x);
        if (32 * c + 32 > width) drop_columns(x, width - 32 * c);
        take_sum(c, x);
      }
    }
    if (!kHold) release();
    if (in && width > 0) a.stats[((a.col0 + t.col) / kCols) * a.ld_stats + t.row] = make_float2(m, s);
    return true;
  }
};

struct ProbEpilogue {
  using Args = CeArgs;
  using State = NoState;
  static constexpr int kEachStages = 16;
  static __device__ __forceinline__ State begin(const Args&) { return {}; }
  static __device__ __forceinline__ void prefetch(const Args&, const EpiTile&, int) {}

  static __device__ __forceinline__ void step(const Args& a, const State&, const EpiTile& t, int c,
                                              float (&x)[32]) {
    const bool in = t.row < t.M;
    const int col = t.col + 32 * c;
    const int64_t d = in ? a.labels[t.row] - a.col0 - col : -1;
    const float lse2 = in ? a.lse2[t.row] : 0.0f;
    // Rows past the last, up to the next multiple of 64 (of those there are),
    // are zeros: the weight gradient's reduction runs over them.
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float p = ex2_approx(fmaf(x[j], kEpiLog2e, -lse2));
      if (j == d) p -= 1.0f;
      x[j] = in ? p : 0.0f;
    }
    EpiTile padded = t;
    padded.rows = static_cast<int>(min(static_cast<int64_t>((t.M + 63) & ~63), a.rows));
    store_bf16(padded, t.out, col, x);
  }

  template <int kCols, bool kHold, class Ready, class Release>
  static __device__ __forceinline__ bool run(const Args& a, const State& st, const EpiTile& t, Ready&& ready,
                                             Release&& release) {
    return epilogue_steps<ProbEpilogue, kCols, kHold>(a, st, t, ready, release);
  }
};

// The products that follow: a tile times a number.
struct StoreEpilogue {
  using Args = StoreArgs;
  using State = float;  // the scale
  static constexpr int kEachStages = 8;
  static __device__ __forceinline__ State begin(const Args& a) { return a.scale ? *a.scale : 1.0f; }

  static __device__ __forceinline__ void prefetch(const Args&, const EpiTile&, int) {}

  static __device__ __forceinline__ void step(const Args& a, const State& scale, const EpiTile& t, int c,
                                              float (&x)[32]) {
    const int col = t.col + 32 * c, n = t.N - col;
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] *= scale;
    if (a.mode == kOutBF16) {
      store_bf16(t, t.out, col, x);
    } else if (a.mode == kOutF32) {
      store_f32(t, t.out, col, x);
    } else if (t.has && t.row < t.M) {
      // added by the L2's reductions: one writer an element, so that they
      // round as a load-add-store would
      float* o = static_cast<float*>(t.out->base) + static_cast<int64_t>(t.row + t.row_off) * t.out->ld + col;
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

  template <int kCols, bool kHold, class Ready, class Release>
  static __device__ __forceinline__ bool run(const Args& a, const State& st, const EpiTile& t, Ready&& ready,
                                             Release&& release) {
    return epilogue_steps<StoreEpilogue, kCols, kHold>(a, st, t, ready, release);
  }
};

}  // namespace

cudaError_t ce_init(bool* regs_ok) {
  cudaError_t e = fused_init_all<StatsEpilogue>(regs_ok);
  if (e == cudaSuccess) e = fused_init_all<ProbEpilogue>(regs_ok);
  return e == cudaSuccess ? fused_init_all<StoreEpilogue>(regs_ok) : e;
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
