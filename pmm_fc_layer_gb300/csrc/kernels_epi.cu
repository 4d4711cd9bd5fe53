// Products with the training epilogues of an FC layer:
//   forward   Z = acc + b;  Y = R + D(act(Z))      (Z stored in bf16 if asked)
//   backward  d = act'(Z) D(acc);  dZ = d + R;  column sums of d
// Both are bound by the tensor cores wherever the reduction is long; the
// epilogue's arithmetic and its reads of R and Z run beside the next tile's
// mainloop.  A thread owns one row and walks its columns 32 at a time.
// Measured, 2.47e12 flops each, medians over four GPUs under the power cap
// (within 3 %): GELU + Z 8192 x 6144 x 24576 1545 us, dropout + residual 8192 x
// 24576 x 6144 1549, backward with GELU' and column sums 8192 x 6144 x 24576
// 1624 (1601, 1597 and 1523 TFLOP/s).
#include "fused_gemm.cuh"

namespace axonn {
namespace {

// The bias of 16 columns (n exist): every lane reads the same addresses.
__device__ __forceinline__ void add_bias16(const EpilogueArgs& a, int col, int n, float* x) {
  if (a.bias_f32) {
    Row16<true> b;
    b.load(a.bias, col, n);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] += b.value(j);
  } else {
    Row16<false> b;
    b.load(a.bias, col, n);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] += b.value(j);
  }
}

__device__ __forceinline__ void drop16(const DropoutArgs& d, const DropRng& g, int row, int col, float* x) {
#pragma unroll
  for (int o = 0; o < 2; ++o) drop8(d, g, static_cast<uint32_t>(row), static_cast<uint32_t>(col) / 8 + o, x + 8 * o);
}

// L2 lines of `cols` columns of a thread's row.
__device__ __forceinline__ void prefetch_row(const void* base, int64_t at, int cols, int bytes) {
  const char* p = static_cast<const char*>(base) + at * bytes;
  for (int b = 0; b < cols * bytes; b += 128) prefetch_l2(p + b);
}

// R over 32 columns: bf16 in one segment, fp32 in two.
template <bool kF32>
struct Residual {
  RowSegment<uint16_t> half;
  __device__ __forceinline__ void start(const EpilogueArgs& a, const EpiTile& t, int col) {
    if constexpr (!kF32) half.start(t, a.residual, a.ld_res, col);
  }
  __device__ __forceinline__ void add(const EpilogueArgs& a, const EpiTile& t, int col, float (&x)[32]) {
    uint32_t w[16];
    if constexpr (!kF32) {
      half.finish(t, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[2 * j] += __uint_as_float(w[j] << 16);
        x[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (col + 16 * h >= t.N) break;
        RowSegment<uint32_t> r;
        r.start(t, a.residual, a.ld_res, col + 16 * h);
        r.finish(t, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[16 * h + j] += __uint_as_float(w[j]);
      }
    }
  }
};

// kF32: the output and the residual are fp32 (else bf16).
template <bool kF32>
__device__ __forceinline__ void store_out(const EpiTile& t, int col, const float (&x)[32]) {
  if constexpr (kF32) store_f32(t, t.out, col, x);
  else store_bf16(t, t.out, col, x);
}

// kJoin: there is dropout or a residual.  The 20-warp kernels hold 64 words a
// thread and spill with either compiled in, which costs the plain form 3 %.
template <bool kF32, bool kJoin>
struct FwdEpilogue {
  using Args = EpilogueArgs;
  using State = DropRng;
  static constexpr int kEachStages = kJoin ? 16 : 8;
  static __device__ __forceinline__ State begin(const Args& a) { return load_rng(a.drop); }

  static __device__ __forceinline__ void prefetch(const Args& a, const EpiTile& t, int cols) {
    if (kJoin && a.residual) prefetch_row(a.residual, t.row * a.ld_res + t.col, cols, kF32 ? 4 : 2);
  }

  static __device__ __forceinline__ void step(const Args& a, const State& rng, const EpiTile& t, int c,
                                              float (&x)[32]) {
    const int col = t.col + 32 * c;
    if (a.bias) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (col + 16 * h < t.N) add_bias16(a, col + 16 * h, t.N - col - 16 * h, x + 16 * h);
    }
    if (a.pre_out) store_bf16(t, t.out2, col, x);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      apply_act16(a.act, x + 16 * h);
      if (kJoin && a.drop.thr != 0) drop16(a.drop, rng, t.row, col + 16 * h, x + 16 * h);
    }
    if (kJoin && a.residual) {
      Residual<kF32> r;
      r.start(a, t, col);
      r.add(a, t, col, x);
    }
    store_out<kF32>(t, col, x);
  }

  template <int kCols, bool kHold, class Ready, class Release>
  static __device__ __forceinline__ bool run(const Args& a, const State& g, const EpiTile& t, Ready&& ready,
                                             Release&& release) {
    return epilogue_steps<FwdEpilogue, kCols, kHold>(a, g, t, ready, release);
  }
};

// Column sums over the 32 rows of a warp: at each step a lane keeps half of
// its columns and hands the other half to the lane across, so that 31
// shuffles (rather than 32 x 5) leave lane j with the sum of column j.  The
// order of the additions is fixed.  x is used up.
__device__ __forceinline__ float column_sum32(float (&x)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float give = up ? x[j] : x[j + w];
      x[j] = (up ? x[j + w] : x[j]) + __shfl_xor_sync(0xFFFFFFFFu, give, w);
    }
  }
  return x[0];
}

template <bool kF32, bool kJoin>
struct BwdEpilogue {
  using Args = EpilogueArgs;
  using State = DropRng;
  static constexpr int kEachStages = kJoin ? 16 : 8;
  static __device__ __forceinline__ State begin(const Args& a) { return load_rng(a.drop); }

  static __device__ __forceinline__ void prefetch(const Args& a, const EpiTile& t, int cols) {
    if (a.act != kActNone) prefetch_row(a.pre_in, t.row * a.ld_pre + t.col, cols, 2);
    if (kJoin && a.residual) prefetch_row(a.residual, t.row * a.ld_res + t.col, cols, kF32 ? 4 : 2);
  }

  static __device__ __forceinline__ void step(const Args& a, const State& rng, const EpiTile& t, int c,
                                              float (&x)[32]) {
    const int col = t.col + 32 * c;
    const bool in = t.row < t.M;
    if (kJoin && a.drop.thr != 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) drop16(a.drop, rng, t.row, col + 16 * h, x + 16 * h);
    }
    if (a.act != kActNone) {
      RowSegment<uint16_t> z;
      z.start(t, a.pre_in, a.ld_pre, col);
      uint32_t w[16];
      z.finish(t, w);
#pragma unroll
      for (int h = 0; h < 2; ++h) apply_slope16(a.act, x + 16 * h, w + 8 * h);
    }
    if (kJoin && a.residual) {
      Residual<kF32> r;
      r.start(a, t, col);
      if (!a.colsum) {
        r.add(a, t, col, x);
        store_out<kF32>(t, col, x);
        return;
      }
      float y[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = x[j];
      r.add(a, t, col, y);
      store_out<kF32>(t, col, y);
    } else {
      store_out<kF32>(t, col, x);
    }
    if (!a.colsum) return;
    // d without the residual; nothing from rows past the end.
    if (!in) {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = 0.0f;
    }
    __syncwarp();
    const float s = column_sum32(x);
    const int at = col + static_cast<int>(threadIdx.x & 31);
    const int64_t group = t.row >> 5;  // the same for the warp: its rows are 32-aligned
    if (at < t.N && (t.row & ~31) < t.M) a.colsum[group * a.ld_colsum + at] = s;
  }

  template <int kCols, bool kHold, class Ready, class Release>
  static __device__ __forceinline__ bool run(const Args& a, const State& g, const EpiTile& t, Ready&& ready,
                                             Release&& release) {
    return epilogue_steps<BwdEpilogue, kCols, kHold>(a, g, t, ready, release);
  }
};

}  // namespace

namespace {
template <template <bool, bool> class Epi>
cudaError_t cluster_init() {
  constexpr int kBytes = FusedLayout<128, kClusterStages, false, 1>::kBytes;
  for (cudaError_t e : {cudaFuncSetAttribute(fused_cluster_kernel<Epi<false, true>>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                        cudaFuncSetAttribute(fused_cluster_kernel<Epi<true, true>>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes)})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}
}  // namespace

cudaError_t fused_init(bool* regs_ok) {
  for (cudaError_t e :
       {fused_init_all<FwdEpilogue<false, false>>(regs_ok), fused_init_all<FwdEpilogue<false, true>>(regs_ok),
        fused_init_all<FwdEpilogue<true, false>>(regs_ok), fused_init_all<FwdEpilogue<true, true>>(regs_ok),
        fused_init_all<BwdEpilogue<false, false>>(regs_ok), fused_init_all<BwdEpilogue<false, true>>(regs_ok),
        fused_init_all<BwdEpilogue<true, false>>(regs_ok), fused_init_all<BwdEpilogue<true, true>>(regs_ok)})
    if (e != cudaSuccess) return e;
  for (cudaError_t e : {cluster_init<FwdEpilogue>(), cluster_init<BwdEpilogue>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

namespace {
template <template <bool, bool> class Epi>
cudaError_t launch_kind(int config, const FusedParams<EpilogueArgs>& p, int units, bool pdl, cudaStream_t s) {
  const bool join = p.epi.residual != nullptr || p.epi.drop.thr != 0;
  if (p.epi.out_f32)
    return join ? fused_launch_config<Epi<true, true>>(config, p, units, pdl, s)
                : fused_launch_config<Epi<true, false>>(config, p, units, pdl, s);
  return join ? fused_launch_config<Epi<false, true>>(config, p, units, pdl, s)
              : fused_launch_config<Epi<false, false>>(config, p, units, pdl, s);
}
}  // namespace

cudaError_t fused_launch(FusedKind kind, int config, const FusedParams<EpilogueArgs>& p, int units,
                         bool pdl, cudaStream_t stream) {
  return kind == kFusedFwd ? launch_kind<FwdEpilogue>(config, p, units, pdl, stream)
                           : launch_kind<BwdEpilogue>(config, p, units, pdl, stream);
}

cudaError_t fused_clusters_resident(int sms, int pieces, int* clusters) {
  using Epi = FwdEpilogue<false, true>;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = fused_cluster_config<Epi>(sms / pieces * pieces, pieces, attr);
  return cudaOccupancyMaxActiveClusters(clusters, reinterpret_cast<const void*>(fused_cluster_kernel<Epi>), &cfg);
}

cudaError_t fused_cluster(FusedKind kind, const FusedParams<EpilogueArgs>& p, int tiles, int pieces, bool pdl,
                          cudaStream_t stream) {
  if (kind == kFusedFwd)
    return p.epi.out_f32 ? fused_cluster_launch<FwdEpilogue<true, true>>(p, tiles, pieces, pdl, stream)
                         : fused_cluster_launch<FwdEpilogue<false, true>>(p, tiles, pieces, pdl, stream);
  return p.epi.out_f32 ? fused_cluster_launch<BwdEpilogue<true, true>>(p, tiles, pieces, pdl, stream)
                       : fused_cluster_launch<BwdEpilogue<false, true>>(p, tiles, pieces, pdl, stream);
}

cudaError_t fused_take_status(unsigned long long* word, cudaStream_t stream) {
  return fused_read_status(word, stream);
}

}  // namespace axonn
