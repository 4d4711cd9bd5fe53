// Products of one or two rows, with the epilogues of the fused products: a
// layer answering single tokens.  B is read once and nothing else counts (one
// row, 6144 x 24576: 302 MB), so there are no tiles and no tensor cores:
// every thread streams 16-byte vectors of B and multiplies them into fp32
// sums, and what is designed is the number of bytes in flight.  The
// reduction is cut over the CTAs of a cluster (see gemv_launch), so that
// short layers keep every SM loading too; their partial sums meet in shared
// memory, in a fixed order, and each CTA finishes its share of the columns.
// HBM-bound: the layer above with GELU takes 50.2 us called again and again
// and 61.4 after other work has filled L2, 6.0 and 4.9 TB/s; 128 x 128 tiles
// of the fused product take 86 (192 tiles are 1.3 rounds).
#include <algorithm>
#include <type_traits>

#include "gemv.h"
#include "vec8.cuh"

namespace axonn {
namespace {

constexpr int kThreads = 256, kWarps = 8;

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint4 load_vec(const uint16_t* p, int64_t left) {
  if (left >= 8) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ F2 pair_of(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// One thread's columns col .. col + 7 (n of them exist) of every row, from
// sums v[row].
template <bool kFwd, bool kF32, int TM>
__device__ __forceinline__ void finish_columns(const GemvArgs& p, int64_t col, int n, float (&v)[TM][8]) {
  const EpilogueArgs& a = p.epi;
  using T = typename std::conditional<kF32, float, uint16_t>::type;
  const DropRng rng = load_rng(a.drop);
  float sum[8] = {};
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    if (m >= p.M) break;
    float(&x)[8] = v[m];
    if constexpr (kFwd) {
      if (a.bias) {
        float b[8];
        if (a.bias_f32) {
          Vec8<float> w;
          w.load(static_cast<const float*>(a.bias) + col, n);
          w.values(b);
        } else {
          Vec8<uint16_t> w;
          w.load(static_cast<const uint16_t*>(a.bias) + col, n);
          w.values(b);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += b[j];
      }
      if (a.pre_out) store8(static_cast<uint16_t*>(p.out2) + m * p.ld_out2 + col, n, x);
      switch (a.act) {
        case kActRelu: act_values<kActRelu, 8>(x); break;
        case kActGelu: act_values<kActGelu, 8>(x); break;
        case kActGeluTanh: act_values<kActGeluTanh, 8>(x); break;
        case kActSilu: act_values<kActSilu, 8>(x); break;
        default: break;
      }
    }
    if (a.drop.thr != 0) drop8(a.drop, rng, m, static_cast<uint32_t>(col / 8), x);
    if constexpr (!kFwd) {
      if (a.act != kActNone) {
        Vec8<uint16_t> z;
        z.load(a.pre_in + m * a.ld_pre + col, n);
        switch (a.act) {
          case kActRelu: act_slopes<kActRelu, 8>(x, z.w); break;
          case kActGelu: act_slopes<kActGelu, 8>(x, z.w); break;
          case kActGeluTanh: act_slopes<kActGeluTanh, 8>(x, z.w); break;
          case kActSilu: act_slopes<kActSilu, 8>(x, z.w); break;
          default: break;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += x[j];
    }
    if (a.residual) {
      Vec8<T> r;
      float b[8];
      r.load(static_cast<const T*>(a.residual) + m * a.ld_res + col, n);
      r.values(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] += b[j];
    }
    store8(static_cast<T*>(p.out) + m * p.ld_out + col, n, x);
  }
  if (!kFwd && a.colsum) store8(a.colsum + col, n, sum);  // one group of rows
}

// CB columns a CTA.  kMN: B stored [R x N], a warp reads 256 / CB rows of CB
// columns at a time, a lane eight columns.  Else B stored [N x R]: a warp has
// eight columns, its lanes split the reduction.
// Six CTAs an SM for one row: 768 of them (6144 x 24576) are then resident at
// once; at four, the last 160 ran as a second wave.
template <bool kMN, int TM>
constexpr int kResident = TM == 1 ? (kMN ? 6 : 4) : 3;
template <bool kFwd, bool kF32, bool kMN, int TM, int CB>
__global__ void __launch_bounds__(kThreads, kResident<kMN, TM>) gemv_kernel(const GemvArgs p) {
  extern __shared__ float smem[];
  float* xs = smem;                          // [TM][p.piece]
  float* part = smem + TM * p.piece;         // [TM][CB], this CTA's sums
  float* sums = part + TM * CB;              // kMN: [kWarps][TM][CB]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), splits = static_cast<int>(cluster_nctarank());
  const int64_t col0 = static_cast<int64_t>(cluster_id_x()) * CB;
  const int64_t k0 = static_cast<int64_t>(rank) * p.piece;
  const int len = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(p.piece), p.R - k0)));
  griddep_wait();
  for (int i = threadIdx.x; i < TM * p.piece; i += kThreads) {
    const int m = i / p.piece, k = i - m * p.piece;
    float x = 0.0f;
    if (m < p.M && k < len) x = bf16_bits_f32(p.A[p.a_mn ? (k0 + k) * p.lda + m : m * p.lda + k0 + k]);
    xs[i] = x;
  }
  __syncthreads();

  if constexpr (kMN) {
    constexpr int kLanes = CB / 8, kRows = 32 / kLanes, kUnroll = TM == 1 ? 4 : 8;
    F2 acc[TM][4];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = f2(0.0f);
    const int64_t col = col0 + 8 * (lane % kLanes);
    const int64_t left = p.N - col;
    const uint16_t* b = p.B + k0 * p.ldb + col;
    const int first = warp * kRows + lane / kLanes;  // this thread's rows: first, + kWarps kRows, ...
    constexpr int kStep = kWarps * kRows;
    if (left > 0) {
      int k = first;
      for (; k + (kUnroll - 1) * kStep < len; k += kUnroll * kStep) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) w[u] = load_vec(b + (k + u * kStep) * p.ldb, left);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const F2 q[4] = {pair_of(w[u].x), pair_of(w[u].y), pair_of(w[u].z), pair_of(w[u].w)};
#pragma unroll
          for (int m = 0; m < TM; ++m) {
            const F2 x = f2(xs[m * p.piece + k + u * kStep]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][j] = fma2(q[j], x, acc[m][j]);
          }
        }
      }
      for (; k < len; k += kStep) {
        const uint4 w = load_vec(b + k * p.ldb, left);
        const F2 q[4] = {pair_of(w.x), pair_of(w.y), pair_of(w.z), pair_of(w.w)};
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const F2 x = f2(xs[m * p.piece + k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][j] = fma2(q[j], x, acc[m][j]);
        }
      }
    }
    // rows of the warp, then the warps in order
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        split(acc[m][j], lo, hi);
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
          lo += __shfl_xor_sync(0xFFFFFFFFu, lo, o);
          hi += __shfl_xor_sync(0xFFFFFFFFu, hi, o);
        }
        if (lane < kLanes) {
          sums[(warp * TM + m) * CB + 8 * lane + 2 * j] = lo;
          sums[(warp * TM + m) * CB + 8 * lane + 2 * j + 1] = hi;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < TM * CB; i += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * TM * CB + i];
      part[i] = s;
    }
  } else {
    static_assert(CB == 8 * kWarps, "a warp's eight columns");
    constexpr int kCols = 4, kUnroll = 8 / kCols;  // columns at a time, 256-element steps in flight
#pragma unroll 1
    for (int half = 0; half < 8 / kCols; ++half) {
      const int64_t n0 = col0 + 8 * warp + kCols * half;
      F2 acc[kCols][TM];
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[c][m] = f2(0.0f);
      for (int k = 8 * lane; k < len; k += 256 * kUnroll) {
        uint4 w[kUnroll][kCols];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            w[u][c] = make_uint4(0, 0, 0, 0);
            if (n0 + c < p.N && k + 256 * u < len)
              w[u][c] = load_vec(p.B + (n0 + c) * p.ldb + k0 + k + 256 * u, len - k - 256 * u);
          }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (k + 256 * u >= len) break;
#pragma unroll
          for (int m = 0; m < TM; ++m) {
            // p.piece is a multiple of 8 and zero-filled past len
            const float4* xp = reinterpret_cast<const float4*>(xs + m * p.piece + k + 256 * u);
            const float4 xa = xp[0], xb = xp[1];
            const F2 x[4] = {f2(xa.x, xa.y), f2(xa.z, xa.w), f2(xb.x, xb.y), f2(xb.z, xb.w)};
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              acc[c][m] = fma2(pair_of(w[u][c].x), x[0], acc[c][m]);
              acc[c][m] = fma2(pair_of(w[u][c].y), x[1], acc[c][m]);
              acc[c][m] = fma2(pair_of(w[u][c].z), x[2], acc[c][m]);
              acc[c][m] = fma2(pair_of(w[u][c].w), x[3], acc[c][m]);
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          float lo, hi;
          split(acc[c][m], lo, hi);
          float s = lo + hi;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
          if (lane == 0) part[m * CB + 8 * warp + kCols * half + c] = s;
        }
    }
  }
  griddep_launch_dependents();
  // Every CTA's sums are there; CTA r finishes the column groups r, r +
  // splits, ..., and no CTA leaves before all have read its sums.
  cluster_sync();
  const int group = rank + splits * static_cast<int>(threadIdx.x);
  if (group < CB / 8 && col0 + 8 * group < p.N) {
    float v[TM][8];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[m][j] = 0.0f;
    for (int s = 0; s < splits; ++s) {
      const uint32_t at = mapa_shared(smem_addr(part), s);
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[m][j] += ld_cluster_f32(at + 4u * (m * CB + 8 * group + j));
    }
    const int64_t col = col0 + 8 * group;
    finish_columns<kFwd, kF32, TM>(p, col, static_cast<int>(min(static_cast<int64_t>(8), p.N - col)), v);
  }
  cluster_sync();
}

template <bool kMN, int TM, int CB>
constexpr int smem_bytes(int piece) {
  return 4 * (TM * piece + TM * CB + (kMN ? kWarps * TM * CB : 0));
}
constexpr int kDefaultSmem = 48 * 1024;  // what a kernel has without asking

// The most that a call can need (see gemv_launch), asked for once: the limit
// is the kernel's, not the launch's, so that a call that set its own would
// change it under another thread's.
template <bool kFwd, bool kF32, bool kMN, int TM, int CB>
cudaError_t allow_smem() {
  constexpr int kMost = smem_bytes<kMN, TM, CB>(static_cast<int>(kGemvPiece));
  if (kMost <= kDefaultSmem) return cudaSuccess;
  return cudaFuncSetAttribute(gemv_kernel<kFwd, kF32, kMN, TM, CB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kMost);
}

template <bool kFwd, bool kF32>
cudaError_t allow_layouts() {
  for (cudaError_t e : {allow_smem<kFwd, kF32, true, 1, 256>(), allow_smem<kFwd, kF32, true, 1, 64>(),
                        allow_smem<kFwd, kF32, false, 1, 64>(), allow_smem<kFwd, kF32, true, 2, 64>(),
                        allow_smem<kFwd, kF32, false, 2, 64>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <bool kFwd, bool kF32, bool kMN, int TM, int CB>
cudaError_t start(const GemvArgs& p, int splits, bool pdl, cudaStream_t stream) {
  auto kernel = gemv_kernel<kFwd, kF32, kMN, TM, CB>;
  const int smem = smem_bytes<kMN, TM, CB>(p.piece);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + CB - 1) / CB * splits), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kFwd, bool kF32, int TM>
cudaError_t start_layout(const GemvArgs& p, bool b_mn, int cols, int splits, bool pdl, cudaStream_t stream) {
  if (!b_mn) return start<kFwd, kF32, false, TM, 64>(p, splits, pdl, stream);
  if constexpr (TM == 1)
    if (cols == 256) return start<kFwd, kF32, true, 1, 256>(p, splits, pdl, stream);
  return start<kFwd, kF32, true, TM, 64>(p, splits, pdl, stream);
}

template <bool kFwd, bool kF32>
cudaError_t start_rows(const GemvArgs& p, bool b_mn, int cols, int splits, bool pdl, cudaStream_t stream) {
  if (p.M == 1) return start_layout<kFwd, kF32, 1>(p, b_mn, cols, splits, pdl, stream);
  return start_layout<kFwd, kF32, 2>(p, b_mn, cols, splits, pdl, stream);
}

}  // namespace

cudaError_t gemv_init() {
  for (cudaError_t e : {allow_layouts<false, false>(), allow_layouts<false, true>(), allow_layouts<true, false>(),
                        allow_layouts<true, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t gemv_launch(FusedKind kind, GemvArgs p, bool b_mn, int sms, bool pdl, cudaStream_t stream) {
  // The reduction in at most eight pieces of at least 256.  One row of a
  // row-major B takes them all, with 256 columns a CTA (whole 512-byte rows)
  // where that still leaves four CTAs for every SM.  The others stop at two
  // CTAs an SM (of pieces that leave several room in shared memory): a longer
  // piece starts its stream and meets its cluster less often.  Two rows, us
  // by 1, 2, 4 and 8 pieces: 6144 x 24576 64, 68, 74 and 65 (68, 70, 74 and 93
  // stored transposed), 24576 x 6144 137, 111, 66 and 70.
  const bool wide = b_mn && p.M == 1;
  int most = 1;
  while (most < 8 && p.R / (2 * most) >= 256) most *= 2;
  int splits = wide ? most : 1;
  while (splits < most && ((p.N + 63) / 64 * splits < 2 * sms || p.R > kGemvPiece * splits)) splits *= 2;
  p.piece = static_cast<int>(((p.R + splits - 1) / splits + 7) / 8 * 8);
  const int cols = wide && (p.N + 255) / 256 * splits >= 4 * sms ? 256 : 64;
  if (kind == kFusedFwd)
    return p.epi.out_f32 ? start_rows<true, true>(p, b_mn, cols, splits, pdl, stream)
                         : start_rows<true, false>(p, b_mn, cols, splits, pdl, stream);
  return p.epi.out_f32 ? start_rows<false, true>(p, b_mn, cols, splits, pdl, stream)
                       : start_rows<false, false>(p, b_mn, cols, splits, pdl, stream);
}

// One and two rows always.  GELU product, us, here and with the best of the
// fused forms (B cold in L2): one row 6144 x 24576 61 and 86, 24576 x 6144 66
// and 78, 768 x 768 10.3 and 12.5; two rows 6144 x 24576 64 and 86, 24576 x
// 6144 66 and 78.  Four rows have too much to multiply: 90 and 86, 96 and 78.
bool gemv_wins(int64_t M, int64_t R) { return M >= 1 && M <= kGemvRows && R <= kGemvReduction; }

}  // namespace axonn
