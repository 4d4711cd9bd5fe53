// bf16 product on the sm_103a tensor cores with an epilogue of the caller's
// choice: C[M x N] = A[M x R] . B[R x N] in fp32 TMEM accumulators, each
// handed to Epi while the next tile's products run.
//
// Persistent and warp-specialised like the plain products: warp 0 loads
// operand stages by TMA, warp 1 issues the MMAs, the others are the
// epilogue.  What differs is the balance.  A fused epilogue costs several
// times a plain store (an activation, a generator call for every eight
// elements, one or two operands to read), so
//  - the accumulator is always double-buffered in TMEM (2 x BN columns):
//    the epilogue has a whole tile's mainloop to finish in, where the
//    512 x 256 tile of the plain products would hold up the next tile's MMAs
//    for as long as the arithmetic takes;
//  - the 256-column tile has two epilogue warps per 32 rows, 128 columns
//    each;
//  - every operand that the epilogue reads is asked for before its use:
//    the first 32 columns before the accumulator is ready, the next 32
//    while the present ones are worked on.
// kPair: a CTA pair shares one 256 x 256 tile (cta_group::2), each CTA
// loading its 128 rows of A and its half of B (32 KB a stage, 6 stages).
// Waits are bounded, and an expired one is recorded and reported, as in the
// plain products.
#pragma once
#include "epilogue.h"
#include "epilogue_math.cuh"
#include "gemm_kernel.cuh"

namespace axonn {

template <int BN, int STAGES, bool kPair>
struct FusedLayout {
  static constexpr int kABytes = 128 * kBK * 2;
  static constexpr int kBCols = kPair ? BN / 2 : BN;  // columns of B one CTA loads
  static constexpr int kBBytes = kBCols * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kNumBars = 2 * STAGES + 5;
  static constexpr int kEpiWarpSets = BN == 256 ? 2 : 1;  // warps per 32 rows
  static constexpr int kEpi = 4 * kEpiWarpSets;
  static constexpr int kThreads = 64 + 32 * kEpi;
  static constexpr int kWarpCols = BN / kEpiWarpSets;
  // 1024 B of slack to align the ring, the ring, barriers, TMEM slot, abort
  static constexpr int kBytes = 1024 + STAGES * kStageBytes + kNumBars * 8 + 16;
};

// Tile t of the grouped rasterisation (see decode_tile in gemm_kernel.cuh):
// group_m > 0 walks that many tile rows before the next tile column,
// group_m < 0 that many tile columns before the next tile row.
__device__ __forceinline__ void fused_tile(int t, int group, int tiles_m, int tiles_n, int& mb, int& nb) {
  if (group > 0) {
    const int per = group * tiles_n, g = t / per, first = g * group;
    const int size = min(group, tiles_m - first), in = t - g * per;
    mb = first + in % size;
    nb = in / size;
  } else {
    const int gn = -group, per = gn * tiles_m, g = t / per, first = g * gn;
    const int size = min(gn, tiles_n - first), in = t - g * per;
    nb = first + in % size;
    mb = in / size;
  }
}

// One epilogue warp's part of a tile: TMEM address of its lanes and first
// column, its row of the output and the output columns [col, col + kCols).
struct EpiTile {
  uint32_t t_row;
  int row, col;
  int M, N;
  bool has;  // false: the reduction is empty and the accumulator is zero
};

__device__ __forceinline__ void load_acc32(const EpiTile& t, int c, float (&x)[32]) {
  uint32_t r[32];
  if (t.has) {
    __syncwarp();  // the whole warp loads: lanes past the last row come back from skipped stores
    tmem_ld_32x32b_x32(t.t_row + c * 32, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
  }
}

template <class Epi, int BN, int STAGES, bool kPair>
__global__ void __launch_bounds__(FusedLayout<BN, STAGES, kPair>::kThreads, 1)
    fused_gemm_kernel(const __grid_constant__ FusedParams<typename Epi::Args> P) {
  using L = FusedLayout<BN, STAGES, kPair>;
  constexpr uint32_t kAccCols = BN < 128 ? 128 : BN;  // TMEM columns of one accumulator
  constexpr uint32_t kTmemCols = 2 * kAccCols;
  constexpr int kTileM = kPair ? 256 : 128;
  static_assert(kTmemCols == 256 || kTmemCols == 512, "TMEM columns");

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_ptr + STAGES * L::kStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  auto full_bar = [&](int s) { return smem_addr(bars + s); };
  auto empty_bar = [&](int s) { return smem_addr(bars + STAGES + s); };
  auto tfull_bar = [&](int b) { return smem_addr(bars + 2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return smem_addr(bars + 2 * STAGES + 2 + b); };
  const uint32_t mma_done_bar = smem_addr(bars + 2 * STAGES + 4);
  auto a_tile = [&](int s) { return ring + s * L::kStageBytes; };
  auto b_tile = [&](int s) { return ring + s * L::kStageBytes + L::kABytes; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int units = kPair ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), (kPair ? 2 : 1) * L::kEpi);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0 && P.num_k > 0) {
    prefetch_tmap(&P.ta);
    prefetch_tmap(&P.tb);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t tmo = P.timeout_ns;
  griddep_wait();  // nothing above touches what the previous kernel writes
  int M = P.M, tiles_m = P.tiles_m, num_k = P.num_k;
  if (P.count_of != 0) {
    const int n = *P.count;
    if (P.count_of == 1) {
      M = n;
      tiles_m = (n + kTileM - 1) / kTileM;
    } else {
      num_k = (n + kBK - 1) / kBK;
    }
  }
  const int total = tiles_m * P.tiles_n;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && P.inject != 1) {
      int stage = 0;
      uint32_t phase = 0, loads = 0;
      bool ok = true;
      const uint64_t pol_a = l2_policy(P.l2_keep == 1, P.l2_keep_frac);
      const uint64_t pol_b = l2_policy(P.l2_keep == 2, P.l2_keep_frac);
      for (int t = unit; ok && t < total; t += units) {
        int mb, nb;
        fused_tile(t, P.group_m, tiles_m, P.tiles_n, mb, nb);
        const int m0 = mb * kTileM + static_cast<int>(rank) * 128;
        const int n0 = nb * BN + static_cast<int>(rank) * L::kBCols;
        for (int k = 0; k < num_k; ++k) {
          ok = wait_bounded(empty_bar(stage), phase ^ 1u, tmo, abort_flag, kSiteProducerEmpty);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(full_bar(stage), (kPair ? 2 : 1) * L::kStageBytes);
          const int r0 = k * kBK;
          if constexpr (kPair) {
            const uint32_t fb = mapa_shared(full_bar(stage), 0);
            if (P.a_3d) {
              tma_load_3d_pair(a_tile(stage), &P.ta, fb, 0, r0, m0 / 64, pol_a);
            } else if (P.a_mn) {
              tma_load_2d_pair(a_tile(stage), &P.ta, fb, m0, r0, pol_a);
              tma_load_2d_pair(a_tile(stage) + kBK * 128, &P.ta, fb, m0 + 64, r0, pol_a);
            } else {
              tma_load_2d_pair(a_tile(stage), &P.ta, fb, r0, m0, pol_a);
            }
            if (P.b_3d) {
              tma_load_3d_pair(b_tile(stage), &P.tb, fb, 0, r0, n0 / 64, pol_b);
            } else if (P.b_mn) {
#pragma unroll
              for (int h = 0; h < L::kBCols / 64; ++h)
                tma_load_2d_pair(b_tile(stage) + h * (kBK * 128), &P.tb, fb, n0 + 64 * h, r0, pol_b);
            } else {
              tma_load_2d_pair(b_tile(stage), &P.tb, fb, r0, n0, pol_b);
            }
          } else {
            const uint32_t fb = full_bar(stage);
            if (P.a_3d) {
              tma_load_3d(a_tile(stage), &P.ta, fb, 0, r0, m0 / 64, pol_a);
            } else if (P.a_mn) {
              tma_load_2d(a_tile(stage), &P.ta, fb, m0, r0, pol_a);
              tma_load_2d(a_tile(stage) + kBK * 128, &P.ta, fb, m0 + 64, r0, pol_a);
            } else {
              tma_load_2d(a_tile(stage), &P.ta, fb, r0, m0, pol_a);
            }
            if (P.b_3d) {
              tma_load_3d(b_tile(stage), &P.tb, fb, 0, r0, n0 / 64, pol_b);
            } else if (P.b_mn) {
#pragma unroll
              for (int h = 0; h < L::kBCols / 64; ++h)
                tma_load_2d(b_tile(stage) + h * (kBK * 128), &P.tb, fb, n0 + 64 * h, r0, pol_b);
            } else {
              tma_load_2d(b_tile(stage), &P.tb, fb, r0, n0, pol_b);
            }
          }
          ++loads;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      griddep_launch_dependents();
      // Drain: the last load of each stage lands before the CTA may exit (a
      // pair's loads all count on the even CTA's barriers).
      if (leader)
        for (int s = 0; s < STAGES; ++s)
          if (loads > static_cast<uint32_t>(s)) {
            const uint32_t n_s = (loads - s + STAGES - 1) / STAGES;
            wait_bounded(full_bar(s), (n_s - 1) & 1u, tmo, abort_flag, kSiteDrainLoads, false);
          }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader && num_k > 0) {
      int stage = 0;
      uint32_t phase = 0, acc = 0;
      bool ok = true;
      for (int t = unit; ok && t < total; t += units, ++acc) {
        const uint32_t b = acc & 1u;
        ok = wait_bounded(tempty_bar(b), ((acc >> 1) & 1u) ^ 1u, tmo, abort_flag, kSiteMmaTmemEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + b * kAccCols;
        for (int k = 0; k < num_k; ++k) {
          ok = wait_bounded(full_bar(stage), phase, tmo, abort_flag, kSiteMmaFull);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t ad = operand_desc<kBK>(a_tile(stage), kk, P.a_mn);
            const uint64_t bd = operand_desc<kBK>(b_tile(stage), kk, P.b_mn);
            const uint32_t add = (k != 0 || kk != 0) ? 1u : 0u;
            if constexpr (kPair) umma_bf16_pair(d_tmem, ad, bd, P.idesc, add);
            else umma_bf16(d_tmem, ad, bd, P.idesc, add);
          }
          if constexpr (kPair) umma_commit_pair_mc(empty_bar(stage), 0x3);
          else umma_commit(empty_bar(stage));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (kPair) umma_commit_pair_mc(tfull_bar(b), 0x3);
        else umma_commit(tfull_bar(b));
      }
      // Every MMA of this thread is done before TMEM is released.
      if constexpr (kPair) umma_commit_pair(mma_done_bar);
      else umma_commit(mma_done_bar);
      wait_bounded(mma_done_bar, 0, tmo, abort_flag, kSiteDrainMma, false);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;         // the TMEM lane quarter this warp may access
    const int set = (warp - 2) >> 2;  // which columns of the tile
    typename Epi::State st = Epi::begin(P.epi);
    uint32_t acc = 0;
    bool ok = true;
    for (int t = unit; ok && t < total; t += units, ++acc) {
      int mb, nb;
      fused_tile(t, P.group_m, tiles_m, P.tiles_n, mb, nb);
      const uint32_t b = acc & 1u;
      EpiTile tile;
      tile.t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * kAccCols + set * L::kWarpCols;
      tile.row = mb * kTileM + static_cast<int>(rank) * 128 + q * 32 + lane;
      tile.col = nb * BN + set * L::kWarpCols;
      tile.M = M;
      tile.N = P.N;
      tile.has = num_k > 0;
      auto ready = [&]() -> bool {
        if (!tile.has) return true;
        int got = 1;
        if (lane == 0)
          got = wait_bounded(tfull_bar(b), (acc >> 1) & 1u, tmo, abort_flag, kSiteEpiTmemFull);
        got = __shfl_sync(0xFFFFFFFFu, got, 0);
        tc_fence_after();
        return got != 0;
      };
      ok = Epi::template run<L::kWarpCols>(P.epi, st, tile, ready);
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (tile.has && lane == 0) {
        if (leader) mbar_arrive(tempty_bar(b));
        else mbar_arrive_cluster(mapa_shared(tempty_bar(b), 0));
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, kTmemCols);
    else tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Shared-memory limit and launch of one instantiation.
template <class Epi, int BN, int STAGES, bool kPair>
struct Fused {
  using L = FusedLayout<BN, STAGES, kPair>;
  static cudaError_t init() {
    return cudaFuncSetAttribute(fused_gemm_kernel<Epi, BN, STAGES, kPair>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  }
  static cudaError_t launch(const FusedParams<typename Epi::Args>& p, int units, bool pdl,
                            cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * units : units), 1, 1);
    cfg.blockDim = dim3(L::kThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
      attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (kPair) {
      attr[n].id = cudaLaunchAttributeClusterDimension;
      attr[n].val.clusterDim.x = 2;
      attr[n].val.clusterDim.y = 1;
      attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
    return cudaLaunchKernelEx(&cfg, fused_gemm_kernel<Epi, BN, STAGES, kPair>, p);
  }
};

constexpr int kFusedPairStages = 6, kFused128Stages = 6, kFused64Stages = 8;

template <class Epi>
cudaError_t fused_init_all() {
  cudaError_t e = Fused<Epi, 256, kFusedPairStages, true>::init();
  if (e == cudaSuccess) e = Fused<Epi, 128, kFused128Stages, false>::init();
  if (e == cudaSuccess) e = Fused<Epi, 64, kFused64Stages, false>::init();
  return e;
}

template <class Epi>
cudaError_t fused_launch_config(int config, const FusedParams<typename Epi::Args>& p, int units, bool pdl,
                                cudaStream_t s) {
  switch (config) {
    case 0: return Fused<Epi, 256, kFusedPairStages, true>::launch(p, units, pdl, s);
    case 1: return Fused<Epi, 128, kFused128Stages, false>::launch(p, units, pdl, s);
    case 2: return Fused<Epi, 64, kFused64Stages, false>::launch(p, units, pdl, s);
    default: return cudaErrorInvalidValue;
  }
}

// Reads, and clears if set, this translation unit's own device error word
// (hence static: one copy for each unit).
static cudaError_t fused_read_status(unsigned long long* word, cudaStream_t stream) {
  *word = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_status_word, sizeof(*word), 0,
                                            cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || *word == 0) return e;
  const unsigned long long zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_word, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace axonn
