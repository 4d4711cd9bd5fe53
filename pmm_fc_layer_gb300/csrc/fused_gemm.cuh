// bf16 product on the sm_103a tensor cores with an epilogue of the caller's
// choice: C[M x N] = A[M x R] . B[R x N] in fp32 TMEM accumulators, each
// handed to Epi while the next tile's products run.
//
// Persistent and warp-specialised like the plain products: warp 0 loads
// operand stages by TMA, warp 1 issues the MMAs, the others are the
// epilogue.  What differs is the balance.  A fused epilogue costs several
// times a plain store (an activation, a generator call for every eight
// elements, one or two operands to read), so it has to run beside the
// mainloop, in one of two ways:
//  - kHalves = 1 (tiles of 128 rows a CTA): the accumulator is
//    double-buffered in TMEM (2 x BN columns), and the epilogue (a warp for
//    every 32 rows x 64 columns) has a whole tile's mainloop to finish in.
//  - kHalves = 2 (a CTA pair's 512 x 256 tile): two accumulators of 128 rows
//    a CTA, which share each B slice (a quarter fewer operand bytes a
//    multiply-add than 256 x 256, and under the power cap 10 to 20 % faster)
//    and fill TMEM.  Sixteen epilogue warps take one half at a time: they
//    move it into registers whole (64 columns a thread), release it, and
//    then work on it.  The MMAs are issued with the halves out of step by
//    kSkew stages: at a tile's end half 0 runs ahead and is done first, at
//    the next one's start it begins first, and the epilogue's work on half 0
//    fits between the two.  Tiles of a last round that fills at most half of
//    the units go to twice as many of them, a half each.
// kPair: a CTA pair shares one tile (cta_group::2), each CTA loading its own
// rows of A and its half of B.
// Waits are bounded, and an expired one is recorded and reported, as in the
// plain products.
//
// Measured (8192 x 6144 x 24576, 512 x 256 tiles): GELU with Z kept 1545 us,
// 1601 TFLOP/s, the tensor pipe busy 86 % of the cycles; under the power cap
// the clock falls as the pipe fills, so the rest is not all idle time.  Short
// reductions are bound by the epilogue's instructions and stores: 8192 x 64 x
// 8192 takes 42 us (3.2 TB/s) plain, 56 with GELU, 94 with dropout and a
// residual, of which the stores are 11, 9 and 5 (256 x 256 tiles).
#pragma once
#include "epilogue.h"
#include "epilogue_math.cuh"
#include "gemm_kernel.cuh"

namespace axonn {

template <int BN, int STAGES, bool kPair, int kHalves>
struct FusedLayout {
  static constexpr int kAHalfBytes = 128 * kBK * 2;
  static constexpr int kABytes = kHalves * kAHalfBytes;
  static constexpr int kBCols = kPair ? BN / 2 : BN;  // columns of B one CTA loads
  static constexpr int kBBytes = kBCols * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kNumBars = 2 * STAGES + 5;
  static constexpr int kSlotBytes = 2048;  // an epilogue warp's staging slot: 32 rows of 64 bytes
  static constexpr int kEpiSets = BN / 64;  // warps per 32 rows, 64 columns each
  static constexpr int kEpi = 4 * kEpiSets;
  static constexpr int kEpiFirst = kHalves == 2 ? 4 : 2;
  static constexpr int kThreads = 32 * (kEpiFirst + kEpi);
  static constexpr int kWarpCols = 64;
  // 1024 B of slack to align the ring, the ring, the staging slots, barriers,
  // TMEM slot, abort flag
  static constexpr int kBytes = 1024 + STAGES * kStageBytes + kEpi * kSlotBytes + kNumBars * 8 + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Registers of a thread of the 20-warp kernels: warpgroup 0 (producer, MMA
// issuer) gives up what the four epilogue warpgroups, which hold 64
// accumulator words a thread, take.  The shares add up to the launch's
// allocation; the host checks that the kernels were built with it.
constexpr int kFusedRegsAtLaunch = 96;
constexpr int kFusedRegsControl = 32;
constexpr int kFusedRegsEpilogue = 112;
static_assert(128 * kFusedRegsControl + 512 * kFusedRegsEpilogue <= 640 * kFusedRegsAtLaunch,
              "register split exceeds the launch allocation");

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
  int rows;                          // rows that stores write: M, unless an epilogue pads
  int row_off;                       // where row 0 of the output lies (a split reduction's range)
  uint32_t slot;                     // shared memory, kSlotBytes
  const OutMatrix* out;
  const OutMatrix* out2;
  bool has;  // false: the reduction is empty and the accumulator is zero
};

__device__ __forceinline__ void load_acc32(const EpiTile& t, int c, float (&x)[32]) {
  uint32_t r[32];
  if (t.has) {
    __syncwarp();  // the whole warp loads: lanes past the last row come back from skipped work
    tmem_ld_32x32b_x32(t.t_row + c * 32, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
  }
}

// The slot's layout: row r's 16-byte chunk c at c ^ (r / 2 % 4) of its 64
// bytes, the 64-byte swizzle of TMA.  A warp's row-wise accesses (a lane its
// own row) and its chunk-wise ones (four lanes a row) both spread over the
// banks.
__device__ __forceinline__ uint32_t slot_at(const EpiTile& t, int row, int chunk) {
  return t.slot + static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) * 16));
}

// 64 bytes of each of the warp's 32 rows of a matrix that the epilogue reads,
// at column `col`.  Four lanes read a row's 64 bytes (a load touches 8 lines;
// a lane reading its own row would touch 32, at 16 bytes a cycle), and the
// slot hands every lane its own row: start() asks for the words, finish()
// exchanges them.  Nothing past row M or column N is read (zeros there).
template <typename T>
struct RowSegment {
  uint4 v[4];
  __device__ __forceinline__ void start(const EpiTile& t, const void* base, int64_t ld, int col) {
    constexpr int kPer16 = 16 / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31;
    const int row0 = t.row - lane, c = col + (lane & 3) * kPer16;
    const T* p = static_cast<const T*>(base) + static_cast<int64_t>(row0 + (lane >> 2)) * ld + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (row0 + 8 * i + (lane >> 2) < t.M && c < t.N) {
        const T* q = p + 8 * i * ld;
        if (c + kPer16 <= t.N) {
          v[i] = *reinterpret_cast<const uint4*>(q);
        } else {  // the row's last, partial 16 bytes
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < kPer16; ++j)
            if (c + j < t.N) {
              if constexpr (sizeof(T) == 4) w[j] = q[j];
              else w[j >> 1] |= static_cast<uint32_t>(q[j]) << (16 * (j & 1));
            }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  // This lane's row: 16 words.
  __device__ __forceinline__ void finish(const EpiTile& t, uint32_t (&w)[16]) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last store has read it
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      st_shared_v4(slot_at(t, 8 * i + (lane >> 2), lane & 3), v[i].x, v[i].y, v[i].z, v[i].w);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 f = ld_shared_v4(slot_at(t, lane, c));
      w[4 * c] = __float_as_uint(f.x);
      w[4 * c + 1] = __float_as_uint(f.y);
      w[4 * c + 2] = __float_as_uint(f.z);
      w[4 * c + 3] = __float_as_uint(f.w);
    }
    __syncwarp();
  }
};

// Writes 64 bytes of each of the warp's 32 rows (16 words a lane, its own
// row's) at column `col` of a matrix: through the warp's staging slot and one
// TMA store.  Row-wise stores from registers, 32 bytes a lane, moved about 18
// bytes a cycle and SM and held up the next tile's MMAs behind the registers
// they came from.  Rows past t.rows and columns past t.N are not written;
// where a row's last 16 bytes are only partly the matrix' own (a TMA store
// writes them whole), that segment goes element by element.
template <typename T>
__device__ __forceinline__ void store_segment(const EpiTile& t, const OutMatrix* m, int col, const uint32_t (&w)[16]) {
  constexpr int kPer16 = 16 / static_cast<int>(sizeof(T)), kCols = 64 / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  if (col + kCols > t.N && t.N % kPer16 != 0) {
    if (t.row < t.rows) {
      T* p = static_cast<T*>(m->base) + static_cast<int64_t>(t.row + t.row_off) * m->ld + col;
      const int n = t.N - col;
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (j < n) p[j] = static_cast<T>(sizeof(T) == 4 ? w[j % 16] : w[(j >> 1) % 16] >> (16 * (j & 1)));
    }
    return;
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the slot has been read
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(slot_at(t, lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0 && t.row < t.rows) {  // lane 0 has the first row
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(&m->map)),
                 "r"(t.slot), "r"(col), "r"(t.row + t.row_off)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// 32 columns of the warp's rows, in bf16 (one rounding) or fp32.
__device__ __forceinline__ void store_bf16(const EpiTile& t, const OutMatrix* m, int col, const float (&x)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
  store_segment<uint16_t>(t, m, col, w);
}
__device__ __forceinline__ void store_f32(const EpiTile& t, const OutMatrix* m, int col, const float (&x)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (col + 16 * h >= t.N) break;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(x[16 * h + j]);
    store_segment<uint32_t>(t, m, col + 16 * h, w);
  }
}

// The 32-column steps of a tile part, for an epilogue given as
//   void prefetch(args, tile, cols)        asks for what it will read into L2
//   void step(args, state, tile, c, x)     works on columns 32 c .. of the part
//   kEachStages                            see wait_warp
// The operands are asked for before the accumulator is ready.  kHold: the
// whole part goes to registers and TMEM is released before any of the work.
template <class Epi, int kCols, bool kHold, class Ready, class Release>
__device__ __forceinline__ bool epilogue_steps(const typename Epi::Args& a, const typename Epi::State& st,
                                               const EpiTile& t, Ready&& ready, Release&& release) {
  if (t.col < t.N && t.row < t.M) Epi::prefetch(a, t, min(kCols, t.N - t.col));
  if (!ready()) return false;
  if constexpr (kHold) {
    float x[kCols / 32][32];
#pragma unroll
    for (int c = 0; c < kCols / 32; ++c)
      if (t.col + 32 * c < t.N) load_acc32(t, c, x[c]);
    release();
#pragma unroll
    for (int c = 0; c < kCols / 32; ++c)
      if (t.col + 32 * c < t.N) Epi::step(a, st, t, c, x[c]);
  } else {
#pragma unroll 1
    for (int c = 0; c < kCols / 32; ++c) {
      if (t.col + 32 * c >= t.N) break;
      float x[32];
      load_acc32(t, c, x);
      Epi::step(a, st, t, c, x);
    }
    release();
  }
  return true;
}

// Barrier of the epilogue's threads that ORs a predicate over them.
template <int kThreads>
__device__ __forceinline__ bool epilogue_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "n"(kThreads)
      : "memory");
  return r != 0;
}

// Bounded wait of a whole warp that polls without suspending it (see
// wait_polling), for reductions of up to Epi::kEachStages stages: 8192 x 64 x
// 8192 takes 15 % less than with one polling warp and a barrier behind it,
// with a light epilogue (stores, an activation) 8192 x 768 x 8192 as long, with
// dropout and a residual still 7 % less, and 8192 x 3000 x 8192 4 to 8 % more:
// its polls' issue slots and power.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                          volatile int* abort_flag, uint32_t site) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) return true;
    bool over = *abort_flag != 0;
    if (!over && global_timer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      if ((threadIdx.x & 31) == 0) record_timeout(site);
      over = true;
    }
    if (__any_sync(0xFFFFFFFFu, over)) return false;
  }
}

template <class Epi, int BN, int STAGES, bool kPair, int kHalves>
__global__ void __launch_bounds__(FusedLayout<BN, STAGES, kPair, kHalves>::kThreads, 1)
    fused_gemm_kernel(const __grid_constant__ FusedParams<typename Epi::Args> P) {
  using L = FusedLayout<BN, STAGES, kPair, kHalves>;
  constexpr uint32_t kAccCols = BN < 128 ? 128 : BN;  // TMEM columns of one accumulator
  constexpr uint32_t kTmemCols = 2 * kAccCols;
  constexpr int kCtaM = 128 * kHalves;
  constexpr int kTileM = kPair ? 2 * kCtaM : kCtaM;
  // Stages by which half 0 runs ahead at a tile's two ends: all the ring
  // holds.
  constexpr int kSkew = STAGES;
  static_assert(kTmemCols == 256 || kTmemCols == 512, "TMEM columns");
  static_assert(kHalves == 1 || kPair, "two halves: a CTA pair's tile");

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - raw);
  const uint32_t slots = ring + STAGES * L::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_ptr + STAGES * L::kStageBytes + L::kEpi * L::kSlotBytes);
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
  int M = P.M, tiles_m = P.tiles_m, all_k = P.num_k;
  if (P.count_of != 0) {
    const int n = *P.count;
    if (P.count_of == 1) {
      M = n;
      tiles_m = (n + kTileM - 1) / kTileM;
    } else {
      all_k = (n + kBK - 1) / kBK;
    }
  }
  int splits = P.splits, split_rows = P.split_rows;
  if (P.parts) {
    const int2 parts = *P.parts;
    splits = parts.x;
    split_rows = parts.y;
  }
  const int per_split = tiles_m * P.tiles_n;
  const int total = per_split * splits;
  // A unit's items: the tiles unit, unit + units, ...; where the last round
  // would leave half the units idle, its tiles' halves are items instead.
  const int over = total % units;
  const int whole = kHalves == 2 && 2 * over <= units ? total - over : total;
  const int items = whole + 2 * (total - whole);
  auto split_of = [&](int t) { return splits == 1 ? 0 : t / per_split; };
  auto item_tile = [&](int i, int& half) {  // half: -1 for all of the tile
    half = i < whole ? -1 : (i - whole) & 1;
    return i < whole ? i : whole + (i - whole) / 2;
  };
  // Range s of the reduction: stages [all_k s / splits, all_k (s + 1) / splits).
  auto range = [&](int split, int& k0) {
    if (splits == 1) {
      k0 = 0;
      return all_k;
    }
    k0 = static_cast<int>(static_cast<int64_t>(all_k) * split / splits);
    return static_cast<int>(static_cast<int64_t>(all_k) * (split + 1) / splits) - k0;
  };

  if constexpr (kHalves == 2) {
    if (warp < L::kEpiFirst) setmaxnreg_dec<kFusedRegsControl>();
  }
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && P.inject != 1) {
      int stage = 0;
      uint32_t phase = 0, loads = 0;
      bool ok = true;
      const uint64_t pol_a = l2_policy(P.l2_keep == 1, P.l2_keep_frac);
      const uint64_t pol_b = l2_policy(P.l2_keep == 2, P.l2_keep_frac);
      for (int i = unit; ok && i < items; i += units) {
        int mb, nb, k_first, only;
        const int t = item_tile(i, only);
        const int split = split_of(t);
        const int num_k = range(split, k_first);
        fused_tile(t - split * per_split, P.group_m, tiles_m, P.tiles_n, mb, nb);
        const uint32_t bytes = P.load_bytes - (only >= 0 ? (kPair ? 2 : 1) * L::kAHalfBytes : 0);
        const int m0 = mb * kTileM + static_cast<int>(rank) * kCtaM;
        const int n0 = nb * BN + static_cast<int>(rank) * L::kBCols;
        for (int k = 0; k < num_k; ++k) {
          ok = wait_bounded(empty_bar(stage), phase ^ 1u, tmo, abort_flag, kSiteProducerEmpty);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes);
          const int r0 = (k_first + k) * kBK;
          if constexpr (kPair) {
            const uint32_t fb = mapa_shared(full_bar(stage), 0);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              const uint32_t at = a_tile(stage) + h * L::kAHalfBytes;
              if (kHalves == 1 || only < 0 || only == h) {
                if (P.a_3d) {
                  tma_load_3d_pair(at, &P.ta, fb, 0, r0, (m0 + 128 * h) / 64, pol_a);
                } else if (P.a_mn) {
                  tma_load_2d_pair(at, &P.ta, fb, m0 + 128 * h, r0, pol_a);
                  tma_load_2d_pair(at + kBK * 128, &P.ta, fb, m0 + 128 * h + 64, r0, pol_a);
                } else {
                  tma_load_2d_pair(at, &P.ta, fb, r0, m0 + 128 * h, pol_a);
                }
              }
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
    if (lane == 0 && leader && all_k > 0) {
      uint32_t acc = 0;
      bool ok = true;
      // The MMAs of one stage into one accumulator.
      auto multiply = [&](int stage, int half, uint32_t d_tmem, bool first) {
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
          const uint64_t ad = operand_desc<kBK>(a_tile(stage) + half * L::kAHalfBytes, kk, P.a_mn);
          const uint64_t bd = operand_desc<kBK>(b_tile(stage), kk, P.b_mn);
          const uint32_t add = (!first || kk != 0) ? 1u : 0u;
          if constexpr (kPair) umma_bf16_pair(d_tmem, ad, bd, P.idesc, add);
          else umma_bf16(d_tmem, ad, bd, P.idesc, add);
        }
      };
      auto commit = [&](uint32_t bar) {
        if constexpr (kPair) umma_commit_pair_mc(bar, 0x3);
        else umma_commit(bar);
      };
      if constexpr (kHalves == 1) {
        int stage = 0;
        uint32_t phase = 0;
        for (int t = unit; ok && t < items; t += units) {
          int k_first;
          const int num_k = range(split_of(t), k_first);
          if (num_k == 0) continue;  // as the epilogue counts
          const uint32_t b = acc & 1u;
          ok = wait_bounded(tempty_bar(b), ((acc >> 1) & 1u) ^ 1u, tmo, abort_flag, kSiteMmaTmemEmpty);
          if (!ok) break;
          tc_fence_after();
          for (int k = 0; k < num_k; ++k) {
            ok = wait_bounded(full_bar(stage), phase, tmo, abort_flag, kSiteMmaFull);
            if (!ok) break;
            tc_fence_after();
            multiply(stage, 0, tmem_base + b * kAccCols, k == 0);
            commit(empty_bar(stage));
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          commit(tfull_bar(b));
          ++acc;
        }
      } else {
        // Half 0 runs stages [0, a), then both halves alternate, then half 0
        // runs [e, num_k); half 1 follows at either end.  No stage is held
        // over more than the ring: kSkew <= STAGES.
        uint32_t base = 0;  // stages consumed before this tile
        auto run = [&](int half, int k0, int k1, bool wait_full, bool free_stage) -> bool {
          for (int k = k0; k < k1; ++k) {
            const uint32_t i = base + k;
            const int stage = static_cast<int>(i % STAGES);
            if (wait_full) {
              if (!wait_bounded(full_bar(stage), (i / STAGES) & 1u, tmo, abort_flag, kSiteMmaFull)) return false;
              tc_fence_after();
            }
            multiply(stage, half, tmem_base + half * kAccCols, k == 0);
            if (free_stage) commit(empty_bar(stage));
          }
          return true;
        };
        uint32_t uses[2] = {0, 0};  // of each half's accumulator
        for (int i = unit; ok && i < items; i += units) {
          int k_first, only;
          const int num_k = range(split_of(item_tile(i, only)), k_first);
          if (num_k == 0) continue;  // as the epilogue counts
          if (only >= 0) {
            ok = wait_bounded(tempty_bar(only), (uses[only] & 1u) ^ 1u, tmo, abort_flag, kSiteMmaTmemEmpty);
            if (!ok) break;
            tc_fence_after();
            ok = run(only, 0, num_k, true, true);
            if (!ok) break;
            commit(tfull_bar(only));
            ++uses[only];
            base += static_cast<uint32_t>(num_k);
            continue;
          }
          const int a = min(kSkew, num_k), e = max(a, num_k - kSkew);
          ok = wait_bounded(tempty_bar(0), (uses[0] & 1u) ^ 1u, tmo, abort_flag, kSiteMmaTmemEmpty);
          if (!ok) break;
          tc_fence_after();
          ok = run(0, 0, a, true, false);
          if (!ok) break;
          if (a == num_k) commit(tfull_bar(0));
          ok = wait_bounded(tempty_bar(1), (uses[1] & 1u) ^ 1u, tmo, abort_flag, kSiteMmaTmemEmpty);
          if (!ok) break;
          tc_fence_after();
          ok = run(1, 0, a, false, true);
          // in step: both halves take a B slice one after the other
          for (int k = a; ok && k < e; ++k) {
            const uint32_t i = base + k;
            const int stage = static_cast<int>(i % STAGES);
            ok = wait_bounded(full_bar(stage), (i / STAGES) & 1u, tmo, abort_flag, kSiteMmaFull);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
              const uint64_t bd = operand_desc<kBK>(b_tile(stage), kk, P.b_mn);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                umma_bf16_pair(tmem_base + h * kAccCols,
                               operand_desc<kBK>(a_tile(stage) + h * L::kAHalfBytes, kk, P.a_mn), bd, P.idesc,
                               (k != 0 || kk != 0) ? 1u : 0u);
            }
            commit(empty_bar(stage));
          }
          ok = ok && run(0, e, num_k, true, false);
          if (!ok) break;
          if (a < num_k) commit(tfull_bar(0));
          run(1, e, num_k, false, true);
          commit(tfull_bar(1));
          base += static_cast<uint32_t>(num_k);
          ++uses[0];
          ++uses[1];
        }
      }
      // Every MMA of this thread is done before TMEM is released.
      if constexpr (kPair) umma_commit_pair(mma_done_bar);
      else umma_commit(mma_done_bar);
      wait_bounded(mma_done_bar, 0, tmo, abort_flag, kSiteDrainMma, false);
    }
  } else if (warp >= L::kEpiFirst) {
    if constexpr (kHalves == 2) setmaxnreg_inc<kFusedRegsEpilogue>();
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // the TMEM lane quarter this warp may access
    const int set = (warp - L::kEpiFirst) >> 2;  // which columns of the tile
    // Short reductions leave the epilogue no time to wait: its warps then go
    // each at its own pace.
    const bool each = all_k <= Epi::kEachStages * splits;
    typename Epi::State st = Epi::begin(P.epi);
    uint32_t uses[2] = {0, 0};  // tiles (one half: uses[0] alone), or of each half's accumulator
    bool ok = true;
    for (int i = unit; ok && i < items; i += units) {
      int mb, nb, k_first, only;
      const int t = item_tile(i, only);
      const int split = split_of(t);
      const bool has = range(split, k_first) > 0;
      fused_tile(t - split * per_split, P.group_m, tiles_m, P.tiles_n, mb, nb);
#pragma unroll 1
      for (int half = 0; ok && half < kHalves; ++half) {
        if (kHalves == 2 && only >= 0 && only != half) continue;
        // buffers alternate by tile (one half), or belong to the halves
        const uint32_t b = kHalves == 1 ? uses[0] & 1u : static_cast<uint32_t>(half);
        const uint32_t parity = kHalves == 1 ? (uses[0] >> 1) & 1u : uses[half] & 1u;
        EpiTile tile;
        tile.t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * kAccCols + set * L::kWarpCols;
        tile.row = mb * kTileM + static_cast<int>(rank) * kCtaM + half * 128 + q * 32 + lane;
        tile.col = nb * BN + set * L::kWarpCols;
        tile.M = tile.rows = M;
        tile.N = P.N;
        tile.slot = slots + static_cast<uint32_t>((warp - L::kEpiFirst) * L::kSlotBytes);
        tile.out = &P.out;
        tile.out2 = &P.out2;
        tile.row_off = split * split_rows;
        tile.has = has;
        auto ready = [&]() -> bool {
          if (!tile.has) return true;
          bool late = false;
          if (each) {
            late = !wait_warp(tfull_bar(b), parity, tmo, abort_flag, kSiteEpiTmemFull);
            tc_fence_after();
            return !late;
          }
          // One warp polls; the others sleep in a hardware barrier, which
          // also tells them how it ended.
          if (warp == L::kEpiFirst) {
            if (lane == 0) late = !wait_bounded(tfull_bar(b), parity, tmo, abort_flag, kSiteEpiTmemFull);
            late = __shfl_sync(0xFFFFFFFFu, late, 0);
          }
          late = epilogue_any<32 * L::kEpi>(late);
          tc_fence_after();
          return !late;
        };
        auto release = [&]() {  // once, when this warp has read its part
          tc_fence_before();
          __syncwarp();
          if (tile.has && lane == 0) {
            if (leader) mbar_arrive(tempty_bar(b));
            else mbar_arrive_cluster(mapa_shared(tempty_bar(b), 0));
          }
        };
        ok = Epi::template run<L::kWarpCols, kHalves == 2>(P.epi, st, tile, ready, release);
        if (has) ++uses[kHalves == 1 ? 0 : half];
      }
    }
    // this warp's stores are complete before the CTA may exit
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// Products of few tiles over a long reduction (a layer answering some tens of
// tokens): a cluster of S CTAs takes one 128 x 128 tile, each CTA a range of
// the reduction.  When its range is done, a CTA leaves its fp32 accumulator
// in the shared memory that held its operands.  The tile's sixteen blocks of
// 32 x 32 are then dealt out to the cluster's warps; a warp adds up the S
// parts of its block in the order of the ranges and runs the epilogue on it.
// One tile a cluster, nothing persistent: it is launched where all CTAs fit
// the GPU at once.  What bounds it is the operands' way into each SM: 64 x
// 24576 x 6144 (302 MB of weights) takes 65 us, 4.6 TB/s, where the best whole
// tile takes 121; 16 x 6144 x 6144 20.5 and 33.5, 512 x 8192 x 512 22.6 and 43.
constexpr int kClusterStages = 6;
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <class Epi>
__global__ void __launch_bounds__(FusedLayout<128, kClusterStages, false, 1>::kThreads, 1)
    fused_cluster_kernel(const __grid_constant__ FusedParams<typename Epi::Args> P) {
  using L = FusedLayout<128, kClusterStages, false, 1>;
  constexpr int STAGES = kClusterStages;
  static_assert(16 * 4096 <= STAGES * L::kStageBytes, "the accumulator fits the ring");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - raw);
  const uint32_t slots = ring + STAGES * L::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_ptr + STAGES * L::kStageBytes + L::kEpi * L::kSlotBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full_bar = [&](int s) { return smem_addr(bars + s); };
  auto empty_bar = [&](int s) { return smem_addr(bars + STAGES + s); };
  const uint32_t tfull_bar = smem_addr(bars + 2 * STAGES);
  auto a_tile = [&](int s) { return ring + s * L::kStageBytes; };
  auto b_tile = [&](int s) { return ring + s * L::kStageBytes + L::kABytes; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0 && P.num_k > 0) {
    prefetch_tmap(&P.ta);
    prefetch_tmap(&P.tb);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t tmo = P.timeout_ns;
  int mb, nb;
  fused_tile(static_cast<int>(cluster_id_x()), P.group_m, P.tiles_m, P.tiles_n, mb, nb);
  const int m0 = mb * 128, n0 = nb * 128;
  const int k0 = static_cast<int>(static_cast<int64_t>(P.num_k) * rank / S);
  const int k1 = static_cast<int>(static_cast<int64_t>(P.num_k) * (rank + 1) / S);
  griddep_wait();

  bool late = false;
  if (warp == 0) {
    if (lane == 0 && P.inject != 1) {
      const uint64_t pol = l2_policy(false, 1.0f);
      int loads = 0;
      for (int k = k0; k < k1; ++k, ++loads) {
        const int stage = loads % STAGES;
        if (!wait_bounded(empty_bar(stage), ((loads / STAGES) & 1) ^ 1u, tmo, abort_flag, kSiteProducerEmpty)) break;
        mbar_arrive_expect_tx(full_bar(stage), P.load_bytes);
        const uint32_t fb = full_bar(stage);
        const int r0 = k * kBK;
        if (P.a_3d) {
          tma_load_3d(a_tile(stage), &P.ta, fb, 0, r0, m0 / 64, pol);
        } else if (P.a_mn) {
          tma_load_2d(a_tile(stage), &P.ta, fb, m0, r0, pol);
          tma_load_2d(a_tile(stage) + kBK * 128, &P.ta, fb, m0 + 64, r0, pol);
        } else {
          tma_load_2d(a_tile(stage), &P.ta, fb, r0, m0, pol);
        }
        if (P.b_3d) {
          tma_load_3d(b_tile(stage), &P.tb, fb, 0, r0, n0 / 64, pol);
        } else if (P.b_mn) {
          tma_load_2d(b_tile(stage), &P.tb, fb, n0, r0, pol);
          tma_load_2d(b_tile(stage) + kBK * 128, &P.tb, fb, n0 + 64, r0, pol);
        } else {
          tma_load_2d(b_tile(stage), &P.tb, fb, r0, n0, pol);
        }
      }
      griddep_launch_dependents();
      for (int s = 0; s < STAGES; ++s)  // the last load of each stage has landed
        if (loads > s)
          wait_bounded(full_bar(s), ((loads - s + STAGES - 1) / STAGES - 1) & 1u, tmo, abort_flag, kSiteDrainLoads,
                       false);
    }
  } else if (warp == 1) {
    if (lane == 0 && k1 > k0) {
      bool ok = true;
      for (int k = k0; k < k1; ++k) {
        const int i = k - k0, stage = i % STAGES;
        ok = wait_bounded(full_bar(stage), (i / STAGES) & 1u, tmo, abort_flag, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem_base, operand_desc<kBK>(a_tile(stage), kk, P.a_mn),
                    operand_desc<kBK>(b_tile(stage), kk, P.b_mn), P.idesc, (i != 0 || kk != 0) ? 1u : 0u);
        umma_commit(empty_bar(stage));
      }
      umma_commit(tfull_bar);  // also where a wait expired: what was issued is drained
      wait_bounded(tfull_bar, 0, tmo, abort_flag, kSiteDrainMma, false);
    }
  } else {
    if (k1 > k0) {
      if (warp == 2) {
        if (lane == 0) late = !wait_bounded(tfull_bar, 0, tmo, abort_flag, kSiteEpiTmemFull) || *abort_flag != 0;
        late = __shfl_sync(0xFFFFFFFFu, late, 0);
      }
      late = epilogue_any<32 * L::kEpi>(late);
      tc_fence_after();
    }
    // Block (q, cc) of the tile, 32 rows x 32 columns, at 4096 (4 q + cc): row
    // r's 16-byte chunk c at c ^ (r & 7) of its 128 bytes.
    const int q = warp & 3, set = (warp - 2) >> 2;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      EpiTile t;
      t.t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + set * 64;
      t.has = k1 > k0 && !late;
      float x[32];
      load_acc32(t, c, x);
      const uint32_t row = ring + 4096u * (4 * q + 2 * set + c) + 128u * lane;
#pragma unroll
      for (int v = 0; v < 8; ++v)
        st_shared_v4(row + 16u * (v ^ (lane & 7)), __float_as_uint(x[4 * v]), __float_as_uint(x[4 * v + 1]),
                     __float_as_uint(x[4 * v + 2]), __float_as_uint(x[4 * v + 3]));
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp >= 2 && !late) {
    typename Epi::State st = Epi::begin(P.epi);
#pragma unroll 1
    for (int u = rank + S * (warp - 2); u < 16; u += S * L::kEpi) {
      EpiTile t;
      t.row = m0 + 32 * (u >> 2) + lane;
      t.col = n0 + 32 * (u & 3);
      t.M = t.rows = P.M;
      t.N = P.N;
      t.row_off = 0;
      t.slot = slots + static_cast<uint32_t>((warp - 2) * L::kSlotBytes);
      t.out = &P.out;
      t.out2 = &P.out2;
      t.has = true;
      if (t.col >= t.N || t.row - lane >= t.M) continue;
      float x[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = 0.0f;
#pragma unroll 1
      for (int s = 0; s < S; ++s) {
        const uint32_t row = mapa_shared(ring + 4096u * u + 128u * lane, s);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float4 f = ld_cluster_v4(row + 16u * (v ^ (lane & 7)));
          x[4 * v] += f.x;
          x[4 * v + 1] += f.y;
          x[4 * v + 2] += f.z;
          x[4 * v + 3] += f.w;
        }
      }
      Epi::step(P.epi, st, t, 0, x);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may read its part
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem_base, 128);
  }
}

template <class Epi>
cudaLaunchConfig_t fused_cluster_config(int ctas, int pieces, cudaLaunchAttribute (&attr)[2]) {
  using L = FusedLayout<128, kClusterStages, false, 1>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(L::kThreads, 1, 1);
  cfg.dynamicSmemBytes = L::kBytes;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(pieces);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <class Epi>
cudaError_t fused_cluster_launch(const FusedParams<typename Epi::Args>& p, int tiles, int pieces, bool pdl,
                                 cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = fused_cluster_config<Epi>(tiles * pieces, pieces, attr);
  cfg.stream = s;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fused_cluster_kernel<Epi>, p);
}

// Shared-memory limit and launch of one instantiation.
template <class Epi, int BN, int STAGES, bool kPair, int kHalves>
struct Fused {
  using L = FusedLayout<BN, STAGES, kPair, kHalves>;
  static cudaError_t init() {
    return cudaFuncSetAttribute(fused_gemm_kernel<Epi, BN, STAGES, kPair, kHalves>,
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
    return cudaLaunchKernelEx(&cfg, fused_gemm_kernel<Epi, BN, STAGES, kPair, kHalves>, p);
  }
};

// The configurations of kFusedConfig, in its order.
template <class Epi>
using FusedC0 = Fused<Epi, 256, 6, true, 1>;
template <class Epi>
using FusedC1 = Fused<Epi, 128, 6, false, 1>;
template <class Epi>
using FusedC2 = Fused<Epi, 64, 8, false, 1>;
template <class Epi>
using FusedC3 = Fused<Epi, 256, 4, true, 2>;

// *regs_ok becomes false if a register split would not find its registers.
template <class Epi>
cudaError_t fused_init_all(bool* regs_ok) {
  cudaFuncAttributes attr = {};
  const cudaError_t q =
      cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(fused_gemm_kernel<Epi, 256, 4, true, 2>));
  if (q != cudaSuccess) return q;
  if (attr.numRegs != kFusedRegsAtLaunch) *regs_ok = false;
  for (cudaError_t e : {FusedC0<Epi>::init(), FusedC1<Epi>::init(), FusedC2<Epi>::init(), FusedC3<Epi>::init()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <class Epi>
cudaError_t fused_launch_config(int config, const FusedParams<typename Epi::Args>& p, int units, bool pdl,
                                cudaStream_t s) {
  switch (config) {
    case 0: return FusedC0<Epi>::launch(p, units, pdl, s);
    case 1: return FusedC1<Epi>::launch(p, units, pdl, s);
    case 2: return FusedC2<Epi>::launch(p, units, pdl, s);
    case 3: return FusedC3<Epi>::launch(p, units, pdl, s);
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
