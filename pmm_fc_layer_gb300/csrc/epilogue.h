// Host interface of the fused-epilogue products (kernels_epi.cu), the
// elementwise kernels beside them (elementwise.cu) and the linear cross
// entropy (linear_ce.cu).  The C entry points that check the arguments are
// in axonn_fc.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace axonn {

enum Activation : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// D(x): an element is dropped where its 16 random bits are below thr, else
// scaled.  thr = 0 is no dropout (rng is not read).
struct DropoutArgs {
  const uint64_t* rng;  // device: seed, offset
  uint32_t thr;         // floor(65536 p + 1/2), 0 .. 65536
  uint32_t above;       // thr 2^16 - 1
  float scale;          // 65536 / (65536 - thr), 0 where thr = 65536
};

// Epilogue of Y = R + D(act(acc + b)), Z = acc + b, and of
// dZ = act'(Z) D(acc) + R with its column sums.
struct EpilogueArgs {
  const void* bias;      // [N] or null
  int32_t pre_out;       // forward: Z is written
  const uint16_t* pre_in;  // backward: Z
  int64_t ld_pre;
  const void* residual;  // of the output's type, or null
  int64_t ld_res;
  float* colsum;         // backward: [ceil(M / 32) x ld_colsum] partial sums, or null
  int64_t ld_colsum;
  DropoutArgs drop;
  int32_t act;
  int32_t out_f32, bias_f32;
};

// Epilogues of the linear cross entropy's products.  Rows are the counted
// rows, packed; columns are [col0, col0 + N) of the vocabulary.
struct CeArgs {
  const int32_t* labels;  // [T], packed
  int64_t rows;           // rows there is room for (T)
  int64_t col0;
  float2* stats;          // [vocabulary groups x ld_stats] (max, sum of exp) of each row and group
  int64_t ld_stats;
  float* label_logit;     // [T]
  int32_t keep_piece;     // the piece [T x N] is written: distances (16 bits), or probabilities (bf16)
  const float* lse2;      // [T] logsumexp in base 2 (the recomputing product)
};

// Output of a product times a number on the device (null: 1): bf16, fp32, or
// added into fp32.
struct StoreArgs {
  const float* scale;
  int32_t mode;  // OutMode: kOutBF16, kOutF32, kOutF32Accum
};

// A matrix that an epilogue writes: by TMA through the map, or element by
// element.
struct OutMatrix {
  CUtensorMap map;
  void* base;
  int64_t ld;
};

// One product with a fused epilogue: C[M x N] = A . B with the operand
// majors of the tensor maps.
template <class Args>
struct FusedParams {
  CUtensorMap ta, tb;
  OutMatrix out;   // the output (the piece, for the linear cross entropy)
  OutMatrix out2;  // the forward's pre-activation
  Args epi;
  // A count on the device that takes the place of M (count_of = 1) or of the
  // reduction's length (2; rows of both operands from the count to the next
  // multiple of 64 are then zero), read when the product starts.
  const int32_t* count;
  int32_t count_of;
  // The reduction in `splits` consecutive ranges, each a product of its own:
  // range s writes the rows from s * split_rows on.
  int32_t splits, split_rows;
  const int2* parts;  // not null: {splits, split_rows} on the device instead
  int32_t M, N, num_k;
  int32_t tiles_m, tiles_n;
  uint32_t idesc;
  int32_t a_mn, b_mn, a_3d, b_3d;
  uint32_t load_bytes;  // of one stage (of both CTAs of a pair)
  int32_t group_m;
  int32_t l2_keep;
  float l2_keep_frac;
  int32_t inject;
  uint64_t timeout_ns;
};

// Tiles of the fused products: 0 a CTA pair's 256 x 256, 1 128 x 128,
// 2 128 x 64, 3 a CTA pair's 512 x 256.
struct FusedConfig {
  int bm, bn;
  bool pair;
  int mma_m;
};
constexpr int kEpilogueCols = 64;  // columns of one epilogue warp: the groups of CeArgs::stats
constexpr int kFusedConfigs = 4;
constexpr FusedConfig kFusedConfig[kFusedConfigs] = {
    {256, 256, true, 256}, {128, 128, false, 128}, {128, 64, false, 128}, {512, 256, true, 256}};

enum FusedKind : int { kFusedFwd = 0, kFusedBwd = 1 };
enum CeKind : int { kCeStats = 0, kCeProb = 1 };

// Shared-memory limits on the current device; *regs_ok = false if a kernel
// was not built with the registers that its split assumes.
cudaError_t fused_init(bool* regs_ok);
cudaError_t fused_launch(FusedKind kind, int config, const FusedParams<EpilogueArgs>& p, int units,
                         bool pdl, cudaStream_t stream);
// How many such clusters the GPU holds at once.
cudaError_t fused_clusters_resident(int sms, int pieces, int* clusters);
// One 128 x 128 tile for every cluster of `pieces` CTAs, the reduction cut
// over them (p as filled for configuration 1).
cudaError_t fused_cluster(FusedKind kind, const FusedParams<EpilogueArgs>& p, int tiles, int pieces, bool pdl,
                          cudaStream_t stream);
cudaError_t fused_take_status(unsigned long long* word, cudaStream_t stream);

cudaError_t ce_init(bool* regs_ok);
cudaError_t ce_launch(CeKind kind, int config, const FusedParams<CeArgs>& p, int units, bool pdl,
                      cudaStream_t stream);
cudaError_t store_launch(int config, const FusedParams<StoreArgs>& p, int units, bool pdl,
                         cudaStream_t stream);
cudaError_t ce_take_status(unsigned long long* word, cudaStream_t stream);

}  // namespace axonn
