// Host interface of the products of one or two rows (gemv.cu).
#pragma once
#include "epilogue.h"

namespace axonn {

struct GemvArgs {
  const uint16_t* A;  // [M x R], or stored [R x M] with a_mn
  int64_t lda;
  const uint16_t* B;  // stored [R x N] or [N x R]
  int64_t ldb;
  int64_t N, R;
  int32_t M, a_mn;
  int32_t piece;  // reduction elements of one CTA (set by the launch)
  void* out;
  int64_t ld_out;
  void* out2;  // the forward's pre-activation
  int64_t ld_out2;
  EpilogueArgs epi;
};

constexpr int64_t kGemvRows = 2;
constexpr int64_t kGemvPiece = 8192;  // 64 KB of x a CTA for two rows
constexpr int64_t kGemvReduction = 8 * kGemvPiece;

// Whether these kernels are the faster ones for a product.
bool gemv_wins(int64_t M, int64_t R);
// Shared-memory limits on the current device.
cudaError_t gemv_init();
cudaError_t gemv_launch(FusedKind kind, GemvArgs p, bool b_mn, int sms, bool pdl, cudaStream_t stream);

}  // namespace axonn
