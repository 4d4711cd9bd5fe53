// Host interface of the elementwise kernels (elementwise.cu).
#pragma once
#include "epilogue.h"

namespace axonn {

struct DropoutKernelArgs {
  const void* x;
  const void* residual;  // or null
  void* y;
  int64_t ld_x, ld_res, ld_y;
  int64_t rows, cols;
  DropoutArgs drop;
};

struct BwdKernelArgs {
  const void* dy;
  const uint16_t* pre;  // not read with act = none
  uint16_t* dz;
  float* colsum;        // [act_bwd_groups(rows) x ld_colsum] or null
  int64_t ld_dy, ld_pre, ld_dz, ld_colsum;
  int64_t rows, cols;
  int32_t act;
  DropoutArgs drop;
};

cudaError_t dropout_launch(const DropoutKernelArgs& a, bool f32, int sms, bool pdl, cudaStream_t stream);
cudaError_t act_bwd_launch(const BwdKernelArgs& a, bool dy_f32, bool pdl, cudaStream_t stream);
int64_t act_bwd_groups(int64_t rows);
cudaError_t colsum_launch(const float* part, int64_t ld, int64_t groups, int64_t cols, float* out,
                          bool pdl, cudaStream_t stream);

}  // namespace axonn
