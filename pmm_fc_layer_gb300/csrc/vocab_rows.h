// Host interface of the kernels over rows of vocabulary logits
// (vocab_rows.cu, distill.cu): log probabilities of given tokens with entropy and top
// alternatives, their way back, and distillation from a teacher's lists.  The
// C entry points that validate arguments and call these are
// axonn_token_logprobs, axonn_token_logprobs_bwd and axonn_distill in
// axonn_fc.cu.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace axonn {

constexpr int kMaxTop = 128;    // longest list axonn_token_logprobs makes
constexpr int kMaxList = 1024;  // longest list axonn_distill reads

// Rows of logits, bf16 or fp32, row stride ld elements.
struct LogitRows {
  const void* logits;
  int64_t ld;
  const uint8_t* keep;  // [rows] or null; 0: the row counts for nothing
  int64_t rows, vocab;
  float temperature;
  int32_t f32;
};

struct LogprobArgs {
  LogitRows in;
  const int32_t* tokens;  // [rows]; null where logprob is
  float* logprob;         // each [rows] or null
  float* entropy;
  float* lse;             // with lse_parts [rows x 2]: the largest logit, ln S
  int32_t* top_index;     // [rows x k], row stride ld_top, or null
  float* top_logprob;     // the same, or null
  int64_t ld_top;
  int32_t k;              // 0: no list
  int32_t lse_parts;
};

struct LogprobBwdArgs {
  LogitRows in;
  const int32_t* tokens;    // [rows] or null (dlogprob is null then)
  const float* lse;         // [rows], with lse_parts [rows x 2]
  const float* dlogprob;    // [rows] or null
  const float* entropy;     // [rows]; null where dentropy is
  const float* dentropy;    // [rows] or null
  void* dlogits;            // of the logits' type, may be the logits
  int64_t ld_dlogits;
  int32_t lse_parts;
};

struct DistillArgs {
  LogitRows in;
  const int32_t* top_index;  // [rows x k], row stride ld_top
  const float* top_logit;
  int64_t ld_top;
  int32_t k;
  float grad_scale;
  float* token_loss;  // [rows]
  float* loss;        // [1]; during the call the kernels' counter
  int32_t* kept;      // [1]
  void* dlogits;      // of the logits' type, may be the logits; or null
  int64_t ld_dlogits;
};

cudaError_t logprobs_launch(const LogprobArgs& a, int sms, bool pdl, cudaStream_t stream);
cudaError_t logprobs_bwd_launch(const LogprobBwdArgs& a, bool pdl, cudaStream_t stream);
cudaError_t distill_init();  // once for each device, before the first launch
cudaError_t distill_launch(const DistillArgs& a, int sms, uint64_t timeout_ns, int inject, bool pdl,
                           cudaStream_t stream);
// Reads (and clears if set) the device error word of the distillation.
cudaError_t distill_take_status(unsigned long long* word, cudaStream_t stream);

}  // namespace axonn
