// Host interface of the linear cross entropy's row kernels (linear_ce.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace axonn {

// Only the rows whose label counts take part: they are packed, in order,
// into the first n of `rows` places, and n stays on the device.
struct CeRowArgs {
  const uint16_t* x;      // bf16 [rows x cols], as the caller has it
  int64_t ld_x;
  const int32_t* labels;  // [rows]
  const uint8_t* keep;    // or null: every label in range counts
  int64_t rows, cols, vocab;
  float grad_scale;
  int32_t* index;         // [rows] packed place -> row
  int32_t* place;         // [rows] row -> packed place, or -1
  int32_t* packed_labels; // [rows]
  uint16_t* packed_x;     // bf16 [rows x ld_packed]
  int64_t ld_packed;
  float* coef;            // [1] grad_scale / n
  uint32_t* done;         // [1] blocks of the combining kernel that have finished
  // dX as fp32 parts of a split reduction: how many, and how many rows apart,
  // follow from n (see ce_index_kernel); part_rows = 0: none.
  int2* parts;            // [1] {parts, rows apart}
  int64_t part_rows;      // rows of all parts together
  int32_t part_units;     // tiles that run at once
  int32_t part_tile, part_tiles_n;  // rows of a tile, tiles across
  int32_t most_parts;
  const float2* stats;    // [groups x rows]
  int64_t groups;
  int32_t group_cols;
  const float* label_logit;  // [rows], packed
  float* lse2;               // [rows], packed
  float* token_loss;         // [rows]
  float* lse;                // [rows] natural logsumexp of the counted rows (0 elsewhere), or null
  float* loss;
  int32_t* kept;
  uint16_t* dx;              // or null
  int64_t ld_dx;
};

// n, the packing, and the losses (0) of the rows that do not count.
cudaError_t ce_index_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream);
cudaError_t ce_gather_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream);
// Each packed row's logsumexp from its groups' statistics, its loss, and the
// mean of the counted losses.
cudaError_t ce_combine_launch(const CeRowArgs& a, bool pdl, cudaStream_t stream);
// The kept distances of columns [col0, col0 + cols) to P = softmax - onehot,
// in place.
cudaError_t ce_scale_launch(const CeRowArgs& a, uint16_t* piece, int64_t ld_piece, int64_t col0,
                            int64_t cols, int sms, bool pdl, cudaStream_t stream);
// dx from its packed rows: bf16, or the sum of fp32 parts, in order; zeros
// where a row does not count.
cudaError_t ce_unpack_launch(const CeRowArgs& a, const void* packed, int64_t ld, bool f32, int sms, bool pdl,
                             cudaStream_t stream);

}  // namespace axonn
