// Internal declarations of the operators around the blocks of a step:
// moe_residual_norm, moe_linear_q4 and moe_logprobs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moeslot.h"

namespace moeslot {

moe_status set_last_error(moe_status st, const char* msg);   // text for moe_last_error()
int sm_count();                                               // of the current device

struct NormArgs {
  const void *x, *gate, *post, *residual, *pre;
  void *sum, *y;                                              // residual_out and y
  int64_t x_stride, gate_stride, residual_stride, sum_stride, y_stride;
  int32_t rows, hidden, gate_kind, gate_sigmoid;
  float scale, eps, offset;
};
cudaError_t launch_residual_norm(const NormArgs& a, int dtype, int residual_dtype, cudaStream_t s);

struct LinearArgs {
  const void* x;
  const uint8_t* codes;                                       // [N][K / 2]
  const void *scales, *bias;                                  // [N][groups], [N]
  void* out;
  int64_t x_stride, out_stride;
  int32_t rows, K, N, groups;
  int32_t x_f32, out_f32;
  int32_t pass_rows, split_log2, chunk, ctas;                       // of the row kernel: k_linear_q4.cu
};
cudaError_t launch_linear_q4(const LinearArgs& a, int group, int scale_dtype, cudaStream_t s);

struct LogprobArgs {
  const void* logits;
  const int32_t* targets;
  float *logp, *entropy, *top_logp;
  int32_t *rank, *top_ids;
  int64_t row_stride;
  int32_t rows, vocab, top;
};
cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s);

}  // namespace moeslot
