// Internal declarations of the operators around the blocks of a step:
// moe_residual_norm, moe_linear_q4 and moe_logprobs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moeslot.h"

namespace moeslot {

moe_status set_last_error(moe_status st, const char* msg);   // text for moe_last_error()
int sm_count();                                               // of the current device
int32_t* step_status();                                       // sticky, on the current device; NULL: not found

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
  int32_t* status;
  int32_t rows, K, N, groups;
  int32_t x_f32, out_f32, scale_f32;
  // of the row kernel: rows of x in a pass, CTAs of a pass, blocks of a slice, slices of x that shared memory
  // holds, stages of the ring, bytes between their rows of codes and floats between those of scales
  int32_t pass_rows, ctas, slice, chunk, depth, pitch, scale_pitch;
  // of the tile kernel: K is whole blocks of 64; x stays in shared memory
  int32_t x_blocks, resident;
};
cudaError_t launch_linear_q4(const LinearArgs& a, int group, cudaStream_t s);
cudaError_t launch_linear_q4_tiles(const LinearArgs& a, int group, cudaStream_t s);      // bf16 x on 16-byte boundaries

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
