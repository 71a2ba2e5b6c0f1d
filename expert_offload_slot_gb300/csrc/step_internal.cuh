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
  int32_t x_f32, out_f32, scale_f32;
  // of the row kernel: rows of x in a pass, CTAs of a pass, blocks of a slice, slices of x that shared memory
  // holds, stages of the ring, bytes between their rows of codes and floats between those of scales
  int32_t pass_rows, ctas, slice, chunk, depth, pitch, scale_pitch;
  // of the tile kernel: K is whole blocks of 64; x stays in shared memory
  int32_t x_blocks, resident;
};
cudaError_t launch_linear_q4(const LinearArgs& a, int group, cudaStream_t s);
cudaError_t launch_linear_q4_tiles(const LinearArgs& a, int group, cudaStream_t s);      // bf16 x on 16-byte boundaries
cudaError_t launch_linear_q4_split(const LinearArgs& a, int group, cudaStream_t s);      // any x
// The first error of each file's kernels on the current device since the last call (blocking).
template <typename T>
cudaError_t take_status(T& symbol, int32_t* st) {
  const int32_t none = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(st, symbol, sizeof none);
  return e == cudaSuccess && *st != 0 ? cudaMemcpyToSymbol(symbol, &none, sizeof none) : e;
}
cudaError_t linear_q4_rows_status(int32_t* st);
cudaError_t linear_q4_tiles_status(int32_t* st);
cudaError_t linear_q4_split_status(int32_t* st);

// x as three bf16 numbers by cutting off bits: the sum is x.  Nothing is left of an infinity or a NaN.
__device__ __forceinline__ float bf16_part(float x, int part) {
  const float h = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  if (part == 0) return (__float_as_uint(x) & 0x7fffffffu) > 0x7f800000u ? __uint_as_float(0x7fc00000u) : h;
  if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) return 0.f;
  const float rest = x - h, m = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
  return part == 1 ? m : rest - m;
}

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
