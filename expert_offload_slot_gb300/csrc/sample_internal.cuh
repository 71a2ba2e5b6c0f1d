// Internal declarations of moe_sample.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moeslot {

struct SampleArgs {
  const void* logits;          // [rows][row_stride] elements
  int64_t row_stride;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* ids;
  float* logp;
  int32_t rows, vocab, chunk;  // chunk: logits per CTA of the row's cluster
};
cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s);

}  // namespace moeslot
