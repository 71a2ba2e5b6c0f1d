// One block per delay: a warp waits on a barrier that another thread arrives at after the delay (ns; negative:
// never).  Every wait and every delay ends.
#include "../expert_offload_slot_gb300/csrc/sm103.cuh"

using namespace moeslot;

__global__ void wait_probe_kernel(const long long* delay, int* answer) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    sm103::bar_init(&bar, 1);
    sm103::bar_init_done();
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    answer[blockIdx.x * 32 + threadIdx.x] = sm103::bar_wait_warp(&bar, 0);
  } else if (threadIdx.x == 32 && delay[blockIdx.x] >= 0) {
    const uint64_t t0 = sm103::now_ns(), d = min(delay[blockIdx.x], 2000000000ll);
    while (sm103::now_ns() - t0 < d) {
    }
    sm103::bar_arrive(&bar);
  }
}

extern "C" __attribute__((visibility("default"))) int wait_probe(const long long* delay, int* answer, int blocks) {
  wait_probe_kernel<<<blocks, 64>>>(delay, answer);
  return cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess;
}
