// Stand-ins for the attention kernels' launchers (see attn_host_stub.cpp).
#include <cuda_runtime.h>

#include <cstring>

#include "../expert_offload_slot_gb300/csrc/attn_internal.cuh"
#include "../expert_offload_slot_gb300/csrc/sample_internal.cuh"

cudaError_t stub_note(const char* what, const void* stream);

namespace {
char last_error[256] = "";
cudaError_t note(const char* what, const void* stream = nullptr) { return stub_note(what, stream); }
}  // namespace

extern "C" __attribute__((visibility("default"))) const char* stub_error() { return last_error; }

namespace moeslot {
moe_status set_last_error(moe_status st, const char* msg) {
  strncpy(last_error, msg, sizeof last_error - 1);
  return st;
}
cudaError_t prepare_attn_f32(int) { return note("prepare"); }
cudaError_t prepare_attn_rows(int) { return note("prepare"); }
cudaError_t prepare_attn_tiles(int) { return note("prepare"); }
cudaError_t prepare_attn_qkv(int, int) { return note("prepare"); }
cudaError_t launch_attn_f32(const AttnArgs&, int, int, cudaStream_t s) { return note("f32", s); }
cudaError_t launch_attn_rows(const AttnArgs&, const CUtensorMap&, const CUtensorMap&, int, int, cudaStream_t s) {
  return note("rows", s);
}
cudaError_t launch_attn_tiles(const AttnArgs&, const CUtensorMap&, const CUtensorMap&, int, int, cudaStream_t s) {
  return note("tiles", s);
}
cudaError_t launch_attn_tables(const TablesArgs&, cudaStream_t s) { return note("tables", s); }
cudaError_t launch_attn_qkv(const QkvArgs&, int, int, int, cudaStream_t s) { return note("qkv", s); }
cudaError_t launch_sample(const SampleArgs&, int, cudaStream_t s) { return note("sample", s); }
}  // namespace moeslot
