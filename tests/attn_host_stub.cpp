// Stand-ins for the CUDA runtime: two devices that exist by name only, and a log of the device that each
// call found current.  Linked with csrc/attn_api.cu and attn_host_stub.cu into a library that needs no GPU.
#include <cuda_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace {
int current = 0;
char text[4096] = "";
unsigned driver_ok(...) { return 0; }
}  // namespace

cudaError_t stub_note(const char* what, const void* stream) {
  char line[64];
  snprintf(line, sizeof line, "%s@%d/%d ", what, current, (int)reinterpret_cast<uintptr_t>(stream));
  strncat(text, line, sizeof text - strlen(text) - 1);
  return cudaSuccess;
}

extern "C" {
__attribute__((visibility("default"))) void stub_set_device(int d) { current = d; }
__attribute__((visibility("default"))) int stub_device() { return current; }
__attribute__((visibility("default"))) const char* stub_log() { return text; }
__attribute__((visibility("default"))) void stub_clear() { text[0] = 0; }

cudaError_t CUDARTAPI cudaGetDeviceCount(int* n) { *n = 2; return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
cudaError_t CUDARTAPI cudaSetDevice(int d) {
  if (d < 0 || d > 1) return cudaErrorInvalidDevice;
  current = d;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t CUDARTAPI cudaMalloc(void** p, size_t) { *p = malloc(64); return stub_note("malloc", nullptr); }
cudaError_t CUDARTAPI cudaFree(void* p) { free(p); return stub_note("free", nullptr); }
cudaError_t CUDARTAPI cudaMemset(void*, int, size_t) { return stub_note("memset", nullptr); }
cudaError_t CUDARTAPI cudaMemcpy(void* to, const void*, size_t n, cudaMemcpyKind) { memset(to, 0, n); return stub_note("memcpy", nullptr); }
cudaError_t CUDARTAPI cudaDeviceSynchronize() { return stub_note("sync", nullptr); }
cudaError_t CUDARTAPI cudaGetLastError() { return cudaSuccess; }
const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return "stub"; }
cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                                       cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(driver_ok);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
// The runtime's registration of compiled device code: nothing is registered.
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}
