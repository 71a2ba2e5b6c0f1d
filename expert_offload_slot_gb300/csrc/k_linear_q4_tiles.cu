// The tile kernels of moe_linear_q4 (linear_q4_tiles.cuh) for bf16 x on 16-byte boundaries, which comes by TMA.
#include "linear_q4_tiles.cuh"

namespace moeslot {
namespace {

template <int G>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  if (a.rows <= 32) return run<Tile<32, G, 0>>(a, s);
  if (a.rows <= 64) return run<Tile<64, G, 0>>(a, s);
  if (a.rows <= 128) return run<Tile<128, G, 0>>(a, s);
  return run<Tile<256, G, 0>>(a, s);
}

}  // namespace

cudaError_t linear_q4_tiles_status(int32_t* st) { return take_status(g_status, st); }

cudaError_t launch_linear_q4_tiles(const LinearArgs& a, int group, cudaStream_t s) {
  return group == 32 ? pick<32>(a, s) : group == 64 ? pick<64>(a, s) : pick<128>(a, s);
}

}  // namespace moeslot
