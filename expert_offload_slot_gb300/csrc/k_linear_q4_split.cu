// The tile kernels of moe_linear_q4 (linear_q4_tiles.cuh) for x through registers: fp32, cut into three bf16 columns a
// row, and bf16 that lies on no 16-byte boundaries.
#include "linear_q4_tiles.cuh"

namespace moeslot {
namespace {

template <int G, int PARTS>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  // The two warps that cut x up set the pace, so a round of the pairs over tiles of 256 columns takes about three times
  // one of 64 (fp32, 4096 inputs: 129 and 41 us); the fewer such units, the better.
  const int64_t pairs = sm_count() / 2, m = (a.N + 255) / 256;
  auto rounds = [&](int rows) { return (m * ((a.rows + rows - 1) / rows) + pairs - 1) / pairs; };
  return rounds(Tile<64, G, PARTS>::ROWS) <= 3 * rounds(Tile<256, G, PARTS>::ROWS) ? run<Tile<64, G, PARTS>>(a, s)
                                                                                   : run<Tile<256, G, PARTS>>(a, s);
}

template <int PARTS>
cudaError_t pick(const LinearArgs& a, int group, cudaStream_t s) {
  return group == 32 ? pick<32, PARTS>(a, s) : group == 64 ? pick<64, PARTS>(a, s) : pick<128, PARTS>(a, s);
}

}  // namespace

cudaError_t linear_q4_split_status(int32_t* st) { return take_status(g_status, st); }

cudaError_t launch_linear_q4_split(const LinearArgs& a, int group, cudaStream_t s) {
  return a.x_f32 ? pick<3>(a, group, s) : pick<1>(a, group, s);
}

}  // namespace moeslot
