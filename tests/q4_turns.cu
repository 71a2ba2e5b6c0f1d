// The converter warpgroups' turns of moe_linear_q4's tile kernels on the host: what each waits for, in its order, as
// (what, slot, parity, 0), and what it does with it; and the waits at the end.
#include "../expert_offload_slot_gb300/csrc/linear_q4_tiles.cuh"

using namespace moeslot;

namespace {

template <typename C>
int walk(int group, int steps, int tile, int tiles, int pairs, int* out, int room) {
  int n = 0;
  auto note = [&](int what, int a, int b, int c) {
    if (n < room) {
      out[4 * n] = what;
      out[4 * n + 1] = a;
      out[4 * n + 2] = b;
      out[4 * n + 3] = c;
    }
    ++n;
  };
  converter_turns<C>(
      group, steps, tile, tiles, pairs, [&](uint32_t ab, uint32_t parity) { note(0, ab, parity, 0); },
      [&](uint32_t st, uint32_t parity) { note(1, st, parity, 0); }, [&](uint32_t st, int half, uint32_t ab) { note(2, st, half, ab); },
      [&](uint32_t st, bool twice) { note(3, st, twice ? 2 : 1, 0); });
  return n;
}

// f(Tile<columns, ...>) of a kernel; -1 for others
template <typename F>
int with(int columns, int parts, F f) {
  if (parts == 0 && columns == 32) return f(Tile<32, 128, 0>());
  if (parts == 0 && columns == 64) return f(Tile<64, 128, 0>());
  if (parts == 0 && columns == 128) return f(Tile<128, 128, 0>());
  if (parts == 0 && columns == 256) return f(Tile<256, 128, 0>());       // one warpgroup: no turns
  if (parts == 1 && columns == 64) return f(Tile<64, 128, 1>());
  if (parts == 3 && columns == 64) return f(Tile<64, 128, 3>());
  return -1;
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int q4_shape(int columns, int parts, int* converters, int* buffers, int* stages) {
  return with(columns, parts, [&](auto tile) {
    typedef decltype(tile) C;
    *converters = C::CONVERTERS;
    *buffers = C::A_BUFS;
    *stages = C::CODE_STAGES;
    return 0;
  });
}

// Notes of a warpgroup over the tiles tile, tile + pairs, ...; how many there are, of which `room` are kept.
extern "C" __attribute__((visibility("default"))) int q4_turns(int columns, int parts, int group, int steps, int tile, int tiles, int pairs,
                                                               int* out, int room) {
  return with(columns, parts, [&](auto shape) { return walk<decltype(shape)>(group, steps, tile, tiles, pairs, out, room); });
}

// The waits of a converter warpgroup after `total` steps, as (what, slot, parity); the stages of x in *stages.
extern "C" __attribute__((visibility("default"))) int q4_end(int columns, int parts, int total, int x_ring, int* out, int* stages) {
  return with(columns, parts, [&](auto shape) {
    int n = 0;
    auto note = [&](int what, int slot, int parity) {
      out[3 * n] = what;
      out[3 * n + 1] = slot;
      out[3 * n++ + 2] = parity;
    };
    *stages = decltype(shape)::X_STAGES;
    converter_end<decltype(shape)>(total, x_ring != 0, [&](uint32_t ab, uint32_t parity) { note(0, ab, parity); },
                                   [&](uint32_t st, uint32_t parity) { note(1, st, parity); });
    return n;
  });
}

// Those of who loads the codes, after `total` loads.
extern "C" __attribute__((visibility("default"))) int q4_codes_end(int columns, int parts, int total, int* out) {
  return with(columns, parts, [&](auto shape) {
    int n = 0;
    last_uses<decltype(shape)::CODE_STAGES>(total, [&](uint32_t st, uint32_t parity) {
      out[2 * n] = st;
      out[2 * n++ + 1] = parity;
    });
    return n;
  });
}
