// The turns of the converter warpgroups of linear_q4_tiles.cuh, apart from what a turn does, and the waits at a kernel's
// end, so that they can be walked through on the host, too (tests/q4_turns.cu).
#pragma once

#include <stdint.h>

namespace moeslot {

// C::CONVERTERS warpgroups, two or four, take turns at the steps of all tiles of a pair (tile, tile + pairs, ... below
// tiles), in one count: each is CONVERTERS steps after its last one.  At a turn it waits for its buffer of expanded codes
// (wait_buffer) and its stage of codes (wait_codes), expands half of the stage and releases it.
//
// A wait on a parity tells the phase before from the one before that only if that one is known to have ended:
// - the buffer: the turn waits for step n - A_BUFS, so step n - 2 A_BUFS has to be known.  At its last turn the warpgroup
//   saw step n - CONVERTERS - A_BUFS end, and products end in their order: A_BUFS >= CONVERTERS.
// - the codes: that the stage CODE_STAGES before this one has come.  Loads may land in any order and a warpgroup has
//   seen its own stages alone, so this follows from the buffers: the codes of a step that has been multiplied, and of all
//   before it, had come.  CODE_STAGES stages hold at least SPAN steps where a tile has two steps or more (of an odd
//   number the last stage has one step, so stages of one step never follow each other), and so the stage in question begins
//   at step n - SPAN or before.  Step n - CONVERTERS - A_BUFS is known from the last turn, n - A_BUFS once
//   this turn's buffer is free: where the first is not late enough, the wait for the buffer comes first.
// Codes first is faster where it may be, as its wait is over when the buffer comes: 100 rows by 4096 x 6144 22.3 us, the other
// way round 23.8 (two warpgroups and buffers).  With four warpgroups both orders take the same (16 rows by 2048 x 131072, 48.4 us).
#pragma nv_exec_check_disable                            // the kernel's callables are device functions, a walk's are not
template <typename C, typename WaitBuffer, typename WaitCodes, typename Expand, typename Release>
__host__ __device__ __forceinline__ void converter_turns(int group, int steps, int tile, int tiles, int pairs, WaitBuffer wait_buffer,
                                                         WaitCodes wait_codes, Expand expand, Release release) {
  static_assert(C::A_BUFS >= C::CONVERTERS, "a warpgroup's waits could meet an older phase of a buffer");
  constexpr int SPAN = C::CODE_STAGES + C::CODE_STAGES / 2;
  static_assert(C::A_BUFS <= SPAN, "or of a stage of codes");
  constexpr bool CODES_FIRST = C::CONVERTERS + C::A_BUFS <= SPAN;
  const uint32_t stages = (steps + 1) / 2;
  uint32_t n = group, nc0 = 0;                           // step, of all tiles; first stage of codes of the tile
  int s = group;                                         // step of the tile
  for (; tile < tiles; tile += pairs, s -= steps, nc0 += stages) {
    for (; s < steps; s += C::CONVERTERS, n += C::CONVERTERS) {
      const uint32_t nc = nc0 + s / 2, st = nc % C::CODE_STAGES, ab = n % C::A_BUFS;
      if (CODES_FIRST) wait_codes(st, (nc / C::CODE_STAGES) & 1);
      wait_buffer(ab, ((n / C::A_BUFS) & 1) ^ 1);
      if (!CODES_FIRST) wait_codes(st, (nc / C::CODE_STAGES) & 1);
      expand(st, s & 1, ab);
      release(st, s + 1 == steps && (s & 1) == 0);       // once for each half of a stage; a tile's last may have one only
    }
  }
}

// The end.  Products report that a buffer or a stage of x is free to the barriers of both CTAs of a pair, and copies land, on
// their own time: a CTA that left before would have them come to memory that is another's by then.  So every barrier's
// last use is waited for, by a converter warp (reports) and by who brings data in, where another warp has given up waiting, too.

// The last N of `total` uses of N barriers in turn, one after another: each wait knows the phase before to be over if that
// holds for the first.
#pragma nv_exec_check_disable
template <uint32_t N, typename Wait>
__host__ __device__ __forceinline__ void last_uses(uint32_t total, Wait wait) {
  for (uint32_t n = total > N ? total - N : 0; n < total; ++n) wait(n % N, (n / N) & 1);
}

// Of a converter warpgroup after `total` steps of all warpgroups.  The first step waited for is total - A_BUFS, and that
// total - 2 A_BUFS is over the warpgroup's last turn told.  After that all steps are known to be multiplied, so each one's
// x had come, which its loader brought once the stage's use before had been reported free.
#pragma nv_exec_check_disable
template <typename C, typename WaitBuffer, typename WaitX>
__host__ __device__ __forceinline__ void converter_end(uint32_t total, bool x_ring, WaitBuffer wait_buffer, WaitX wait_x) {
  last_uses<C::A_BUFS>(total, wait_buffer);
  if (x_ring) last_uses<C::X_STAGES>(total, wait_x);
}

}  // namespace moeslot
