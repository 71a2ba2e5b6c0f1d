// moe_linear_q4 for many columns of x or many outputs: the products of k_linear_q4.cu on tcgen05, codes
// expanded into tensor memory.  Two files make its kernels: k_linear_q4_tiles.cu for x by TMA, k_linear_q4_split.cu
// for x through registers.
//
// Two CTAs work as a pair (cluster of two, cta_group::2) on tiles of 256 outputs by BN rows of x:
// M = 256 outputs, 128 in each CTA, N up to 128 rows of x, half of them in each CTA's shared memory.
// K goes in steps of 128.  A converter thread owns one output: it reads its 128 codes of a step from
// shared memory and stores them as bf16 into its lane of tensor memory, which is the products' A
// operand, so that the expanded weights (four times the codes) never pass through shared
// memory.  The accumulator of a group of inputs is exact up to the tensor core's sums; the
// drain threads, one output each, too, take it from tensor memory, scale it in fp32 and
// add it to their registers, while the next group's products run into another accumulator.
// With BN = 256 a step has two accumulators of 128 rows, each expanded code being used twice.
//
// Expansion of a word of eight codes: nibbles 0, 2, 4, 6 and 1, 3, 5, 7 each into the bytes of a
// word, u = code ^ 8 = code + 8 in each byte; a byte permutation puts bytes i of the two into the
// halves of a word, zeros above.  Read as bf16 such a half is u 2^-133 (a subnormal), and
// u 2^-133 2^127 - 8 2^-6 = code 2^-6, exactly, in one fma.  The sums are multiplied by 2^6 at the end.
//
// Roles: warp 0 loads x by TMA, warp 2 the codes, warp 1 of the first CTA issues the products; then the
// converters (one, two or four warpgroups that take turns at the steps), then two warpgroups of drain
// threads, which take half of an accumulator's columns each.
// Where all rows of x fit one tile and shared memory, x is loaded once and stays (`resident`): few rows
// by many outputs are a stream of codes.
// Tensor memory (512 columns): two to six steps of expanded codes of 64 columns, then three or four accumulators.
//
// What bounds it.  2048 rows by 4096 x 6144 (103 GFLOP): 77 us, 1.34 PFLOP/s or 68 % of cuBLAS's bf16 burst
// rate; the products alone take 52, with the drain beside them 69: each accumulator's 64 KB pass
// through tensor memory's port once more for every 512 cycles of products, and an SM's TMA unit, at some 35
// bytes a cycle, needs 1170 cycles for the x and codes of a step whose products take 1024.  Groups of 64 and 32
// have two and four accumulators a step: 116 and 206 us.  The drain's loop unrolled over four groups cost 6 us.
// 16 rows by 2048 x 131072 (147 MB): 48 us, 3.1 TB/s: a step's own instructions, barriers and
// waits, in each role one after another, take 475 cycles in the products' warp alone (28 us) and 830 with all
// roles beside it; HBM would allow 350.  With x brought in for every step, and two converter
// warpgroups instead of four, it took 56; with codes by cp.async of two warps 67.  A warp's own instructions
// being the cost, barriers' phases are kept where that is cheap, and a wait that need not wait is a test and a branch.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "linear_q4_turns.cuh"
#include "sm103.cuh"
#include "step_internal.cuh"

namespace moeslot {
namespace {
using namespace sm103;

typedef __nv_bfloat16 bf16;
constexpr int kCodeStage = 128 * 128;          // 128 outputs by 256 codes: two steps
constexpr int kShared = 225 * 1024;
__device__ int32_t g_status;                   // of this file's kernels: set where a wait ran out
constexpr int kXBars = 8;                      // barriers of the stages of x, or of eighths of a resident x

// PARTS 0: x is bf16 and comes by TMA; 1: bf16 on any boundary, 3: fp32, cut into three columns a row, both by two warps.
template <int BN_, int G_, int PARTS_>
struct Tile {
  static constexpr int BN = BN_, G = G_, PARTS = PARTS_, P = 128 / G;
  static constexpr int HN = BN < 128 ? BN : 128, HALVES = BN / HN;       // columns of an accumulator
  static constexpr int BUFS = HN == 128 ? 3 : 4;                         // accumulators
  static constexpr int A_BUFS = (512 - BUFS * HN) / 64 < 6 ? (512 - BUFS * HN) / 64 : 6;       // expanded steps
  static constexpr int D0 = A_BUFS * 64;                 // tensor memory: the accumulators' first column
  static constexpr int COLS = HN / 2;                    // of a CTA's shared memory and of a drain thread
  static constexpr int COL_ROWS = PARTS == 3 ? COLS / 3 : COLS, ROWS = 2 * HALVES * COL_ROWS;  // rows of x there, and in a tile
  static constexpr int CONVERTERS = BN <= 64 ? 4 : BN <= 128 ? 2 : 1;    // warpgroups
  static constexpr int THREADS = 128 * (1 + CONVERTERS + 2);
  static constexpr int X_PART = HN / 2 * 128;            // this CTA's rows by 64 inputs
  static constexpr int X_STAGE = HALVES * 2 * X_PART;    // [half][64 inputs][rows][128 bytes]
  static constexpr int X_STAGES = BN >= 256 ? 3 : 4;
  static constexpr int CODE_STAGES = BN >= 256 ? 6 : 5;
  static constexpr int X_BYTES = BN >= 256 ? X_STAGES * X_STAGE : 128 * 1024;      // its ring, or all of a resident x
  static constexpr int BYTES = CODE_STAGES * kCodeStage + X_BYTES + 1024;
  static_assert(X_STAGES * X_STAGE <= X_BYTES, "room for the ring");
  // registers of a thread at launch and after the split: (1 + CONVERTERS + 2) * launch >= the sum of the shares
  static constexpr int REGS = CONVERTERS == 4 ? 72 : CONVERTERS == 2 ? 96 : 128, MISC = CONVERTERS == 1 ? 64 : 56;
  static constexpr int CONVERT = CONVERTERS == 4 ? 64 : CONVERTERS == 2 ? 72 : 80;
  static constexpr int DRAIN = CONVERTERS == 4 ? 96 : CONVERTERS == 2 ? 136 : 184;
  static_assert(MISC + CONVERTERS * CONVERT + 2 * DRAIN <= (3 + CONVERTERS) * REGS, "the split waits for ever otherwise");
  static_assert(BYTES <= kShared, "shared memory");
};

// Eight codes as four pairs of code 2^-6 in bf16, in their order.
__device__ __forceinline__ void widen(uint32_t w, uint32_t* p) {
  uint32_t lo, hi;                             // (w & 0x0f0f0f0f) ^ 0x08080808, and of w >> 4
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(lo) : "r"(w), "r"(0x0f0f0f0fu), "r"(0x08080808u));
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(hi) : "r"(w >> 4), "r"(0x0f0f0f0fu), "r"(0x08080808u));
  constexpr uint32_t sel[4] = {0xc480, 0xd591, 0xe6a2, 0xf7b3};          // 8 + n: the sign of byte n, eight times: 0
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(u) : "r"(lo), "r"(hi), "r"(sel[i]));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(p[i]) : "r"(u), "r"(0x7f007f00u), "r"(0xbe00be00u));
  }
}

// Eight inputs of row t from k on (k is a multiple of 8, as K is); zeros past K and the rows.
template <int PARTS>
struct Eight {
  float v[PARTS == 3 ? 8 : 4];                 // fp32, or pairs of bf16
  __device__ __forceinline__ void get(const LinearArgs& a, int t, int k, bool wide) {
#pragma unroll
    for (int i = 0; i < (PARTS == 3 ? 8 : 4); ++i) v[i] = 0.f;
    if (t >= a.rows || k >= a.K) return;
    if constexpr (PARTS == 1) {
      const uint16_t* p = static_cast<const uint16_t*>(a.x) + t * a.x_stride + k;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(p[2 * i] | (uint32_t)p[2 * i + 1] << 16);
    } else {
      const float* p = static_cast<const float*>(a.x) + t * a.x_stride + k;
      if (wide) {
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
        *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(p + 4);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[i];
      }
    }
  }
  __device__ __forceinline__ uint4 part(int q) const {       // as bf16
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (PARTS == 1) w[i] = __float_as_uint(v[i]);
      else w[i] = __float_as_uint(bf16_part(v[2 * i], q)) >> 16 | (__float_as_uint(bf16_part(v[2 * i + 1], q)) & 0xffff0000u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A ring's place, and the parity of its barriers' phase there.
template <int N>
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float* v) {
  if constexpr (N == 16) tmem_ld16(addr, v);
  else tmem_ld32(addr, v);
}

template <typename C>
__global__ __cluster_dims__(2, 1, 1) __launch_bounds__(C::THREADS, 1)
void linear_q4_tiles_kernel(const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mx, const LinearArgs a) {
  extern __shared__ uint8_t raw[];
  // x_full, a_full and d_empty are the first CTA's, who issues the products, for both; the others are of each its own
  __shared__ __align__(8) uint64_t c_full[C::CODE_STAGES], c_empty[C::CODE_STAGES], x_full[kXBars], x_empty[C::X_STAGES],
      a_full[C::A_BUFS], a_empty[C::A_BUFS], d_full[C::BUFS], d_empty[C::BUFS], drained;
  __shared__ uint32_t tmem_slot;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t codes = smem_addr(smem), xs = codes + C::CODE_STAGES * kCodeStage;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, rank = (int)pair_rank();
  if (tid == 0) {
    for (int s = 0; s < C::CODE_STAGES; ++s) {
      bar_init(c_full + s, 1);
      bar_init(c_empty + s, C::CONVERTERS == 1 ? 4 : 8);
    }
    for (int s = 0; s < kXBars; ++s) bar_init(x_full + s, C::PARTS == 0 ? 2 : 4);
    for (int s = 0; s < C::X_STAGES; ++s) bar_init(x_empty + s, 1);
    for (int s = 0; s < C::A_BUFS; ++s) {
      bar_init(a_full + s, 8);
      bar_init(a_empty + s, 1);
    }
    for (int s = 0; s < C::BUFS; ++s) {
      bar_init(d_full + s, 1);
      bar_init(d_empty + s, 16);
    }
    bar_init(&drained, 1);
    bar_init_done();
  }
  if (wid == 2) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  pair_sync();                                           // the other CTA's barriers are ready, too
  tc_fence_after();
  grid_wait();
  const uint32_t tmem = tmem_slot;

  const int steps = (a.K + 127) / 128, n_tiles = (a.rows + C::ROWS - 1) / C::ROWS, tiles = (a.N + 255) / 256 * n_tiles;
  const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
  const int eighth = (steps + kXBars - 1) / kXBars;      // steps behind one barrier of a resident x
  const uint32_t mine = (uint32_t)((tiles - pair + pairs - 1) / pairs);  // tiles of this pair
  bool alive = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {        // bounded; after a timeout nothing waits any more
    if (!bar_test(b, parity) && alive && !bar_wait(b, parity)) {
      alive = false;
      atomicCAS(&g_status, 0, MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  };

  if (wid < 4) {
    regs_give<C::MISC>();
    if (C::PARTS > 0 && (wid == 0 || wid == 3)) {
      // ------------------------------------------------- x, through registers
      // A lane takes eight inputs of a row and stores them in each of the row's columns, swizzled; zeros past K and rows.
      constexpr int PARTS = C::PARTS > 0 ? C::PARTS : 1, UNITS = C::HALVES * C::COL_ROWS * 16;
      const bool wide = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.x_stride * (PARTS == 3 ? 4 : 2) % 16 == 0;
      const uint32_t lead_full = lead_addr(x_full);
      Ring<C::X_STAGES> rx;
      rx.phase = 1;
      for (int tile = pair; tile < tiles; tile += pairs) {
        const int t0 = tile % n_tiles * C::ROWS + rank * C::COL_ROWS;
        for (int s = 0; s < steps; ++s) {
          wait(x_empty + rx.i, rx.phase);
          uint8_t* stage = smem + (xs - codes) + rx.i * C::X_STAGE;
          constexpr int FLIGHT = 4;            // loads on their way
          for (int u0 = (wid ? 32 : 0) + lane; u0 < UNITS; u0 += 64 * FLIGHT) {
            Eight<PARTS> x[FLIGHT];
#pragma unroll
            for (int f = 0; f < FLIGHT; ++f) {
              const int u = u0 + 64 * f, r = u >> 4, h = r / C::COL_ROWS;
              x[f].get(a, u < UNITS ? t0 + h * C::COL_ROWS + r : a.rows, s * 128 + (u & 15) * 8, wide);      // 2 h COL_ROWS + r - h COL_ROWS
            }
#pragma unroll
            for (int f = 0; f < FLIGHT; ++f) {
              const int u = u0 + 64 * f, chunk = u & 15, r = u >> 4, h = r / C::COL_ROWS;
              if (u >= UNITS) break;
              uint8_t* to = stage + (2 * h + (chunk >> 3)) * C::X_PART;
#pragma unroll
              for (int p = 0; p < PARTS; ++p) {
                const int n = (r - h * C::COL_ROWS) * PARTS + p;
                *reinterpret_cast<uint4*>(to + n * 128 + (((chunk & 7) ^ (n & 7)) << 4)) = x[f].part(p);
              }
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive_at(lead_full + rx.i * 8);
          rx.next();
        }
      }
    } else if (wid == 0) {
      // ------------------------------------------------------------ x, by TMA
      uint32_t st = 0, phase = 1;
      auto load = [&](uint32_t dst, uint32_t bar, int s, int t) {        // a step: one box, or two where K ends inside 64
        if (a.x_blocks) {
          if (lane < C::HALVES) tma_3d_pair(dst + lane * 2 * C::X_PART, &mx, bar, 0, t + lane * C::HN, 2 * s);
        } else if (lane < 2 * C::HALVES) {
          tma_3d_pair(dst + lane * C::X_PART, &mx, bar, s * 128 + (lane & 1) * 64, t + (lane >> 1) * C::HN, 0);
        }
      };
      auto announce = [&](uint64_t* bar, int bytes) {
        if (lane == 0) {
          if (rank == 0) bar_expect(bar, 2 * bytes);     // of both CTAs
          else bar_arrive_at(lead_addr(bar));
        }
        __syncwarp();
      };
      if (a.resident) {
        for (int s = 0; s < steps; ++s) {
          uint64_t* bar = x_full + s / eighth;
          if (s % eighth == 0) announce(bar, min(eighth, steps - s) * C::X_STAGE);
          load(xs + s * C::X_STAGE, lead_addr(bar), s, rank * (C::HN / 2));
        }
        if (rank == 0)
          for (int s = 0; s < steps; s += eighth) wait(x_full + s / eighth, 0);
      } else {
        for (int tile = pair; tile < tiles; tile += pairs) {
          const int t0 = tile % n_tiles * C::BN + rank * (C::HN / 2);
          for (int s = 0; s < steps; ++s) {
            wait(x_empty + st, phase);
            announce(x_full + st, C::X_STAGE);
            load(xs + st * C::X_STAGE, lead_addr(x_full + st), s, t0);
            if (++st == C::X_STAGES) {
              st = 0;
              phase ^= 1;
            }
          }
        }
        if (rank == 0) last_uses<C::X_STAGES>(mine * steps, [&](uint32_t i, uint32_t parity) { wait(x_full + i, parity); });
      }
      if (!alive) {                                      // bounded: copies in flight land before the memory is given up
        const uint64_t t = now_ns();
        while (now_ns() - t < 1000000ull) __nanosleep(1000);
      }
    } else if (wid == 2) {
      // --------------------------------------------------------------- codes
      uint32_t st = 0, phase = 1;
      for (int tile = pair; tile < tiles; tile += pairs) {
        const int m0 = tile / n_tiles * 256 + rank * 128;
        for (int at = 0; at < a.K / 2; at += 128) {
          wait(c_empty + st, phase);
          if (lane == 0) {
            bar_expect(c_full + st, kCodeStage);
            tma_2d(codes + st * kCodeStage, &mc, c_full + st, at, m0);
          }
          if (++st == C::CODE_STAGES) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      last_uses<C::CODE_STAGES>(mine * ((steps + 1) / 2), [&](uint32_t i, uint32_t parity) { wait(c_full + i, parity); });
      if (!alive) {
        const uint64_t t = now_ns();
        while (now_ns() - t < 1000000ull) __nanosleep(1000);
      }
    } else if (wid == 1 && rank == 0) {
      // ----------------------------------------------------------------- MMAs
      const uint32_t lead = elect_lead();
      constexpr uint32_t kDesc = tc_idesc(C::HN, false);
      const uint64_t x_desc = tc_desc<128>(xs);
      uint32_t seen = 0;                                 // eighths of a resident x that have come
      // Descriptors are made once; a stage or a sixteen of K adds to their address field (units of 16 bytes).
      Ring<C::A_BUFS> ra;
      Ring<C::X_STAGES> rx;
      Ring<C::BUFS> rd;
      rd.phase = 1;
      for (int tile = pair; tile < tiles; tile += pairs) {
        for (int s = 0; s < steps; ++s) {
          uint64_t xd = x_desc;
          wait(a_full + ra.i, ra.phase);
          if (!a.resident) {
            wait(x_full + rx.i, rx.phase);
            xd += rx.i * (C::X_STAGE >> 4);
          } else {
            if (s == (int)seen * eighth && tile == pair) wait(x_full + seen++, 0);
            xd += s * (C::X_STAGE >> 4);
          }
          const uint32_t ad = tmem + ra.i * 64;
#pragma unroll
          for (int p = 0; p < C::P; ++p) {
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
              wait(d_empty + rd.i, rd.phase);
              tc_fence_after();
              const uint32_t dd = tmem + C::D0 + rd.i * C::HN;
#pragma unroll
              for (int k = 0; k < C::G / 16; ++k) {
                const int at = p * (C::G / 16) + k;      // sixteens of the step
                tc_mma_ts(lead, dd, ad + at * 8, xd + (((2 * h + (at >> 2)) * C::X_PART + (at & 3) * 32) >> 4), kDesc, k > 0);
              }
              tc_commit(lead, d_full + rd.i);
              rd.next();
            }
          }
          tc_commit(lead, a_empty + ra.i);
          ra.next();
          if (!a.resident) {
            tc_commit(lead, x_empty + rx.i);
            rx.next();
          }
        }
      }
      // products in flight end before the memory is given up, also where the drain has given up waiting for them
      tc_commit(lead, &drained, 1);
      if (!bar_wait(&drained, 0)) atomicCAS(&g_status, 0, MOE_ERR_TIMEOUT);
    }
  } else if (wid < 4 + 4 * C::CONVERTERS) {
    regs_give<C::CONVERT>();
    // ------------------------------------------------------------- expansion
    const int group = (wid >> 2) - 1, row = (wid & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wid & 3) << 21), lead_full = lead_addr(a_full);
    auto expand = [&](uint32_t st, int half, uint32_t ab) {              // half a stage of codes into buffer ab
      const uint8_t* src = smem + st * kCodeStage + row * 128;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {                      // 64 codes at a time
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + (((half * 4 + q * 2 + i) ^ (row & 7)) << 4));
          widen(u.x, w + i * 16);
          widen(u.y, w + i * 16 + 4);
          widen(u.z, w + i * 16 + 8);
          widen(u.w, w + i * 16 + 12);
        }
        tmem_st32(lanes + ab * 64 + q * 32, w);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_at(lead_full + ab * 8);
    };
    auto wait_buffer = [&](uint32_t ab, uint32_t parity) { wait(a_empty + ab, parity); };
    if constexpr (C::CONVERTERS == 1) {                  // its own loop: 2048 rows by 4096 x 6144 77 us, by the other one 82
      Ring<C::CODE_STAGES> rc;
      Ring<C::A_BUFS> ra;
      ra.phase = 1;
      for (int tile = pair; tile < tiles; tile += pairs) {
        for (int s0 = 0; s0 < steps; s0 += 2, rc.next()) {
          wait(c_full + rc.i, rc.phase);
#pragma unroll 1
          for (int half = 0; half < 2 && s0 + half < steps; ++half, ra.next()) {
            wait(a_empty + ra.i, ra.phase);
            expand(rc.i, half, ra.i);
          }
          if (lane == 0) bar_arrive(c_empty + rc.i);
        }
      }
    } else {
      converter_turns<C>(
          group, steps, pair, tiles, pairs, wait_buffer, [&](uint32_t st, uint32_t parity) { wait(c_full + st, parity); }, expand,
          [&](uint32_t st, bool twice) {
            if (lane == 0) {
              bar_arrive(c_empty + st);
              if (twice) bar_arrive(c_empty + st);
            }
          });
    }
    // one warp: waits of all of them slow the drain of the last products (32 rows by 2048 x 2048 10.0 instead of 9.7 us)
    if (wid == 4) converter_end<C>(mine * steps, !a.resident, wait_buffer, [&](uint32_t i, uint32_t parity) { wait(x_empty + i, parity); });
  } else {
    regs_take<C::DRAIN>();
    // ----------------------------------------------- scaling, sums and output
    constexpr int COLS = C::COLS, PIECE = COLS < 32 ? COLS : 32;         // of an accumulator, of a load
    const int side = (wid - 4 - 4 * C::CONVERTERS) >> 2, row = (wid & 3) * 32 + lane;
    const uint32_t d_addr = tmem + ((uint32_t)(wid & 3) << 21) + C::D0 + side * COLS, lead_empty = lead_addr(d_empty);
    Ring<C::BUFS> rd;
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int n = tile / n_tiles * 256 + rank * 128 + row, t0 = tile % n_tiles * C::ROWS + side * C::COL_ROWS;
      const int64_t at = (int64_t)min(n, a.N - 1) * a.groups;
      auto scale = [&](int g) {
        if (g >= a.groups) return 0.f;
        return a.scale_f32 ? static_cast<const float*>(a.scales)[at + g] : __bfloat162float(static_cast<const bf16*>(a.scales)[at + g]);
      };
      uint64_t acc[C::HALVES][COLS / 2];                 // pairs of fp32
#pragma unroll
      for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) acc[h][j] = 0;
      constexpr int AHEAD = 4;                           // scales on their way
      float next[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) next[k] = scale(k);
      const int groups = steps * C::P;                   // those past the end of K have no scale and zeros of x
#pragma unroll 1
      for (int g = 0; g < groups; ++g) {
          const float now = next[0];
#pragma unroll
          for (int k = 0; k < AHEAD - 1; ++k) next[k] = next[k + 1];
          next[AHEAD - 1] = scale(g + AHEAD);
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h) {
            wait(d_full + rd.i, rd.phase);
            tc_fence_after();
            const uint64_t factor = pack2(now, now);
#pragma unroll
            for (int j0 = 0; j0 < COLS; j0 += PIECE) {
              float d[PIECE];
              tmem_load<PIECE>(d_addr + rd.i * C::HN + j0, d);
              if (j0 + PIECE == COLS) {                  // read: the products may go on
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_at(lead_empty + rd.i * 8);
              }
#pragma unroll
              for (int j = 0; j < PIECE; j += 2)
                acc[h][(j0 + j) / 2] = fma2(factor, pack2(d[j], d[j + 1]), acc[h][(j0 + j) / 2]);
            }
            rd.next();
          }
      }
      if (n < a.N) {
        float bias = 0.f;
        if (a.bias) bias = C::PARTS == 3 ? static_cast<const float*>(a.bias)[n] : __bfloat162float(static_cast<const bf16*>(a.bias)[n]);
        auto column = [&](int h, int j) {
          float lo, hi;
          unpack2(acc[h][j / 2], lo, hi);
          return j & 1 ? hi : lo;
        };
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
          for (int j = 0; j < C::COL_ROWS; ++j) {
            const int t = t0 + 2 * h * C::COL_ROWS + j;
            if (t >= a.rows) break;
            const float sum = C::PARTS == 3 ? column(h, 3 * j) + (column(h, 3 * j + 1) + column(h, 3 * j + 2)) : column(h, j);
            const float v = fmaf(sum, 64.f, bias);
            if (a.out_f32) static_cast<float*>(a.out)[t * a.out_stride + n] = v;
            else static_cast<bf16*>(a.out)[t * a.out_stride + n] = __float2bfloat16_rn(v);
          }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();                                           // neither CTA's memory or barriers are used any more
  tc_fence_after();
  if (wid == 2) tmem_free(tmem, 512);
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  static const auto encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  const cuuint32_t one[3] = {1, 1, 1};
  return encode && encode(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes as [N][K / 2] bytes: a box is a stage.
bool code_map(CUtensorMap* m, const LinearArgs& a) {
  const cuuint64_t dims[2] = {(cuuint64_t)a.K / 2, (cuuint64_t)a.N}, strides[1] = {(cuuint64_t)a.K / 2};
  const cuuint32_t box[2] = {128, 128};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, dims, strides, box);
}

// x as [K / 64][rows][64] (one box brings the 128 inputs of a step) or, where K ends inside 64, as [1][rows][K].
bool x_map(CUtensorMap* m, const LinearArgs& a, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)(a.x_blocks ? 64 : a.K), (cuuint64_t)a.rows, (cuuint64_t)(a.x_blocks ? a.K / 64 : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)a.x_stride * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)(a.x_blocks ? 2 : 1)};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.x, dims, strides, box);
}

template <typename C>
cudaError_t run(LinearArgs a, cudaStream_t s) {
  a.x_blocks = a.K % 64 == 0;
  const int steps = (a.K + 127) / 128;
  a.resident = C::PARTS == 0 && a.rows <= C::ROWS && steps * C::X_STAGE <= C::X_BYTES;
  CUtensorMap mc = {}, mx = {};
  if (!code_map(&mc, a) || (C::PARTS == 0 && !x_map(&mx, a, C::COLS))) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};       // devices whose kernel has the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(linear_q4_tiles_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t tiles = (int64_t)((a.N + 255) / 256) * ((a.rows + C::ROWS - 1) / C::ROWS), pairs = sm_count() / 2;
  return sm103::launch(linear_q4_tiles_kernel<C>, 2 * (int)(tiles < pairs ? tiles : pairs), C::THREADS, C::BYTES, s, mc, mx, a);
}

}  // namespace
}  // namespace moeslot
