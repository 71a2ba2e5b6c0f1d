// moe_linear_q4 for many columns of x or many outputs, bf16 inputs: the products of
// k_linear_q4.cu on tcgen05, codes expanded into tensor memory.
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
// Roles: warp 0 loads codes and x by TMA, warp 1 of the first CTA issues the products; then the
// converters (one warpgroup, or two that take turns at the steps), then two warpgroups of drain threads,
// which take half of an accumulator's columns each.
// Tensor memory (512 columns): four steps of expanded codes of 64 columns, then the accumulators.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "sm103.cuh"
#include "step_internal.cuh"

namespace moeslot {
namespace {
using namespace sm103;

typedef __nv_bfloat16 bf16;
constexpr int kSteps = 4;                      // buffers of expanded codes
constexpr int kCodeStage = 128 * 128;          // 128 outputs by 256 codes: two steps
constexpr int kShared = 225 * 1024;

template <int BN_, int G_>
struct Tile {
  static constexpr int BN = BN_, G = G_, P = 128 / G;
  static constexpr int HN = BN < 128 ? BN : 128, HALVES = BN / HN;       // columns of an accumulator
  static constexpr int BUFS = 256 / HN < 4 ? 256 / HN : 4;               // accumulators
  static constexpr int CONVERTERS = BN <= 128 ? 2 : 1;                   // warpgroups
  static constexpr int THREADS = 128 * (1 + CONVERTERS + 2);
  static constexpr int X_PART = HN / 2 * 128;            // this CTA's rows by 64 inputs
  static constexpr int X_STAGE = HALVES * 2 * X_PART;    // [half][64 inputs][rows][128 bytes]
  static constexpr int X_STAGES = BN >= 256 ? 3 : 4;
  static constexpr int CODE_STAGES = BN >= 256 ? 6 : 8;
  static constexpr int BYTES = CODE_STAGES * kCodeStage + X_STAGES * X_STAGE + 1024;
  // registers of a thread at launch and after the split: (1 + CONVERTERS + 2) * launch >= the sum of the shares
  static constexpr int REGS = CONVERTERS == 2 ? 96 : 128, MISC = 56, CONVERT = CONVERTERS == 2 ? 72 : 80;
  static constexpr int DRAIN = CONVERTERS == 2 ? 136 : 184;
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
  __shared__ __align__(8) uint64_t c_full[C::CODE_STAGES], c_empty[C::CODE_STAGES], x_full[C::X_STAGES], x_empty[C::X_STAGES],
      a_full[kSteps], a_empty[kSteps], d_full[C::BUFS], d_empty[C::BUFS], drained;
  __shared__ uint32_t tmem_slot;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t codes = smem_addr(smem), xs = codes + C::CODE_STAGES * kCodeStage;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, rank = (int)pair_rank();
  if (tid == 0) {
    for (int s = 0; s < C::CODE_STAGES; ++s) {
      bar_init(c_full + s, 1);
      bar_init(c_empty + s, 4 * C::CONVERTERS);
    }
    for (int s = 0; s < C::X_STAGES; ++s) {
      bar_init(x_full + s, 2);
      bar_init(x_empty + s, 1);
    }
    for (int s = 0; s < kSteps; ++s) {
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

  const int steps = (a.K + 127) / 128, n_tiles = (a.rows + C::BN - 1) / C::BN, tiles = (a.N + 255) / 256 * n_tiles;
  const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
  bool alive = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {        // bounded; after a timeout nothing waits any more
    if (alive && !bar_wait(b, parity)) {
      alive = false;
      atomicCAS(a.status, 0, MOE_ERR_TIMEOUT);
    }
  };

  if (wid < 4) {
    regs_give<C::MISC>();
    if (wid == 0) {
      // ---------------------------------------------------------------- loads
      uint32_t nc = 0, nx = 0;
      for (int tile = pair; tile < tiles; tile += pairs) {
        const int m0 = tile / n_tiles * 256 + rank * 128, t0 = tile % n_tiles * C::BN + rank * (C::HN / 2);
        for (int s = 0; s < steps; ++s) {
          if ((s & 1) == 0) {
            const int st = nc % C::CODE_STAGES;
            wait(c_empty + st, ((nc / C::CODE_STAGES) & 1) ^ 1);
            __syncwarp();
            if (lane == 0) {
              bar_expect(c_full + st, kCodeStage);
              tma_2d(codes + st * kCodeStage, &mc, c_full + st, s * 64, m0);
            }
            ++nc;
          }
          const int st = nx % C::X_STAGES;
          const uint32_t lead_full = lead_addr(x_full + st);
          wait(x_empty + st, ((nx / C::X_STAGES) & 1) ^ 1);
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) bar_expect(x_full + st, 2 * C::X_STAGE);      // of both CTAs
            else bar_arrive_at(lead_full);
          }
          __syncwarp();
          if (lane < 2 * C::HALVES)
            tma_2d_pair(xs + st * C::X_STAGE + lane * C::X_PART, &mx, lead_full, s * 128 + (lane & 1) * 64, t0 + (lane >> 1) * C::HN);
          ++nx;
        }
      }
      if (!alive) {                                      // bounded: copies in flight land (on the first CTA's barriers,
        const uint64_t t = now_ns();                     // which this one cannot test) before the memory is given up
        while (now_ns() - t < 1000000ull) __nanosleep(1000);
      }
    } else if (wid == 1 && rank == 0) {
      // ----------------------------------------------------------------- MMAs
      const uint32_t lead = elect_lead();
      constexpr uint32_t kDesc = tc_idesc(C::HN, false);
      const uint64_t x_desc = tc_desc<128>(xs);
      uint32_t n = 0, nd = 0;                            // steps, accumulators
      for (int tile = pair; tile < tiles; tile += pairs) {
        for (int s = 0; s < steps; ++s, ++n) {
          const uint32_t ab = n % kSteps, st = n % C::X_STAGES;
          wait(a_full + ab, (n / kSteps) & 1);
          wait(x_full + st, (n / C::X_STAGES) & 1);
#pragma unroll
          for (int p = 0; p < C::P; ++p) {
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h, ++nd) {
              const uint32_t buf = nd % C::BUFS;
              wait(d_empty + buf, ((nd / C::BUFS) & 1) ^ 1);
              __syncwarp();
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < C::G / 16; ++k) {
                const int at = p * (C::G / 16) + k;      // sixteens of the step
                tc_mma_ts(lead, tmem + 256 + buf * C::HN, tmem + ab * 64 + at * 8,
                          x_desc + ((st * C::X_STAGE + (2 * h + (at >> 2)) * C::X_PART + (at & 3) * 32) >> 4), kDesc, k > 0);
              }
              tc_commit(lead, d_full + buf);
            }
          }
          tc_commit(lead, a_empty + ab);
          tc_commit(lead, x_empty + st);
        }
      }
      if (!alive) {                                      // bounded: products in flight end before the memory is given up
        tc_commit(lead, &drained);
        bar_wait(&drained, 0);
      }
    }
  } else if (wid < 4 + 4 * C::CONVERTERS) {
    regs_give<C::CONVERT>();
    // ------------------------------------------------------------- expansion
    const int group = (wid >> 2) - 1, row = (wid & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wid & 3) << 21);
    uint32_t nc = 0, n0 = 0;                             // stages of codes; steps of the tiles before
    for (int tile = pair; tile < tiles; tile += pairs, n0 += steps) {
      for (int s0 = 0; s0 < steps; s0 += 2, ++nc) {
        const int st = nc % C::CODE_STAGES;
        wait(c_full + st, (nc / C::CODE_STAGES) & 1);
        __syncwarp();
#pragma unroll 1
        for (int half = C::CONVERTERS == 2 ? group : 0; half < (C::CONVERTERS == 2 ? group + 1 : 2); ++half) {
          if (s0 + half >= steps) break;
          const uint32_t n = n0 + s0 + half, ab = n % kSteps;
          const uint8_t* src = smem + st * kCodeStage + row * 128;
          wait(a_empty + ab, ((n / kSteps) & 1) ^ 1);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 2; ++q) {                  // 64 codes at a time
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
          if (lane == 0) bar_arrive_at(lead_addr(a_full + ab));
        }
        __syncwarp();
        if (lane == 0) bar_arrive(c_empty + st);
      }
    }
  } else {
    regs_take<C::DRAIN>();
    // ----------------------------------------------- scaling, sums and output
    constexpr int COLS = C::HN / 2, PIECE = COLS < 32 ? COLS : 32;       // of an accumulator, of a load
    const int side = (wid - 4 - 4 * C::CONVERTERS) >> 2, row = (wid & 3) * 32 + lane;
    const uint32_t d_addr = tmem + ((uint32_t)(wid & 3) << 21) + 256 + side * COLS;
    uint32_t nd = 0;
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int n = tile / n_tiles * 256 + rank * 128 + row, t0 = tile % n_tiles * C::BN + side * COLS;
      const int64_t at = (int64_t)min(n, a.N - 1) * a.groups;
      auto scale = [&](int g) {
        if (g >= a.groups) return 0.f;
        return a.scale_f32 ? static_cast<const float*>(a.scales)[at + g] : __bfloat162float(static_cast<const bf16*>(a.scales)[at + g]);
      };
      float acc[C::HALVES][COLS];
#pragma unroll
      for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
        for (int j = 0; j < COLS; ++j) acc[h][j] = 0.f;
      constexpr int AHEAD = 4;                           // scales on their way
      float next[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) next[k] = scale(k);
      const int groups = steps * C::P;                   // those past the end of K have no scale and zeros of x
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += AHEAD) {
        float now[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          now[k] = next[k];
          next[k] = scale(g0 + AHEAD + k);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          if (g0 + k >= groups) break;
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h, ++nd) {
            const uint32_t buf = nd % C::BUFS;
            wait(d_full + buf, (nd / C::BUFS) & 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int j0 = 0; j0 < COLS; j0 += PIECE) {
              float d[PIECE];
              tmem_load<PIECE>(d_addr + buf * C::HN + j0, d);
#pragma unroll
              for (int j = 0; j < PIECE; ++j) acc[h][j0 + j] = fmaf(now[k], d[j], acc[h][j0 + j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_at(lead_addr(d_empty + buf));
          }
        }
      }
      if (n < a.N) {
        const float bias = a.bias ? __bfloat162float(static_cast<const bf16*>(a.bias)[n]) : 0.f;
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
          for (int j = 0; j < COLS; ++j) {
            const int t = t0 + h * C::HN + j;
            if (t >= a.rows) break;
            const float v = fmaf(acc[h][j], 64.f, bias);
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

bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows, int64_t pitch, int box_cols,
            int box_rows) {
  static const auto encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C>
cudaError_t run(const LinearArgs& a, cudaStream_t s) {
  CUtensorMap mc, mx;
  if (!map_2d(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.K / 2, a.N, a.K / 2, 128, 128) ||
      !map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.rows, a.x_stride * 2, 64, C::HN / 2))
    return cudaErrorInvalidValue;
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
  const int64_t tiles = (int64_t)((a.N + 255) / 256) * ((a.rows + C::BN - 1) / C::BN), pairs = sm_count() / 2;
  return sm103::launch(linear_q4_tiles_kernel<C>, 2 * (int)(tiles < pairs ? tiles : pairs), C::THREADS, C::BYTES, s, mc, mx, a);
}

template <int G>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  if (a.rows <= 32) return run<Tile<32, G>>(a, s);
  if (a.rows <= 64) return run<Tile<64, G>>(a, s);
  if (a.rows <= 128) return run<Tile<128, G>>(a, s);
  return run<Tile<256, G>>(a, s);
}

}  // namespace

cudaError_t launch_linear_q4_tiles(const LinearArgs& a, int group, cudaStream_t s) {
  return group == 32 ? pick<32>(a, s) : group == 64 ? pick<64>(a, s) : pick<128>(a, s);
}

}  // namespace moeslot
