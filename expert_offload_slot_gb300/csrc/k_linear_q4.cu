// moe_linear_q4: out[t, n] = bias[n] + sum_g scale[n, g] sum_{k in group g} code[n, k] x[t, k],
// 4-bit codes in -8..7 with one scale for each group of 32, 64 or 128 inputs.
//
// Row kernel.  A warp takes tiles of 16 outputs by up to 32 columns of x on mma.sync (M the
// outputs, N the columns).  A code is exact in bf16, so products and the sums of a group
// are the tensor core's, exact up to fp32 sums; a group's sum is scaled in fp32.  An fp32
// x is cut into three bf16 numbers that add up to it (8 bits of its 24 each) and takes
// three columns.
//
// The order of k inside a group is free as long as codes and x agree: lane (g, t) of the
// warp takes for row g (and g + 8) the quarter t of each group, so that it reads its codes
// with one load and no exchange.  The eight codes of a 32-bit word turn into four
// bf16 pairs (k, k + 4) by one and-xor each: nibble ^ 8 below the bits of 128.0 is
// 136 + code, exact, less 136 is the code.  x lies in shared memory in the same order, 16
// bytes for each word.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "sm103.cuh"
#include "step_internal.cuh"

namespace moeslot {
namespace {

typedef __nv_bfloat16 bf16;
constexpr int NT = 512, NWARP = NT / 32;
constexpr int kTile = 16;            // outputs of a warp's tile
constexpr int kBlock = 128;          // inputs of a step
constexpr int kColumn = 20;          // floats between the columns of a tile in shared memory: no bank conflicts
constexpr int kShared = 220 * 1024;  // dynamic shared memory of a CTA

// Codes of a word as four pairs (k, k + 4) of bf16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) {
  const __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));   // 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) ^ 0x43084308u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), top);
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// x as three bf16 numbers by cutting off bits: the sum is x.  Nothing is left of an infinity or a NaN.
__device__ __forceinline__ float part_of(float x, int part) {
  const float h = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  if (part == 0) return (__float_as_uint(x) & 0x7fffffffu) > 0x7f800000u ? __uint_as_float(0x7fc00000u) : h;
  if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) return 0.f;
  const float rest = x - h, m = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
  return part == 1 ? m : rest - m;
}

// Eight inputs k0 .. k0 + 7 of a column, in the order of widen()'s pairs.
__device__ __forceinline__ uint4 column8(const LinearArgs& a, int64_t row, int part, int k0, bool wide) {
  uint32_t w[4];
  if (a.x_f32) {
    const float* p = static_cast<const float*>(a.x) + row * a.x_stride + k0;
    float v[8];
    if (wide) {
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __float_as_uint(part_of(v[i], part)) >> 16 | (__float_as_uint(part_of(v[i + 4], part)) & 0xffff0000u);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.x) + row * a.x_stride + k0;
    uint16_t v[8];
    if (wide) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i] | (uint32_t)v[i + 4] << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }

// What a warp reads for one step of a tile: rows g and g + 8.
template <int P>
struct Step {
  uint32_t code[2][4];
  float scale[2][P];
};

template <typename S, int G>
__device__ __forceinline__ void fetch(const LinearArgs& a, int tile, int block, Step<kBlock / G>& st) {
  constexpr int P = kBlock / G, WORDS = G / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t n = min(tile * kTile + g + 8 * i, a.N - 1);
    const uint8_t* row = a.codes + n * (a.K / 2);
    const S* scales = static_cast<const S*>(a.scales) + n * a.groups;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int k = block * kBlock + p * G + t * (G / 4);
      uint32_t* c = st.code[i] + p * WORDS;
      if (k < a.K) {
        if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(c) = __ldcs(reinterpret_cast<const uint4*>(row + k / 2));
        else if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(c) = __ldcs(reinterpret_cast<const uint2*>(row + k / 2));
        else *c = __ldcs(reinterpret_cast<const uint32_t*>(row + k / 2));
      } else {
#pragma unroll
        for (int j = 0; j < WORDS; ++j) c[j] = 0;
      }
      const int group = block * P + p;
      st.scale[i][p] = group < a.groups ? to_float(scales[group]) : 0.f;
    }
  }
}

// Grid: for each pass over `pass_rows` rows of x, the CTAs that share the tiles.
// Shared memory: x of the pass, [block][word][column][t][8], then the warps' tiles.
template <typename S, int G, int N8>
__global__ void __launch_bounds__(NT, 1) linear_q4_rows_kernel(const LinearArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int P = kBlock / G, WORDS = G / 32, COLS = 8 * N8, U = 2;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int blocks = (a.K + kBlock - 1) / kBlock, chunk = min(a.chunk, blocks);
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float* red = reinterpret_cast<float*>(smem + (size_t)chunk * 4 * COLS * 64);
  const int pass = blockIdx.x / a.ctas, cta = blockIdx.x - pass * a.ctas;
  const int row0 = pass * a.pass_rows, rows = min(a.pass_rows, a.rows - row0);
  const int splits = 1 << a.split_log2, team = wid >> a.split_log2, part = wid & (splits - 1), teams = NWARP >> a.split_log2;
  const int tiles = (a.N + kTile - 1) / kTile;
  const bool whole = chunk == blocks;
  const int esize = a.x_f32 ? 4 : 2, parts = a.x_f32 ? 3 : 1;
  const bool wide = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.x_stride * esize % 16 == 0;
  sm103::grid_wait();

  auto stage = [&](int b0) {                   // blocks b0 .. of x; zeros past its end and its rows
    const int groups8 = chunk * (kBlock / 8);
    for (int u = tid; u < groups8 * COLS; u += NT) {
      const int col = u / groups8, q = u - col * groups8, k0 = b0 * kBlock + q * 8;
      const int in_block = q * 8 % kBlock, p = in_block / G, in_group = in_block % G;
      const int t = in_group / (G / 4), word = p * WORDS + in_group % (G / 4) / 8;
      const int row = a.x_f32 ? col / 3 : col;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows && col < rows * parts && k0 < a.K) v = column8(a, row0 + row, col - row * parts, k0, wide);
      xs[((q / (kBlock / 8) * 4 + word) * COLS + col) * 4 + t] = v;
    }
  };

  const int stride = a.ctas * teams, first = cta * teams + team;
  float acc[N8][4];
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < N8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  };
  auto work = [&](const Step<P>& st, int block) {       // block: within the staged ones
    const uint4* xb = xs + (size_t)block * 4 * COLS * 4 + (lane >> 2) * 4 + (lane & 3);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float sum[N8][4];
#pragma unroll
      for (int j = 0; j < N8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[j][i] = 0.f;
#pragma unroll
      for (int w = p * WORDS; w < (p + 1) * WORDS; ++w) {
        uint32_t lo[4], hi[4];
        widen(st.code[0][w], lo);
        widen(st.code[1][w], hi);
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          const uint4 b = xb[(w * COLS + 8 * j) * 4];
          sm103::mma16816(sum[j], a0, b.x, b.y);
          sm103::mma16816(sum[j], a1, b.z, b.w);
        }
      }
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        acc[j][0] = fmaf(st.scale[0][p], sum[j][0], acc[j][0]);
        acc[j][1] = fmaf(st.scale[0][p], sum[j][1], acc[j][1]);
        acc[j][2] = fmaf(st.scale[1][p], sum[j][2], acc[j][2]);
        acc[j][3] = fmaf(st.scale[1][p], sum[j][3], acc[j][3]);
      }
    }
  };
  int turn = 0;
  auto finish = [&](int tile) {                // the team's parts joined, in their order, and written
    float* mine = red + (size_t)(turn * NWARP + wid) * COLS * kColumn;
    const float* base = red + (size_t)(turn * NWARP + team * splits) * COLS * kColumn;
    turn ^= 1;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < N8; ++j) {
      mine[(8 * j + 2 * t) * kColumn + g] = acc[j][0];
      mine[(8 * j + 2 * t + 1) * kColumn + g] = acc[j][1];
      mine[(8 * j + 2 * t) * kColumn + g + 8] = acc[j][2];
      mine[(8 * j + 2 * t + 1) * kColumn + g + 8] = acc[j][3];
    }
    if (splits == 1) __syncwarp();
    else sm103::named_sync(1 + team, splits * 32);
    for (int u = part * 32 + lane; u < rows * kTile; u += splits * 32) {
      const int row = u / kTile, i = u % kTile, n = tile * kTile + i;
      if (n >= a.N) continue;
      float v = 0.f;
      for (int s = 0; s < splits; ++s) {
        const float* from = base + (size_t)s * COLS * kColumn + i;
        if (parts == 1) v += from[row * kColumn];
        else v += from[3 * row * kColumn] + (from[(3 * row + 1) * kColumn] + from[(3 * row + 2) * kColumn]);
      }
      if (a.bias) v += a.x_f32 ? static_cast<const float*>(a.bias)[n] : to_float(static_cast<const bf16*>(a.bias)[n]);
      const int64_t at = (row0 + row) * a.out_stride + n;
      if (a.out_f32) static_cast<float*>(a.out)[at] = v;
      else static_cast<bf16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
    if (splits == 1) __syncwarp();
  };

  if (whole) {
    // the steps of all this warp's tiles in one run, U of them on their way
    Step<P> st[U];
    const int per = (blocks - part + splits - 1) / splits;               // steps of a tile (splits <= blocks)
    const int mine = first < tiles ? (tiles - first + stride - 1) / stride : 0;
    int ft = first, fb = part;
    auto ahead = [&](Step<P>& s) {
      if (ft < tiles) fetch<S, G>(a, ft, fb, s);
      fb += splits;
      if (fb >= blocks) {
        fb = part;
        ft += stride;
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) ahead(st[u]);
    stage(0);
    __syncthreads();
    int tile = first, block = part;
    clear();
    const int total = mine * per;
    for (int i = 0; i < total; i += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u < total) {
          work(st[u], block);
          ahead(st[u]);
          block += splits;
          if (block >= blocks) {
            finish(tile);
            clear();
            block = part;
            tile += stride;
          }
        }
      }
    }
  } else {                                     // x in chunks: all warps of the CTA go through them together
    const int rounds = (tiles + stride - 1) / stride;
    for (int i = 0; i < rounds; ++i) {
      const int tile = first + i * stride;
      clear();
      for (int b0 = 0; b0 < blocks; b0 += chunk) {
        __syncthreads();
        stage(b0);
        __syncthreads();
        for (int b = b0 + part; b < min(b0 + chunk, blocks) && tile < tiles; b += splits) {
          Step<P> st;
          fetch<S, G>(a, tile, b, st);
          work(st, b - b0);
        }
      }
      if (tile < tiles) finish(tile);
    }
  }
}

template <typename S, int G, int N8>
cudaError_t run(LinearArgs a, cudaStream_t s) {
  constexpr int cols = 8 * N8;
  const int sms = sm_count(), blocks = (a.K + kBlock - 1) / kBlock, tiles = (a.N + kTile - 1) / kTile;
  const size_t joint = (size_t)2 * NWARP * cols * kColumn * sizeof(float), block_bytes = (size_t)4 * cols * 64;
  const int fit = (int)((kShared - joint) / block_bytes);
  a.chunk = blocks < fit ? blocks : fit;
  a.pass_rows = a.x_f32 ? cols / 3 : cols;
  const int passes = (a.rows + a.pass_rows - 1) / a.pass_rows;
  // warps that share a tile's inputs: those that need the fewest steps, a tile's end counted as one
  int64_t least = 0;
  a.split_log2 = 0;
  const int ctas = passes < sms ? sms / passes : 1;
  for (int log = 0; log <= 4 && (1 << log) <= a.chunk; ++log) {
    const int64_t at_once = (int64_t)ctas * (NWARP >> log), rounds = (tiles + at_once - 1) / at_once;
    const int64_t cost = rounds * ((blocks + (1 << log) - 1) / (1 << log) + 1);
    if (log == 0 || cost < least) {
      least = cost;
      a.split_log2 = log;
    }
  }
  const int teams = NWARP >> a.split_log2, need = (tiles + teams - 1) / teams;
  static std::atomic<uint64_t> ready{0};       // devices whose kernel has the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(linear_q4_rows_kernel<S, G, N8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  a.ctas = need < ctas ? need : ctas;
  cfg.gridDim = dim3((unsigned)a.ctas * passes);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = joint + a.chunk * block_bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, linear_q4_rows_kernel<S, G, N8>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename S, int G>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  const int64_t cols = (int64_t)a.rows * (a.x_f32 ? 3 : 1);
  if (cols <= 8) return run<S, G, 1>(a, s);
  if (cols <= 16) return run<S, G, 2>(a, s);
  return run<S, G, 4>(a, s);
}

template <typename S>
cudaError_t pick(const LinearArgs& a, int group, cudaStream_t s) {
  return group == 32 ? pick<S, 32>(a, s) : group == 64 ? pick<S, 64>(a, s) : pick<S, 128>(a, s);
}

}  // namespace

cudaError_t launch_linear_q4(const LinearArgs& a, int group, int scale_dtype, cudaStream_t s) {
  return scale_dtype == MOE_F32 ? pick<float>(a, group, s) : pick<bf16>(a, group, s);
}

}  // namespace moeslot
