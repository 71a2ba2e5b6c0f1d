// moe_linear_q4: out[t, n] = bias[n] + sum_g scale[n, g] sum_{k in group g} code[n, k] x[t, k],
// 4-bit codes in -8..7 with one scale for each group of 32, 64 or 128 inputs.
//
// Row kernel, for few columns of x (launch_linear_q4 says when; linear_q4_tiles.cuh has the others).
// The codes are all there is to read, so the kernel is a stream of them: a CTA takes tiles
// of 16 to 64 outputs, four warps copy their codes (cp.async, a row of a slice of K each)
// into a ring in shared memory, two more bring the scales, and 16 warps share the slice, a
// block of 128 inputs each (one group of warps for all rows, or two), on mma.sync with M the
// outputs and N the columns of x.  A code is exact in bf16, so products and the sums of a
// group are the tensor core's, exact up to fp32 sums; a group's sum is scaled in fp32.  At a
// tile's end the warps' parts are added up in their order.  An fp32 x is cut into three bf16
// numbers that add up to it (8 bits of its 24 each) and takes three columns.
//
// What bounds it: for small matrices the launch and the latencies of x, codes and joins one
// after another (one row, 2048 x 5120, 5.2 MB of codes: 6.0 us); for large ones the instructions that
// expand a code (11 for a word of eight, most on a pipe of half rate) and feed the products, 66 us for
// 2048 x 131072 where HBM needs 20: without the products 50, without the copies 38.  Registers filled by plain loads
// instead of the ring took 59 there but 11.3 instead of 9.5 us for one row of 4096 x 6144; bulk copies instead of cp.async 71.
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
constexpr int NWARP = 16, NT = NWARP * 32;     // consumers
constexpr int kCodeWarps = 4, kScaleWarps = 2, kThreads = NT + 32 * (kCodeWarps + kScaleWarps);
constexpr int kBlock = 128;                    // inputs of a warp's part of a slice
constexpr int kRing = 8;                       // stages at most
constexpr int kShared = 225 * 1024;            // dynamic shared memory of a CTA
__device__ int32_t g_status;                   // set where a wait ran out

// Codes of a word as four pairs (k, k + 4) of bf16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) {
  const __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));   // 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u;                                // ((w >> 4 i) & 0x000f000f) ^ 0x43084308
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(u) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43084308u));
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), top);
    p[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
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
      w[i] = __float_as_uint(bf16_part(v[i], part)) >> 16 | (__float_as_uint(bf16_part(v[i + 4], part)) & 0xffff0000u);
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

// Shapes of a row kernel: N8 * 8 columns of x; a warp has 16 * MT outputs; RG groups of warps have outputs of
// their own, the 16 / RG warps of a group the blocks of a slice.
template <int N8_, int MT_, int RG_, int G_>
struct Shape {
  static constexpr int N8 = N8_, MT = MT_, RG = RG_, G = G_;
  static constexpr int COLS = 8 * N8, ROWS = 16 * MT * RG, PARTS = NWARP / RG, P = kBlock / G, WORDS = G / 32;
  static constexpr int COLUMN = 16 * MT + 4;   // floats between a tile's columns in shared memory: no bank conflicts
  static constexpr int RED = NWARP * COLS * COLUMN * 4;
  static constexpr int X_BLOCK = 4 * COLS * 64;          // bytes of a block of x
};

// Grid: for each pass over `pass_rows` rows of x, the CTAs that share the tiles.
// Shared memory: x [block][word][column][t][8], the warps' parts, then the ring: codes, `pitch` bytes a row, and
// scales, `scale_pitch` floats a row.  Rows are apart by half a group's bytes more than a multiple of 128: no bank
// conflicts among the eight rows that a load instruction reads.
template <typename H>
__global__ void __launch_bounds__(kThreads, 1) linear_q4_rows_kernel(const LinearArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kRing], empty[kRing];
  constexpr int G = H::G, P = H::P, WORDS = H::WORDS, COLS = H::COLS, N8 = H::N8, MT = H::MT;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int blocks = (a.K + kBlock - 1) / kBlock;
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float* red = reinterpret_cast<float*>(smem + (size_t)a.chunk * a.slice * H::X_BLOCK);
  uint8_t* ring = reinterpret_cast<uint8_t*>(red) + H::RED;
  const int stage_bytes = H::ROWS * (a.pitch + a.scale_pitch * 4);
  const int pass = blockIdx.x / a.ctas, cta = blockIdx.x - pass * a.ctas;
  const int row0 = pass * a.pass_rows, rows = min(a.pass_rows, a.rows - row0);
  const int tiles = (a.N + H::ROWS - 1) / H::ROWS, mine = (tiles - cta + a.ctas - 1) / a.ctas;
  const int slices = (blocks + a.slice - 1) / a.slice;
  const int64_t steps = (int64_t)mine * slices;
  if (tid == 0) {
    for (int s = 0; s < a.depth; ++s) {
      sm103::bar_init(full + s, 32 * kCodeWarps + 1);
      sm103::bar_init(empty + s, NWARP);
    }
    sm103::bar_init_done();
  }
  __syncthreads();
  sm103::grid_wait();

  if (wid >= NWARP && wid < NWARP + kCodeWarps) {        // ---------------------- the codes
    int st = 0, slice = 0, tile = cta;
    uint32_t phase = 0;
    for (int64_t i = 0; i < steps; ++i) {
      if (i >= a.depth && !sm103::bar_wait_warp(empty + st, phase ^ 1)) {
        if (lane == 0) atomicCAS(&g_status, 0, MOE_ERR_TIMEOUT);
        break;
      }
      const int at = slice * a.slice * (kBlock / 2), bytes = min(a.slice * (kBlock / 2), a.K / 2 - at);
      const int n0 = tile * H::ROWS, n = min(H::ROWS, a.N - n0);
      const uint32_t dst = sm103::smem_addr(ring) + st * stage_bytes;
      const uint8_t* src = a.codes + (int64_t)n0 * (a.K / 2) + at;
      for (int r = wid - NWARP; r < n; r += kCodeWarps)
        for (int c = lane * 16; c < bytes; c += 512) sm103::cp_async16(dst + r * a.pitch + c, src + (int64_t)r * (a.K / 2) + c, 16);
      sm103::cp_async_arrive(full + st);
      if (++slice == slices) {
        slice = 0;
        tile += a.ctas;
      }
      if (++st == a.depth) {
        st = 0;
        phase ^= 1;
      }
    }
    sm103::cp_async_wait();
    return;
  }
  if (wid >= NWARP) {                          // ------------------------------- the scales, every other stage
    const int per = a.slice * P;               // of a row in a stage
    const uint32_t mul = 0xffffffffu / per + 1;          // k / per for k below 2^16 and per above 1
    auto row_of = [&](uint32_t k) { return per == 1 ? k : __umulhi(k, mul); };
    int slice = (wid - NWARP - kCodeWarps) % slices, tile = cta + (wid - NWARP - kCodeWarps) / slices * a.ctas;
    for (int64_t i = wid - NWARP - kCodeWarps; i < steps; i += kScaleWarps) {
      const int st = (int)(i % a.depth);
      const uint32_t phase = (uint32_t)(i / a.depth) & 1;
      if (i >= a.depth && !sm103::bar_wait_warp(empty + st, phase ^ 1)) return;
      float* dst = reinterpret_cast<float*>(ring + st * stage_bytes + H::ROWS * a.pitch);
      const int n0 = tile * H::ROWS, g0 = slice * per, groups = min(per, a.groups - g0);
      for (int k0 = lane; k0 < H::ROWS * per; k0 += 32 * 16) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t k = k0 + 32 * j, r = row_of(k), g = k - r * per;
          v[j] = 0.f;
          if (k < H::ROWS * per && n0 + (int)r < a.N && (int)g < groups) {
            const int64_t at = (int64_t)(n0 + r) * a.groups + g0 + g;
            v[j] = a.scale_f32 ? static_cast<const float*>(a.scales)[at] : __bfloat162float(static_cast<const bf16*>(a.scales)[at]);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t k = k0 + 32 * j, r = row_of(k), g = k - r * per;
          if (k < H::ROWS * per) dst[r * a.scale_pitch + g] = v[j];
        }
      }
      __syncwarp();
      if (lane == 0) sm103::bar_arrive(full + st);
      slice += kScaleWarps;
      while (slice >= slices) {
        slice -= slices;
        tile += a.ctas;
      }
    }
    return;
  }

  // ------------------------------------------------------------------------------ the products
  const int g = lane >> 2, t = lane & 3, group = wid % H::RG, part = wid / H::RG;
  const int esize = a.x_f32 ? 4 : 2, parts = a.x_f32 ? 3 : 1;
  const bool wide = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.x_stride * esize % 16 == 0;
  auto stage_x = [&](int b0) {                 // `chunk` slices of x from block b0; zeros past its end and its rows
    const int eights = a.chunk * a.slice * (kBlock / 8);
    for (int u = tid; u < eights * COLS; u += NT) {
      const int col = u / eights, q = u - col * eights, row = a.x_f32 ? col / 3 : col;
      const int k0 = b0 * kBlock + q * 8, in_block = q * 8 % kBlock, p = in_block / G, in_group = in_block % G;
      const int tx = in_group / (G / 4), word = p * WORDS + in_group % (G / 4) / 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows && k0 < a.K) v = column8(a, row0 + row, col - row * parts, k0, wide);
      xs[((q / (kBlock / 8) * 4 + word) * COLS + col) * 4 + tx] = v;
    }
  };
  float acc[MT][N8][4];
  int st = 0, slice = 0, tile = cta;
  uint32_t phase = 0;
  bool alive = true;                           // without it the others' barriers are still met, and nothing waited for
  for (int64_t i = 0; i < steps; ++i) {
    const int held = slice % a.chunk;          // slice of x within the ones in shared memory
    if (held == 0 && (i == 0 || a.chunk < slices)) {
      if (i > 0) sm103::named_sync(1, NT);     // all are through with the last ones
      stage_x(slice * a.slice);
      sm103::named_sync(1, NT);
    }
    if (slice == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < N8; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][j][k] = 0.f;
    }
    if (alive && !(alive = sm103::bar_wait_warp(full + st, phase)) && lane == 0) atomicCAS(&g_status, 0, MOE_ERR_TIMEOUT);
    const int block = slice * a.slice + part;
    if (part < a.slice && block < blocks) {
      const uint8_t* codes = ring + st * stage_bytes + (group * 16 * MT + g) * a.pitch + part * (kBlock / 2) + t * (G / 8);
      const float* scales = reinterpret_cast<const float*>(ring + st * stage_bytes + H::ROWS * a.pitch) +
                            (group * 16 * MT + g) * a.scale_pitch + part * P;
      const uint4* xb = xs + (size_t)(held * a.slice + part) * 4 * COLS * 4 + lane;
      // past the end of K x is zero and any code finite
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint32_t code[MT][2][WORDS];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* c = codes + (m * 16 + h * 8) * a.pitch + p * (G / 2);
            if constexpr (WORDS == 4) {
              const uint4 u = *reinterpret_cast<const uint4*>(c);
              code[m][h][0] = u.x; code[m][h][1] = u.y; code[m][h][2] = u.z; code[m][h][3] = u.w;
            } else if constexpr (WORDS == 2) {
              const uint2 u = *reinterpret_cast<const uint2*>(c);
              code[m][h][0] = u.x; code[m][h][1] = u.y;
            } else {
              code[m][h][0] = *reinterpret_cast<const uint32_t*>(c);
            }
          }
        float sum[MT][N8][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < N8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[m][j][k] = 0.f;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          uint4 b[N8];
#pragma unroll
          for (int j = 0; j < N8; ++j) b[j] = xb[((p * WORDS + w) * COLS + 8 * j) * 4];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t lo[4], hi[4];
            widen(code[m][0][w], lo);
            widen(code[m][1][w], hi);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
            for (int j = 0; j < N8; ++j) {
              sm103::mma16816(sum[m][j], a0, b[j].x, b[j].y);
              sm103::mma16816(sum[m][j], a1, b[j].z, b[j].w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float s0 = scales[m * 16 * a.scale_pitch + p], s1 = scales[(m * 16 + 8) * a.scale_pitch + p];
#pragma unroll
          for (int j = 0; j < N8; ++j) {
            acc[m][j][0] = fmaf(s0, sum[m][j][0], acc[m][j][0]);
            acc[m][j][1] = fmaf(s0, sum[m][j][1], acc[m][j][1]);
            acc[m][j][2] = fmaf(s1, sum[m][j][2], acc[m][j][2]);
            acc[m][j][3] = fmaf(s1, sum[m][j][3], acc[m][j][3]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) sm103::bar_arrive(empty + st);
    if (++st == a.depth) {
      st = 0;
      phase ^= 1;
    }
    if (++slice < slices) continue;
    // ---------------------------------------------------- the parts added up, in their order
    slice = 0;
    sm103::named_sync(1, NT);                  // the last tile's have been read
    float* to = red + (size_t)wid * COLS * H::COLUMN + g;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        to[(8 * j + 2 * t) * H::COLUMN + m * 16] = acc[m][j][0];
        to[(8 * j + 2 * t + 1) * H::COLUMN + m * 16] = acc[m][j][1];
        to[(8 * j + 2 * t) * H::COLUMN + m * 16 + 8] = acc[m][j][2];
        to[(8 * j + 2 * t + 1) * H::COLUMN + m * 16 + 8] = acc[m][j][3];
      }
    sm103::named_sync(1, NT);
    const int used = min(H::PARTS, min(a.slice, blocks));
    for (int u = tid; u < rows * H::ROWS; u += NT) {
      const int row = u / H::ROWS, o = u % H::ROWS, n = tile * H::ROWS + o;
      if (n >= a.N) continue;
      const float* from = red + (size_t)(o / (16 * MT)) * COLS * H::COLUMN + o % (16 * MT) + (size_t)row * parts * H::COLUMN;
      float v = 0.f;
      for (int s = 0; s < used; ++s, from += H::RG * COLS * H::COLUMN)
        v += parts == 1 ? from[0] : from[0] + (from[H::COLUMN] + from[2 * H::COLUMN]);
      if (a.bias) v += a.x_f32 ? static_cast<const float*>(a.bias)[n] : __bfloat162float(static_cast<const bf16*>(a.bias)[n]);
      const int64_t at = (row0 + row) * a.out_stride + n;
      if (a.out_f32) static_cast<float*>(a.out)[at] = v;
      else static_cast<bf16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
    tile += a.ctas;
  }
}

template <typename H>
cudaError_t run(LinearArgs a, cudaStream_t s) {
  const int sms = sm_count(), blocks = (a.K + kBlock - 1) / kBlock, tiles = (a.N + H::ROWS - 1) / H::ROWS;
  a.pass_rows = a.x_f32 ? H::COLS / 3 : H::COLS;
  const int passes = (a.rows + a.pass_rows - 1) / a.pass_rows;
  const int slices = (blocks + H::PARTS - 1) / H::PARTS;
  a.slice = (blocks + slices - 1) / slices;
  a.pitch = (a.slice * (kBlock / 2) + 127) / 128 * 128 + H::G / 2;
  a.scale_pitch = a.slice * H::P | 1;
  const int stage = H::ROWS * (a.pitch + a.scale_pitch * 4);
  // all of x where three stages still fit beside it, else as many slices as do
  const int room = kShared - H::RED, x_slice = a.slice * H::X_BLOCK;
  a.chunk = (blocks + a.slice - 1) / a.slice;
  while (a.chunk > 1 && a.chunk * x_slice + 3 * stage > room) --a.chunk;
  a.depth = (room - a.chunk * x_slice) / stage;
  if (a.depth > kRing) a.depth = kRing;
  const size_t bytes = H::RED + (size_t)a.chunk * x_slice + (size_t)a.depth * stage;
  const int share = passes < sms ? sms / passes : 1;
  a.ctas = tiles < share ? tiles : share;
  static std::atomic<uint64_t> ready{0};       // devices whose kernel has the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(linear_q4_rows_kernel<H>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return sm103::launch(linear_q4_rows_kernel<H>, a.ctas * passes, kThreads, bytes, s, a);
}

template <int G>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  const int64_t cols = (int64_t)a.rows * (a.x_f32 ? 3 : 1);
  const bool large = a.N >= 64 * 2 * sm_count();
  if (cols <= 8) return large ? run<Shape<1, 2, 2, G>>(a, s) : run<Shape<1, 1, 1, G>>(a, s);
  if (cols <= 16) return large ? run<Shape<2, 2, 2, G>>(a, s) : run<Shape<2, 1, 1, G>>(a, s);
  return large ? run<Shape<4, 1, 2, G>>(a, s) : run<Shape<4, 1, 1, G>>(a, s);
}

}  // namespace

namespace {

// Which kernel for up to 16 rows of bf16: the row kernel's time goes by the bytes of codes (us a MB: 0.56 up to 8
// rows, 1 up to 16, twice that where x does not fit shared memory), the tile kernel's by steps of 128 inputs and rounds of its
// pairs of CTAs, 0.47 us each; both begin with some 2.5 us.  Measured, row and tile kernel in us: one row, 2048 x 5120 6.0, 10.0;
// 4096 x 6144 9.5, 16.3; 8192 x 8192 20, 30; 4096 x 16000 18.1, 17.5; 2048 x 131072 66, 48.  12 rows, 4096 x 6144 16.1, 16.6;
// 2048 x 10000 12.1, 10.8; 8192 x 8192 68, 31.  More rows have the tile kernel: 32 rows, 4096 x 6144 57, 17.
bool rows_are_faster(const LinearArgs& a) {
  if (a.rows > 16) return false;
  const int64_t pairs = sm_count() / 2, blocks = (a.K + kBlock - 1) / kBlock, cols = a.rows <= 8 ? 8 : 16;
  const bool fits = blocks * 4 * cols * 64 <= 150 * 1024;
  const int64_t rows_ns = (int64_t)a.N * (a.K / 2) * (a.rows <= 8 ? 56 : 100) * (fits ? 1 : 2) / 100000;
  const int64_t tiles_ns = 470 * blocks * (((a.N + 255) / 256 + pairs - 1) / pairs);
  return rows_ns <= tiles_ns;
}

}  // namespace

cudaError_t linear_q4_rows_status(int32_t* st) { return take_status(g_status, st); }

cudaError_t launch_linear_q4(const LinearArgs& a, int group, cudaStream_t s) {
  const bool tiles = a.K >= 256, aligned = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.x_stride % 8 == 0;
  if (tiles && !a.x_f32 && aligned && !rows_are_faster(a)) return launch_linear_q4_tiles(a, group, s);
  if (tiles && (a.x_f32 ? a.rows > 5 : a.rows > 32 && !aligned)) return launch_linear_q4_split(a, group, s);
  return group == 32 ? pick<32>(a, s) : group == 64 ? pick<64>(a, s) : pick<128>(a, s);
}

}  // namespace moeslot
