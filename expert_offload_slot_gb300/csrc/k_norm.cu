// moe_residual_norm: a block's output joined into the residual stream, with the
// norms on either side of it.
//
//   n  = x / sqrt(mean x^2 + eps) * (offset + post)      (x itself without post)
//   r' = r + scale * act(gate) * n                       (r itself without x)
//   y  = r' / sqrt(mean r'^2 + eps) * (offset + pre)
//
// A row stays in the registers of its threads from the first load to the last
// store, so each input is read once; everything between is fp32, and r' goes
// into its norm unrounded.
//
// What bounds it: HBM for many rows (8192 rows of 4096: bf16 44 us, 6.1 TB/s or 90 % of a copy's rate; with an
// fp32 stream and both norms 71 us, 5.7 TB/s), once the next row's loads are on their way while this one's sums go
// through the barriers (without that 66 and 85 us); the launch for few (one row of 2048: 1.6 us).  Widths or rows off
// 16-byte boundaries go element by element: 777 rows of 1537 fp32, 9.5 us for 19 MB.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm103.cuh"
#include "step_internal.cuh"

namespace moeslot {
namespace {

typedef __nv_bfloat16 bf16;

// W consecutive elements as they lie in memory, and as numbers: 8 (16-byte loads) or one.
template <typename T, int W>
struct Raw {
  T v;
  __device__ __forceinline__ void get(const T* p) { v = *p; }
  __device__ __forceinline__ void to(float (&x)[1]) const { x[0] = (float)v; }
};
template <>
struct Raw<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void get(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void to(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <>
struct Raw<bf16, 8> {
  uint4 u;
  __device__ __forceinline__ void get(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void to(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
template <int W>
__device__ __forceinline__ void store(float* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}
template <int W>
__device__ __forceinline__ void store(bf16* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(sm103::pack_bf16(v[0], v[1]), sm103::pack_bf16(v[2], v[3]),
                                              sm103::pack_bf16(v[4], v[5]), sm103::pack_bf16(v[6], v[7]));
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// Sum over the TPR threads of a row; `turn` alternates between two buffers, so that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sm, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    float* buf = sm + (turn ^= NW);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += buf[w];
  }
  return v;
}

// TPR threads a row, C pieces of W elements each.  TPR 32: a warp a row, four rows a CTA; else a CTA a row.
// Of one piece of 8 a thread (LEAN) the next row is asked for before this one is summed up, and 16-bit weights
// stay in registers (KEEP).
// GATED: by channel or element.
template <int TPR, int W>
constexpr int kCtas = TPR == 1024 ? 1 : (W == 8 ? 1024 : 1536) / (TPR == 32 ? 128 : TPR);      // of an SM

template <typename T, typename R, int TPR, int C, int W, bool GATED>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, (kCtas<TPR, W>)) residual_norm_kernel(const NormArgs a) {
  __shared__ float sm[TPR > 32 ? 2 * (TPR / 32) : 1];
  constexpr int PER_CTA = TPR == 32 ? 4 : 1;
  constexpr bool LEAN = C == 1 && W == 8, KEEP = LEAN && sizeof(T) == 2;
  const int tid = TPR == 32 ? threadIdx.x & 31 : threadIdx.x, sub = TPR == 32 ? threadIdx.x >> 5 : 0;
  const float inv_n = 1.f / (float)a.hidden;
  const int64_t stride = (int64_t)gridDim.x * PER_CTA;
  int turn = 0;
  sm103::grid_wait();
  Raw<T, W> x_raw[C], post, pre;
  Raw<R, W> r_raw[C];
  auto ask = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + tid) * W;
      if (e < a.hidden) {
        r_raw[c].get(static_cast<const R*>(a.residual) + row * a.residual_stride + e);
        if (a.x) x_raw[c].get(static_cast<const T*>(a.x) + row * a.x_stride + e);
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * PER_CTA + sub;
  if (LEAN) {
    if (row < a.rows) ask(row);
    if (KEEP && tid * W < a.hidden) {
      if (a.post) post.get(static_cast<const T*>(a.post) + tid * W);
      if (a.y && a.pre) pre.get(static_cast<const T*>(a.pre) + tid * W);
    }
  }
  for (; row < a.rows; row += stride) {
    if (!LEAN) ask(row);
    float r[C][W], n[C][W];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if ((c * TPR + tid) * W < a.hidden) {
        r_raw[c].to(r[c]);
        if (a.x) x_raw[c].to(n[c]);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) r[c][k] = n[c][k] = 0.f;
      }
    }
    if (a.x) {
      float f = a.scale;
      if (a.gate_kind == MOE_RESIDUAL_GATE_ROW) {
        const float g = (float)static_cast<const T*>(a.gate)[row * a.gate_stride];
        f *= a.gate_sigmoid ? 1.f / (1.f + expf(-g)) : g;
      }
      if (LEAN && row + stride < a.rows) ask(row + stride);
      float inv = 1.f;
      if (a.post) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < W; ++k) ss += n[c][k] * n[c][k];
        inv = 1.f / sqrtf(row_sum<TPR>(ss, sm, turn) * inv_n + a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = (c * TPR + tid) * W;
        if (e >= a.hidden) continue;
        if (a.post) {
          float w[W];
          if (!KEEP) post.get(static_cast<const T*>(a.post) + e);
          post.to(w);
#pragma unroll
          for (int k = 0; k < W; ++k) n[c][k] = n[c][k] * inv * (a.offset + w[k]);
        }
        if (GATED) {
          Raw<T, W> raw;
          float g[W];
          raw.get(static_cast<const T*>(a.gate) + row * a.gate_stride + e);
          raw.to(g);
#pragma unroll
          for (int k = 0; k < W; ++k) n[c][k] *= a.gate_sigmoid ? 1.f / (1.f + expf(-g[k])) : g[k];
        }
#pragma unroll
        for (int k = 0; k < W; ++k) r[c][k] = fmaf(f, n[c][k], r[c][k]);
        store<W>(static_cast<R*>(a.sum) + row * a.sum_stride + e, r[c]);
      }
    } else if (LEAN && row + stride < a.rows) {
      ask(row + stride);
    }
    if (!a.y) continue;
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < W; ++k) ss += r[c][k] * r[c][k];
    const float inv = 1.f / sqrtf(row_sum<TPR>(ss, sm, turn) * inv_n + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + tid) * W;
      if (e >= a.hidden) continue;
      if (a.pre) {
        float w[W];
        if (!KEEP) pre.get(static_cast<const T*>(a.pre) + e);
        pre.to(w);
#pragma unroll
        for (int k = 0; k < W; ++k) r[c][k] = r[c][k] * inv * (a.offset + w[k]);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) r[c][k] *= inv;
      }
      store<W>(static_cast<T*>(a.y) + row * a.y_stride + e, r[c]);
    }
  }
}

template <typename T, typename R, int TPR, int C, int W>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  constexpr int threads = TPR == 32 ? 128 : TPR, per = TPR == 32 ? 4 : 1;
  const int64_t ctas = ((int64_t)a.rows + per - 1) / per, most = (int64_t)sm_count() * kCtas<TPR, W>;
  const int grid = (int)(ctas < most ? ctas : most);
  return a.gate_kind >= MOE_RESIDUAL_GATE_CHANNEL
             ? sm103::launch(residual_norm_kernel<T, R, TPR, C, W, true>, grid, threads, 0, s, a)
             : sm103::launch(residual_norm_kernel<T, R, TPR, C, W, false>, grid, threads, 0, s, a);
}

template <typename T, typename R>
cudaError_t pick(const NormArgs& a, cudaStream_t s) {
  auto wide = [](const void* p, int64_t stride, int size) {       // 8 elements at 16-byte boundaries in every row
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * size % 16 == 0);
  };
  const int ts = sizeof(T), rs = sizeof(R), h = a.hidden;
  const bool vec = h % 8 == 0 && wide(a.x, a.x_stride, ts) && wide(a.residual, a.residual_stride, rs) &&
                   wide(a.sum, a.sum_stride, rs) && wide(a.y, a.y_stride, ts) && wide(a.post, 0, ts) && wide(a.pre, 0, ts) &&
                   (a.gate_kind < MOE_RESIDUAL_GATE_CHANNEL || wide(a.gate, a.gate_stride, ts));
  if (vec) {
    if (h <= 32 * 8) return run<T, R, 32, 1, 8>(a, s);
    if (h <= 64 * 8) return run<T, R, 64, 1, 8>(a, s);
    if (h <= 128 * 8) return run<T, R, 128, 1, 8>(a, s);
    if (h <= 256 * 8) return run<T, R, 256, 1, 8>(a, s);
    if (h <= 512 * 8) return run<T, R, 512, 1, 8>(a, s);
    if (h <= 1024 * 8) return run<T, R, 1024, 1, 8>(a, s);
    return run<T, R, 1024, 2, 8>(a, s);
  }
  if (h <= 32 * 4) return run<T, R, 32, 4, 1>(a, s);
  if (h <= 128 * 8) return run<T, R, 128, 8, 1>(a, s);
  if (h <= 256 * 8) return run<T, R, 256, 8, 1>(a, s);
  if (h <= 512 * 8) return run<T, R, 512, 8, 1>(a, s);
  return run<T, R, 1024, 16, 1>(a, s);
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a, int dtype, int residual_dtype, cudaStream_t s) {
  if (dtype == MOE_F32) return pick<float, float>(a, s);
  return residual_dtype == MOE_F32 ? pick<bf16, float>(a, s) : pick<bf16, bf16>(a, s);
}

}  // namespace moeslot
