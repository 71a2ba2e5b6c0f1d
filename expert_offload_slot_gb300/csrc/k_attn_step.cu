// The two small operators ahead of the attention of a step.
//
// moe_attn_tables: block tables and row maps from the requests' lengths.
//   have_r = ceil(ctx_r / P), need_r = ceil((ctx_r + new_r) / P)
//   off_r  = sum over earlier requests of (need - have)
//   table[r, j] = free_pages[head + off_r + j - have_r]      have_r <= j < need_r
//   row t of request r: pos = ctx_r + t - row_start_r, slot = table[r, pos / P] * P + pos % P
// Every CTA scans the lengths of all requests itself (they are a few KB that L2
// serves), so one launch does it all and no CTA waits for another.
//
// moe_attn_qkv: y = x / sqrt(mean(x^2) + eps) * w for each query and key head,
// then the rotation (a, b) -> (a cos - b sin, b cos + a sin) of its first
// `rotary` elements, and K and V into their cache slots, in one pass: each head
// is read once and written once.
#include "attn_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
namespace {

// ------------------------------------------------------------------- tables
constexpr int TT = 256;
constexpr int kMaxLen = 1 << 30;

struct Lens {
  int ctx, fresh, have, need;
};

// The lengths of request r, made such that no sum of them leaves 32 bits (the host bounds R and
// rows); the rows past `rows` are reported, not written.
__device__ __forceinline__ Lens lens_of(const TablesArgs& a, int r, bool& bad) {
  Lens v;
  v.ctx = a.ctx[r];
  v.fresh = a.fresh[r];
  bad |= v.ctx < 0 || v.fresh < 0 || v.ctx > kMaxLen;
  v.ctx = min(max(v.ctx, 0), kMaxLen);
  v.fresh = min(max(v.fresh, 0), a.rows + 1);
  v.have = (v.ctx + a.page - 1) >> a.page_log2;
  v.need = (v.ctx + v.fresh + a.page - 1) >> a.page_log2;
  return v;
}

__global__ __launch_bounds__(TT) void attn_tables_kernel(const TablesArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* s_row = sm;                       // [R + 1] first row of each request
  int32_t* s_off = sm + a.R + 1;             // [R]     pages taken by the requests before it
  __shared__ int32_t s_warp[2][TT / 32];
  __shared__ int32_t s_carry[2];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  sm103::grid_wait();
  const int head = *a.head_in;
  bool bad = false, full = false;
  if (tid < 2) s_carry[tid] = 0;
  for (int r0 = 0; r0 < a.R; r0 += TT) {
    __syncthreads();
    const int r = r0 + tid;
    int rows = 0, pages = 0;
    if (r < a.R) {
      const Lens v = lens_of(a, r, bad);
      rows = v.fresh;
      pages = v.need - v.have;
      if (blockIdx.x == 0) a.seq_len[r] = v.ctx + v.fresh;
    }
    int ri = rows, pi = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, ri, o), y = __shfl_up_sync(0xffffffffu, pi, o);
      if (lane >= o) { ri += x; pi += y; }
    }
    if (lane == 31) { s_warp[0][wid] = ri; s_warp[1][wid] = pi; }
    __syncthreads();
    int rb = s_carry[0], pb = s_carry[1];
    for (int w = 0; w < wid; ++w) { rb += s_warp[0][w]; pb += s_warp[1][w]; }
    if (r < a.R) {
      s_row[r] = rb + ri - rows;
      s_off[r] = pb + pi - pages;
      if (r == a.R - 1) s_row[a.R] = rb + ri;
    }
    __syncthreads();
    if (tid == TT - 1) { s_carry[0] = rb + ri; s_carry[1] = pb + pi; }
  }
  if (a.R == 0 && tid == 0) s_row[0] = 0;
  __syncthreads();
  const int total = s_row[a.R], taken = s_carry[1];
  full |= total > a.rows;
  auto fresh_page = [&](int at) -> int {     // entry `at` of the free list beyond the head; -1 when it is short
    if (head < 0 || (int64_t)head + at >= a.num_free) { full = true; return -1; }
    return a.free_pages[head + at];
  };
  // the row starts, and the new table entries: a warp per request
  const int warps = gridDim.x * (TT / 32);
  for (int r = blockIdx.x * TT + tid; r <= a.R; r += gridDim.x * TT) a.row_start[r] = s_row[r];
  for (int r = blockIdx.x * (TT / 32) + wid; r < a.R; r += warps) {
    const Lens v = lens_of(a, r, bad);
    full |= v.need > a.table_stride;
    for (int j = v.have + lane; j < min(v.need, a.table_stride); j += 32)
      a.table[(size_t)r * a.table_stride + j] = fresh_page(s_off[r] + j - v.have);
  }
  // the rows
  for (int t = blockIdx.x * TT + tid; t < a.rows; t += gridDim.x * TT) {
    int pos = 0, slot = -1;
    if (t < total) {
      int lo = 0, hi = a.R - 1;
      while (lo < hi) {                      // last request that starts at or before row t
        const int mid = (lo + hi + 1) >> 1;
        if (s_row[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const Lens v = lens_of(a, lo, bad);
      pos = v.ctx + t - s_row[lo];
      const int j = pos >> a.page_log2;
      if (j < a.table_stride) {
        const int page = j >= v.have ? fresh_page(s_off[lo] + j - v.have) : a.table[(size_t)lo * a.table_stride + j];
        if (page >= 0) slot = (page << a.page_log2) + (pos & (a.page - 1));
        else bad = bad || j < v.have;
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  if (bad) atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
  if (full) atomicCAS(a.status, 0, MOE_ERR_CAPACITY);
  // head_out may be head_in: the last CTA to have read the head writes it
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
      *a.ticket = 0;
      *a.head_out = head + taken;
    }
  }
}

// ---------------------------------------------------------------------- qkv
constexpr int QT = 256;

template <typename T>
struct Vec;                                   // 16 bytes of a head
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const void* p, float* v) {
    const float4 x = *static_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
  static __device__ __forceinline__ void store(void* p, const float* v) {
    *static_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const void* p, float* v) {
    const uint4 x = *static_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A CTA per row: a group of D * sizeof(T) / 16 lanes takes a head at a time, its cosines, sines and
// norm weights in registers for all of the row's heads, U heads in flight.
template <typename T, int D>
__global__ __launch_bounds__(QT, 4) void attn_qkv_kernel(const QkvArgs a) {
  constexpr int N = Vec<T>::N, G = D / N, GROUPS = QT / G, U = 2;
  const int heads = a.Hq + 2 * a.Hkv, t = blockIdx.x, group = threadIdx.x / G, sub = threadIdx.x % G, e0 = sub * N;
  const int lane = threadIdx.x & 31, half = a.rotary / 2;
  sm103::grid_wait();
  const int64_t slot = a.slots[t];
  const int64_t pos = a.rotary > 0 ? a.positions[t] : 0;
  const T* src = static_cast<const T*>(a.qkv) + (size_t)t * a.qkv_stride + e0;
  float x[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (group + u * GROUPS < heads) Vec<T>::load(src + (size_t)(group + u * GROUPS) * D, x[u]);
  const bool in_table = pos >= 0 && pos < a.rope_len, turn = e0 < a.rotary && in_table;
  const bool first = e0 < half;
  float cs[N], sn[N];                         // of this lane's elements (MOE_ROTARY_PAIRS: the first N / 2)
  if (turn) {
    const float* row = a.rope + pos * a.rotary;
    const int i0 = a.pairs ? e0 / 2 : first ? e0 : e0 - half;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.pairs && i >= N / 2) break;
      cs[i] = row[i0 + i];
      sn[i] = row[half + i0 + i];
    }
  }
  if (a.rotary > 0 && !in_table && threadIdx.x == 0) atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
  if (slot >= a.num_slots && threadIdx.x == 0) atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
  const bool cached = slot >= 0 && slot < a.num_slots;
  const int64_t page = slot >> a.page_log2, in = slot & ((1 << a.page_log2) - 1);
  const int peer = e0 < a.rotary ? (first ? lane + half / N : lane - half / N) : lane;
  for (int h0 = group; h0 - group < heads; h0 += U * GROUPS) {       // the same number of rounds in every group
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int head = h0 + u * GROUPS;
      const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hkv;
      float y[N], ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        y[i] = x[u][i];
        ss += y[i] * y[i];
      }
      if (head + U * GROUPS < heads) Vec<T>::load(src + (size_t)(head + U * GROUPS) * D, x[u]);   // of the next round
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const void* w = is_q ? a.q_norm : a.k_norm;
      if (!is_v && w) {
        float g[N];
        Vec<T>::load(static_cast<const T*>(w) + e0, g);
        const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = y[i] * inv * g[i];
      }
      if (a.pairs) {
        if (turn && !is_v) {
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float p = y[i], q = y[i + 1];
            y[i] = p * cs[i / 2] - q * sn[i / 2];
            y[i + 1] = q * cs[i / 2] + p * sn[i / 2];
          }
        }
      } else if (a.rotary > 0) {              // uniform: every lane takes part in the exchange
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float z = __shfl_sync(0xffffffffu, y[i], peer);
          if (turn && !is_v) y[i] = first ? y[i] * cs[i] - z * sn[i] : y[i] * cs[i] + z * sn[i];
        }
      }
      if (head >= heads) continue;
      if (is_q) {
        Vec<T>::store(static_cast<T*>(a.q) + ((size_t)t * a.Hq + head) * D + e0, y);
      } else if (cached) {
        const int h = head - a.Hq - (is_v ? a.Hkv : 0);
        T* dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache);
        Vec<T>::store(dst + ((((page * a.Hkv + h) << a.page_log2) + in) * D + e0), y);
      }
    }
  }
}

template <typename T, int D>
cudaError_t qkv(const QkvArgs& a, cudaStream_t s) {
  return sm103::launch(attn_qkv_kernel<T, D>, a.rows, QT, 0, s, a);
}

}  // namespace

cudaError_t launch_attn_tables(const TablesArgs& a, cudaStream_t s) {
  const int work = a.rows > a.R * 32 ? a.rows : a.R * 32;
  int grid = (work + TT - 1) / TT;
  grid = grid < 1 ? 1 : grid > 152 ? 152 : grid;
  return sm103::launch(attn_tables_kernel, grid, TT, (2 * a.R + 1) * sizeof(int32_t), s, a);
}

cudaError_t launch_attn_qkv(const QkvArgs& a, int dtype, int D, cudaStream_t s) {
  if (dtype == MOE_F32) return D == 64 ? qkv<float, 64>(a, s) : qkv<float, 128>(a, s);
  return D == 64 ? qkv<__nv_bfloat16, 64>(a, s) : qkv<__nv_bfloat16, 128>(a, s);
}

}  // namespace moeslot
