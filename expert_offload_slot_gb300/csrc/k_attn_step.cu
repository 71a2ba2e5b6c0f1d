// The two small operators ahead of the attention of a step.
//
// moe_attn_tables: block tables and row maps from the requests' lengths.
//   have_r = ceil(ctx_r / P), need_r = ceil((ctx_r + new_r) / P)
//   off_r  = sum over earlier requests of (need - have)
//   table[r, j] = free_pages[head + off_r + j - have_r]      have_r <= j < need_r
//   row t of request r: pos = ctx_r + t - row_start_r, slot = table[r, pos / P] * P + pos % P
// Without a free list every page is in the table already: nothing is written there or taken.
// Every CTA scans the lengths of all requests itself (they are a few KB that L2
// serves), so one launch does it all and no CTA waits for another.  A step moves
// a few hundred KB at most, so the launch bounds it: 384 requests with 25k new
// rows take 7.6 us a call, 16 requests with one row each 7.5.
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
  const bool given = a.num_free == 0;        // the tables are complete: only the maps are wanted
  const int total = s_row[a.R], taken = given ? 0 : s_carry[1];
  full |= total > a.rows;
  auto is_short = [&](int at) { return head < 0 || (int64_t)head + at >= a.num_free; };
  auto fresh_page = [&](int at) -> int {     // entry `at` of the free list beyond the head; -1 when it is short
    if (is_short(at)) { full = true; return -1; }
    return a.free_pages[head + at];
  };
  // the row starts, and the new table entries: a warp per request
  const int warps = gridDim.x * (TT / 32);
  for (int r = blockIdx.x * TT + tid; r <= a.R; r += gridDim.x * TT) a.row_start[r] = s_row[r];
  for (int r = blockIdx.x * (TT / 32) + wid; r < a.R; r += warps) {
    const Lens v = lens_of(a, r, bad);
    full |= v.need > a.table_stride;
    if (given) continue;
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
        const bool fresh = j >= v.have && !given;
        const int at = s_off[lo] + j - v.have, page = fresh ? fresh_page(at) : a.table[(size_t)lo * a.table_stride + j];
        // a page whose slots need more than 31 bits would come out as the slots of another
        if ((uint32_t)page <= 0x7fffffffu >> a.page_log2) slot = (page << a.page_log2) + (pos & (a.page - 1));
        else bad |= !(fresh && is_short(at));
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

// Eight consecutive elements.
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(sm103::pack_bf16(v[0], v[1]), sm103::pack_bf16(v[2], v[3]),
                                            sm103::pack_bf16(v[4], v[5]), sm103::pack_bf16(v[6], v[7]));
}

// D / 16 lanes a head, 16 elements a lane in two chunks of eight.  With MOE_ROTARY_HALF a lane of the
// turning part has elements i .. i+7 and their partners i + half .. i + half + 7, so the rotation
// needs no exchange; the lanes after it have the rest in order (rotary_dim is a multiple of 16, so
// the two parts fill whole lanes).
template <int D>
struct HeadLane {
  static constexpr int G = D / 16;
  int sub, e0, e1;
  bool turn;
  __device__ __forceinline__ explicit HeadLane(const QkvArgs& a) {
    const int half = a.rotary / 2;
    sub = threadIdx.x % G;
    const bool split = !a.pairs && 8 * sub < half;
    turn = split || (a.pairs && 16 * sub < a.rotary);
    e0 = split ? 8 * sub : a.pairs ? 16 * sub : a.rotary + 16 * (sub - half / 8);
    e1 = split ? half + 8 * sub : e0 + 8;
  }
  // Norm and rotation of a query or key head; `rope`: the row's cosines and sines, or none.
  template <typename T>
  __device__ __forceinline__ void work(const QkvArgs& a, const T* w, const float* rope, float (&x)[16]) const {
    if (w) {
      float ss = 0.f, g[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += x[i] * x[i];
      const uint32_t lanes = ((1u << G) - 1) << ((threadIdx.x & 31) / G * G);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
      load8(w + e0, g);
      load8(w + e1, g + 8);
      const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * inv * g[i];
    }
    if (turn && rope) {
      float cs[8], sn[8];
      load8(rope + 8 * sub, cs);
      load8(rope + a.rotary / 2 + 8 * sub, sn);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = a.pairs ? x[2 * i] : x[i], v = a.pairs ? x[2 * i + 1] : x[i + 8];
        const float y = u * cs[i] - v * sn[i], z = v * cs[i] + u * sn[i];
        if (a.pairs) {
          x[2 * i] = y;
          x[2 * i + 1] = z;
        } else {
          x[i] = y;
          x[i + 8] = z;
        }
      }
    }
  }
  // The head's place in q or, by its row's slot (>= 0), in the cache.
  template <typename T>
  __device__ __forceinline__ T* place(const QkvArgs& a, int t, int head, int64_t slot) const {
    if (head < a.Hq) return static_cast<T*>(a.q) + ((size_t)t * a.Hq + head) * D;
    const bool is_v = head >= a.Hq + a.Hkv;
    const int64_t page = slot >> a.page_log2, in = slot & ((1 << a.page_log2) - 1);
    const int h = head - a.Hq - (is_v ? a.Hkv : 0);
    return static_cast<T*>(is_v ? a.v_cache : a.k_cache) + (((page * a.Hkv + h) << a.page_log2) + in) * D;
  }
};

// Few rows: every (row, head) is independent, a group of lanes each.
template <typename T, int D>
__global__ __launch_bounds__(QT) void attn_qkv_kernel(const QkvArgs a) {
  constexpr int G = D / 16;
  const HeadLane<D> lane(a);
  const uint32_t unit = blockIdx.x * (QT / G) + threadIdx.x / G;
  sm103::grid_wait();
  if (unit >= (uint32_t)a.rows * a.heads) return;            // whole groups of lanes
  const int t = (int)(((uint64_t)unit * a.unit_mul) >> a.unit_shift), head = (int)(unit - (uint32_t)t * a.heads);
  float x[16];
  const T* src = static_cast<const T*>(a.qkv) + (size_t)t * a.qkv_stride + (size_t)head * D;
  load8(src + lane.e0, x);
  load8(src + lane.e1, x + 8);
  const int64_t slot = head < a.Hq ? 0 : a.slots[t];
  if (head < a.Hq + a.Hkv) {
    const int64_t pos = a.rotary > 0 ? a.positions[t] : 0;
    const bool in_table = pos >= 0 && pos < a.rope_len;
    if (a.rotary > 0 && !in_table && lane.sub == 0) atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
    lane.work(a, static_cast<const T*>(head < a.Hq ? a.q_norm : a.k_norm), in_table ? a.rope + pos * a.rotary : nullptr, x);
  }
  if (slot < 0) return;                                      // a padding row
  if (slot >= a.num_slots) {
    atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
    return;
  }
  T* dst = lane.template place<T>(a, t, head, slot);
  store8(dst + lane.e0, x);
  store8(dst + lane.e1, x + 8);
}

// Many rows: persistent CTAs whose last warp brings rows (or pieces of long ones) and their rotation
// into a ring in shared memory by bulk copies, so that HBM is read ahead of the work: in the kernel
// above a group of lanes waits for its position, then for the rotation's row, and nothing is in
// flight while it does.  HBM bounds it: 16384 rows of 32 + 2 x 4 heads of 128, bf16 (344 MB moved),
// 58 us or 5.9 TB/s, 75 us by the kernel above; 2048 rows with 2 x 8 heads (51 MB) 13.1 us, 15.6.
// With 1024 such rows, 48 heads of 8 lanes, the two are level (8.5 and 8.9 us), below that the one
// above is ahead (256 rows: 3.1 and 4.3 us): so it takes up to 4096 lanes per SM.
constexpr int ST = QT + 32, kRing = 4, kPiece = 16384;       // kPiece: bytes of a piece at most
constexpr int kLanes = 4096;
struct RowMeta {
  int64_t slot;
  int32_t rope;                                              // the rotation's row is there
};
template <typename T, int D>
__global__ __launch_bounds__(ST, 4) void attn_qkv_rows_kernel(const QkvArgs a) {
  constexpr int G = D / 16;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kRing], empty[kRing];
  __shared__ RowMeta meta[kRing];
  const int tid = threadIdx.x, stage = a.chunk_heads * D * (int)sizeof(T) + a.rotary * 4;
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      sm103::bar_init(full + s, 1);
      sm103::bar_init(empty + s, QT / 32);
    }
    sm103::bar_init_done();
  }
  __syncthreads();
  sm103::grid_wait();
  const uint32_t units = (uint32_t)a.rows * a.chunks;
  if (tid >= QT) {                                           // the loading warp, its first lane
    if (tid > QT) return;
    uint32_t it = 0;
    bool alive = true;
    for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x, ++it) {
      const int t = (int)(((uint64_t)unit * a.unit_mul) >> a.unit_shift), h0 = (int)(unit - (uint32_t)t * a.chunks) * a.chunk_heads;
      const int n = min(a.chunk_heads, a.heads - h0), st = it % kRing;
      RowMeta m = {0, 0};
      int64_t pos = 0;
      if (h0 + n > a.Hq) m.slot = a.slots[t];
      if (a.rotary > 0 && h0 < a.Hq + a.Hkv) {
        pos = a.positions[t];
        m.rope = pos >= 0 && pos < a.rope_len;
        if (!m.rope) atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
      }
      if (m.slot >= a.num_slots) {
        atomicCAS(a.status, 0, MOE_ERR_BOUNDS);
        m.slot = -1;
      }
      if (it >= kRing && !(alive = sm103::bar_wait(empty + st, (it / kRing - 1) & 1))) break;
      meta[st] = m;
      const uint32_t dst = sm103::smem_addr(ring) + st * stage, bytes = n * D * (uint32_t)sizeof(T);
      sm103::bar_expect(full + st, bytes + (m.rope ? a.rotary * 4 : 0));
      sm103::bulk_load(dst, static_cast<const T*>(a.qkv) + (size_t)t * a.qkv_stride + (size_t)h0 * D, bytes, full + st);
      if (m.rope) sm103::bulk_load(dst + stage - a.rotary * 4, a.rope + pos * a.rotary, a.rotary * 4, full + st);
    }
    if (!alive) atomicCAS(a.status, 0, MOE_ERR_TIMEOUT);
    // the memory is not given up before the last copies have landed
    for (uint32_t k = it > kRing ? it - kRing : 0; k < it; ++k) sm103::bar_wait(full + k % kRing, (k / kRing) & 1);
    return;
  }
  const HeadLane<D> lane(a);
  constexpr int groups = QT / G;
  uint32_t it = 0;
  int first = tid / G;                                       // each row begins with the group after the last one's
  for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x, ++it) {
    const int t = (int)(((uint64_t)unit * a.unit_mul) >> a.unit_shift), h0 = (int)(unit - (uint32_t)t * a.chunks) * a.chunk_heads;
    const int n = min(a.chunk_heads, a.heads - h0), st = it % kRing;
    if (!sm103::bar_wait_warp(full + st, (it / kRing) & 1)) {
      atomicCAS(a.status, 0, MOE_ERR_TIMEOUT);
      return;
    }
    const T* row = reinterpret_cast<const T*>(ring + st * stage);
    const float* rope = reinterpret_cast<const float*>(ring + (st + 1) * stage - a.rotary * 4);
    const RowMeta m = meta[st];
    int k = first;
    for (; k < n; k += groups) {
      const int head = h0 + k;
      float x[16];
      load8(row + k * D + lane.e0, x);
      load8(row + k * D + lane.e1, x + 8);
      if (head < a.Hq + a.Hkv)
        lane.work(a, static_cast<const T*>(head < a.Hq ? a.q_norm : a.k_norm), m.rope ? rope : nullptr, x);
      if (head >= a.Hq && m.slot < 0) continue;              // a padding row
      T* dst = lane.template place<T>(a, t, head, m.slot);
      store8(dst + lane.e0, x);
      store8(dst + lane.e1, x + 8);
    }
    first = k - n;
    __syncwarp();
    if ((tid & 31) == 0) sm103::bar_arrive(empty + st);
  }
}

template <typename T, int D>
cudaError_t qkv(QkvArgs a, int sms, cudaStream_t s) {
  const int64_t units = (int64_t)a.rows * a.heads;
  if (units * (D / 16) > (int64_t)kLanes * sms) {
    constexpr int most = kPiece / (D * (int)sizeof(T));
    a.chunks = (a.heads + most - 1) / most;
    a.chunk_heads = (a.heads + a.chunks - 1) / a.chunks;
    a.chunks = (a.heads + a.chunk_heads - 1) / a.chunk_heads;
    divider(a.chunks, a.unit_mul, a.unit_shift);
    const int bytes = kRing * (a.chunk_heads * D * (int)sizeof(T) + a.rotary * 4);
    const int fit = 225 * 1024 / (bytes + 2048), per_sm = fit < 4 ? fit : 4;
    const int64_t pieces = (int64_t)a.rows * a.chunks, grid = (int64_t)per_sm * sms;
    return sm103::launch(attn_qkv_rows_kernel<T, D>, (int)(pieces < grid ? pieces : grid), ST, bytes, s, a);
  }
  constexpr int per = QT / (D / 16);
  divider(a.heads, a.unit_mul, a.unit_shift);
  return sm103::launch(attn_qkv_kernel<T, D>, (int)((units + per - 1) / per), QT, 0, s, a);
}

template <typename T, int D>
cudaError_t qkv_prepare() {
  return cudaFuncSetAttribute(attn_qkv_rows_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * (kPiece + D * 4));
}

}  // namespace

cudaError_t launch_attn_tables(const TablesArgs& a, cudaStream_t s) {
  const int work = a.rows > a.R * 32 ? a.rows : a.R * 32;
  int grid = (work + TT - 1) / TT;
  grid = grid < 1 ? 1 : grid > 152 ? 152 : grid;
  return sm103::launch(attn_tables_kernel, grid, TT, (2 * a.R + 1) * sizeof(int32_t), s, a);
}

cudaError_t prepare_attn_qkv(int dtype, int D) {
  if (dtype == MOE_F32) return D == 64 ? qkv_prepare<float, 64>() : qkv_prepare<float, 128>();
  return D == 64 ? qkv_prepare<__nv_bfloat16, 64>() : qkv_prepare<__nv_bfloat16, 128>();
}

cudaError_t launch_attn_qkv(const QkvArgs& a, int dtype, int D, int sms, cudaStream_t s) {
  if (dtype == MOE_F32) return D == 64 ? qkv<float, 64>(a, sms, s) : qkv<float, 128>(a, sms, s);
  return D == 64 ? qkv<__nv_bfloat16, 64>(a, sms, s) : qkv<__nv_bfloat16, 128>(a, sms, s);
}

}  // namespace moeslot
