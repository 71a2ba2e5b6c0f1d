// moe_logprobs: the log probability and rank of a given token in each row of logits, the
// row's entropy and its most probable tokens.
//
//   lse = max + log sum exp(x - max), logp = x_t - lse, entropy = lse - sum p x
//
// One pass over the row, shared by the CTAs of a cluster: each thread keeps the running
// maximum m of its logits in log2 units (rounded, so one number is the reference of all) and,
// relative to it, s = sum e and w = sum e z with z = x log2(e) - m, one rounding, e = 2^z; when
// m grows by -d, s becomes 2^d s and w 2^d (w + d s).  Then logp = (z_t - log2 s) log(2) and
// entropy = (log2 s - w / s) log(2): differences of numbers of different signs, nothing cancels.
//
// The best tokens need no second pass over the row: the n-th largest of 32 or 64 groups' maxima
// is a bound that n logits reach, only the logits of threads whose own maximum reaches it are looked at
// again, and the few that do are sorted by (x, index).  Rows where the bound does
// not help (equal logits in thousands, hardly any token) are searched by bisection, some fifty passes: one row of 131072
// with three tokens above -inf 81 us.
//
// NaN counts as -inf.  Logits far from zero, where the products with log2(e) lose the
// differences, and rows without a token take a second, careful pass.
//
// What bounds it: of many rows HBM and, near it, the instructions of a logit, which therefore
// are taken in pairs (bf16 comparisons and maxima, fp32 sums): 2048 rows of 131072 bf16 logits without
// best tokens 90 us (6.0 TB/s, 88 % of a copy's rate), with five 102, with twenty 126; an exponential, a
// product and two sums for each logit by itself took 128 (five).  One row of 131072: 5.0 us, 8.5 with twenty
// best tokens: loads, two exchanges in the cluster, the bound and the sorting one after another.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm103.cuh"
#include "step_internal.cuh"

namespace moeslot {
namespace {
namespace cg = cooperative_groups;
typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

constexpr int kMaxCluster = 8, kMaxThreads = 512;
constexpr int kTop = MOE_LOGPROBS_MAX_TOP;
constexpr int kGroups = 64;                    // whose maxima bound the best tokens; twice kTop
constexpr int kFew = 20;                       // of 32 groups' maxima: some 32 ln(32 / 12) = 31 logits reach the 20th
constexpr int kList = 256;                     // tokens that reach the bound, at most
static_assert(kGroups >= 2 * kTop && kList >= kMaxCluster * kTop, "room for every list");
constexpr float kLow = -1e38f;                 // logits are held above it (so -inf and NaN are there, too) and, below
constexpr float kNone = -9e37f;                // this first maximum, add nothing; rows without a larger one are `far`
constexpr float kFar = 1048576.f;              // up to it (log2 units) the rounding of m leaves e below 1.05
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct Soft {                                  // part of a row: see above; m in log2 units
  float m, s, w;
};
__device__ __forceinline__ void join(Soft& a, const Soft& b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m - m, db = b.m - m, fa = sm103::ex2(da), fb = sm103::ex2(db);
  // an exponential of zero ends a part, whatever its sums are
  const float wa = fa > 0.f ? fa * fmaf(da, a.s, a.w) : 0.f, wb = fb > 0.f ? fb * fmaf(db, b.s, b.w) : 0.f;
  a.m = m;
  a.s = fa * a.s + fb * b.s;
  a.w = wa + wb;
}

struct Shared {                                // of a CTA; the cluster reads the second part
  Soft warp[kMaxThreads / 32];
  int32_t count[kMaxThreads / 32];
  float best[kMaxThreads];
  u64 list[kList];
  float bound;
  int32_t found, owners;
  int16_t owner[kMaxThreads];
  // shown to the cluster
  Soft soft;
  float most;
  int32_t rank, kept;
  u64 top[kTop];
};

__device__ __forceinline__ float clean(float x) {  // NaN counts as -inf, -0 as +0
  x += 0.f;
  return x == x ? x : -INFINITY;
}
// Descending logits, equal ones by ascending index, as descending keys.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ u64 key_of(float x, int i) { return (u64)ordered(x) << 32 | (0xffffffffu - (uint32_t)i); }
__device__ __forceinline__ int index_of(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float raw(float v) { return v; }
__device__ __forceinline__ float raw(bf16 v) { return __bfloat162float(v); }

// 16 bytes of logits: two at a time held above kLow, and the number above the target (or equal: before it),
// summed up in `Count`s of up to 256 logits.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int W = 4;
  typedef int Count;
  static __device__ __forceinline__ Count none() { return 0; }
  static __device__ __forceinline__ int total(Count n) { return n; }
  template <bool before>
  static __device__ __forceinline__ void above(const uint4& u, float xt, Count& n) {
    const float v[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
#pragma unroll
    for (int k = 0; k < 4; ++k) n += before ? v[k] >= xt : v[k] > xt;
  }
  static __device__ __forceinline__ void hold(uint4& u) {
    u.x = __float_as_uint(fmaxf(__uint_as_float(u.x), kLow));
    u.y = __float_as_uint(fmaxf(__uint_as_float(u.y), kLow));
    u.z = __float_as_uint(fmaxf(__uint_as_float(u.z), kLow));
    u.w = __float_as_uint(fmaxf(__uint_as_float(u.w), kLow));
  }
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    float m = kLow;
#pragma unroll
    for (int k = 0; k < N; ++k)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u[k].x), __uint_as_float(u[k].y)), fmaxf(__uint_as_float(u[k].z), __uint_as_float(u[k].w))));
    return m;
  }
  template <typename F>
  static __device__ __forceinline__ void pairs(const uint4& u, F f) {
    f(__uint_as_float(u.x), __uint_as_float(u.y));
    f(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <>
struct Vec<bf16> {
  static constexpr int W = 8;
  typedef __nv_bfloat162 Count;                // two counts, exact up to 256
  static __device__ __forceinline__ Count none() { return __float2bfloat162_rn(0.f); }
  static __device__ __forceinline__ int total(Count n) { return (int)(__low2float(n) + __high2float(n)); }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
  static __device__ __forceinline__ uint32_t word(__nv_bfloat162 p) { return *reinterpret_cast<const uint32_t*>(&p); }
  template <bool before>
  static __device__ __forceinline__ void above(const uint4& u, float xt, Count& n) {
    const __nv_bfloat162 t = __float2bfloat162_rn(xt);               // a logit: exact
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) n = __hadd2(n, before ? __hge2(pair(w[k]), t) : __hgt2(pair(w[k]), t));
  }
  static __device__ __forceinline__ void hold(uint4& u) {
    const __nv_bfloat162 low = __float2bfloat162_rn(kLow);
    u.x = word(__hmax2(pair(u.x), low));
    u.y = word(__hmax2(pair(u.y), low));
    u.z = word(__hmax2(pair(u.z), low));
    u.w = word(__hmax2(pair(u.w), low));
  }
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    __nv_bfloat162 m = pair(u[0].x);
#pragma unroll
    for (int k = 0; k < N; ++k) m = __hmax2(m, __hmax2(__hmax2(pair(u[k].x), pair(u[k].y)), __hmax2(pair(u[k].z), pair(u[k].w))));
    return fmaxf(__low2float(m), __high2float(m));
  }
  template <typename F>
  static __device__ __forceinline__ void pairs(const uint4& u, F f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  }
};

// The logits of a CTA: [head | vectors v0 .. v1 | tail], the vectors on 16-byte boundaries; head and tail
// are less than a vector and belong to the first and the last CTA.
template <typename T>
struct Share {
  static constexpr int W = Vec<T>::W;
  const T* x;
  int lead, v0, v1, head, tail0, tail;         // logit of vector 0; elements before it; first of and elements of the tail
  __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(x + lead); }
  // the element of thread `tid` outside of the vectors, or -1
  __device__ __forceinline__ int single(int tid) const {
    if (tid < head) return tid;
    return tid >= 32 && tid - 32 < tail ? tail0 + tid - 32 : -1;
  }
  // f(x, index) for every logit, spread over the CTA's threads
  template <typename F>
  __device__ __forceinline__ void each(int tid, int nt, F f) const {
    const int i = single(tid);
    if (i >= 0) f(clean(raw(x[i])), i);
    const int from = lead + v0 * W, to = lead + v1 * W;
    for (int k = from + tid; k < to; k += nt) f(clean(raw(x[k])), k);
  }
};

template <typename T, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 2) logprobs_kernel(const LogprobArgs a) {
  constexpr int W = Vec<T>::W, NW = NT / 32, U = 4;
  static_assert(NT <= kMaxThreads, "room for every thread");
  __shared__ Shared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), row = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  sm103::grid_wait();
  Share<T> in;
  in.x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
  in.lead = min((int)((16 - (reinterpret_cast<uintptr_t>(in.x) & 15)) & 15) / (int)sizeof(T), a.vocab);
  const int vectors = (a.vocab - in.lead) / W;
  in.v0 = (int)((int64_t)rank * vectors / cs);
  in.v1 = (int)((int64_t)(rank + 1) * vectors / cs);
  in.head = rank == 0 ? in.lead : 0;
  in.tail0 = in.lead + vectors * W;
  in.tail = rank == cs - 1 ? a.vocab - in.tail0 : 0;

  const int target = a.targets[row];
  const bool asked = target >= 0 && target < a.vocab;
  const float xt = asked ? clean(raw(in.x[target])) : INFINITY;

  // ------------------------------------------------ one pass
  Soft soft = {kNone * kLog2e, 0.f, 0.f};
  float mine = kNone;                          // this thread's maximum
  int above = 0;
  {
    using sm103::pack2;
    const uint64_t log2e2 = pack2(kLog2e, kLog2e);
    uint64_t s2 = 0, w2 = 0;                   // two sums each, of even and odd logits
    auto grow = [&](float m) {                 // to a maximum m
      mine = m;
      m *= kLog2e;
      const float d = soft.m - m, f = sm103::ex2(d);
      float s0, s1, w0, w1;
      sm103::unpack2(s2, s0, s1);
      sm103::unpack2(w2, w0, w1);
      w2 = f > 0.f ? pack2(f * fmaf(d, s0, w0), f * fmaf(d, s1, w1)) : 0;
      s2 = pack2(s0 * f, s1 * f);
      soft.m = m;
    };
    auto add = [&](float x, float y) {
      float z0, z1;
      const uint64_t z = sm103::fma2(pack2(x, y), log2e2, pack2(-soft.m, -soft.m));
      sm103::unpack2(z, z0, z1);
      const uint64_t e = pack2(sm103::ex2(z0), sm103::ex2(z1));
      s2 = sm103::add2(s2, e);
      w2 = sm103::fma2(e, z, w2);
    };
    const int i = in.single(tid);
    if (i >= 0) {
      const float x = raw(in.x[i]), v = fmaxf(x, kLow);
      above += i < target ? x >= xt : x > xt;
      if (v > mine) grow(v);
      add(v, kLow);
    }
    const uint4* p = in.vectors();
    // N vectors, NT apart, from `vec` on
    auto take = [&](auto& u, int vec) {
      constexpr int N = sizeof(u) / sizeof(uint4);
      typename Vec<T>::Count n = Vec<T>::none();
      const int first = in.lead + vec * W;
      if (first + (N - 1) * NT * W < target) {
#pragma unroll
        for (int k = 0; k < N; ++k) Vec<T>::template above<true>(u[k], xt, n);
      } else if (first >= target) {
#pragma unroll
        for (int k = 0; k < N; ++k) Vec<T>::template above<false>(u[k], xt, n);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (first + k * NT * W < target) Vec<T>::template above<true>(u[k], xt, n);
          else Vec<T>::template above<false>(u[k], xt, n);
        }
      }
      above += Vec<T>::total(n);
#pragma unroll
      for (int k = 0; k < N; ++k) Vec<T>::hold(u[k]);
      const float m = Vec<T>::largest(u);
      if (m > mine) grow(m);
#pragma unroll
      for (int k = 0; k < N; ++k) Vec<T>::pairs(u[k], add);
    };
    int v = in.v0 + tid;
    for (; v + (U - 1) * NT < in.v1; v += U * NT) {
      uint4 u[U];
#pragma unroll
      for (int k = 0; k < U; ++k) u[k] = __ldg(p + v + k * NT);
      take(u, v);
    }
    for (; v < in.v1; v += NT) {
      uint4 u[1] = {__ldg(p + v)};
      take(u, v);
    }
    float s0, s1, w0, w1;
    sm103::unpack2(s2, s0, s1);
    sm103::unpack2(w2, w0, w1);
    soft.s = s0 + s1;
    soft.w = w0 + w1;
  }
  // the target's own vector counted all its equals: those from the target on do not stand before it
  if (asked && target > in.lead && target < in.tail0) {
    const int vec = (target - in.lead) / W;
    if (vec >= in.v0 && vec < in.v1 && (vec - in.v0) % NT == tid && in.lead + vec * W < target)
      for (int i = target; i < in.lead + (vec + 1) * W; ++i) above -= raw(in.x[i]) == xt;
  }
  if (asked && xt == -INFINITY) {              // NaN is equal to it, which the comparisons do not see
    above = 0;
    in.each(tid, NT, [&](float x, int i) { above += x > xt || i < target; });
  }

  auto reduce = [&](Soft& v, int& n) {         // over the CTA, into every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Soft other;
      other.m = __shfl_xor_sync(0xffffffffu, v.m, o);
      other.s = __shfl_xor_sync(0xffffffffu, v.s, o);
      other.w = __shfl_xor_sync(0xffffffffu, v.w, o);
      join(v, other);
    }
    n = (int)__reduce_add_sync(0xffffffffu, (uint32_t)n);
    __syncthreads();
    if (lane == 0) {
      sm.warp[wid] = v;
      sm.count[wid] = n;
    }
    __syncthreads();
    v = sm.warp[0];
    n = sm.count[0];
    for (int w = 1; w < NW; ++w) {
      join(v, sm.warp[w]);
      n += sm.count[w];
    }
  };
  sm.best[tid] = mine;
  reduce(soft, above);                         // its barriers show the maxima, too
  if (tid == 0) {
    sm.soft = soft;
    sm.rank = above;
    sm.found = sm.owners = 0;
  }

  // ------------------------------------------------ the CTA's best tokens, sorted
  const int n = min(a.top, a.vocab);
  if (n > 0) {
    auto count = [&](auto pred) -> int {       // logits of the CTA that satisfy it
      int c = 0;
      in.each(tid, NT, [&](float x, int i) { c += pred(x, i); });
      c = (int)__reduce_add_sync(0xffffffffu, (uint32_t)c);
      __syncthreads();
      if (lane == 0) sm.count[wid] = c;
      __syncthreads();
      c = 0;
      for (int w = 0; w < NW; ++w) c += sm.count[w];
      return c;
    };
    if (wid == 0) {                            // the n-th largest maximum of 64 groups, or of 32
      float g[2] = {kNone, kNone};
#pragma unroll
      for (int k = 0; k < NT / kGroups; ++k) {
        g[0] = fmaxf(g[0], sm.best[lane + k * kGroups]);
        g[1] = fmaxf(g[1], sm.best[lane + 32 + k * kGroups]);
      }
      int larger[2] = {0, 0};
      if (n <= kFew) {                         // 32 groups do
        g[0] = fmaxf(g[0], g[1]);
        g[1] = kNone;
        larger[1] = n;
#pragma unroll
        for (int k = 0; k < 32; ++k) larger[0] += __shfl_sync(0xffffffffu, g[0], k) > g[0];
      } else {
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
          const float p = __shfl_sync(0xffffffffu, g[0], k), q = __shfl_sync(0xffffffffu, g[1], k);
          larger[0] += (p > g[0]) + (q > g[0]);
          larger[1] += (p > g[1]) + (q > g[1]);
        }
      }
      const uint32_t least = min(larger[0] < n ? ordered(g[0]) : 0xffffffffu, larger[1] < n ? ordered(g[1]) : 0xffffffffu);
      const uint32_t bound = __reduce_min_sync(0xffffffffu, least);
      if (lane == 0) sm.bound = value_of((u64)bound << 32);
    }
    __syncthreads();
    const float bound = sm.bound;
    bool listed = bound > kNone;
    if (listed) {
      // the logits of the threads that reach it, by all threads, four vectors on their way
      auto offer = [&](float x, int i) {
        if (x >= bound) {
          const int at = atomicAdd(&sm.found, 1);
          if (at < kList) sm.list[at] = key_of(x + 0.f, i);
        }
      };
      if (mine >= bound) {
        sm.owner[atomicAdd(&sm.owners, 1)] = (int16_t)tid;
        const int i = in.single(tid);
        if (i >= 0) offer(raw(in.x[i]), i);
      }
      __syncthreads();
      const int per = max(1, (in.v1 - in.v0 + NT - 1) / NT), all = sm.owners * per;
      for (int j = tid; j < all; j += 4 * NT) {
        uint4 u[4];
        int at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int which = (j + k * NT) / per, v = in.v0 + (j + k * NT - which * per) * NT + (j + k * NT < all ? sm.owner[which] : 0);
          at[k] = j + k * NT < all && v < in.v1 ? v : -1;
          if (at[k] >= 0) u[k] = __ldg(in.vectors() + v);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (at[k] < 0) continue;
          int i = in.lead + at[k] * W;
          Vec<T>::pairs(u[k], [&](float x, float y) {
            offer(x, i);
            offer(y, i + 1);
            i += 2;
          });
        }
      }
      __syncthreads();
      listed = sm.found <= kList;
    }
    if (!listed) {                             // bisection over the ordered logits, then over the index of the last ones
      __syncthreads();
      if (tid == 0) sm.found = 0;
      const uint32_t none = ordered(-INFINITY);
      const int want = min(n, count([&](float x, int) { return ordered(x) > none; }));
      if (want > 0) {
        uint32_t lo = none + 1, hi = 0xffffffffu;                    // the largest key that `want` logits reach
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2 + 1;
          if (count([&](float x, int) { return ordered(x) >= mid; }) >= want) lo = mid;
          else hi = mid - 1;
        }
        const int ties = want - count([&](float x, int) { return ordered(x) > lo; });
        int first = 0, last = a.vocab - 1;     // the lowest index up to which enough are equal to it
        while (first < last) {
          const int mid = first + (last - first) / 2;
          if (count([&](float x, int i) { return ordered(x) == lo && i <= mid; }) >= ties) last = mid;
          else first = mid + 1;
        }
        in.each(tid, NT, [&](float x, int i) {
          if (ordered(x) > lo || (ordered(x) == lo && i <= first)) sm.list[atomicAdd(&sm.found, 1)] = key_of(x, i);
        });
      }
      __syncthreads();
    }
    const int m = sm.found;
    if (tid < m) {                             // sorted by counting: keys are unique
      const u64 key = sm.list[tid];
      int at = 0;
#pragma unroll 4
      for (int k = 0; k < m; ++k) at += sm.list[k] > key;
      if (at < n) sm.top[at] = key;
    }
    if (tid == 0) sm.kept = min(m, n);
  }

  // ------------------------------------------------ the cluster's parts joined
  cluster.sync();
  {                                            // a lane a CTA, in every warp
    const Shared* o = cluster.map_shared_rank(&sm, min(lane, cs - 1));
    soft = o->soft;
    above = lane < cs ? o->rank : 0;
    if (lane >= cs) soft = {kNone * kLog2e, 0.f, 0.f};
#pragma unroll
    for (int k = kMaxCluster / 2; k > 0; k >>= 1) {
      Soft other;
      other.m = __shfl_xor_sync(0xffffffffu, soft.m, k);
      other.s = __shfl_xor_sync(0xffffffffu, soft.s, k);
      other.w = __shfl_xor_sync(0xffffffffu, soft.w, k);
      join(soft, other);
      above += __shfl_xor_sync(0xffffffffu, above, k);
    }
    soft.m = __shfl_sync(0xffffffffu, soft.m, 0);        // lanes 0 .. 7 hold it
    soft.s = __shfl_sync(0xffffffffu, soft.s, 0);
    soft.w = __shfl_sync(0xffffffffu, soft.w, 0);
  }
  float entropy;
  const bool far = !(fabsf(soft.m) <= kFar);
  if (far) {              // a careful pass: the same for all CTAs of the row
    float m = -INFINITY;
    in.each(tid, NT, [&](float x, int) { m = fmaxf(m, x); });
    auto whole = [&](auto op, float v, float* slot) {                // over the cluster
      for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
      __syncthreads();
      if (lane == 0) sm.warp[wid].m = v;
      __syncthreads();
      v = sm.warp[0].m;
      for (int w = 1; w < NW; ++w) v = op(v, sm.warp[w].m);
      cluster.sync();
      if (tid == 0) *slot = v;
      cluster.sync();
      v = *cluster.map_shared_rank(slot, 0);
      for (int c = 1; c < cs; ++c) v = op(v, *cluster.map_shared_rank(slot, c));
      return v;
    };
    auto larger = [](float p, float q) { return fmaxf(p, q); };
    auto plus = [](float p, float q) { return p + q; };
    m = whole(larger, m, &sm.most);
    float s = 0.f, w = 0.f;
    in.each(tid, NT, [&](float x, int) {
      const float d = x == m ? 0.f : x - m, e = expf(d);
      s += e;
      if (e > 0.f) w = fmaf(e, d, w);
    });
    s = whole(plus, s, &sm.most);
    w = whole(plus, w, &sm.most);
    const float ls = logf(s);
    entropy = m == -INFINITY ? 0.f : ls - w / s;
    soft.m = m;
    soft.s = ls;
  } else {
    const float ls = log2f(soft.s);
    entropy = (ls - soft.w / soft.s) * kLn2;
    soft.s = ls;
  }
  auto log_p = [&](float x) {
    if (x == -INFINITY) return x;
    const float l = far ? (x == soft.m ? 0.f : x - soft.m) - soft.s
                        : x < -1e30f ? x : (fmaf(x, kLog2e, -soft.m) - soft.s) * kLn2;
    return fminf(l, 0.f);
  };
  if (rank == 0) {
    if (tid == 0) {
      a.logp[row] = asked ? log_p(xt) : 0.f;
      if (a.entropy) a.entropy[row] = fmaxf(entropy, 0.f);
      if (a.rank) a.rank[row] = asked ? above : -1;
    }
    if (a.top > 0) {
      int have = 0, place = 0;                 // tokens of all CTAs; this thread's place among its own CTA's
      u64 key = 0;
      const int c = tid / kTop, i = tid % kTop;
      static_assert(kMaxCluster * kTop <= 256 && kTop == 32, "a thread a token");
      if (c < cs) {                            // a warp a CTA: its sorted list, behind the others' in shared memory
        const Shared* o = cluster.map_shared_rank(&sm, c);
        const int kept = o->kept;
        key = i < kept ? o->top[i] : 0;        // no token's key is 0
        sm.list[tid] = key;
      }
      __syncthreads();
      for (int k = 0; k < cs; ++k) {           // sorted lists: how many of each are before this one
        const u64* list = sm.list + k * kTop;
        int lo = 0;
#pragma unroll
        for (int step = kTop / 2; step > 0; step >>= 1) lo += list[lo + step - 1] > key ? step : 0;
        lo += list[lo] > key;
        place += lo;
        have += __popc(__ballot_sync(0xffffffffu, list[lane] != 0));
      }
      if (key != 0 && place < a.top) {
        const int64_t to = (int64_t)row * a.top + place;
        a.top_ids[to] = index_of(key);
        a.top_logp[to] = log_p(value_of(key));
      }
      for (int at = have + tid; at < a.top; at += NT) {              // fewer tokens than asked for
        const int64_t to = (int64_t)row * a.top + at;
        a.top_ids[to] = -1;
        a.top_logp[to] = -INFINITY;
      }
    }
  }
  cluster.sync();                              // no CTA leaves while its memory is read
}

template <typename T>
cudaError_t run(const LogprobArgs& a, cudaStream_t s) {
  const int sms = sm_count();
  // CTAs a row: as many of 512 threads as the GPU holds at once, two on an SM, with 4096 logits each or more; where
  // even one does not fit, of 256 threads, five on an SM, and two a row if those fit (48 rows of 131072 bf16 logits: 4 CTAs
  // of 512 threads each 12.6 us, 8 of 256 14.8, 2 of 512 14.4; 333 rows of 50257: 2 of 256 15.6, one of 256 19.8).
  int cs = 1;
  while (cs < kMaxCluster && (int64_t)a.rows * cs * 2 <= 2 * sms && a.vocab / (2 * cs) >= 4096) cs *= 2;
  const bool few = (int64_t)a.rows * cs <= 2 * sms;
  if (!few && (int64_t)a.rows * 2 <= 5 * sms && a.vocab >= 8192) cs = 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * cs));
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, logprobs_kernel<T, 512>, a) : cudaLaunchKernelEx(&cfg, logprobs_kernel<T, 256>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s) {
  return dtype == MOE_F32 ? run<float>(a, s) : run<bf16>(a, s);
}

}  // namespace moeslot
