// moe_sample: the next token of each row from its logits and one given uniform
// number: temperature, top-k, top-p, min-p.
//
//   z_i = (x_i - max x) / T,  w_i = floor(exp(z_i) 2^40)     (fp32 up to the floor)
//   descending x (equal ones by ascending index): the first top_k; of them, with
//   mass M, those whose preceding mass is below top_p M; of them those with
//   w_i >= min_p 2^40.  With kept mass K the token is the lowest index whose
//   inclusive prefix of kept w, in index order, exceeds floor(u K).
//
// The weights are 64-bit integers so that every sum is exact: no order of
// summation, split over CTAs or atomic changes a token.  2^40 keeps weights down
// to e^-27.7 of the largest.
//
// A cluster of CTAs holds a row: each CTA keeps its share of the logits in shared
// memory, so HBM is read once.  A cut (of top-k by count, of top-p by mass) is found
// over the distance d = max x - x in [0, 28 T), beyond which no token has weight:
// one pass adds the tokens up in 2048 bins of count or 1024 of mass with shared-memory
// atomics on integers, the cluster adds its CTAs' bins over distributed shared memory,
// and the tokens of the bin that holds the cut are collected and sorted by (x, index).
// Where top-k leaves 256 tokens or fewer down to the end of that bin (1024 where top-p
// follows), all of them are collected instead and the first CTA does the rest on its
// sorted list.  A bin with
// more tokens than the list holds (equal logits) is resolved by a radix descent over
// the ordered bits of x and a count of the ties in index order.
//
// What bounds it: few CTAs walk a row (48 rows of 100277 fp32 logits: 240 CTAs, 40000 logits
// an SM), so a pass over all logits costs 3 to 8 us by its instructions, and each cut two or
// three exchanges in the cluster of about 3 us; HBM's part is 4 us.  48 such rows, read from
// HBM: greedy 11.8 us, temperature alone 16.9, top-k of 50 20.5 and of 1000 31.5, top-p of 0.9
// 37.5, top-k of 1000 with top-p and min-p 36.5.  One row of 131072 bf16 logits: 4.7, 7.4, 12.3,
// 20, 23, 25.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/moeslot.h"
#include "sample_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
int sm_count();

namespace {
namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int NT = 512, NWARP = NT / 32;
constexpr int DIGIT = 2, BINS = 1 << DIGIT;    // bits a pass of the radix descent
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;                    // tokens that are collected and sorted
constexpr int kFinish = 256;                   // of top-k alone, so many that one CTA does the rest on the list
constexpr float kHead = 10.f;
constexpr int kCountBins = 2048, kMassBins = 1024, kCountShift = 13, kMassShift = 14;
constexpr int kScratch = kCountBins * 4 + 3 * kList * 8;       // bins and three lists, or the descent's counters
static_assert(BINS * NT * 8 <= kScratch, "the counters share the lists' memory");
constexpr int kShared = 230400;                // dynamic shared memory of a CTA, beside about 1 KB of static
static_assert((kShared - kScratch) / 4 / 8 * 8 * kMaxCluster >= MOE_SAMPLE_MAX_VOCAB, "the largest row must fit");
constexpr u64 kMassMask = (1ull << 48) - 1;    // a thread's counter: count in the top 16 bits, mass below

struct Exchange {                              // what a CTA shows its cluster; two of them take turns
  u64 mass[BINS];
  uint32_t count[BINS];
  float best;
  int32_t first;
};

struct Cut {                                   // kept: logits above it, and of the equal ones those up to an index
  float x;
  int32_t index;
};

__device__ __forceinline__ float value(float x) {  // NaN counts as -inf, -0 as +0
  x += 0.f;
  return x == x ? x : -INFINITY;
}
// Order-preserving key.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
// The weight of a logit: floor(2^40 e), e = 2^((x - best) log2(e) / T).  log2(e) / T is held in two
// floats, so the exponent is off by the roundings of x - best and of the product alone.  T in
// [1e-30, 1e30], best finite.
struct Softener {
  float best, hi, lo, least;
  __device__ __forceinline__ Softener(float b, float temp) : best(b), least(-30.f * temp) {
    constexpr double l2e = 1.4426950408889634074;
    constexpr float l2e_hi = (float)l2e, l2e_lo = (float)(l2e - (double)l2e_hi);
    hi = l2e_hi / temp;
    lo = (fmaf(-hi, temp, l2e_hi) + l2e_lo) / temp;
  }
  __device__ __forceinline__ float power(float x) const {
    const float d = fmaxf(x - best, least);      // 30 T below the maximum nothing is left of 2^40
    return sm103::ex2(fmaf(d, hi, d * lo));
  }
};
// floor(2^40 e) of e in [0, 1] as `high` 2^20 + `low`: the sum with 2^23, rounded towards zero, has the
// integer part in its lowest bits (64-bit conversions run at a small part of the rate).  Both come
// with the bits of 2^23 on top.
constexpr uint32_t kMagic = 0x4b000000u;
__device__ __forceinline__ void fixed(float e, uint32_t& high, uint32_t& low) {
  const float h = __fmaf_rz(e, 1048576.f, 8388608.f), l = fmaf(e, 1048576.f, 8388608.f - h);
  high = __float_as_uint(h);
  low = __float_as_uint(__fmaf_rz(l, 1048576.f, 8388608.f));
}
__device__ __forceinline__ u64 weight_of(float e) {
  uint32_t h, l;
  fixed(e, h, l);
  return ((u64)(h - kMagic) << 20) + (l - kMagic);
}
// A sum of weights, up to 4000 of them: the two parts apart.
struct Mass {
  uint32_t high = 0, low = 0;
  __device__ __forceinline__ void add(float e) {
    uint32_t h, l;
    fixed(e, h, l);
    high += h - kMagic;
    low += l - kMagic;
  }
  __device__ __forceinline__ u64 sum() const { return ((u64)high << 20) + low; }
};
__device__ __forceinline__ u64 warp_add(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
constexpr int kVec = 16 / sizeof(T);           // logits per 16 bytes
__device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {   // of values that are bf16 already
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// This CTA's share into shared memory, NaN as -inf and -0 as +0, padded with -inf to whole vectors.
// Returns the thread's maximum.
template <typename T>
__device__ __forceinline__ float load_share(const T* src, T* xs, int n) {
  constexpr int V = kVec<T>;
  float best = -INFINITY;
  const bool aligned = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  const int nv = aligned ? n / V : 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += NT) {
    float x[V];
    unpack(__ldcs(reinterpret_cast<const uint4*>(src) + i), x);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = value(x[j]);
      best = fmaxf(best, x[j]);
    }
    reinterpret_cast<uint4*>(xs)[i] = pack(x);
  }
#pragma unroll 8
  for (int i = nv * V + threadIdx.x; i < n; i += NT) {
    const float x = value((float)src[i]);
    xs[i] = (T)x;
    best = fmaxf(best, x);
  }
  for (int i = n + threadIdx.x; i < (n + V - 1) / V * V; i += NT) xs[i] = (T)-INFINITY;
  return best;
}

template <typename T>
__global__ __launch_bounds__(NT, 2) void sample_kernel(const SampleArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / CS, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  extern __shared__ __align__(16) uint8_t raw[];
  u64* bins = reinterpret_cast<u64*>(raw);                       // [BINS][NT]
  T* xs = reinterpret_cast<T*>(raw + kScratch);
  __shared__ Exchange ex[2];
  __shared__ u64 s_mass[NWARP];
  __shared__ uint32_t s_count[NWARP];
  __shared__ float s_best[NWARP];
  __shared__ u64 t_mass[BINS];                                   // the cluster's sums of a pass
  __shared__ uint32_t t_count[BINS];
  // in the counters' place: the bins of the first pass, this CTA's list, the cluster's, its prefix sums
  uint32_t* hist = reinterpret_cast<uint32_t*>(raw);             // [kCountBins], or low and high words [2][kMassBins]
  u64* own = bins + kCountBins / 2;                              // [kList] ~key << 32 | index: ascending in (-x, index)
  u64* all = own + kList;                                        // [kList]
  u64* sums = all + kList;                                       // [kList]
  __shared__ int32_t list_n;
  __shared__ Cut s_cut;
  __shared__ u64 s_kept, s_goal, s_above;
  __shared__ int32_t s_bin, s_in;
  int turn = 0;

  sm103::grid_wait();
  const int chunk = a.chunk;
  const int i0 = min(rank * chunk, a.vocab), n = min(i0 + chunk, a.vocab) - i0;
  float temp = a.temperature ? a.temperature[row] : 1.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const float u = a.u[row];
  const float mine_best = load_share(static_cast<const T*>(a.logits) + (size_t)row * a.row_stride + i0, xs, n);
  float best = mine_best;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s_best[wid] = best;
  if (tid == 0) list_n = 0;
  __syncthreads();
  best = s_best[0];
#pragma unroll
  for (int w = 1; w < NWARP; ++w) best = fmaxf(best, s_best[w]);
  if (tid == 0) ex[0].best = best;
  cluster.sync();
  best = lane < CS ? cluster.map_shared_rank(&ex[0], lane)->best : -INFINITY;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  best = __shfl_sync(0xffffffffu, best, 0);
  turn = 1;

  const bool greedy = !(temp > 0.f);
  temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
  const bool none = best == -INFINITY;                           // no token has any weight
  if (greedy || none) {
    int first = 0x7fffffff;
    for (int i = tid; i < n; i += NT)
      if ((float)(xs[i]) == best) { first = i0 + i; break; }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) s_count[wid] = (uint32_t)first;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < NWARP; ++w) first = min(first, (int)s_count[w]);
      ex[1].first = first;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < CS; ++c) first = min(first, cluster.map_shared_rank(&ex[1], c)->first);
      a.ids[row] = none ? -1 : first;
      if (a.logp) a.logp[row] = none ? -INFINITY : 0.f;
    }
    cluster.sync();                                              // no CTA leaves while its memory is read
    return;
  }

  float mine = mine_best;
  if (best == INFINITY) {                                        // infinite ones share all mass: as zeros above nothing
    for (int i = tid; i < n; i += NT) xs[i] = (float)xs[i] == INFINITY ? (T)0.f : (T)-INFINITY;
    mine = mine_best == INFINITY ? 0.f : -INFINITY;
    best = 0.f;
    __syncthreads();
  }
  const Softener soft(best, temp);
  // The cluster's sums over the threads' counters, into t_mass and t_count.
  auto add_up = [&]() {
    __syncthreads();
    if (wid < BINS) {                                            // one warp per bin
      u64 mass = 0;
      uint32_t count = 0;
#pragma unroll
      for (int t = 0; t < NT; t += 32) {
        const u64 v = bins[wid * NT + t + lane];
        mass += v & kMassMask;
        count += (uint32_t)(v >> 48);
      }
      mass = warp_add(mass);
      count = __reduce_add_sync(0xffffffffu, count);
      if (lane == 0) {
        ex[turn].mass[wid] = mass;
        ex[turn].count[wid] = count;
      }
    }
    cluster.sync();
    if (tid < BINS * kMaxCluster) {
      const int b = tid / kMaxCluster, c = tid % kMaxCluster;
      const Exchange* e = cluster.map_shared_rank(&ex[turn], c < CS ? c : 0);
      u64 m = c < CS ? e->mass[b] : 0;
      uint32_t k = c < CS ? e->count[b] : 0;
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) {
        m += __shfl_xor_sync(0xffffffffu, m, o);
        k += __shfl_xor_sync(0xffffffffu, k, o);
      }
      if (c == 0) {
        t_mass[b] = m;
        t_count[b] = k;
      }
    }
    turn ^= 1;
    __syncthreads();
  };
  auto clear = [&]() {
#pragma unroll
    for (int b = 0; b < BINS; ++b) bins[b * NT + tid] = 0;
  };
  // First digit from the top at which the running sum reaches `limit`; `above` moves past the
  // digits before it.  Every warp finds the same.
  auto find = [&](bool by_mass, u64 limit, u64& above) -> int {
    const int b = BINS - 1 - lane;
    const u64 v = lane < BINS ? by_mass ? t_mass[b] : (u64)t_count[b] : 0;
    u64 run = v;
#pragma unroll
    for (int o = 1; o < BINS; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < BINS && above + run >= limit);
    const int at = hit ? __ffs(hit) - 1 : BINS - 1;
    above += __shfl_sync(0xffffffffu, run - v, at);
    return BINS - 1 - at;
  };

  // Walks this CTA's logits, a vector at a time: f(values, index of the first).
  constexpr int V = kVec<T>;
  auto each = [&](auto&& f) {
    const int nv = (n + V - 1) / V;
    for (int v = tid; v - lane < nv; v += NT) {                  // whole warps; past the end -inf
      float x[V];
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = -INFINITY;
      if (v < nv) unpack(reinterpret_cast<const uint4*>(xs)[v], x);
      f(x, i0 + v * V);
    }
  };
  const float to_q = 16777216.f / 28.f / temp;                   // d in [0, 28 T) to [0, 2^24)
  auto q_of = [&](float x) -> uint32_t { return (uint32_t)fminf((best - x) * to_q, 16777216.f); };

  // Inclusive sum over the threads; every thread gets the total.
  auto scan = [&](u64 v, u64& total) -> u64 {
    u64 inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_mass[wid] = inc;
    __syncthreads();
    const u64 w = lane < NWARP ? s_mass[lane] : 0;
    total = warp_add(w);
    return inc + warp_add(lane < wid ? w : 0);
  };
  // The first bin at which the cluster's running sum reaches a limit: s_bin, the sum before it s_above,
  // the tokens in it s_in (by count), in every CTA.  The limit follows from the total, to which each
  // CTA adds `rest`.  Each CTA adds up a share of the bins only: reading all bins of all CTAs took most of
  // a top-p call.  False when the bins' sum stays below the limit.
  auto find_bin = [&](bool by_mass, u64 rest, u64& total, auto&& limit_of) -> bool {
    const int nb = by_mass ? kMassBins : kCountBins, Q = by_mass ? 2 : 4, per = ((nb + CS - 1) / CS + 3) / 4 * 4;
    const int b0 = min(rank * per, nb), b1 = min(b0 + per, nb), b = b0 + Q * tid;
    cluster.sync();                                              // the bins are complete
    u64 v[4] = {0, 0, 0, 0};
    if (b < b1) {
#pragma unroll 1
      for (int c0 = 0; c0 < CS; c0 += 4) {                       // four CTAs' loads in flight together
        uint4 k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* h = cluster.map_shared_rank(hist, min(c0 + c, CS - 1)) + b;
          if (by_mass) {
            const uint2 lo = *reinterpret_cast<const uint2*>(h), hi = *reinterpret_cast<const uint2*>(h + kMassBins);
            k[c] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            k[c] = *reinterpret_cast<const uint4*>(h);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c0 + c >= CS) break;
          v[0] += by_mass ? (u64)k[c].z << 32 | k[c].x : (u64)k[c].x;
          v[1] += by_mass ? (u64)k[c].w << 32 | k[c].y : (u64)k[c].y;
          v[2] += by_mass ? 0 : k[c].z;
          v[3] += by_mass ? 0 : k[c].w;
        }
      }
    }
    const u64 sum = v[0] + v[1] + v[2] + v[3];
    u64 share;
    const u64 inc = scan(sum, share);
    if (tid == 0) {
      ex[turn].mass[0] = share;
      ex[turn].mass[1] = rest;
    }
    cluster.sync();
    const Exchange* e = cluster.map_shared_rank(&ex[turn], lane < CS ? lane : 0);
    const u64 shares = lane < CS ? e->mass[0] : 0, rests = lane < CS ? e->mass[1] : 0;
    turn ^= 1;
    const u64 before = warp_add(lane < rank ? shares : 0), all = warp_add(shares);
    total = all + warp_add(rests);
    const u64 limit = limit_of(total);
    u64 run = before + inc - sum;
    if (run < limit && run + sum >= limit) {                     // one thread of the cluster tells all CTAs
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (run < limit && run + v[j] >= limit) {
          for (int c = 0; c < CS; ++c) {
            *cluster.map_shared_rank(&s_bin, c) = b0 + Q * tid + j;
            *cluster.map_shared_rank(&s_above, c) = run;
            *cluster.map_shared_rank(&s_in, c) = (int)v[j];
          }
        }
        run += v[j];
      }
    }
    cluster.sync();
    return all >= limit;
  };
  // Sorts the first m of list (at most kList, all different), ascending: few, one a thread, by counting the
  // smaller ones; more in a bitonic network (Batcher) over the next power of two, two neighbours a thread.
  // Partners within a warp meet by shuffles; only those further apart pass through memory (10 of the
  // 55 steps of 1024).
  auto sort = [&](u64* list, int m) {
    if (m <= NT / 2) {
      __syncthreads();
      const u64 x = tid < m ? list[tid] : 0;
      int place = 0;
      if (tid < m) {
#pragma unroll 8
        for (int j = 0; j < m; ++j) place += list[j] < x;
      }
      __syncthreads();
      if (tid < m) list[place] = x;
      __syncthreads();
      return;
    }
    int top = NT;
    while (top < m) top <<= 1;
    const bool on = tid < top / 2;                               // whole warps
    u64 a = ~0ull, b = ~0ull;
    __syncthreads();
    if (2 * tid < m) a = list[2 * tid];
    if (2 * tid + 1 < m) b = list[2 * tid + 1];
    for (int size = 2; size <= top; size <<= 1) {
      const bool up = ((2 * tid) & size) == 0;
      int apart = size / 4;                                      // threads between partners; 0: the thread's own two
      for (; apart >= 32; apart >>= 1) {
        __syncthreads();
        if (on) *reinterpret_cast<ulonglong2*>(list + 2 * tid) = make_ulonglong2(a, b);
        __syncthreads();
        if (on) {
          const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(list + 2 * (tid ^ apart));
          const bool least = ((tid & apart) == 0) == up;
          a = (o.x < a) == least ? o.x : a;
          b = (o.y < b) == least ? o.y : b;
        }
      }
      if (!on) continue;
      for (; apart >= 1; apart >>= 1) {
        const u64 x = __shfl_xor_sync(0xffffffffu, a, apart), y = __shfl_xor_sync(0xffffffffu, b, apart);
        const bool least = ((tid & apart) == 0) == up;
        a = (x < a) == least ? x : a;
        b = (y < b) == least ? y : b;
      }
      if ((b < a) == up) {
        const u64 x = a;
        a = b;
        b = x;
      }
    }
    __syncthreads();
    if (on) *reinterpret_cast<ulonglong2*>(list + 2 * tid) = make_ulonglong2(a, b);
    __syncthreads();
  };
  auto key_in = [](u64 item) -> uint32_t { return ~(uint32_t)(item >> 32); };
  auto x_of = [](uint32_t key) -> float { return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key); };

  // A logit below this is in no bin up to `to` (with room for rounding).
  auto floor_of = [&](uint32_t to, int shift) {
    return best - (float)((to + 1) << shift) / to_q * 1.0001f - 1e-6f * fabsf(best);
  };

  Cut cut = {-INFINITY, 0x7fffffff};                             // everything
  constexpr int EACH = kList / NT;                               // list entries of a thread
  auto passes = [&](float x, int i) { return x > cut.x || (x == cut.x && i <= cut.index); };
  // Collects the tokens of bins [from, to], those that pass the cut, and sorts them into `all` (in the
  // first CTA only, or in every one): their number, or -1 when they are too many.
  auto collect = [&](int shift, uint32_t from, uint32_t to, bool leader) -> int {
    if (tid == 0) list_n = 0;
    __syncthreads();
    // below `floor` and above `roof` nothing can be in the bins: most vectors are passed over at once
    const float floor = floor_of(to, shift);
    const float roof = best - (float)(from << shift) / to_q * 0.9999f + 1e-6f * fabsf(best);
    each([&](const float (&x)[V], int i) {
      bool any = false;
#pragma unroll
      for (int j = 0; j < V; ++j) any |= !(x[j] < floor) && !(x[j] > roof);
      if (!any) return;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (x[j] < floor || x[j] > roof) continue;
        const uint32_t q = q_of(x[j]), bin = q >> shift, key = key_of(x[j]);
        if (bin >= from && bin <= to && q < 16777216u && passes(x[j], i + j)) {
          const int at = atomicAdd(&list_n, 1);
          if (at < kList) own[at] = (u64)(~key) << 32 | (uint32_t)(i + j);
        }
      }
    });
    __syncthreads();
    if (tid == 0) ex[turn].first = list_n;
    cluster.sync();
    const int mine = lane < CS ? cluster.map_shared_rank(&ex[turn], lane)->first : 0;
    turn ^= 1;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int total = __shfl_sync(0xffffffffu, inc, kMaxCluster - 1);
    if (total > kList) return -1;                                // the same in every CTA
    if (!leader || rank == 0) {
      const int c = wid % kMaxCluster;                           // two warps per CTA of the cluster
      const int m = __shfl_sync(0xffffffffu, mine, c), at = __shfl_sync(0xffffffffu, inc - mine, c);
      const u64* r = cluster.map_shared_rank(own, min(c, CS - 1));
      for (int i = lane + 32 * (wid / kMaxCluster); i < m; i += 32 * (NWARP / kMaxCluster)) all[at + i] = r[i];
      sort(all, total);
    }
    cluster.sync();                                              // every list has been read
    return total;
  };
  auto add_to = [&](uint32_t* bin, u64 w) {                      // a 64-bit sum in two words: the carry is seen here
    const uint32_t low = (uint32_t)w, old = atomicAdd(bin, low);
    const uint32_t up = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
    if (up) atomicAdd(bin + kMassBins, up);
  };
  auto clear_hist = [&]() {
    for (int b = tid; b < kCountBins; b += NT) hist[b] = 0;
    __syncthreads();
  };

  const bool cut_p = top_p < 1.f;
  const float scale40 = 1099511627776.f;
  const float least = min_p > 0.f ? ceilf(fminf(min_p, 1.f) * scale40) / scale40 : 0.f;   // exact: scalings by 2^40
  u64 kept_mass = 0;
  for (int what = 0; what < 2; ++what) {                         // 0: top-k by count, 1: top-p by mass
    u64 limit = 0, above = 0, above_mass = 0, total;
    if (what == 0 ? !(top_k > 0 && top_k < a.vocab) : !cut_p) continue;
    clear_hist();
    if (what == 0) {
      limit = (u64)top_k;
      // The k-th largest of the threads' maxima is no larger than the k-th largest logit, and only about
      // k + k^2 / threads logits reach it: its bin bounds what has to be looked at, and where so many fit
      // the list they are all collected at once.  Otherwise the logits down to there are counted.
      int count = -1, bound = kCountBins - 1;
      const int64_t threads = CS * NT;
      // With a top-p cut to follow, the list saves a pass of weights: worth sorting up to all of it (48 rows
      // of 100277, top-k of 1000: 37 against 47 us, but without top-p 37 against 31).
      const int finish = cut_p ? kList : kFinish;
      if (2 * (int64_t)top_k <= threads) {
        const uint32_t q = q_of(mine);
        if (q < 16777216u) atomicAdd(hist + (q >> kCountShift), 1u);
        if (find_bin(false, 0, total, [&](u64) { return limit; })) {
          bound = s_bin;
          if (top_k + (int64_t)top_k * top_k / threads <= finish * 7 / 8) count = collect(kCountShift, 0, bound, true);
        }
        clear_hist();
      }
      int bin = 0;
      if (count < 0) {
        const float floor = floor_of(bound, kCountShift);
        each([&](const float (&x)[V], int) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (x[j] < floor) continue;
            const uint32_t q = q_of(x[j]);
            if (q < 16777216u) atomicAdd(hist + (q >> kCountShift), 1u);
          }
        });
        // below the limit: every token that has weight is among the first
        if (!find_bin(false, 0, total, [&](u64) { return limit; })) continue;
        above = s_above;
        bin = s_bin;
        if (above + s_in <= (u64)finish) count = collect(kCountShift, 0, bin, true);
      }
      if (count >= 0) {
        // all that may be kept, in one list
        if (rank != 0) return;
        count = min(count, top_k);
        u64 w[EACH], sum = 0;                                    // consecutive tokens a thread
        float e[EACH];
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          e[j] = EACH * tid + j < count ? soft.power(x_of(key_in(all[EACH * tid + j]))) : 0.f;
          w[j] = weight_of(e[j]);
          sum += w[j];
        }
        u64 run = scan(sum, total) - sum;
        if (tid == 0) {
          s_kept = ~0ull;
          if (cut_p) {
            const double goal = ceil((double)fmaxf(top_p, 0.f) * (double)total);
            s_kept = goal > 1.0 ? (u64)goal : 1ull;
          }
          list_n = 0;
        }
        __syncthreads();
        limit = s_kept;
        int kept = 0;                                            // the kept ones are the first of the list
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          if (w[j] && e[j] >= least && run < limit) ++kept;
          run += w[j];
          sums[EACH * tid + j] = run;
        }
        kept = __reduce_add_sync(0xffffffffu, kept);
        if (lane == 0 && kept) atomicAdd(&list_n, kept);
        __syncthreads();
        kept = list_n;
        total = sums[kept - 1];
        if (tid == 0) s_goal = u > 0.f ? (u64)((double)u * (double)total) : 0ull;
        // in the order of the index; of many only those of the bin of indices that holds the goal
        u64 before = 0;
        const bool narrow = kept > NT / 4;
        int shift = 0;
        while (a.vocab - 1 >> shift >= kMassBins) ++shift;
        if (narrow) {
          clear_hist();
#pragma unroll
          for (int j = 0; j < EACH; ++j) {
            const int i = EACH * tid + j;
            if (i < kept) add_to(hist + ((uint32_t)all[i] >> shift), w[j]);
          }
          __syncthreads();
          const u64 v0 = (u64)hist[2 * tid + kMassBins] << 32 | hist[2 * tid];
          const u64 v1 = (u64)hist[2 * tid + 1 + kMassBins] << 32 | hist[2 * tid + 1];
          u64 sum_all;
          const u64 inc = scan(v0 + v1, sum_all), goal = min(s_goal, total - 1);
          if (goal < inc && goal >= inc - v0 - v1) {             // one thread
            const bool second = goal >= inc - v1;
            s_bin = 2 * tid + second;
            s_above = second ? inc - v1 : inc - v0 - v1;
          }
          if (tid == 0) list_n = 0;
          __syncthreads();
          before = s_above;
          for (int i = tid; i < kept; i += NT) {
            const uint32_t index = (uint32_t)all[i];
            if ((int)(index >> shift) == s_bin) own[atomicAdd(&list_n, 1)] = (u64)index << 32 | (uint32_t)i;
          }
          __syncthreads();
          kept = list_n;
        } else {
          for (int i = tid; i < kept; i += NT) own[i] = (u64)(uint32_t)all[i] << 32 | (uint32_t)i;
        }
        sort(own, kept);
        const u64 goal = min(s_goal, total - 1);
        sum = 0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const int i = EACH * tid + j < kept ? (int)(uint32_t)own[EACH * tid + j] : -1;
          w[j] = i < 0 ? 0 : sums[i] - (i ? sums[i - 1] : 0);
          sum += w[j];
        }
        u64 all_mass;
        run = before + scan(sum, all_mass) - sum;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          if (run <= goal && goal < run + w[j]) {
            a.ids[row] = (int32_t)(own[EACH * tid + j] >> 32);
            if (a.logp) a.logp[row] = logf((float)w[j] / (float)total);
          }
          run += w[j];
        }
        return;
      }
    } else {
      // Bins for the tokens up to kHead T below the maximum; the mass of the others in one sum, unless
      // the cut turns out to lie among them.
      // A warp's atomic takes as long for one logit as for 32, and few are near the maximum: each thread
      // queues its own.
      constexpr int kQueue = 3 * kList * 2 / NT;
      float* queue = reinterpret_cast<float*>(own) + tid;
      int queued = 0;
      auto to_bins = [&]() {
        for (int k = 0; __any_sync(0xffffffffu, k < queued); ++k) {
          if (k >= queued) continue;
          const float x = queue[k * NT];
          const uint32_t b = min(q_of(x), 16777215u) >> kMassShift;
          add_to(hist + b, weight_of(soft.power(x)));
        }
        queued = 0;
      };
      float edge = best - kHead * temp;
      for (;;) {
        Mass rest;
        each([&](const float (&x)[V], int i) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const bool kept = passes(x[j], i + j), near = kept && x[j] > edge;
            const float e = soft.power(x[j]);
            rest.add(kept && !near ? e : 0.f);
            if (near) queue[queued++ * NT] = x[j];
          }
          if (__any_sync(0xffffffffu, queued > kQueue - V)) to_bins();
        });
        to_bins();
        u64 sum;
        scan(rest.sum(), sum);
        const bool found = find_bin(true, sum, kept_mass, [&](u64 all_mass) -> u64 {
          if (tid == 0) {                                        // one thread: fp64 is slow here
            const double goal = ceil((double)fmaxf(top_p, 0.f) * (double)all_mass);
            s_kept = goal > 1.0 ? (u64)goal : 1ull;
          }
          __syncthreads();
          return s_kept;
        });
        limit = s_kept;
        if (found || edge == -INFINITY) break;
        edge = -INFINITY;
        clear_hist();
      }
      above_mass = s_above;
    }
    const int bin = s_bin, count = collect(what == 0 ? kCountShift : kMassShift, bin, bin, false);
    if (count >= 0) {
      u64 v[EACH], sum = 0;
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        v[j] = EACH * tid + j < count ? what == 0 ? 1ull : weight_of(soft.power(x_of(key_in(all[EACH * tid + j])))) : 0ull;
        sum += v[j];
      }
      u64 run = (what == 0 ? above : above_mass) + scan(sum, total) - sum;
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        if (run < limit && run + v[j] >= limit) s_cut = Cut{x_of(key_in(all[EACH * tid + j])), (int32_t)(uint32_t)all[EACH * tid + j]};
        run += v[j];
      }
      __syncthreads();
      cut = s_cut;                                               // never above an earlier cut: its tokens alone were counted
      __syncthreads();
      continue;
    }
    // crowded: radix descent over the keys, then the index of the last tie that is kept
    constexpr int kLastShift = sizeof(T) == 2 ? 16 : 0;        // a bf16's lower key bits say nothing more
    above = 0;
    uint32_t prefix = 0;
    for (int shift = 32 - DIGIT; shift >= kLastShift; shift -= DIGIT) {
      clear();
      for (int i = tid; i < n; i += NT) {
        const float x = (float)(xs[i]);
        const uint32_t key = key_of(x);
        if (shift == 32 - DIGIT || (key >> (shift + DIGIT)) == prefix)
          bins[((key >> shift) & (BINS - 1)) * NT + tid] += (1ull << 48) + weight_of(soft.power(x));
      }
      add_up();
      prefix = prefix << DIGIT | find(what == 1, limit, above);
      __syncthreads();
    }
    uint32_t key = prefix << kLastShift;
    if (sizeof(T) == 2 && !(key >> 31)) key |= 0xffffu;        // a negative bf16's low key bits are ones
    const u64 w = weight_of(soft.power(x_of(key)));
    const u64 ties = what == 0 ? limit - above : w ? (limit - above + w - 1) / w : 1;   // kept of the equal ones
    const int span = ((n + NWARP - 1) / NWARP + 31) / 32 * 32;
    const int w0 = min(wid * span, n), w1 = min(w0 + span, n);
    uint32_t mine = 0;
    for (int i = w0 + lane; i < w1; i += 32) mine += key_of((float)(xs[i])) == key;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s_count[wid] = mine;
    __syncthreads();
    if (tid == 0) {
      uint32_t sum = 0;
      for (int v = 0; v < NWARP; ++v) sum += s_count[v];
      ex[turn].count[0] = sum;
      ex[turn].first = 0x7fffffff;
    }
    cluster.sync();
    u64 before = 0;
    for (int c = 0; c < rank; ++c) before += cluster.map_shared_rank(&ex[turn], c)->count[0];
    for (int v = 0; v < wid; ++v) before += s_count[v];
    if (before < ties && before + mine >= ties) {              // one warp of the cluster
      for (int i = w0; i < w1; i += 32) {
        const bool tie = i + lane < w1 && key_of((float)(xs[min(i + lane, w1 - 1)])) == key;
        const uint32_t votes = __ballot_sync(0xffffffffu, tie);
        if (before + __popc(votes) >= ties) {
          if (tie && before + __popc(votes & ((2u << lane) - 1)) == ties) ex[turn].first = i0 + i + lane;
          break;
        }
        before += __popc(votes);
      }
    }
    cluster.sync();
    Cut found = {x_of(key), 0x7fffffff};
    for (int c = 0; c < CS; ++c) found.index = min(found.index, cluster.map_shared_rank(&ex[turn], c)->first);
    if (found.x > cut.x || (found.x == cut.x && found.index < cut.index)) cut = found;
    cluster.sync();                                            // read by all before it is written again
  }

  // kept mass of every warp's span of indices
  const int span = ((n + NWARP - 1) / NWARP + 31) / 32 * 32;
  const int w0 = min(wid * span, n), w1 = min(w0 + span, n);
  auto kept = [&](int i, int end) -> float {                     // 2^-40 of the token's weight if it is kept
    const float x = i < end ? (float)xs[i] : -INFINITY, e = soft.power(x);
    return passes(x, i0 + i) && e >= least ? e : 0.f;
  };
  Mass spans;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) spans.add(kept(i, w1));
  u64 mass = spans.sum();
  mass = warp_add(mass);
  if (lane == 0) s_mass[wid] = mass;
  __syncthreads();
  if (tid == 0) {
    u64 sum = 0;
    for (int w = 0; w < NWARP; ++w) sum += s_mass[w];
    ex[turn].mass[0] = sum;
  }
  cluster.sync();
  u64 before = 0, total = 0;
  {
    const u64 v = lane < CS ? cluster.map_shared_rank(&ex[turn], lane)->mass[0] : 0;
    before = warp_add(lane < rank ? v : 0);
    total = warp_add(v);
    before += warp_add(lane < wid ? s_mass[lane & (NWARP - 1)] : 0);
  }
  if (tid == 0) s_goal = u > 0.f ? (u64)((double)u * (double)total) : 0ull;
  __syncthreads();
  u64 goal = s_goal;
  if (goal >= total) goal = total - 1;
  if (tid == 0) list_n = -1;
  __syncthreads();
  if (lane == 0 && goal >= before && goal < before + mass) {     // one warp of the cluster
    list_n = wid;
    s_kept = before;
  }
  __syncthreads();
  if (list_n >= 0) {                                             // its span, by all warps of its CTA
    const int sub = (span / NWARP + 31) / 32 * 32;
    const int end = min(list_n * span + span, n), v0 = min(list_n * span + wid * sub, end), v1 = min(v0 + sub, end);
    Mass sub_mass;
    for (int i = v0 + lane; i < v1; i += 32) sub_mass.add(kept(i, v1));
    const u64 part = warp_add(sub_mass.sum());
    if (lane == 0) s_mass[wid] = part;
    __syncthreads();
    u64 run = s_kept + warp_add(lane < wid ? s_mass[lane & (NWARP - 1)] : 0);
    if (goal >= run && goal < run + part) {
      for (int i = v0; i < v1; i += 32) {
        const u64 w = weight_of(kept(i + lane, v1));
        u64 inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run + inc > goal);
        if (past) {
          if (lane == __ffs(past) - 1) {
            a.ids[row] = i0 + i + lane;
            if (a.logp) a.logp[row] = logf((float)w / (float)total);
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  cluster.sync();                                                // no CTA leaves while its memory is read
}

// Clusters of c CTAs that the GPU holds at once, with one or two CTAs on an SM: a GPC's SMs do not
// divide by every size (as cudaOccupancyMaxActiveClusters says for GB300).
int clusters_at_once(int c, int per_sm) {
  static const int at[2][kMaxCluster] = {{152, 76, 46, 36, 28, 23, 15, 15}, {304, 152, 97, 74, 58, 46, 38, 36}};
  return at[per_sm - 1][c - 1];
}

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  // CTAs per row: those that need the least time by a simple account.  A CTA takes as long as kFixed
  // logits beside its own, and two on an SM get about 0.6 of its pace each; clusters that do not fit
  // at once take another round (48 rows of 100277 fp32 logits with top-p of 0.9: 3 CTAs each, two
  // rounds, 67.7 us; 5 CTAs each, two on an SM, one round, 38.1 us).
  constexpr int64_t kFixed = 12000;
  int cs = 0;
  int64_t cheapest = 0;
  for (int c = 1; c <= kMaxCluster; ++c) {
    const int64_t chunk = ((a.vocab + c - 1) / c + 7) / 8 * 8, bytes = kScratch + chunk * (int64_t)sizeof(T);
    if (bytes > kShared || (c > 1 && chunk < 2048)) continue;
    const int per_sm = 2 * (bytes + 3 * 1024) <= 228 * 1024 ? 2 : 1;   // 1 KB of each is the system's, 2 KB static
    const int64_t fit = clusters_at_once(c, per_sm), rounds = (a.rows + fit - 1) / fit;
    const bool shared = per_sm == 2 && (int64_t)a.rows * c > sm_count();
    const int64_t cost = rounds * (kFixed + (shared ? chunk * 5 / 3 : chunk));
    if (cs == 0 || cost < cheapest) {
      cs = c;
      cheapest = cost;
    }
  }
  a.chunk = ((a.vocab + cs - 1) / cs + 7) / 8 * 8;               // every share is aligned as the row is
  const size_t bytes = kScratch + (size_t)a.chunk * sizeof(T);
  static std::atomic<uint64_t> ready{0};                         // devices whose kernel has the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows * cs);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
  return dtype == MOE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace moeslot
