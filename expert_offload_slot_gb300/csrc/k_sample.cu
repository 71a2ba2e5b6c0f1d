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
// memory, so HBM is read once, and the cut of top-k and that of top-p are each
// found by a radix descent over the ordered bits of x (four bits a pass; a bf16
// logit has 16, an fp32 one 32).  In a pass every thread adds (count, mass) of its
// own logits to its own 16 counters in shared memory — no atomics — and the
// cluster adds up the counters over distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moeslot.h"
#include "sample_internal.cuh"

namespace moeslot {
namespace {
namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int NT = 512, NWARP = NT / 32, BINS = 16;
constexpr int kMaxCluster = 8;
constexpr u64 kMassMask = (1ull << 48) - 1;    // a thread's counter: count in the top 16 bits, mass below

struct Exchange {                              // what a CTA shows its cluster; two of them take turns
  u64 mass[BINS];
  uint32_t count[BINS];
  float best;
  int32_t first;
};

// Order-preserving key; -0 counts as +0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ u64 weight_of(float x, float best, float temp) {
  if (x == best) return 1ull << 40;
  const float e = expf((x - best) / temp) * 1099511627776.f;
  return e >= 1.f ? (u64)e : 0ull;             // NaN (inf temperature against -inf) compares false
}

__device__ __forceinline__ u64 warp_add(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ __launch_bounds__(NT) void sample_kernel(const SampleArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / CS, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  extern __shared__ __align__(16) uint8_t raw[];
  u64* bins = reinterpret_cast<u64*>(raw);                       // [BINS][NT]
  float* xs = reinterpret_cast<float*>(raw + sizeof(u64) * BINS * NT);
  __shared__ Exchange ex[2];
  __shared__ u64 s_mass[NWARP];
  __shared__ uint32_t s_count[NWARP];
  __shared__ float s_best[NWARP];
  __shared__ u64 t_mass[BINS];                                   // the cluster's sums of a pass
  __shared__ uint32_t t_count[BINS];
  int turn = 0;

  const int chunk = (a.vocab + CS - 1) / CS;
  const int i0 = min(rank * chunk, a.vocab), n = min(i0 + chunk, a.vocab) - i0;
  const T* src = static_cast<const T*>(a.logits) + (size_t)row * a.row_stride + i0;
  float best = -INFINITY;
  for (int i = tid; i < n; i += NT) {
    float x = (float)src[i];
    if (x != x) x = -INFINITY;
    xs[i] = x;
    best = fmaxf(best, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s_best[wid] = best;
  __syncthreads();
  best = s_best[0];
#pragma unroll
  for (int w = 1; w < NWARP; ++w) best = fmaxf(best, s_best[w]);
  if (tid == 0) ex[0].best = best;
  cluster.sync();
  for (int c = 0; c < CS; ++c) best = fmaxf(best, cluster.map_shared_rank(&ex[0], c)->best);
  turn = 1;

  const float temp = a.temperature ? a.temperature[row] : 1.f;
  const bool greedy = !(temp > 0.f);
  const bool none = best == -INFINITY;                           // no token has any weight
  if (greedy || none) {
    int first = 0x7fffffff;
    for (int i = tid; i < n; i += NT)
      if (xs[i] == best) { first = i0 + i; break; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
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

  // The cluster's (count, mass) of every 4-bit digit of the keys whose upper bits equal `prefix`.
  auto histogram = [&](uint32_t prefix, int shift) {
#pragma unroll
    for (int b = 0; b < BINS; ++b) bins[b * NT + tid] = 0;
    for (int i = tid; i < n; i += NT) {
      const float x = xs[i];
      const uint32_t key = key_of(x);
      if (shift == 28 || (key >> (shift + 4)) == prefix)
        bins[((key >> shift) & 15) * NT + tid] += (1ull << 48) + weight_of(x, best, temp);
    }
    __syncthreads();
    u64 mass = 0;
    uint32_t count = 0;
    for (int t = lane; t < NT; t += 32) {                        // one warp per digit
      const u64 v = bins[wid * NT + t];
      mass += v & kMassMask;
      count += (uint32_t)(v >> 48);
    }
    mass = warp_add(mass);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      ex[turn].mass[wid] = mass;
      ex[turn].count[wid] = count;
    }
    cluster.sync();
    if (tid < BINS) {
      u64 m = 0;
      uint32_t k = 0;
      for (int c = 0; c < CS; ++c) {
        const Exchange* e = cluster.map_shared_rank(&ex[turn], c);
        m += e->mass[tid];
        k += e->count[tid];
      }
      t_mass[tid] = m;
      t_count[tid] = k;
    }
    turn ^= 1;
    __syncthreads();
  };
  constexpr int kLastShift = sizeof(T) == 2 ? 16 : 0;            // a bf16's lower key bits say nothing more
  constexpr uint32_t kLowMask = sizeof(T) == 2 ? 0xffffu : 0u;

  // cut: keys above cut_key are kept, and the first `ties` (by index) of those equal to it
  bool cut = false;
  uint32_t cut_key = 0;
  u64 ties = 0, kept_mass = 0;
  bool have_mass = false;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f;
  for (int what = 0; what < 2; ++what) {                         // 0: top-k by count, 1: top-p by mass
    if (what == 0 ? top_k <= 0 || top_k >= a.vocab : !(top_p < 1.f)) continue;
    u64 limit = (u64)top_k, above = 0, above_mass = 0;
    uint32_t prefix = 0;
    for (int shift = 28; shift >= kLastShift; shift -= 4) {
      histogram(prefix, shift);
      if (what == 1 && shift == 28) {
        if (!have_mass) {
          kept_mass = 0;
          for (int b = 0; b < BINS; ++b) kept_mass += t_mass[b];
        }
        const double goal = ceil((double)fmaxf(top_p, 0.f) * (double)kept_mass);
        limit = goal > 1.0 ? (u64)goal : 1ull;
      }
      int digit = 0;
      for (int b = BINS - 1; b >= 0; --b) {
        const u64 v = what == 0 ? (u64)t_count[b] : t_mass[b];
        if (above + v >= limit) { digit = b; break; }
        above += v;
        above_mass += t_mass[b];
      }
      prefix = (prefix << 4) | digit;
      __syncthreads();                                           // the sums are read: the next pass may write them
    }
    uint32_t key = prefix << kLastShift;
    if (kLowMask && !(key >> 31)) key |= kLowMask;               // a negative bf16's low key bits are ones
    const u64 w = weight_of(value_of(key), best, temp);
    if (what == 0) {
      cut_key = key;
      ties = limit - above;
      kept_mass = above_mass + ties * w;
      have_mass = true;
    } else {                                                     // never below the cut of top-k: limit <= its mass
      const u64 t = w ? (limit - above + w - 1) / w : 1;
      ties = cut && key == cut_key && ties < t ? ties : t;
      cut_key = key;
    }
    cut = true;
  }

  // kept mass of every warp's span of indices
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const double least = min_p > 0.f ? (double)fminf(min_p, 1.f) * 1099511627776.0 : 0.0;
  const int span = ((n + NWARP - 1) / NWARP + 31) / 32 * 32;
  const int w0 = min(wid * span, n), w1 = min(w0 + span, n);
  u64 tie_base = 0;
  if (cut) {
    uint32_t mine = 0;
    for (int i = w0 + lane; i < w1; i += 32) mine += key_of(xs[i]) == cut_key;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s_count[wid] = mine;
    __syncthreads();
    if (tid == 0) {
      uint32_t sum = 0;
      for (int w = 0; w < NWARP; ++w) sum += s_count[w];
      ex[turn].count[0] = sum;
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) tie_base += cluster.map_shared_rank(&ex[turn], c)->count[0];
    for (int w = 0; w < wid; ++w) tie_base += s_count[w];
    turn ^= 1;
  }
  // weight of index i if it is kept, walking a warp's span 32 indices at a time
  auto kept = [&](int i, u64& tie_rank) -> u64 {
    const float x = i < w1 ? xs[i] : -INFINITY;
    const uint32_t key = key_of(x);
    const bool tie = cut && i < w1 && key == cut_key;
    const uint32_t votes = __ballot_sync(0xffffffffu, tie);
    const u64 rank_here = tie_rank + __popc(votes & ((1u << lane) - 1));
    tie_rank += __popc(votes);
    if (i >= w1 || (cut && (key < cut_key || (tie && rank_here >= ties)))) return 0;
    const u64 w = weight_of(x, best, temp);
    return (double)w >= least ? w : 0;
  };
  u64 mass = 0, tr = tie_base;
  for (int i = w0; i < w1; i += 32) mass += kept(i + lane, tr);
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
  for (int c = 0; c < CS; ++c) {
    const u64 v = cluster.map_shared_rank(&ex[turn], c)->mass[0];
    before += c < rank ? v : 0;
    total += v;
  }
  for (int w = 0; w < wid; ++w) before += s_mass[w];
  const float u = a.u[row];
  u64 goal = u > 0.f ? (u64)((double)u * (double)total) : 0ull;
  if (goal >= total) goal = total - 1;
  if (goal >= before && goal < before + mass) {                  // one warp of the cluster
    u64 run = before;
    tr = tie_base;
    for (int i = w0; i < w1; i += 32) {
      const u64 w = kept(i + lane, tr);
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
  cluster.sync();                                                // no CTA leaves while its memory is read
}

template <typename T>
cudaError_t launch(const SampleArgs& a, cudaStream_t s) {
  int cs = kMaxCluster;
  while (cs > 1 && (a.vocab + cs / 2 - 1) / (cs / 2) <= 4096) cs /= 2;
  const int chunk = (a.vocab + cs - 1) / cs;
  const size_t bytes = sizeof(u64) * BINS * NT + (size_t)chunk * 4;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows * cs);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
  return dtype == MOE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace moeslot
