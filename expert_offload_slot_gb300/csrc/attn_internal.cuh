// Internal declarations of the attention step (moe_attn_*): the handle, the
// arguments the kernels get, and the division of an attention call's work
// among its CTAs.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moeslot.h"

namespace moeslot {

moe_status set_last_error(moe_status st, const char* msg);   // text for moe_last_error()

constexpr int kAttnRowsTile = 16;     // query rows per item of the row kernel
constexpr int kAttnTile = 512;        // and of the tile kernel, by a pair of CTAs
constexpr int kAttnF32Tile = 64;      // of the fp32 kernel
constexpr int kAttnF32Few = 8;        // and of the one for few rows
// Cached + new tokens of a request, at most: positions, down to MOE_ATTN_MAX_ROWS below zero, less a window
// and plus a unit stay within 32 bits.
constexpr int kAttnMaxKeys = 0x7fffffff - 2 * MOE_ATTN_MAX_ROWS;

// floor(n / d) as (n * mul) >> shift for n below 2^31: mul = ceil(2^(31 + l) / d) with 2^l >= d; what
// that adds to n / d is below n / 2^(31 + l) <= 1 / d, too little to reach the next integer.
inline void divider(uint32_t d, uint32_t& mul, int32_t& shift) {
  int l = 0;
  while ((1u << l) < d) ++l;
  shift = 31 + l;
  mul = (uint32_t)(((1ull << shift) + d - 1) / d);
}

struct AttnArgs {
  const void* q;               // [rows][q_stride] elements, heads contiguous
  void* out;                   // [rows][Hq][D]
  const void* k_cache;         // [num_pages][Hkv][P][D]
  const void* v_cache;
  const int32_t* row_start;    // [R+1]
  const int32_t* seq_len;      // [R]
  const int32_t* table;        // [R][table_stride]
  int64_t q_stride;
  int32_t R, rows, max_new, table_stride, num_pages;
  int32_t Hq, Hkv, group, page, page_log2, window;
  float scale, scale_log2;     // softmax_scale, and times log2(e)
  // workspace: one CTA owns partial slots 2c (a piece that begins inside an item) and 2c+1
  float* part_o;               // [2 * grid][rows per slot][D]
  float2* part_ml;             // [2 * grid][rows per slot]  (running maximum, sum of exponentials)
  uint32_t* arrived;           // [grid] pieces of the split item that starts in CTA c; self-resetting
  int32_t* status;             // sticky
  uint32_t group_mul;          // token of a row without a division: (row * group_mul) >> group_shift,
  int32_t group_shift;         // exact below 2^31 (group_mul = ceil(2^group_shift / group))
  __device__ __forceinline__ int token(int row) const { return (int)(((uint64_t)(uint32_t)row * group_mul) >> group_shift); }
  __device__ __forceinline__ int head_of(int row) const { return row - token(row) * group; }
};

__device__ __forceinline__ void attn_status(int32_t* status, int32_t code) { atomicCAS(status, 0, code); }

// ------------------------------------------------------------------ the items
// An item is (request r, row tile i, kv head h).  Its rows are the query rows
// of the request's new tokens for the heads that share kv head h, token-major
// ((token, head in group) flattened), tile i taking rows [i*BM, (i+1)*BM).  Its
// keys are [lo, hi): all that any of its rows may see, cut into units of
// `unit` keys aligned to multiples of `unit`.
struct AttnRequest {
  int32_t start, n, seq;       // first row, new tokens, cached + new tokens
};

__device__ __forceinline__ AttnRequest attn_request(const AttnArgs& a, int r) {
  AttnRequest q;
  q.start = a.row_start[r];
  int n = a.row_start[r + 1] - q.start;
  int seq = a.seq_len[r];
  const int64_t cap = min((int64_t)a.table_stride * a.page, (int64_t)kAttnMaxKeys);
  bool bad = q.start < 0 || n < 0 || n > a.max_new || seq < 0 || seq > cap || (int64_t)q.start + n > a.rows;
  if (q.start < 0 || q.start >= a.rows || n < 0) n = 0;
  n = min(n, min(a.max_new, a.rows - q.start));
  if (n <= 0) n = 0;
  seq = max(0, (int)min((int64_t)seq, cap));
  if (bad) attn_status(a.status, MOE_ERR_BOUNDS);
  q.n = n;
  q.seq = seq;
  return q;
}

// Keys of row tile i: first unit and number of units (at least one, so that rows without a
// key are still written).
template <int BM>
__device__ __forceinline__ void attn_units(const AttnArgs& a, const AttnRequest& q, int i, int unit, int& u0, int& nu) {
  const int first = a.token(i * BM);                                   // first and last token of the tile
  const int last = min(q.n - 1, a.token((i + 1) * BM - 1));
  const int hi = q.seq - q.n + last + 1;
  int lo = a.window > 0 ? max(0, q.seq - q.n + first - a.window + 1) : 0;
  lo = min(lo, max(hi - 1, 0));
  u0 = lo / unit;
  nu = hi > 0 ? (hi + unit - 1) / unit - u0 : 1;
}

template <int BM>
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, const AttnRequest& q) {
  return (q.n * a.group + BM - 1) / BM;
}

// Units of a call, at most: more are refused, so that counts of them fit in 32 bits.  So many would take
// any of the kernels seconds (heads of 128: bf16, 512 rows by 128 keys a unit, 36 PFLOP or 24 s; 16 rows, 70
// TB of keys and values; fp32, 64 rows by 32 keys, 1.1 PFLOP or 36 s; 8 rows, 35 TB).
constexpr int64_t kAttnMaxUnits = 1 << 30;

// Sum over the warp's lanes of 64-bit counts below 2^52.
__device__ __forceinline__ int64_t attn_warp_sum(int64_t v) {
  const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x3ffffffu);
  const uint32_t high = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 26));
  return ((int64_t)high << 26) + low;
}

// Units of a request's row tiles for one kv head, and the most of one tile: its lane by itself where
// there are few tiles, else the whole warp for one lane after another.  2^20 rows of 1024 heads over
// 2^31 keys have 2^24 tiles of 2^26 units, so the sum has 64 bits.
template <int BM>
__device__ __forceinline__ void attn_count_units(const AttnArgs& a, const AttnRequest& q, int nt, int unit, int64_t& sum,
                                                 int& longest) {
  const int lane = threadIdx.x & 31;
  sum = longest = 0;
  int u0, nu;
  for (int i = 0; i < min(nt, 2); ++i) {
    attn_units<BM>(a, q, i, unit, u0, nu);
    sum += nu;
    longest = max(longest, nu);
  }
  for (uint32_t todo = __ballot_sync(0xffffffffu, nt > 2); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    AttnRequest x;
    x.start = 0;
    x.n = __shfl_sync(0xffffffffu, q.n, src);
    x.seq = __shfl_sync(0xffffffffu, q.seq, src);
    const int xt = __shfl_sync(0xffffffffu, nt, src);
    int64_t total = 0;
    int top = 0;
    for (int i = lane; i < xt; i += 32) {
      attn_units<BM>(a, x, i, unit, u0, nu);
      total += nu;
      top = max(top, nu);
    }
    total = attn_warp_sum(total);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == src) {
      sum = total;
      longest = top;
    }
  }
}

// How a call's units are divided among its parts (a part: a CTA, or a pair of them).  Every CTA
// finds its share by scanning the requests itself: no schedule is built ahead and nothing waits.
// Pieces: each item is cut into equal pieces, one part each, of at most L units, L the smallest
// for which the parts suffice.  Ranges: the units of all items, item after item, are cut into
// equal ranges; that balances any lengths, but a part whose range crosses an item's end has to
// finish one piece before it goes on with the next, which costs it `overhead` units.  So pieces
// are taken where L is at most that much above an even share.  An item of several pieces is
// finished by the last of its parts to arrive.
struct AttnCursor {
  int32_t r, i, h;             // item
  int32_t at;                  // unit offset inside the item
  int32_t left;                // units left in this CTA's range
  int32_t item_first;          // global index of the item's first unit
  AttnRequest q;
  int32_t u0, nu;              // the item's units
};

struct AttnSplit {
  int32_t W, parts;            // ranges
  int32_t first, count;        // pieces: first part and number of parts of this part's item (count 0: ranges)
  __device__ __forceinline__ int begin(int c) const { return (int)((int64_t)c * W / parts); }
  __device__ __forceinline__ int owner(int x) const { return (int)((((int64_t)x + 1) * parts - 1) / W); }
  __device__ __forceinline__ void pieces(const AttnCursor& c, int& c0, int& n) const {
    c0 = count ? first : owner(c.item_first);
    n = count ? count : owner(c.item_first + c.nu - 1) - c0 + 1;
  }
};

// Called by all threads of the CTA (NT of them) for part c of at most `most`.  `sm` holds 64 ints, on 8
// bytes.  False when the part has no work, or the call too many units (reported).  Up to 32 requests, every
// warp finds the part by itself with a request in each lane: no barrier stands before the first load of the
// cache.
// `join`: units that the join of one piece takes; k pieces of an item of nu units take nu / k + join k,
// so shorter ones than sqrt(join nu) are not made (tile kernel, 204 tokens over 2000 keys, 8 q heads and
// one kv head: 37 us with pieces of one unit, 24 with 4).  0 where a join takes a small part of a unit.
template <int BM, int NT, int unit, int overhead, int join>
__device__ __forceinline__ bool attn_find_range(const AttnArgs& a, int c, int most, int32_t* sm, AttnSplit& sp,
                                                AttnCursor& cur) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  constexpr int NW = NT / 32;
  const bool alone = a.R <= 32;
  const int per = alone ? 1 : (a.R + NT - 1) / NT;
  const int r0 = alone ? lane : min(tid * per, a.R), r1 = alone ? min(lane + 1, a.R) : min(r0 + per, a.R);
  AttnRequest q = {0, 0, 0};                   // of the last request looked at: the only one when per is 1
  int64_t units = 0;
  int longest = 0;
  for (int k = 0; k < per; ++k) {
    if (r0 + k < r1) q = attn_request(a, r0 + k);
    else q.n = 0;
    int64_t sum;
    attn_count_units<BM>(a, q, attn_tiles<BM>(a, q), unit, sum, longest);
    units += sum * a.Hkv;
  }
  int64_t all = 0;                             // of all requests: 32 small numbers need no adding up
  if (!alone || __any_sync(0xffffffffu, units > kAttnMaxUnits / 32)) all = attn_warp_sum(units);
  if (!alone) {
    if (lane == 0) reinterpret_cast<int2*>(sm)[wid] = make_int2((int)(all & 0x3ffffff), (int)(all >> 26));
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) all += ((int64_t)sm[2 * w + 1] << 26) + sm[2 * w];
  }
  if (all > kAttnMaxUnits) {                   // no CTA takes any
    if (tid == 0) attn_status(a.status, MOE_ERR_CAPACITY);
    return false;
  }
  const int mine = (int)units;
  // sum over the requests before this thread's, and over all
  auto scan = [&](int v, int& before, int& total) {
    int run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    before = run - v;
    total = __shfl_sync(0xffffffffu, run, 31);
    if (alone) return;
    __syncthreads();
    if (lane == 31) sm[wid] = run;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      before += w < wid ? sm[w] : 0;
      total += sm[w];
    }
  };
  int lo, W;
  scan(mine, lo, W);
  sp.W = W;
  sp.parts = max(1, min(most, W));
  sp.count = 0;
  if (W == 0) return false;
  int found[12] = {-1};                        // r, tile, head, first and last unit, request, u0, nu, first part, pieces
  bool here = false, pieces = false;
  if (per == 1) {
    const int items = attn_tiles<BM>(a, q) * a.Hkv;                    // of this thread's request
    int before, own, total;
    auto parts_for = [&](int L) -> int {       // parts for pieces of at most L units
      own = items > 0 ? items * ((longest + L - 1) / L) : 0;
      scan(own, before, total);
      return total;
    };
    int least = (W + most - 1) / most;
    if (join > 0 && alone) least = max(least, (int)sqrtf((float)join * (float)__reduce_max_sync(0xffffffffu, longest)));
    int top = least + overhead;
    if (alone) {                               // the even share, which few keys get; then all others at once
      auto fits = [&](int L) {
        return __reduce_add_sync(0xffffffffu, items > 0 ? items * ((longest + L - 1) / L) : 0) <= most;
      };
      pieces = fits(least);
      if (!pieces) {
        uint32_t fit = 0;
#pragma unroll
        for (int k = 1; k <= overhead; ++k) fit |= (uint32_t)fits(least + k) << k;
        pieces = fit != 0;
        least += pieces ? __ffs(fit) - 1 : 0;
      }
    } else if (parts_for(top) <= most) {
      pieces = true;
      while (least < top) {
        const int mid = (least + top) / 2;
        if (parts_for(mid) <= most) top = mid;
        else least = mid + 1;
      }
    }
    if (pieces) {
      parts_for(least);
      if (c >= total) return false;
      if (c >= before && c < before + own) {                           // one thread (of each warp)
        const int per_item = own / items, local = c - before, item = local / per_item, p = local - item * per_item;
        const int i = item / a.Hkv;
        int u0, nu;
        attn_units<BM>(a, q, i, unit, u0, nu);
        const int n = min(per_item, nu);                               // a short tile has fewer pieces
        here = true;
        if (p < n) {
          found[0] = r0; found[1] = i; found[2] = item - i * a.Hkv;
          found[3] = (int)((int64_t)p * nu / n); found[4] = (int)((int64_t)(p + 1) * nu / n);
          found[5] = q.start; found[6] = q.n; found[7] = q.seq; found[8] = u0; found[9] = nu;
          found[10] = c - p; found[11] = n;
        }
      }
    }
  }
  if (!pieces) {
    if (c >= sp.parts) return false;
    const int x0 = sp.begin(c), x1 = sp.begin(c + 1);
    const uint32_t has = __ballot_sync(0xffffffffu, x0 >= lo && x0 < lo + mine);
    if (has) {                                 // one warp (or each), whose lane `src` has the request
      const int src = __ffs(has) - 1;
      int r = __shfl_sync(0xffffffffu, r0, src);
      lo = __shfl_sync(0xffffffffu, lo, src);
      AttnRequest y;
      y.start = __shfl_sync(0xffffffffu, q.start, src);
      y.n = __shfl_sync(0xffffffffu, q.n, src);
      y.seq = __shfl_sync(0xffffffffu, q.seq, src);
      for (;; ++r) {                           // the whole warp, over the lane's requests and 32 tiles at a time
        if (per > 1) y = attn_request(a, r);
        const int nt = attn_tiles<BM>(a, y);
        for (int i0 = 0; i0 < nt && !__any_sync(0xffffffffu, here); i0 += 32) {
          int u0 = 0, nu = 0;
          if (i0 + lane < nt) attn_units<BM>(a, y, i0 + lane, unit, u0, nu);
          int run = nu * a.Hkv;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
          }
          const int before = lo + run - nu * a.Hkv;
          if (nu > 0 && x0 >= before && x0 < before + nu * a.Hkv) {
            const int h = (x0 - before) / nu;
            here = true;
            found[0] = r; found[1] = i0 + lane; found[2] = h;
            found[3] = x0 - before - h * nu; found[4] = found[3] + x1 - x0;
            found[5] = y.start; found[6] = y.n; found[7] = y.seq; found[8] = u0; found[9] = nu;
            found[10] = before + h * nu; found[11] = 0;
          }
          lo += __shfl_sync(0xffffffffu, run, 31);
        }
        if (__any_sync(0xffffffffu, here) || r + 1 >= a.R) break;
      }
    }
  }
  if (alone) {
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
#pragma unroll
    for (int k = 0; k < 12; ++k) found[k] = __shfl_sync(0xffffffffu, found[k], src);
  } else {
    __syncthreads();
    if (here) {
#pragma unroll
      for (int k = 0; k < 12; ++k) sm[40 + k] = found[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 12; ++k) found[k] = sm[40 + k];
  }
  if (found[0] < 0) return false;
  cur.r = found[0]; cur.i = found[1]; cur.h = found[2]; cur.at = found[3]; cur.left = found[4] - found[3];
  cur.q.start = found[5]; cur.q.n = found[6]; cur.q.seq = found[7]; cur.u0 = found[8]; cur.nu = found[9];
  cur.item_first = pieces ? 0 : found[10];
  sp.first = found[10];
  sp.count = found[11];
  return true;
}

// Units of the current item that fall into this CTA's range.
__device__ __forceinline__ int attn_piece(const AttnCursor& c) { return min(c.nu - c.at, c.left); }

// Step past the current piece; false at the end of the range.
template <int BM>
__device__ __forceinline__ bool attn_next(const AttnArgs& a, int unit, AttnCursor& c) {
  const int took = attn_piece(c);
  c.left -= took;
  if (c.left <= 0) return false;
  c.item_first += c.nu;
  c.at = 0;
  if (++c.h < a.Hkv) return true;
  c.h = 0;
  if (++c.i >= attn_tiles<BM>(a, c.q)) {
    c.i = 0;
    do {
      c.q = attn_request(a, ++c.r);
    } while (c.q.n == 0 && c.r < a.R - 1);
  }
  attn_units<BM>(a, c.q, c.i, unit, c.u0, c.nu);
  return true;
}

// Partial slot of part `part`'s piece of a split item.
__device__ __forceinline__ int attn_slot(const AttnCursor& c, int part) { return 2 * part + (c.at == 0 ? 1 : 0); }

// All threads, after the piece's partial results are stored: true in the CTA whose piece is the
// last of the item to arrive, with c0 and n the item's first CTA and number of pieces.
__device__ __forceinline__ bool attn_arrive(const AttnArgs& a, const AttnSplit& sp, const AttnCursor& c, int32_t* flag,
                                            int& c0, int& n) {
  sp.pieces(c, c0, n);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(a.arrived + c0, 1u) == (uint32_t)(n - 1);
    if (last) a.arrived[c0] = 0;
    *flag = last;
  }
  __syncthreads();
  const bool last = *flag;
  if (last) __threadfence();
  return last;
}

__device__ __forceinline__ void attn_store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void attn_store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&lo);
  u.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = u;
}

// Joins the n pieces of a split item, in piece order (so the sum does not depend on which CTA
// arrives last), and writes the item's output rows.  All threads; a warp per row, whose lanes take
// the pieces' maxima and sums at once and then D / 32 columns each; of few rows a power of two of
// warps per row, over equal shares of the pieces, joined through `scratch` (NT / 32 * (D + 4)
// floats).  U: pieces whose columns are in flight together (one token over 64000 keys, 8 q heads and
// one kv head, 152 pieces: 22 us with 8, 20 with 16; 16 decodes of few pieces 28.7 and 29.0).  LOG2: the maxima are in log2 units.
template <typename T, int D, int BM, int NT, int U, bool LOG2>
__device__ __forceinline__ void attn_join(const AttnArgs& a, const AttnCursor& c, int c0, int n, float* scratch) {
  constexpr int COLS = D / 32, NW = NT / 32, LD = D + 4;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, rows = min(BM, c.q.n * a.group - c.i * BM);
  int log_parts = 0;
  while ((rows << log_parts) * 2 <= NW && (16 << log_parts) < n) ++log_parts;
  auto slot = [&](int p) { return (size_t)(2 * (c0 + p) + (p == 0 ? 1 : 0)) * BM; };
  auto power = [](float x) { return LOG2 ? exp2f(x) : expf(x); };
  auto finish = [&](int row, float l, const float (&o)[COLS]) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int fr = c.i * BM + row;
    T* dst = static_cast<T*>(a.out) + ((size_t)(c.q.start + a.token(fr)) * a.Hq + c.h * a.group + a.head_of(fr)) * D + lane * COLS;
    if constexpr (COLS == 4) {
      attn_store4(dst, make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv));
    } else {
#pragma unroll
      for (int k = 0; k < COLS; ++k) dst[k] = (T)(o[k] * inv);
    }
  };
  for (int x = wid; x < rows << log_parts; x += NW) {
    const int row = x >> log_parts, part = x & ((1 << log_parts) - 1);
    const int q0 = (int)((int64_t)part * n >> log_parts), q1 = (int)((int64_t)(part + 1) * n >> log_parts);
    float v[U][COLS], M = -INFINITY, l = 0.f, o[COLS];
    auto load = [&](int p0) {                  // columns of pieces p0 .. p0 + U - 1
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* src = a.part_o + (slot(min(p0 + u, q1 - 1)) + row) * D + lane * COLS;
        if constexpr (COLS == 4) *reinterpret_cast<float4*>(v[u]) = __ldcg(reinterpret_cast<const float4*>(src));
        else *reinterpret_cast<float2*>(v[u]) = __ldcg(reinterpret_cast<const float2*>(src));
      }
    };
    auto stats = [&](int p) { return p < q1 ? __ldcg(a.part_ml + slot(p) + row) : make_float2(-INFINITY, 0.f); };
    float2 next = stats(q0 + lane);
    load(q0);                                  // one latency for both
#pragma unroll
    for (int k = 0; k < COLS; ++k) o[k] = 0.f;
    for (int p0 = q0; p0 < q1; p0 += 32) {
      const float2 ml = next;
      next = stats(p0 + 32 + lane);
      float top = ml.x;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float last = M;
      M = fmaxf(M, top);
      top = M == -INFINITY ? 0.f : M;
      const float f = power(last - top), g = power(ml.x - top), gl = g * ml.y;
      l *= f;
#pragma unroll
      for (int k = 0; k < COLS; ++k) o[k] *= f;
      const int m = min(32, q1 - p0);
      for (int p = 0; p < m; p += U) {
        if (p0 + p > q0) load(p0 + p);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float w = __shfl_sync(0xffffffffu, g, p + u), y = __shfl_sync(0xffffffffu, gl, p + u);
          if (p + u < m) {
            l += y;
#pragma unroll
            for (int k = 0; k < COLS; ++k) o[k] += w * v[u][k];
          }
        }
      }
    }
    if (log_parts == 0) {
      finish(row, l, o);
      continue;
    }
    float* to = scratch + wid * LD;
#pragma unroll
    for (int k = 0; k < COLS; ++k) to[lane * COLS + k] = o[k];
    if (lane == 0) {
      to[D] = M;
      to[D + 1] = l;
    }
  }
  if (log_parts == 0) return;
  __syncthreads();
  if (wid < rows) {
    const float* from = scratch + (wid << log_parts) * LD;
    const int parts = 1 << log_parts;
    float M = -INFINITY, l = 0.f, o[COLS];
    for (int k = 0; k < parts; ++k) M = fmaxf(M, from[k * LD + D]);
    const float top = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < COLS; ++k) o[k] = 0.f;
    for (int p = 0; p < parts; ++p) {
      const float g = power(from[p * LD + D] - top);
      l += g * from[p * LD + D + 1];
#pragma unroll
      for (int k = 0; k < COLS; ++k) o[k] += g * from[p * LD + lane * COLS + k];
    }
    finish(wid, l, o);
  }
  __syncthreads();                             // the scratch is read
}

// ------------------------------------------------------------------ launchers
// prepare_*: once per device, before the first launch
cudaError_t prepare_attn_f32(int D);
cudaError_t prepare_attn_rows(int D);
cudaError_t prepare_attn_tiles(int D);
cudaError_t launch_attn_f32(const AttnArgs& a, int D, int grid, cudaStream_t s);
cudaError_t launch_attn_rows(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int D, int grid,
                             cudaStream_t s);
cudaError_t launch_attn_tiles(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int D, int grid,
                              cudaStream_t s);
inline int attn_grid(int sms) { return 2 * sms; }   // CTAs of the largest grid: two per SM

struct TablesArgs {
  const int32_t *ctx, *fresh, *free_pages, *head_in;
  int32_t *table, *head_out, *row_start, *seq_len, *positions, *slots, *status;
  uint32_t* ticket;
  int32_t R, table_stride, num_free, rows, page, page_log2;
};
cudaError_t launch_attn_tables(const TablesArgs& a, cudaStream_t s);

struct QkvArgs {
  const void *qkv, *q_norm, *k_norm;
  const float* rope;           // [rope_len][rotary]: cosines, then sines
  const int32_t *positions, *slots;
  void *q, *k_cache, *v_cache;
  int32_t* status;
  int64_t qkv_stride, num_slots;
  int32_t rows, heads, Hq, Hkv, page_log2, rotary, pairs, rope_len;
  int32_t chunks, chunk_heads; // pieces of a row, and heads in each but the last
  uint32_t unit_mul;           // row of a (row, head) or (row, piece) unit without a division, as AttnArgs::group_mul
  int32_t unit_shift;
  float eps;
};
cudaError_t prepare_attn_qkv(int dtype, int D);
cudaError_t launch_attn_qkv(const QkvArgs& a, int dtype, int D, int sms, cudaStream_t s);

}  // namespace moeslot
