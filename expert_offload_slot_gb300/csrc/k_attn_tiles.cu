// Attention of new tokens over the paged cache, bf16, for chunks of tokens: both
// products on the tensor cores (tcgen05, accumulators in tensor memory).
//
//   out[t, head] = sum_j softmax_j(scale q[t, head] . k[j]) v[j],
//   j in (pos - window, pos], pos = seq_len - new + t
//
// Two CTAs work as a pair (cluster of two, tcgen05 cta_group::2).  An item is 512 query
// rows (all heads of one kv head's group, token-major, so that a key tile serves the
// whole group) as two M = 256 tiles A and B, half of each in either CTA.  Per 128 keys
// and tile: S = Q K^T (K-major operands from shared memory), the softmax in registers,
// one thread per row, P in bf16 back into tensor memory over S, and O += P V with P as
// the tensor-memory operand and V as an MN-major operand, straight from its [key][d]
// layout.  While one tile is in the softmax the tensor cores work on the other.
//
// Why pairs: each CTA keeps and loads only half of every K tile (64 of the keys) and V
// tile (half of the columns).  An SM's TMA unit brings swizzled boxes of 16, 64 and 128
// rows in at 20, 31 and 35 bytes a cycle (measured, L2 hits), and one CTA alone would want
// 64 KB every 2048 cycles that its products take; its shared memory would be busy with
// operands in all of them (128 bytes a cycle).
//
// The running maximum m is only raised (and O, l rescaled by 2^(m - m')) when a
// score exceeds it by more than 2^8: P stays below 256, which bf16 and fp32 hold
// with the same relative precision, and the rescaling of O through tensor memory
// becomes rare.  O and l are divided once at the end, so the choice of m cancels.
// P is rounded to bf16 because both factors of a product have one type; l sums it
// before that.  Against 64 bits the outputs are off by 2.0 (prompts) to 2.3 10^-3
// (1024 tokens over 31k keys) of their norm, where P in fp32 gives 1.6 to 1.7.
//
// Roles (three warpgroups in each CTA): warps 0..3 and 4..7 softmax and output of this
// CTA's rows of tiles A and B; warp 8 loads K and V by TMA, one box per page and 64-column
// half; warp 9 of the first CTA issues the MMAs.  A softmax thread holds its row's 128
// scores, so the third warpgroup gives registers up: launched with 168 each (384 x 168 =
// 64512), 216 for the first two and 72 for the third (256 x 216 + 128 x 72 = 64512).
// Tensor memory (512 columns): S/P of A, S/P of B, O of A, O of B.
//
// Measured, 32 q heads of 128: 1024 tokens over 31000 keys, 8 kv heads (531 GFLOP) 345 to 354 us,
// 1.5 PFLOP/s or 79 % of cuBLAS's burst rate and 89 % of its rate under the power cap, which such a
// call reaches.  Three prompts of 700 to 1100 tokens, 4 kv heads: 36.6 us, of which the products are 11
// and the causal tiles' masked part another 3: the first scores are there after 8.5 us (lengths, page
// table, first keys and queries from HBM one after another), a unit of 128 keys takes 1.4 us, and an
// item ends in 2.2 us of masked scores, output and the next item's first scores, two or three times a
// pair.  Two threads a row (16 softmax warps) made the large call 352 instead of 327 us, steps of 64
// keys with their scores a step ahead 357: an MMA of 64 columns reads the queries from shared memory
// as often as one of 128.
//
// With 168 registers at launch ptxas spills 464 bytes a thread (48 of stack).  They belong to the division of
// the work, which each CTA finds once before the roles begin: without the ranges 120 bytes are left, without
// any division none; leaving the joins, the masks or the rescaling out changes them by 60 or less.
#include "attn_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
namespace {
using namespace sm103;

constexpr int NT = 384, BM = kAttnTile, UNIT = 128;
constexpr float kRaise = 8.f;                  // log2 of the growth of P that m lets pass

template <int D>
struct TileCfg {
  static constexpr int kQ = 128 * D * 2;                 // this CTA's rows of a Q tile: [D / 64][128][128 bytes]
  static constexpr int kTile = 64 * D * 2;               // its half of a K tile [D / 64][64 keys][128 bytes]
                                                         // or of a V tile [128 keys][D bytes]
  static constexpr int kStages = D == 128 ? 8 : 16;
  static constexpr int kOut = 8 * 32 * 128;              // a warp's rows on their way out, 64 columns at a time
  static constexpr int kBytes = 2 * kQ + kStages * kTile + kOut + 1024;
};

// A call's work is divided in one of two ways, chosen from the lengths by every CTA alike.
// Whole: the items, longest first, are dealt out to the pairs to and fro, so that long and
// short ones meet in each; nothing is split.  Ranges: the keys of all items are cut into
// equal ranges (attn_find_range), which balances any lengths but has split items join their
// pieces through memory; that takes about as long as kJoin units.  So items stay whole unless
// the longest takes kJoin units more than an even share.
struct TileCursor : AttnCursor {
  int32_t next;                                // whole items: place of the next one in the pair's list
};
constexpr int kListMax = 32, kJoin = 6;

struct TileWork {
  AttnSplit sp;
  bool whole;
  int count;                                   // whole: items of this pair
  int4* list;                                  // [2 * kListMax] (request, head, tile, units), (first row, new, seq, first unit)
};

__device__ __forceinline__ void tile_take(const TileWork& w, TileCursor& c) {
  const int4 x = w.list[2 * c.next], y = w.list[2 * c.next + 1];
  ++c.next;
  c.r = x.x;
  c.h = x.y;
  c.i = x.z;
  c.nu = c.left = x.w;
  c.q.start = y.x;
  c.q.n = y.y;
  c.q.seq = y.z;
  c.u0 = y.w;
  c.at = 0;
  c.item_first = 0;
}

__device__ __forceinline__ bool tile_next(const AttnArgs& a, const TileWork& w, TileCursor& c) {
  if (!w.whole) return attn_next<BM>(a, UNIT, c);
  if (c.next >= w.count) return false;
  tile_take(w, c);
  return true;
}

// All threads; sm: 64 ints, scratch: 24 KB of shared memory that nothing else uses yet.
__device__ __forceinline__ bool tile_work(const AttnArgs& a, int32_t* sm, uint8_t* scratch, TileWork& w, TileCursor& c) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, G = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
  int32_t* s_nu = reinterpret_cast<int32_t*>(scratch);                   // [NT] units of each row tile
  int32_t* s_tile = s_nu + NT;                                           // [R + 1] first row tile of each request
  int4* s_req = reinterpret_cast<int4*>(scratch + 6144);                 // [R] (first row, new, seq)
  static_assert((NT + MOE_ATTN_MAX_REQUESTS + 1) * 4 <= 6144 && 6144 + MOE_ATTN_MAX_REQUESTS * 16 <= 24 * 1024, "scratch");
  const int per = (a.R + NT - 1) / NT;
  const int r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
  AttnRequest q = {0, 0, 0};
  int64_t units = 0;
  int tiles = 0, longest = 0;
  for (int k = 0; k < per; ++k) {
    q.n = 0;
    if (r0 + k < r1) {
      q = attn_request(a, r0 + k);
      s_req[r0 + k] = make_int4(q.start, q.n, q.seq, 0);
    }
    const int nt = attn_tiles<BM>(a, q);
    int64_t sum;
    int top;
    attn_count_units<BM>(a, q, nt, UNIT, sum, top);
    units += sum;
    tiles += nt;
    longest = max(longest, top);
  }
  int inc = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  units = attn_warp_sum(units);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) sm[wid] = inc;
  if (lane == 0) {
    sm[16 + wid] = (int)(units & 0x3ffffff);
    sm[32 + wid] = (int)(units >> 26);
    sm[48 + wid] = longest;
  }
  __syncthreads();
  int base = 0, T = 0, top = 0;                              // row tiles, and the most units of one
  int64_t sum = 0;                                           // units of one kv head
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    base += k < wid ? sm[k] : 0;
    T += sm[k];
    sum += ((int64_t)sm[32 + k] << 26) + sm[16 + k];
    top = max(top, sm[48 + k]);
  }
  if (sum * a.Hkv > kAttnMaxUnits) {                         // no CTA takes any
    if (tid == 0) attn_status(a.status, MOE_ERR_CAPACITY);
    return false;
  }
  const int W = (int)(sum * a.Hkv);
  if (W == 0) return false;
  const int all = T * a.Hkv;
  w.whole = top <= (W + G - 1) / G + kJoin && all <= G * kListMax;
  w.count = 0;
  if (!w.whole) {
    __syncthreads();
    return attn_find_range<BM, NT, UNIT, kJoin, 1>(a, pair, G, sm, w.sp, c);
  }
  int at = base + inc - tiles;
  for (int r = r0; r < r1; ++r) {
    s_tile[r] = at;
    at += (s_req[r].y * a.group + BM - 1) / BM;
  }
  if (tid == 0) s_tile[a.R] = T;
  __syncthreads();
  const bool sort = a.R > 1 && T <= NT;
  for (int x0 = 0; x0 < T; x0 += NT) {                       // one row tile a thread
    const int x = min(x0 + tid, T - 1);
    int lo = 0, hi = a.R - 1;
    while (lo < hi) {                                        // last request that starts at or before tile x
      const int mid = (lo + hi + 1) >> 1;
      if (s_tile[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    const int4 e = s_req[lo];
    const AttnRequest y = {e.x, e.y, e.z};
    const int i = x - s_tile[lo];
    int u0, nu, place = T - 1 - x;                           // the tiles of one request grow with i
    attn_units<BM>(a, y, i, UNIT, u0, nu);
    // Of several requests: the place by length.  More tiles than threads go as they come: then a pair
    // has so many items that they even out.
    if (sort) {
      s_nu[tid] = x0 + tid < T ? nu : 0;         // T <= NT: one turn; a tile has one unit or more
      __syncthreads();
      place = 0;
      for (int z = 0; z < T && wid * 32 < T; z += 4) {                   // the warps that have a tile
        const int4 v = *reinterpret_cast<const int4*>(s_nu + z);         // past the end: nothing counts
        place += (v.x > nu || (v.x == nu && z < x)) + (v.y > nu || (v.y == nu && z + 1 < x)) +
                 (v.z > nu || (v.z == nu && z + 2 < x)) + (v.w > nu || (v.w == nu && z + 3 < x));
      }
    }
    if (x0 + tid >= T) continue;
    int j = place * a.Hkv / G, pos = place * a.Hkv - j * G;  // round and place in it
    for (int h = 0; h < a.Hkv; ++h) {
      if (pos == ((j & 1) ? G - 1 - pair : pair)) {
        w.list[2 * j] = make_int4(lo, h, i, nu);
        w.list[2 * j + 1] = make_int4(y.start, y.n, y.seq, u0);
      }
      if (++pos == G) {
        pos = 0;
        ++j;
      }
    }
  }
  const int last = (all - 1) / G;              // round of the last item; only that round may lack one
  const int k = (last & 1) ? (last + 1) * G - 1 - pair : last * G + pair;
  w.count = last + (k < all);
  __syncthreads();
  if (w.count == 0) return false;
  c.next = 0;
  tile_take(w, c);
  return true;
}

template <int D>
__global__ __cluster_dims__(2, 1, 1) __launch_bounds__(NT, 1)
void attn_tiles_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const AttnArgs a) {
  using C = TileCfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) int32_t sched[64];
  // full, q_full and p_full are the first CTA's, who issues the products, for both; the others are of each its own
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], edge[C::kStages], drain, q_full[2], s_full[2],
      p_full[2][2], o_full[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t last_flag[2];
  __shared__ int4 items[2 * kListMax];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sq = smem_addr(smem), ring = sq + 2 * C::kQ;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)pair_rank(), part = (int)blockIdx.x / 2;
  // What needs no input comes first: with the launch set up early it runs beside the previous kernel's end.
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      bar_init(full + s, 2);
      bar_init(empty + s, 1);
      bar_init(edge + s, 1);
    }
    bar_init(&drain, 1);
    for (int t = 0; t < 2; ++t) {
      bar_init(q_full + t, 8);
      bar_init(s_full + t, 1);
      bar_init(&p_full[t][0], 8);
      bar_init(&p_full[t][1], 8);
      bar_init(o_full + t, 1);
    }
    bar_init_done();
  }
  if (wid == 9) tmem_alloc(&tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  pair_sync();                                           // the other CTA's barriers are ready, too
  tc_fence_after();
  grid_wait();
  TileWork work;
  TileCursor c;
  work.list = items;
  if (!tile_work(a, sched, smem, work, c)) {             // the same answer in every thread of the pair
    if (wid == 9) tmem_free(tmem_slot, 512);
    return;
  }
  fence_async_smem();                                    // the scratch of tile_work becomes the loads' memory
  __syncthreads();
  const uint32_t tmem = tmem_slot;

  bool alive = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {        // bounded; after a timeout nothing waits any more
    if (alive && !bar_wait(b, parity)) {
      alive = false;
      attn_status(a.status, MOE_ERR_TIMEOUT);
    }
  };

  if (wid >= 8) {
    regs_give<72>();
    if (wid == 8) {
      // ---------------------------------------------------------------- loads
      // A K tile as 64 keys x D (one box per page and 64 columns), a V tile as 128 keys x D / 2.
      const int row_limit = (int)((int64_t)a.num_pages * a.Hkv * a.page);   // out of range: zeros arrive
      const int k_box = min(a.page, 64), k_boxes = 64 / k_box, v_box = min(a.page, UNIT), v_boxes = UNIT / v_box;
      const bool my_k = lane < k_boxes * (D / 64), my_v = lane < v_boxes;
      const int k_col = lane / k_boxes, my_key = rank * 64 + lane % k_boxes * k_box;
      const uint32_t k_dst = k_col * (64 * 128) + lane % k_boxes * k_box * 128, v_dst = lane * v_box * D;
      uint32_t n = 0, edge_phase = 0;
      // Row of the cache map where a box of keys begins.  No table entry is read for one that no row of the
      // item sees: behind the first row's window it may be anything.
      auto row_of = [&](int key, int box, int lo) -> int {
        if (key >= c.q.seq || key + box <= lo) return row_limit;
        const int page = a.table[(size_t)c.r * a.table_stride + (key >> a.page_log2)];
        if ((uint32_t)page < (uint32_t)a.num_pages) return ((page * a.Hkv + c.h) << a.page_log2) + (key & (a.page - 1));
        attn_status(a.status, MOE_ERR_BOUNDS);
        return row_limit;
      };
      do {
        const int first = a.token(c.i * BM), last = min(c.q.n - 1, a.token((c.i + 1) * BM - 1));
        const int hi = c.q.seq - c.q.n + last + 1;
        const int lo = a.window > 0 ? max(0, c.q.seq - c.q.n + first - a.window + 1) : 0;
        const int units = attn_piece(c);
        // a unit's pages are looked up while the one before it is issued: a lookup takes about half as long
        // as the boxes of a unit of small pages
        const int piece0 = (c.u0 + c.at) * UNIT;
        int k_at = my_k ? row_of(piece0 + my_key, k_box, lo) : 0;
        int v_at = my_v ? row_of(piece0 + lane * v_box, v_box, lo) : 0;
        for (int j = 0; j < units; ++j) {
          const int key0 = piece0 + j * UNIT;
          const bool ahead = j + 1 < units;
          const int k_next = my_k && ahead ? row_of(key0 + UNIT + my_key, k_box, lo) : 0;
          const int v_next = my_v && ahead ? row_of(key0 + UNIT + lane * v_box, v_box, lo) : 0;
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int st = n % C::kStages;
            const uint32_t stage = ring + st * C::kTile, lead_full = lead_addr(full + st);
            wait(empty + st, ((n / C::kStages) & 1) ^ 1);
            __syncwarp();
            // Values of keys that no row of the item sees may be anything (0 x NaN is NaN): they are
            // zeroed here, in the first and last unit of an item, once they have landed.
            const bool clean = kv == 1 && (key0 < lo || key0 + UNIT > hi);
            if (clean) {
              if (lane == 0) bar_expect(edge + st, C::kTile);
              __syncwarp();
              if (my_v) tma_3d(stage + v_dst, &mv, edge + st, 0, v_at, rank);
              // the barrier's phase is that of its uses, not of the ring: one bit per stage
              wait(edge + st, (edge_phase >> st) & 1);
              edge_phase ^= 1u << st;
              __syncwarp();
              for (int r = lane; r < UNIT; r += 32) {
                if (key0 + r >= lo && key0 + r < hi) continue;
                for (int ch = 0; ch < D / 16; ++ch)
                  *reinterpret_cast<uint4*>(smem + (stage - sq) + r * D + ch * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) bar_arrive_at(lead_full);
              continue;
            }
            if (lane == 0) {
              if (rank == 0) bar_expect(full + st, 2 * C::kTile);      // of both CTAs
              else bar_arrive_at(lead_full);
            }
            __syncwarp();
            if (kv == 0 ? my_k : my_v)
              tma_3d_pair(stage + (kv == 0 ? k_dst : v_dst), kv == 0 ? &mk : &mv, lead_full, 0, kv == 0 ? k_at : v_at,
                          kv == 0 ? k_col : rank);
          }
          k_at = k_next;
          v_at = v_next;
        }
      } while (tile_next(a, work, c));
      if (!alive) {                                      // bounded: copies in flight land (on the first CTA's barriers,
        const uint64_t t0 = now_ns();                    // which this one cannot test) before the memory is given up
        while (now_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    } else if (wid == 9 && rank == 0) {
      // ----------------------------------------------------------------- MMAs
      const uint32_t lead = elect_lead();
      constexpr uint32_t kS = tc_idesc(UNIT, false), kO = tc_idesc(D, true);
      uint32_t n = 0;                                    // ring position
      uint32_t np[2] = {0, 0}, pieces[2] = {0, 0};       // P tiles and Q tiles taken
      // Descriptors are made once; a step in K or to another stage adds to their address field (units
      // of 16 bytes).
      const uint64_t q_desc = tc_desc<128>(sq), k_desc = tc_desc<128>(ring), v_desc = tc_desc<D>(ring);
      auto scores = [&](int t, uint32_t stage) {
        const uint64_t qd = q_desc + t * (C::kQ >> 4), kd = k_desc + stage * (C::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_ss(lead, tmem + t * UNIT, qd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                    kd + (((k >> 2) * (64 * 128) + (k & 3) * 32) >> 4), kS, k > 0);
        tc_commit(lead, s_full + t);
      };
      do {
        const int tiles = c.q.n * a.group - c.i * BM > 256 ? 2 : 1;
        const int units = attn_piece(c);
        wait(full + n % C::kStages, (n / C::kStages) & 1);
        for (int t = 0; t < tiles; ++t) {
          wait(q_full + t, pieces[t]++ & 1);
          __syncwarp();
          tc_fence_after();
          scores(t, n % C::kStages);
        }
        tc_commit(lead, empty + n % C::kStages);
        ++n;
        for (int j = 0; j < units; ++j) {
          const uint32_t vs = n % C::kStages, ks = (n + 1) % C::kStages;
          const bool more = j + 1 < units;
          wait(full + vs, (n / C::kStages) & 1);
          const uint64_t vd = v_desc + vs * (C::kTile >> 4);
          for (int t = 0; t < tiles; ++t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {                // P comes in halves of 64 keys
              wait(&p_full[t][h], np[t] & 1);
              __syncwarp();
              tc_fence_after();
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                tc_mma_ts(lead, tmem + 256 + t * 128, tmem + t * UNIT + k * 8, vd + k * (16 * D >> 4), kO, k > 0 || j > 0);
            }
            ++np[t];
            if (more) {
              if (t == 0) wait(full + ks, ((n + 1) / C::kStages) & 1);
              __syncwarp();
              scores(t, ks);
            } else {
              tc_commit(lead, o_full + t);
            }
          }
          tc_commit(lead, empty + vs);
          if (more) tc_commit(lead, empty + ks);
          n += more ? 2 : 1;
        }
      } while (tile_next(a, work, c));
      if (!alive) {                                      // bounded: products in flight end before the memory is given up
        tc_commit(lead, &drain);
        bar_wait(&drain, 0);
      }
    }
  } else {
    regs_take<216>();
    // ------------------------------------------------- softmax and output of tile t
    const int t = wid >> 2, row = (wid & 3) * 32 + lane;
    const int f_off = t * 256 + rank * 128;                           // this CTA's first row of the tile
    const uint32_t lanes = tmem + ((uint32_t)(wid & 3) << 21);        // this warp's 32 lanes of tensor memory
    const uint32_t s_addr = lanes + t * UNIT, o_addr = lanes + 256 + t * 128;
    const uint32_t lead_p[2] = {lead_addr(&p_full[t][0]), lead_addr(&p_full[t][1])}, lead_q = lead_addr(q_full + t);
    uint32_t ns = 0, no = 0;
    // This warp's 32 rows of tile t, 128-byte swizzled: D / 8 lanes read a row together.
    auto load_q = [&](const AttnCursor& x) {
      constexpr int PER = 32 / (D / 8);
      const int limit = x.q.n * a.group, ch = lane % (D / 8);
      const uint32_t dst = sq + t * C::kQ + (ch >> 3) * (128 * 128);
#pragma unroll
      for (int k = 0; k < 32; k += PER) {
        const int r = (wid & 3) * 32 + k + lane / (D / 8), f = x.i * BM + f_off + r, token = a.token(f);
        const bool live = f < limit;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q);
        if (live) src += (size_t)(x.q.start + token) * a.q_stride + (size_t)(x.h * a.group + f - token * a.group) * D;
        cp_async16(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + ch * 8, live ? 16 : 0);
      }
    };
    auto q_loaded = [&]() {
      cp_async_wait();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive_at(lead_q);
    };
    auto has_tile = [&](const AttnCursor& x) { return x.q.n * a.group - x.i * BM > t * 256; };
    bool mine = has_tile(c);
    if (mine) {
      load_q(c);
      q_loaded();
    }
    bool more;
    do {
      if (!mine) {                                       // an item of 256 rows or fewer has no tile B
        more = tile_next(a, work, c);
        mine = more && has_tile(c);
        if (mine) {
          load_q(c);
          q_loaded();
        }
        continue;
      }
      const int f0 = c.i * BM + f_off, f = f0 + row;
      const int rows = c.q.n * a.group - f0;             // of this CTA's part of the tile: may exceed 128, or be none
      const int base_pos = c.q.seq - c.q.n;
      const int pos = row < rows ? base_pos + a.token(f) : -1;
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      // keys that every row of this part of the tile sees need no mask
      const int all_hi = base_pos + a.token(f0) + 1;
      const int all_lo = a.window > 0 ? max(0, base_pos + a.token(f0 + max(0, min(rows, 128) - 1)) - a.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      const int units = attn_piece(c);
      for (int j = 0; j < units; ++j) {
        const int key0 = (c.u0 + c.at + j) * UNIT;
        wait(s_full + t, ns++ & 1);
        __syncwarp();
        tc_fence_after();
        float s[UNIT];
        tmem_ld64(s_addr, s);
        tmem_ld64(s_addr + 64, s + 64);
        if (key0 < all_lo || key0 + UNIT > all_hi) {
          const int first = lo - key0, last = pos - key0;
          if (a.window > 0) {
#pragma unroll
            for (int i = 0; i < UNIT; ++i)
              if (i < first) s[i] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < UNIT; ++i)
            if (i > last) s[i] = -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < UNIT; ++i) top[i & 3] = fmaxf(top[i & 3], s[i]);
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
        const bool raise = mx > m + kRaise || (m == -INFINITY && mx > m);
        float fac = 1.f;
        if (raise) {
          fac = ex2(m - mx);                             // 0 from -inf
          m = mx;
          l *= fac;
        }
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            float o[32];
            tmem_ld32(o_addr + d, o);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * fac);
            tmem_st32(o_addr + d, w);
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;     // no key yet: every exponential is 0, not NaN
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), neg2 = pack2(neg, neg);
        uint64_t sum2[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x, y;
            unpack2(fma2(pack2(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]), scale2, neg2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum2[i & 1] = add2(sum2[i & 1], pack2(x, y));
            w[i] = pack_bf16(x, y);
          }
          tmem_st32(s_addr + 32 * h, w);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_at(lead_p[h]);       // its product may start
        }
        float x, y;
        unpack2(add2(sum2[0], sum2[1]), x, y);
        l += x + y;
      }
      // Every product that reads this tile's Q has ended with the last scores; the next Q comes while the
      // last product and the output run.
      TileCursor nx = c;
      more = tile_next(a, work, nx);
      const bool next_mine = more && has_tile(nx);
      if (next_mine) load_q(nx);
      wait(o_full + t, no++ & 1);
      __syncwarp();
      tc_fence_after();
      const bool whole = units == c.nu;
      // Partial results lie a warp's 32 rows together, [D / 4][32 rows][4]: a warp stores and loads 512
      // contiguous bytes at a time, a row staying in its thread.
      const size_t warp_rows = f_off + (wid & 3) * 32;
      const size_t part_slot = (size_t)attn_slot(c, part) * BM;
      float* part_dst = a.part_o + (part_slot + warp_rows) * D + lane * 4;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      __nv_bfloat16* out_rows[8];                        // this lane's part of rows lane / 8, + 4, ... of the warp's
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = f0 + (wid & 3) * 32 + 4 * k + lane / 8, token = a.token(r);
        out_rows[k] = static_cast<__nv_bfloat16*>(a.out) +
                      ((size_t)(c.q.start + token) * a.Hq + c.h * a.group + r - token * a.group) * D + lane % 8 * 8;
      }
      // A row per thread would touch 32 lines with every store; turned in shared memory, a store
      // writes 128 bytes of each of four rows.
      const uint32_t turn = sq + 2 * C::kQ + C::kStages * C::kTile + wid * (32 * 128);
      auto send = [&](const uint32_t* w, int d) {        // 64 columns of the warp's rows from column d on
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
          *reinterpret_cast<uint4*>(smem + (turn - sq) + lane * 128 + ((ch ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + lane / 8, ch = lane % 8;
          const uint4 v = *reinterpret_cast<const uint4*>(smem + (turn - sq) + r * 128 + ((ch ^ (r & 7)) << 4));
          const int tr = (wid & 3) * 32 + r;
          if (tr < rows) *reinterpret_cast<uint4*>(out_rows[k] + d) = v;
        }
      };
#pragma unroll 1
      for (int d = 0; d < D; d += 64) {
        float o[64];
        __syncwarp();
        tmem_ld64(o_addr + d, o);
        if (d + 64 == D && next_mine) q_loaded();        // the next item's first scores run beside the rest
        if (whole) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
          send(w, d);
        } else if (row < rows) {
#pragma unroll
          for (int i = 0; i < 64; i += 4)
            attn_store4(part_dst + (d + i) * 32, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
        }
      }
      if (!whole && rows > 0) {
        if (row < rows) a.part_ml[part_slot + f_off + row] = make_float2(m, l);
        int c0, n;
        work.sp.pieces(c, c0, n);
        uint32_t* counter = a.arrived + 4 * c0 + 2 * t + rank;
        __threadfence();
        named_sync(1 + t, 128);
        if (tid == t * 128) {
          const bool last = atomicAdd(counter, 1u) == (uint32_t)(n - 1);
          if (last) *counter = 0;
          last_flag[t] = last;
        }
        named_sync(1 + t, 128);
        if (last_flag[t]) {                              // the last of the item's pieces to arrive joins these rows, in
          __threadfence();                               // piece order (rows past the end as they come: not sent)
          auto slot = [&](int p) { return (size_t)(2 * (c0 + p) + (p == 0)) * BM; };
          const float2* ml = a.part_ml + f_off + row;
          float M = -INFINITY, sum = 0.f;
#pragma unroll 4
          for (int p = 0; p < n; ++p) M = fmaxf(M, __ldcg(ml + slot(p)).x);
          const float top = M == -INFINITY ? 0.f : M;
#pragma unroll 4
          for (int p = 0; p < n; ++p) {
            const float2 v = __ldcg(ml + slot(p));
            sum += ex2(v.x - top) * v.y;
          }
          const float in = sum > 0.f ? 1.f / sum : 0.f;
          const float* src = a.part_o + warp_rows * D + lane * 4;
#pragma unroll 1
          for (int d = 0; d < D; d += 64) {
            float o[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i] = 0.f;
#pragma unroll 1
            for (int p = 0; p < n; ++p) {
              const float g = ex2(__ldcg(ml + slot(p)).x - top) * in;
              float4 v[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                v[i] = __ldcg(reinterpret_cast<const float4*>(src + slot(p) * D + (d + 4 * i) * 32));
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                o[4 * i] += g * v[i].x;
                o[4 * i + 1] += g * v[i].y;
                o[4 * i + 2] += g * v[i].z;
                o[4 * i + 3] += g * v[i].w;
              }
            }
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
            send(w, d);
          }
        }
      }
      more = tile_next(a, work, c);
      mine = next_mine;
    } while (more);
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();                                           // neither CTA's memory or barriers are used any more
  tc_fence_after();
  if (wid == 9) tmem_free(tmem, 512);
}

template <int D>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t s) {
  return sm103::launch(attn_tiles_kernel<D>, grid, NT, TileCfg<D>::kBytes, s, mk, mv, a);
}

template <int D>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<D>::kBytes);
}

}  // namespace

cudaError_t prepare_attn_tiles(int D) { return D == 64 ? prepare<64>() : prepare<128>(); }

cudaError_t launch_attn_tiles(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int D, int grid,
                              cudaStream_t s) {
  return D == 64 ? launch<64>(a, mk, mv, grid, s) : launch<128>(a, mk, mv, grid, s);
}

}  // namespace moeslot
