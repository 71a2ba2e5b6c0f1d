// Attention of new tokens over the paged cache, bf16, for few query rows per
// request (decode): the kernel streams the cache and is bound by HBM.
//
//   out[t, head] = sum_j softmax_j(scale q[t, head] . k[j]) v[j],
//   j in (pos - window, pos], pos = seq_len - new + t
//
// One pass over the keys with the running maximum m and sum l of the softmax,
// both fp32; scores and outputs accumulate in fp32.  The probabilities are
// rounded to bf16 for the second product, whose other factor is bf16: each is off
// by at most 2^-8 of itself, as the output is by its own rounding, and over many
// keys the errors average out (off from 64 bits by 1.7 to 1.8 10^-3 of the outputs'
// norm where probabilities in fp32 give 1.7).  l sums them before that rounding.
//
// An item's query rows are all heads of one kv head's group (times the new
// tokens), so that a key is read from HBM once for the whole group.  The eight
// warps of a CTA take the 16-key steps of the CTA's piece in turn; each warp
// owns a ring of stages that one lane fills by TMA (128-byte-swizzled tiles,
// two copies of 16 keys x D a stage) and keeps its own m, l, O, so no barrier
// lies in the stream; the warps join once per piece.  Both products run on
// mma.sync m16n8k16: with 16 rows or fewer of queries the tensor work is a few
// percent of the stream, and its fragments give the softmax its row in four
// lanes without a pass through tensor memory.
//
// Measured: four requests of 100000 keys, 8 kv heads (1.6 GB) 252 us, 6.4 TB/s or
// 95 % of a plain copy's rate; 16 requests of 60 to 8191 keys, 4 kv heads (114 MB)
// 29 us: 4 pass before the first load is out (lengths, then pages, each an HBM
// latency), 3 to 5 after the last (warps and pieces joined), and pieces are uneven.  One
// request of 1000 keys takes 9.0 us.  Units of 64 and 32 keys in place of 128 gain 1 % or
// nothing, and the one request then takes 0.7 and 2.7 us longer: more pieces to join.
#include "attn_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
namespace {
using namespace sm103;

constexpr int NW = 8, NT = NW * 32, BM = kAttnRowsTile, STEP = 16;
constexpr int UNIT = STEP * NW;            // keys per unit of the split: one step of every warp

template <int D>
struct RowsCfg {
  static constexpr int kHalf = STEP * 128;                 // bytes of one 64-column half of a 16-key tile
  static constexpr int kTile = kHalf * (D / 64);           // K or V of a stage
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRing = NW * kStages * 2 * kTile;
  static constexpr int kJoin = (NW / 2) * BM * D * 4;      // O of the warps being joined
  static constexpr int kBytes = kRing + kJoin + 1024;
};

template <int D>
__global__ __launch_bounds__(NT, 1) void attn_rows_kernel(const __grid_constant__ CUtensorMap mk,
                                                          const __grid_constant__ CUtensorMap mv, const AttnArgs a) {
  using C = RowsCfg<D>;
  constexpr int KS = D / 16, ND = D / 8;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) int32_t sched[64];
  __shared__ __align__(8) uint64_t bars[NW * C::kStages];
  __shared__ float sm_m[NW / 2][BM], sm_l[NW / 2][BM], all_m[NW][8], all_l[NW][8];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(smem + C::kRing);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) bar_init(bars + wid * C::kStages + s, 1);
    bar_init_done();
  }
  grid_wait();
  AttnSplit sp;
  AttnCursor c;
  if (!attn_find_range<BM, NT, UNIT, 5, 0>(a, blockIdx.x, gridDim.x, sched, sp, c)) return;

  uint64_t* bar = bars + wid * C::kStages;
  const uint32_t ring = smem_addr(smem) + wid * C::kStages * 2 * C::kTile;
  const int row_limit = (int)((int64_t)a.num_pages * a.Hkv * a.page);      // out of range: the TMA unit writes zeros
  const int g = lane >> 2, t4 = lane & 3;

  // the loading side: its own cursor, ahead of the computing side by up to kStages steps
  AttnCursor pc = c;
  int p_step = wid, p_steps = attn_piece(pc) * NW;   // steps of the piece, this warp takes wid, wid + NW, ...
  bool p_more = true;
  int p_page = 0, p_page_base = -1;                  // table entries of the next 32 steps, one per lane
  uint32_t issued = 0;
  auto issue = [&]() -> bool {                       // warp-uniform
    while (p_more && p_step >= p_steps) {
      p_more = attn_next<BM>(a, UNIT, pc);
      p_step = wid;
      p_steps = attn_piece(pc) * NW;
      p_page_base = -1;
    }
    if (!p_more) return false;
    const int idx = p_step / NW;                     // this warp's step number in the piece
    if (p_page_base < 0 || idx >= p_page_base + 32) {
      p_page_base = idx;
      const int key = (pc.u0 + pc.at) * UNIT + (p_step + lane * NW) * STEP;
      // the entries of pages that lie wholly before the tile's first window may be anything, too
      const int lo = a.window > 0 ? pc.q.seq - pc.q.n + a.token(pc.i * BM) - a.window + 1 : 0;
      p_page = p_step + lane * NW < p_steps && key < pc.q.seq && key + STEP > lo
                   ? a.table[(size_t)pc.r * a.table_stride + (key >> a.page_log2)] : -2;
    }
    const int page = __shfl_sync(0xffffffffu, p_page, idx - p_page_base);
    const int st = issued % C::kStages;
    if (lane == 0) {
      const int key = (pc.u0 + pc.at) * UNIT + p_step * STEP;
      int at = row_limit;
      if ((uint32_t)page < (uint32_t)a.num_pages) at = ((page * a.Hkv + pc.h) << a.page_log2) + (key & (a.page - 1));
      else if (page != -2) attn_status(a.status, MOE_ERR_BOUNDS);
      const uint32_t dst = ring + st * 2 * C::kTile;
      bar_expect(bar + st, 2 * C::kTile);
      tma_3d(dst, &mk, bar + st, 0, at, 0);
      tma_3d(dst + C::kTile, &mv, bar + st, 0, at, 0);
    }
    ++issued;
    p_step += NW;
    return true;
  };
  __syncwarp();
  for (int s = 0; s < C::kStages; ++s) issue();

  uint32_t taken = 0;
  bool alive = true;
  do {
    const int rows = min(BM, c.q.n * a.group - c.i * BM);
    // query rows g and g + 8 of the tile as A fragments
    uint32_t qf[KS][4];
    int pos[2], lo[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int row = g + 8 * hh, f = c.i * BM + row;
      pos[hh] = row < rows ? c.q.seq - c.q.n + a.token(f) : -1;
      lo[hh] = a.window > 0 ? max(0, pos[hh] - a.window + 1) : 0;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                 (size_t)(c.q.start + a.token(f)) * a.q_stride +
                                 (size_t)(c.h * a.group + a.head_of(f)) * D + t4 * 2;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][hh] = row < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
        qf[k][2 + hh] = row < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
      }
    }
    float o[ND][4];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[d][k] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // keys that every row of the tile sees need no mask: [all_lo, all_hi)
    const int first = a.token(c.i * BM), last = min(c.q.n - 1, a.token((c.i + 1) * BM - 1));
    const int tile_hi = c.q.seq - c.q.n + last + 1;
    const int tile_lo = a.window > 0 ? max(0, c.q.seq - c.q.n + first - a.window + 1) : 0;
    const int all_hi = c.q.seq - c.q.n + first + 1;
    const int all_lo = a.window > 0 ? max(0, c.q.seq - c.q.n + last - a.window + 1) : 0;

    const int steps = attn_piece(c) * NW;
    for (int step = wid; step < steps; step += NW) {
      const int key0 = (c.u0 + c.at) * UNIT + step * STEP;
      const int st = taken % C::kStages;
      const uint32_t parity = (taken / C::kStages) & 1;
      if (alive) {
        alive = bar_wait_warp(bar + st, parity);
        if (!alive) {
          attn_status(a.status, MOE_ERR_TIMEOUT);
          p_more = false;                    // load nothing more; the results are void
          p_step = p_steps;
        }
      }
      ++taken;
      const uint32_t kb = ring + st * 2 * C::kTile, vb = kb + C::kTile;
      if (key0 < tile_hi && key0 + STEP > tile_lo) {
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int mi = lane >> 3, rr = lane & 7;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          const int tok = (mi >> 1) * 8 + rr, ch = (k & 3) * 2 + (mi & 1);
          ldsm4(kb + (k >> 2) * C::kHalf + tok * 128 + ((ch ^ rr) << 4), b);
          mma16816(s[0], qf[k], b[0], b[1]);
          mma16816(s[1], qf[k], b[2], b[3]);
        }
        const bool mask = key0 < all_lo || key0 + STEP > all_hi;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float top = m[hh];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = s[j][2 * hh + e];
              x *= a.scale_log2;
              if (mask) {
                const int key = key0 + 8 * j + 2 * t4 + e;
                if (key < lo[hh] || key > pos[hh]) x = -INFINITY;
              }
              top = fmaxf(top, x);
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float base = top == -INFINITY ? 0.f : top;   // no key yet: every exponential is 0, not NaN
          const float f = ex2(m[hh] - base);
          m[hh] = top;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = s[j][2 * hh + e];
              x = ex2(x - base);
              sum += x;
            }
          l[hh] = l[hh] * f + sum;           // this lane's keys; the four lanes of a row are summed at the end
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            o[d][2 * hh] *= f;
            o[d][2 * hh + 1] *= f;
          }
        }
        uint32_t p[4];
        p[0] = pack_bf16(s[0][0], s[0][1]);
        p[1] = pack_bf16(s[0][2], s[0][3]);
        p[2] = pack_bf16(s[1][0], s[1][1]);
        p[3] = pack_bf16(s[1][2], s[1][3]);
        // values of keys that no row of the tile sees may be anything (0 x NaN is NaN): as zeros
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        const bool edge = key0 < tile_lo || key0 + STEP > tile_hi;
        if (edge) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = key0 + 8 * j + 2 * t4;
            keep[j] = (key >= tile_lo && key < tile_hi ? 0x0000ffffu : 0u) |
                      (key + 1 >= tile_lo && key + 1 < tile_hi ? 0xffff0000u : 0u);
          }
        }
#pragma unroll
        for (int d = 0; d < ND / 2; ++d) {
          uint32_t b[4];
          const int tok = (mi & 1) * 8 + rr, ch = (d & 3) * 2 + (mi >> 1);
          ldsm4_t(vb + (d >> 2) * C::kHalf + tok * 128 + ((ch ^ rr) << 4), b);
          if (edge) {
            b[0] &= keep[0]; b[1] &= keep[1]; b[2] &= keep[0]; b[3] &= keep[1];
          }
          mma16816(o[2 * d], p, b[0], b[1]);
          mma16816(o[2 * d + 1], p, b[2], b[3]);
        }
      }
      __syncwarp();                          // every lane has read the stage: it may be filled again
      issue();
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    }
    const bool whole = attn_piece(c) == c.nu;
    if (rows <= 8) {
      // All warps' results side by side, then a warp per row over them in order: one barrier.
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *reinterpret_cast<float2*>(join + (wid * 8 + g) * D + ((d ^ g) * 8) % D + 2 * t4) = make_float2(o[d][0], o[d][1]);
      if (t4 == 0) {
        all_m[wid][g] = m[0];
        all_l[wid][g] = l[0];
      }
      __syncthreads();
      if (wid < rows) {
        constexpr int COLS = D / 32;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, all_m[w][wid]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, x[COLS];
#pragma unroll
        for (int k = 0; k < COLS; ++k) x[k] = 0.f;
        const int col = lane * COLS, at = ((col >> 3) ^ wid) * 8 + (col & 7);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = ex2(all_m[w][wid] - base);
          sum += f * all_l[w][wid];
          const float* src = join + (w * 8 + wid) * D + at;
#pragma unroll
          for (int k = 0; k < COLS; ++k) x[k] += f * src[k];
        }
        const int fr = c.i * BM + wid;
        if (whole) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                               ((size_t)(c.q.start + a.token(fr)) * a.Hq + c.h * a.group + a.head_of(fr)) * D + col;
#pragma unroll
          for (int k = 0; k < COLS; k += 2) *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16(x[k] * inv, x[k + 1] * inv);
        } else {
          const size_t slot = (size_t)attn_slot(c, blockIdx.x) * BM + wid;
          if (lane == 0) a.part_ml[slot] = make_float2(top, sum);
#pragma unroll
          for (int k = 0; k < COLS; k += 2)
            *reinterpret_cast<float2*>(a.part_o + slot * D + col + k) = make_float2(x[k], x[k + 1]);
        }
      }
    } else {
      // join the warps in a fixed tree: 4..7 into 0..3, 2..3 into 0..1, 1 into 0
#pragma unroll
      for (int half = NW / 2; half > 0; half >>= 1) {
        if (wid >= half && wid < 2 * half) {
          float* dst = join + (wid - half) * BM * D;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int row = g + 8 * hh;
            if (t4 == 0) {
              sm_m[wid - half][row] = m[hh];
              sm_l[wid - half][row] = l[hh];
            }
#pragma unroll
            for (int d = 0; d < ND; ++d)
              *reinterpret_cast<float2*>(dst + row * D + ((d ^ g) * 8) % D + 2 * t4) = make_float2(o[d][2 * hh], o[d][2 * hh + 1]);
          }
        }
        __syncthreads();
        if (wid < half) {
          const float* src = join + wid * BM * D;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int row = g + 8 * hh;
            const float m2 = sm_m[wid][row], l2 = sm_l[wid][row];
            const float top = fmaxf(m[hh], m2), base = top == -INFINITY ? 0.f : top;
            const float f1 = ex2(m[hh] - base), f2 = ex2(m2 - base);
            m[hh] = top;
            l[hh] = l[hh] * f1 + l2 * f2;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const float2 v = *reinterpret_cast<const float2*>(src + row * D + ((d ^ g) * 8) % D + 2 * t4);
              o[d][2 * hh] = o[d][2 * hh] * f1 + v.x * f2;
              o[d][2 * hh + 1] = o[d][2 * hh + 1] * f1 + v.y * f2;
            }
          }
        }
        if (half > 1) __syncthreads();
      }
      if (wid == 0) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int row = g + 8 * hh, f = c.i * BM + row;
          if (row >= rows) continue;
          if (whole) {
            const float inv = l[hh] > 0.f ? 1.f / l[hh] : 0.f;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                                 ((size_t)(c.q.start + a.token(f)) * a.Hq + c.h * a.group + a.head_of(f)) * D + 2 * t4;
#pragma unroll
            for (int d = 0; d < ND; ++d)
              *reinterpret_cast<uint32_t*>(dst + 8 * d) = pack_bf16(o[d][2 * hh] * inv, o[d][2 * hh + 1] * inv);
          } else {
            const size_t at = (size_t)attn_slot(c, blockIdx.x) * BM + row;
            if (t4 == 0) a.part_ml[at] = make_float2(m[hh], l[hh]);
#pragma unroll
            for (int d = 0; d < ND; ++d)
              *reinterpret_cast<float2*>(a.part_o + at * D + 8 * d + 2 * t4) = make_float2(o[d][2 * hh], o[d][2 * hh + 1]);
          }
        }
      }
    }
    __syncthreads();                         // the join's memory is read: the next piece may write it
    if (!whole) {
      int c0, n;
      if (attn_arrive(a, sp, c, sched, c0, n)) attn_join<__nv_bfloat16, D, BM, NT, 16, true>(a, c, c0, n, join);
    }
  } while (attn_next<BM>(a, UNIT, c));
  if (!alive)                                // bounded: let the copies in flight land before the memory is given up
    for (uint32_t k = issued > C::kStages ? issued - C::kStages : 0; k < issued; ++k)
      bar_wait(bar + k % C::kStages, (k / C::kStages) & 1);
}

template <int D>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t s) {
  return sm103::launch(attn_rows_kernel<D>, grid, NT, RowsCfg<D>::kBytes, s, mk, mv, a);
}

template <int D>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsCfg<D>::kBytes);
}

}  // namespace

cudaError_t prepare_attn_rows(int D) { return D == 64 ? prepare<64>() : prepare<128>(); }

cudaError_t launch_attn_rows(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int D, int grid,
                             cudaStream_t s) {
  return D == 64 ? launch<64>(a, mk, mv, grid, s) : launch<128>(a, mk, mv, grid, s);
}

}  // namespace moeslot
