// Attention of new tokens over the paged cache, fp32: q, caches and out are
// fp32 and every product and sum is fp32 on the CUDA cores (the tensor cores'
// tf32 would drop 13 bits of each factor).
//
//   out[t, head] = sum_j softmax_j(scale q[t, head] . k[j]) v[j],
//   j in (pos - window, pos], pos = seq_len - new + t
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// a tile's scores s raise m to m', and O and l are scaled by exp(m - m').
// A CTA holds 64 query rows (all heads of a kv head's group together, so that a key
// read once serves the whole group) and walks its units of 32 keys.  A thread has
// four rows with two keys' scores, then with D / 16 output columns, so that its 32
// products need six (then three) reads of shared memory; two CTAs share an SM, so
// that one's loads run beside the other's products.  With half the rows and one product
// for each read of K and V a 512-token prompt (32 q heads) took 225 us; so it takes 92 to 95 us,
// 23 TFLOP/s, and the last 200 of 2000 tokens 203 instead of 573 us, 31 TFLOP/s.  Shared memory and the
// instructions bound it together: its pipe is busy 66 % of the time, issue slots 67 %, the FMA pipe 52 %, as
// loads of a tile and its products take turns behind two barriers.
#include "attn_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
namespace {

constexpr int NT = 256, BM = kAttnF32Tile, BN = 32;

template <int D>
struct F32Cfg {
  static constexpr int LD = D + 4, LP = BM + 4;       // padded rows: eight rows' float4 reads hit 32 banks
  static constexpr int kBytes = (BM * LD + 2 * BN * LD + BN * LP) * 4;
};

template <int D>
__global__ __launch_bounds__(NT, 2) void attn_f32_kernel(const AttnArgs a) {
  using C = F32Cfg<D>;
  constexpr int LD = C::LD, LP = C::LP, COLS = D / 16;
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;                         // [BM][LD]
  float* sk = sq + BM * LD;                 // [BN][LD]
  float* sv = sk + BN * LD;                 // [BN][LD]
  float* prob = sv + BN * LD;               // [BN][LP] probabilities, rows innermost
  __shared__ __align__(8) int32_t sched[64];
  sm103::grid_wait();
  AttnSplit sp;
  AttnCursor c;
  if (!attn_find_range<BM, NT, BN, 4, 0>(a, blockIdx.x, gridDim.x, sched, sp, c)) return;
  const int tid = threadIdx.x, tx = tid % 16, r0 = tid / 16 * 4;
  do {
    const int rows = min(BM, c.q.n * a.group - c.i * BM);
    const int first = a.token(c.i * BM), last = min(c.q.n - 1, a.token((c.i + 1) * BM - 1));
    const int tile_hi = c.q.seq - c.q.n + last + 1;
    const int tile_lo = a.window > 0 ? max(0, c.q.seq - c.q.n + first - a.window + 1) : 0;
    int pos[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pos[i] = r0 + i < rows ? c.q.seq - c.q.n + a.token(c.i * BM + r0 + i) : -1;
      lo[i] = a.window > 0 ? max(0, pos[i] - a.window + 1) : 0;
    }
    __syncthreads();
    for (int e = tid * 4; e < BM * D; e += NT * 4) {
      const int rr = e / D, d = e % D, f = c.i * BM + rr;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows)
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (size_t)(c.q.start + a.token(f)) * a.q_stride +
                                             (size_t)(c.h * a.group + a.head_of(f)) * D + d);
      *reinterpret_cast<float4*>(sq + rr * LD + d) = v;
    }
    float o[4][COLS], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < COLS; ++k) o[i][k] = 0.f;
    }
    const int piece = attn_piece(c);
    for (int u = 0; u < piece; ++u) {
      const int key0 = (c.u0 + c.at + u) * BN;
      __syncthreads();
      constexpr int LANES = D / 4;
#pragma unroll 4
      for (int kr = tid / LANES; kr < BN; kr += NT / LANES) {
        const int key = key0 + kr, d = tid % LANES * 4;
        size_t at = 0;
        uint32_t bytes = 0;
        if (key >= tile_lo && key < tile_hi) {   // what no row of the tile sees may hold anything: it counts as zero
          const int page = a.table[(size_t)c.r * a.table_stride + (key >> a.page_log2)];
          if ((uint32_t)page < (uint32_t)a.num_pages) {
            at = ((((size_t)page * a.Hkv + c.h) << a.page_log2) + (key & (a.page - 1))) * D + d;
            bytes = 16;
          } else {
            attn_status(a.status, MOE_ERR_BOUNDS);
          }
        }
        const uint32_t dst = sm103::smem_addr(sk + kr * LD + d);
        sm103::cp_async16(dst, static_cast<const float*>(a.k_cache) + at, bytes);
        sm103::cp_async16(dst + BN * LD * 4, static_cast<const float*>(a.v_cache) + at, bytes);
      }
      sm103::cp_async_wait();
      __syncthreads();
      float s[4][2] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(sk + tx * LD + d);
        const float4 k1 = *reinterpret_cast<const float4*>(sk + (tx + 16) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(sq + (r0 + i) * LD + d);
          s[i][0] += x.x * k0.x + x.y * k0.y + x.z * k0.z + x.w * k0.w;
          s[i][1] += x.x * k1.x + x.y * k1.y + x.z * k1.z + x.w * k1.w;
        }
      }
      float p[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = key0 + tx + 16 * j;
          s[i][j] = key >= lo[i] && key <= pos[i] ? s[i][j] * a.scale : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float base = top == -INFINITY ? 0.f : top;   // no key yet: every exponential is 0, not NaN
        const float f = expf(m[i] - base);
        m[i] = top;
#pragma unroll
        for (int j = 0; j < 2; ++j) p[j][i] = expf(s[i][j] - base);
        l[i] = l[i] * f + (p[0][i] + p[1][i]);             // this thread's keys; the row's 16 threads sum at the end
#pragma unroll
        for (int k = 0; k < COLS; ++k) o[i][k] *= f;
      }
      // a row's probabilities are written and read by the same 16 lanes
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float4*>(prob + (tx + 16 * j) * LP + r0) = make_float4(p[j][0], p[j][1], p[j][2], p[j][3]);
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < BN; ++k) {
        const float4 w = *reinterpret_cast<const float4*>(prob + k * LP + r0);
#pragma unroll
        for (int j = 0; j < COLS / 4; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(sv + k * LD + tx * 4 + 64 * j);
          const float pw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i][4 * j] += pw[i] * v.x; o[i][4 * j + 1] += pw[i] * v.y;
            o[i][4 * j + 2] += pw[i] * v.z; o[i][4 * j + 3] += pw[i] * v.w;
          }
        }
      }
    }
    const bool whole = piece == c.nu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
      if (r0 + i >= rows) continue;
      const int fr = c.i * BM + r0 + i;
      const float inv = whole ? (l[i] > 0.f ? 1.f / l[i] : 0.f) : 1.f;
      const size_t slot = (size_t)attn_slot(c, blockIdx.x) * BM + r0 + i;
      float* dst = whole ? static_cast<float*>(a.out) +
                               ((size_t)(c.q.start + a.token(fr)) * a.Hq + c.h * a.group + a.head_of(fr)) * D
                         : a.part_o + slot * D;
      if (!whole && tx == 0) a.part_ml[slot] = make_float2(m[i], l[i]);
#pragma unroll
      for (int j = 0; j < COLS / 4; ++j)
        attn_store4(dst + tx * 4 + 64 * j, make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                                                       o[i][4 * j + 3] * inv));
    }
    if (!whole) {
      int c0, n;
      if (attn_arrive(a, sp, c, sched, c0, n)) attn_join<float, D, BM, NT, 8, false>(a, c, c0, n, prob);
    }
  } while (attn_next<BM>(a, BN, c));
}

// ------------------------------------------------- few query rows per request (decode)
// Eight query rows a CTA: the kernel above computes 64 for every key (16 requests of 5000 keys, 8 kv
// heads: 707 us with 32; this one 185 us, 3.5 TB/s, half of HBM's rate: four barriers a tile of 32 keys keep
// its products and softmax apart, with shared memory's pipe busy 59 % of the time and issue slots 54 %).
// Tiles of 32 keys come by 16-byte asynchronous copies into three stages; two CTAs share an SM, so that the
// copies and the phases between barriers of one run beside the other's.  Scores: a lane has one key, a warp an eighth of D, so that K is read once from
// shared memory and q by broadcast; softmax: a warp per row; output: a thread per column and group
// of keys, eight rows in its registers.
constexpr int FM = kAttnF32Few, FN = 32, FSTAGES = 3, DQ = NT / 32;

template <int D>
struct FewCfg {
  static constexpr int LD = D + 4;
  static constexpr int KG = NT / D;                              // groups of keys of the output phase
  static constexpr int kStage = 2 * FN * LD;                     // floats: K and V
  static constexpr int kBytes = (FSTAGES * kStage + FM * D + DQ * FM * FN + FN * FM + 4 * FM) * 4;
};

template <int D>
__global__ __launch_bounds__(NT, 2) void attn_f32_few_kernel(const AttnArgs a) {
  using C = FewCfg<D>;
  constexpr int LD = C::LD, KG = C::KG;
  extern __shared__ __align__(16) float smem[];
  float* stage = smem;                                           // [FSTAGES][K, V][FN][LD]
  float* sq = stage + FSTAGES * C::kStage;                       // [FM][D]
  float* part = sq + FM * D;                                     // [DQ][FM][FN] scores over a part of D each
  float* prob = part + DQ * FM * FN;                             // [FN][FM]
  float* fac = prob + FN * FM;                                   // [FM] scale of this step; then m, l
  __shared__ __align__(8) int32_t sched[64];
  sm103::grid_wait();
  AttnSplit sp;
  AttnCursor c;
  if (!attn_find_range<FM, NT, FN, 4, 0>(a, blockIdx.x, gridDim.x, sched, sp, c)) return;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int col = tid % D, kg = tid / D;                         // output phase
  AttnCursor pc = c;                                             // the loading side, FSTAGES - 1 units ahead
  int p_unit = 0;
  bool p_more = true;
  auto issue = [&](int st) {
    if (p_more && p_unit >= attn_piece(pc)) {
      p_more = attn_next<FM>(a, FN, pc);
      p_unit = 0;
    }
    if (p_more) {
      const int first = a.token(pc.i * FM), last = min(pc.q.n - 1, a.token((pc.i + 1) * FM - 1));
      const int hi = pc.q.seq - pc.q.n + last + 1;
      const int lo = a.window > 0 ? max(0, pc.q.seq - pc.q.n + first - a.window + 1) : 0;
      const int key0 = (pc.u0 + pc.at + p_unit) * FN;
      constexpr int LANES = D / 4;
      for (int kr = tid / LANES; kr < FN; kr += NT / LANES) {    // what no row sees may be anything: zeros come
        const int key = key0 + kr, d = tid % LANES * 4;
        size_t at = 0;
        uint32_t bytes = 0;
        if (key >= lo && key < hi) {
          const int page = a.table[(size_t)pc.r * a.table_stride + (key >> a.page_log2)];
          if ((uint32_t)page < (uint32_t)a.num_pages) {
            at = ((((size_t)page * a.Hkv + pc.h) << a.page_log2) + (key & (a.page - 1))) * D + d;
            bytes = 16;
          } else {
            attn_status(a.status, MOE_ERR_BOUNDS);
          }
        }
        const uint32_t dst = sm103::smem_addr(stage + st * C::kStage + kr * LD + d);
        sm103::cp_async16(dst, static_cast<const float*>(a.k_cache) + at, bytes);
        sm103::cp_async16(dst + FN * LD * 4, static_cast<const float*>(a.v_cache) + at, bytes);
      }
      ++p_unit;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s < FSTAGES - 1; ++s) issue(s);
  int st = 0;
  do {
    const int rows = min(FM, c.q.n * a.group - c.i * FM);
    __syncthreads();
    for (int e = tid * 4; e < FM * D; e += NT * 4) {
      const int rr = e / D, d = e % D, f = c.i * FM + rr;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows)
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (size_t)(c.q.start + a.token(f)) * a.q_stride +
                                             (size_t)(c.h * a.group + a.head_of(f)) * D + d);
      *reinterpret_cast<float4*>(sq + e) = v;
    }
    // softmax phase: warp w has row w
    const int f = c.i * FM + wid, pos = wid < rows ? c.q.seq - c.q.n + a.token(f) : -1;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    float m = -INFINITY, l = 0.f, o[FM];
#pragma unroll
    for (int r = 0; r < FM; ++r) o[r] = 0.f;
    const int piece = attn_piece(c);
    for (int u = 0; u < piece; ++u) {
      const int key0 = (c.u0 + c.at + u) * FN;
      issue((st + FSTAGES - 1) % FSTAGES);                       // the stage read last: the barrier below was after it
      asm volatile("cp.async.wait_group %0;" ::"n"(FSTAGES - 1) : "memory");
      __syncthreads();
      const float* sk = stage + st * C::kStage;
      const float* sv = sk + FN * LD;
      {
        constexpr int PART = D / DQ;                             // a warp: 32 keys, a part of D
        float s[FM];
#pragma unroll
        for (int r = 0; r < FM; ++r) s[r] = 0.f;
#pragma unroll
        for (int d = wid * PART; d < (wid + 1) * PART; d += 4) {
          const float4 k = *reinterpret_cast<const float4*>(sk + lane * LD + d);
#pragma unroll
          for (int r = 0; r < FM; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(sq + r * D + d);
            s[r] += x.x * k.x + x.y * k.y + x.z * k.z + x.w * k.w;
          }
        }
#pragma unroll
        for (int r = 0; r < FM; ++r) part[(wid * FM + r) * FN + lane] = s[r];
      }
      __syncthreads();
      {
        const int key = key0 + lane;
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < DQ; ++k) x += part[(k * FM + wid) * FN + lane];
        x = key >= lo && key <= pos ? x * a.scale : -INFINITY;
        float top = fmaxf(m, x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float base = top == -INFINITY ? 0.f : top;         // no key yet: every exponential is 0, not NaN
        const float scale = expf(m - base), p = expf(x - base);
        m = top;
        l = l * scale + p;                                       // this lane's keys
        prob[lane * FM + wid] = p;
        if (lane == 0) fac[wid] = scale;
      }
      __syncthreads();
      {
        const float4 f0 = *reinterpret_cast<const float4*>(fac), f1 = *reinterpret_cast<const float4*>(fac + 4);
        o[0] *= f0.x; o[1] *= f0.y; o[2] *= f0.z; o[3] *= f0.w;
        o[4] *= f1.x; o[5] *= f1.y; o[6] *= f1.z; o[7] *= f1.w;
#pragma unroll 8
        for (int k = kg * (FN / KG); k < (kg + 1) * (FN / KG); ++k) {
          const float v = sv[k * LD + col];
          const float4 p0 = *reinterpret_cast<const float4*>(prob + k * FM), p1 = *reinterpret_cast<const float4*>(prob + k * FM + 4);
          o[0] += p0.x * v; o[1] += p0.y * v; o[2] += p0.z * v; o[3] += p0.w * v;
          o[4] += p1.x * v; o[5] += p1.y * v; o[6] += p1.z * v; o[7] += p1.w * v;
        }
      }
      __syncthreads();
      st = (st + 1) % FSTAGES;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    // the groups of keys join in order; `part` holds [KG][FM][D] at most
    static_assert(KG * FM * D <= DQ * FM * FN, "the groups' sums fit where scores and probabilities were");
#pragma unroll
    for (int r = 0; r < FM; ++r) part[(kg * FM + r) * D + col] = o[r];
    if (lane == 0) {
      fac[FM + wid] = m;
      fac[2 * FM + wid] = l;
    }
    __syncthreads();
    const bool whole = piece == c.nu;
    for (int e = tid; e < rows * D; e += NT) {
      const int r = e / D, d = e % D, fr = c.i * FM + r;
      float x = part[r * D + d];
#pragma unroll
      for (int k = 1; k < KG; ++k) x += part[(k * FM + r) * D + d];
      const float rl = fac[2 * FM + r];
      if (whole)
        static_cast<float*>(a.out)[((size_t)(c.q.start + a.token(fr)) * a.Hq + c.h * a.group + a.head_of(fr)) * D + d] =
            rl > 0.f ? x / rl : 0.f;
      else
        a.part_o[((size_t)attn_slot(c, blockIdx.x) * FM + r) * D + d] = x;
    }
    if (!whole) {
      if (tid < rows) a.part_ml[(size_t)attn_slot(c, blockIdx.x) * FM + tid] = make_float2(fac[FM + tid], fac[2 * FM + tid]);
      int c0, n;
      if (attn_arrive(a, sp, c, sched, c0, n)) attn_join<float, D, FM, NT, 16, false>(a, c, c0, n, part);
    }
  } while (attn_next<FM>(a, FN, c));
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t s) {
  // Up to four tiles of eight rows the few-row kernel is ahead although it reads the keys once for each:
  // 8 requests of 3000 keys, 8 kv heads, 16, 24 and 32 rows per kv head: 113, 168 and 218 us against the
  // other's 228 to 230 (a fifth tile would add 55 us); 2 requests of 400 keys, 32 rows: 19 us against 25.
  if ((int64_t)a.max_new * a.group <= 4 * FM)
    return sm103::launch(attn_f32_few_kernel<D>, grid, NT, FewCfg<D>::kBytes, s, a);
  return sm103::launch(attn_f32_kernel<D>, grid, NT, F32Cfg<D>::kBytes, s, a);
}

template <int D>
cudaError_t prepare() {
  const cudaError_t e = cudaFuncSetAttribute(attn_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32Cfg<D>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_f32_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<D>::kBytes);
}

}  // namespace

cudaError_t prepare_attn_f32(int D) { return D == 64 ? prepare<64>() : prepare<128>(); }

cudaError_t launch_attn_f32(const AttnArgs& a, int D, int grid, cudaStream_t s) {
  return D == 64 ? launch<64>(a, grid, s) : launch<128>(a, grid, s);
}

}  // namespace moeslot
