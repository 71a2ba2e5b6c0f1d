// Attention of new tokens over the paged cache, fp32: q, caches and out are
// fp32 and every product and sum is fp32 on the CUDA cores (the tensor cores'
// tf32 would drop 13 bits of each factor).
//
//   out[t, head] = sum_j softmax_j(scale q[t, head] . k[j]) v[j],
//   j in (pos - window, pos], pos = seq_len - new + t
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// a tile's scores s raise m to m', and O and l are scaled by exp(m - m').
// A CTA holds 32 query rows (all heads of a kv head's group together, so a key
// read once serves the whole group) and walks its units of 32 keys.
#include "attn_internal.cuh"
#include "sm103.cuh"

namespace moeslot {
namespace {

constexpr int NT = 256, BM = kAttnF32Tile, BN = 32;

template <int D>
__global__ __launch_bounds__(NT) void attn_f32_kernel(const AttnArgs a) {
  constexpr int LD = D + 4;                 // padded rows: eight rows' float4 reads hit 32 banks
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;                         // [BM][LD]
  float* sk = sq + BM * LD;                 // [BN][LD]
  float* sv = sk + BN * LD;                 // [BN][LD]
  float* spr = sv + BN * LD;                // [BM][BN + 1]
  __shared__ int32_t sched[128];
  sm103::grid_wait();
  AttnSplit sp;
  AttnCursor c;
  if (!attn_find_range<BM, NT>(a, BN, 4, blockIdx.x, gridDim.x, sched, sp, c)) return;
  const int tid = threadIdx.x, row = tid / 8, sub = tid % 8;
  do {
    const int rows = min(BM, c.q.n * a.group - c.i * BM);
    const int fr = c.i * BM + row;
    const int pos = row < rows ? c.q.seq - c.q.n + a.token(fr) : -1;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int first = a.token(c.i * BM), last = min(c.q.n - 1, a.token((c.i + 1) * BM - 1));
    const int tile_hi = c.q.seq - c.q.n + last + 1;
    const int tile_lo = a.window > 0 ? max(0, c.q.seq - c.q.n + first - a.window + 1) : 0;
    __syncthreads();
    for (int e = tid * 4; e < BM * D; e += NT * 4) {
      const int rr = e / D, d = e % D;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows) {
        const int f = c.i * BM + rr;
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                             (size_t)(c.q.start + a.token(f)) * a.q_stride +
                                             (size_t)(c.h * a.group + a.head_of(f)) * D + d);
      }
      *reinterpret_cast<float4*>(sq + rr * LD + d) = v;
    }
    float o[D / 8];
#pragma unroll
    for (int k = 0; k < D / 8; ++k) o[k] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int piece = attn_piece(c);
    for (int u = 0; u < piece; ++u) {
      const int key0 = (c.u0 + c.at + u) * BN;
      __syncthreads();
      for (int e = tid * 4; e < BN * D; e += NT * 4) {
        const int kr = e / D, d = e % D, key = key0 + kr;
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (key >= tile_lo && key < tile_hi) {   // what no row of the tile sees may hold anything: it counts as zero
          const int page = a.table[(size_t)c.r * a.table_stride + (key >> a.page_log2)];
          if ((uint32_t)page < (uint32_t)a.num_pages) {
            const size_t at = ((((size_t)page * a.Hkv + c.h) << a.page_log2) + (key & (a.page - 1))) * D + d;
            kv = *reinterpret_cast<const float4*>(static_cast<const float*>(a.k_cache) + at);
            vv = *reinterpret_cast<const float4*>(static_cast<const float*>(a.v_cache) + at);
          } else {
            attn_status(a.status, MOE_ERR_BOUNDS);
          }
        }
        *reinterpret_cast<float4*>(sk + kr * LD + d) = kv;
        *reinterpret_cast<float4*>(sv + kr * LD + d) = vv;
      }
      __syncthreads();
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 x = *reinterpret_cast<const float4*>(sq + row * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(sk + (sub + 8 * j) * LD + d);
          s[j] += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + sub + 8 * j;
        s[j] = key >= lo && key <= pos ? s[j] * a.scale : -INFINITY;
        top = fmaxf(top, s[j]);
      }
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float mn = fmaxf(m, top);
      const float base = mn == -INFINITY ? 0.f : mn;     // no key yet: every exponential is 0, not NaN
      const float f = expf(m - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[j] - base);
        spr[row * (BN + 1) + sub + 8 * j] = p;
        sum += p;
      }
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      l = l * f + sum;
      m = mn;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) o[k] *= f;
      __syncwarp();
#pragma unroll 4
      for (int j = 0; j < BN; ++j) {
        const float p = spr[row * (BN + 1) + j];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(sv + j * LD + sub * 4 + 32 * k);
          o[4 * k] += p * v.x; o[4 * k + 1] += p * v.y; o[4 * k + 2] += p * v.z; o[4 * k + 3] += p * v.w;
        }
      }
    }
    if (piece == c.nu) {
      if (row < rows) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        float* dst = static_cast<float*>(a.out) +
                     ((size_t)(c.q.start + a.token(fr)) * a.Hq + c.h * a.group + a.head_of(fr)) * D + sub * 4;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          attn_store4(dst + 32 * k, make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv));
      }
    } else {
      const size_t at = (size_t)attn_slot(c, blockIdx.x) * BM + row;
      if (sub == 0) a.part_ml[at] = make_float2(m, l);
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        attn_store4(a.part_o + at * D + sub * 4 + 32 * k, make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
      int c0, n;
      if (attn_arrive(a, sp, c, sched, c0, n)) attn_join<float, D, BM, NT, false>(a, c, c0, n);
    }
  } while (attn_next<BM>(a, BN, c));
}

template <int D>
constexpr int f32_bytes() {
  return ((BM + 2 * BN) * (D + 4) + BM * (BN + 1)) * 4;
}

template <int D>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t s) {
  return sm103::launch(attn_f32_kernel<D>, grid, NT, f32_bytes<D>(), s, a);
}

template <int D>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, f32_bytes<D>());
}

}  // namespace

cudaError_t prepare_attn_f32(int D) { return D == 64 ? prepare<64>() : prepare<128>(); }

cudaError_t launch_attn_f32(const AttnArgs& a, int D, int grid, cudaStream_t s) {
  return D == 64 ? launch<64>(a, grid, s) : launch<128>(a, grid, s);
}

}  // namespace moeslot
