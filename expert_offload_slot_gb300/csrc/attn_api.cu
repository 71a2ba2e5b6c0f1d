// C ABI of the attention step and the token choice (declared in
// include/moeslot.h): argument checks, the handle's workspace, the tensor maps
// of a call's caches and the launches.  No call synchronises, and only
// moe_attn_create allocates, so a step can be captured into a CUDA graph.
#include <cudaTypedefs.h>

#include <cstdarg>
#include <cstdio>
#include <new>

#include "attn_internal.cuh"
#include "sample_internal.cuh"

using namespace moeslot;

struct moe_attn {
  moe_attn_config cfg;
  int device = 0, sms = 0, page_log2 = 0;
  void* work = nullptr;        // one allocation: partial results, counters, status
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  uint32_t* arrived = nullptr;
  uint32_t* ticket = nullptr;
  int32_t* status = nullptr;
  size_t zero_bytes = 0;       // counters and status, from `arrived` on
  // tensor maps of caches of map_pages pages, for the row kernel [0] and the tile kernel [1]: K and V
  // differ in the box; a call sets its caches' addresses into a copy
  CUtensorMap maps[2][2];
  int32_t map_pages[2] = {0, 0};
};

namespace {

moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_last_error(st, buf);
}

moe_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Makes a handle's device current for a call and gives the thread its own back at the end: the stream
// of a call may be the default one, which is that of the current device.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    error = cudaGetDevice(&before);
    if (error == cudaSuccess && before != device) {
      error = cudaSetDevice(device);
      changed = error == cudaSuccess;
    }
  }
  ~DeviceGuard() {
    if (changed) cudaSetDevice(before);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
  cudaError_t error;

 private:
  int before = 0;
  bool changed = false;
};

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

moe_status check_config(const moe_attn_config* c) {
  if (!c) return fail(MOE_ERR_INVALID, "config is NULL");
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return fail(MOE_ERR_INVALID, "dtype must be MOE_F32 or MOE_BF16");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(MOE_ERR_INVALID, "head_dim must be 64 or 128");
  if (c->num_kv_heads < 1 || c->num_kv_heads > 256) return fail(MOE_ERR_INVALID, "num_kv_heads must be in 1..256");
  if (c->num_q_heads < c->num_kv_heads || c->num_q_heads > 1024 || c->num_q_heads % c->num_kv_heads)
    return fail(MOE_ERR_INVALID, "num_q_heads must be a multiple of num_kv_heads, at most 1024");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(MOE_ERR_INVALID, "page_size must be 16, 32, 64 or 128");
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 16)
    return fail(MOE_ERR_INVALID, "rotary_dim must be a multiple of 16 in 0..head_dim");
  if (c->rotary_style != MOE_ROTARY_HALF && c->rotary_style != MOE_ROTARY_PAIRS)
    return fail(MOE_ERR_INVALID, "unknown rotary_style");
  if (c->window < 0) return fail(MOE_ERR_INVALID, "window must be >= 0");
  if (!(c->softmax_scale > 0.f) || c->softmax_scale > 1e30f)
    return fail(MOE_ERR_INVALID, "softmax_scale must be positive and finite");
  if (!(c->norm_eps >= 0.f) || c->norm_eps > 1e30f) return fail(MOE_ERR_INVALID, "norm_eps must be >= 0 and finite");
  return MOE_OK;
}

template <typename F>
F driver_call(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    p = nullptr;
  return reinterpret_cast<F>(p);
}

// A cache [num_pages][Hkv][P][D] as [D / cols][num_pages * Hkv * P][cols] bf16, cols 64 or 32: a box
// of `rows` consecutive keys of one head comes as `blocks` tiles of rows of 2 cols bytes, swizzled
// over as many.
bool cache_map(CUtensorMap* m, const void* base, int64_t keys, int D, int rows, int cols, int blocks) {
  static const auto encode = driver_call<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled");
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)keys, (cuuint64_t)(D / cols)};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)cols * 2};
  const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)rows, (cuuint32_t)blocks}, one[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// This call's maps: made anew when the number of pages changes, else the kept ones with this call's
// addresses (making two costs more than the launch).
bool call_maps(moe_attn* A, bool few, const void* k, const void* v, int32_t num_pages, CUtensorMap& mk, CUtensorMap& mv) {
  static const auto replace = driver_call<PFN_cuTensorMapReplaceAddress_v12000>("cuTensorMapReplaceAddress");
  if (!replace) return false;
  const moe_attn_config& c = A->cfg;
  CUtensorMap* kept = A->maps[few ? 0 : 1];
  if (A->map_pages[few ? 0 : 1] != num_pages) {
    const int64_t keys = (int64_t)num_pages * c.num_kv_heads * c.page_size;
    const int D = c.head_dim;
    A->map_pages[few ? 0 : 1] = 0;
    // the row kernel takes 16 keys of a head at a time, all columns; of the tile kernel's pairs each CTA
    // takes half a K tile, 64 keys, and half a V tile, half the columns
    const bool ok = few ? cache_map(kept, k, keys, D, 16, 64, D / 64) && cache_map(kept + 1, v, keys, D, 16, 64, D / 64)
                        : cache_map(kept, k, keys, D, c.page_size < 64 ? c.page_size : 64, 64, 1) &&
                              cache_map(kept + 1, v, keys, D, c.page_size, D / 2, 1);
    if (!ok) return false;
    A->map_pages[few ? 0 : 1] = num_pages;
  }
  mk = kept[0];
  mv = kept[1];
  return replace(&mk, const_cast<void*>(k)) == CUDA_SUCCESS && replace(&mv, const_cast<void*>(v)) == CUDA_SUCCESS;
}

moe_status check_cache(const moe_attn* A, const void* k, const void* v, int32_t num_pages) {
  if (!k || !v) return fail(MOE_ERR_INVALID, "k_cache and v_cache must not be NULL");
  if (misaligned(k, 16) || misaligned(v, 16)) return fail(MOE_ERR_INVALID, "k_cache and v_cache must be 16-byte aligned");
  if (num_pages < 1) return fail(MOE_ERR_INVALID, "num_pages must be >= 1");
  if ((int64_t)num_pages * A->cfg.num_kv_heads * A->cfg.page_size > 0x7fffffff - 65536)
    return fail(MOE_ERR_INVALID, "num_pages * num_kv_heads * page_size must stay below 2^31 - 65536");
  return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_attn_create(const moe_attn_config* cfg, int device, moe_attn** out) {
  if (!out) return fail(MOE_ERR_INVALID, "out is NULL");
  *out = nullptr;
  const moe_status st = check_config(cfg);
  if (st != MOE_OK) return st;
  int ndev = 0;
  cudaError_t e = cudaGetDeviceCount(&ndev);
  if (e != cudaSuccess) return launched(e, "cudaGetDeviceCount");
  if (device < 0 || device >= ndev) return fail(MOE_ERR_INVALID, "device %d out of range", device);
  const DeviceGuard guard(device);
  if (guard.error != cudaSuccess) return launched(guard.error, "selecting the device");
  e = cfg->dtype == MOE_F32 ? prepare_attn_f32(cfg->head_dim) : prepare_attn_rows(cfg->head_dim);
  if (e == cudaSuccess && cfg->dtype == MOE_BF16) e = prepare_attn_tiles(cfg->head_dim);
  if (e == cudaSuccess) e = prepare_attn_qkv(cfg->dtype, cfg->head_dim);
  if (e != cudaSuccess) return launched(e, "preparing the attention kernels");
  moe_attn* A = new (std::nothrow) moe_attn;
  if (!A) return fail(MOE_ERR_OOM, "host allocation failed");
  A->cfg = *cfg;
  A->device = device;
  while ((1 << A->page_log2) < cfg->page_size) ++A->page_log2;
  cudaDeviceGetAttribute(&A->sms, cudaDevAttrMultiProcessorCount, device);
  if (A->sms < 1) A->sms = 1;
  // two partial slots of a row tile per CTA: the fp32 kernel has two CTAs per SM, the others one
  const size_t slots = (size_t)2 * attn_grid(A->sms);
  const size_t part_rows = cfg->dtype == MOE_F32 ? slots * kAttnF32Tile : (size_t)A->sms * kAttnTile;
  const size_t o_bytes = part_rows * cfg->head_dim * sizeof(float), ml_bytes = part_rows * sizeof(float2);
  A->zero_bytes = (slots + 8) * sizeof(uint32_t);
  e = cudaMalloc(&A->work, o_bytes + ml_bytes + A->zero_bytes);
  if (e != cudaSuccess) {
    delete A;
    cudaGetLastError();
    return fail(MOE_ERR_OOM, "workspace of %zu bytes: %s", o_bytes + ml_bytes, cudaGetErrorString(e));
  }
  uint8_t* p = static_cast<uint8_t*>(A->work);
  A->part_o = reinterpret_cast<float*>(p);
  A->part_ml = reinterpret_cast<float2*>(p + o_bytes);
  A->arrived = reinterpret_cast<uint32_t*>(p + o_bytes + ml_bytes);
  A->ticket = A->arrived + slots;
  A->status = reinterpret_cast<int32_t*>(A->ticket + 4);
  e = cudaMemset(A->arrived, 0, A->zero_bytes);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(A->work);
    delete A;
    return launched(e, "clearing the workspace");
  }
  *out = A;
  return MOE_OK;
}

MOE_API moe_status moe_attn_destroy(moe_attn* A) {
  if (!A) return MOE_OK;
  const DeviceGuard guard(A->device);
  cudaDeviceSynchronize();
  cudaFree(A->work);
  delete A;
  return MOE_OK;
}

MOE_API moe_status moe_attn_get_status(moe_attn* A) {
  if (!A) return fail(MOE_ERR_INVALID, "handle is NULL");
  int32_t st = 0;
  const DeviceGuard guard(A->device);
  cudaError_t e = guard.error;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&st, A->status, sizeof st, cudaMemcpyDeviceToHost);
  return e == cudaSuccess ? static_cast<moe_status>(st) : launched(e, "reading the status");
}

MOE_API moe_status moe_attn_clear_status(moe_attn* A) {
  if (!A) return fail(MOE_ERR_INVALID, "handle is NULL");
  const DeviceGuard guard(A->device);
  cudaError_t e = guard.error;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemset(A->arrived, 0, A->zero_bytes);   // counters a timed-out call may have left, too
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return launched(e, "clearing the status");
}

MOE_API moe_status moe_attn_tables(moe_attn* A, const int32_t* ctx_len, const int32_t* new_len, int32_t R,
                                   int32_t* block_table, int32_t table_stride, const int32_t* free_pages,
                                   int32_t num_free, const int32_t* free_head, int32_t* free_head_out, int32_t rows,
                                   int32_t* row_start, int32_t* seq_len, int32_t* positions, int32_t* slot_map,
                                   void* stream) {
  if (!A) return fail(MOE_ERR_INVALID, "handle is NULL");
  if (R < 0 || R > MOE_ATTN_MAX_REQUESTS) return fail(MOE_ERR_INVALID, "R must be in 0..%d", MOE_ATTN_MAX_REQUESTS);
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (table_stride < 1) return fail(MOE_ERR_INVALID, "table_stride must be >= 1");
  if (num_free < 0) return fail(MOE_ERR_INVALID, "num_free must be >= 0");
  if (!free_head || !free_head_out || !row_start) return fail(MOE_ERR_INVALID, "NULL argument");
  if (R > 0 && (!ctx_len || !new_len || !block_table || !seq_len)) return fail(MOE_ERR_INVALID, "NULL argument");
  if (rows > 0 && (!positions || !slot_map)) return fail(MOE_ERR_INVALID, "NULL argument");
  if (num_free > 0 && !free_pages) return fail(MOE_ERR_INVALID, "free_pages is NULL but num_free is %d", num_free);
  if (R > 0 && (seq_len == ctx_len || seq_len == new_len || row_start == ctx_len || row_start == new_len))
    return fail(MOE_ERR_INVALID, "seq_len and row_start must not be the lengths they are computed from");
  const void* all[] = {ctx_len, new_len, block_table, free_pages, free_head, free_head_out, row_start, seq_len, positions, slot_map};
  for (const void* p : all)
    if (misaligned(p, 4)) return fail(MOE_ERR_INVALID, "every array must be 4-byte aligned");
  TablesArgs a;
  a.ctx = ctx_len; a.fresh = new_len; a.free_pages = free_pages; a.head_in = free_head; a.table = block_table;
  a.head_out = free_head_out; a.row_start = row_start; a.seq_len = seq_len; a.positions = positions; a.slots = slot_map;
  a.status = A->status; a.ticket = A->ticket; a.R = R; a.table_stride = table_stride; a.num_free = num_free; a.rows = rows;
  a.page = A->cfg.page_size; a.page_log2 = A->page_log2;
  const DeviceGuard guard(A->device);
  if (guard.error != cudaSuccess) return launched(guard.error, "selecting the device");
  return launched(launch_attn_tables(a, static_cast<cudaStream_t>(stream)), "moe_attn_tables");
}

MOE_API moe_status moe_attn_qkv(moe_attn* A, const void* qkv, int64_t qkv_stride, int32_t rows, const void* q_norm,
                                const void* k_norm, const float* rope, int32_t rope_len, const int32_t* positions,
                                const int32_t* slot_map, void* q, void* k_cache, void* v_cache, int32_t num_pages,
                                void* stream) {
  if (!A) return fail(MOE_ERR_INVALID, "handle is NULL");
  const moe_attn_config& c = A->cfg;
  const int es = c.dtype == MOE_F32 ? 4 : 2;
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (qkv_stride < (int64_t)(c.num_q_heads + 2 * c.num_kv_heads) * c.head_dim)
    return fail(MOE_ERR_INVALID, "qkv_stride is below (num_q_heads + 2 num_kv_heads) * head_dim");
  if (qkv_stride * es % 16) return fail(MOE_ERR_INVALID, "qkv rows must start on 16-byte boundaries");
  const moe_status st = check_cache(A, k_cache, v_cache, num_pages);
  if (st != MOE_OK) return st;
  if (c.rotary_dim > 0 && (!rope || rope_len < 1)) return fail(MOE_ERR_INVALID, "rope is missing but rotary_dim is %d", c.rotary_dim);
  if (rows == 0) return MOE_OK;
  if (!qkv || !slot_map || !q || (c.rotary_dim > 0 && !positions)) return fail(MOE_ERR_INVALID, "NULL argument");
  if (misaligned(qkv, 16) || misaligned(q, 16) || misaligned(q_norm, 16) || misaligned(k_norm, 16))
    return fail(MOE_ERR_INVALID, "qkv, q, q_norm and k_norm must be 16-byte aligned");
  if (misaligned(rope, 16)) return fail(MOE_ERR_INVALID, "rope must be 16-byte aligned");
  if (misaligned(positions, 4) || misaligned(slot_map, 4))
    return fail(MOE_ERR_INVALID, "positions and slot_map must be 4-byte aligned");
  QkvArgs a;
  a.qkv = qkv; a.q_norm = q_norm; a.k_norm = k_norm; a.rope = rope; a.positions = positions; a.slots = slot_map; a.q = q;
  a.k_cache = k_cache; a.v_cache = v_cache; a.status = A->status; a.qkv_stride = qkv_stride;
  a.num_slots = (int64_t)num_pages * c.page_size; a.rows = rows; a.Hq = c.num_q_heads; a.Hkv = c.num_kv_heads;
  a.page_log2 = A->page_log2; a.rotary = c.rotary_dim; a.pairs = c.rotary_style == MOE_ROTARY_PAIRS; a.rope_len = rope_len;
  a.eps = c.norm_eps;
  a.heads = a.Hq + 2 * a.Hkv;
  const DeviceGuard guard(A->device);
  if (guard.error != cudaSuccess) return launched(guard.error, "selecting the device");
  return launched(launch_attn_qkv(a, c.dtype, c.head_dim, A->sms, static_cast<cudaStream_t>(stream)), "moe_attn_qkv");
}

MOE_API moe_status moe_attn_forward(moe_attn* A, const void* q, int64_t q_stride, int32_t rows, const int32_t* row_start,
                                    const int32_t* seq_len, int32_t R, int32_t max_new, const void* k_cache,
                                    const void* v_cache, int32_t num_pages, const int32_t* block_table,
                                    int32_t table_stride, void* out, void* stream) {
  if (!A) return fail(MOE_ERR_INVALID, "handle is NULL");
  const moe_attn_config& c = A->cfg;
  const int es = c.dtype == MOE_F32 ? 4 : 2;
  if (R < 0 || R > MOE_ATTN_MAX_REQUESTS) return fail(MOE_ERR_INVALID, "R must be in 0..%d", MOE_ATTN_MAX_REQUESTS);
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (max_new < 0 || max_new > rows) return fail(MOE_ERR_INVALID, "max_new must be in 0..rows");
  if (table_stride < 1) return fail(MOE_ERR_INVALID, "table_stride must be >= 1");
  if (q_stride < (int64_t)c.num_q_heads * c.head_dim) return fail(MOE_ERR_INVALID, "q_stride is below num_q_heads * head_dim");
  if (q_stride * es % 16) return fail(MOE_ERR_INVALID, "q rows must start on 16-byte boundaries");
  moe_status st = check_cache(A, k_cache, v_cache, num_pages);
  if (st != MOE_OK) return st;
  if (R == 0 || rows == 0 || max_new == 0) return MOE_OK;
  if (!q || !row_start || !seq_len || !block_table || !out) return fail(MOE_ERR_INVALID, "NULL argument");
  if (misaligned(q, 16) || misaligned(out, 16)) return fail(MOE_ERR_INVALID, "q and out must be 16-byte aligned");
  if (misaligned(row_start, 4) || misaligned(seq_len, 4) || misaligned(block_table, 4))
    return fail(MOE_ERR_INVALID, "row_start, seq_len and block_table must be 4-byte aligned");
  AttnArgs a = {};
  a.q = q; a.out = out; a.k_cache = k_cache; a.v_cache = v_cache; a.row_start = row_start; a.seq_len = seq_len;
  a.table = block_table; a.q_stride = q_stride; a.R = R; a.rows = rows; a.max_new = max_new; a.table_stride = table_stride;
  a.num_pages = num_pages; a.Hq = c.num_q_heads; a.Hkv = c.num_kv_heads; a.group = c.num_q_heads / c.num_kv_heads;
  a.page = c.page_size; a.page_log2 = A->page_log2; a.window = c.window < kAttnMaxKeys ? c.window : 0; a.scale = c.softmax_scale;
  a.scale_log2 = c.softmax_scale * 1.44269504088896340736f;
  a.part_o = A->part_o; a.part_ml = A->part_ml; a.arrived = A->arrived; a.status = A->status;
  divider(a.group, a.group_mul, a.group_shift);
  const DeviceGuard guard(A->device);
  if (guard.error != cudaSuccess) return launched(guard.error, "selecting the device");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.dtype == MOE_F32) return launched(launch_attn_f32(a, c.head_dim, attn_grid(A->sms), s), "moe_attn_forward");
  // Up to two row tiles of 16 the row kernel is ahead of the tile kernel although it reads the keys
  // once for each: 16 requests of 8192 keys, 4 kv heads, 24 and 32 query rows per kv head: 90 and 91 us
  // against 96 and 95; with 64 rows 168 against 97.  One chunk decides for all requests of the call: 16
  // decodes over 8192 keys beside a chunk of 512 tokens 199 us, in two calls 144.
  const bool few = (int64_t)max_new * a.group <= 2 * kAttnRowsTile;
  CUtensorMap mk, mv;
  if (!call_maps(A, few, k_cache, v_cache, num_pages, mk, mv))
    return fail(MOE_ERR_CUDA, "the driver made no tensor map of the caches");
  const int D = c.head_dim;
  return launched(few ? launch_attn_rows(a, mk, mv, D, A->sms, s) : launch_attn_tiles(a, mk, mv, D, A->sms / 2 * 2, s),
                  "moe_attn_forward");
}

MOE_API moe_status moe_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                              const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                              const float* u, int32_t* ids, float* logp, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_INVALID, "dtype must be MOE_F32 or MOE_BF16");
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (vocab < 1 || vocab > MOE_SAMPLE_MAX_VOCAB) return fail(MOE_ERR_INVALID, "vocab must be in 1..%d", MOE_SAMPLE_MAX_VOCAB);
  if (row_stride < vocab) return fail(MOE_ERR_INVALID, "row_stride is below vocab");
  if (rows == 0) return MOE_OK;
  if (!logits || !u || !ids) return fail(MOE_ERR_INVALID, "logits, u and ids must not be NULL");
  if (misaligned(logits, dtype == MOE_F32 ? 4 : 2)) return fail(MOE_ERR_INVALID, "logits must be aligned to their elements");
  const void* all[] = {temperature, top_k, top_p, min_p, u, ids, logp};
  for (const void* p : all)
    if (misaligned(p, 4)) return fail(MOE_ERR_INVALID, "the per-row arrays must be 4-byte aligned");
  SampleArgs a;
  a.logits = logits; a.row_stride = row_stride; a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.u = u; a.ids = ids; a.logp = logp; a.rows = rows; a.vocab = vocab;
  return launched(launch_sample(a, dtype, static_cast<cudaStream_t>(stream)), "moe_sample");
}
