// C ABI of the operators around a step's blocks (declared in include/moeslot.h):
// argument checks and launches.  They need no handle and no workspace, run on the
// current device and neither allocate nor synchronise.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "step_internal.cuh"

using namespace moeslot;

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

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
bool bad_dtype(int32_t t) { return t != MOE_F32 && t != MOE_BF16; }
int size_of(int32_t t) { return t == MOE_F32 ? 4 : 2; }

}  // namespace

MOE_API moe_status moe_step_status(void) {
  cudaError_t e = cudaDeviceSynchronize();
  int32_t first = 0;
  for (auto take : {linear_q4_rows_status, linear_q4_tiles_status, linear_q4_split_status}) {
    int32_t st = 0;
    if (e == cudaSuccess) e = take(&st);
    if (first == 0) first = st;
  }
  return e == cudaSuccess ? static_cast<moe_status>(first) : launched(e, "reading the status");
}

MOE_API moe_status moe_residual_norm(const moe_norm_config* c, const void* x, int64_t x_stride, const void* gate,
                                     int64_t gate_stride, const void* post_weight, const void* residual,
                                     int64_t residual_stride, void* residual_out, int64_t residual_out_stride,
                                     const void* pre_weight, void* y, int64_t y_stride, int32_t rows, void* stream) {
  if (!c) return fail(MOE_ERR_INVALID, "config is NULL");
  if (bad_dtype(c->dtype)) return fail(MOE_ERR_INVALID, "dtype must be MOE_F32 or MOE_BF16");
  if (c->residual_dtype != c->dtype && c->residual_dtype != MOE_F32)
    return fail(MOE_ERR_INVALID, "residual_dtype must be dtype or MOE_F32");
  if (c->hidden < 1 || c->hidden > MOE_NORM_MAX_HIDDEN) return fail(MOE_ERR_INVALID, "hidden must be in 1..%d", MOE_NORM_MAX_HIDDEN);
  if (c->gate < MOE_RESIDUAL_GATE_NONE || c->gate > MOE_RESIDUAL_GATE_ELEMENT) return fail(MOE_ERR_INVALID, "unknown gate");
  if (c->gate_sigmoid != 0 && c->gate_sigmoid != 1) return fail(MOE_ERR_INVALID, "gate_sigmoid must be 0 or 1");
  if (!std::isfinite(c->residual_scale) || !std::isfinite(c->weight_offset))
    return fail(MOE_ERR_INVALID, "residual_scale and weight_offset must be finite");
  if (!(c->norm_eps >= 0.f) || c->norm_eps > 1e30f) return fail(MOE_ERR_INVALID, "norm_eps must be >= 0 and finite");
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  const bool gated = c->gate != MOE_RESIDUAL_GATE_NONE;
  const int64_t h = c->hidden;
  if (residual_stride < h) return fail(MOE_ERR_INVALID, "residual_stride is below hidden");
  if (x && x_stride < h) return fail(MOE_ERR_INVALID, "x_stride is below hidden");
  if (x && residual_out_stride < h) return fail(MOE_ERR_INVALID, "residual_out_stride is below hidden");
  if (y && y_stride < h) return fail(MOE_ERR_INVALID, "y_stride is below hidden");
  if (gated && c->gate == MOE_RESIDUAL_GATE_ELEMENT && gate_stride < h) return fail(MOE_ERR_INVALID, "gate_stride is below hidden");
  if (gated && c->gate == MOE_RESIDUAL_GATE_ROW && gate_stride < 1) return fail(MOE_ERR_INVALID, "gate_stride must be >= 1");
  if (rows == 0) return MOE_OK;
  if (!residual) return fail(MOE_ERR_INVALID, "residual must not be NULL");
  if (x && !residual_out) return fail(MOE_ERR_INVALID, "residual_out must not be NULL where x is given");
  if (gated && !gate) return fail(MOE_ERR_INVALID, "gate is NULL but the config has one");
  if (!x && (residual_out || post_weight || gated)) return fail(MOE_ERR_INVALID, "residual_out, post_weight and a gate need x");
  if (!x && !y) return fail(MOE_ERR_INVALID, "x and y must not both be NULL");
  const int es = size_of(c->dtype), rs = size_of(c->residual_dtype);
  const void* same[] = {x, gate, post_weight, pre_weight, y};
  for (const void* p : same)
    if (misaligned(p, es)) return fail(MOE_ERR_INVALID, "every tensor must be aligned to its elements");
  if (misaligned(residual, rs) || misaligned(residual_out, rs))
    return fail(MOE_ERR_INVALID, "every tensor must be aligned to its elements");
  NormArgs a;
  a.x = x; a.gate = gate; a.post = post_weight; a.residual = residual; a.pre = pre_weight; a.sum = residual_out; a.y = y;
  a.x_stride = x_stride; a.gate_stride = c->gate == MOE_RESIDUAL_GATE_CHANNEL ? 0 : gate_stride;
  a.residual_stride = residual_stride; a.sum_stride = residual_out_stride; a.y_stride = y_stride;
  a.rows = rows; a.hidden = c->hidden; a.gate_kind = c->gate; a.gate_sigmoid = c->gate_sigmoid;
  a.scale = c->residual_scale; a.eps = c->norm_eps; a.offset = c->weight_offset;
  return launched(launch_residual_norm(a, c->dtype, c->residual_dtype, static_cast<cudaStream_t>(stream)), "moe_residual_norm");
}

MOE_API moe_status moe_q4_pack(const float* w, int32_t out_features, int32_t in_features, int32_t group, uint8_t* codes,
                               float* scales) {
  if (group != 32 && group != 64 && group != 128) return fail(MOE_ERR_INVALID, "group must be 32, 64 or 128");
  if (in_features < 32 || in_features > MOE_LINEAR_MAX_IN || in_features % 32)
    return fail(MOE_ERR_INVALID, "in_features must be a multiple of 32 in 32..%d", MOE_LINEAR_MAX_IN);
  if (out_features < 1 || out_features > MOE_LINEAR_MAX_OUT)
    return fail(MOE_ERR_INVALID, "out_features must be in 1..%d", MOE_LINEAR_MAX_OUT);
  if (!w || !codes || !scales) return fail(MOE_ERR_INVALID, "NULL argument");
  const int64_t K = in_features, groups = (K + group - 1) / group;
  for (int64_t n = 0; n < out_features; ++n)
    for (int64_t g = 0; g < groups; ++g) {
      const int64_t k0 = g * group, k1 = k0 + group < K ? k0 + group : K;
      const float* src = w + n * K;
      float amax = 0.f;
      for (int64_t k = k0; k < k1; ++k) {
        if (!std::isfinite(src[k])) return fail(MOE_ERR_INVALID, "weight [%lld, %lld] is not finite", (long long)n, (long long)k);
        amax = std::fmax(amax, std::fabs(src[k]));
      }
      float scale = amax / 7.f;
      if (!(scale > 0.f)) scale = 1.f;
      scales[n * groups + g] = scale;
      uint8_t* dst = codes + n * (K / 2);
      for (int64_t k = k0; k < k1; k += 2) {
        const float lo = std::fmin(std::fmax(std::nearbyint(src[k] / scale), -7.f), 7.f);
        const float hi = std::fmin(std::fmax(std::nearbyint(src[k + 1] / scale), -7.f), 7.f);
        dst[k / 2] = (uint8_t)(((int)lo & 15) | ((int)hi & 15) << 4);
      }
    }
  return MOE_OK;
}

MOE_API moe_status moe_linear_q4(const void* x, int32_t dtype, int64_t x_stride, int32_t rows, int32_t in_features,
                                 const uint8_t* codes, const void* scales, int32_t scale_dtype, int32_t group,
                                 const void* bias, int32_t out_features, void* out, int32_t out_dtype, int64_t out_stride,
                                 void* stream) {
  if (bad_dtype(dtype) || bad_dtype(scale_dtype)) return fail(MOE_ERR_INVALID, "dtype and scale_dtype must be MOE_F32 or MOE_BF16");
  if (out_dtype != dtype && out_dtype != MOE_F32) return fail(MOE_ERR_INVALID, "out_dtype must be dtype or MOE_F32");
  if (group != 32 && group != 64 && group != 128) return fail(MOE_ERR_INVALID, "group must be 32, 64 or 128");
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (in_features < 32 || in_features > MOE_LINEAR_MAX_IN || in_features % 32)
    return fail(MOE_ERR_INVALID, "in_features must be a multiple of 32 in 32..%d", MOE_LINEAR_MAX_IN);
  if (out_features < 1 || out_features > MOE_LINEAR_MAX_OUT)
    return fail(MOE_ERR_INVALID, "out_features must be in 1..%d", MOE_LINEAR_MAX_OUT);
  if (x_stride < in_features) return fail(MOE_ERR_INVALID, "x_stride is below in_features");
  if (out_stride < out_features) return fail(MOE_ERR_INVALID, "out_stride is below out_features");
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !out) return fail(MOE_ERR_INVALID, "x, codes, scales and out must not be NULL");
  if (misaligned(codes, 16)) return fail(MOE_ERR_INVALID, "codes must be 16-byte aligned");
  if (misaligned(x, size_of(dtype)) || misaligned(bias, size_of(dtype)) || misaligned(scales, size_of(scale_dtype)) ||
      misaligned(out, size_of(out_dtype)))
    return fail(MOE_ERR_INVALID, "every tensor must be aligned to its elements");
  LinearArgs a = {};
  a.x = x; a.codes = codes; a.scales = scales; a.bias = bias; a.out = out; a.x_stride = x_stride; a.out_stride = out_stride;
  a.rows = rows; a.K = in_features; a.N = out_features; a.groups = (in_features + group - 1) / group;
  a.x_f32 = dtype == MOE_F32; a.out_f32 = out_dtype == MOE_F32; a.scale_f32 = scale_dtype == MOE_F32;
  return launched(launch_linear_q4(a, group, static_cast<cudaStream_t>(stream)), "moe_linear_q4");
}

MOE_API moe_status moe_logprobs(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                                const int32_t* targets, int32_t top, float* logp, float* entropy, int32_t* rank,
                                int32_t* top_ids, float* top_logp, void* stream) {
  if (bad_dtype(dtype)) return fail(MOE_ERR_INVALID, "dtype must be MOE_F32 or MOE_BF16");
  if (rows < 0 || rows > MOE_ATTN_MAX_ROWS) return fail(MOE_ERR_INVALID, "rows must be in 0..%d", MOE_ATTN_MAX_ROWS);
  if (vocab < 1 || vocab > MOE_SAMPLE_MAX_VOCAB) return fail(MOE_ERR_INVALID, "vocab must be in 1..%d", MOE_SAMPLE_MAX_VOCAB);
  if (row_stride < vocab) return fail(MOE_ERR_INVALID, "row_stride is below vocab");
  if (top < 0 || top > MOE_LOGPROBS_MAX_TOP) return fail(MOE_ERR_INVALID, "top must be in 0..%d", MOE_LOGPROBS_MAX_TOP);
  if (rows == 0) return MOE_OK;
  if (!logits || !targets || !logp) return fail(MOE_ERR_INVALID, "logits, targets and logp must not be NULL");
  if (top > 0 && (!top_ids || !top_logp)) return fail(MOE_ERR_INVALID, "top_ids and top_logp must not be NULL where top is above 0");
  if (misaligned(logits, size_of(dtype))) return fail(MOE_ERR_INVALID, "logits must be aligned to their elements");
  const void* all[] = {targets, logp, entropy, rank, top_ids, top_logp};
  for (const void* p : all)
    if (misaligned(p, 4)) return fail(MOE_ERR_INVALID, "the per-row arrays must be 4-byte aligned");
  LogprobArgs a;
  a.logits = logits; a.targets = targets; a.logp = logp; a.entropy = entropy; a.rank = rank; a.top_ids = top_ids;
  a.top_logp = top_logp; a.row_stride = row_stride; a.rows = rows; a.vocab = vocab; a.top = top;
  return launched(launch_logprobs(a, dtype, static_cast<cudaStream_t>(stream)), "moe_logprobs");
}
