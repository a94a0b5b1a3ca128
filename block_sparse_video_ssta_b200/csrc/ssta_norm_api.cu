// C ABI of the norms, gated residuals and 8-bit checkpoints around the attention:
// argument validation, size planning and dispatch.  Declared in include/ssta.h.
// Nothing here allocates or synchronises.
#include <math.h>

#include <initializer_list>

#include "ssta_api_common.h"
#include "ssta_norm.h"

namespace ssta {
namespace {

constexpr int kMaxChannels = 8192;   // one block holds a row

bool known_dtype(int d) { return d == SSTA_BF16 || d == SSTA_F32; }
bool known_norm(int n) { return n == SSTA_NORM_NONE || n == SSTA_NORM_LAYER || n == SSTA_NORM_RMS; }

ssta_status check_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return SSTA_ERR_ALIGNMENT;
  return SSTA_OK;
}

// A checkpoint argument: NULL is absent (all-zero copy), anything else must be whole.
ssta_status take(const ssta_checkpoint* c, ssta_checkpoint* out) {
  *out = ssta_checkpoint{};
  if (c == nullptr) return SSTA_OK;
  if (c->codes == nullptr || c->exponents == nullptr) return SSTA_ERR_INVALID_ARG;
  if (c->format != SSTA_INT8 && c->format != SSTA_E4M3) return SSTA_ERR_INVALID_ARG;
  if (!aligned(c->codes, 16) || !aligned(c->exponents, 16)) return SSTA_ERR_ALIGNMENT;
  *out = *c;
  return SSTA_OK;
}

ssta_status check_workspace(const NormGeom& g, const void* workspace, size_t bytes) {
  if (workspace == nullptr || bytes < norm_bwd_workspace_bytes(g)) return SSTA_ERR_WORKSPACE;
  return aligned(workspace, 256) ? SSTA_OK : SSTA_ERR_ALIGNMENT;
}

}  // namespace

ssta_status make_norm_geom(const ssta_norm_desc* d, NormGeom* g) {
  if (d == nullptr || g == nullptr) return SSTA_ERR_INVALID_ARG;
  if (d->rows < 1 || d->C < 1 || d->mod_rows < 0 || d->mod_stride < 0) return SSTA_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || !known_dtype(d->param_dtype)) return SSTA_ERR_INVALID_ARG;
  if (!known_norm(d->norm) || !known_norm(d->post_norm)) return SSTA_ERR_INVALID_ARG;
  if (!(d->eps > 0.0f) || isinf(d->eps) || !isfinite(d->res_scale)) return SSTA_ERR_INVALID_ARG;
  if (d->mod_stride > 0 && d->mod_stride < d->C) return SSTA_ERR_INVALID_ARG;
  if (d->rows >= (int64_t)1 << 31) return SSTA_ERR_UNSUPPORTED;
  if (d->C % 8 != 0 || d->C > kMaxChannels || d->mod_stride % 8 != 0) return SSTA_ERR_UNSUPPORTED;
  NormGeom x{};
  x.rows = d->rows;
  x.mod_rows = d->mod_rows == 0 || d->mod_rows > d->rows ? d->rows : d->mod_rows;
  x.mod_stride = d->mod_stride == 0 ? d->C : d->mod_stride;
  x.groups = (x.rows + x.mod_rows - 1) / x.mod_rows;
  x.C = d->C;
  x.norm = d->norm;
  x.post_norm = d->post_norm;
  x.eps = d->eps;
  x.res_scale = d->res_scale;
  x.bf16 = d->dtype == SSTA_BF16;
  x.param_f32 = d->param_dtype == SSTA_F32;
  *g = x;
  return SSTA_OK;
}

}  // namespace ssta

using namespace ssta;

#define SSTA_TRY(expr)                          \
  do {                                          \
    const ssta_status st_ = (expr);             \
    if (st_ != SSTA_OK) return st_;             \
  } while (0)

extern "C" {

ssta_status ssta_norm_plan(const ssta_norm_desc* desc, ssta_norm_plan_info* info) {
  if (info == nullptr) return SSTA_ERR_INVALID_ARG;
  NormGeom g;
  SSTA_TRY(make_norm_geom(desc, &g));
  info->groups = g.groups;
  info->exponents_per_row = (g.C + 127) / 128;
  info->bwd_workspace_bytes = norm_bwd_workspace_bytes(g);
  return SSTA_OK;
}

ssta_status ssta_norm_fwd(const ssta_norm_desc* desc, const void* x, const void* weight, const void* scale,
                          const void* shift, void* y, float* mean, float* rstd, const ssta_checkpoint* x_save,
                          void* stream) {
  NvtxRange nvtx("ssta_norm_fwd");
  NormGeom g;
  SSTA_TRY(make_norm_geom(desc, &g));
  if (g.norm == SSTA_NORM_NONE || x == nullptr || y == nullptr) return SSTA_ERR_INVALID_ARG;
  if (g.norm != SSTA_NORM_LAYER && mean != nullptr) return SSTA_ERR_INVALID_ARG;
  NormFwdArgs a{};
  SSTA_TRY(take(x_save, &a.r_save));
  SSTA_TRY(check_aligned({x, weight, scale, shift, y, mean, rstd}));
  a.x = x;
  a.weight = weight;
  a.scale = scale;
  a.shift = shift;
  a.n = y;
  a.mean = mean;
  a.rstd = rstd;
  return from_cuda(launch_norm_fwd(g, a, static_cast<cudaStream_t>(stream)));
}

ssta_status ssta_norm_bwd(const ssta_norm_desc* desc, const void* dy, const void* x, const ssta_checkpoint* x_saved,
                          const float* mean, const float* rstd, const void* weight, const void* scale,
                          const void* dres, void* dx, float* dweight, float* dscale, float* dshift, void* workspace,
                          size_t workspace_bytes, void* stream) {
  NvtxRange nvtx("ssta_norm_bwd");
  NormGeom g;
  SSTA_TRY(make_norm_geom(desc, &g));
  if (g.norm == SSTA_NORM_NONE || dy == nullptr || dx == nullptr || rstd == nullptr) return SSTA_ERR_INVALID_ARG;
  if ((x == nullptr) == (x_saved == nullptr)) return SSTA_ERR_INVALID_ARG;
  if ((g.norm == SSTA_NORM_LAYER) != (mean != nullptr)) return SSTA_ERR_INVALID_ARG;
  NormBwdArgs a{};
  SSTA_TRY(take(x_saved, &a.r_saved));
  SSTA_TRY(check_aligned({dy, x, mean, rstd, weight, scale, dres, dx, dweight, dscale, dshift}));
  SSTA_TRY(check_workspace(g, workspace, workspace_bytes));
  g.post_norm = SSTA_NORM_NONE;
  a.dr = dres;
  a.dn = dy;
  a.r = x;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.scale = scale;
  a.dx = dx;
  a.dweight = dweight;
  a.dscale = dscale;
  a.dshift = dshift;
  return from_cuda(launch_norm_bwd(g, a, workspace, static_cast<cudaStream_t>(stream)));
}

ssta_status ssta_residual_norm_fwd(const ssta_norm_desc* desc, const void* x, const void* y, const void* post_weight,
                                   const void* gate, const void* weight, const void* scale, const void* shift,
                                   void* r, void* n, float* post_mean, float* post_rstd, float* mean, float* rstd,
                                   const ssta_checkpoint* y_save, const ssta_checkpoint* r_save, void* stream) {
  NvtxRange nvtx("ssta_residual_norm_fwd");
  NormGeom g;
  SSTA_TRY(make_norm_geom(desc, &g));
  if (x == nullptr || y == nullptr || r == nullptr) return SSTA_ERR_INVALID_ARG;
  if ((g.norm == SSTA_NORM_NONE) != (n == nullptr)) return SSTA_ERR_INVALID_ARG;
  if (g.norm == SSTA_NORM_NONE && (weight != nullptr || scale != nullptr || shift != nullptr || rstd != nullptr))
    return SSTA_ERR_INVALID_ARG;
  if (g.norm != SSTA_NORM_LAYER && mean != nullptr) return SSTA_ERR_INVALID_ARG;
  if (g.post_norm == SSTA_NORM_NONE && (post_weight != nullptr || post_rstd != nullptr)) return SSTA_ERR_INVALID_ARG;
  if (g.post_norm != SSTA_NORM_LAYER && post_mean != nullptr) return SSTA_ERR_INVALID_ARG;
  NormFwdArgs a{};
  SSTA_TRY(take(y_save, &a.y_save));
  SSTA_TRY(take(r_save, &a.r_save));
  SSTA_TRY(check_aligned({x, y, post_weight, gate, weight, scale, shift, r, n, post_mean, post_rstd, mean, rstd}));
  a.x = x;
  a.y = y;
  a.post_weight = post_weight;
  a.gate = gate;
  a.weight = weight;
  a.scale = scale;
  a.shift = shift;
  a.r = r;
  a.n = n;
  a.post_mean = post_mean;
  a.post_rstd = post_rstd;
  a.mean = mean;
  a.rstd = rstd;
  return from_cuda(launch_norm_fwd(g, a, static_cast<cudaStream_t>(stream)));
}

ssta_status ssta_residual_norm_bwd(const ssta_norm_desc* desc, const void* dr, const void* dn, const void* r,
                                   const ssta_checkpoint* r_saved, const void* y, const ssta_checkpoint* y_saved,
                                   const float* post_mean, const float* post_rstd, const float* mean,
                                   const float* rstd, const void* post_weight, const void* gate, const void* weight,
                                   const void* scale, void* dx, void* dy, float* dpost_weight, float* dgate,
                                   float* dweight, float* dscale, float* dshift, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  NvtxRange nvtx("ssta_residual_norm_bwd");
  NormGeom g;
  SSTA_TRY(make_norm_geom(desc, &g));
  if (dx == nullptr || dy == nullptr || (dr == nullptr && dn == nullptr)) return SSTA_ERR_INVALID_ARG;
  if ((r != nullptr && r_saved != nullptr) || (y != nullptr && y_saved != nullptr)) return SSTA_ERR_INVALID_ARG;
  const bool has_r = r != nullptr || r_saved != nullptr, has_y = y != nullptr || y_saved != nullptr;
  if (dn != nullptr) {
    if (g.norm == SSTA_NORM_NONE || !has_r || rstd == nullptr) return SSTA_ERR_INVALID_ARG;
    if (g.norm == SSTA_NORM_LAYER && mean == nullptr) return SSTA_ERR_INVALID_ARG;
  } else if (dweight != nullptr || dscale != nullptr || dshift != nullptr) {
    return SSTA_ERR_INVALID_ARG;
  }
  if (g.post_norm != SSTA_NORM_NONE) {
    if (!has_y || post_rstd == nullptr || (g.post_norm == SSTA_NORM_LAYER && post_mean == nullptr))
      return SSTA_ERR_INVALID_ARG;
  } else if (post_weight != nullptr || dpost_weight != nullptr) {
    return SSTA_ERR_INVALID_ARG;
  }
  if (dgate != nullptr && !has_y) return SSTA_ERR_INVALID_ARG;
  NormBwdArgs a{};
  // what no formula reads is left alone
  const bool use_r = dn != nullptr;
  const bool use_y = g.post_norm != SSTA_NORM_NONE || dgate != nullptr || dpost_weight != nullptr;
  SSTA_TRY(take(r_saved, &a.r_saved));
  SSTA_TRY(take(y_saved, &a.y_saved));
  if (!use_r) a.r_saved = ssta_checkpoint{};
  if (!use_y) a.y_saved = ssta_checkpoint{};
  if (use_r && use_y) {
    if ((a.r_saved.codes != nullptr) != (a.y_saved.codes != nullptr)) return SSTA_ERR_INVALID_ARG;
    if (a.r_saved.codes != nullptr && a.r_saved.format != a.y_saved.format) return SSTA_ERR_INVALID_ARG;
  }
  SSTA_TRY(check_aligned({dr, dn, r, y, post_mean, post_rstd, mean, rstd, post_weight, gate, weight, scale, dx, dy,
                          dpost_weight, dgate, dweight, dscale, dshift}));
  SSTA_TRY(check_workspace(g, workspace, workspace_bytes));
  a.dr = dr;
  a.dn = dn;
  a.r = use_r ? r : nullptr;
  a.y = use_y ? y : nullptr;
  a.post_mean = post_mean;
  a.post_rstd = post_rstd;
  a.mean = mean;
  a.rstd = rstd;
  a.post_weight = post_weight;
  a.gate = gate;
  // (without dn the norm's vectors would multiply zeros, and an infinity or a NaN among them make a NaN)
  a.weight = use_r ? weight : nullptr;
  a.scale = use_r ? scale : nullptr;
  a.dx = dx;
  a.dy = dy;
  a.dpost_weight = dpost_weight;
  a.dgate = dgate;
  a.dweight = dweight;
  a.dscale = dscale;
  a.dshift = dshift;
  return from_cuda(launch_norm_bwd(g, a, workspace, static_cast<cudaStream_t>(stream)));
}

static ssta_status checkpoint_args(int64_t rows, int C, int dtype, const void* x, const ssta_checkpoint* c,
                                   ssta_checkpoint* out) {
  if (rows < 1 || C < 1 || !known_dtype(dtype) || x == nullptr || c == nullptr) return SSTA_ERR_INVALID_ARG;
  if (C % 8 != 0 || rows > ((int64_t)1 << 36) / ((C + 127) / 128)) return SSTA_ERR_UNSUPPORTED;
  SSTA_TRY(take(c, out));
  return aligned(x, 16) ? SSTA_OK : SSTA_ERR_ALIGNMENT;
}

ssta_status ssta_checkpoint_save(int64_t rows, int C, int dtype, const void* x, const ssta_checkpoint* out,
                                 void* stream) {
  NvtxRange nvtx("ssta_checkpoint_save");
  ssta_checkpoint c;
  SSTA_TRY(checkpoint_args(rows, C, dtype, x, out, &c));
  return from_cuda(launch_checkpoint_save(rows, C, dtype == SSTA_BF16, x, c, static_cast<cudaStream_t>(stream)));
}

ssta_status ssta_checkpoint_load(int64_t rows, int C, int dtype, const ssta_checkpoint* in, void* x, void* stream) {
  NvtxRange nvtx("ssta_checkpoint_load");
  ssta_checkpoint c;
  SSTA_TRY(checkpoint_args(rows, C, dtype, x, in, &c));
  return from_cuda(launch_checkpoint_load(rows, C, dtype == SSTA_BF16, &c, &x, 1, static_cast<cudaStream_t>(stream)));
}

// Bytes of one packed tensor's values, in whole 256-byte steps.
static size_t packed_bytes(const Geom& g) {
  return ((size_t)g.B * g.H * g.Lq * g.D * g.esize + 255) / 256 * 256;
}

ssta_status ssta_attention_bwd_checkpoint_workspace(const ssta_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return SSTA_ERR_INVALID_ARG;
  Geom g;
  SSTA_TRY(make_geom(desc, &g));
  *bytes = bwd_workspace_layout(g).total + 3 * packed_bytes(g);
  return SSTA_OK;
}

ssta_status ssta_attention_bwd_checkpoint(const ssta_desc* desc, const ssta_checkpoint* q, const ssta_checkpoint* k,
                                          const ssta_checkpoint* v, const ssta_checkpoint* o, const float* lse,
                                          const void* do_packed, const int32_t* kv_idx, const int32_t* kv_cnt,
                                          void* dq_packed, void* dk_packed, void* dv_packed, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  NvtxRange nvtx("ssta_attention_bwd_checkpoint");
  Geom g;
  SSTA_TRY(make_geom(desc, &g));
  if (g.dtype == SSTA_BF16 && g.N % 128 != 0) return SSTA_ERR_UNSUPPORTED;
  size_t need = 0;
  SSTA_TRY(ssta_attention_bwd_checkpoint_workspace(desc, &need));
  if (workspace == nullptr || workspace_bytes < need) return SSTA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSTA_ERR_ALIGNMENT;
  const bool empty = (int64_t)g.B * g.H == 0;
  const ssta_checkpoint* in[4] = {q, k, v, o};
  ssta_checkpoint c[4];
  for (int i = 0; i < 4; ++i) {
    if (!empty && in[i] == nullptr) return SSTA_ERR_INVALID_ARG;
    if (!empty) SSTA_TRY(take(in[i], &c[i]));
    if (!empty && c[i].format != c[0].format) return SSTA_ERR_INVALID_ARG;
  }
  const void* rest[] = {lse, do_packed, kv_idx, kv_cnt, dq_packed, dk_packed, dv_packed};
  for (const void* p : rest) {
    if (!empty && p == nullptr) return SSTA_ERR_INVALID_ARG;
    if (!aligned(p, 16)) return SSTA_ERR_ALIGNMENT;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(int32_t), s) != cudaSuccess) return SSTA_ERR_LAUNCH;
  if (empty) return SSTA_OK;
  // The tensor-core kernel takes its operands by TMA, so the values of q, k and v are
  // written out once (bf16: with the row statistics, where O is decoded too; fp32: O's
  // values go to dq's place, which the dQ kernel overwrites last).
  uint8_t* values = static_cast<uint8_t*>(workspace) + bwd_workspace_layout(g).total;
  void* x[3] = {values, values + packed_bytes(g), values + 2 * packed_bytes(g)};
  const bool bf16 = g.dtype == SSTA_BF16;
  if (!bf16) {
    const int64_t rows = (int64_t)g.B * g.H * g.Lq;
    cudaError_t e = launch_checkpoint_load(rows, g.D, false, c, x, 3, s);
    if (e == cudaSuccess) e = launch_checkpoint_load(rows, g.D, false, &c[3], &dq_packed, 1, s);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return from_cuda(launch_attention_bwd(g, x[0], x[1], x[2], bf16 ? nullptr : dq_packed, bf16 ? c : nullptr, lse,
                                        do_packed, kv_idx, kv_cnt, dq_packed, dk_packed, dv_packed, workspace, s));
}

}  // extern "C"
