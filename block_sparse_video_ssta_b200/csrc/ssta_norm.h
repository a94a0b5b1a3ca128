// Host-side declarations of the norm, gated-residual and checkpoint kernels.
#pragma once

#include "ssta_internal.h"

namespace ssta {

// Modulation rows: row i of the activations uses row i / mod_rows.
struct NormGeom {
  int64_t rows, mod_rows, mod_stride;
  int64_t groups;
  int C;
  int norm, post_norm;
  float eps, res_scale;
  bool bf16, param_f32;
};

ssta_status make_norm_geom(const ssta_norm_desc* d, NormGeom* g);

// One pass over the rows: [h = post_norm(y), r = res_scale * x + gate * h,] n = norm(r).
// Without y (y == NULL) r is x itself and is not written; n may be NULL (norm none).
struct NormFwdArgs {
  const void *x, *y, *post_weight, *gate, *weight, *scale, *shift;
  void *r, *n;
  float *post_mean, *post_rstd, *mean, *rstd;
  ssta_checkpoint y_save, r_save;   // codes == NULL: none
};
cudaError_t launch_norm_fwd(const NormGeom& g, const NormFwdArgs& a, cudaStream_t s);

// Backward of the same pass.  Without a gated residual (dy == NULL) dx = dR.
struct NormBwdArgs {
  const void *dr, *dn, *r, *y;              // dense activations (NULL: absent, or kept as a checkpoint)
  ssta_checkpoint r_saved, y_saved;         // codes == NULL: none
  const float *post_mean, *post_rstd, *mean, *rstd;
  const void *post_weight, *gate, *weight, *scale;
  void *dx, *dy;
  float *dpost_weight, *dgate, *dweight, *dscale, *dshift;
};
size_t norm_bwd_workspace_bytes(const NormGeom& g);
cudaError_t launch_norm_bwd(const NormGeom& g, const NormBwdArgs& a, void* workspace, cudaStream_t s);

cudaError_t launch_checkpoint_save(int64_t rows, int C, bool bf16, const void* x, const ssta_checkpoint& out,
                                   cudaStream_t s);
// `count` checkpoints of one shape and format at once (at most 3).
cudaError_t launch_checkpoint_load(int64_t rows, int C, bool bf16, const ssta_checkpoint* in, void* const* x, int count,
                                   cudaStream_t s);

}  // namespace ssta
