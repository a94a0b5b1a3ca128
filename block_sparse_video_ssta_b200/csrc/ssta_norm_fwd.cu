// Forward of the norms around a block: y = norm(x) * w * (1 + scale) + shift, and behind
// a block r = res_scale * x + gate * post_norm(y) with the next norm of r, in one pass.
//
// Every row is read once, held in registers, and written once: the statistics (mean, then
// the mean square of the differences, both fp32) are sums over registers and warp
// shuffles, so the kernel moves 2 (norm) or 4 (residual) elements per channel and is
// bound by HBM.  A row belongs to one warp up to 2,048 channels (half a warp up to 128)
// and to 2 or 4 warps above, which exchange their partial sums through shared memory;
// up to 8 vectors of 8 channels per lane and array keep enough loads in flight without
// any staging.  Weights and modulation rows are shared by many rows and come from L1/L2.
// An 8-bit checkpoint of an input or of r is written in the same pass from the registers.
#include "ssta_norm.h"
#include "ssta_rows.cuh"

#include <algorithm>

namespace ssta {
namespace {

using namespace rows;

constexpr int kFwdThreads = 256;

struct FwdParams {
  NormFwdArgs a;
  uint32_t rows, mod_rows;
  int64_t mod_stride;
  int C, norm, post_norm, groups_per_row;
  float eps, res_scale, inv_c;
};

// Sum of v over the lanes (and warps) of a row; every thread of the row gets it.
template <int LPR, int WPR>
__device__ __forceinline__ float row_sum(float v, float* exchange, int slot) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) exchange[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(WPR * 32) : "memory");
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += exchange[slot * WPR + w];
  }
  return v;
}

// mean and 1 / deviation of the row in v (lanes beyond C hold zeros in v and are left out).
template <int NV, int LPR, int WPR>
__device__ __forceinline__ void row_stats(const float (&v)[NV][kVec], const FwdParams& p, int kind, int lane,
                                          float* exchange, int slot, float& mean, float& rstd) {
  mean = 0.f;
  if (kind == SSTA_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s += v[i][j];
    mean = row_sum<LPR, WPR>(s, exchange, slot) * p.inv_c;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * LPR * WPR + lane) * kVec < p.C) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float d = v[i][j] - mean;
        q = fmaf(d, d, q);
      }
    }
  }
  // exchange + 8: the second sum of a row never meets readers of the first
  rstd = rsqrtf(row_sum<LPR, WPR>(q, exchange + kFwdThreads / 32, slot) * p.inv_c + p.eps);
}

template <int NV, int LPR, int WPR>
__device__ __forceinline__ void save_row(const float (&v)[NV][kVec], const FwdParams& p, const ssta_checkpoint& c,
                                         uint32_t row, int lane, bool alive) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = (i * LPR * WPR + lane) * kVec;
    const int E = group_exponent(group_amax(v[i]), c.format);
    if (alive && ch < p.C) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.codes) + (int64_t)row * p.C + ch) = encode8(v[i], E, c.format);
      if (ch % kGroup == 0) c.exponents[(int64_t)row * p.groups_per_row + ch / kGroup] = (uint8_t)E;
    }
  }
}

// NV vectors per lane, LPR lanes and WPR warps per row; POST: with a gated residual.
template <typename T, typename P, int NV, int LPR, int WPR, bool POST>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_kernel(const __grid_constant__ FwdParams p) {
  constexpr int kRowThreads = LPR * WPR, kSlots = kFwdThreads / kRowThreads;
  __shared__ float exchange[4][kFwdThreads / 32];
  const int slot = threadIdx.x / kRowThreads, lane = threadIdx.x % kRowThreads;
  const uint32_t row = blockIdx.x * kSlots + slot;
  const bool alive = row < p.rows;   // dead rows go along with the shuffles and barriers
  const NormFwdArgs& a = p.a;
  const int64_t base = (int64_t)row * p.C;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* y = static_cast<const T*>(a.y) + base;
  Raw<T> xr[NV], yr[POST ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = (i * kRowThreads + lane) * kVec;
    const bool in = alive && ch < p.C;
    xr[i] = in ? load_raw(x + ch) : zero_raw<T>();
    if constexpr (POST) yr[i] = in ? load_raw(y + ch) : zero_raw<T>();
  }
  const int64_t mod = p.mod_rows < p.rows ? (int64_t)(row / p.mod_rows) * p.mod_stride : 0;
  float v[NV][kVec];
  if constexpr (POST) {
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack(yr[i], v[i]);
    if (a.y_save.codes != nullptr) save_row<NV, LPR, WPR>(v, p, a.y_save, row, lane, alive);
    float pm = 0.f, pr = 1.f;
    if (p.post_norm != SSTA_NORM_NONE) {
      row_stats<NV, LPR, WPR>(v, p, p.post_norm, lane, exchange[0], slot, pm, pr);
      if (alive && lane == 0) {
        if (a.post_mean != nullptr) a.post_mean[row] = pm;
        if (a.post_rstd != nullptr) a.post_rstd[row] = pr;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * kRowThreads + lane) * kVec;
      if (!(alive && ch < p.C)) continue;   // stays zero
      if (p.post_norm != SSTA_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] = (v[i][j] - pm) * pr;
        if (a.post_weight != nullptr) {
          float w[kVec];
          load8(static_cast<const P*>(a.post_weight) + ch, w);
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[i][j] *= w[j];
        }
      }
      if (a.gate != nullptr) {
        float w[kVec];
        load8(static_cast<const P*>(a.gate) + mod + ch, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] = __fmul_rn(v[i][j], w[j]);
      }
      // products and sum rounded one by one: r does not depend on what the compiler fuses
      float xv[kVec];
      unpack(xr[i], xv);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = __fadd_rn(__fmul_rn(p.res_scale, xv[j]), v[i][j]);
      const Raw<T> out = pack(v[i], T());
      store_raw(static_cast<T*>(a.r) + base + ch, out);
      xr[i] = out;   // r as stored, for its checkpoint
    }
    if (a.r_save.codes != nullptr) {
      float s[NV][kVec];
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack(xr[i], s[i]);
      save_row<NV, LPR, WPR>(s, p, a.r_save, row, lane, alive);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack(xr[i], v[i]);
    if (a.r_save.codes != nullptr) save_row<NV, LPR, WPR>(v, p, a.r_save, row, lane, alive);
  }
  if (p.norm == SSTA_NORM_NONE) return;
  float mean, rstd;
  row_stats<NV, LPR, WPR>(v, p, p.norm, lane, exchange[2], slot, mean, rstd);
  if (alive && lane == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = (i * kRowThreads + lane) * kVec;
    if (!(alive && ch < p.C)) continue;
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = (v[i][j] - mean) * rstd;
    if (a.weight != nullptr) {
      float w[kVec];
      load8(static_cast<const P*>(a.weight) + ch, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] *= w[j];
    }
    if (a.scale != nullptr) {
      float w[kVec];
      load8(static_cast<const P*>(a.scale) + mod + ch, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = fmaf(v[i][j], w[j], v[i][j]);
    }
    if (a.shift != nullptr) {
      float w[kVec];
      load8(static_cast<const P*>(a.shift) + mod + ch, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] += w[j];
    }
    store8(static_cast<T*>(a.n) + base + ch, v[i]);
  }
}

template <typename T, typename P, int NV, int LPR, int WPR>
cudaError_t launch_shape(const FwdParams& p, cudaStream_t s) {
  constexpr int kSlots = kFwdThreads / (LPR * WPR);
  const unsigned blocks = (p.rows + kSlots - 1) / kSlots;
  if (p.a.y != nullptr)
    norm_fwd_kernel<T, P, NV, LPR, WPR, true><<<blocks, kFwdThreads, 0, s>>>(p);
  else
    norm_fwd_kernel<T, P, NV, LPR, WPR, false><<<blocks, kFwdThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t launch_types(const FwdParams& p, cudaStream_t s) {
  if (p.C <= 128) return launch_shape<T, P, 1, 16, 1>(p, s);
  if (p.C <= 256) return launch_shape<T, P, 1, 32, 1>(p, s);
  if (p.C <= 512) return launch_shape<T, P, 2, 32, 1>(p, s);
  if (p.C <= 1024) return launch_shape<T, P, 4, 32, 1>(p, s);
  if (p.C <= 2048) return launch_shape<T, P, 8, 32, 1>(p, s);
  if (p.C <= 4096) return launch_shape<T, P, 8, 32, 2>(p, s);
  return launch_shape<T, P, 8, 32, 4>(p, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormGeom& g, const NormFwdArgs& a, cudaStream_t s) {
  FwdParams p{};
  p.a = a;
  p.rows = (uint32_t)g.rows;
  p.mod_rows = (uint32_t)g.mod_rows;
  p.mod_stride = g.mod_stride;
  p.C = g.C;
  p.norm = g.norm;
  p.post_norm = g.post_norm;
  p.groups_per_row = groups_per_row(g.C);
  p.eps = g.eps;
  p.res_scale = g.res_scale;
  p.inv_c = 1.0f / (float)g.C;
  if (g.bf16) return g.param_f32 ? launch_types<__nv_bfloat16, float>(p, s) : launch_types<__nv_bfloat16, __nv_bfloat16>(p, s);
  return g.param_f32 ? launch_types<float, float>(p, s) : launch_types<float, __nv_bfloat16>(p, s);
}

}  // namespace ssta
