// Forward of the norms around a block: y = norm(x) * w * (1 + scale) + shift, and behind
// a block r = res_scale * x + gate * post_norm(y) with the next norm of r, in one pass.
//
// Every row is read once, held in registers, and written once: the statistics (mean, then
// the mean square of the differences, both fp32) are sums over registers and warp
// shuffles, so the kernel moves 2 (norm) or 4 (residual) elements per channel and is
// bound by HBM.  A row belongs to one warp up to 1,024 channels (half a warp up to 128; two
// warps from 769 on where a residual adds a second array) and to 2, 4 or 8 warps above,
// which exchange their partial sums through shared memory; a thread holds two to four
// vectors of 8 channels per array, of one wide row or of several narrow ones, which keeps
// enough loads in flight without any staging.  Weights and modulation rows are shared by
// many rows and come from L1/L2.  An 8-bit checkpoint of an input or of r is written in the
// same pass from the registers.
// Measured, passes back to back (of the measured copy rate; in parentheses with L2 flushed
// between passes, which leaves the GPU pauses): residual and norm of 111,600 x 2,048 bf16
// 309 us, 0.90 (295 us, 0.94), with two int8 saves 444 us, 0.78; RMS norm of 1,785,600 x 128
// bf16 154-164 us, 0.86-0.90 (152 us, 0.93); 97,656 x 1,024 fp32 (0.98).
#include "ssta_norm.h"
#include "ssta_rows.cuh"

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

// Sums of v[u] over the lanes (and warps) of U rows; every thread of a row gets its row's.
// `exchange` is used by one call only: a second sum never meets readers of the first.
template <int U, int LPR, int WPR>
__device__ __forceinline__ void row_sums(float (&v)[U], float (*exchange)[kFwdThreads / 32], int slot) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], off);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) exchange[u][warp] = v[u];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(WPR * 32) : "memory");
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) v[u] += exchange[u][slot * WPR + w];
    }
  }
}

// mean and 1 / deviation of U rows (channels beyond C hold zeros in v and are left out).
template <int NV, int U, int LPR, int WPR>
__device__ __forceinline__ void row_stats(const V8 (&v)[U][NV], const FwdParams& p, int kind, int lane,
                                          float (*exchange)[kFwdThreads / 32], int slot, float (&mean)[U],
                                          float (&rstd)[U]) {
  float t[U];
#pragma unroll
  for (int u = 0; u < U; ++u) mean[u] = 0.f;
  if (kind == SSTA_NORM_LAYER) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      V8 s = v[u][0];
#pragma unroll
      for (int i = 1; i < NV; ++i) s = add(s, v[u][i]);
      t[u] = sum(s);
    }
    row_sums<U, LPR, WPR>(t, exchange, slot);
#pragma unroll
    for (int u = 0; u < U; ++u) mean[u] = t[u] * p.inv_c;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    V8 q = fill(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const V8 d = add(v[u][i], fill((i * LPR * WPR + lane) * kVec < p.C ? -mean[u] : 0.f));
      q = fma(d, d, q);
    }
    t[u] = sum(q);
  }
  row_sums<U, LPR, WPR>(t, exchange + U, slot);
#pragma unroll
  for (int u = 0; u < U; ++u) rstd[u] = rsqrtf(t[u] * p.inv_c + p.eps);
}

__device__ __forceinline__ void save8(const V8& v, const FwdParams& p, const ssta_checkpoint& c, uint32_t row, int ch,
                                      bool in) {
  const int E = group_exponent(group_amax(v), c.format);
  if (in) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.codes) + (int64_t)row * p.C + ch) = encode8(v, E, c.format);
    if (ch % kGroup == 0) c.exponents[(int64_t)row * p.groups_per_row + ch / kGroup] = (uint8_t)E;
  }
}

// Eight elements of an optional vector (`other` where it is absent).
template <typename P>
__device__ __forceinline__ V8 param8(const void* v, int64_t at, bool in, float other) {
  return v == nullptr ? fill(other) : in ? load8(static_cast<const P*>(v) + at) : fill(0.f);
}

// NV vectors per lane and row, U rows per thread, LPR lanes and WPR warps per row; POST:
// with a gated residual.  Blocks per SM: four without a residual (64 registers, for which the
// kernels with four vectors per thread up to 512 channels store 24 to 80 bytes per thread to
// local memory; three and 76 registers take 162 us instead of 152 us for 1,785,600 rows of
// 128 bf16 channels, and so do two rows per thread with five blocks), three with one (80 registers), two where more is held.
template <typename T, typename P, int NV, int U, int LPR, int WPR, bool POST>
__global__ void __launch_bounds__(kFwdThreads, !POST ? 4 : sizeof(T) == 2 && WPR > 1 ? 3 : 2) norm_fwd_kernel(const __grid_constant__ FwdParams p) {
  constexpr int kRowThreads = LPR * WPR, kSlots = kFwdThreads / kRowThreads;
  __shared__ float exchange[4 * U][kFwdThreads / 32];
  const int slot = threadIdx.x / kRowThreads, lane = threadIdx.x % kRowThreads;
  const uint32_t row0 = (blockIdx.x * kSlots + slot) * U;   // rows past the end go along with shuffles and barriers
  const NormFwdArgs& a = p.a;
  const int64_t base = (int64_t)row0 * p.C;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* y = static_cast<const T*>(a.y) + base;
  Raw<T> xr[U][NV], yr[POST ? U : 1][POST ? NV : 1];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * kRowThreads + lane) * kVec;
      const bool in = row0 + u < p.rows && ch < p.C;
      xr[u][i] = in ? load_raw(x + u * p.C + ch) : zero_raw<T>();
      if constexpr (POST) yr[u][i] = in ? load_raw(y + u * p.C + ch) : zero_raw<T>();
    }
  }
  // rows of a thread may belong to different modulation rows
  int64_t mod[U];
#pragma unroll
  for (int u = 0; u < U; ++u) mod[u] = p.mod_rows < p.rows ? (int64_t)((row0 + u) / p.mod_rows) * p.mod_stride : 0;
  // A thread with one vector fetches its parameters together with it: few rows are a matter
  // of latency, and the loads would otherwise start behind each reduction.
  constexpr bool kEarly = NV * U == 1;
  V8 early[kEarly ? 5 : 1];
  if constexpr (kEarly) {
    const int ch = lane * kVec;
    const bool in = row0 < p.rows && ch < p.C;
    early[0] = param8<P>(a.weight, ch, in, 1.f);
    early[1] = param8<P>(a.scale, mod[0] + ch, in, 0.f);
    early[2] = param8<P>(a.shift, mod[0] + ch, in, 0.f);
    if constexpr (POST) {
      early[3] = param8<P>(a.post_weight, ch, in, 1.f);
      early[4] = param8<P>(a.gate, mod[0] + ch, in, 1.f);
    }
  }
  V8 v[U][NV];
  float mean[U], rstd[U];
  if constexpr (POST) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[u][i] = unpack(yr[u][i]);
    if (a.y_save.codes != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int ch = (i * kRowThreads + lane) * kVec;
          save8(v[u][i], p, a.y_save, row0 + u, ch, row0 + u < p.rows && ch < p.C);
        }
    }
    if (p.post_norm != SSTA_NORM_NONE) {
      row_stats<NV, U, LPR, WPR>(v, p, p.post_norm, lane, exchange, slot, mean, rstd);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (row0 + u < p.rows && lane == 0) {
          if (a.post_mean != nullptr) a.post_mean[row0 + u] = mean[u];
          if (a.post_rstd != nullptr) a.post_rstd[row0 + u] = rstd[u];
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = (i * kRowThreads + lane) * kVec;
        const V8 w = kEarly ? early[kEarly ? 3 : 0] : param8<P>(a.post_weight, ch, ch < p.C, 1.f);
#pragma unroll
        for (int u = 0; u < U; ++u) v[u][i] = mul(mul(add(v[u][i], fill(-mean[u])), rstd[u]), w);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = (i * kRowThreads + lane) * kVec;
        const bool in = row0 + u < p.rows && ch < p.C;
        if (a.gate != nullptr) v[u][i] = mul(v[u][i], kEarly ? early[kEarly ? 4 : 0] : param8<P>(a.gate, mod[u] + ch, in, 1.f));
        // products and sum rounded one by one: r does not depend on what gets fused
        v[u][i] = add(mul(unpack(xr[u][i]), p.res_scale), v[u][i]);
        if (!in) v[u][i] = fill(0.f);
        xr[u][i] = pack(v[u][i], T());   // r as stored
        if (in) store_raw(static_cast<T*>(a.r) + base + u * p.C + ch, xr[u][i]);
      }
    }
    if (a.r_save.codes != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int ch = (i * kRowThreads + lane) * kVec;
          save8(unpack(xr[u][i]), p, a.r_save, row0 + u, ch, row0 + u < p.rows && ch < p.C);
        }
    }
    if (p.norm == SSTA_NORM_NONE) return;
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = (i * kRowThreads + lane) * kVec;
        v[u][i] = unpack(xr[u][i]);
        if (a.r_save.codes != nullptr) save8(v[u][i], p, a.r_save, row0 + u, ch, row0 + u < p.rows && ch < p.C);
      }
    }
  }
  row_stats<NV, U, LPR, WPR>(v, p, p.norm, lane, exchange + 2 * U, slot, mean, rstd);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row0 + u < p.rows && lane == 0) {
      if (a.mean != nullptr) a.mean[row0 + u] = mean[u];
      if (a.rstd != nullptr) a.rstd[row0 + u] = rstd[u];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = (i * kRowThreads + lane) * kVec;
    const V8 w = kEarly ? early[0] : param8<P>(a.weight, ch, ch < p.C, 1.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = row0 + u < p.rows && ch < p.C;
      V8 n = mul(add(v[u][i], fill(-mean[u])), rstd[u]);
      if (a.weight != nullptr) n = mul(n, w);
      if (a.scale != nullptr) n = fma(n, kEarly ? early[kEarly ? 1 : 0] : param8<P>(a.scale, mod[u] + ch, in, 0.f), n);
      if (a.shift != nullptr) n = add(n, kEarly ? early[kEarly ? 2 : 0] : param8<P>(a.shift, mod[u] + ch, in, 0.f));
      if (in) store8(static_cast<T*>(a.n) + base + u * p.C + ch, n);
    }
  }
}

template <typename T, typename P, int NV, int U, int LPR, int WPR, bool POST>
cudaError_t launch_rows(const FwdParams& p, cudaStream_t s) {
  constexpr int kRows = kFwdThreads / (LPR * WPR) * U;
  norm_fwd_kernel<T, P, NV, U, LPR, WPR, POST><<<(p.rows + kRows - 1) / kRows, kFwdThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P, int WPR, bool POST>
cudaError_t launch_wide(const FwdParams& p, cudaStream_t s) {
  return p.C <= 768 * WPR ? launch_rows<T, P, 3, 1, 32, WPR, POST>(p, s) : launch_rows<T, P, 4, 1, 32, WPR, POST>(p, s);
}

template <typename T, typename P, bool POST>
cudaError_t launch_shape(const FwdParams& p, cudaStream_t s) {
  constexpr int kU = POST ? 2 : 4;   // four vectors per thread, of one array or of two
  if (p.C <= 128) return launch_rows<T, P, 1, kU, 16, 1, POST>(p, s);
  if (p.C <= 256) return launch_rows<T, P, 1, kU, 32, 1, POST>(p, s);
  // Few rows, all of them resident at once with a vector per thread (two blocks of 256
  // threads per SM): 256 x 2048 takes 7.7 us with four vectors per thread.
  if (p.C <= 2048) {
    const int warps = p.C <= 512 ? 2 : p.C <= 1024 ? 4 : 8;
    if ((int64_t)p.rows * warps <= 148 * 2 * (kFwdThreads / 32)) {
      if (warps == 2) return launch_rows<T, P, 1, 1, 32, 2, POST>(p, s);
      if (warps == 4) return launch_rows<T, P, 1, 1, 32, 4, POST>(p, s);
      return launch_rows<T, P, 1, 1, 32, 8, POST>(p, s);
    }
  }
  if (p.C <= 512) return launch_rows<T, P, 2, kU / 2, 32, 1, POST>(p, s);
  // Three or four vectors per thread, whichever leaves fewer lanes idle (100 M elements in
  // rows of 1,536 channels: 82 us with four).
  if (p.C <= 1024) {
    if (p.C <= 768) return launch_rows<T, P, 3, 1, 32, 1, POST>(p, s);
    // two arrays of four vectors need 113 registers: 184 us, against 151 us for two warps
    if constexpr (POST) return launch_rows<T, P, 2, 1, 32, 2, POST>(p, s);
    return launch_rows<T, P, 4, 1, 32, 1, POST>(p, s);
  }
  if (p.C <= 2048) return launch_wide<T, P, 2, POST>(p, s);
  if (p.C <= 4096) return launch_wide<T, P, 4, POST>(p, s);
  return launch_wide<T, P, 8, POST>(p, s);
}

template <typename T, typename P>
cudaError_t launch_types(const FwdParams& p, cudaStream_t s) {
  return p.a.y != nullptr ? launch_shape<T, P, true>(p, s) : launch_shape<T, P, false>(p, s);
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
