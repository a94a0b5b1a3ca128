// 8-bit activation checkpoints on their own: save (quantise) and load (values back).
// Elementwise over groups of 128 channels, one half-warp per group (8 channels per lane:
// a group's largest magnitude is three register steps and four shuffles), bound by HBM:
// 3 bytes per bf16 element and 1/128 byte of exponents in either direction.  219,600 x
// 2,048 bf16 there and back: 400 us, 6.8 TB/s, 1.03 of the measured copy rate.
#include "ssta_norm.h"
#include "ssta_rows.cuh"

namespace ssta {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / kGroupLanes;
constexpr int kPerThread = 4;   // groups per half-warp, every load issued before the first use

struct CkptParams {
  const void* in[3];
  void* out[3];
  const uint8_t* exps[3];   // load; save writes exps[0]
  int64_t groups;
  int C, gpr, format;
};

// Element offset of vector `lane` of group gi, or -1 where the row ends inside the group.
__device__ __forceinline__ int64_t vec_offset(const CkptParams& p, int64_t gi, int lane) {
  if (gi >= p.groups) return -1;
  if (p.C % kGroup == 0) return gi * kGroup + lane * kVec;   // groups follow one another
  const int64_t row = gi / p.gpr;
  const int ch = (int)(gi - row * p.gpr) * kGroup + lane * kVec;
  return ch < p.C ? row * p.C + ch : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_save_kernel(const __grid_constant__ CkptParams p) {
  const int lane = threadIdx.x % kGroupLanes;
  const int64_t g0 = (int64_t)blockIdx.x * (kHalfWarps * kPerThread) + threadIdx.x / kGroupLanes;
  Raw<T> raw[kPerThread];
  int64_t off[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    off[i] = vec_offset(p, g0 + i * kHalfWarps, lane);
    raw[i] = off[i] >= 0 ? load_raw(static_cast<const T*>(p.in[0]) + off[i]) : zero_raw<T>();
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const V8 v = unpack(raw[i]);
    const int E = group_exponent(group_amax(v), p.format);
    if (off[i] >= 0) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out[0]) + off[i]) = encode8(v, E, p.format);
      if (lane == 0) const_cast<uint8_t*>(p.exps[0])[g0 + i * kHalfWarps] = (uint8_t)E;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_load_kernel(const __grid_constant__ CkptParams p) {
  const int lane = threadIdx.x % kGroupLanes;
  const int64_t g0 = (int64_t)blockIdx.x * (kHalfWarps * kPerThread) + threadIdx.x / kGroupLanes;
  const uint8_t* codes = static_cast<const uint8_t*>(p.in[blockIdx.y]);
  const uint8_t* exps = p.exps[blockIdx.y];
  T* out = static_cast<T*>(p.out[blockIdx.y]);
  uint2 c[kPerThread];
  int E[kPerThread];
  int64_t off[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    off[i] = vec_offset(p, g0 + i * kHalfWarps, lane);
    if (off[i] >= 0) {
      c[i] = *reinterpret_cast<const uint2*>(codes + off[i]);
      E[i] = exps[g0 + i * kHalfWarps];
    }
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (off[i] < 0) continue;
    store8(out + off[i], mul(decode8(c[i], p.format), code_scale(E[i])));
  }
}

unsigned blocks_for(int64_t groups) {
  const int64_t per_block = kHalfWarps * kPerThread;
  return (unsigned)((groups + per_block - 1) / per_block);
}

}  // namespace

cudaError_t launch_checkpoint_save(int64_t rows, int C, bool bf16, const void* x, const ssta_checkpoint& out,
                                   cudaStream_t s) {
  CkptParams p{};
  p.in[0] = x;
  p.out[0] = out.codes;
  p.exps[0] = out.exponents;
  p.C = C;
  p.gpr = groups_per_row(C);
  p.groups = rows * p.gpr;
  p.format = out.format;
  if (bf16)
    checkpoint_save_kernel<__nv_bfloat16><<<blocks_for(p.groups), kThreads, 0, s>>>(p);
  else
    checkpoint_save_kernel<float><<<blocks_for(p.groups), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_load(int64_t rows, int C, bool bf16, const ssta_checkpoint* in, void* const* x, int count,
                                   cudaStream_t s) {
  CkptParams p{};
  for (int i = 0; i < count; ++i) {
    p.in[i] = in[i].codes;
    p.exps[i] = in[i].exponents;
    p.out[i] = x[i];
  }
  p.C = C;
  p.gpr = groups_per_row(C);
  p.groups = rows * p.gpr;
  p.format = in[0].format;
  const dim3 grid(blocks_for(p.groups), count);
  if (bf16)
    checkpoint_load_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else
    checkpoint_load_kernel<float><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssta
