// 8-bit activation checkpoints on their own: save (quantise) and load (values back).
// Elementwise over groups of 128 channels, one half-warp per group (8 channels per lane:
// a group's largest magnitude is three register steps and four shuffles), bound by HBM:
// 3 bytes per bf16 element and 1/128 byte of exponents in either direction.  219,600 x
// 2,048 bf16 there and back: 408-423 us back to back, 0.97-1.01 of the measured copy rate (400
// us with L2 flushed between passes).
#include "ssta_checkpoint.cuh"

namespace ssta {
namespace {

using namespace ckpt;

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_save_kernel(const __grid_constant__ Params p) {
  const int lane = threadIdx.x % kGroupLanes;
  const int64_t g0 = (int64_t)blockIdx.x * kBlockGroups + threadIdx.x / kGroupLanes;
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
__global__ void __launch_bounds__(kThreads) checkpoint_load_kernel(const __grid_constant__ Params p) {
  load_block<T>(p, blockIdx.y, blockIdx.x);
}

}  // namespace

cudaError_t launch_checkpoint_save(int64_t rows, int C, bool bf16, const void* x, const ssta_checkpoint& out,
                                   cudaStream_t s) {
  Params p = params(rows, C, out.format);
  p.in[0] = x;
  p.out[0] = out.codes;
  p.exps[0] = out.exponents;
  if (bf16)
    checkpoint_save_kernel<__nv_bfloat16><<<blocks_for(p.groups), kThreads, 0, s>>>(p);
  else
    checkpoint_save_kernel<float><<<blocks_for(p.groups), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_load(int64_t rows, int C, bool bf16, const ssta_checkpoint* in, void* const* x, int count,
                                   cudaStream_t s) {
  Params p = params(rows, C, in[0].format);
  for (int i = 0; i < count; ++i) {
    p.in[i] = in[i].codes;
    p.exps[i] = in[i].exponents;
    p.out[i] = x[i];
  }
  const dim3 grid(blocks_for(p.groups), count);
  if (bf16)
    checkpoint_load_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else
    checkpoint_load_kernel<float><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssta
