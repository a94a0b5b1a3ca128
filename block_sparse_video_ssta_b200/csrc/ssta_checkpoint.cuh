// Reading 8-bit checkpoints by blocks of 256 threads: the body of the load kernel, which the
// attention backward's first kernel shares.
#pragma once

#include "ssta_norm.h"
#include "ssta_rows.cuh"

namespace ssta {
namespace ckpt {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / kGroupLanes;
constexpr int kPerThread = 4;   // groups per half-warp, every load issued before the first use
constexpr int kBlockGroups = kHalfWarps * kPerThread;

struct Params {
  const void* in[3];
  void* out[3];
  const uint8_t* exps[3];   // load; save writes exps[0]
  int64_t groups;
  int C, gpr, format;
};

// Element offset of vector `lane` of group gi, or -1 where the row ends inside the group.
__device__ __forceinline__ int64_t vec_offset(const Params& p, int64_t gi, int lane) {
  if (gi >= p.groups) return -1;
  if (p.C % kGroup == 0) return gi * kGroup + lane * kVec;   // groups follow one another
  const int64_t row = gi / p.gpr;
  const int ch = (int)(gi - row * p.gpr) * kGroup + lane * kVec;
  return ch < p.C ? row * p.C + ch : -1;
}

// Values of the groups of block `block` of tensor `which`.
template <typename T>
__device__ __forceinline__ void load_block(const Params& p, int which, int64_t block) {
  const int lane = threadIdx.x % kGroupLanes;
  const int64_t g0 = block * kBlockGroups + threadIdx.x / kGroupLanes;
  const uint8_t* codes = static_cast<const uint8_t*>(p.in[which]);
  const uint8_t* exps = p.exps[which];
  T* out = static_cast<T*>(p.out[which]);
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

inline Params params(int64_t rows, int C, int format) {
  Params p{};
  p.C = C;
  p.gpr = groups_per_row(C);
  p.groups = rows * p.gpr;
  p.format = format;
  return p;
}
inline unsigned blocks_for(int64_t groups) { return (unsigned)((groups + kBlockGroups - 1) / kBlockGroups); }

}  // namespace ckpt
}  // namespace ssta
