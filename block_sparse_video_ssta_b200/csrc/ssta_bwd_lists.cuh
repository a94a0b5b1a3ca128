// The transposed kept lists of the attention backward, for its fp32 and bf16 kernels.
#pragma once

#include "ssta_internal.h"

namespace ssta {

// For key tile j of head bh: tidx[bh][j][0..tcnt) = query tiles i (ascending) whose
// kept list holds j.  Lists are ascending (as ssta_build_block_mask writes them).
// One warp, for w = bh * NQ + j.
__device__ __forceinline__ void transpose_lists(const Geom& g, int64_t w, const int32_t* __restrict__ kv_idx,
                                                const int32_t* __restrict__ kv_cnt, int32_t* __restrict__ tidx,
                                                int32_t* __restrict__ tcnt, int32_t* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)g.B * g.H * g.NQ) return;
  const int64_t bh = w / g.NQ;
  const int j = (int)(w - bh * g.NQ);
  int32_t* out = tidx + w * g.NQ;
  int n = 0;
  for (int i0 = 0; i0 < g.NQ; i0 += 32) {
    const int i = i0 + lane;
    bool keeps = false;
    if (i < g.NQ) {
      const int64_t lr = bh * g.NQ + i;
      int c = kv_cnt[lr];
      if (c < 0 || c > g.max_kept) {
        atomicExch(status, (int)SSTA_ERR_DEVICE_BOUNDS);
        c = c < 0 ? 0 : g.max_kept;
      }
      const int32_t* l = kv_idx + lr * g.max_kept;
      int lo = 0, hi = c;                      // first entry >= j
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (l[mid] < j) lo = mid + 1; else hi = mid;
      }
      keeps = lo < c && l[lo] == j;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, keeps);
    if (keeps) out[n + __popc(m & ((1u << lane) - 1u))] = i;
    n += __popc(m);
  }
  if (lane == 0) tcnt[w] = n;
}

}  // namespace ssta
