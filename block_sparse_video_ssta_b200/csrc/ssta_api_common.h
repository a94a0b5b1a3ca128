// Helpers of the C ABI's entry points.
#pragma once

#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

namespace ssta {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// NVTX range over one library call (host side: validation and kernel enqueue), so a
// timeline tool shows each call by name; without a tool attached it costs a few ns.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace ssta
