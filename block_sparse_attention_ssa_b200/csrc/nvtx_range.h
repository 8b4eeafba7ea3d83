// NVTX range of one entry-point call.
#pragma once

#include <nvtx3/nvToolsExt.h>

namespace ssa {

// One NVTX range per entry-point call, named after the call, so a profiler
// timeline (nsys, ncu --nvtx) shows which call enqueued which kernels.
// Header-only NVTX 3: without an attached tool the push / pop are no-ops.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace ssa
