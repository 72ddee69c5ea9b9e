// api_util.cuh -- helpers of the entry-point files.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace hsa {

// An NVTX range around each launching entry point, named after it, so that a
// timeline (nsys, ncu's range filters) shows the library's calls.  Header-only
// NVTX: without an attached tool a range costs a null check.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

}  // namespace hsa

#define HSA_TRY(expr)                       \
    do {                                    \
        hsa_status_t s_ = (expr);           \
        if (s_ != HSA_OK) return s_;        \
    } while (0)
