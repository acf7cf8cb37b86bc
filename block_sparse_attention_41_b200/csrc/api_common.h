// What the C entry points of the library share: the per-thread error text, the status helpers and
// the checks of pointers, sizes and the current device (defined in sol_attn_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sol_attn.h"

namespace sol {
namespace api {

void clear_error();
sol_status fail(sol_status s, const char* fmt, ...);
sol_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool size_ok(long long v, long long lim) { return v >= 1 && v <= lim; }

// The failure-detection test hook, taken by the launch that it is for (the attention or a linear layer): what the launch
// leaves out, or 0, and the limit of its device waits.
int take_drop(bool linear, uint64_t* wait_limit_ns);

// An sm_100 GPU is current: SOL_OK and its SM count.
sol_status current_device(int* num_sms);

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's driver entry point (no link-time libcuda), or null.
EncodeTiledFn encode_fn();

}  // namespace api
}  // namespace sol
