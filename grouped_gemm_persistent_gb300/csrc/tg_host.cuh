// tg_host.cuh - what the translation units of the host API share: failures and their
// messages, the state of the current device, the workspace pool, tensor maps and the
// launch counter.  Defined in tg_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg.h"
#include "tg_kernel.cuh"

namespace tg {
namespace host {

constexpr int64_t MAX_DIM = (int64_t(1) << 31) - 1;

// Record the message of a failing call and return its status.
tg_status fail(tg_status s, const char* fmt, ...);
tg_status cuda_fail(cudaError_t e, const char* what);

// The current device, checked to be sm_103 (once per device; allocates nothing).
struct Device {
    int id = 0;
    int sms = 0;
    ErrorRecord* err = nullptr;
};
tg_status device(Device* out);

// `bytes` of the library's stream-ordered pool on the current device; released with cudaFreeAsync.
tg_status workspace(size_t bytes, cudaStream_t stream, const char* what, void** out);

// Look up cuTensorMapEncodeTiled (once); encode_bytes needs it.
tg_status encoder();

// Tensor map of 8-bit elements with 128-byte swizzle: dims and box innermost first, strides in
// bytes for the outer dimensions.
tg_status encode_bytes(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                       const uint32_t* box, const char* what);

// The launch-wide fields of Params: error record, wait budget and the armed withhold hook
// (consumed; an armed trace is left for the next launch that records one).
void launch_params(Params* p, ErrorRecord* err);

void count_launches(int n);

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace host
}  // namespace tg
