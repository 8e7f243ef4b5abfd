// Host-side services of the C ABI layer that its files share (defined in api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace dr {

// The calling thread's error message (dr_last_error): cleared by an entry point, set by a failure,
// which returns its status.
void host_clear_error();
int host_fail(int status, const char* fmt, ...);
// Stream-ordered memory from the library's pool of the current device (released with hipFreeAsync).
hipError_t host_workspace(size_t bytes, hipStream_t stream, void** ptr);
// With DR_DEBUG_VALIDATE set: cu_seqlens [nseq + 1] copied to the host and checked (synchronises).
int host_check_offsets(const int32_t* cu, int64_t nseq, int64_t tokens, hipStream_t stream);

}  // namespace dr
