// Host-side services of the C ABI layer that its files share (defined in api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace dr {

// The calling thread's error message (dr_last_error): cleared by an entry point, set by a failure,
// which returns its status.
void host_clear_error();
int host_fail(int status, const char* fmt, ...);
// A call's workspace: the caller's `given` (checked for its alignment and size), or with none stream-ordered memory
// from the library's pool of the current device (`owned`: given back with hipFreeAsync). The pool is refused while the
// stream is being captured: a graph would hold it as memory nodes, and a replay of one of two such graphs has run its
// kernels on addresses that were not mapped. Returns a status.
int host_space(const char* what, int64_t need, void* given, int64_t given_bytes, uintptr_t align, hipStream_t stream,
               unsigned char** ws, bool* owned);
// With DR_DEBUG_VALIDATE set: cu_seqlens [nseq + 1] copied to the host and checked (synchronises).
int host_check_offsets(const int32_t* cu, int64_t nseq, int64_t tokens, hipStream_t stream);

}  // namespace dr
