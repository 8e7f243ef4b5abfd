// 8-bit state cache: parameter block and launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dr {

struct CacheParams {
  float* S;              // [nstates, H, d_k, d_v]
  uint8_t* codes;        // [nslots, H, d_k, d_v]
  float* scales;         // [nslots, H, d_k]
  const int32_t* state_idx;  // [count], null: n
  const int32_t* slot_idx;   // [count], null: n
  int64_t count, nstates, nslots;
  int32_t H, DK, DV;
};

constexpr int CACHE_VPT = 4;                  // float4 per thread
constexpr int CACHE_BLOCK = 256 * CACHE_VPT;  // float4 per workgroup
// Workgroups of one head's state, and whether a launch over `heads` states of one head fits (its work items are a 32-bit number).
constexpr int64_t cache_parts(int hsz) { return (hsz / 4 + CACHE_BLOCK - 1) / CACHE_BLOCK; }
constexpr bool cache_fits(int64_t heads, int hsz) { return heads * cache_parts(hsz) * 256 <= (int64_t)UINT32_MAX; }

hipError_t launch_state_pack(const CacheParams& p, bool e4m3, hipStream_t s);
hipError_t launch_state_unpack(const CacheParams& p, bool e4m3, hipStream_t s);

}  // namespace dr
