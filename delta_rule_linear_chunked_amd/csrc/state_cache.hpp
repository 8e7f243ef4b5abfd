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

hipError_t launch_state_pack(const CacheParams& p, bool e4m3, hipStream_t s);
hipError_t launch_state_unpack(const CacheParams& p, bool e4m3, hipStream_t s);

}  // namespace dr
