// Stand-ins for the launches of the decayed linear attention and the state cache, for a host-only build of the C ABI
// under the address and undefined-behaviour sanitizers: every launch reports that there is no device.
#include "../../delta_rule_linear_chunked_amd/csrc/decay.hpp"
#include "../../delta_rule_linear_chunked_amd/csrc/state_cache.hpp"

namespace dr {

hipError_t launch_decay_fwd(DecayParams, const DecayPlan&, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_decay_step(const DecayParams&, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_decay_bwd(DecayParams, const DecayPlan&, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_state_pack(const CacheParams&, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_state_unpack(const CacheParams&, bool, hipStream_t) { return hipErrorNoDevice; }

}  // namespace dr
