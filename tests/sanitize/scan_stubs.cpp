// Stand-ins for the launches of the selective scan, the convolution and the norm, for a host-only build of the C ABI under the
// address and undefined-behaviour sanitizers: every launch reports that there is no device.
#include "../../delta_rule_linear_chunked_amd/csrc/scan.hpp"

namespace dr {

hipError_t launch_conv_fwd(ConvParams, int, bool, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_conv_step(const ConvParams&, int, bool, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_conv_bwd(ConvParams, int, bool, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_scan_fwd(ScanParams, const ScanPlan&, int, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_scan_step(const ScanParams&, int, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_scan_bwd(ScanParams, int, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm_fwd(const NormParams&, int, bool, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm_bwd(const NormParams&, bool, bool, hipStream_t) { return hipErrorNoDevice; }

}  // namespace dr
