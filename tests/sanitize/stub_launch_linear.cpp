// Test-only launchers of linear attention and layer norm for the host-only build of the C-ABI layer
// under AddressSanitizer and UndefinedBehaviorSanitizer (beside stub_launch.cpp): no device is present.
#include "gdn_linear_launch.h"
namespace gdn {
hipError_t launch_linear_decode(const LinearArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_linear_prefill(const LinearArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_linear_backward(const LinearBackwardArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_layer_norm(const NormArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_layer_norm_backward(const NormBackwardArgs&, hipStream_t) { return hipErrorNoDevice; }
}
