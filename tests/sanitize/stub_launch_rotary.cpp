// Test-only launchers of the rotation and norm of queries and keys for the host-only build of the C-ABI layer
// under AddressSanitizer and UndefinedBehaviorSanitizer (beside stub_launch.cpp): no device is present.
#include "gdn_rotary_launch.h"
namespace gdn {
hipError_t launch_rope(const RotaryArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_qk_norm_rope(const RotaryArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_qk_norm_rope_backward(const RotaryArgs&, hipStream_t) { return hipErrorNoDevice; }
}
