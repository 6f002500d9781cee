// Test-only launchers of the gated linear recurrence for the host-only build of the C-ABI layer under
// AddressSanitizer and UndefinedBehaviorSanitizer (beside stub_launch.cpp): no device is present.
#include "gdn_scan_launch.h"
namespace gdn {
hipError_t launch_scan_decode(const ScanArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_scan_prefill(const ScanArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_scan_backward(const ScanArgs&, hipStream_t) { return hipErrorNoDevice; }
}
