// layer_stubs.cpp -- stand-ins for the layer operators' device launchers, for a
// host-only build of layer_api.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer (test infrastructure).  The driver only makes
// calls that must be rejected: a launcher that is reached aborts.
#include <cstdio>
#include <cstdlib>

#include "layer_launch.hpp"

namespace ssd {

[[noreturn]] static void reached(const char* what) {
  std::fprintf(stderr, "launcher reached on arguments that should have been rejected: %s\n", what);
  std::abort();
}

bool scan_dstate_supported(int64_t N) { return N > 0 && N % 4 == 0 && N <= 256; }
size_t conv_backward_ws_bytes(int64_t B, int64_t, int64_t D, int W) { return (size_t)B + (size_t)D * (size_t)W; }
size_t scan_forward_ws_bytes(int64_t, int64_t L, int64_t D, int64_t, int64_t) { return (size_t)(L + D); }
size_t scan_backward_ws_bytes(int64_t, int64_t L, int64_t D, int64_t, int64_t) { return 2 * (size_t)(L + D); }
size_t norm_backward_ws_bytes(int64_t, int64_t D) { return (size_t)D * 8; }
hipError_t launch_conv_forward(const ConvArgs&, bool, hipStream_t) { reached("conv_forward"); }
hipError_t launch_conv_backward(const ConvArgs&, bool, hipStream_t) { reached("conv_backward"); }
hipError_t launch_conv_step(const ConvArgs&, const void*, void*, bool, hipStream_t) { reached("conv_step"); }
hipError_t launch_scan_forward(const ScanArgs&, bool, hipStream_t) { reached("scan_forward"); }
hipError_t launch_scan_backward(const ScanArgs&, bool, hipStream_t) { reached("scan_backward"); }
hipError_t launch_scan_step(const ScanArgs&, const float*, float*, bool, hipStream_t) { reached("scan_step"); }
hipError_t launch_norm_forward(const NormArgs&, bool, hipStream_t) { reached("norm_forward"); }
hipError_t launch_norm_backward(const NormArgs&, bool, hipStream_t) { reached("norm_backward"); }

}  // namespace ssd
