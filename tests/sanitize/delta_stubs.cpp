// delta_stubs.cpp -- stand-ins for the device launchers of the delta rule, the
// group norm and 8-bit storage, for a host-only build of delta_api.cpp and
// group_api.cpp under AddressSanitizer and UndefinedBehaviorSanitizer (test
// infrastructure).  A launcher that is reached aborts.
#include <cstdio>
#include <cstdlib>

#include "delta_launch.hpp"
#include "group_launch.hpp"

namespace ssd {

[[noreturn]] static void reached(const char* what) {
  std::fprintf(stderr, "launcher reached on arguments that should have been rejected: %s\n", what);
  std::abort();
}

size_t delta_forward_ws_bytes(int64_t B, int64_t L, int64_t, int64_t, int64_t, int64_t) { return (size_t)(B + L); }
size_t delta_backward_ws_bytes(int64_t B, int64_t L, int64_t, int64_t, int64_t, int64_t) { return 2 * (size_t)(B + L); }
hipError_t launch_delta_forward(const DeltaArgs&, bool, hipStream_t) { reached("delta_forward"); }
hipError_t launch_delta_backward(const DeltaArgs&, bool, hipStream_t) { reached("delta_backward"); }
hipError_t launch_delta_step(const DeltaArgs&, const float*, float*, bool, hipStream_t) { reached("delta_step"); }
size_t group_norm_backward_ws_bytes(int64_t, int64_t D, int64_t) { return (size_t)D * 8; }
hipError_t launch_group_norm_forward(const GroupNormArgs&, bool, hipStream_t) { reached("group_norm_forward"); }
hipError_t launch_group_norm_backward(const GroupNormArgs&, bool, hipStream_t) { reached("group_norm_backward"); }
hipError_t launch_pack8(int64_t, int64_t, const void*, int64_t, bool, int8_t*, uint16_t*, hipStream_t) { reached("pack8"); }
hipError_t launch_unpack8(int64_t, int64_t, const int8_t*, const uint16_t*, void*, int64_t, bool, hipStream_t) {
  reached("unpack8");
}

}  // namespace ssd
