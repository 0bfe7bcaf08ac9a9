// group_launch.hpp -- host-side launchers of the group norm and of activations
// in 8 bits.  Arguments are validated by the C ABI layer (group_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

struct GroupNormArgs {
  int64_t rows, D, G;      // D columns in G groups
  bool rms, gate_first, silu, shared;
  float eps;
  const void* x;           // kept8: int8
  const void* z;           // may be null
  int64_t z_row, dz_row;
  const uint16_t* xs;      // scales of x, z in 8 bits, or null
  const uint16_t* zs;
  const float* w;
  const float* bias;       // may be null
  void* y;
  float* mean;             // null for rms
  float* rstd;
  // backward
  const void* dy;
  void* dx;
  void* dz;                // null exactly when z is
  float* dw;
  float* db;               // may be null
  float* ws;
};
constexpr int64_t kGroupNormMaxSize = 16384;  // columns of a group
size_t group_norm_backward_ws_bytes(int64_t rows, int64_t D, int64_t G);
hipError_t launch_group_norm_forward(const GroupNormArgs& a, bool bf16, hipStream_t s);
hipError_t launch_group_norm_backward(const GroupNormArgs& a, bool bf16, hipStream_t s);

constexpr int64_t kPackBlock = 64;  // values that share a scale
hipError_t launch_pack8(int64_t rows, int64_t D, const void* x, int64_t x_row, bool bf16, int8_t* q, uint16_t* scale,
                        hipStream_t s);
hipError_t launch_unpack8(int64_t rows, int64_t D, const int8_t* q, const uint16_t* scale, void* x, int64_t x_row,
                          bool bf16, hipStream_t s);

}  // namespace ssd
