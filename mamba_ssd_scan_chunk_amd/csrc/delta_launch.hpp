// delta_launch.hpp -- host-side launchers of the gated delta rule.  Arguments
// are validated by the C ABI layer (delta_api.cpp) before any of these is
// called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

constexpr int64_t kDeltaC = 64;        // tokens a window
constexpr int64_t kDeltaMaxDim = 256;  // of a key or value head
constexpr int64_t kDeltaMaxStates = 65535;  // states after tokens

struct DeltaRows {
  int64_t q, k, v, dt, beta;  // elements from a token to the next
};
struct DeltaArgs {
  int64_t B, L, H, G, N, P;
  DeltaRows rows, grows;
  bool softplus, sigmoid, qk_norm;
  bool f32_products;  // of bf16 inputs; fp32 ones have no others
  float scale;
  const void *q, *k, *v, *dt, *beta;
  const float *A, *dt_bias;  // dt_bias may be null
  const float* h0;           // [B,H,N,P] or null
  const int* seq_idx;        // [B,L] or null
  void* y;
  float* hfin;               // may be null
  int64_t nseq;
  const int64_t* seq_last;
  float* seq_states;         // [nseq,H,N,P]
  // backward
  const void* dy;
  const float* dfinal;       // may be null
  void *dq, *dk, *dv, *ddt, *dbeta;
  float *dA, *ddt_bias, *dinit;  // ddt_bias, dinit may be null
  char* ws;
};
size_t delta_forward_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P);
size_t delta_backward_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P);
hipError_t launch_delta_forward(const DeltaArgs& a, bool bf16, hipStream_t s);
hipError_t launch_delta_backward(const DeltaArgs& a, bool bf16, hipStream_t s);
hipError_t launch_delta_step(const DeltaArgs& a, const float* state, float* state_out, bool bf16, hipStream_t s);

}  // namespace ssd
