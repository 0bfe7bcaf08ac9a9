// layer_launch.hpp -- host-side launchers of the layer operators around the
// scan: causal convolution, selective scan and layer norm.  Arguments are
// validated by the C ABI layer (layer_api.cpp) before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

int device_cu_count();

// A flat grid of n < 2^32 blocks of up to 1024 threads.  A launch takes fewer
// than 2^32 threads a dimension, so past kGridX blocks the others lie along y;
// flat_block() in the kernel is the block's place, n and more for the last few.
constexpr uint32_t kGridX = 1u << 21;
inline dim3 flat_grid(int64_t n) {
  return n <= kGridX ? dim3((unsigned)n) : dim3(kGridX, (unsigned)((n + kGridX - 1) / kGridX));
}

// ---- causal convolution ----
struct ConvArgs {
  int64_t B, L, D;
  int W;
  bool silu;
  int64_t x_row, dx_row;  // elements between consecutive tokens of x / dx
  const void* x;
  const float* w;
  const float* bias;         // may be null
  const void* init;          // [B,W-1,D] or null
  const int* seq_idx;        // [B,L] or null
  void* y;
  void* final_state;         // [B,W-1,D] or null
  int64_t nseq;
  const int64_t* seq_last;
  void* seq_states;          // [nseq,W-1,D]
  // backward
  const void* dy;
  const void* dfinal;        // [B,W-1,D] or null
  void* dx;
  float* dw;
  float* dbias;              // may be null
  void* dinit;               // may be null
  float* ws;
};
size_t conv_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int W);
hipError_t launch_conv_forward(const ConvArgs& a, bool bf16, hipStream_t s);
hipError_t launch_conv_backward(const ConvArgs& a, bool bf16, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, bool bf16, hipStream_t s);

// ---- selective scan ----
struct ScanRows {
  int64_t u, dt, b, c, z;
};
struct ScanArgs {
  int64_t B, L, D, N, G;
  ScanRows rows, grows;
  bool softplus;
  const void *u, *dt, *Bm, *Cm, *z;  // z may be null
  const float *A, *D_skip, *dt_bias; // D_skip, dt_bias may be null
  const int* seq_idx;                // may be null
  const float* h0;                   // may be null
  void* y;
  float* hfin;                       // may be null
  int64_t nseq;
  const int64_t* seq_last;
  float* seq_states;
  // backward
  const void* dy;
  const float* dfinal;               // may be null
  void *du, *ddt, *dB, *dC, *dz;     // dz null when z is
  float *dA, *dD, *ddt_bias, *dinit; // dD, ddt_bias, dinit may be null
  void* ws;
};
bool scan_dstate_supported(int64_t N);
size_t scan_forward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G);
size_t scan_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G);
hipError_t launch_scan_forward(const ScanArgs& a, bool bf16, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, bool bf16, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, const float* state, float* state_out, bool bf16, hipStream_t s);

// ---- layer norm ----
struct NormArgs {
  int64_t rows, D;
  float eps;
  bool rms;
  const void* x;
  bool res_bf16;            // type of residual / residual_out (forward), of x / dresidual (backward)
  const void* residual;     // may be null
  void* residual_out;       // null exactly when residual is
  const float* w;
  const float* bias;        // may be null
  void* y;
  float* mean;              // null for rms
  float* rstd;
  // backward
  const void* dy;
  const void* dres;         // gradient arriving at the residual stream, or null
  void* dx;                 // type of dy
  void* dres_out;           // type of x, or null
  float* dw;
  float* db;                // or null
  float* ws;
};
constexpr int64_t kNormMaxDim = 16384;
size_t norm_backward_ws_bytes(int64_t rows, int64_t D);
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, hipStream_t s);

}  // namespace ssd
