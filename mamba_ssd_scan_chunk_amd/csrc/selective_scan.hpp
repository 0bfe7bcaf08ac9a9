// selective_scan.hpp -- what the selective scan's forward and backward kernels
// share: the split of the work over waves and the scalar loads of B and C.
#pragma once

#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

constexpr int kScanT = 16;  // tokens held in registers at a time

struct ScanGrid {
  int64_t Q, nc;  // tokens a chunk (a multiple of kScanT), chunks
  int64_t ncb;    // blocks of 64 channels per group
};

struct ScanWs {
  float* carry;  // [B,nc,N,D] states
  float* sdt;    // [B,nc,D] summed dt of a chunk (since its last restart)
  int* cut;      // [B,nc] whether a sequence starts inside the chunk
  float* adj;    // backward: [B,nc,N,D] adjoint states
};

struct ScanBlock {
  int64_t b, c, grp, d0, dend, t0, t1;
};

// Grid (G * ncb, chunks, B): consecutive blocks take neighbouring channels of
// the same tokens, which share their rows of B and C.
__device__ __forceinline__ ScanBlock scan_block(const ScanGrid& g, const ScanArgs& a) {
  ScanBlock k;
  const int64_t gd = a.D / a.G;
  k.grp = blockIdx.x / (unsigned)g.ncb;
  k.d0 = k.grp * gd + (blockIdx.x % (unsigned)g.ncb) * 64;
  k.dend = (k.grp + 1) * gd;
  k.c = blockIdx.y;
  k.b = blockIdx.z;
  k.t0 = k.c * g.Q;
  k.t1 = k.t0 + g.Q < a.L ? k.t0 + g.Q : a.L;
  return k;
}

// Four consecutive elements at an address that is the same for all lanes
// (4-byte aligned): scalar loads, widened on the scalar unit.
template <class IO>
__device__ __forceinline__ void uniform4(const typename IO::type* p, float (&o)[4]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
  if constexpr (IO::kVec == 8) {
    const uint32_t w0 = w[0], w1 = w[1];
    o[0] = __uint_as_float(w0 << 16);
    o[1] = __uint_as_float(w0 & 0xffff0000u);
    o[2] = __uint_as_float(w1 << 16);
    o[3] = __uint_as_float(w1 & 0xffff0000u);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __uint_as_float(w[k]);
  }
}

// Element n of a row at an address that is the same for all lanes (the row
// 4-byte aligned).
template <class IO>
__device__ __forceinline__ float uniform1(const typename IO::type* row, int n) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
  if constexpr (IO::kVec == 8) {
    const uint32_t v = w[n >> 1];
    return __uint_as_float((n & 1) ? (v & 0xffff0000u) : (v << 16));
  } else {
    return __uint_as_float(w[n]);
  }
}

}  // namespace ssd
