// layer_reduce.hip -- column sums of fp32 partials, in a fixed order.
#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

constexpr int kSlices = 16;  // row slices (waves) of a block

// One block per 64 columns: wave w sums rows w, w + 16, ... ; the slices meet
// in LDS and are added in wave order.
__global__ __launch_bounds__(64 * kSlices) void colsum_kernel(const float* __restrict__ in, int64_t R, int64_t C,
                                                              float* __restrict__ out) {
  __shared__ float part[kSlices][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const bool ok = c < C;
  const float* p = in + (ok ? c : C - 1);
  float acc = 0.f;
  int64_t r = w;
  for (; r + 7 * kSlices < R; r += 8 * kSlices) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p[(r + k * kSlices) * C];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc += v[k];
  }
  for (; r < R; r += kSlices) acc += p[r * C];
  part[w][lane] = acc;
  __syncthreads();
  if (w == 0 && ok) {
    float s = part[0][lane];
#pragma unroll
    for (int k = 1; k < kSlices; ++k) s += part[k][lane];
    out[c] = s;
  }
}

hipError_t launch_colsum(const float* in, int64_t R, int64_t C, float* out, hipStream_t s) {
  hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((C + 63) / 64)), dim3(64 * kSlices), 0, s, in, R, C, out);
  return hipGetLastError();
}

}  // namespace ssd
