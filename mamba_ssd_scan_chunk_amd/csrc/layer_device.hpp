// layer_device.hpp -- device helpers of the layer operators: element types,
// the sigmoid and softplus they share.
#pragma once

#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {

// The block's place in a flat_grid.
__device__ __forceinline__ uint32_t flat_block() { return blockIdx.y * kGridX + blockIdx.x; }

// Element type of activations in memory; arithmetic is always fp32.
struct IoBF16 {
  typedef uint16_t type;
  static constexpr int kVec = 8;  // elements in 16 bytes
  __device__ __forceinline__ static float get(uint16_t v) { return bf16_bits_to_f32(v); }
  __device__ __forceinline__ static uint16_t put(float v) { return (uint16_t)f32_to_bf16_bits(v); }
};
struct IoF32 {
  typedef float type;
  static constexpr int kVec = 4;
  __device__ __forceinline__ static float get(float v) { return v; }
  __device__ __forceinline__ static float put(float v) { return v; }
};

// V consecutive elements as fp32: one 16-byte access per IO::kVec elements
// (V a multiple of it), one 8-byte access (four bf16), or a single element.
template <class IO, int V>
__device__ __forceinline__ void load_vec(const typename IO::type* p, float* o) {
  if constexpr (V == 1) {
    o[0] = IO::get(p[0]);
  } else if constexpr (IO::kVec == 8 && V == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    o[0] = __uint_as_float(q.x << 16);
    o[1] = __uint_as_float(q.x & 0xffff0000u);
    o[2] = __uint_as_float(q.y << 16);
    o[3] = __uint_as_float(q.y & 0xffff0000u);
  } else if constexpr (IO::kVec == 8) {
#pragma unroll
    for (int k = 0; k < V; k += 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + k);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[k + 2 * e] = __uint_as_float(w[e] << 16);
        o[k + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + k);
      o[k] = q.x; o[k + 1] = q.y; o[k + 2] = q.z; o[k + 3] = q.w;
    }
  }
}
template <class IO, int V>
__device__ __forceinline__ void store_vec(typename IO::type* p, const float* v) {
  if constexpr (V == 1) {
    p[0] = IO::put(v[0]);
  } else if constexpr (IO::kVec == 8 && V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else if constexpr (IO::kVec == 8) {
#pragma unroll
    for (int k = 0; k < V; k += 8)
      *reinterpret_cast<uint4*>(p + k) = make_uint4(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]),
                                                    pack_bf16x2(v[k + 4], v[k + 5]), pack_bf16x2(v[k + 6], v[k + 7]));
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  }
}

// 1 / (1 + e^-v): hardware exponential and reciprocal, about 2 ulp.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-v * kLog2e));
}
// the same of w ln 2
__device__ __forceinline__ float sigmoid2(float w) { return __builtin_amdgcn_rcpf(1.f + fast_exp2(-w)); }
// d/dv [v sigmoid(v)] from v and its sigmoid
__device__ __forceinline__ float dsilu(float v, float s) { return s * fmaf(v, 1.f - s, 1.f); }

// log2(1 + 2^w).  With e = 2^w and u = 1 + e rounded it is log2(u) plus what
// rounding u lost, log2(e) (e - (u-1)) / u to first order, which matters where
// log2(u) is small; there 1/u is near 1 - e/2 (above e = 2 the term is below
// half a unit and left out).  It is never below w: the maximum also covers the
// e that overflows.  Branch-free, about a third of the library's log1p, whose
// branches also kept a tile's loads from overlapping.
__device__ __forceinline__ float softplus2(float w) {
  const float e = fast_exp2(w);
  const float u = 1.f + e;
  const float lost = e - (u - 1.f);
  const float l = fmaf(lost, fmaxf(fmaf(-0.5f * kLog2e, e, kLog2e), 0.f), __builtin_amdgcn_logf(u));
  return fmaxf(l, w);
}

// Sum of a column of fp32 partials, p[0], p[stride], .. (R of them), for a
// block of 16 waves that take 64 columns a lane each: wave w adds rows w,
// w + 16, .., the waves' sums meet in LDS (a float a thread) and are added in
// order.  Valid in the first wave; every thread must call it.
constexpr int kColsumThreads = 1024;
__device__ __forceinline__ float column_sum(const float* p, int64_t R, int64_t stride, float* lds) {
  constexpr int S = kColsumThreads / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float acc = 0.f;
  int64_t r = w;
  for (; r + 7 * S < R; r += 8 * S) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[(r + e * S) * stride];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc += v[e];
  }
  for (; r < R; r += S) acc += p[r * stride];
  lds[threadIdx.x] = acc;
  __syncthreads();
  float s = lds[lane];
#pragma unroll
  for (int e = 1; e < S; ++e) s += lds[e * 64 + lane];
  return s;
}

}  // namespace ssd
