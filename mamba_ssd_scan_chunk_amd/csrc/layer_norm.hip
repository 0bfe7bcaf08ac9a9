// layer_norm.hip -- layer norm (or RMS norm) with the residual add in front,
// and its gradients.
//
// Per row: r = x + residual (stored, in the residual's type; the stored value
// is what is normalised), mean and variance of r in fp32 with the squared
// deviations taken from the mean (a second pass over registers), and
//     xh = (r - mean) rstd,  y = xh w + bias,  rstd = 1/sqrt(var + eps)
// (RMS: mean = 0, no mean in the gradient).  Backward, with v = w dy:
//     dr = rstd (v - mean(v) - xh mean(v xh)) + dresidual
//     dw = sum over rows of dy xh,  dbias = sum over rows of dy
//
// Bound by memory.  A row stays in registers between its one read and its one
// write: 64, 256 or 1024 threads a row by its length, 16 bytes a load (single
// elements where rows are not whole 16-byte units).  The backward keeps dw and
// dbias of its columns in registers over the rows a block walks; the blocks'
// partial sums are added in a fixed order.
#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

// Sum over the TPR threads of a row (TPR = 64: the wave; else the block).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < TPR / 64; ++k) v += red[k];
  }
  return v;
}

// Loads V elements at column c (below D) as fp32, zeros past the row.
template <class IO, int V>
__device__ __forceinline__ void load_cols(const void* base, int64_t row0, int64_t c, int64_t D, float* o) {
  if (c < D) {
    load_vec<IO, V>(static_cast<const typename IO::type*>(base) + row0 + c, o);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
  }
}

template <class IO, class RO, int V, int NV, int TPR>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_forward_kernel(NormArgs a) {
  __shared__ float red[TPR == 64 ? 1 : TPR / 64];
  const int64_t row = TPR == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (TPR == 64 && row >= a.rows) return;
  const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t r0 = row * a.D;
  float x[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_cols<IO, V>(a.x, r0, ((int64_t)j * TPR + tid) * V, a.D, x[j]);
  if (a.residual) {
    float q[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_cols<RO, V>(a.residual, r0, ((int64_t)j * TPR + tid) * V, a.D, q[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)j * TPR + tid) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) x[j][e] = RO::get(RO::put(x[j][e] + q[j][e]));
      if (c < a.D) store_vec<RO, V>(static_cast<typename RO::type*>(a.residual_out) + r0 + c, x[j]);
    }
  }
  const float inv = 1.f / (float)a.D;
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s += x[j][e];
    mean = row_sum<TPR>(s, red) * inv;
  }
  float s2 = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = ((int64_t)j * TPR + tid) * V < a.D;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[j][e] -= mean;
      s2 = in ? fmaf(x[j][e], x[j][e], s2) : s2;
    }
  }
  const float rstd = 1.f / sqrtf(fmaf(row_sum<TPR>(s2, red), inv, a.eps));
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = ((int64_t)j * TPR + tid) * V;
    if (c < a.D) {
      float w[V], b[V], o[V];
      load_vec<IoF32, V>(a.w + c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) b[e] = 0.f;
      if (a.bias) load_vec<IoF32, V>(a.bias + c, b);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(x[j][e] * rstd, w[e], b[e]);
      store_vec<IO, V>(static_cast<typename IO::type*>(a.y) + r0 + c, o);
    }
  }
}

// IO: type of dy and dx; RO: type of x, dres and dres_out.
template <class IO, class RO, int V, int NV, int TPR>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void norm_backward_kernel(NormArgs a) {
  __shared__ float red[TPR == 64 ? 1 : TPR / 64];
  const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t first = TPR == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = TPR == 64 ? (int64_t)gridDim.x * 4 : gridDim.x;
  const float inv = 1.f / (float)a.D;
  float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_cols<IoF32, V>(a.w, 0, ((int64_t)j * TPR + tid) * V, a.D, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  for (int64_t row = first; row < a.rows; row += step) {
    const int64_t r0 = row * a.D;
    const float rstd = a.rstd[row], mean = a.mean ? a.mean[row] : 0.f;
    float x[NV][V], g[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_cols<RO, V>(a.x, r0, ((int64_t)j * TPR + tid) * V, a.D, x[j]);
      load_cols<IO, V>(a.dy, r0, ((int64_t)j * TPR + tid) * V, a.D, g[j]);
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (x[j][e] - mean) * rstd;
        dw[j][e] = fmaf(g[j][e], xh, dw[j][e]);
        db[j][e] += g[j][e];
        const float v = g[j][e] * w[j][e];  // zero past the row
        s1 += v;
        s2 = fmaf(v, xh, s2);
        x[j][e] = xh;
        g[j][e] = v;
      }
    s2 = row_sum<TPR>(s2, red) * inv;
    s1 = a.rms ? 0.f : row_sum<TPR>(s1, red) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)j * TPR + tid) * V;
      if (c < a.D) {
        float q[V], o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) q[e] = 0.f;
        if (a.dres) load_vec<RO, V>(static_cast<const typename RO::type*>(a.dres) + r0 + c, q);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(rstd, g[j][e] - fmaf(x[j][e], s2, s1), q[e]);
        store_vec<IO, V>(static_cast<typename IO::type*>(a.dx) + r0 + c, o);
        if (a.dres_out) store_vec<RO, V>(static_cast<typename RO::type*>(a.dres_out) + r0 + c, o);
      }
    }
  }
  // partial sums: ws[first][2][D]
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = ((int64_t)j * TPR + tid) * V;
    if (c < a.D) {
      store_vec<IoF32, V>(a.ws + first * 2 * a.D + c, dw[j]);
      store_vec<IoF32, V>(a.ws + first * 2 * a.D + a.D + c, db[j]);
    }
  }
}

__global__ __launch_bounds__(256) void norm_weight_kernel(const float* __restrict__ sums, int64_t D,
                                                          float* __restrict__ dw, float* __restrict__ db) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  dw[c] = sums[c];
  if (db) db[c] = sums[D + c];
}

// Threads a row: a wave up to 64 values a thread, then 256, then 1024.
static int norm_tpr(int64_t D) { return D <= 64 * 64 ? 64 : D <= 256 * 64 ? 256 : 1024; }

// Rows of partial sums the backward leaves: one per wave or block that walks rows.
static int64_t norm_bwd_walkers(int64_t rows, int64_t D) {
  const int64_t cus = device_cu_count();
  const int64_t w = norm_tpr(D) == 64 ? cus * 8 : norm_tpr(D) == 256 ? cus * 2 : cus;
  return rows < w ? rows : w;
}

size_t norm_backward_ws_bytes(int64_t rows, int64_t D) {
  return sizeof(float) * (size_t)(2 * D) * (size_t)(norm_bwd_walkers(rows, D) + 3 + 1);
}

template <class IO, class RO, int V, int NV, int TPR, bool BWD>
static hipError_t norm_go(const NormArgs& a, hipStream_t s) {
  if (!BWD) {
    const int64_t blocks = TPR == 64 ? (a.rows + 3) / 4 : a.rows;
    hipLaunchKernelGGL((norm_forward_kernel<IO, RO, V, NV, TPR>), dim3((unsigned)blocks), dim3(TPR == 64 ? 256 : TPR), 0,
                       s, a);
    return hipGetLastError();
  }
  int64_t walkers = norm_bwd_walkers(a.rows, a.D);
  if (TPR == 64) walkers = (walkers + 3) / 4 * 4;  // whole blocks of four waves
  hipLaunchKernelGGL((norm_backward_kernel<IO, RO, V, NV, TPR>), dim3((unsigned)(TPR == 64 ? walkers / 4 : walkers)),
                     dim3(TPR == 64 ? 256 : TPR), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* sums = a.ws + walkers * 2 * a.D;
  if ((e = launch_colsum(a.ws, walkers, 2 * a.D, sums, s)) != hipSuccess) return e;
  hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((a.D + 255) / 256)), dim3(256), 0, s, sums, a.D, a.dw, a.db);
  return hipGetLastError();
}

// Values a thread holds: NV runs of V (the loads past a short row are skipped).
template <class IO, class RO, int V, int TPR, bool BWD>
static hipError_t norm_nv(const NormArgs& a, hipStream_t s) {
  const int64_t per = (a.D + TPR - 1) / TPR;  // elements a thread
  if (per <= 8) return norm_go<IO, RO, V, 8 / V, TPR, BWD>(a, s);
  if (per <= 16) return norm_go<IO, RO, V, 16 / V, TPR, BWD>(a, s);
  if (per <= 24) return norm_go<IO, RO, V, 24 / V, TPR, BWD>(a, s);
  if (per <= 40) return norm_go<IO, RO, V, 40 / V, TPR, BWD>(a, s);
  return norm_go<IO, RO, V, 64 / V, TPR, BWD>(a, s);
}

template <class IO, class RO, bool BWD>
static hipError_t norm_types(const NormArgs& a, hipStream_t s) {
  const int tpr = norm_tpr(a.D);
  // 16-byte loads of the narrower type: whole units of 8 elements a row
  if (a.D % 8 == 0) {
    if (tpr == 64) return norm_nv<IO, RO, 8, 64, BWD>(a, s);
    if (tpr == 256) return norm_nv<IO, RO, 8, 256, BWD>(a, s);
    return norm_nv<IO, RO, 8, 1024, BWD>(a, s);
  }
  if (tpr == 64) return norm_nv<IO, RO, 1, 64, BWD>(a, s);
  if (tpr == 256) return norm_nv<IO, RO, 1, 256, BWD>(a, s);
  return norm_nv<IO, RO, 1, 1024, BWD>(a, s);
}

template <bool BWD>
static hipError_t norm_io(const NormArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.res_bf16 ? norm_types<IoBF16, IoBF16, BWD>(a, s) : norm_types<IoBF16, IoF32, BWD>(a, s);
  return a.res_bf16 ? norm_types<IoF32, IoBF16, BWD>(a, s) : norm_types<IoF32, IoF32, BWD>(a, s);
}

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, hipStream_t s) { return norm_io<false>(a, bf16, s); }
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, hipStream_t s) { return norm_io<true>(a, bf16, s); }

}  // namespace ssd
