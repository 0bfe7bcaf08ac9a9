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
// write.  Forward: a wave a row up to 4096 columns, 256 threads beyond, 16
// bytes a load (single elements where rows are not whole units of 8).
// Backward: 64, 256 or 1024 threads a row, 16 values a thread at most, so that
// the five values a column (x, dy, w, dw, dbias) leave room for waves beside;
// blocks walk rows, the next row's loads in flight behind the sums of this
// one, and keep dw and dbias of their columns in registers.  The blocks'
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
__global__ __launch_bounds__(256) void norm_forward_kernel(NormArgs a) {
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

// Both sums of a row at once over its TPR threads; `red` holds two rounds of
// them, so that one barrier a row is enough.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int k = 0; k < TPR / 64; ++k) {
      a += red[k].x;
      b += red[k].y;
    }
  }
  return make_float2(a, b);
}

// Threads of a backward block: whole rows of TPR threads, four rows for TPR = 64.
constexpr int norm_bwd_threads(int tpr) { return tpr == 64 ? 256 : tpr; }

// IO: type of dy and dx; RO: type of x, dres and dres_out.
template <class IO, class RO, int V, int NV, int TPR>
__global__ __launch_bounds__(norm_bwd_threads(TPR)) void norm_backward_kernel(NormArgs a) {
  __shared__ float2 red[2][TPR == 64 ? 1 : TPR / 64];
  __shared__ float part[TPR == 64 ? 3 * 2 * 64 * NV * V : 1];
  const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = threadIdx.x >> 6;
  const int64_t first = TPR == 64 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int64_t step = TPR == 64 ? (int64_t)gridDim.x * 4 : gridDim.x;
  const float inv = 1.f / (float)a.D;
  auto col = [&](int j) { return ((int64_t)j * TPR + tid) * V; };
  float w[NV][V], dw[NV][V], db[NV][V], x[NV][V], g[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_cols<IoF32, V>(a.w, 0, col(j), a.D, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_cols<RO, V>(a.x, row * a.D, col(j), a.D, x[j]);
      load_cols<IO, V>(a.dy, row * a.D, col(j), a.D, g[j]);
    }
  };
  // the next row's loads in flight behind this one's sums, but for the blocks
  // of 1024 threads whose 128 registers do not hold both
  constexpr bool kAhead = TPR < 1024 || NV * V <= 8;
  if (kAhead && first < a.rows) fetch(first);
  int round = 0;
  for (int64_t row = first; row < a.rows; row += step, round ^= 1) {
    const int64_t r0 = row * a.D;
    if (!kAhead) fetch(row);
    const float rstd = a.rstd[row], mean = a.mean ? a.mean[row] : 0.f;
    float xh[NV][V], v[NV][V], q[NV][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (a.dres) {
        load_cols<RO, V>(a.dres, r0, col(j), a.D, q[j]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) q[j][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[j][e] = (x[j][e] - mean) * rstd;
        dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
        db[j][e] += g[j][e];
        v[j][e] = g[j][e] * w[j][e];  // zero past the row
        s1 += v[j][e];
        s2 = fmaf(v[j][e], xh[j][e], s2);
      }
    }
    if (kAhead && row + step < a.rows) fetch(row + step);
    const float2 s = row_sum2<TPR>(s1, s2, red[round]);
    const float m1 = a.rms ? 0.f : s.x * inv, m2 = s.y * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (col(j) < a.D) {
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(rstd, v[j][e] - fmaf(xh[j][e], m2, m1), q[j][e]);
        store_vec<IO, V>(static_cast<typename IO::type*>(a.dx) + r0 + col(j), o);
        if (a.dres_out) store_vec<RO, V>(static_cast<typename RO::type*>(a.dres_out) + r0 + col(j), o);
      }
    }
  }
  // a row of partial sums a block: ws[block][2][D]; with four waves a block
  // they meet first
  if constexpr (TPR == 64) {
    constexpr int P = 64 * NV * V;
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          part[((wave - 1) * 2) * P + (j * V + e) * 64 + tid] = dw[j][e];
          part[((wave - 1) * 2 + 1) * P + (j * V + e) * 64 + tid] = db[j][e];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          dw[j][e] += part[(k * 2) * P + (j * V + e) * 64 + tid];
          db[j][e] += part[(k * 2 + 1) * P + (j * V + e) * 64 + tid];
        }
      }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (col(j) < a.D) {
      store_vec<IoF32, V>(a.ws + (int64_t)blockIdx.x * 2 * a.D + col(j), dw[j]);
      store_vec<IoF32, V>(a.ws + (int64_t)blockIdx.x * 2 * a.D + a.D + col(j), db[j]);
    }
  }
}

// dw and dbias [D] from the walkers' partial sums [R][2][D]
__global__ __launch_bounds__(kColsumThreads) void norm_param_kernel(const float* __restrict__ part, int64_t R, int64_t D,
                                                                    float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float lds[kColsumThreads];
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const float s = column_sum(part + (c < 2 * D ? c : 2 * D - 1), R, 2 * D, lds);
  if (threadIdx.x >= 64 || c >= 2 * D) return;
  if (c < D) dw[c] = s;
  else if (db) db[c - D] = s;
}

// Backward: threads a row, for 16 values a thread at most.
static int norm_bwd_tpr(int64_t D) { return D <= 64 * 16 ? 64 : D <= 256 * 16 ? 256 : 1024; }

// Blocks the backward walks the rows with, each leaving a row of partial sums:
// two a compute unit (one of 1024 threads), but four rows a walker at least
// where that still leaves half a block a unit: the partial sums cost as much
// as reading one fp32 row each, and their addition as much again.
static int64_t norm_bwd_blocks(int64_t rows, int64_t D) {
  const int64_t cus = device_cu_count();
  const int tpr = norm_bwd_tpr(D);
  const int64_t walkers = tpr == 64 ? (rows + 3) / 4 : rows;  // if each walked one row
  int64_t b = tpr == 1024 ? cus : 2 * cus;
  const int64_t quarter = (walkers + 3) / 4;
  if (quarter < b) b = quarter > cus / 2 ? quarter : cus / 2;
  return walkers < b ? walkers : b;
}

size_t norm_backward_ws_bytes(int64_t rows, int64_t D) {
  return sizeof(float) * (size_t)(2 * D) * (size_t)norm_bwd_blocks(rows, D);
}

template <class IO, class RO, int V, int NV, int TPR>
static hipError_t norm_fwd_go(const NormArgs& a, hipStream_t s) {
  const int64_t blocks = TPR == 64 ? (a.rows + 3) / 4 : a.rows;
  hipLaunchKernelGGL((norm_forward_kernel<IO, RO, V, NV, TPR>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <class IO, class RO, int V, int NV, int TPR>
static hipError_t norm_bwd_go(const NormArgs& a, hipStream_t s) {
  const int64_t blocks = norm_bwd_blocks(a.rows, a.D);
  hipLaunchKernelGGL((norm_backward_kernel<IO, RO, V, NV, TPR>), dim3((unsigned)blocks), dim3(norm_bwd_threads(TPR)), 0,
                     s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_param_kernel, dim3((unsigned)((2 * a.D + 63) / 64)), dim3(kColsumThreads), 0, s, a.ws, blocks,
                     a.D, a.dw, a.db);
  return hipGetLastError();
}

// Values a thread holds: NV runs of V (the loads past a short row are skipped).
template <class IO, class RO, int V, int TPR>
static hipError_t norm_fwd_nv(const NormArgs& a, hipStream_t s) {
  const int64_t per = (a.D + TPR - 1) / TPR;
  if (per <= 8) return norm_fwd_go<IO, RO, V, 8 / V, TPR>(a, s);
  if (per <= 16) return norm_fwd_go<IO, RO, V, 16 / V, TPR>(a, s);
  if (per <= 40) return norm_fwd_go<IO, RO, V, 40 / V, TPR>(a, s);
  return norm_fwd_go<IO, RO, V, 64 / V, TPR>(a, s);
}
template <class IO, class RO, int V, int TPR>
static hipError_t norm_bwd_nv(const NormArgs& a, hipStream_t s) {
  const int64_t per = (a.D + TPR - 1) / TPR;
  if (per <= 8) return norm_bwd_go<IO, RO, V, 8 / V, TPR>(a, s);
  if (per <= 12) return norm_bwd_go<IO, RO, V, 12 / V, TPR>(a, s);
  return norm_bwd_go<IO, RO, V, 16 / V, TPR>(a, s);
}

template <class IO, class RO, bool BWD>
static hipError_t norm_types(const NormArgs& a, hipStream_t s) {
  if constexpr (BWD) {
    const int tpr = norm_bwd_tpr(a.D);
    if (a.D % 4 == 0) {
      if (tpr == 64) return norm_bwd_nv<IO, RO, 4, 64>(a, s);
      if (tpr == 256) return norm_bwd_nv<IO, RO, 4, 256>(a, s);
      return norm_bwd_nv<IO, RO, 4, 1024>(a, s);
    }
    if (tpr == 64) return norm_bwd_nv<IO, RO, 1, 64>(a, s);
    if (tpr == 256) return norm_bwd_nv<IO, RO, 1, 256>(a, s);
    return norm_bwd_nv<IO, RO, 1, 1024>(a, s);
  } else {
    const bool wave = a.D <= 64 * 64;
    if (a.D % 8 == 0) return wave ? norm_fwd_nv<IO, RO, 8, 64>(a, s) : norm_fwd_nv<IO, RO, 8, 256>(a, s);
    return wave ? norm_fwd_nv<IO, RO, 1, 64>(a, s) : norm_fwd_nv<IO, RO, 1, 256>(a, s);
  }
}

template <bool BWD>
static hipError_t norm_io(const NormArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.res_bf16 ? norm_types<IoBF16, IoBF16, BWD>(a, s) : norm_types<IoBF16, IoF32, BWD>(a, s);
  return a.res_bf16 ? norm_types<IoF32, IoBF16, BWD>(a, s) : norm_types<IoF32, IoF32, BWD>(a, s);
}

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, hipStream_t s) { return norm_io<false>(a, bf16, s); }
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, hipStream_t s) { return norm_io<true>(a, bf16, s); }

}  // namespace ssd
