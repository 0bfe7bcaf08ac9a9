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
// write: 16384 rows of 2560 columns (bf16, fp32 residual) 100 us forward, 5.0
// TB/s, and 124 us backward, 5.4 TB/s, where a copy reaches 4.95.
// Forward: a wave a row up to 4096 columns, 256 threads beyond, 8 or 4
// elements a load.  Rows that are not whole groups of 4 begin anywhere in one:
// in bf16 their threads take the groups as memory has them, the first beginning
// up to 3 columns before the row and the last ending after it (4866 rows of
// 1669 columns, bf16 with bf16 residual: 51 us an element a load, 20 so).
// Backward: 64, 256 or 1024 threads a row, 16 values a thread at most, so that
// the five values a column (x, dy, w, dw, dbias) leave room for waves beside;
// blocks walk rows, the next row's loads in flight behind the sums of this
// one, and keep dw and dbias of their columns in registers (walking in steps
// of 4 rows, they find the same columns in each also where rows begin inside
// groups).  The blocks' partial sums are
// added in a fixed order.
#include <type_traits>

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

// Columns of the row before its first group of V in memory: rows of whole
// groups (SHIFT false) begin with one.
template <int V, bool SHIFT>
__device__ __forceinline__ int row_shift(int64_t r0) {
  return SHIFT ? (int)(r0 & (V - 1)) : 0;
}
// Whether column c + e of a group at c is in the row.
template <bool SHIFT>
__device__ __forceinline__ bool in_row(int c, int e, int D) {
  return SHIFT ? (unsigned)(c + e) < (unsigned)D : c < D;
}
// V elements at column c, zeros outside the row, held as loaded until they are
// widened: widened in the branch that loads them each group would be waited
// for before the next is asked for (4866 rows of 1669 columns, bf16 with bf16
// residual: 26 us, 20 so; gradients of 16384 x 2560, bf16 with fp32 residual,
// 142 and 124).  Groups over a row's ends hold elements of its neighbours, all
// within the `total` elements but for the last row's.  (Loads of groups past the
// row made unconditional, to leave no branches, cost more in traffic than they
// saved.)
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <class IO, int V, bool SHIFT>
struct Cols {
  typedef typename IO::type T;
  static constexpr bool kWords = sizeof(T) == 2 && V > 1;  // bf16 in whole words
  typedef std::conditional_t<kWords, std::conditional_t<V == 8, u32x4_t, u32x2_t>, T> Q;
  Q q[kWords ? 1 : V];
  __device__ __forceinline__ void load(const void* base, int64_t row0, int c, int D, int64_t total) {
    const T* p = static_cast<const T*>(base) + row0 + c;
#pragma unroll
    for (int e = 0; e < (kWords ? 1 : V); ++e) q[e] = Q(0);
    if (c < D && (!SHIFT || row0 + c + V <= total)) {
      if constexpr (kWords || V == 1) {
        q[0] = *reinterpret_cast<const Q*>(p);
      } else {
        load_vec<IO, V>(p, q);
      }
    } else if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (in_row<SHIFT>(c, e, D)) {
          if constexpr (kWords) q[0][e / 2] |= (uint32_t)p[e] << (e % 2 * 16);
          else q[e] = p[e];
        }
      }
    }
  }
  __device__ __forceinline__ void widen(int c, int D, float* o) const {
    if constexpr (kWords) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = __uint_as_float(e % 2 ? q[0][e / 2] & 0xffff0000u : q[0][e / 2] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = IO::get(q[e]);
    }
    if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = in_row<SHIFT>(c, e, D) ? o[e] : 0.f;
    }
  }
};
template <class IO, int V, bool SHIFT>
__device__ __forceinline__ void store_cols(void* base, int64_t row0, int c, int D, const float* v) {
  typename IO::type* p = static_cast<typename IO::type*>(base) + row0 + c;
  if (SHIFT ? c >= 0 && c + V <= D : c < D) {
    store_vec<IO, V>(p, v);
  } else if (SHIFT) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (in_row<SHIFT>(c, e, D)) p[e] = IO::put(v[e]);
  }
}
// The same of an fp32 vector of D, whose groups are aligned only without a shift.
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
template <int V, bool SHIFT>
__device__ __forceinline__ void load_param(const float* p, int c, int D, float* o) {
  if constexpr (SHIFT) {
    if (c >= 0 && c + V <= D) {
      const f32x4_any_t q = *reinterpret_cast<const f32x4_any_t*>(p + c);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = q[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = in_row<SHIFT>(c, e, D) ? p[c + e] : 0.f;
    }
  } else {
    Cols<IoF32, V, false> q;
    q.load(p, 0, c, D, D);
    q.widen(c, D, o);
  }
}

template <class IO, class RO, int V, bool SHIFT, int NV, int TPR>
__global__ __launch_bounds__(256) void norm_forward_kernel(NormArgs a) {
  __shared__ float red[TPR == 64 ? 1 : TPR / 64];
  const int64_t row = TPR == 64 ? (int64_t)flat_block() * 4 + (threadIdx.x >> 6) : flat_block();
  if (row >= a.rows) return;  // whole waves, or the whole block
  const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t r0 = row * a.D;
  const int D = (int)a.D, m = row_shift<V, SHIFT>(r0);
  const int64_t total = a.rows * a.D;
  auto col = [&](int j) { return (j * TPR + tid) * V - m; };
  float x[NV][V];
  Cols<IO, V, SHIFT> xq[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) xq[j].load(a.x, r0, col(j), D, total);
  if (a.residual) {
    Cols<RO, V, SHIFT> q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) q[j].load(a.residual, r0, col(j), D, total);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float t[V];
      xq[j].widen(col(j), D, x[j]);
      q[j].widen(col(j), D, t);
#pragma unroll
      for (int e = 0; e < V; ++e) x[j][e] = RO::get(RO::put(x[j][e] + t[e]));
      store_cols<RO, V, SHIFT>(a.residual_out, r0, col(j), D, x[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) xq[j].widen(col(j), D, x[j]);
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
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[j][e] -= mean;
      s2 = in_row<SHIFT>(col(j), e, D) ? fmaf(x[j][e], x[j][e], s2) : s2;
    }
  }
  const float rstd = 1.f / sqrtf(fmaf(row_sum<TPR>(s2, red), inv, a.eps));
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (col(j) < D) {
      float w[V], b[V], o[V];
      load_param<V, SHIFT>(a.w, col(j), D, w);
#pragma unroll
      for (int e = 0; e < V; ++e) b[e] = 0.f;
      if (a.bias) load_param<V, SHIFT>(a.bias, col(j), D, b);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(x[j][e] * rstd, w[e], b[e]);
      store_cols<IO, V, SHIFT>(a.y, r0, col(j), D, o);
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
template <class IO, class RO, int V, bool SHIFT, int NV, int TPR>
__global__ __launch_bounds__(norm_bwd_threads(TPR)) void norm_backward_kernel(NormArgs a) {
  __shared__ float2 red[2][TPR == 64 ? 1 : TPR / 64];
  __shared__ float part[TPR == 64 ? 3 * 2 * 64 * NV * V : 1];
  const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = threadIdx.x >> 6;
  const int64_t first = TPR == 64 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  const int64_t step = TPR == 64 ? (int64_t)gridDim.x * 4 : gridDim.x;
  const float inv = 1.f / (float)a.D;
  const int D = (int)a.D, m = row_shift<V, SHIFT>(first * a.D);  // of each of the walker's rows
  const int64_t total = a.rows * a.D;
  auto col = [&](int j) { return (j * TPR + tid) * V - m; };
  float w[NV][V], dw[NV][V], db[NV][V];
  Cols<RO, V, SHIFT> x[NV];
  Cols<IO, V, SHIFT> g[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_param<V, SHIFT>(a.w, col(j), D, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j].load(a.x, row * a.D, col(j), D, total);
      g[j].load(a.dy, row * a.D, col(j), D, total);
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
    float xh[NV][V], v[NV][V];
    Cols<RO, V, SHIFT> q[NV];
    if (a.dres) {
#pragma unroll
      for (int j = 0; j < NV; ++j) q[j].load(a.dres, r0, col(j), D, total);
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float xv[V], gv[V];
      x[j].widen(col(j), D, xv);
      g[j].widen(col(j), D, gv);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[j][e] = (xv[e] - mean) * rstd;
        dw[j][e] = fmaf(gv[e], xh[j][e], dw[j][e]);
        db[j][e] += gv[e];
        v[j][e] = gv[e] * w[j][e];  // zero past the row
        s1 += v[j][e];
        s2 = fmaf(v[j][e], xh[j][e], s2);
      }
    }
    if (kAhead && row + step < a.rows) fetch(row + step);
    const float2 s = row_sum2<TPR>(s1, s2, red[round]);
    const float m1 = a.rms ? 0.f : s.x * inv, m2 = s.y * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (col(j) < D) {
        float o[V], t[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t[e] = 0.f;
        if (a.dres) q[j].widen(col(j), D, t);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(rstd, v[j][e] - fmaf(xh[j][e], m2, m1), t[e]);
        store_cols<IO, V, SHIFT>(a.dx, r0, col(j), D, o);
        if (a.dres_out) store_cols<RO, V, SHIFT>(a.dres_out, r0, col(j), D, o);
      }
    }
  }
  // a row of partial sums a block: ws[block][2][D]; with four waves a block
  // they meet first
  if constexpr (TPR == 64) {
    static_assert(!SHIFT, "the waves of a block share their columns");
    constexpr int P = 64 * NV * V;
    // a lane's values side by side with the other lanes'
    auto place = [&](int j, int e) { return (j * V + e) * 64 + tid; };
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          part[((wave - 1) * 2) * P + place(j, e)] = dw[j][e];
          part[((wave - 1) * 2 + 1) * P + place(j, e)] = db[j][e];
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
          dw[j][e] += part[(k * 2) * P + place(j, e)];
          db[j][e] += part[(k * 2 + 1) * P + place(j, e)];
        }
      }
  }
  float* ws = a.ws + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (in_row<SHIFT>(col(j), e, D)) {
          ws[col(j) + e] = dw[j][e];
          ws[a.D + col(j) + e] = db[j][e];
        }
      }
    } else {
      store_cols<IoF32, V, false>(ws, 0, col(j), D, dw[j]);
      store_cols<IoF32, V, false>(ws + a.D, 0, col(j), D, db[j]);
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

// Columns a row's threads have to cover: with the most that the first group can
// begin before a row that is not whole groups of 4.
static int64_t norm_cover(int64_t D) { return D % 4 == 0 ? D : D + (D % 2 ? 3 : 2); }

// Backward: threads a row, for 16 values a thread at most (but one row length).
static int norm_bwd_tpr(int64_t D) {
  const int64_t n = norm_cover(D);
  return n <= 64 * 16 ? 64 : n <= 256 * 16 ? 256 : 1024;
}

// Blocks the backward walks the rows with, each leaving a row of partial sums:
// two a compute unit (one of 1024 threads), but four rows a walker at least
// where that still leaves half a block a unit: the partial sums cost as much
// as reading one fp32 row each, and their addition as much again.  Where rows
// begin inside groups, steps in whole fours.
static int64_t norm_bwd_blocks(int64_t rows, int64_t D) {
  const int64_t cus = device_cu_count();
  const int tpr = norm_bwd_tpr(D);
  const int64_t walkers = tpr == 64 ? (rows + 3) / 4 : rows;  // if each walked one row
  int64_t b = tpr == 1024 ? cus : 2 * cus;
  const int64_t quarter = (walkers + 3) / 4;
  if (quarter < b) b = quarter > cus / 2 ? quarter : cus / 2;
  b = (b + 3) / 4 * 4;
  return walkers < b ? walkers : b;
}

size_t norm_backward_ws_bytes(int64_t rows, int64_t D) {
  return sizeof(float) * (size_t)(2 * D) * (size_t)norm_bwd_blocks(rows, D);
}

template <class IO, class RO, int V, bool SHIFT, int NV, int TPR>
static hipError_t norm_fwd_go(const NormArgs& a, hipStream_t s) {
  const int64_t blocks = TPR == 64 ? (a.rows + 3) / 4 : a.rows;
  hipLaunchKernelGGL((norm_forward_kernel<IO, RO, V, SHIFT, NV, TPR>), flat_grid(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <class IO, class RO, int V, bool SHIFT, int NV, int TPR>
static hipError_t norm_bwd_go(const NormArgs& a, hipStream_t s) {
  const int64_t blocks = norm_bwd_blocks(a.rows, a.D);
  hipLaunchKernelGGL((norm_backward_kernel<IO, RO, V, SHIFT, NV, TPR>), dim3((unsigned)blocks),
                     dim3(norm_bwd_threads(TPR)), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_param_kernel, dim3((unsigned)((2 * a.D + 63) / 64)), dim3(kColsumThreads), 0, s, a.ws, blocks,
                     a.D, a.dw, a.db);
  return hipGetLastError();
}

// Values a thread holds: NV groups of V (the loads past a short row are
// skipped).  Fewer than a row's most leave registers for more waves: forward
// 40 beside 64 (16384 x 2557, bf16 with fp32 residual 109 us, 64 131; 16000 x
// 2557 fp32 150 and 199; whole groups do not mind, 16384 x 2560 99 and 96), 16
// (40960 x 1024 bf16 31 us, 64 46), 8 (262144 x 128 135, 64 280); backward 12
// (3400 x 12288 137 us, 16 158; no difference with fewer threads a row).
// 16383 columns, the one length that its shift takes over the most
// that 16384 need, get a group more.
template <class IO, class RO, int V, bool SHIFT, int TPR>
static hipError_t norm_fwd_nv(const NormArgs& a, hipStream_t s) {
  const int64_t per = ((SHIFT ? norm_cover(a.D) : a.D) + TPR - 1) / TPR;
  if (per <= 8) return norm_fwd_go<IO, RO, V, SHIFT, 8 / V, TPR>(a, s);
  if (per <= 16) return norm_fwd_go<IO, RO, V, SHIFT, 16 / V, TPR>(a, s);
  if (per <= 40) return norm_fwd_go<IO, RO, V, SHIFT, 40 / V, TPR>(a, s);
  if (per <= 64) return norm_fwd_go<IO, RO, V, SHIFT, 64 / V, TPR>(a, s);
  if constexpr (SHIFT && TPR == 256) return norm_fwd_go<IO, RO, V, SHIFT, 64 / V + 1, TPR>(a, s);
  return hipErrorInvalidValue;
}
template <class IO, class RO, int V, bool SHIFT, int TPR>
static hipError_t norm_bwd_nv(const NormArgs& a, hipStream_t s) {
  const int64_t per = ((SHIFT ? norm_cover(a.D) : a.D) + TPR - 1) / TPR;
  if (per <= 8) return norm_bwd_go<IO, RO, V, SHIFT, 8 / V, TPR>(a, s);
  if (per <= 12) return norm_bwd_go<IO, RO, V, SHIFT, 12 / V, TPR>(a, s);
  if (per <= 16) return norm_bwd_go<IO, RO, V, SHIFT, 16 / V, TPR>(a, s);
  if constexpr (SHIFT && TPR == 1024) return norm_bwd_go<IO, RO, V, SHIFT, 16 / V + 1, TPR>(a, s);
  return hipErrorInvalidValue;
}

template <class IO, class RO, int V, bool SHIFT>
static hipError_t norm_fwd_rows(const NormArgs& a, hipStream_t s) {
  return norm_cover(a.D) <= 64 * 64 ? norm_fwd_nv<IO, RO, V, SHIFT, 64>(a, s) : norm_fwd_nv<IO, RO, V, SHIFT, 256>(a, s);
}
template <class IO, class RO, int V>
static hipError_t norm_bwd_rows(const NormArgs& a, hipStream_t s) {
  switch (norm_bwd_tpr(a.D)) {
    case 64: return norm_bwd_nv<IO, RO, V, false, 64>(a, s);
    case 256: return norm_bwd_nv<IO, RO, V, false, 256>(a, s);
    default: return norm_bwd_nv<IO, RO, V, false, 1024>(a, s);
  }
}

// Rows that are not whole groups.  Forward: shifted groups where a type is
// bf16, single elements in fp32 (bf16 without residual 11753 x 1021 14 us,
// single elements 23; fp32 with residual 11753 x 1021 38, groups 45; bf16 rows of
// 61 and fp32 ones past 2048 columns would be the other way: 72 and 49, 4692 x
// 2557 51 and 43).  Gradients, whose five values a column weigh more than the
// loads: single elements (bf16 without residual 7189 x 1669 31 us, groups 36;
// bf16 with fp32 residual 196721 x 61 142 and 269, 999 x 12001 59 and 96) but
// for the longest bf16 rows (732 x 16382 bf16 residual 115 and 93; fp32
// residual 99 and 144).
template <class IO, class RO, bool BWD>
static hipError_t norm_types(const NormArgs& a, hipStream_t s) {
  constexpr bool bf16 = IO::kVec == 8 || RO::kVec == 8;
  if constexpr (BWD) {
    if (a.D % 4 == 0) return norm_bwd_rows<IO, RO, 4>(a, s);
    if constexpr (bf16) {
      if (a.D > 12 * 1024) return norm_bwd_nv<IO, RO, 4, true, 1024>(a, s);
    }
    return norm_bwd_rows<IO, RO, 1>(a, s);
  } else {
    if (a.D % 8 == 0) return norm_fwd_rows<IO, RO, 8, false>(a, s);
    if (a.D % 4 == 0) return norm_fwd_rows<IO, RO, 4, false>(a, s);
    return norm_fwd_rows<IO, RO, bf16 ? 4 : 1, bf16>(a, s);
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
