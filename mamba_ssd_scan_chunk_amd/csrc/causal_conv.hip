// causal_conv.hip -- the short depthwise causal convolution in front of a
// state-space scan, with bias and SiLU, its gradients and its single-token
// step.
//
// Per channel d and token t, with W taps:
//     pre[t] = bias + sum_k w[k] x[t-W+1+k],   y[t] = pre sigmoid(pre)   (or pre)
// Taps before the row come from the initial state (its last W-1 inputs), taps
// of another packed sequence are zero.  Backward:
//     dpre[t] = dy[t] silu'(pre[t]),  dx[t] = sum_k w[k] dpre[t+W-1-k],
//     dw[k] = sum_t dpre[t] x[t-W+1+k],  dbias = sum_t dpre[t]
//
// Bound by memory: 2 elements moved per output (3 backward) against 2W + 4
// operations.  A thread owns 16 bytes of channels (one channel where rows or
// widths are not whole 16-byte units) and walks a run of tokens with the last
// W-1 inputs in registers, so each input is read once plus a halo of W-1 rows
// per run; consecutive lanes take consecutive channels of one row.
#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

constexpr int kConvThreads = 256;
constexpr int kConvBatch = 8;  // token rows whose loads are in flight together

// Window of the W-1 inputs before the current token, oldest first.
template <int W, int V>
struct Window {
  float v[W - 1][V];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) v[k][e] = 0.f;
  }
  __device__ __forceinline__ void push(const float* x) {
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) v[k][e] = v[k + 1][e];
#pragma unroll
    for (int e = 0; e < V; ++e) v[W - 2][e] = x[e];
  }
};

template <class IO, int V, int W>
__device__ __forceinline__ void load_weights(const float* w, const float* bias, int64_t d, float (&wv)[W][V],
                                             float (&bv)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) wv[k][e] = w[(d + e) * W + k];
    bv[e] = bias ? bias[d + e] : 0.f;
  }
}

// The window entering token t0 of row b: the W-1 inputs before it, zero from
// where another sequence starts.
template <class IO, int V, int W, bool PACKED>
__device__ __forceinline__ void window_at(const ConvArgs& a, const typename IO::type* xr, const int* sr, int64_t b,
                                          int64_t d, int64_t t0, Window<W, V>& win) {
  win.clear();
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int64_t j = t0 - (W - 1) + k;
    float x[V];
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = 0.f;
    if (j >= 0) {
      if (PACKED && j > 0 && sr[j] != sr[j - 1]) win.clear();
      load_vec<IO, V>(xr + j * a.x_row, x);
    } else if (a.init) {
      load_vec<IO, V>(static_cast<const typename IO::type*>(a.init) + (b * (W - 1) + j + W - 1) * a.D + d, x);
    }
    win.push(x);
  }
  if (PACKED && t0 > 0 && t0 < a.L && sr[t0] != sr[t0 - 1]) win.clear();
}

template <class IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_forward_kernel(ConvArgs a, int64_t nrun, int run, int64_t total) {
  typedef typename IO::type T;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (idx >= total) return;
  const int64_t Dv = a.D / V;
  const int64_t d = (idx % Dv) * V;
  const int64_t rb = idx / Dv;
  const int64_t b = rb / nrun, t0 = (rb % nrun) * run;
  const int64_t t1 = t0 + run < a.L ? t0 + run : a.L;
  const T* xr = static_cast<const T*>(a.x) + b * a.L * a.x_row + d;
  const int* sr = PACKED ? a.seq_idx + b * a.L : nullptr;
  T* yr = static_cast<T*>(a.y) + b * a.L * a.D + d;
  float wv[W][V], bv[V];
  load_weights<IO, V, W>(a.w, a.bias, d, wv, bv);
  Window<W, V> win;
  window_at<IO, V, W, PACKED>(a, xr, sr, b, d, t0, win);
  for (int64_t t = t0; t < t1; t += kConvBatch) {
    float x[kConvBatch][V];
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i)
      load_vec<IO, V>(xr + (t + i < t1 ? t + i : t1 - 1) * a.x_row, x[i]);
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i) {
      if (t + i >= t1) break;
      if (PACKED && t + i > t0 && sr[t + i] != sr[t + i - 1]) win.clear();
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float p = bv[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) p = fmaf(wv[k][e], win.v[k][e], p);
        p = fmaf(wv[W - 1][e], x[i][e], p);
        o[e] = SILU ? p * sigmoid(p) : p;
      }
      store_vec<IO, V>(yr + (t + i) * a.D, o);
      win.push(x[i]);
    }
  }
  if (t1 == a.L && a.final_state) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      store_vec<IO, V>(static_cast<T*>(a.final_state) + (b * (W - 1) + k) * a.D + d, win.v[k]);
  }
}

// Convolution states after given tokens (packed prompts that go on decoding).
template <class IO, int W>
__global__ __launch_bounds__(kConvThreads) void conv_seq_states_kernel(ConvArgs a) {
  typedef typename IO::type T;
  const int64_t d = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t s = blockIdx.y;
  if (d >= a.D) return;
  const int64_t tok = a.seq_last[s];
  if (tok < 0 || tok >= a.B * a.L) return;
  const int64_t b = tok / a.L, t = tok % a.L;
  const T* xr = static_cast<const T*>(a.x) + b * a.L * a.x_row + d;
  const int* sr = a.seq_idx ? a.seq_idx + b * a.L : nullptr;
  T* o = static_cast<T*>(a.seq_states) + s * (W - 1) * a.D + d;
  bool same = true;
#pragma unroll
  for (int k = W - 2; k >= 0; --k) {
    const int64_t j = t - (W - 2) + k;
    if (sr && j + 1 > 0 && j + 1 <= t && sr[j + 1] != sr[j < 0 ? 0 : j]) same = false;
    T v = IO::put(0.f);
    if (same && j >= 0) v = xr[j * a.x_row];
    else if (same && a.init) v = static_cast<const T*>(a.init)[(b * (W - 1) + j + W - 1) * a.D + d];
    o[k * a.D] = v;
  }
}

// Backward.  Walking a run of tokens forwards, token t's dpre (taps of x from
// the window) reaches dx of t-W+1 .. t; the pending sums of the last W-1
// inputs ride in registers beside the window.  A run also computes the W-1
// dpre after its end, for its own last inputs.  Inputs before the run belong
// to the run before it (or to the initial state).
template <class IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_backward_kernel(ConvArgs a, int64_t nrun, int run, int64_t total) {
  typedef typename IO::type T;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (idx >= total) return;
  const int64_t Dv = a.D / V;
  const int64_t d = (idx % Dv) * V;
  const int64_t rb = idx / Dv;
  const int64_t b = rb / nrun, t0 = (rb % nrun) * run;
  const int64_t t1 = t0 + run < a.L ? t0 + run : a.L;
  const int64_t t2 = t1 + W - 1 < a.L ? t1 + W - 1 : a.L;  // dpre needed up to here
  const T* xr = static_cast<const T*>(a.x) + b * a.L * a.x_row + d;
  const T* gr = static_cast<const T*>(a.dy) + b * a.L * a.D + d;
  const int* sr = PACKED ? a.seq_idx + b * a.L : nullptr;
  T* dxr = static_cast<T*>(a.dx) + b * a.L * a.dx_row + d;
  float wv[W][V], bv[V];
  load_weights<IO, V, W>(a.w, a.bias, d, wv, bv);
  Window<W, V> win, pend;  // pend.v[k]: dx collected so far of the input win.v[k]
  window_at<IO, V, W, PACKED>(a, xr, sr, b, d, t0, win);
  pend.clear();
  float dw[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][e] = 0.f;
  }
  // A sequence start at t ends every pending sum: the inputs before it are
  // complete.  The W-1 pending inputs of token t are t-W+1 .. t-1.
  auto finish = [&](int64_t j, const float* g) {  // dx of input j is complete
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = g[e];
    if (j >= 0) {
      if (j >= t0 && j < t1) {
        if (a.dfinal && j >= a.L - (W - 1) ) {
          bool own = true;
          if (PACKED)
            for (int64_t q = j + 1; q < a.L; ++q) own = own && sr[q] == sr[q - 1];
          if (own) {
            float f[V];
            load_vec<IO, V>(static_cast<const T*>(a.dfinal) + (b * (W - 1) + j - (a.L - (W - 1))) * a.D + d, f);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] += f[e];
          }
        }
        store_vec<IO, V>(dxr + j * a.dx_row, o);
      }
    } else if (t0 == 0 && a.dinit) {
      // row j of the initial state; with fewer tokens than taps part of it is
      // still in the final state
      const int64_t k = j + W - 1;
      const int64_t kf = k - a.L;  // its place in the final state
      if (a.dfinal && kf >= 0) {
        bool own = true;
        if (PACKED)
          for (int64_t q = 1; q < a.L; ++q) own = own && sr[q] == sr[q - 1];
        if (own) {
          float f[V];
          load_vec<IO, V>(static_cast<const T*>(a.dfinal) + (b * (W - 1) + kf) * a.D + d, f);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += f[e];
        }
      }
      store_vec<IO, V>(static_cast<T*>(a.dinit) + (b * (W - 1) + k) * a.D + d, o);
    }
  };
  for (int64_t t = t0; t < t2; t += kConvBatch) {
    float x[kConvBatch][V], g[kConvBatch][V];
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i) {
      const int64_t tc = t + i < t2 ? t + i : t2 - 1;
      load_vec<IO, V>(xr + tc * a.x_row, x[i]);
      load_vec<IO, V>(gr + tc * a.D, g[i]);
    }
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i) {
      if (t + i >= t2) break;
      const int64_t tt = t + i;
      bool live[W - 1];  // whether pending input k shares the token's sequence
#pragma unroll
      for (int k = 0; k < W - 1; ++k) live[k] = true;
      if (PACKED) {
        bool same = true;
#pragma unroll
        for (int k = W - 2; k >= 0; --k) {
          const int64_t j = tt - (W - 1) + k;
          if (j + 1 > 0 && sr[j + 1] != sr[j < 0 ? 0 : j]) same = false;
          live[k] = same;
        }
        if (tt > 0 && sr[tt] != sr[tt - 1]) win.clear();
      }
      const bool in = tt < t1;
      float fresh[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float p = bv[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) p = fmaf(wv[k][e], win.v[k][e], p);
        p = fmaf(wv[W - 1][e], x[i][e], p);
        float dp = g[i][e];
        if (SILU) dp *= dsilu(p, sigmoid(p));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          const float c = dp * wv[k][e];
          pend.v[k][e] += (!PACKED || live[k]) ? c : 0.f;
        }
        fresh[e] = dp * wv[W - 1][e];
        if (in) {
#pragma unroll
          for (int k = 0; k < W - 1; ++k) dw[k][e] = fmaf(dp, win.v[k][e], dw[k][e]);
          dw[W - 1][e] = fmaf(dp, x[i][e], dw[W - 1][e]);
          db[e] += dp;
        }
      }
      finish(tt - (W - 1), pend.v[0]);
      win.push(x[i]);
      pend.push(fresh);
    }
  }
  if (t2 == a.L) {  // no dpre after the row: what is pending is complete
#pragma unroll
    for (int k = 0; k < W - 1; ++k) finish(a.L - (W - 1) + k, pend.v[k]);
  }
  // partial sums of this run: ws[rb][W+1][D]
  float* ws = a.ws + rb * (W + 1) * a.D + d;
#pragma unroll
  for (int k = 0; k < W; ++k) store_vec<IoF32, V>(ws + k * a.D, dw[k]);
  store_vec<IoF32, V>(ws + W * a.D, db);
}

// dw [D,W] and dbias [D] from the column sums [W+1][D]
template <int W>
__global__ __launch_bounds__(kConvThreads) void conv_weight_kernel(const float* __restrict__ sums, int64_t D,
                                                                   float* __restrict__ dw, float* __restrict__ db) {
  const int64_t d = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (d >= D) return;
#pragma unroll
  for (int k = 0; k < W; ++k) dw[d * W + k] = sums[k * D + d];
  if (db) db[d] = sums[W * D + d];
}

template <class IO, int V, int W, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(ConvArgs a, const typename IO::type* state,
                                                                 typename IO::type* state_out, int64_t total) {
  typedef typename IO::type T;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (idx >= total) return;
  const int64_t Dv = a.D / V;
  const int64_t d = (idx % Dv) * V, b = idx / Dv;
  float wv[W][V], bv[V], x[V], o[V], st[W - 1][V];
  load_vec<IO, V>(static_cast<const T*>(a.x) + b * a.x_row + d, x);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) load_vec<IO, V>(state + (b * (W - 1) + k) * a.D + d, st[k]);
  load_weights<IO, V, W>(a.w, a.bias, d, wv, bv);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float p = bv[e];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) p = fmaf(wv[k][e], st[k][e], p);
    p = fmaf(wv[W - 1][e], x[e], p);
    o[e] = SILU ? p * sigmoid(p) : p;
  }
  store_vec<IO, V>(static_cast<T*>(a.y) + b * a.D + d, o);
#pragma unroll
  for (int k = 0; k + 1 < W - 1; ++k) store_vec<IO, V>(state_out + (b * (W - 1) + k) * a.D + d, st[k + 1]);
  store_vec<IO, V>(state_out + (b * (W - 1) + W - 2) * a.D + d, x);
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 16-byte accesses need whole 16-byte units in every row
static bool conv_vec(const ConvArgs& a, int kvec) {
  return a.D % kvec == 0 && a.x_row % kvec == 0 && a.dx_row % kvec == 0 && al16(a.x) && al16(a.dx);
}

// Tokens a thread walks: runs of 32 keep the halo under a tenth of the reads;
// short runs where 32 would leave compute units without a wave.
static int conv_run(int64_t B, int64_t L, int64_t Dv) {
  int run = 32;
  while (run > kConvBatch && B * ((L + run - 1) / run) * Dv < (int64_t)device_cu_count() * 8 * 64) run /= 2;
  return run;
}

template <class IO, int V, int W, bool PACKED>
static hipError_t conv_forward_v(const ConvArgs& a, hipStream_t s) {
  const int64_t Dv = a.D / V;
  const int run = conv_run(a.B, a.L, Dv);
  const int64_t nrun = (a.L + run - 1) / run, total = a.B * nrun * Dv;
  const dim3 grid((unsigned)((total + kConvThreads - 1) / kConvThreads));
  if (a.silu)
    hipLaunchKernelGGL((conv_forward_kernel<IO, V, W, PACKED, true>), grid, dim3(kConvThreads), 0, s, a, nrun, run, total);
  else
    hipLaunchKernelGGL((conv_forward_kernel<IO, V, W, PACKED, false>), grid, dim3(kConvThreads), 0, s, a, nrun, run, total);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nseq == 0) return e;
  hipLaunchKernelGGL((conv_seq_states_kernel<IO, W>),
                     dim3((unsigned)((a.D + kConvThreads - 1) / kConvThreads), (unsigned)a.nseq), dim3(kConvThreads), 0,
                     s, a);
  return hipGetLastError();
}

// Partial rows of dw / dbias: one per run of tokens.
static int conv_bwd_run(int64_t B, int64_t L, int64_t Dv) {
  int run = 64;
  while (run > kConvBatch && B * ((L + run - 1) / run) * Dv < (int64_t)device_cu_count() * 8 * 64) run /= 2;
  return run;
}

template <class IO, int V, int W, bool PACKED>
static hipError_t conv_backward_v(const ConvArgs& a, hipStream_t s) {
  const int64_t Dv = a.D / V;
  const int run = conv_bwd_run(a.B, a.L, Dv);
  const int64_t nrun = (a.L + run - 1) / run, total = a.B * nrun * Dv;
  const dim3 grid((unsigned)((total + kConvThreads - 1) / kConvThreads));
  if (a.silu)
    hipLaunchKernelGGL((conv_backward_kernel<IO, V, W, PACKED, true>), grid, dim3(kConvThreads), 0, s, a, nrun, run, total);
  else
    hipLaunchKernelGGL((conv_backward_kernel<IO, V, W, PACKED, false>), grid, dim3(kConvThreads), 0, s, a, nrun, run, total);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t C = (W + 1) * a.D;
  float* sums = a.ws + a.B * nrun * C;
  if ((e = launch_colsum(a.ws, a.B * nrun, C, sums, s)) != hipSuccess) return e;
  hipLaunchKernelGGL((conv_weight_kernel<W>), dim3((unsigned)((a.D + kConvThreads - 1) / kConvThreads)),
                     dim3(kConvThreads), 0, s, sums, a.D, a.dw, a.dbias);
  return hipGetLastError();
}

size_t conv_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int W) {
  // the widest thread leaves the shortest runs: size for the smaller of both
  const int r8 = conv_bwd_run(B, L, D / 8 > 0 ? D / 8 : 1), r1 = conv_bwd_run(B, L, D);
  const int run = r8 < r1 ? r8 : r1;
  const int64_t nrun = (L + run - 1) / run;
  return sizeof(float) * (size_t)((B * nrun + 1) * (W + 1) * D);
}

template <class IO, int V, int W>
static hipError_t conv_step_v(const ConvArgs& a, const void* st, void* so, hipStream_t s) {
  typedef typename IO::type T;
  const int64_t total = a.B * (a.D / V);
  const dim3 grid((unsigned)((total + kConvThreads - 1) / kConvThreads));
  if (a.silu)
    hipLaunchKernelGGL((conv_step_kernel<IO, V, W, true>), grid, dim3(kConvThreads), 0, s, a,
                       static_cast<const T*>(st), static_cast<T*>(so), total);
  else
    hipLaunchKernelGGL((conv_step_kernel<IO, V, W, false>), grid, dim3(kConvThreads), 0, s, a,
                       static_cast<const T*>(st), static_cast<T*>(so), total);
  return hipGetLastError();
}

template <class F>
static hipError_t with_width(int W, F f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
  }
  return hipErrorInvalidValue;
}
template <class F>
static hipError_t with_io(bool bf16, F f) {
  return bf16 ? f(IoBF16{}) : f(IoF32{});
}

hipError_t launch_conv_forward(const ConvArgs& a, bool bf16, hipStream_t s) {
  return with_io(bf16, [&](auto io) {
    typedef decltype(io) IO;
    return with_width(a.W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (conv_vec(a, IO::kVec))
        return a.seq_idx ? conv_forward_v<IO, IO::kVec, W, true>(a, s) : conv_forward_v<IO, IO::kVec, W, false>(a, s);
      return a.seq_idx ? conv_forward_v<IO, 1, W, true>(a, s) : conv_forward_v<IO, 1, W, false>(a, s);
    });
  });
}

hipError_t launch_conv_backward(const ConvArgs& a, bool bf16, hipStream_t s) {
  return with_io(bf16, [&](auto io) {
    typedef decltype(io) IO;
    return with_width(a.W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (conv_vec(a, IO::kVec))
        return a.seq_idx ? conv_backward_v<IO, IO::kVec, W, true>(a, s) : conv_backward_v<IO, IO::kVec, W, false>(a, s);
      return a.seq_idx ? conv_backward_v<IO, 1, W, true>(a, s) : conv_backward_v<IO, 1, W, false>(a, s);
    });
  });
}

hipError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, bool bf16, hipStream_t s) {
  return with_io(bf16, [&](auto io) {
    typedef decltype(io) IO;
    return with_width(a.W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (conv_vec(a, IO::kVec)) return conv_step_v<IO, IO::kVec, W>(a, state, state_out, s);
      return conv_step_v<IO, 1, W>(a, state, state_out, s);
    });
  });
}

}  // namespace ssd
