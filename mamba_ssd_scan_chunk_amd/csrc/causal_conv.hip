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
// operations.  A wave takes 64 neighbouring groups of V channels (8 bytes a
// lane; one channel where rows are not whole 8-byte units) and walks a run of
// tokens with the last W-1 inputs in registers, so each input is read once
// plus a halo of W-1 rows per run.  The run, its row addresses and its
// sequence starts are the same for the whole wave and live in scalars.
// 2 x 8192 tokens of 5376 channels (bf16): 71 us forward, 5.0 TB/s, and 113 us
// backward, 4.7 TB/s, where a copy reaches 4.95.
#include <type_traits>

#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

constexpr int kConvWaves = 4;  // runs of a block
constexpr int kConvThreads = 64 * kConvWaves;
constexpr int kConvBatch = 8;     // token rows whose loads are in flight together, forward
constexpr int kConvBwdBatch = 4;  // and backward, of two inputs

// The wave's run of tokens and its lane's channels.
struct ConvRun {
  int64_t group, rb, b, t0, t1;  // the block's runs are those of a group
  int64_t d0, d;  // first channel of the wave, and of the lane
  bool live;      // the run exists
  bool ok;        // the lane has channels (one without repeats the last ones')
};
template <int V>
__device__ __forceinline__ ConvRun conv_run_of(const ConvArgs& a, int64_t nrun, int run, int64_t ncb) {
  ConvRun r;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t block = flat_block();
  r.group = block / (unsigned)ncb;
  r.rb = r.group * kConvWaves + wave;
  r.live = r.rb < a.B * nrun;
  const int64_t rb = r.live ? r.rb : 0;
  r.b = rb / nrun;
  r.t0 = (rb - r.b * nrun) * run;
  r.t1 = r.t0 + run < a.L ? r.t0 + run : a.L;
  r.d0 = (int64_t)(block % (unsigned)ncb) * 64 * V;
  r.d = r.d0 + (threadIdx.x & 63) * V;
  r.ok = r.d < a.D;
  if (!r.ok) r.d = a.D - V;
  return r;
}

// Bit i of the result (uniform): token t + i, i < n <= 64, lies in the row and
// begins another sequence than its predecessor's.
__device__ __forceinline__ uint64_t start_bits(const int* sr, int64_t t, int n, int64_t L) {
  const int64_t j = t + (threadIdx.x & 63);
  bool s = false;
  if ((int)(threadIdx.x & 63) < n && j > 0 && j < L) s = sr[j] != sr[j - 1];
  return __ballot(s);
}

// V elements as loaded and stored, by a buffer's uniform offset `so` and the
// lane's own.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <class IO, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(typename IO::type);
  typedef std::conditional_t<kBytes == 2, uint16_t,
                             std::conditional_t<kBytes == 4, uint32_t, std::conditional_t<kBytes == 8, u32x2_t, u32x4_t>>>
      type;
  __device__ __forceinline__ static type load(__amdgpu_buffer_rsrc_t r, int off, int so) {
    if constexpr (kBytes == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, so, 0);
    else if constexpr (kBytes == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, off, so, 0);
    else if constexpr (kBytes == 8) return __builtin_amdgcn_raw_buffer_load_b64(r, off, so, 0);
    else return __builtin_amdgcn_raw_buffer_load_b128(r, off, so, 0);
  }
  __device__ __forceinline__ static void widen(const type& q, float* o) {
    if constexpr (kBytes == 2) {
      o[0] = IO::get(q);
    } else if constexpr (kBytes == 4) {
      o[0] = __uint_as_float(q);
    } else if constexpr (kBytes == 8) {
      o[0] = __uint_as_float(q.x << 16);
      o[1] = __uint_as_float(q.x & 0xffff0000u);
      o[2] = __uint_as_float(q.y << 16);
      o[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __uint_as_float(q[e]);
    }
  }
  __device__ __forceinline__ static void store(__amdgpu_buffer_rsrc_t r, int off, int so, const float* v) {
    if constexpr (kBytes == 2) {
      __builtin_amdgcn_raw_buffer_store_b16(IO::put(v[0]), r, off, so, 0);
    } else if constexpr (kBytes == 4) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, off, so, 0);
    } else if constexpr (kBytes == 8) {
      const u32x2_t q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      __builtin_amdgcn_raw_buffer_store_b64(q, r, off, so, 0);
    } else {
      const u32x4_t q = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      __builtin_amdgcn_raw_buffer_store_b128(q, r, off, so, 0);
    }
  }
};
template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const T* row) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(row), 0, 0x7fffffff, 0x00027000);
}

// A batch of rows, the last of n again past it.
template <class IO, int V, int NB>
struct Rows {
  typename Raw<IO, V>::type q[NB];
  __device__ __forceinline__ void load(const typename IO::type* row, int64_t stride, int n, int off) {
    const __amdgpu_buffer_rsrc_t r = rows_at(row);
    const int step = (int)stride * (int)sizeof(typename IO::type);
    int so = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      q[i] = Raw<IO, V>::load(r, off, so);
      so += i + 1 < n ? step : 0;
      asm volatile("" : "+s"(so));  // one running offset, not a multiple a row
    }
  }
  // Waits for the rows here.  Where a loop is entered with loads in flight the
  // compiler would else wait in it for the stores behind the next loads, too.
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : : "v"(q[i]));
  }
  __device__ __forceinline__ void get(int i, float* o) const { Raw<IO, V>::widen(q[i], o); }
  // the first row, and the others move up
  __device__ __forceinline__ void next(float* o) {
    get(0, o);
#pragma unroll
    for (int i = 0; i + 1 < NB; ++i) q[i] = q[i + 1];
  }
};

template <int NB>
__device__ __forceinline__ int tokens_left(int64_t t, int64_t end) {
  return (int)(end - t < NB ? end - t : NB);
}
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

template <int V, int W>
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
// where another sequence starts.  `ask` loads them, all at once, `fill` takes
// them; the run's first rows are asked for in between.
template <class IO, int V, int W, bool PACKED>
struct WindowAt {
  typename Raw<IO, V>::type q[W - 1];
  __device__ __forceinline__ void ask(const ConvArgs& a, const typename IO::type* xr, int64_t b, int64_t d, int64_t t0) {
    const typename IO::type* init = static_cast<const typename IO::type*>(a.init) + b * (W - 1) * a.D + d;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int64_t j = t0 - (W - 1) + k;
      const typename IO::type* p = j >= 0 ? xr + j * a.x_row : a.init ? init + (j + W - 1) * a.D : xr;
      q[k] = *reinterpret_cast<const typename Raw<IO, V>::type*>(p);
    }
  }
  // st: the starts from token t0 - W + 1 on
  __device__ __forceinline__ void fill(const ConvArgs& a, int64_t t0, uint64_t st, Window<W, V>& win) const {
    win.clear();
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      float x[V];
      Raw<IO, V>::widen(q[k], x);
      const bool there = t0 - (W - 1) + k >= 0 || a.init;
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = there ? x[e] : 0.f;
      if (PACKED && (st >> k & 1)) win.clear();
      win.push(x);
    }
    if (PACKED && (st >> (W - 1) & 1)) win.clear();
  }
};

template <class IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_forward_kernel(ConvArgs a, int64_t nrun, int run, int64_t ncb) {
  typedef typename IO::type T;
  const ConvRun r = conv_run_of<V>(a, nrun, run, ncb);
  if (!r.live) return;  // whole waves only: sequence starts are found by ballot
  const T* xr = static_cast<const T*>(a.x) + r.b * a.L * a.x_row + r.d;
  const int* sr = PACKED ? a.seq_idx + r.b * a.L : nullptr;
  float wv[W][V], bv[V];
  load_weights<V, W>(a.w, a.bias, r.d, wv, bv);
  WindowAt<IO, V, W, PACKED> before;
  before.ask(a, xr, r.b, r.d, r.t0);
  auto out = [&](const float (&tap)[W][V], float* o) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float p = bv[e];
#pragma unroll
      for (int k = 0; k < W; ++k) p = fmaf(wv[k][e], tap[k][e], p);
      o[e] = SILU ? p * sigmoid(p) : p;
    }
  };
  const int off = (int)((r.d - r.d0) * sizeof(T));
  const T* xb = static_cast<const T*>(a.x) + (r.b * a.L + r.t0) * a.x_row + r.d0;  // the batch's first row
  T* yb = static_cast<T*>(a.y) + (r.b * a.L + r.t0) * a.D + r.d0;
  Rows<IO, V, kConvBatch> x;
  x.load(xb, a.x_row, tokens_left<kConvBatch>(r.t0, r.t1), off);
  // the starts that the run can see, from token t0 - W + 1 on
  uint64_t starts = PACKED ? start_bits(sr, r.t0 - (W - 1), (int)(r.t1 - r.t0) + W - 1, a.L) : 0;
  Window<W, V> win;
  before.fill(a, r.t0, starts, win);
  starts = starts >> (W - 1) & ~uint64_t(1);  // from t0 on, whose own the window has seen
  x.settle();
  for (int64_t t = r.t0; t < r.t1; t += kConvBatch) {
    const int n = tokens_left<kConvBatch>(t, r.t1);
    const uint32_t st = PACKED ? (uint32_t)(starts >> (t - r.t0)) & 0xffu : 0;
    xb += kConvBatch * a.x_row;
    if (n == kConvBatch && st == 0) {
      // outputs first, then the next batch's loads, then the stores: loads
      // asked for behind the stores would be waited for with them
      float v[W - 1 + kConvBatch][V], o[kConvBatch][V];
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = win.v[k][e];
#pragma unroll
      for (int i = 0; i < kConvBatch; ++i) {
        x.get(i, v[W - 1 + i]);
        out(reinterpret_cast<const float(&)[W][V]>(v[i]), o[i]);
      }
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) win.v[k][e] = v[kConvBatch + k][e];
      const bool more = t + kConvBatch < r.t1;
      if (more) x.load(xb, a.x_row, tokens_left<kConvBatch>(t + kConvBatch, r.t1), off);
      const __amdgpu_buffer_rsrc_t yr = rows_at(yb);
      int so = 0;
#pragma unroll
      for (int i = 0; i < kConvBatch; ++i) {
        Raw<IO, V>::store(yr, off, so, o[i]);
        so += (int)a.D * (int)sizeof(T);
        asm volatile("" : "+s"(so));
      }
      yb += kConvBatch * a.D;
    } else {
#pragma unroll
      for (int i = 0; i < kConvBatch; ++i) {
        if (i >= n) break;
        if (PACKED && (st >> i & 1)) win.clear();
        float tap[W][V], o[V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) tap[k][e] = win.v[k][e];
        x.get(i, tap[W - 1]);
        out(tap, o);
        Raw<IO, V>::store(rows_at(yb), off, 0, o);
        yb += a.D;
        win.push(tap[W - 1]);
      }
      if (t + kConvBatch < r.t1) {
        x.load(xb, a.x_row, tokens_left<kConvBatch>(t + kConvBatch, r.t1), off);
        x.settle();
      }
    }
  }
  if (r.t1 == a.L && a.final_state && r.ok) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      store_vec<IO, V>(static_cast<T*>(a.final_state) + (r.b * (W - 1) + k) * a.D + r.d, win.v[k]);
  }
}

// Convolution states after given tokens (packed prompts that go on decoding).
template <class IO, int W>
__global__ __launch_bounds__(kConvThreads) void conv_seq_states_kernel(ConvArgs a) {
  typedef typename IO::type T;
  const int64_t s = blockIdx.y;
  const int64_t tok = a.seq_last[s];
  if (tok < 0 || tok >= a.B * a.L) return;
  const int64_t b = tok / a.L, t = tok % a.L;
  const int* sr = a.seq_idx ? a.seq_idx + b * a.L : nullptr;
  for (int64_t d = (int64_t)blockIdx.x * kConvThreads + threadIdx.x; d < a.D; d += (int64_t)gridDim.x * kConvThreads) {
    const T* xr = static_cast<const T*>(a.x) + b * a.L * a.x_row + d;
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
}

// Backward.  Walking a run of tokens forwards, token t's dpre (taps of x from
// the window) reaches dx of t-W+1 .. t; the pending sums of the last W-1
// inputs ride in registers beside the window.  A run also computes the W-1
// dpre after its end, for its own last inputs.  Inputs before the run belong
// to the run before it (or to the initial state).  The block's runs meet in
// LDS before dw and dbias go to memory.
// Whole batches without a sequence start take the straight path: inputs and
// sums in arrays whose indices the compiler knows (moving a window token by
// token cost a third of the instructions), the next loads before the stores
// (2 x 88022 tokens of 136 channels, fp32: 230 us with them after, 80 so).  The
// others, and the run's end, go a token at a time.
template <class IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_backward_kernel(ConvArgs a, int64_t nrun, int run, int64_t ncb) {
  typedef typename IO::type T;
  constexpr int NB = kConvBwdBatch;
  static_assert(NB >= W - 1, "only a run's first batch reaches inputs before the run");
  __shared__ float part[kConvWaves][(W + 1) * V][64];
  const ConvRun r = conv_run_of<V>(a, nrun, run, ncb);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float dw[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][e] = 0.f;
  }
  if (r.live) {
    const int64_t t0 = r.t0, t1 = r.t1, b = r.b, d = r.d;
    const int64_t t2 = t1 + W - 1 < a.L ? t1 + W - 1 : a.L;  // dpre needed up to here
    const T* xr = static_cast<const T*>(a.x) + b * a.L * a.x_row + d;
    const int* sr = PACKED ? a.seq_idx + b * a.L : nullptr;
    T* dxr = static_cast<T*>(a.dx) + b * a.L * a.dx_row + d;
    float wv[W][V], bv[V];
    load_weights<V, W>(a.w, a.bias, d, wv, bv);
    WindowAt<IO, V, W, PACKED> before;
    before.ask(a, xr, b, d, t0);
    Window<W, V> win, pend;  // pend.v[k]: dx collected so far of the input win.v[k]
    pend.clear();
    auto finish = [&](int64_t j, const float* g) {  // dx of input j is complete
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = g[e];
      // with dfinal: the place of input j in the final state, if it is there
      // and no sequence starts after it
      const int64_t f = j - (a.L - (W - 1));
      if (a.dfinal && f >= 0) {
        bool own = true;
        if (PACKED)
          for (int64_t q = j < 0 ? 1 : j + 1; q < a.L; ++q) own = own && sr[q] == sr[q - 1];
        if (own) {
          float v[V];
          load_vec<IO, V>(static_cast<const T*>(a.dfinal) + (b * (W - 1) + f) * a.D + d, v);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += v[e];
        }
      }
      if (!r.ok) return;
      if (j >= 0) {
        if (j >= t0 && j < t1) store_vec<IO, V>(dxr + j * a.dx_row, o);
      } else if (t0 == 0 && a.dinit) {
        store_vec<IO, V>(static_cast<T*>(a.dinit) + (b * (W - 1) + j + W - 1) * a.D + d, o);
      }
    };
    auto dpre = [&](const float (&tap)[W][V], const float* g, float* dp) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float p = bv[e];
#pragma unroll
        for (int k = 0; k < W; ++k) p = fmaf(wv[k][e], tap[k][e], p);
        dp[e] = g[e];
        if (SILU) dp[e] *= dsilu(p, sigmoid(p));
      }
    };
    auto sums = [&](const float (&tap)[W][V], const float* dp) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][e] = fmaf(dp[e], tap[k][e], dw[k][e]);
        db[e] += dp[e];
      }
    };
    const int off = (int)((d - r.d0) * sizeof(T));
    const T* xb = static_cast<const T*>(a.x) + (b * a.L + t0) * a.x_row + r.d0;  // the batch's first rows
    const T* gb = static_cast<const T*>(a.dy) + (b * a.L + t0) * a.D + r.d0;
    Rows<IO, V, NB> x, g;
    x.load(xb, a.x_row, tokens_left<NB>(t0, t2), off);
    g.load(gb, a.D, tokens_left<NB>(t0, t2), off);
    // starts from token t0 - W + 1 on, all the run can see
    const uint64_t starts = PACKED ? start_bits(sr, t0 - (W - 1), (int)(t2 - t0) + W - 1, a.L) : 0;
    before.fill(a, t0, starts, win);
    x.settle();
    g.settle();
    // bit of token t in `starts`
    auto bit = [&](int64_t t) { return (int)(t - t0) + W - 1; };
    // no start in the batch nor in the W-2 tokens before it
    auto plain = [&](int64_t t) {
      return !PACKED || (starts >> (bit(t) - (W - 2)) & ((uint64_t(1) << (NB + W - 2)) - 1)) == 0;
    };
    int64_t t = t0;
    while (t < t2) {
      for (; t + NB <= t1 && plain(t); t += NB) {
        const int left = t + NB < t2 ? tokens_left<NB>(t + NB, t2) : 0;
        xb += NB * a.x_row;
        gb += NB * a.D;
        // v[k], dx[k]: inputs t - (W-1) + k and what has reached them; all
        // arithmetic first, then the next loads, then the stores (loads asked
        // for behind the stores would be waited for with them)
        float v[W - 1 + NB][V], dx[W - 1 + NB][V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            v[k][e] = win.v[k][e];
            dx[k][e] = pend.v[k][e];
          }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          float gv[V], dp[V];
          x.get(i, v[W - 1 + i]);
          g.get(i, gv);
          const float(&tap)[W][V] = reinterpret_cast<const float(&)[W][V]>(v[i]);
          dpre(tap, gv, dp);
          sums(tap, dp);
#pragma unroll
          for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) dx[i + k][e] = fmaf(dp[e], wv[k][e], dx[i + k][e]);
            dx[i + W - 1][e] = dp[e] * wv[W - 1][e];
          }
          __builtin_amdgcn_sched_barrier(0);  // token by token, in fewer registers
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            win.v[k][e] = v[NB + k][e];
            pend.v[k][e] = dx[NB + k][e];
          }
        if (left > 0) {
          x.load(xb, a.x_row, left, off);
          g.load(gb, a.D, left, off);
        }
        const __amdgpu_buffer_rsrc_t o = rows_at(static_cast<T*>(a.dx) + (b * a.L + t - (W - 1)) * a.dx_row + r.d0);
        int so = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if (i >= W - 1 || t > t0) Raw<IO, V>::store(o, off, so, dx[i]);
          else if (t0 == 0 && a.dinit) store_vec<IO, V>(static_cast<T*>(a.dinit) + (b * (W - 1) + i) * a.D + d, dx[i]);
          so += (int)a.dx_row * (int)sizeof(T);
          asm volatile("" : "+s"(so));
        }
      }
      if (t >= t2) break;
      const int n = tokens_left<NB>(t, t2);
#pragma clang loop unroll(disable)
      for (int i = 0; i < n; ++i) {
        // tokens since the last start, the token of the start itself counting
        // 0; no more than W-1 matter
        int since = W;
        if (PACKED) {
          const uint64_t m = starts << (63 - bit(t) - i);
          since = m ? __builtin_clzll(m) : W;
        }
        float tap[W][V], gv[V], dp[V], fresh[V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) tap[k][e] = win.v[k][e] = PACKED && since == 0 ? 0.f : win.v[k][e];
        x.next(tap[W - 1]);
        g.next(gv);
        dpre(tap, gv, dp);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          const bool same = !PACKED || W - 1 - k <= since;  // the input is of the token's sequence
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float f = fmaf(dp[e], wv[k][e], pend.v[k][e]);
            pend.v[k][e] = same ? f : pend.v[k][e];
          }
        }
        if (t + i < t1) sums(tap, dp);
#pragma unroll
        for (int e = 0; e < V; ++e) fresh[e] = dp[e] * wv[W - 1][e];
        finish(t + i - (W - 1), pend.v[0]);
        win.push(tap[W - 1]);
        pend.push(fresh);
      }
      t += n;
      if (t < t2) {
        xb += NB * a.x_row;
        gb += NB * a.D;
        x.load(xb, a.x_row, tokens_left<NB>(t, t2), off);
        g.load(gb, a.D, tokens_left<NB>(t, t2), off);
        x.settle();
        g.settle();
      }
    }
    if (t2 == a.L) {  // no dpre after the row: what is pending is complete
#pragma unroll
      for (int k = 0; k < W - 1; ++k) finish(a.L - (W - 1) + k, pend.v[k]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) part[wave][k * V + e][lane] = dw[k][e];
    part[wave][W * V + e][lane] = db[e];
  }
  __syncthreads();
  // partial sums of the block's runs: ws[row group][W+1][D]; a block past the
  // last one has none (left to here: asked at the start it costs registers, 170
  // instead of 166 leave two waves a SIMD of three, 2 x 8192 x 5376 112 -> 128 us)
  if (r.ok && r.group * kConvWaves < a.B * nrun) {
    float* ws = a.ws + r.group * (W + 1) * a.D + r.d;
    for (int k = wave; k <= W; k += kConvWaves) {
      float s[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[e] = 0.f;
#pragma unroll
        for (int q = 0; q < kConvWaves; ++q) s[e] += part[q][k * V + e][lane];
      }
      store_vec<IoF32, V>(ws + k * a.D, s);
    }
  }
}

// dw [D,W] and dbias [D] from the row groups' partial sums [R][W+1][D]
template <int W>
__global__ __launch_bounds__(kColsumThreads) void conv_param_kernel(const float* __restrict__ part, int64_t R, int64_t D,
                                                                    float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float lds[kColsumThreads];
  const int64_t c = (int64_t)flat_block() * 64 + (threadIdx.x & 63), C = (W + 1) * D;
  const float s = column_sum(part + (c < C ? c : C - 1), R, C, lds);
  if (threadIdx.x >= 64 || c >= C) return;
  const int64_t k = c / D, d = c - k * D;
  if (k < W) dw[d * W + k] = s;
  else if (db) db[d] = s;
}

// Single-token step, V channels a thread: the time of a launch (1 x 1792
// channels 2.4 to 2.8 us).
template <class IO, int V, int W, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(ConvArgs a, const typename IO::type* state,
                                                                 typename IO::type* state_out, int64_t total) {
  typedef typename IO::type T;
  const int64_t idx = (int64_t)flat_block() * kConvThreads + threadIdx.x;
  if (idx >= total) return;
  const int64_t Dv = a.D / V;
  const int64_t d = (idx % Dv) * V, b = idx / Dv;
  float wv[W][V], bv[V], x[V], o[V], st[W - 1][V];
  load_vec<IO, V>(static_cast<const T*>(a.x) + b * a.x_row + d, x);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) load_vec<IO, V>(state + (b * (W - 1) + k) * a.D + d, st[k]);
  load_weights<V, W>(a.w, a.bias, d, wv, bv);
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

// Vector accesses (four channels a lane) need rows in whole multiples of them
static bool conv_vec(const ConvArgs& a, int es) {
  const uintptr_t m = 4 * es - 1;
  return a.D % 4 == 0 && a.x_row % 4 == 0 && a.dx_row % 4 == 0 && (reinterpret_cast<uintptr_t>(a.x) & m) == 0 &&
         (reinterpret_cast<uintptr_t>(a.dx) & m) == 0;
}

// Tokens of a run: `most` (the halo is then a small part of the reads), less
// where that leaves a compute unit fewer than four waves (gradients of 4 x 2048
// tokens of 1792 channels: 33 us where eight are asked for, 30.5 so).
static int conv_run(int64_t B, int64_t L, int64_t ncb, int most) {
  int run = most;
  while (run > kConvBatch && B * ((L + run - 1) / run) * ncb < (int64_t)device_cu_count() * 4) run /= 2;
  return run;
}
static int64_t conv_blocks_of(int64_t D, int V) { return (D / V + 63) / 64; }

struct ConvGrid {
  int run;
  int64_t nrun, ncb, groups;  // groups of kConvWaves runs
};
static ConvGrid conv_grid(int64_t B, int64_t L, int64_t D, int V, int most) {
  ConvGrid g;
  g.ncb = conv_blocks_of(D, V);
  g.run = conv_run(B, L, g.ncb, most);
  g.nrun = (L + g.run - 1) / g.run;
  g.groups = (B * g.nrun + kConvWaves - 1) / kConvWaves;
  return g;
}
// Measured at 2 x 8192 tokens of 5376 channels (bf16): forward runs of 16 tokens
// 71 us, 8 79, 24 71, 32 72, 64 75; backward runs of 32 112 us, of 40, 48 and 56
// 2 to 5% more (4 x 8192 tokens of 2304 channels in packed rows: 101, 3 to 7%).
constexpr int kConvFwdRun = 16, kConvBwdRun = 32;

template <class IO, int V, int W, bool PACKED>
static hipError_t conv_forward_v(const ConvArgs& a, hipStream_t s) {
  const ConvGrid g = conv_grid(a.B, a.L, a.D, V, kConvFwdRun);
  const dim3 grid = flat_grid(g.groups * g.ncb);
  auto kern = a.silu ? conv_forward_kernel<IO, V, W, PACKED, true> : conv_forward_kernel<IO, V, W, PACKED, false>;
  hipLaunchKernelGGL(kern, grid, dim3(kConvThreads), 0, s, a, g.nrun, g.run, g.ncb);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nseq == 0) return e;
  hipLaunchKernelGGL((conv_seq_states_kernel<IO, W>),
                     dim3(flat_grid((a.D + kConvThreads - 1) / kConvThreads).x, (unsigned)a.nseq), dim3(kConvThreads), 0,
                     s, a);
  return hipGetLastError();
}

template <class IO, int V, int W, bool PACKED>
static hipError_t conv_backward_v(const ConvArgs& a, hipStream_t s) {
  const ConvGrid g = conv_grid(a.B, a.L, a.D, V, kConvBwdRun);
  const dim3 grid = flat_grid(g.groups * g.ncb);
  auto kern = a.silu ? conv_backward_kernel<IO, V, W, PACKED, true> : conv_backward_kernel<IO, V, W, PACKED, false>;
  hipLaunchKernelGGL(kern, grid, dim3(kConvThreads), 0, s, a, g.nrun, g.run, g.ncb);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((conv_param_kernel<W>), flat_grid(((W + 1) * a.D + 63) / 64), dim3(kColsumThreads), 0, s,
                     a.ws, g.groups, a.D, a.dw, a.dbias);
  return hipGetLastError();
}

size_t conv_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int W) {
  // vector or single-element accesses depend on the pointers: the larger of both
  const int64_t g4 = D >= 4 ? conv_grid(B, L, D, 4, kConvBwdRun).groups : 0;
  const int64_t g1 = conv_grid(B, L, D, 1, kConvBwdRun).groups;
  return sizeof(float) * (size_t)(g4 > g1 ? g4 : g1) * (size_t)((W + 1) * D);
}

template <class IO, int V, int W>
static hipError_t conv_step_v(const ConvArgs& a, const void* st, void* so, hipStream_t s) {
  typedef typename IO::type T;
  const int64_t total = a.B * (a.D / V);
  const dim3 grid = flat_grid((total + kConvThreads - 1) / kConvThreads);
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
      if (conv_vec(a, sizeof(typename IO::type)))
        return a.seq_idx ? conv_forward_v<IO, 4, W, true>(a, s) : conv_forward_v<IO, 4, W, false>(a, s);
      return a.seq_idx ? conv_forward_v<IO, 1, W, true>(a, s) : conv_forward_v<IO, 1, W, false>(a, s);
    });
  });
}

hipError_t launch_conv_backward(const ConvArgs& a, bool bf16, hipStream_t s) {
  return with_io(bf16, [&](auto io) {
    typedef decltype(io) IO;
    return with_width(a.W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (conv_vec(a, sizeof(typename IO::type)))
        return a.seq_idx ? conv_backward_v<IO, 4, W, true>(a, s) : conv_backward_v<IO, 4, W, false>(a, s);
      return a.seq_idx ? conv_backward_v<IO, 1, W, true>(a, s) : conv_backward_v<IO, 1, W, false>(a, s);
    });
  });
}

hipError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, bool bf16, hipStream_t s) {
  return with_io(bf16, [&](auto io) {
    typedef decltype(io) IO;
    return with_width(a.W, [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (conv_vec(a, sizeof(typename IO::type))) return conv_step_v<IO, 4, W>(a, state, state_out, s);
      return conv_step_v<IO, 1, W>(a, state, state_out, s);
    });
  });
}

}  // namespace ssd
