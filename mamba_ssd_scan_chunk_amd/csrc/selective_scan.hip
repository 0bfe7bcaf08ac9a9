// selective_scan.hip -- the selective state-space scan: per batch b, channel d
// (group g = d / (D/G)) and state n
//     dt[t]   = softplus(raw[t,d] + bias[d])                    (or without)
//     h[t,n]  = exp(dt[t] A[d,n]) h[t-1,n] + dt[t] u[t,d] B[t,g,n]
//     y[t,d]  = (sum_n C[t,g,n] h[t,n] + D[d] u[t,d]) * z sigmoid(z)
// for whole prompts, and its single-token step.
//
// Each (channel, state) pair decays at its own rate, so unlike a scan with one
// decay a head there is no matrix product in it: per token, channel and state
// it costs a multiply and an exponential for the decay, a multiply and a fused
// multiply-add for the state and one for the output, on the vector ALUs.  With
// 16 states that outweighs the 8 bytes (bf16, gated) moved per token and
// channel.
//
// One wave takes 64 channels (a lane each) and a chunk of tokens; states stay
// in LDS, four of them in registers at a time over 16 tokens.  B and C are the
// same for all lanes, so they come through scalar loads as scalar operands.
// Where channels alone leave compute units idle the tokens are split: a first
// pass takes every chunk's state from zero, a second carries the states from
// chunk to chunk (decays multiply as exp of the summed dt), and the last
// computes the outputs from the carried states.
#include "layer_device.hpp"
#include "layer_launch.hpp"
#include "selective_scan.hpp"

namespace ssd {

// State passes: FINAL writes outputs from the chunk's entering state, else
// only the state the chunk leaves and its summed dt.
template <class IO, bool PACKED, bool FINAL>
__global__ __launch_bounds__(64) void scan_chunk_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  typedef typename IO::type T;
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  const ScanBlock k = scan_block(g, a);
  const int N = (int)a.N;
  float* hs = lds;  // h[n][lane]
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;

  const float* h_in = nullptr;
  if (FINAL && g.nc > 1) h_in = ws.carry + (k.b * g.nc + k.c) * N * a.D;
  if (k.c == 0) h_in = a.h0 ? a.h0 + k.b * N * a.D : nullptr;
  for (int n = 0; n < N; ++n) hs[n * 64 + lane] = h_in ? h_in[(int64_t)n * a.D + d] : 0.f;
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
  const float skip = a.D_skip ? a.D_skip[d] : 0.f;
  const int64_t row0 = k.b * a.L;
  const T* up = static_cast<const T*>(a.u) + row0 * a.rows.u + d;
  const T* dp = static_cast<const T*>(a.dt) + row0 * a.rows.dt + d;
  const T* zp = a.z ? static_cast<const T*>(a.z) + row0 * a.rows.z + d : nullptr;
  const T* Bp = static_cast<const T*>(a.Bm) + row0 * a.rows.b + k.grp * N;
  const T* Cp = static_cast<const T*>(a.Cm) + row0 * a.rows.c + k.grp * N;
  const int* sq = PACKED ? a.seq_idx + row0 : nullptr;
  T* yp = FINAL ? static_cast<T*>(a.y) + row0 * a.D + d : nullptr;

  float sdt = 0.f;
  bool restarted = false;
  for (int64_t t0 = k.t0; t0 < k.t1; t0 += kScanT) {
    const int nt = (int)(k.t1 - t0 < kScanT ? k.t1 - t0 : kScanT);
    float dt[kScanT], x[kScanT], y[kScanT];
    uint32_t starts = 0;  // bit i: token t0 + i begins another sequence
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      const int64_t t = t0 + (i < nt ? i : nt - 1);
      const float u = IO::get(up[t * a.rows.u]);
      const float raw = IO::get(dp[t * a.rows.dt]) + bias;
      const float v = a.softplus ? softplus(raw) : raw;
      dt[i] = i < nt ? v : 0.f;          // tokens past the chunk: decay 1, input 0
      x[i] = i < nt ? v * u : 0.f;
      if (FINAL) y[i] = skip * u;
      if (PACKED && i < nt && t > 0 && sq[t] != sq[t - 1]) starts |= 1u << i;
    }
    if (!FINAL) {
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        sdt = (PACKED && (starts >> i & 1)) ? dt[i] : sdt + dt[i];
      }
      if (PACKED) restarted = restarted || starts != 0;
    }
    for (int n0 = 0; n0 < N; n0 += 4) {
      const float4 av = *reinterpret_cast<const float4*>(a.A + d * N + n0);
      const float a2[4] = {av.x * kLog2e, av.y * kLog2e, av.z * kLog2e, av.w * kLog2e};
      float h[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) h[s] = hs[(n0 + s) * 64 + lane];
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        const int64_t t = t0 + (i < nt ? i : nt - 1);
        float bv[4], cv[4];
        uniform4<IO>(Bp + t * a.rows.b + n0, bv);
        if (FINAL) uniform4<IO>(Cp + t * a.rows.c + n0, cv);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float dec = fast_exp2(dt[i] * a2[s]);
          const float hp = (PACKED && (starts >> i & 1)) ? 0.f : h[s];
          h[s] = fmaf(dec, hp, x[i] * bv[s]);
          if (FINAL) y[i] = fmaf(cv[s], h[s], y[i]);
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) hs[(n0 + s) * 64 + lane] = h[s];
    }
    if (FINAL) {
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        if (i < nt) {
          float o = y[i];
          if (zp) {
            const float z = IO::get(zp[(t0 + i) * a.rows.z]);
            o *= z * sigmoid(z);
          }
          if (ok) yp[(t0 + i) * a.D] = IO::put(o);
        }
      }
    }
  }
  if (FINAL) {
    if (k.c == g.nc - 1 && a.hfin && ok)
      for (int n = 0; n < N; ++n) a.hfin[(k.b * N + n) * a.D + d] = hs[n * 64 + lane];
  } else if (ok) {
    float* o = ws.carry + (k.b * g.nc + k.c) * N * a.D + d;
    for (int n = 0; n < N; ++n) o[(int64_t)n * a.D] = hs[n * 64 + lane];
    ws.sdt[(k.b * g.nc + k.c) * a.D + d] = sdt;
    if (PACKED && lane == 0 && k.d0 == 0) ws.cut[k.b * g.nc + k.c] = restarted;
  }
}

// Carry: from the states the chunks leave (slot c) to the states entering them
// (in place; slot 0, whose state is the initial one, is not rewritten).
template <bool PACKED>
__global__ __launch_bounds__(256) void scan_carry_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= a.B * a.N * a.D) return;
  const int64_t d = idx % a.D, n = idx / a.D % a.N, b = idx / a.D / a.N;
  const float a2 = a.A[d * a.N + n] * kLog2e;
  float* s = ws.carry + (b * g.nc * a.N + n) * a.D + d;
  const float* sd = ws.sdt + b * g.nc * a.D + d;
  const int64_t cs = a.N * a.D;
  float run = s[0];
  constexpr int U = 8;
  for (int64_t c0 = 1; c0 < g.nc; c0 += U) {
    float v[U], p[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + i < g.nc - 1 ? c0 + i : g.nc - 2;  // the last chunk left no state
      v[i] = c > 0 ? s[c * cs] : 0.f;
      p[i] = fast_exp2(sd[c * a.D] * a2);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + i;
      if (c < g.nc) {
        s[c * cs] = run;
        if (PACKED && c < g.nc - 1 && ws.cut[b * g.nc + c]) run = v[i];
        else run = fmaf(p[i], run, v[i]);
      }
    }
  }
}

// States after given tokens: from the state entering the token's chunk.
template <class IO>
__global__ __launch_bounds__(64) void scan_seq_states_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  typedef typename IO::type T;
  const int lane = threadIdx.x;
  const int64_t s = blockIdx.z;
  const int64_t tok = a.seq_last[s];
  if (tok < 0 || tok >= a.B * a.L) return;
  const int64_t b = tok / a.L, t = tok % a.L;
  const int64_t c = t / g.Q, gd = a.D / a.G;
  const int64_t grp = blockIdx.x / g.ncb;
  const int64_t d = grp * gd + (blockIdx.x % g.ncb) * 64 + lane;
  if (d >= (grp + 1) * gd) return;
  const int n = blockIdx.y;
  const int N = (int)a.N;
  const float a2 = a.A[d * N + n] * kLog2e;
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
  const float* h_in = c > 0 ? ws.carry + (b * g.nc + c) * N * a.D : (a.h0 ? a.h0 + b * N * a.D : nullptr);
  float h = h_in ? h_in[(int64_t)n * a.D + d] : 0.f;
  const int64_t row0 = b * a.L;
  const T* up = static_cast<const T*>(a.u) + row0 * a.rows.u + d;
  const T* dp = static_cast<const T*>(a.dt) + row0 * a.rows.dt + d;
  const T* Bp = static_cast<const T*>(a.Bm) + row0 * a.rows.b + grp * N + n;
  for (int64_t j = c * g.Q; j <= t; ++j) {
    const float raw = IO::get(dp[j * a.rows.dt]) + bias;
    const float dt = a.softplus ? softplus(raw) : raw;
    if (a.seq_idx && j > 0 && a.seq_idx[row0 + j] != a.seq_idx[row0 + j - 1]) h = 0.f;
    h = fmaf(fast_exp2(dt * a2), h, dt * IO::get(up[j * a.rows.u]) * IO::get(Bp[j * a.rows.b]));
  }
  a.seq_states[(s * N + n) * a.D + d] = h;
}

// Single-token step.  A lane takes one channel and all its states; the states
// (8 bytes each, read and written) bound it.
template <class IO>
__global__ __launch_bounds__(64) void scan_step_kernel(ScanArgs a, const float* state, float* state_out) {
  typedef typename IO::type T;
  const int64_t gd = a.D / a.G, ncb = (gd + 63) / 64;
  const int64_t grp = blockIdx.x / ncb;
  const int64_t d = grp * gd + (blockIdx.x % ncb) * 64 + threadIdx.x;
  const int64_t b = blockIdx.y;
  if (d >= (grp + 1) * gd) return;
  const int N = (int)a.N;
  const float u = IO::get(static_cast<const T*>(a.u)[b * a.rows.u + d]);
  const float raw = IO::get(static_cast<const T*>(a.dt)[b * a.rows.dt + d]) + (a.dt_bias ? a.dt_bias[d] : 0.f);
  const float dt = a.softplus ? softplus(raw) : raw;
  const float x = dt * u;
  const T* Bp = static_cast<const T*>(a.Bm) + b * a.rows.b + grp * N;
  const T* Cp = static_cast<const T*>(a.Cm) + b * a.rows.c + grp * N;
  const float* st = state + b * N * a.D + d;
  float* so = state_out + b * N * a.D + d;
  float y = a.D_skip ? a.D_skip[d] * u : 0.f;
  for (int n0 = 0; n0 < N; n0 += 4) {
    float bv[4], cv[4], h[4], av[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      h[s] = st[(int64_t)(n0 + s) * a.D];
      av[s] = a.A[d * N + n0 + s];
    }
    uniform4<IO>(Bp + n0, bv);
    uniform4<IO>(Cp + n0, cv);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      h[s] = fmaf(fast_exp2(dt * (av[s] * kLog2e)), h[s], x * bv[s]);
      y = fmaf(cv[s], h[s], y);
      so[(int64_t)(n0 + s) * a.D] = h[s];
    }
  }
  if (a.z) {
    const float z = IO::get(static_cast<const T*>(a.z)[b * a.rows.z + d]);
    y *= z * sigmoid(z);
  }
  static_cast<T*>(a.y)[b * a.D + d] = IO::put(y);
}

bool scan_dstate_supported(int64_t N) { return N > 0 && N % 4 == 0 && N <= 256; }

// Chunk length: enough waves for four a SIMD, in whole 16-token steps; the
// carried states then cost little beside the inputs.
static ScanGrid forward_grid(int64_t B, int64_t L, int64_t D, int64_t G) {
  ScanGrid g;
  g.ncb = (D / G + 63) / 64;
  const int64_t waves = B * G * g.ncb, want = (int64_t)device_cu_count() * 16;
  int64_t nc = (want + waves - 1) / waves;
  const int64_t most = (L + 63) / 64;
  if (nc > most) nc = most;
  if (nc < 1) nc = 1;
  g.Q = ((L + nc - 1) / nc + kScanT - 1) / kScanT * kScanT;
  g.nc = (L + g.Q - 1) / g.Q;
  return g;
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t scan_forward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanGrid g = forward_grid(B, L, D, G);
  if (g.nc == 1) return 0;
  return up256(sizeof(float) * B * g.nc * N * D) + up256(sizeof(float) * B * g.nc * D) +
         up256(sizeof(int) * B * g.nc);
}

template <class IO, bool PACKED>
static hipError_t scan_forward_t(const ScanArgs& a, hipStream_t s) {
  const ScanGrid g = forward_grid(a.B, a.L, a.D, a.G);
  ScanWs ws = {};
  char* base = static_cast<char*>(a.ws);
  ws.carry = reinterpret_cast<float*>(base);
  ws.sdt = reinterpret_cast<float*>(base + up256(sizeof(float) * a.B * g.nc * a.N * a.D));
  ws.cut = reinterpret_cast<int*>(reinterpret_cast<char*>(ws.sdt) + up256(sizeof(float) * a.B * g.nc * a.D));
  const size_t lds = 64 * sizeof(float) * a.N;  // 64 KB at N = 256
  hipError_t e;
  if (g.nc > 1) {
    const dim3 grid((unsigned)(a.G * g.ncb), (unsigned)(g.nc - 1), (unsigned)a.B);
    hipLaunchKernelGGL((scan_chunk_kernel<IO, PACKED, false>), grid, dim3(64), lds, s, a, g, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((scan_carry_kernel<PACKED>), dim3((unsigned)((a.B * a.N * a.D + 255) / 256)), dim3(256), 0, s, a,
                       g, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_chunk_kernel<IO, PACKED, true>),
                     dim3((unsigned)(a.G * g.ncb), (unsigned)g.nc, (unsigned)a.B), dim3(64), lds, s, a, g, ws);
  if ((e = hipGetLastError()) != hipSuccess || a.nseq == 0) return e;
  hipLaunchKernelGGL((scan_seq_states_kernel<IO>), dim3((unsigned)(a.G * g.ncb), (unsigned)a.N, (unsigned)a.nseq),
                     dim3(64), 0, s, a, g, ws);
  return hipGetLastError();
}

hipError_t launch_scan_forward(const ScanArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.seq_idx ? scan_forward_t<IoBF16, true>(a, s) : scan_forward_t<IoBF16, false>(a, s);
  return a.seq_idx ? scan_forward_t<IoF32, true>(a, s) : scan_forward_t<IoF32, false>(a, s);
}

hipError_t launch_scan_step(const ScanArgs& a, const float* state, float* state_out, bool bf16, hipStream_t s) {
  const int64_t ncb = (a.D / a.G + 63) / 64;
  const dim3 grid((unsigned)(a.G * ncb), (unsigned)a.B);
  if (bf16) hipLaunchKernelGGL((scan_step_kernel<IoBF16>), grid, dim3(64), 0, s, a, state, state_out);
  else hipLaunchKernelGGL((scan_step_kernel<IoF32>), grid, dim3(64), 0, s, a, state, state_out);
  return hipGetLastError();
}

}  // namespace ssd
