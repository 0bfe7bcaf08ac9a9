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
// in LDS, one at a time in a register over 16 tokens whose time steps, inputs
// and outputs stay in registers.  B and C come as scalar operands.
// Where channels alone leave compute units idle the tokens are split: a first
// pass takes every chunk's state from zero, a second carries the states from
// chunk to chunk (decays multiply as exp of the summed dt), and the last
// computes the outputs from the carried states.  2 x 8192 tokens of 5120
// channels and 16 states, bf16, gated: 491 us, of which the two passes' instructions come to
// 461 at the rates measured for them; 65536 tokens of 1024 channels: 418.
#include "layer_device.hpp"
#include "layer_launch.hpp"
#include "selective_scan.hpp"

namespace ssd {

// Packs B ln 2 and C to [B,G,tile,N][kEntry] in fp32 (tokens past the row:
// zero), A to [N,D], and the sequence starts to a bit a token.  Small beside
// the scan (2 G N of each token's elements against 3 D or more), it spares the
// inner loops the address arithmetic and the widening of scalars.
// A block turns one tile of one group through LDS, so that reads go along the
// states and writes along the entries; the blocks after those take A and the
// starts.
template <class IO>
__global__ __launch_bounds__(256) void scan_pack_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  typedef typename IO::type T;
  extern __shared__ float turn[];  // [N][kEntry + 1]
  const int N = (int)a.N;
  const int64_t tiles = a.B * a.G * g.ntile;
  const int64_t block = flat_block();
  if (block < tiles) {
    const int64_t bg = block / g.ntile, tile = block - bg * g.ntile;
    const int64_t b = bg / a.G, grp = bg - b * a.G;
    for (int e = threadIdx.x; e < kEntry * N; e += 256) {
      const int isC = e / (kScanT * N), r = e - isC * kScanT * N, tok = r / N, n = r - tok * N;
      const int64_t t = tile * kScanT + tok, row = b * a.L + t;
      float v = 0.f;
      if (t < a.L)
        v = isC ? IO::get(static_cast<const T*>(a.Cm)[row * a.rows.c + grp * N + n])
                : IO::get(static_cast<const T*>(a.Bm)[row * a.rows.b + grp * N + n]) * kLn2;
      turn[n * (kEntry + 1) + tok / kHalf * kScanT + isC * kHalf + tok % kHalf] = v;
    }
    __syncthreads();
    float* o = ws.bc + block * N * kEntry;
    for (int e = threadIdx.x; e < kEntry * N; e += 256) o[e] = turn[e / kEntry * (kEntry + 1) + e % kEntry];
    return;
  }
  const int64_t k = (block - tiles) * 256 + threadIdx.x, na = N * a.D;
  if (k < na) {
    ws.at[k] = a.A[k % a.D * N + k / a.D];
  } else if (ws.starts && k - na < a.B * g.ntile) {
    const int64_t q = k - na, b = q / g.ntile, t0 = q % g.ntile * kScanT;
    const int* sq = a.seq_idx + b * a.L;
    uint32_t m = 0;
    for (int e = 0; e < kScanT; ++e) {
      const int64_t t = t0 + e;
      if (t > 0 && t < a.L && sq[t] != sq[t - 1]) m |= 1u << e;
    }
    ws.starts[q] = m;
  }
}

hipError_t launch_scan_pack(const ScanArgs& a, const ScanGrid& g, const ScanWs& ws, bool bf16, hipStream_t s) {
  const int64_t rest = a.N * a.D + (ws.starts ? a.B * g.ntile : 0);
  const dim3 grid = flat_grid(a.B * a.G * g.ntile + (rest + 255) / 256);
  const size_t lds = sizeof(float) * a.N * (kEntry + 1);
  if (bf16) hipLaunchKernelGGL((scan_pack_kernel<IoBF16>), grid, dim3(256), lds, s, a, g, ws);
  else hipLaunchKernelGGL((scan_pack_kernel<IoF32>), grid, dim3(256), lds, s, a, g, ws);
  return hipGetLastError();
}

// State passes: FINAL writes outputs from the chunk's entering state, else
// only the state the chunk leaves and its summed dt.  Four waves a SIMD, which
// the compiler would give up for a register (164 of them: 563 -> 593 us); the
// packed last pass spills 9 registers for them (fp32 12).
template <class IO, bool PACKED, bool FINAL>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(4, 4))) void scan_chunk_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  typedef typename IO::type T;
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  const ScanBlock k = scan_block(g, a);
  const int N = (int)a.N;
  float* hs = lds + lane;   // hs[n*64]: state
  float* as = hs + N * 64;  // as[n*64]: A
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;

  const float* h_in = nullptr;
  if (FINAL && g.nc > 1) h_in = ws.carry + (k.b * g.nc + k.c) * N * a.D;
  if (k.c == 0) h_in = a.h0 ? a.h0 + k.b * N * a.D : nullptr;
  const float* ep = ws.bc + (((k.b * a.G + k.grp) * g.ntile + k.t0 / kScanT) * N) * kEntry;
  Touch ahead;
  ahead.entries(ep, N, lane);
  if (h_in) {
    rows_to_lds(hs, h_in + d, a.D, N);
  } else {
    for (int n = 0; n < N; ++n) hs[n * 64] = 0.f;
  }
  rows_to_lds(as, ws.at + d, a.D, N);
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const float skip = a.D_skip ? a.D_skip[d] : 0.f;
  const int64_t row0 = k.b * a.L;
  const int off = (int)((d - k.d0) * sizeof(T));
  const T* up = static_cast<const T*>(a.u) + row0 * a.rows.u + k.d0;
  const T* dp = static_cast<const T*>(a.dt) + row0 * a.rows.dt + k.d0;
  const T* zp = a.z ? static_cast<const T*>(a.z) + row0 * a.rows.z + k.d0 : nullptr;
  T* yp = FINAL ? static_cast<T*>(a.y) + row0 * a.D + k.d0 : nullptr;
  BCPair<FINAL> cur;
  cur.load(ep);
  float a_n = as[0], h_n = hs[0];
  RawTile<IO> ru, rd, rz;
  ru.load(up, a.rows.u, k.t0, tile_tokens(k, k.t0), off);
  rd.load(dp, a.rows.dt, k.t0, tile_tokens(k, k.t0), off);

  float sdt = 0.f;
  bool restarted = false;
  for (int64_t t0 = k.t0; t0 < k.t1; t0 += kScanT) {
    pace(t0 - k.t0, k.t1 - k.t0);
    const int nt = tile_tokens(k, t0);
    const uint32_t starts = PACKED ? ws.starts[k.b * g.ntile + t0 / kScanT] : 0;
    float dt[kScanT], x[kScanT], y[kScanT];
    time_steps(rd, bias, a.softplus, nt, dt);
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      x[i] = dt[i] * ru.at(i);
      if (FINAL) y[i] = skip * ru.at(i);
    }
    if (nt < kScanT) {  // past the row u is the last token's, which may be anything
#pragma unroll
      for (int i = 0; i < kScanT; ++i)
        if (i >= nt) x[i] = 0.f;
    }
    // the gate of this tile and the next tile's inputs arrive behind the states
    ahead.settle();
    ahead.entries(t0 + kScanT < k.t1 ? ep + N * kEntry : ep, N, lane);
    if (FINAL && zp) rz.load(zp, a.rows.z, t0, nt, off);
    if (t0 + kScanT < k.t1) {
      ru.load(up, a.rows.u, t0 + kScanT, tile_tokens(k, t0 + kScanT), off);
      rd.load(dp, a.rows.dt, t0 + kScanT, tile_tokens(k, t0 + kScanT), off);
    }
    if (!FINAL) {
#pragma unroll
      for (int i = 0; i < kScanT; ++i) sdt = (PACKED && (starts >> i & 1)) ? dt[i] : sdt + dt[i];
      if (PACKED) restarted = restarted || starts != 0;
    }
    if (PACKED && starts) {
      // the tiles in which a sequence starts, one state after the other: the
      // starts' selects would cost every tile a fifth of its arithmetic (4 x
      // 8192 tokens of 2048 channels, 9 sequences a row: 495 us, so 450)
      for (int n = 0; n < N; ++n) {
        cur.settle();
        float h = hs[n * 64];
        const float an = as[n * 64];
#pragma unroll
        for (int i = 0; i < kScanT; ++i) {
          const float dec = fast_exp2(dt[i] * an);
          h = (starts >> i & 1) ? 0.f : h;
          h = fmaf(dec, h, x[i] * cur.b(i));
          if (FINAL) y[i] = fmaf(cur.c(i), h, y[i]);
        }
        hs[n * 64] = h;
        ep += kEntry;
        cur.load(ep);
      }
      a_n = as[0];
      h_n = hs[0];
    } else {
      for (int n0 = 0; n0 < N; n0 += 4) {
        // the last one's successor is the next tile's first
        float* hq = hs + n0 * 64;
        const float* aq = as + n0 * 64;
        const int next = n0 + 4 < N ? 4 * 64 : -n0 * 64;
  #pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float an = a_n;
          float h = h_n;
          cur.settle();
          ep += kEntry;
          BCPair<FINAL> nxt;
          nxt.load(ep);
          a_n = s < 3 ? aq[(s + 1) * 64] : aq[next];
          if (s < 3) h_n = hq[(s + 1) * 64];
  #pragma unroll
          for (int i = 0; i < kScanT; ++i) {
            const float dec = fast_exp2(dt[i] * an);
            h = fmaf(dec, h, x[i] * cur.b(i));
            if (FINAL) y[i] = fmaf(cur.c(i), h, y[i]);
          }
          cur = nxt;
          hq[s * 64] = h;
          if (s == 3) h_n = hq[next];
        }
      }
    }
    if (FINAL) {
      if (zp) {
#pragma unroll
        for (int i = 0; i < kScanT; ++i) {
          const float z = rz.at(i);
          y[i] *= z * sigmoid(z);
        }
      }
      if (ok) store_tile<IO>(yp, a.D, t0, nt, off, y);
    }
  }
  if (FINAL) {
    if (k.c == g.nc - 1 && a.hfin && ok)
      for (int n = 0; n < N; ++n) a.hfin[(k.b * N + n) * a.D + d] = hs[n * 64];
  } else if (ok) {
    float* o = ws.carry + (k.b * g.nc + k.c) * N * a.D + d;
    for (int n = 0; n < N; ++n) o[(int64_t)n * a.D] = hs[n * 64];
    ws.sdt[(k.b * g.nc + k.c) * a.D + d] = sdt;
    if (PACKED && lane == 0 && k.d0 == 0) ws.cut[k.b * g.nc + k.c] = restarted;
  }
}

// Carry, in place.  Forward (z < B): from the states the chunks leave to the
// states entering them; chunk 0 leaves its full state (it started from the
// initial one) and what enters it is not used.  Backward (z >= B): from what
// each chunk sends back to the gradient reaching its last state, the last
// chunk's being dfinal.  One fused multiply-add a chunk, bound by the latency
// of the loads: the waves of a block take up to kCarryAhead chunks each, whose
// loads are in flight together, compose them, and then, with what the waves
// before let through, write their carries.  Longer stretches are walked twice,
// or once by one wave where the columns alone fill the chip.
// Lanes past D repeat its last column.  Pointers step from chunk to chunk: with
// a product of 64 bits an address the code outgrew the time it took to fetch.
constexpr int kCarryAhead = 16, kCarryWaves = 16;
template <bool PACKED>
__global__ __launch_bounds__(64 * kCarryWaves) void scan_carry_kernel(ScanArgs a, ScanGrid g, ScanWs ws, int part) {
  __shared__ float left[kCarryWaves][64], kept[kCarryWaves][64];
  const bool rev = blockIdx.z >= a.B;
  const int64_t b = rev ? blockIdx.z - a.B : blockIdx.z, n = blockIdx.y;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)(blockDim.x >> 6);
  int64_t d = (int64_t)blockIdx.x * 64 + lane;
  if (d >= a.D) d = a.D - 1;
  const float an = ws.at[n * a.D + d];
  // The chunks in walking order, from the first or back from the last; the last
  // one's slot takes what reaches it and is not read.
  const int steps = (int)g.nc - 1;
  const int q0 = wave * part < steps ? wave * part : steps, q1 = q0 + part < steps ? q0 + part : steps;
  const int64_t sign = rev ? -1 : 1, c0 = b * g.nc + (rev ? steps - q0 : q0);
  const int64_t cs = sign * a.N * a.D, ds = sign * a.D;
  float* const s0 = (rev ? ws.adj : ws.carry) + (c0 * a.N + n) * a.D + d;
  const float* const sd0 = ws.sdt + c0 * a.D + d;
  const int* const cut0 = ws.cut + c0;
  float v[kCarryAhead], p[kCarryAhead];
  uint32_t cuts = 0;  // bit i: a sequence starts in chunk i, nothing that enters leaves it
  auto load = [&](int q) {  // past q1: nothing added, nothing decays
    const float *s = s0 + (q - q0) * cs, *sd = sd0 + (q - q0) * ds;
    const int* cut = cut0 + (q - q0) * sign;
    cuts = 0;
#pragma unroll
    for (int i = 0; i < kCarryAhead; ++i) {
      v[i] = *s;
      p[i] = *sd;
      const bool more = q + i + 1 < q1;
      if (PACKED) {
        cuts |= (*cut != 0 ? 1u : 0u) << i;
        cut += more ? sign : 0;
      }
      s += more ? cs : 0;
      sd += more ? ds : 0;
    }
#pragma unroll
    for (int i = 0; i < kCarryAhead; ++i) {
      if (q + i >= q1) v[i] = p[i] = 0.f;
    }
    if (!rev && q == 0) p[0] = 0.f;  // chunk 0 leaves its full state
    if (PACKED && q1 - q < kCarryAhead) cuts &= (1u << (q1 - q)) - 1;
  };
  auto after = [&](float run, int i) {
    const float r = fmaf(fast_exp2(p[i] * an), run, v[i]);
    return PACKED && (cuts >> i & 1) ? v[i] : r;
  };
  const float first = rev && wave == 0 && a.dfinal ? a.dfinal[(b * a.N + n) * a.D + d] : 0.f;
  const bool held = part <= kCarryAhead;  // this wave's chunks stay in registers
  float run = first;
  if (held) load(q0);
  if (waves > 1) {
    float sum = 0.f;  // time steps of the stretch
    uint32_t any = 0;
    for (int q = q0; q < q1; q += kCarryAhead) {
      if (!held) load(q);
#pragma unroll
      for (int i = 0; i < kCarryAhead; ++i) {
        // (a stretch starts from nothing: not even an overflowing decay of it)
        run = i == 0 && q == q0 && wave > 0 ? v[0] : after(run, i);
        sum += p[i];
      }
      any |= cuts;
    }
    left[wave][lane] = run;
    kept[wave][lane] = any ? -1.f : fast_exp2(sum * an);  // -1: nothing gets through
    __syncthreads();
    run = wave == 0 ? first : left[0][lane];
    for (int w = 1; w < wave; ++w) {
      const float k = kept[w][lane], l = left[w][lane];
      run = k < 0.f || run == 0.f ? l : fmaf(k, run, l);
    }
  }
  float* s = s0;
  for (int q = q0; q < q1; q += kCarryAhead) {
    if (!held) load(q);
#pragma unroll
    for (int i = 0; i < kCarryAhead; ++i) {
      if (q + i < q1) {
        *s = run;
        s += cs;
        run = after(run, i);
      }
    }
  }
  if (wave == waves - 1) *s = run;
}

hipError_t launch_scan_carry(const ScanArgs& a, const ScanGrid& g, const ScanWs& ws, hipStream_t s) {
  const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)a.N, (unsigned)(ws.adj ? 2 * a.B : a.B));
  const int64_t blocks = (int64_t)grid.x * grid.y * grid.z;
  const int steps = (int)g.nc - 1;
  int waves = (steps + kCarryAhead - 1) / kCarryAhead;
  if (waves > kCarryWaves) waves = blocks < (int64_t)device_cu_count() * 8 ? kCarryWaves : 1;
  if (waves < 1) waves = 1;
  auto kern = ws.starts ? scan_carry_kernel<true> : scan_carry_kernel<false>;
  hipLaunchKernelGGL(kern, grid, dim3((unsigned)(64 * waves)), 0, s, a, g, ws, (steps + waves - 1) / waves);
  return hipGetLastError();
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
  const float an = a.A[d * N + n];
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const float* h_in = c > 0 ? ws.carry + (b * g.nc + c) * N * a.D : (a.h0 ? a.h0 + b * N * a.D : nullptr);
  float h = h_in ? h_in[(int64_t)n * a.D + d] : 0.f;
  const int64_t row0 = b * a.L;
  const T* up = static_cast<const T*>(a.u) + row0 * a.rows.u + d;
  const T* dp = static_cast<const T*>(a.dt) + row0 * a.rows.dt + d;
  const T* Bp = static_cast<const T*>(a.Bm) + row0 * a.rows.b + grp * N + n;
  for (int64_t j = c * g.Q; j <= t; ++j) {
    const float raw = fmaf(IO::get(dp[j * a.rows.dt]), kLog2e, bias);
    const float dt = a.softplus ? softplus2(raw) : raw;
    if (a.seq_idx && j > 0 && a.seq_idx[row0 + j] != a.seq_idx[row0 + j - 1]) h = 0.f;
    h = fmaf(fast_exp2(dt * an), h, dt * IO::get(up[j * a.rows.u]) * (IO::get(Bp[j * a.rows.b]) * kLn2));
  }
  a.seq_states[(s * N + n) * a.D + d] = h;
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

// Single-token step.  A lane takes one channel and all its states; the states
// (8 bytes each, read and written) bound it: 64 x 5120 channels of 16 states in
// 10.5 us, 4.3 TB/s.
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
  const float raw = (IO::get(static_cast<const T*>(a.dt)[b * a.rows.dt + d]) + (a.dt_bias ? a.dt_bias[d] : 0.f)) * kLog2e;
  const float dt = a.softplus ? softplus2(raw) : raw;  // in units of ln 2
  const float x = dt * u * kLn2;
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
      h[s] = fmaf(fast_exp2(dt * av[s]), h[s], x * bv[s]);
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

// Chunk length: enough waves for four a SIMD, in whole 16-token tiles; the
// carried states then cost little beside the inputs.  Short problems go down to
// a tile a chunk (1 x 512 tokens of 1536 channels: chunks of 64 tokens 57 us,
// 32 39, 16 30), but rows of up to three tiles stay whole: two passes and a
// carry take as long as three tiles in one.
static ScanGrid forward_grid(int64_t B, int64_t L, int64_t D, int64_t G) {
  ScanGrid g;
  g.ncb = (D / G + 63) / 64;
  const int64_t waves = B * G * g.ncb, want = (int64_t)device_cu_count() * 16;
  int64_t nc = want / waves;  // rounded down: one wave too many would run in a round of its own
  const int64_t most = L <= 3 * kScanT ? 1 : (L + kScanT - 1) / kScanT;
  if (nc > most) nc = most;
  if (nc < 1) nc = 1;
  g.Q = ((L + nc - 1) / nc + kScanT - 1) / kScanT * kScanT;
  g.nc = (L + g.Q - 1) / g.Q;
  g.ntile = (L + kScanT - 1) / kScanT;
  return g;
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct FwdLayout {
  size_t carry, sdt, cut, bc, at, starts, total;
};
static FwdLayout forward_layout(const ScanGrid& g, int64_t B, int64_t D, int64_t N, int64_t G) {
  FwdLayout w;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t r = o; o += up256(bytes); return r; };
  const int64_t nc = g.nc > 1 ? g.nc : 0;  // nothing is carried inside one chunk
  w.carry = take(sizeof(float) * B * nc * N * D);
  w.sdt = take(sizeof(float) * B * nc * D);
  w.cut = take(sizeof(int) * B * nc);
  w.bc = take(sizeof(float) * scan_bc_floats(B, G, g.ntile, N));
  w.at = take(sizeof(float) * N * D);
  w.starts = take(sizeof(uint32_t) * B * g.ntile);
  w.total = o;
  return w;
}
size_t scan_forward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  return forward_layout(forward_grid(B, L, D, G), B, D, N, G).total;
}

template <class IO, bool PACKED>
static hipError_t scan_forward_t(const ScanArgs& a, hipStream_t s) {
  const ScanGrid g = forward_grid(a.B, a.L, a.D, a.G);
  const FwdLayout w = forward_layout(g, a.B, a.D, a.N, a.G);
  char* base = static_cast<char*>(a.ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const ScanWs ws = {at(w.carry), at(w.sdt), reinterpret_cast<int*>(base + w.cut), nullptr, at(w.bc), at(w.at),
                     PACKED ? reinterpret_cast<uint32_t*>(base + w.starts) : nullptr, nullptr, nullptr};
  const size_t lds = 2 * 64 * sizeof(float) * a.N;
  hipError_t e = launch_scan_pack(a, g, ws, IO::kVec == 8, s);
  if (e != hipSuccess) return e;
  if (lds > 64 * 1024) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_chunk_kernel<IO, PACKED, false>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_chunk_kernel<IO, PACKED, true>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  if (g.nc > 1) {
    const dim3 grid((unsigned)(a.G * g.ncb), (unsigned)(g.nc - 1), (unsigned)a.B);
    hipLaunchKernelGGL((scan_chunk_kernel<IO, PACKED, false>), grid, dim3(64), lds, s, a, g, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_scan_carry(a, g, ws, s)) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_chunk_kernel<IO, PACKED, true>),
                     dim3((unsigned)(a.G * g.ncb), (unsigned)g.nc, (unsigned)a.B), dim3(64), lds, s, a,
                     g, ws);
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
