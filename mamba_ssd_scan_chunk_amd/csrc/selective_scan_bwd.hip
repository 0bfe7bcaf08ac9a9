// selective_scan_bwd.hip -- gradients of the selective scan.
//
// With dy' = dy z sigmoid(z) (the gradient at y before the gate), the adjoint
// state runs back over the tokens,
//     g[t,n] = C[t,n] dy'[t] + a[t+1,n] g[t+1,n],      a[t,n] = exp(dt[t] A[n])
// and with q[t,n] = g[t,n] a[t,n] h[t-1,n], s[t] = sum_n g[t,n] B[t,n]:
//     du = dt s + D dy'      ddt = u s + sum_n A[n] q      draw = ddt sigmoid(raw)
//     dB[t,n] = sum_d g dt u     dC[t,n] = sum_d h dy'     (over the group's channels)
//     dA[n] = sum_t dt q     dD = sum_t u dy'      dz = dy y silu'(z)
//     dinitial[n] = a[0,n] g[0,n]
// A sequence start at t cuts both recurrences between t-1 and t.
//
// Three passes over chunks of tokens, a wave per (64 channels, chunk): the
// state each chunk leaves and the adjoint it sends back, each from zero; the
// carry of both over the chunks; then the chunk itself, whose states are
// recomputed forwards 16 tokens at a time (from the states the first pass left
// at every 16th token) and swept backwards.  The sums over channels go through
// LDS, 16 tokens of one state at a time; the channel blocks' partial sums are
// then added in order.  No atomics: results do not depend on timing.  2 x 2048
// tokens of 5120 channels and 16 states, bf16, gated: 425 us, 306 of them the
// third pass and 116 the first, bound by the vector ALUs.
#include "layer_device.hpp"
#include "layer_launch.hpp"
#include "selective_scan.hpp"

namespace ssd {

struct BwdWs {
  float* bc;     // [ncb][B L][G N] dB partial sums, then the same for dC
  float* dDb;    // [B nc][2][D] dD, then ddt_bias
};

// One row of the batch (b) of each input, from the wave's first channel on;
// lanes add their own.
template <class IO>
struct RowPtrs {
  typedef typename IO::type T;
  const T *u, *dt, *z, *dy;
  __device__ __forceinline__ RowPtrs(const ScanArgs& a, int64_t b, int64_t d0) {
    const int64_t r = b * a.L;
    u = static_cast<const T*>(a.u) + r * a.rows.u + d0;
    dt = static_cast<const T*>(a.dt) + r * a.rows.dt + d0;
    z = a.z ? static_cast<const T*>(a.z) + r * a.rows.z + d0 : nullptr;
    dy = static_cast<const T*>(a.dy) + r * a.D + d0;
  }
};

// dy z sigmoid(z), or dy
template <class IO>
__device__ __forceinline__ void gated(const RawTile<IO>& rg, const RawTile<IO>& rz, bool gate, float (&g)[kScanT]) {
#pragma unroll
  for (int i = 0; i < kScanT; ++i) g[i] = rg.at(i);
  if (gate) {
#pragma unroll
    for (int i = 0; i < kScanT; ++i) g[i] *= rz.at(i) * sigmoid(rz.at(i));
  }
}

// Pass 1: carry = the state the chunk leaves (chunk 0 from the initial state,
// others from zero), adj = what the chunk's outputs send back to its entering
// state, sdt = its summed dt.
template <class IO, bool PACKED>
__global__ __launch_bounds__(64) void scan_bwd_local_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  const ScanBlock k = scan_block(g, a);
  const int N = (int)a.N;
  float* hs = lds + lane;  // hs[n*64]: state
  float* gs = hs + N * 64;                       // gs[n*64]: what goes back to the entering state
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;
  const float* h_in = k.c == 0 && a.h0 ? a.h0 + k.b * N * a.D : nullptr;
  const float* ep = ws.bc + (((k.b * a.G + k.grp) * g.ntile + k.t0 / kScanT) * N) * kEntry;
  Touch ahead;
  ahead.entries(ep, N, lane);
  for (int n = 0; n < N; ++n) hs[n * 64] = gs[n * 64] = 0.f;
  if (h_in) rows_to_lds(hs, h_in + d, a.D, N);
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const RowPtrs<IO> p(a, k.b, k.d0);
  const int off = (int)((d - k.d0) * sizeof(typename IO::type));
  const float* atp = ws.at + d;
  BCPair<true> e;
  e.load(ep);
  float a_n = atp[0];
  float sdt = 0.f;        // since the chunk's start
  float last = 0.f;       // since its last restart
  bool cut = false;
  for (int64_t t0 = k.t0; t0 < k.t1; t0 += kScanT) {
    pace(t0 - k.t0, k.t1 - k.t0);
    const int nt = tile_tokens(k, t0);
    float dt[kScanT], x[kScanT], dy[kScanT];
    const uint32_t starts = PACKED ? ws.starts[k.b * g.ntile + t0 / kScanT] : 0;
    RawTile<IO> ru, rd, rg, rz;
    rd.load(p.dt, a.rows.dt, t0, nt, off);
    ru.load(p.u, a.rows.u, t0, nt, off);
    rg.load(p.dy, a.D, t0, nt, off);
    if (p.z) rz.load(p.z, a.rows.z, t0, nt, off);
    time_steps(rd, bias, a.softplus, nt, dt);
    gated(rg, rz, p.z, dy);
#pragma unroll
    for (int i = 0; i < kScanT; ++i) x[i] = dt[i] * ru.at(i);
    if (nt < kScanT) {  // past the row: decay 1, nothing added
#pragma unroll
      for (int i = 0; i < kScanT; ++i)
        if (i >= nt) x[i] = dy[i] = 0.f;
    }
    // tokens of this step that still reach the chunk's entering state
    const int live = cut ? 0 : (starts ? __builtin_ctz(starts) : kScanT);
    const float sdt0 = PACKED && cut ? 0.f : sdt;  // behind a start r is zero, but time steps may be anything
    // The state entering the next tile.  Stored always, from every lane (a lane
    // past the group repeats its last channel, value and all): behind a
    // condition the next state's load would wait for the store too.  What
    // enters the next chunk is not read back; the row after the last tile need
    // only be there.
    const int64_t next = k.b * g.ntile + t0 / kScanT + 1;
    float* ts = ws.tstate + next * N * a.D + d;
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      last = (PACKED && (starts >> i & 1)) ? dt[i] : last + dt[i];
      sdt += dt[i];
    }
    ahead.settle();
    ahead.entries(t0 + kScanT < k.t1 ? ep + N * kEntry : ep, N, lane);
    for (int n = 0; n < N; ++n) {
      const float an = a_n;
      e.settle();
      ep += kEntry;
      BCPair<true> nxt;
      nxt.load(ep);
      a_n = atp[(int64_t)(n + 1 < N ? n + 1 : 0) * a.D];
      float h = hs[n * 64];
      float dec[kScanT];
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        dec[i] = fast_exp2(dt[i] * an);
        if (PACKED && (starts >> i & 1)) h = 0.f;
        h = fmaf(dec[i], h, x[i] * e.b(i));
      }
      // what the tile's live tokens send back to the state entering it
      float r = 0.f;
#pragma unroll
      for (int i = kScanT - 1; i >= 0; --i) {
        const float v = fmaf(e.c(i), dy[i], r) * dec[i];
        r = (!PACKED || i < live) ? v : 0.f;
      }
      e = nxt;
      hs[n * 64] = h;
      gs[n * 64] = fmaf(fast_exp2(sdt0 * an), r, gs[n * 64]);
      ts[(int64_t)n * a.D] = h;
    }
    cut = cut || starts != 0;
    ws.tsdt[next * a.D + d] = last;
  }
  if (ok) {
    const int64_t o = (k.b * g.nc + k.c) * N * a.D + d;
    for (int n = 0; n < N; ++n) {
      ws.carry[o + (int64_t)n * a.D] = hs[n * 64];
      ws.adj[o + (int64_t)n * a.D] = gs[n * 64];
    }
    ws.sdt[(k.b * g.nc + k.c) * a.D + d] = last;
    if (PACKED && lane == 0 && k.d0 == 0) ws.cut[k.b * g.nc + k.c] = cut;
  }
}

// Pass 2 is the carry of both, shared with the forward.

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// Sum over the 64 lanes of 16 values a lane, through LDS: red[t*kRedRow + lane]
// holds them; lane l sums token l >> 2 over the 16 lanes of its quarter l & 3,
// and the four quarters meet by data-parallel moves: the whole sum of token
// l >> 2 in each of its four lanes.  (Halving the values with each lane bit in
// registers instead took 45 issue slots a state against 18.)
constexpr int kRedRow = 68;  // rows of 64 lanes shifted by four banks each
__device__ __forceinline__ float lane_sums(const float* red, int lane) {
  const float4* p = reinterpret_cast<const float4*>(red + (lane >> 2) * kRedRow + (lane & 3) * 16);
  float4 v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = p[e];
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s += (v[e].x + v[e].y) + (v[e].z + v[e].w);
  s += dpp_mov<0x4E>(s);
  s += dpp_mov<0xB1>(s);
  return s;
}

// Pass 3, two waves a SIMD: six values a token in registers beside the state's
// own leave no room for a third (forced to three the compiler spills: 792 us;
// tiles of 8 tokens at three waves read and write twice the states and take as
// long over most shapes).  306 us at 2 x 2048 tokens of 5120 channels and 16
// states, the vector ALUs busy for 72% of it.  LDS of a wave: the adjoint
// riding backwards and the summed dA, per state and lane, and the values being
// summed over lanes, dC's beside dB's: one wait for both sums, behind the sweep.
template <class IO, bool PACKED>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(2, 2))) void scan_bwd_chunk_kernel(ScanArgs a, ScanGrid g, ScanWs ws, BwdWs bw) {
  typedef typename IO::type T;
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  const ScanBlock k = scan_block(g, a);
  const int N = (int)a.N;
  float* red = lds;
  float* redc = red + kScanT * kRedRow;
  float* gs = lds + 2 * kScanT * kRedRow + lane;  // gs[n*64]
  float* as = gs + N * 64;                    // dA
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;
  const int64_t co = (k.b * g.nc + k.c) * N * a.D + d;  // this chunk's slot
  // the state entering the chunk; with none, any readable row times zero
  const float* h_in = k.c == 0 ? (a.h0 ? a.h0 + k.b * N * a.D + d : nullptr) : ws.carry + co;
  const bool entered = h_in != nullptr;
  if (!entered) h_in = ws.carry + co;
  const int nstep = (int)((k.t1 - k.t0 + kScanT - 1) / kScanT);
  const float* e0 = ws.bc + (((k.b * a.G + k.grp) * g.ntile + k.t0 / kScanT) * N) * kEntry;
  Touch ahead;
  ahead.entries(e0 + (int64_t)(nstep - 1) * N * kEntry, N, lane);
  rows_to_lds(gs, ws.adj + co, a.D, N);
  for (int n = 0; n < N; ++n) as[n * 64] = 0.f;
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const float skip = a.D_skip ? a.D_skip[d] : 0.f;
  const RowPtrs<IO> p(a, k.b, k.d0);
  const int off = (int)((d - k.d0) * sizeof(typename IO::type));
  const float* atp = ws.at + d;
  const bool whole = k.d0 + 64 <= k.dend;
  float dDsum = 0.f, dbsum = 0.f;
  const int64_t BL = a.B * a.L;
  const int64_t GN = a.G * N;
  float* dBp = bw.bc + (k.cb * BL + k.b * a.L) * GN + k.grp * N;
  float* dCp = dBp + g.ncb * BL * GN;
  for (int j = nstep - 1; j >= 0; --j) {
    pace(nstep - 1 - j, nstep);
    const int64_t t0 = k.t0 + j * kScanT, tile = k.b * g.ntile + t0 / kScanT;
    const int nt = tile_tokens(k, t0);
    float dt[kScanT], x[kScanT], gy[kScanT], y[kScanT], sB[kScanT], sA[kScanT];
    const uint32_t starts = PACKED ? ws.starts[tile] : 0;
    // what reaches this tile of the chunk's entering state
    bool reached = entered && (j == 0 || k.c > 0);  // chunk 0 started from the initial state
    if (PACKED) {
      for (int q = 0; q < j; ++q) reached = reached && ws.starts[tile - j + q] == 0;
    }
    const float tsd = j ? ws.tsdt[tile * a.D + d] : 0.f;
    const float* ts = ws.tstate + tile * N * a.D + d;
    {
      RawTile<IO> ru, rd, rg, rz;
      rd.load(p.dt, a.rows.dt, t0, nt, off);
      ru.load(p.u, a.rows.u, t0, nt, off);
      rg.load(p.dy, a.D, t0, nt, off);
      if (p.z) rz.load(p.z, a.rows.z, t0, nt, off);
      time_steps(rd, bias, a.softplus, nt, dt);
      gated(rg, rz, p.z, gy);
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        x[i] = dt[i] * ru.at(i);
        y[i] = skip * ru.at(i);
        sB[i] = 0.f;
        sA[i] = 0.f;
      }
      if (nt < kScanT) {
#pragma unroll
        for (int i = 0; i < kScanT; ++i)
          if (i >= nt) x[i] = gy[i] = 0.f;
      }
      if (!whole) {  // lanes past the group add nothing to its sums
#pragma unroll
        for (int i = 0; i < kScanT; ++i) {
          x[i] = ok ? x[i] : 0.f;
          gy[i] = ok ? gy[i] : 0.f;
        }
      }
    }
    BCPair<true> e;
    const float* ep = e0 + (int64_t)j * N * kEntry;
    e.load(ep);
    ahead.settle();
    ahead.entries(j ? ep - N * kEntry : ep, N, lane);
    float a_n = atp[0], in_n = h_in[0], ts_n = j ? ts[0] : 0.f;
    float rB = 0.f, rC = 0.f;  // of token lane >> 2, state lane & 3 of four
    for (int n = 0; n < N; ++n) {
      const float an = a_n;
      float h0 = ts_n;
      if (reached) h0 = fmaf(fast_exp2(tsd * an), in_n, h0);
      e.settle();
      {
        const int64_t nn = (int64_t)(n + 1 < N ? n + 1 : n) * a.D;
        a_n = atp[nn];
        in_n = h_in[nn];
        if (j) ts_n = ts[nn];
      }
      float dec[kScanT], h[kScanT];
      float hp = h0;
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        dec[i] = fast_exp2(dt[i] * an);
        if (PACKED && (starts >> i & 1)) hp = 0.f;
        hp = fmaf(dec[i], hp, x[i] * e.b(i));
        h[i] = hp;
        y[i] = fmaf(e.c(i), hp, y[i]);
        redc[i * kRedRow + lane] = hp * gy[i];
      }
      float ga = gs[n * 64], dA = as[n * 64];
#pragma unroll
      for (int i = kScanT - 1; i >= 0; --i) {
        const float gt = fmaf(e.c(i), gy[i], ga);
        red[i * kRedRow + lane] = gt * x[i];
        sB[i] = fmaf(gt, e.b(i), sB[i]);
        ga = gt * dec[i];
        float q = ga * (i ? h[i > 0 ? i - 1 : 0] : h0);
        if (PACKED && (starts >> i & 1)) {
          ga = 0.f;
          q = 0.f;
        }
        sA[i] = fmaf(an, q, sA[i]);
        dA = fmaf(dt[i], q, dA);
      }
      // summed here and now: put off past the branch below, the terms would
      // stay in registers beside the sums
#pragma unroll
      for (int i = 0; i < kScanT; ++i) asm volatile("" : "+v"(sA[i]), "+v"(sB[i]), "+v"(y[i]));
      asm volatile("" : "+v"(dA));
      // B and C are in use up to here; the next entry arrives behind the sums
      // (asked for earlier, the 64 scalar registers of two entries spill)
      ep += kEntry;
      e.load(ep);
      gs[n * 64] = ga;
      as[n * 64] = dA;
      __builtin_amdgcn_wave_barrier();
      const float sumB = lane_sums(red, lane), sumC = lane_sums(redc, lane);
      __builtin_amdgcn_wave_barrier();
      const bool mine = (n & 3) == (lane & 3);
      rB = mine ? sumB : rB;
      rC = mine ? sumC : rC;
      if ((n & 3) == 3) {
        const int i = lane >> 2;
        if (i < nt) {
          dBp[(t0 + i) * GN + n - 3 + (lane & 3)] = rB;
          dCp[(t0 + i) * GN + n - 3 + (lane & 3)] = rC;
        }
      }
    }
    // gradients of this tile's tokens; its inputs once more, from cache (by an
    // offset the compiler cannot tell from the first one's: it would keep
    // their 64 registers through the loop instead)
    const int64_t r0 = k.b * a.L;
    int off2 = off;
    asm volatile("" : "+v"(off2));
    RawTile<IO> ru, rd, rg, rz;
    ru.load(p.u, a.rows.u, t0, nt, off2);
    if (a.softplus) rd.load(p.dt, a.rows.dt, t0, nt, off2);
    if (p.z) {
      rg.load(p.dy, a.D, t0, nt, off2);
      rz.load(p.z, a.rows.z, t0, nt, off2);
    }
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      sA[i] = fmaf(sB[i] * kLog2e, ru.at(i), sA[i]);  // sB holds B ln 2, dt units of ln 2
      sB[i] = fmaf(dt[i], sB[i], skip * gy[i]);
    }
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < kScanT; ++i) sA[i] *= sigmoid2(fmaf(rd.at(i), kLog2e, bias));
    }
    if (nt < kScanT) {  // past the row: gy is zero already
#pragma unroll
      for (int i = 0; i < kScanT; ++i)
        if (i >= nt) sA[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      dbsum += sA[i];
      dDsum = fmaf(gy[i], ru.at(i), dDsum);
    }
    if (p.z) {
#pragma unroll
      for (int i = 0; i < kScanT; ++i) y[i] *= rg.at(i) * dsilu(rz.at(i), sigmoid(rz.at(i)));
    }
    if (ok) {
      store_tile<IO>(static_cast<T*>(a.du) + r0 * a.grows.u + k.d0, a.grows.u, t0, nt, off, sB);
      store_tile<IO>(static_cast<T*>(a.ddt) + r0 * a.grows.dt + k.d0, a.grows.dt, t0, nt, off, sA);
      if (p.z) store_tile<IO>(static_cast<T*>(a.dz) + r0 * a.grows.z + k.d0, a.grows.z, t0, nt, off, y);
    }
  }
  if (ok) {
    if (k.c == 0 && a.dinit)
      for (int n = 0; n < N; ++n) a.dinit[(k.b * N + n) * a.D + d] = gs[n * 64];
    // the chunk's adjoint has been used: its slot takes the chunk's dA
    for (int n = 0; n < N; ++n) ws.adj[co + (int64_t)n * a.D] = as[n * 64];
    bw.dDb[(k.b * g.nc + k.c) * 2 * a.D + d] = dDsum;
    bw.dDb[((k.b * g.nc + k.c) * 2 + 1) * a.D + d] = dbsum;
  }
}

// dB, dC [B L][G N] from the channel blocks' partial sums, added in order.
template <class IO>
__global__ __launch_bounds__(256) void scan_bc_reduce_kernel(ScanArgs a, int64_t ncb, const float* __restrict__ part) {
  typedef typename IO::type T;
  const int64_t GN = a.G * a.N, n = a.B * a.L * GN;
  const int64_t idx = (int64_t)flat_block() * 256 + threadIdx.x;
  if (idx >= 2 * n) return;
  const bool c = idx >= n;
  const int64_t e = c ? idx - n : idx;
  const float* q = part + (c ? ncb * n : 0) + e;
  float acc = 0.f;
  int64_t k = 0;
  for (; k + 8 <= ncb; k += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q[(k + i) * n];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += v[i];
  }
  for (; k < ncb; ++k) acc += q[k * n];
  const int64_t row = e / GN, col = e % GN;
  if (c) static_cast<T*>(a.dC)[row * a.grows.c + col] = IO::put(acc);
  else static_cast<T*>(a.dB)[row * a.grows.b + col] = IO::put(acc * kLn2);  // dt in units of ln 2
}

// dA [D,N], dD and ddt_bias [D] from the chunks' partial sums ([R][N D] and
// [R][2 D])
__global__ __launch_bounds__(kColsumThreads) void scan_param_kernel(const float* __restrict__ dAp,
                                                                    const float* __restrict__ dDb, int64_t R, int64_t D,
                                                                    int64_t N, float* __restrict__ dA,
                                                                    float* __restrict__ dD, float* __restrict__ db) {
  __shared__ float lds[kColsumThreads];
  int64_t c = (int64_t)flat_block() * 64 + (threadIdx.x & 63);
  const bool ok = c < (N + 2) * D;
  if (!ok) c = (N + 2) * D - 1;
  const bool isA = c < N * D;
  const float s = column_sum(isA ? dAp + c : dDb + c - N * D, R, isA ? N * D : 2 * D, lds);
  if (threadIdx.x >= 64 || !ok) return;
  if (isA) dA[c % D * N + c / D] = s * kLn2;  // dt in units of ln 2
  else if (c < (N + 1) * D) { if (dD) dD[c - N * D] = s; }
  else if (db) db[c - (N + 1) * D] = s;
}

// Chunks of four tiles: the carried states then cost a quarter of the per-tile
// states.  Shorter ones, down to one tile, where four would leave the third
// pass's two waves a SIMD unfilled (3 x 777 tokens of 1002 channels, fp32:
// 122 us with four tiles where two took 97).
static ScanGrid backward_grid(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  ScanGrid g;
  g.ncb = (D / G + 63) / 64;
  const int64_t slots = (int64_t)device_cu_count() * 8;
  int tiles = 4;
  while (tiles > 1 && B * G * g.ncb * ((L + kScanT * tiles - 1) / (kScanT * tiles)) < slots) tiles /= 2;
  g.Q = kScanT * tiles;
  g.nc = (L + g.Q - 1) / g.Q;
  g.ntile = (L + kScanT - 1) / kScanT;
  return g;
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct BwdLayout {
  size_t carry, adj, sdt, cut, pack, at, starts, tstate, tsdt, bc, dDb, total;
};
static BwdLayout backward_layout(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanGrid g = backward_grid(B, L, D, N, G);
  BwdLayout w;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t r = o; o += up256(bytes); return r; };
  w.carry = take(sizeof(float) * B * g.nc * N * D);
  w.adj = take(sizeof(float) * B * g.nc * N * D);
  w.sdt = take(sizeof(float) * B * g.nc * D);
  w.cut = take(sizeof(int) * B * g.nc);
  w.pack = take(sizeof(float) * scan_bc_floats(B, G, g.ntile, N));
  w.at = take(sizeof(float) * N * D);
  w.starts = take(sizeof(uint32_t) * B * g.ntile);
  w.tstate = take(sizeof(float) * (B * g.ntile + 1) * N * D);
  w.tsdt = take(sizeof(float) * (B * g.ntile + 1) * D);
  w.bc = take(sizeof(float) * 2 * g.ncb * B * L * G * N);
  w.dDb = take(sizeof(float) * B * g.nc * 2 * D);
  w.total = o;
  return w;
}
size_t scan_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  return backward_layout(B, L, D, N, G).total;
}

template <class IO, bool PACKED>
static hipError_t scan_backward_t(const ScanArgs& a, hipStream_t s) {
  const ScanGrid g = backward_grid(a.B, a.L, a.D, a.N, a.G);
  const BwdLayout w = backward_layout(a.B, a.L, a.D, a.N, a.G);
  char* base = static_cast<char*>(a.ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const ScanWs ws = {at(w.carry), at(w.sdt), reinterpret_cast<int*>(base + w.cut), at(w.adj), at(w.pack), at(w.at),
                     PACKED ? reinterpret_cast<uint32_t*>(base + w.starts) : nullptr, at(w.tstate), at(w.tsdt)};
  const BwdWs bw = {at(w.bc), at(w.dDb)};
  const dim3 grid((unsigned)(a.G * g.ncb), (unsigned)g.nc, (unsigned)a.B), block(64);
  const size_t per = 64 * sizeof(float) * a.N;
  const size_t lds1 = 2 * per, lds3 = 2 * per + 2 * sizeof(float) * kScanT * kRedRow;
  hipError_t e;
  if (lds1 > 64 * 1024 || lds3 > 64 * 1024) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_bwd_local_kernel<IO, PACKED>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds1);
    if (e != hipSuccess) return e;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_bwd_chunk_kernel<IO, PACKED>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds3);
    if (e != hipSuccess) return e;
  }
  if ((e = launch_scan_pack(a, g, ws, IO::kVec == 8, s)) != hipSuccess) return e;
  if (g.ntile > 1) {  // a single tile has nothing to pass on
    hipLaunchKernelGGL((scan_bwd_local_kernel<IO, PACKED>), grid, block, lds1, s, a, g, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if ((e = launch_scan_carry(a, g, ws, s)) != hipSuccess) return e;
  hipLaunchKernelGGL((scan_bwd_chunk_kernel<IO, PACKED>), grid, block, lds3, s, a, g, ws, bw);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t nbc = 2 * a.B * a.L * a.G * a.N;
  hipLaunchKernelGGL((scan_bc_reduce_kernel<IO>), flat_grid((nbc + 255) / 256), dim3(256), 0, s, a, g.ncb, bw.bc);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t np = (a.N + 2) * a.D;
  hipLaunchKernelGGL(scan_param_kernel, flat_grid((np + 63) / 64), dim3(kColsumThreads), 0, s, ws.adj, bw.dDb,
                     a.B * g.nc, a.D, a.N, a.dA, a.dD, a.ddt_bias);
  return hipGetLastError();
}

hipError_t launch_scan_backward(const ScanArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.seq_idx ? scan_backward_t<IoBF16, true>(a, s) : scan_backward_t<IoBF16, false>(a, s);
  return a.seq_idx ? scan_backward_t<IoF32, true>(a, s) : scan_backward_t<IoF32, false>(a, s);
}

}  // namespace ssd
