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
// recomputed forwards 16 tokens at a time (the steps' entering states in LDS)
// and swept backwards.  The sums over channels take a wave reduction that
// halves the number of values with each lane bit it sums over, so 16 tokens x
// 4 states end as one value a lane; the channel blocks' partial sums are then
// added in order.  No atomics: results do not depend on timing.
#include "layer_device.hpp"
#include "layer_launch.hpp"
#include "selective_scan.hpp"

namespace ssd {

struct BwdWs {
  float* bc;     // [ncb][B L][G N] dB partial sums, then the same for dC
  float* dDp;    // [B nc][D]
  float* dbp;    // [B nc][D]
};

// One row of the batch (b) of each input; lanes add their channel.
template <class IO>
struct RowPtrs {
  typedef typename IO::type T;
  const T *u, *dt, *z, *dy;
  __device__ __forceinline__ RowPtrs(const ScanArgs& a, int64_t b) {
    const int64_t r = b * a.L;
    u = static_cast<const T*>(a.u) + r * a.rows.u;
    dt = static_cast<const T*>(a.dt) + r * a.rows.dt;
    z = a.z ? static_cast<const T*>(a.z) + r * a.rows.z : nullptr;
    dy = static_cast<const T*>(a.dy) + r * a.D;
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
__global__ __launch_bounds__(64 * kScanWaves) void scan_bwd_local_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63;
  ScanBlock k;
  if (!scan_block(g, a, k)) return;
  const int N = (int)a.N;
  float* hs = lds + k.wave * 2 * N * 64 + lane;  // hs[n*64]: state
  float* gs = hs + N * 64;                       // gs[n*64]: what goes back to the entering state
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;
  const float* h_in = k.c == 0 && a.h0 ? a.h0 + k.b * N * a.D : nullptr;
  for (int n = 0; n < N; ++n) {
    hs[n * 64] = h_in ? h_in[(int64_t)n * a.D + d] : 0.f;
    gs[n * 64] = 0.f;
  }
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const RowPtrs<IO> p(a, k.b);
  const int off = (int)(d * sizeof(typename IO::type));
  const float* atp = ws.at + d;
  const float* ep = ws.bc + (((k.b * a.G + k.grp) * g.ntile + k.t0 / kScanT) * N) * kEntry;
  BCHalf<true> lo, hi;
  lo.load(ep);
  float a_n = atp[0];
  float sdt = 0.f;        // since the chunk's start
  float last = 0.f;       // since its last restart
  bool cut = false;
  for (int64_t t0 = k.t0; t0 < k.t1; t0 += kScanT) {
    const int nt = tile_tokens(k, t0);
    float dt[kScanT], x[kScanT], dy[kScanT];
    const uint32_t starts = PACKED ? ws.starts[k.b * g.ntile + t0 / kScanT] : 0;
    RawTile<IO> ru, rd, rg, rz;
    rd.load(p.dt, a.rows.dt, t0, nt, off);
    ru.load(p.u, a.rows.u, t0, nt, off);
    rg.load(p.dy, a.D, t0, nt, off);
    if (p.z) rz.load(p.z, a.rows.z, t0, nt, off);
    time_steps<IO>(rd, bias, a.softplus, nt, dt);
    gated<IO>(rg, rz, p.z, dy);
#pragma unroll
    for (int i = 0; i < kScanT; ++i) x[i] = dt[i] * ru.at(i);
    if (nt < kScanT) {  // past the row: decay 1, nothing added
#pragma unroll
      for (int i = 0; i < kScanT; ++i)
        if (i >= nt) x[i] = dy[i] = 0.f;
    }
    // tokens of this step that still reach the chunk's entering state
    const int live = cut ? 0 : (starts ? __builtin_ctz(starts) : kScanT);
    const float sdt0 = sdt;
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      last = (PACKED && (starts >> i & 1)) ? dt[i] : last + dt[i];
      sdt += dt[i];
    }
    for (int n = 0; n < N; ++n) {
      const float an = a_n;
      lo.settle();
      hi.load(ep + kScanT);
      a_n = atp[(int64_t)(n + 1 < N ? n + 1 : 0) * a.D];
      float h = hs[n * 64], acc = gs[n * 64], pr = fast_exp2(sdt0 * an);
      auto half = [&](const BCHalf<true>& e, int i0) {
#pragma unroll
        for (int i = i0; i < i0 + kHalf; ++i) {
          const float dec = fast_exp2(dt[i] * an);
          if (PACKED && (starts >> i & 1)) h = 0.f;
          h = fmaf(dec, h, x[i] * e.b(i - i0));
          pr *= dec;
          const float v = fmaf(pr, e.c(i - i0) * dy[i], acc);
          acc = (!PACKED || i < live) ? v : acc;
        }
      };
      half(lo, 0);
      hi.settle();
      ep += kEntry;
      lo.load(ep);
      half(hi, kHalf);
      hs[n * 64] = h;
      gs[n * 64] = acc;
    }
    cut = cut || starts != 0;
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

// Pass 2, in place: carry[c] = state entering chunk c (c >= 1; chunk 0 enters
// with the initial state), adj[c] = gradient reaching chunk c's last state
// from the tokens after it.
template <bool PACKED>
__global__ __launch_bounds__(256) void scan_bwd_carry_kernel(ScanArgs a, ScanGrid g, ScanWs ws) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= a.B * a.N * a.D) return;
  const int64_t d = idx % a.D, n = idx / a.D % a.N, b = idx / a.D / a.N;
  const float an = a.A[d * a.N + n];
  const float* sd = ws.sdt + b * g.nc * a.D + d;
  const int* cut = ws.cut + b * g.nc;
  const int64_t cs = a.N * a.D, o = (b * g.nc * a.N + n) * a.D + d;
  constexpr int U = 8;
  if (blockIdx.y == 0) {
    float* s = ws.carry + o;
    float run = 0.f;
    for (int64_t c0 = 0; c0 < g.nc; c0 += U) {
      float v[U], p[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 + i < g.nc ? c0 + i : g.nc - 1;
        v[i] = s[c * cs];
        p[i] = fast_exp2(sd[c * a.D] * an);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 + i;
        if (c < g.nc) {
          s[c * cs] = run;
          // chunk 0's left state already holds the initial state
          run = (c == 0 || (PACKED && cut[c])) ? v[i] : fmaf(p[i], run, v[i]);
        }
      }
    }
  } else {
    float* s = ws.adj + o;
    float run = a.dfinal ? a.dfinal[(b * a.N + n) * a.D + d] : 0.f;
    for (int64_t c0 = g.nc - 1; c0 >= 0; c0 -= U) {
      float v[U], p[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 - i > 0 ? c0 - i : 0;
        v[i] = s[c * cs];
        p[i] = fast_exp2(sd[c * a.D] * an);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 - i;
        if (c >= 0) {
          s[c * cs] = run;
          run = (PACKED && cut[c]) ? v[i] : fmaf(p[i], run, v[i]);
        }
      }
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
  return __uint_as_float(
      __builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// v0 summed over the two halves where the lane bit is clear, v1 where it is
// set (lane bits 5 and 4 by the row swaps, lower ones by data-parallel moves).
__device__ __forceinline__ float pair_sum32(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v0), __float_as_uint(v1), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float pair_sum16(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v0), __float_as_uint(v1), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ float pair_sum_dpp(float v0, float v1, bool set) {
  const float s0 = v0 + dpp_mov<CTRL>(v0), s1 = v1 + dpp_mov<CTRL>(v1);
  return set ? s1 : s0;
}
// 16 values a lane -> one: lane l holds value l >> 2, summed over the 16 lanes
// that share its low two bits up to the mirroring of the last step; two more
// pair sums over lane bits 1 and 0 complete it.
__device__ __forceinline__ float lane_sum16(const float (&v)[16], int lane) {
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pair_sum32(v[i], v[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pair_sum16(w[i], w[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = pair_sum_dpp<0x128>(w[i], w[i + 2], lane & 8);
  return pair_sum_dpp<0x141>(w[0], w[1], lane & 4);
}
__device__ __forceinline__ float lane_sum4(const float (&r)[4], int lane) {
  const float a = pair_sum_dpp<0x4E>(r[0], r[2], lane & 2);
  const float b = pair_sum_dpp<0x4E>(r[1], r[3], lane & 2);
  return pair_sum_dpp<0xB1>(a, b, lane & 1);
}

// Pass 3.  LDS per state and lane: the adjoint riding backwards, the summed
// dA, and the state entering each 16-token step but the first.
template <class IO, bool PACKED>
__global__ __launch_bounds__(64 * kScanWaves) void scan_bwd_chunk_kernel(ScanArgs a, ScanGrid g, ScanWs ws, BwdWs bw) {
  typedef typename IO::type T;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63;
  ScanBlock k;
  if (!scan_block(g, a, k)) return;
  const int N = (int)a.N;
  const int st = N * 64;
  float* gs = lds + k.wave * (int)(g.Q / kScanT + 1) * st + lane;  // gs[n*64]
  float* as = gs + st;               // dA
  float* hs = as + st;               // hs[(j-1)*st + n*64]: state entering step j >= 1
  const int64_t d = k.d0 + lane < k.dend ? k.d0 + lane : k.dend - 1;
  const bool ok = k.d0 + lane < k.dend;
  const int64_t co = (k.b * g.nc + k.c) * N * a.D + d;  // this chunk's slot
  const float* h_in = ws.carry + co;
  if (k.c == 0) h_in = a.h0 ? a.h0 + k.b * N * a.D + d : nullptr;
  for (int n = 0; n < N; ++n) {
    gs[n * 64] = ws.adj[co + (int64_t)n * a.D];
    as[n * 64] = 0.f;
  }
  const float bias = a.dt_bias ? a.dt_bias[d] * kLog2e : 0.f;
  const float skip = a.D_skip ? a.D_skip[d] : 0.f;
  const RowPtrs<IO> p(a, k.b);
  const int off = (int)(d * sizeof(typename IO::type));
  const int nstep = (int)((k.t1 - k.t0 + kScanT - 1) / kScanT);

  const float* atp = ws.at + d;
  const float* e0 = ws.bc + (((k.b * a.G + k.grp) * g.ntile + k.t0 / kScanT) * N) * kEntry;

  // states entering steps 1 .. nstep-1
  if (nstep > 1) {
    const float* ep = e0;
    BCHalf<false> lo, hi;
    lo.load(ep);
    float a_n = atp[0];
    for (int j = 0; j + 1 < nstep; ++j) {
      const int64_t t0 = k.t0 + j * kScanT;
      float dt[kScanT], x[kScanT];
      const uint32_t starts = PACKED ? ws.starts[k.b * g.ntile + t0 / kScanT] : 0;
      RawTile<IO> ru, rd;  // whole tiles: only the last one can be ragged
      rd.load(p.dt, a.rows.dt, t0, kScanT, off);
      ru.load(p.u, a.rows.u, t0, kScanT, off);
      time_steps<IO>(rd, bias, a.softplus, kScanT, dt);
#pragma unroll
      for (int i = 0; i < kScanT; ++i) x[i] = dt[i] * ru.at(i);
      for (int n = 0; n < N; ++n) {
        const float an = a_n;
        lo.settle();
        hi.load(ep + kScanT);
        a_n = atp[(int64_t)(n + 1 < N ? n + 1 : 0) * a.D];
        float h = j ? hs[(j - 1) * st + n * 64] : (h_in ? h_in[(int64_t)n * a.D] : 0.f);
        auto half = [&](const BCHalf<false>& e, int i0) {
#pragma unroll
          for (int i = i0; i < i0 + kHalf; ++i) {
            if (PACKED && (starts >> i & 1)) h = 0.f;
            h = fmaf(fast_exp2(dt[i] * an), h, x[i] * e.b(i - i0));
          }
        };
        half(lo, 0);
        hi.settle();
        ep += kEntry;
        lo.load(ep);
        half(hi, kHalf);
        hs[j * st + n * 64] = h;
      }
    }
  }

  const bool whole = k.d0 + 64 <= k.dend;
  float dDsum = 0.f, dbsum = 0.f;
  const int64_t BL = a.B * a.L;
  const int64_t GN = a.G * N;
  float* dBp = bw.bc + (k.cb * BL + k.b * a.L) * GN + k.grp * N;
  float* dCp = dBp + g.ncb * BL * GN;
  for (int j = nstep - 1; j >= 0; --j) {
    const int64_t t0 = k.t0 + j * kScanT;
    const int nt = tile_tokens(k, t0);
    float dt[kScanT], x[kScanT], gy[kScanT], y[kScanT], sB[kScanT], sA[kScanT];
    const uint32_t starts = PACKED ? ws.starts[k.b * g.ntile + t0 / kScanT] : 0;
    {
      RawTile<IO> ru, rd, rg, rz;
      rd.load(p.dt, a.rows.dt, t0, nt, off);
      ru.load(p.u, a.rows.u, t0, nt, off);
      rg.load(p.dy, a.D, t0, nt, off);
      if (p.z) rz.load(p.z, a.rows.z, t0, nt, off);
      time_steps<IO>(rd, bias, a.softplus, nt, dt);
      gated<IO>(rg, rz, p.z, gy);
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
    const float* ep = e0 + (int64_t)j * N * kEntry;
    BCHalf<true> lo, hi;
    lo.load(ep);
    hi.load(ep + kScanT);
    auto bv = [&](int i) { return i < kHalf ? lo.b(i) : hi.b(i - kHalf); };
    auto cv = [&](int i) { return i < kHalf ? lo.c(i) : hi.c(i - kHalf); };
    float a_n = atp[0];
    float rB[4] = {}, rC[4] = {};  // the last four states' sums
    for (int n = 0; n < N; ++n) {
      const float an = a_n;
      a_n = atp[(int64_t)(n + 1 < N ? n + 1 : 0) * a.D];
      float dec[kScanT], h[kScanT], v[kScanT];
      const float h0 = j ? hs[(j - 1) * st + n * 64] : (h_in ? h_in[(int64_t)n * a.D] : 0.f);
      float hp = h0;
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        dec[i] = fast_exp2(dt[i] * an);
        if (PACKED && (starts >> i & 1)) hp = 0.f;
        hp = fmaf(dec[i], hp, x[i] * bv(i));
        h[i] = hp;
        y[i] = fmaf(cv(i), hp, y[i]);
        v[i] = hp * gy[i];
      }
      const float sC = lane_sum16(v, lane);
      float ga = gs[n * 64], dA = as[n * 64];
#pragma unroll
      for (int i = kScanT - 1; i >= 0; --i) {
        const float gt = fmaf(cv(i), gy[i], ga);
        v[i] = gt * x[i];
        sB[i] = fmaf(gt, bv(i), sB[i]);
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
      ep += kEntry;
      lo.load(ep);
      hi.load(ep + kScanT);
      gs[n * 64] = ga;
      as[n * 64] = dA;
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        rB[e] = rB[e + 1];
        rC[e] = rC[e + 1];
      }
      rC[3] = sC;
      rB[3] = lane_sum16(v, lane);
      if ((n & 3) == 3) {
        const float vB = lane_sum4(rB, lane), vC = lane_sum4(rC, lane);
        const int i = lane >> 2;
        if (i < nt) {
          dBp[(t0 + i) * GN + n - 3 + (lane & 3)] = vB;
          dCp[(t0 + i) * GN + n - 3 + (lane & 3)] = vC;
        }
      }
    }
    // gradients of this tile's tokens (its inputs once more, from cache)
    const int64_t r0 = k.b * a.L;
    RawTile<IO> ru, rd, rg, rz;
    ru.load(p.u, a.rows.u, t0, nt, off);
    if (a.softplus) rd.load(p.dt, a.rows.dt, t0, nt, off);
    if (p.z) {
      rg.load(p.dy, a.D, t0, nt, off);
      rz.load(p.z, a.rows.z, t0, nt, off);
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
      store_tile<IO>(static_cast<T*>(a.du) + r0 * a.grows.u, a.grows.u, t0, nt, off, sB);
      store_tile<IO>(static_cast<T*>(a.ddt) + r0 * a.grows.dt, a.grows.dt, t0, nt, off, sA);
      if (p.z) store_tile<IO>(static_cast<T*>(a.dz) + r0 * a.grows.z, a.grows.z, t0, nt, off, y);
    }
  }
  if (ok) {
    if (k.c == 0 && a.dinit)
      for (int n = 0; n < N; ++n) a.dinit[(k.b * N + n) * a.D + d] = gs[n * 64];
    // the chunk's adjoint has been used: its slot takes the chunk's dA
    for (int n = 0; n < N; ++n) ws.adj[co + (int64_t)n * a.D] = as[n * 64];
    bw.dDp[(k.b * g.nc + k.c) * a.D + d] = dDsum;
    bw.dbp[(k.b * g.nc + k.c) * a.D + d] = dbsum;
  }
}

// dB, dC [B L][G N] from the channel blocks' partial sums, added in order.
template <class IO>
__global__ __launch_bounds__(256) void scan_bc_reduce_kernel(ScanArgs a, int64_t ncb, const float* __restrict__ part) {
  typedef typename IO::type T;
  const int64_t GN = a.G * a.N, n = a.B * a.L * GN;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
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

// dA [D,N] from the chunk sums' [N][D]
__global__ __launch_bounds__(256) void scan_da_kernel(const float* __restrict__ s, int64_t D, int64_t N,
                                                      float* __restrict__ dA) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= D * N) return;
  dA[idx] = s[idx % N * D + idx / N] * kLn2;  // dt in units of ln 2
}

// Steps of 16 tokens a chunk: as many as leave eight waves a compute unit
// their LDS (N <= 32: four), fewer for large N.
static ScanGrid backward_grid(int64_t L, int64_t D, int64_t N, int64_t G) {
  ScanGrid g;
  g.ncb = (D / G + 63) / 64;
  g.Q = kScanT * (N <= 32 ? 4 : N <= 64 ? 2 : 1);
  g.nc = (L + g.Q - 1) / g.Q;
  g.ntile = (L + kScanT - 1) / kScanT;
  g.wpb = scan_wpb(g.ncb, 64 * (int64_t)sizeof(float) * N * (g.Q / kScanT + 1));
  return g;
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct BwdLayout {
  size_t carry, adj, sdt, cut, pack, at, starts, bc, dDp, dbp, sums, total;
};
static BwdLayout backward_layout(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanGrid g = backward_grid(L, D, N, G);
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
  w.bc = take(sizeof(float) * 2 * g.ncb * B * L * G * N);
  w.dDp = take(sizeof(float) * B * g.nc * D);
  w.dbp = take(sizeof(float) * B * g.nc * D);
  w.sums = take(sizeof(float) * N * D);
  w.total = o;
  return w;
}
size_t scan_backward_ws_bytes(int64_t B, int64_t L, int64_t D, int64_t N, int64_t G) {
  return backward_layout(B, L, D, N, G).total;
}

template <class IO, bool PACKED>
static hipError_t scan_backward_t(const ScanArgs& a, hipStream_t s) {
  const ScanGrid g = backward_grid(a.L, a.D, a.N, a.G);
  const BwdLayout w = backward_layout(a.B, a.L, a.D, a.N, a.G);
  char* base = static_cast<char*>(a.ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const ScanWs ws = {at(w.carry), at(w.sdt), reinterpret_cast<int*>(base + w.cut), at(w.adj), at(w.pack), at(w.at),
                     PACKED ? reinterpret_cast<uint32_t*>(base + w.starts) : nullptr};
  const BwdWs bw = {at(w.bc), at(w.dDp), at(w.dbp)};
  const dim3 grid((unsigned)scan_blocks(g, a.G), (unsigned)g.nc, (unsigned)a.B), block(64 * g.wpb);
  const size_t per = 64 * sizeof(float) * a.N * g.wpb;
  const size_t lds1 = 2 * per, lds3 = per * (2 + g.Q / kScanT - 1);
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
  hipLaunchKernelGGL((scan_bwd_local_kernel<IO, PACKED>), grid, block, lds1, s, a, g, ws);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((scan_bwd_carry_kernel<PACKED>), dim3((unsigned)((a.B * a.N * a.D + 255) / 256), 2), dim3(256), 0,
                     s, a, g, ws);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((scan_bwd_chunk_kernel<IO, PACKED>), grid, block, lds3, s, a, g, ws, bw);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t nbc = 2 * a.B * a.L * a.G * a.N;
  hipLaunchKernelGGL((scan_bc_reduce_kernel<IO>), dim3((unsigned)((nbc + 255) / 256)), dim3(256), 0, s, a, g.ncb, bw.bc);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  float* sums = at(w.sums);
  if ((e = launch_colsum(ws.adj, a.B * g.nc, a.N * a.D, sums, s)) != hipSuccess) return e;
  hipLaunchKernelGGL(scan_da_kernel, dim3((unsigned)((a.N * a.D + 255) / 256)), dim3(256), 0, s, sums, a.D, a.N, a.dA);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.dD && (e = launch_colsum(bw.dDp, a.B * g.nc, a.D, a.dD, s)) != hipSuccess) return e;
  if (a.ddt_bias && (e = launch_colsum(bw.dbp, a.B * g.nc, a.D, a.ddt_bias, s)) != hipSuccess) return e;
  return hipSuccess;
}

hipError_t launch_scan_backward(const ScanArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.seq_idx ? scan_backward_t<IoBF16, true>(a, s) : scan_backward_t<IoBF16, false>(a, s);
  return a.seq_idx ? scan_backward_t<IoF32, true>(a, s) : scan_backward_t<IoF32, false>(a, s);
}

}  // namespace ssd
