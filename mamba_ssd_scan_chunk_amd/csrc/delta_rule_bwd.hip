// delta_rule_bwd.hip -- gradients of the gated delta rule.  With the forward's
// names (delta_rule.hpp), D the gradient of the state behind a piece and dy of
// its outputs,
//     du = P^T dy + diag(e^{G_end - G}) k D,   du += R^T (b du),   dw = b du,
//     dv = dw,   D' = e^{G_end} D + q^T diag(e^G) dy - k^T diag(e^G) dw,
//     db_t = du_t . w_t,
//     dQK_ts = e^{G_t - G_s} dy_t.u_s (s <= t),  dKK_ts = -e^{G_t - G_s} dw_t.u_s (s < t),
//     dq = diag(e^G) dy S^T + dQK k,
//     dk = -diag(e^G) dw S^T + diag(e^{G_end - G}) u D^T + dQK^T q + (dKK + dKK^T) k.
// The log decay g_t stands between what is written before t and what is read
// from t on:
//     dg_t = sum_{s < t <= r} Z_rs + sum_{r >= t} rowS_r + sum_{s < t} colD_s + e^{G_end} <S, D>
// with Z = dQK (q.k) + dKK (k.k), rowS and colD the shares of the state in
// front and of the one behind in q.dq + k.dk.  Taken as differences of q.dq
// and k.dk the pairs on one side of t would cancel only up to the products'
// rounding; from one Z they cancel exactly.
//
// Five launches: the preparation and the forward chain (delta_rule.hip), which
// leave the states in front of the windows and w; delta_reverse_kernel, a wave
// 16 value columns as there, which leaves D of every window and du;
// delta_grad_kernel, a block a (window, head), all windows at once; and
// delta_finish_kernel, which adds the heads of a key group and takes the
// gradients through the unit length.
#include "delta_rule.hpp"

namespace ssd {

constexpr int kTP = kC + 4;

// ---------------------------------------------------------------- the chain, back to front
template <class M, int NP>
constexpr int rev_pitch() { return NP + 16 / (int)sizeof(typename M::IO::type); }
template <class M, int NP>
constexpr size_t rev_lds() {
  return (size_t)2 * kC * rev_pitch<M, NP>() * sizeof(typename M::IO::type) + 5 * kC * 4;
}

template <class M, int NP, bool VL>
__global__ __launch_bounds__(256) void delta_reverse_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename M::IO::type T;
  typedef typename M::Two Two;
  constexpr int NT = NP / 16, KS = NP / 32, LP = rev_pitch<M, NP>(), V = M::IO::kVec;
  extern __shared__ __align__(16) char lds[];
  T* kt = reinterpret_cast<T*>(lds);
  T* qt = kt + kC * LP;
  float* gt = reinterpret_cast<float*>(qt + kC * LP);
  const float *sBeta = gt, *sKin = gt + kC, *sQin = gt + 2 * kC, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nthr = blockDim.x, c = lane & 15, g = lane >> 4;
  const uint32_t bid = near_block(blockIdx.x, gridDim.x);
  const uint32_t slices = (uint32_t)(a.P / 16) / (nthr / 64);
  const int64_t bh = bid / slices, h = bh % a.H, b = bh / a.H, grp = h / (a.H / a.G);
  const int64_t p = ((bid % slices) * (nthr / 64) + wave) * 16 + c;
  const int N = (int)a.N;
  const int64_t row = b * a.L;

  f32x4_t D[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nn = 16 * j + 4 * g + r;
      D[j][r] = a.dfinal && nn < N ? a.dfinal[(bh * N + nn) * a.P + p] : 0.f;
    }

  for (int64_t win = ws.nw - 1; win >= 0; --win) {
    const int64_t t0 = win * kC, bhw = bh * ws.nw + win;
    const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC);
    Cuts cuts = {0, 0};
    if constexpr (VL) cuts = window_cuts(a.seq_idx, nullptr, row, t0, a.L, lane);
    {
      float* out = reinterpret_cast<float*>(a.ws + ws.D) + bhw * N * a.P + p;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int nn = 16 * j + 4 * g + r;
          if (nn < N) out[nn * a.P] = D[j][r];
        }
    }
    const char* fr = a.ws + ws.up_r + bhw * kTriBytes;
    const char* fp = a.ws + ws.up_p + bhw * kTriBytes;
    int end = n;
    while (end > 0) {
      const int begin = VL ? piece_begin(cuts.piece, end) : 0;
      __syncthreads();
      for (int i = tid; i < kC * (NP / V); i += nthr) {
        const int t = i / (NP / V), col = i % (NP / V) * V;
        uint4 kv = make_uint4(0, 0, 0, 0), qv = kv;
        if (t >= begin && t < end && col < N) {
          kv = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + (row + t0 + t) * a.rows.k + grp * N + col);
          qv = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (row + t0 + t) * a.rows.q + grp * N + col);
        }
        *reinterpret_cast<uint4*>(kt + t * LP + col) = kv;
        *reinterpret_cast<uint4*>(qt + t * LP + col) = qv;
      }
      const float* gsrc = reinterpret_cast<const float*>(reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw);
      for (int i = tid; i < 5 * kC; i += nthr) gt[i] = i % kC >= begin && i % kC < end ? gsrc[i] : 0.f;
      __syncthreads();

      f32x4_t dy[4], du[4];
      const T* yp = static_cast<const T*>(a.dy) + ((row + t0) * a.H + h) * a.P + p;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          dy[i][r] = t >= begin && t < end ? M::IO::get(yp[t * a.H * a.P]) : 0.f;
          du[i][r] = 0.f;
        }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float v[8];
        slots(D[2 * s], D[2 * s + 1], v);
        const Two db = M::two(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const T* kp = kt + (16 * i + c) * LP + 32 * s + 4 * g;
          du[i] = M::mma(lds_4x2<M>(kp, kp + 16), db, du[i]);
        }
      }
      float be[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          be[i][r] = sBeta[t];
          du[i][r] *= sKout[t];
        }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8];
        slots(dy[2 * s], dy[2 * s + 1], v);
        const typename M::One yb = M::one(v);
#pragma unroll
        for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(M::load(fp + up_frag(i, s) * 2048, lane), yb, du[i]);
      }
      // du += R^T (b du); the products read what was before them
      Two xb[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 32 * s + 16 * (e / 4) + 4 * g + e % 4;
          v[e] = !VL || (t >= begin && t < end) ? be[2 * s + e / 4][e % 4] * du[2 * s + e / 4][e % 4] : 0.f;
        }
        xb[s] = M::two(v);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(M::load(fr + up_frag(i, s) * 2048, lane), xb[s], du[i]);
      float* out = reinterpret_cast<float*>(a.ws + ws.du) + bhw * kC * a.P + p;
      T* dvp = static_cast<T*>(a.dv) + (row + t0) * a.grows.v + h * a.P + p;
      f32x4_t dw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          const bool on = t >= begin && t < end;
          dw[i][r] = !VL || on ? be[i][r] * du[i][r] : 0.f;
          if (on) {
            out[t * a.P] = du[i][r];
            dvp[t * a.grows.v] = M::IO::put(dw[i][r]);
          }
        }
      const float whole = sIn[end - 1];
#pragma unroll
      for (int j = 0; j < NT; ++j) D[j] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8], x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 32 * s + 16 * (e / 4) + 4 * g + e % 4;
          v[e] = sQin[t] * dy[2 * s + e / 4][e % 4];
          x[e] = -sKin[t] * dw[2 * s + e / 4][e % 4];
        }
        const Two yb = M::two(v), wb = M::two(x);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          D[j] = M::mma(M::transposed(qt + 32 * s * LP + 16 * j, LP, lane), yb, D[j]);
          D[j] = M::mma(M::transposed(kt + 32 * s * LP + 16 * j, LP, lane), wb, D[j]);
        }
      }
      if (VL && (cuts.fresh >> begin & 1)) {  // nothing goes back past a sequence's start
#pragma unroll
        for (int j = 0; j < NT; ++j) D[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      end = begin;
    }
  }
  if (a.dinit) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int nn = 16 * j + 4 * g + r;
        if (nn < N) a.dinit[(bh * N + nn) * a.P + p] = D[j][r];
      }
  }
}

// ---------------------------------------------------------------- the same of bf16 inputs
// C column waves and C helpers, as in the forward chain.  What the next piece
// adds whatever D is, P^T dy to its values and q^T diag(e^G) dy to D, the helpers
// work out a step ahead and leave in LDS as accumulators.
template <int NP, int C>
struct ReverseLds {
  static constexpr int kPitch = NP + 8;
  static constexpr int kRows = kC * kPitch * 2;
  static constexpr int kX = (NP / 16 + 4) * 1024;
  static constexpr int k = 0, r = k + kRows, g = r + kTriBytes, half = g + 5 * kC * 4;
  static constexpr int q = 2 * half, x = q + 2 * kRows, total = x + 2 * C * kX;
};

template <int NP, int C, bool VL>
__global__ __launch_bounds__(128 * C, C) void delta_reverse_bf16_kernel(DeltaArgs a, DeltaWs ws) {
  typedef DeltaB M;
  typedef DeltaB::One One;
  typedef DeltaB::Two Two;
  typedef ReverseLds<NP, C> Lay;
  constexpr int NT = NP / 16, KS = NP / 32, LP = Lay::kPitch, NH = 64 * C;
  extern __shared__ __align__(16) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t bid = near_block(blockIdx.x, gridDim.x);
  const uint32_t slices = (uint32_t)(a.P / 16) / C;
  const int64_t bh = bid / slices, h = bh % a.H, b = bh / a.H, grp = h / (a.H / a.G);
  const uint32_t p = ((bid % slices) * C + wave % C) * 16 + c;
  const int N = (int)a.N;
  const uint32_t P = (uint32_t)a.P;
  const int64_t row = b * a.L;
  Pieces pc;
  pc.last(VL ? reinterpret_cast<const Cuts*>(a.ws + ws.cuts) + b * ws.nw : nullptr, ws.nw, a.L);

  if (wave >= C) {
    // ---- helper
    const int ht = tid - NH;
    RowTile<NP, NH> kt, qt;
    TriTile<NH> rt;
    GateTile<NH> gt;
    Column dy;
    f32x4_t qin[4];
    const uint32_t krow = (uint32_t)a.rows.k, qrow = (uint32_t)a.rows.q, yrow = (uint32_t)(a.H * a.P);
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + row * a.rows.k + grp * N;
    const uint16_t* qb = static_cast<const uint16_t*>(a.q) + row * a.rows.q + grp * N;
    auto gates = [&](const Pieces& s) {
      return reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bh * ws.nw + s.win;
    };
    auto ask = [&](const Pieces& s) {
      kt.load(kb + s.win * kC * a.rows.k, krow, N, s.n, ht);
      rt.load(a.ws + ws.up_r + (bh * ws.nw + s.win) * kTriBytes, ht);
      gt.load(gates(s), ht);
    };
    auto put = [&](const Pieces& s, int half) {
      char* o = lds + half * Lay::half;
      kt.template store<VL>(reinterpret_cast<uint16_t*>(o + Lay::k), LP, s.begin, s.end, ht);
      rt.store(o + Lay::r, ht);
      gt.template store<VL>(reinterpret_cast<float*>(o + Lay::g), s.begin, s.end, ht);
    };
    auto ask_q = [&](const Pieces& s) { qt.load(qb + s.win * kC * a.rows.q, qrow, N, s.n, ht); };
    auto put_q = [&](const Pieces& s, int half) {
      qt.template store<VL>(reinterpret_cast<uint16_t*>(lds + Lay::q + half * Lay::kRows), LP, s.begin, s.end, ht);
    };
    auto ask_dy = [&](const Pieces& s) {
      dy.load(static_cast<const uint16_t*>(a.dy) + ((row + s.win * kC) * a.H + h) * a.P, yrow, 4 * g * yrow + p, s.n);
#pragma unroll
      for (int i = 0; i < 4; ++i) qin[i] = *reinterpret_cast<const f32x4_t*>(gates(s)->qin + 16 * i + 4 * g);
    };
    // P^T dy and q^T diag(e^G) dy of piece s, whose q is in LDS
    auto work = [&](const Pieces& s, int half) {
      const char* fp = a.ws + ws.up_p + (bh * ws.nw + s.win) * kTriBytes;
      Two pf[kTriFrags];
#pragma unroll
      for (int f = 0; f < kTriFrags; ++f) pf[f] = M::load(fp + f * 2048, lane);
      const uint16_t* ql = reinterpret_cast<const uint16_t*>(lds + Lay::q + half * Lay::kRows);
      char* x = lds + Lay::x + (half * C + wave % C) * Lay::kX;
      One yb[2];
      f32x4_t Y[NT], py[4];
#pragma unroll
      for (int j = 0; j < NT; ++j) Y[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) py[i] = Y[0];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        One qT[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) qT[j] = M::transposed(ql + 32 * t * LP + 16 * j, LP, lane);
        float v[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 2 * t + e / 4, r = e % 4, tok = 16 * i + 4 * g + r;
          const bool on = !VL || (tok >= s.begin && tok < s.end);
          v[e] = on ? dy.get(i, r) : 0.f;
          w[e] = on ? qin[i][r] * v[e] : 0.f;
        }
        yb[t] = M::one(v);
        const Two wb = M::two(w);
#pragma unroll
        for (int j = 0; j < NT; ++j) Y[j] = M::mma(qT[j], wb.lo, Y[j]);
#pragma unroll
        for (int j = 0; j < NT; ++j) Y[j] = M::mma(qT[j], wb.hi, Y[j]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 2 * t + 2; ++i) py[i] = M::mma(pf[up_frag(i, t)].lo, yb[t], py[i]);
#pragma unroll
        for (int i = 0; i < 2 * t + 2; ++i) py[i] = M::mma(pf[up_frag(i, t)].hi, yb[t], py[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4_t*>(x + i * 1024 + 16 * lane) = py[i];
#pragma unroll
      for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4_t*>(x + (4 + j) * 1024 + 16 * lane) = Y[j];
    };
    // before the first piece: its operands, q of it and of the next, its products
    Pieces n1 = pc;
    n1.step_back();
    ask(pc);
    ask_q(pc);
    ask_dy(pc);
    put(pc, 0);
    put_q(pc, 0);
    if (n1.valid_back()) ask_q(n1);
    __syncthreads();
    work(pc, 0);
    if (n1.valid_back()) {
      put_q(n1, 1);
      ask_dy(n1);
    }
    __syncthreads();
    for (int j = 0;; ++j) {
      // pc: piece j, which the column waves take now; n1: the next
      if (!n1.valid_back()) {
        __syncthreads();
        break;
      }
      Pieces n2 = n1;
      n2.step_back();
      ask(n1);
      if (n2.valid_back()) ask_q(n2);
      work(n1, (j + 1) & 1);
      put(n1, (j + 1) & 1);
      if (n2.valid_back()) {
        put_q(n2, j & 1);
        ask_dy(n2);
      }
      n1 = n2;
      __syncthreads();
    }
    return;
  }

  // ---- column wave
  f32x4_t D[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nn = 16 * j + 4 * g + r;
      D[j][r] = a.dfinal && nn < N ? a.dfinal[(bh * N + nn) * a.P + p] : 0.f;
    }
  const uint32_t vrow = (uint32_t)a.grows.v;
  uint16_t* dvb = static_cast<uint16_t*>(a.dv) + row * a.grows.v + h * a.P;
  __syncthreads();
  __syncthreads();
  for (int step = 0; pc.valid_back(); ++step) {
    const int begin = pc.begin, end = pc.end, n = pc.n;
    const int64_t win = pc.win, bhw = bh * ws.nw + win;
    const char* in = lds + (step & 1) * Lay::half;
    const uint16_t* kt = reinterpret_cast<const uint16_t*>(in + Lay::k);
    const float* gt = reinterpret_cast<const float*>(in + Lay::g);
    const float *sBeta = gt, *sKin = gt + kC, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC;
    const char* x = lds + Lay::x + ((step & 1) * C + wave) * Lay::kX;
    One kf[KS][4], kT[2][NT];
    Two rf[kTriFrags];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* kp = kt + (16 * i + c) * LP + 32 * s + 4 * g;
        kf[s][i] = lds_4x2<M>(kp, kp + 16);
      }
    __builtin_amdgcn_sched_barrier(0);
    if (!VL || end == n)
      put_state<NT>(reinterpret_cast<float*>(a.ws + ws.D) + bhw * N * a.P, N, P, 4 * g * P + p, D);
    f32x4_t du[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) du[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float v[8];
      slots(D[2 * s], D[2 * s + 1], v);
      const Two db = M::two(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) du[i] = M::mma(kf[s][i], db.lo, du[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) du[i] = M::mma(kf[s][i], db.hi, du[i]);
      if (s == 0) {
#pragma unroll
        for (int f = 0; f < kTriFrags; ++f) rf[f] = M::load(in + Lay::r + f * 2048, lane);
      }
    }
#pragma unroll
    for (int e = 0; e < 8 * KS; ++e) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
    }
    float ki[4][4], be[4][4], ko[4][4];
    f32x4_t py[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_vec<IoF32, 4>(sKin + 16 * i + 4 * g, ki[i]);
      load_vec<IoF32, 4>(sBeta + 16 * i + 4 * g, be[i]);
      load_vec<IoF32, 4>(sKout + 16 * i + 4 * g, ko[i]);
      py[i] = *reinterpret_cast<const f32x4_t*>(x + i * 1024 + 16 * lane);
    }
    const float whole = sIn[end - 1];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) kT[s][j] = M::transposed(kt + 32 * s * LP + 16 * j, LP, lane);
    __builtin_amdgcn_sched_barrier(0);
    // du = P^T dy + e^{G_end - G} k D, then R^T of what it is here
    Two xb[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 2 * s + e / 4, r = e % 4, t = 16 * i + 4 * g + r;
        du[i][r] = fmaf(ko[i][r], du[i][r], py[i][r]);
        v[e] = !VL || (t >= begin && t < end) ? be[i][r] * du[i][r] : 0.f;
      }
      xb[s] = M::two(v);
    }
    pc.step_back();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(rf[up_frag(i, s)].hi, xb[s].lo, du[i]);
#pragma unroll
      for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(rf[up_frag(i, s)].lo, xb[s].hi, du[i]);
#pragma unroll
      for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(rf[up_frag(i, s)].hi, xb[s].hi, du[i]);
    }
    f32x4_t Y[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) Y[j] = *reinterpret_cast<const f32x4_t*>(x + (4 + j) * 1024 + 16 * lane);
    Column::put<VL>(reinterpret_cast<float*>(a.ws + ws.du) + bhw * kC * a.P, P, 4 * g * P + p, kC, du, begin, end, g);
    f32x4_t dw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * g + r;
        dw[i][r] = !VL || (t >= begin && t < end) ? be[i][r] * du[i][r] : 0.f;
      }
    Column::put<VL>(dvb + win * kC * a.grows.v, vrow, 4 * g * vrow + p, n, dw, begin, end, g);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) D[j][r] = fmaf(whole, D[j][r], Y[j][r]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = -ki[2 * s + e / 4][e % 4] * dw[2 * s + e / 4][e % 4];
      const Two wb = M::two(v);
#pragma unroll
      for (int j = 0; j < NT; ++j) D[j] = M::mma(kT[s][j], wb.lo, D[j]);
#pragma unroll
      for (int j = 0; j < NT; ++j) D[j] = M::mma(kT[s][j], wb.hi, D[j]);
    }
    if constexpr (VL) {
      // nothing goes back past a sequence's start
      const Cuts* list = reinterpret_cast<const Cuts*>(a.ws + ws.cuts) + b * ws.nw;
      if (uniform64(list[win].fresh) >> begin & 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) D[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
    __syncthreads();
  }
  if (a.dinit) put_state<NT>(a.dinit + bh * N * a.P, N, P, 4 * g * P + p, D);
}

// ---------------------------------------------------------------- all windows at once
// Left operands of 64 tokens by 64 value columns in LDS.
template <class M> struct GradTile;
template <> struct GradTile<DeltaB> {
  static constexpr int kPitch = 72, kPlane = kC * kPitch;
  uint16_t* p;  // dy, u hi, u lo, dw hi, dw lo
  __device__ __forceinline__ explicit GradTile(char* lds) : p(reinterpret_cast<uint16_t*>(lds)) {}
  static constexpr size_t bytes() { return (size_t)5 * kPlane * 2; }
  __device__ __forceinline__ void put8(int t, int col, const float* dy, const float* u, const float* dw) {
    const DeltaB::Two x = DeltaB::two(u), y = DeltaB::two(dw);
    uint16_t* q = p + t * kPitch + col;
    *reinterpret_cast<uint4*>(q) = DeltaB::one(dy).v;
    *reinterpret_cast<uint4*>(q + kPlane) = x.hi.v;
    *reinterpret_cast<uint4*>(q + 2 * kPlane) = x.lo.v;
    *reinterpret_cast<uint4*>(q + 3 * kPlane) = y.hi.v;
    *reinterpret_cast<uint4*>(q + 4 * kPlane) = y.lo.v;
  }
  __device__ __forceinline__ DeltaB::One dy(int t, int col) const { return DeltaB::global8(p + t * kPitch + col); }
  __device__ __forceinline__ DeltaB::Two two(int plane, int t, int col) const {
    DeltaB::Two x;
    x.hi = DeltaB::global8(p + plane * kPlane + t * kPitch + col);
    x.lo = DeltaB::global8(p + (plane + 1) * kPlane + t * kPitch + col);
    return x;
  }
  __device__ __forceinline__ DeltaB::Two u(int t, int col) const { return two(1, t, col); }
  __device__ __forceinline__ DeltaB::Two dw(int t, int col) const { return two(3, t, col); }
};
template <> struct GradTile<DeltaF> {
  static constexpr int kPitch = 68, kPlane = kC * kPitch;
  float* p;  // dy, u, dw
  __device__ __forceinline__ explicit GradTile(char* lds) : p(reinterpret_cast<float*>(lds)) {}
  static constexpr size_t bytes() { return (size_t)3 * kPlane * 4; }
  __device__ __forceinline__ void put8(int t, int col, const float* dy, const float* u, const float* dw) {
    float* q = p + t * kPitch + col;
    Lds<OpF32>::store8(q, dy);
    Lds<OpF32>::store8(q + kPlane, u);
    Lds<OpF32>::store8(q + 2 * kPlane, dw);
  }
  __device__ __forceinline__ DeltaF::One dy(int t, int col) const { return DeltaF::global8(p + t * kPitch + col); }
  __device__ __forceinline__ DeltaF::Two u(int t, int col) const { return DeltaF::global8(p + kPlane + t * kPitch + col); }
  __device__ __forceinline__ DeltaF::Two dw(int t, int col) const {
    return DeltaF::global8(p + 2 * kPlane + t * kPitch + col);
  }
};
template <class M>
constexpr size_t grad_lds() {
  const size_t tile = GradTile<M>::bytes(), tri = (size_t)3 * kC * kTP * 4;
  return (tile > tri ? tile : tri) + (size_t)(7 + 4 + 4 + 4 + 1 + 1) * kC * 4 + kC * 8 + 16 * 4;
}

// Sum over the 16 lanes of a group, in every lane.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Four waves; a wave takes NTW 16-row tiles of the state (dq and dk columns)
// for all 64 tokens, and rows 16 wave .. of the token-by-token matrices.
template <class M, int NTW, bool VL>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename M::IO::type T;
  typedef typename M::One One;
  typedef typename M::Two Two;
  extern __shared__ __align__(16) char lds[];
  constexpr size_t kBig = GradTile<M>::bytes() > (size_t)3 * kC * kTP * 4 ? GradTile<M>::bytes() : (size_t)3 * kC * kTP * 4;
  GradTile<M> tile(lds);
  float(*M1)[kTP] = reinterpret_cast<float(*)[kTP]>(lds);
  float(*M2)[kTP] = M1 + kC;
  float(*M3)[kTP] = M2 + kC;
  double* sG = reinterpret_cast<double*>(lds + kBig);
  float* gt = reinterpret_cast<float*>(sG + kC);
  const float *sBeta = gt, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC, *sRk = gt + 5 * kC, *sRq = gt + 6 * kC;
  float(*rowS)[kC] = reinterpret_cast<float(*)[kC]>(gt + 7 * kC);  // by wave
  float(*colD)[kC] = rowS + 4;
  float(*colZ)[kC] = colD + 4;
  float* rowZ = reinterpret_cast<float*>(colZ + 4);
  float* sDb = rowZ + kC;
  float* sSD = sDb + kC;  // by wave

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int64_t bid = near_block(blockIdx.x, gridDim.x);
  const int64_t h = bid % a.H, win = bid / a.H % ws.nw, b = bid / a.H / ws.nw;
  const int64_t row = b * a.L, t0 = win * kC, bhw = (b * a.H + h) * ws.nw + win;
  const int64_t grp = h / (a.H / a.G);
  const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC), N = (int)a.N, P = (int)a.P;
  Cuts cuts = {0, 0};
  if constexpr (VL) cuts = window_cuts(a.seq_idx, nullptr, row, t0, a.L, lane);
  const DeltaGates* gates = reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw;
  for (int i = tid; i < 7 * kC; i += 256) gt[i] = reinterpret_cast<const float*>(gates)[i];
  if (tid < kC) sG[tid] = gates->G[tid];
  const float* wsw = reinterpret_cast<const float*>(a.ws + ws.w) + bhw * kC * P;
  const float* wsu = reinterpret_cast<const float*>(a.ws + ws.du) + bhw * kC * P;
  const float* wsS = reinterpret_cast<const float*>(a.ws + ws.S) + bhw * N * P;
  const float* wsD = reinterpret_cast<const float*>(a.ws + ws.D) + bhw * N * P;
  const T* kbase = static_cast<const T*>(a.k) + (row + t0) * a.rows.k + grp * N;
  const T* qbase = static_cast<const T*>(a.q) + (row + t0) * a.rows.q + grp * N;
  const T* ybase = static_cast<const T*>(a.dy) + ((row + t0) * a.H + h) * P;
  float sumA = 0.f, sumB = 0.f;  // of dA and ddt_bias, in wave 0
  const f32x4_t zero4 = {0.f, 0.f, 0.f, 0.f};

  int begin = 0;
  while (begin < n) {
    const int end = VL ? piece_end(cuts.piece, begin, n) : n;
    // only a row's first piece begins with a state, only its last one hands one on
    const bool first = begin == 0, last = end == n;
    f32x4_t qS[NTW][4], wS[NTW][4], uD[NTW][4], dP[4], dE[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dP[i] = dE[i] = zero4;
#pragma unroll
      for (int m = 0; m < NTW; ++m) qS[m][i] = wS[m][i] = uD[m][i] = zero4;
    }
    float sd = 0.f, db = 0.f;
    for (int p0 = 0; p0 < P; p0 += 64) {
      __syncthreads();
      {
        const int t = tid >> 2, col = (tid & 3) * 16;
        const bool on = t >= begin && t < end && p0 + col < P;
        const float beta = on ? sBeta[t] : 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          float w[8], du[8], dy[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = du[k] = dy[k] = 0.f;
          if (on) {
            load_vec<IoF32, 8>(wsw + t * P + p0 + col + e, w);
            load_vec<IoF32, 8>(wsu + t * P + p0 + col + e, du);
            load_vec<typename M::IO, 8>(ybase + t * a.H * P + p0 + col + e, dy);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            db = fmaf(w[k], du[k], db);
            w[k] *= beta;
            du[k] *= beta;
          }
          tile.put8(t, col + e, dy, w, du);
        }
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (p0 + 32 * s >= P) break;
        const int col = 32 * s + 8 * g;
        One ya[4];
        Two ua[4], wa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ya[i] = tile.dy(16 * i + c, col);
          ua[i] = tile.u(16 * i + c, col);
          wa[i] = tile.dw(16 * i + c, col);
        }
#pragma unroll
        for (int m = 0; m < NTW; ++m) {
          const int nn = 16 * (wave + 4 * m) + c;
          float sv[8], dv[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) sv[k] = dv[k] = 0.f;
          if (nn < N && p0 + col < P) {
            if (first) load_vec<IoF32, 8>(wsS + nn * P + p0 + col, sv);
            if (last) load_vec<IoF32, 8>(wsD + nn * P + p0 + col, dv);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) sd = fmaf(sv[k], dv[k], sd);
          const Two sf = M::two(sv), df = M::two(dv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qS[m][i] = M::mma(ya[i], sf, qS[m][i]);
            wS[m][i] = M::mma(wa[i], sf, wS[m][i]);
            uD[m][i] = M::mma(ua[i], df, uD[m][i]);
          }
        }
        const One yr = tile.dy(16 * wave + c, col);
        const Two wr = tile.dw(16 * wave + c, col);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j > wave) continue;
          dP[j] = M::mma(yr, ua[j], dP[j]);
          dE[j] = M::mma(wr, ua[j], dE[j]);
        }
      }
    }
    db += __shfl_xor(db, 1, 64);
    db += __shfl_xor(db, 2, 64);
    if ((tid & 3) == 0) sDb[tid >> 2] = db;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sd += __shfl_xor(sd, o, 64);
    if (lane == 0) sSD[wave] = sd;

    // Gram products of rows 16 wave ..
    f32x4_t kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero4;
    for (int s = 0; s * 32 < N; ++s) {
      const int col = 32 * s + 8 * g;
      auto load = [&](const T* base, int64_t stride, int i) {
        const int t = 16 * i + c;
        return t >= begin && t < end && col < N ? M::global8(base + t * stride + col) : M::zero();
      };
      const One ka = load(kbase, a.rows.k, wave), qa = load(qbase, a.rows.q, wave);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > wave) continue;
        const One kb = load(kbase, a.rows.k, j);
        kk[j] = M::mma(ka, kb, kk[j]);
        qk[j] = M::mma(qa, kb, qk[j]);
      }
    }
    __syncthreads();  // the tile's place is the matrices' from here
    float rz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = 16 * j + c;
      float cz = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * wave + 4 * g + r;
        float m1 = 0.f, m2 = 0.f, lo = 0.f, up = 0.f;
        if (j <= wave && s >= begin && s <= t && t < end) {
          const float rel = fast_exp2((float)(sG[t] - sG[s]));
          const float dqk = rel * dP[j][r];
          m1 = dqk * sRk[s];
          m2 = dqk * sRq[t];
          if (s < t) {
            const float dkk = -rel * dE[j][r];
            lo = dkk * sRk[s];
            up = dkk * sRk[t];
            const float z = m1 * sRq[t] * qk[j][r] + lo * sRk[t] * kk[j][r];
            rz[r] += z;
            cz += z;
          }
        }
        M1[t][s] = m1;
        M2[t][s] = m2;
        if (j <= wave) {
          if (s < t || j < wave) M3[t][s] = lo;
          if (s < t) M3[s][t] = up;
          if (s == t) M3[t][s] = 0.f;
        }
      }
      cz += __shfl_xor(cz, 16, 64);
      cz += __shfl_xor(cz, 32, 64);
      if (g == 0) colZ[wave][s] = cz;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float z = sum16(rz[r]);
      if (c == 0) rowZ[16 * wave + 4 * g + r] = z;
    }
    __syncthreads();
    // dq and dk of the wave's columns
    float rs[4][4], cd[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) rs[i][r] = cd[i][r] = 0.f;
    One kb[NTW][2], qb[NTW][2];
#pragma unroll
    for (int m = 0; m < NTW; ++m) {
      const int nn = 16 * (wave + 4 * m) + c;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float kv[8], qv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 32 * s + 16 * (e / 4) + 4 * g + e % 4;
          const bool on = nn < N && t >= begin && t < end;
          kv[e] = on ? M::IO::get(kbase[t * a.rows.k + nn]) : 0.f;
          qv[e] = on ? M::IO::get(qbase[t * a.rows.q + nn]) : 0.f;
          const int i = 2 * s + e / 4, r = e % 4;
          const float in = on ? sIn[t] : 0.f, kout = on ? sKout[t] : 0.f;
          const float x = in * qS[m][i][r], y = in * wS[m][i][r], z = uD[m][i][r];
          rs[i][r] += (sRq[t] * qv[e]) * x - (sRk[t] * kv[e]) * y;
          cd[i][r] = fmaf(kout * kv[e], z, cd[i][r]);
          qS[m][i][r] = x;
          wS[m][i][r] = (kout / sRk[t]) * z - y;
        }
        kb[m][s] = M::one(kv);
        qb[m][s] = M::one(qv);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = sum16(rs[i][r]), y = sum16(cd[i][r]);
        if (c == 0) {
          rowS[wave][16 * i + 4 * g + r] = x;
          colD[wave][16 * i + 4 * g + r] = y;
        }
      }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[8];
        if (2 * s <= i) {  // rows 16 i .. of M1, columns 32 s ..
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = M1[16 * i + c][32 * s + 16 * (e / 4) + 4 * g + e % 4];
          const Two f = M::two(v);
#pragma unroll
          for (int m = 0; m < NTW; ++m) qS[m][i] = M::mma(f, kb[m][s], qS[m][i]);
        }
        if (i < 2 * s + 2) {  // columns 16 i .. of M2, rows 32 s ..
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = M2[32 * s + 16 * (e / 4) + 4 * g + e % 4][16 * i + c];
          const Two f = M::two(v);
#pragma unroll
          for (int m = 0; m < NTW; ++m) wS[m][i] = M::mma(f, qb[m][s], wS[m][i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = M3[16 * i + c][32 * s + 16 * (e / 4) + 4 * g + e % 4];
        const Two f = M::two(v);
#pragma unroll
        for (int m = 0; m < NTW; ++m) wS[m][i] = M::mma(f, kb[m][s], wS[m][i]);
      }
    float* dq = reinterpret_cast<float*>(a.ws + ws.dq) + bhw * kC * N;
    float* dk = reinterpret_cast<float*>(a.ws + ws.dk) + bhw * kC * N;
#pragma unroll
    for (int m = 0; m < NTW; ++m) {
      const int nn = 16 * (wave + 4 * m) + c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          if (nn < N && t >= begin && t < end) {
            dq[t * N + nn] = qS[m][i][r];
            dk[t * N + nn] = wS[m][i][r];
          }
        }
    }
    __syncthreads();
    if (wave == 0) {
      const bool on = lane >= begin && lane < end;
      auto waves = [&](float(*q)[kC]) { return ((q[0][lane] + q[1][lane]) + q[2][lane]) + q[3][lane]; };
      double x = on ? (double)rowZ[lane] - waves(colZ) + waves(rowS) : 0.0, y = on ? (double)waves(colD) : 0.0;
      const double mine = y;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double ox = __shfl_down(x, off, 64), oy = __shfl_up(y, off, 64);
        if (lane + off < 64) x += ox;
        if (lane >= off) y += oy;
      }
      const float whole = first && last ? sIn[end - 1] * (((sSD[0] + sSD[1]) + sSD[2]) + sSD[3]) : 0.f;
      float dg = (float)(x + (y - mine) + (double)whole);
      if (VL && lane == begin && (cuts.fresh >> begin & 1)) dg = 0.f;  // nothing comes in
      float pa = 0.f, pb = 0.f;
      if (on) {
        const int64_t t = row + t0 + lane;
        float raw = M::IO::get(static_cast<const T*>(a.dt)[t * a.rows.dt + h]);
        if (a.dt_bias) raw += a.dt_bias[h];
        const float step = a.softplus ? softplus2(raw * kLog2e) * kLn2 : raw;
        float d = dg * a.A[h];
        if (a.softplus) d *= sigmoid(raw);
        pa = dg * step;
        pb = d;
        static_cast<T*>(a.ddt)[t * a.grows.dt + h] = M::IO::put(d);
        float e = sDb[lane];
        if (a.sigmoid) {
          const float be = sBeta[lane];
          e *= be * (1.f - be);
        }
        static_cast<T*>(a.dbeta)[t * a.grows.beta + h] = M::IO::put(e);
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        pa += __shfl_xor(pa, o, 64);
        pb += __shfl_xor(pb, o, 64);
      }
      sumA += pa;
      sumB += pb;
    }
    begin = end;
  }
  if (tid == 0) {
    float* part = reinterpret_cast<float*>(a.ws + ws.part) + 2 * ((b * ws.nw + win) * a.H + h);
    part[0] = sumA;
    part[1] = sumB;
  }
}

// ---------------------------------------------------------------- heads of a group together, unit length
// A wave a (token, key group); blockIdx.y: q or k.
template <class IO>
__global__ __launch_bounds__(256) void delta_finish_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename IO::type T;
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= a.B * a.L * a.G) return;
  const int64_t grp = i % a.G, t = i / a.G, b = t / a.L, tl = t % a.L;
  const bool isk = blockIdx.y;
  const int N = (int)a.N, rep = (int)(a.H / a.G);
  const T* x = static_cast<const T*>(isk ? a.k : a.q) + t * (isk ? a.rows.k : a.rows.q) + grp * N;
  T* out = static_cast<T*>(isk ? a.dk : a.dq) + t * (isk ? a.grows.k : a.grows.q) + grp * N;
  const float* d = reinterpret_cast<const float*>(a.ws + (isk ? ws.dk : ws.dq));
  const float scale = isk ? 1.f : a.scale;
  constexpr int E = (int)kDeltaMaxDim / 64;
  float v[E], xv[E], ss = 0.f, dot = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int nn = lane + 64 * e;
    v[e] = xv[e] = 0.f;
    if (nn < N) {
      for (int r = 0; r < rep; ++r)
        v[e] += d[(((b * a.H + grp * rep + r) * ws.nw + tl / kC) * kC + tl % kC) * N + nn];
      v[e] *= scale;
      xv[e] = IO::get(x[nn]);
    }
    ss = fmaf(xv[e], xv[e], ss);
    dot = fmaf(xv[e], v[e], dot);
  }
  float rn = 1.f, back = 0.f;
  if (a.qk_norm) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      ss += __shfl_xor(ss, o, 64);
      dot += __shfl_xor(dot, o, 64);
    }
    rn = 1.f / sqrtf(ss + kQkEps);
    back = dot * rn * rn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 64 * e < N) out[lane + 64 * e] = IO::put(rn * (v[e] - xv[e] * back));
}

// dA and ddt_bias: a block a head, the windows' sums in a fixed order.
__global__ __launch_bounds__(256) void delta_param_kernel(DeltaArgs a, DeltaWs ws) {
  __shared__ float red[2][256];
  const int64_t h = blockIdx.x;
  const float* part = reinterpret_cast<const float*>(a.ws + ws.part);
  float x = 0.f, y = 0.f;
  for (int64_t i = threadIdx.x; i < a.B * ws.nw; i += 256) {
    x += part[2 * (i * a.H + h)];
    y += part[2 * (i * a.H + h) + 1];
  }
  red[0][threadIdx.x] = x;
  red[1][threadIdx.x] = y;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) {
      red[0][threadIdx.x] += red[0][threadIdx.x + o];
      red[1][threadIdx.x] += red[1][threadIdx.x + o];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.dA[h] = red[0][0];
    if (a.ddt_bias) a.ddt_bias[h] = red[1][0];
  }
}

// ---------------------------------------------------------------- launches
size_t delta_backward_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
  return delta_ws(B, L, H, N, P, true).total;
}

template <class M, int NP, bool VL>
static hipError_t reverse(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_reverse_kernel<M, NP, VL>;
  const size_t lds = rev_lds<M, NP>();
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const int w = delta_chain_waves(a.B, a.H, a.P);
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * (a.P / 16 / w))), dim3(64 * w), lds, s, a, ws);
  return hipGetLastError();
}
template <int NP, int C, bool VL>
static hipError_t reverse_bf16(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_reverse_bf16_kernel<NP, C, VL>;
  const size_t lds = ReverseLds<NP, C>::total;
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * (a.P / 16 / C))), dim3(128 * C), lds, s, a, ws);
  return hipGetLastError();
}
template <class M, int NP, bool VL>
static hipError_t reverse_at(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  if constexpr (sizeof(typename M::IO::type) == 2 && NP <= 128)
    return a.P % 32 == 0 ? reverse_bf16<NP, 2, VL>(a, ws, s) : reverse_bf16<NP, 1, VL>(a, ws, s);
  else
    return reverse<M, NP, VL>(a, ws, s);
}
template <class M, int NTW, bool VL>
static hipError_t grad(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_grad_kernel<M, NTW, VL>;
  const size_t lds = grad_lds<M>();
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * ws.nw * a.H)), dim3(256), lds, s, a, ws);
  return hipGetLastError();
}
template <class M, bool VL>
static hipError_t back_of(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  hipError_t e = a.N <= 32    ? reverse_at<M, 32, VL>(a, ws, s)
                 : a.N <= 64  ? reverse_at<M, 64, VL>(a, ws, s)
                 : a.N <= 128 ? reverse_at<M, 128, VL>(a, ws, s)
                              : reverse_at<M, 256, VL>(a, ws, s);
  if (e != hipSuccess) return e;
  e = a.N <= 64 ? grad<M, 1, VL>(a, ws, s) : a.N <= 128 ? grad<M, 2, VL>(a, ws, s) : grad<M, 4, VL>(a, ws, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(delta_finish_kernel<typename M::IO>, dim3((unsigned)((a.B * a.L * a.G + 3) / 4), 2), dim3(256), 0,
                     s, a, ws);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(delta_param_kernel, dim3((unsigned)a.H), dim3(256), 0, s, a, ws);
  return hipGetLastError();
}

hipError_t launch_delta_backward(const DeltaArgs& a, bool bf16, hipStream_t s) {
  const DeltaWs ws = delta_ws(a.B, a.L, a.H, a.N, a.P, true);
  hipError_t e = launch_delta_prepare(a, ws, true, bf16, s);
  if (e == hipSuccess) e = launch_delta_chain(a, ws, true, bf16, s);
  if (e != hipSuccess) return e;
  if (bf16) return a.seq_idx ? back_of<DeltaB, true>(a, ws, s) : back_of<DeltaB, false>(a, ws, s);
  return a.seq_idx ? back_of<DeltaF, true>(a, ws, s) : back_of<DeltaF, false>(a, ws, s);
}

}  // namespace ssd
