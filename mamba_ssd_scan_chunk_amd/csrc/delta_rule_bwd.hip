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
// Six launches: the preparation and the forward chain (delta_rule.hip), which
// leave the states in front of the windows and w; delta_reverse_kernel, a wave
// 16 value columns as there, which leaves D of every window and du;
// delta_grad_kernel, a block a (window, head), all windows at once;
// delta_finish_kernel, which adds the heads of a key group and takes the
// gradients through the unit length; and delta_param_kernel, which adds dA and the
// bias' gradient over the windows.
#include "delta_rule.hpp"

namespace ssd {

constexpr int kTP = kC + 4;

// ---------------------------------------------------------------- the chain, back to front
// fp32 products, and bf16 inputs of more than 128 key columns; the waves as in the
// forward's general chain.  2 x 777 tokens, N = 48, P = 80, fp32: 96 us, the
// length of the chain (224 where every wave staged for itself).
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
  constexpr int NT = NP / 16, KS = NP / 32, LP = rev_pitch<M, NP>();
  extern __shared__ __align__(16) char lds[];
  T* kt = reinterpret_cast<T*>(lds);
  T* qt = kt + kC * LP;
  float* gt = reinterpret_cast<float*>(qt + kC * LP);
  const float *sBeta = gt, *sKin = gt + kC, *sQin = gt + 2 * kC, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = chain_columns(a.P), c = lane & 15, g = lane >> 4;
  const bool column = wave < w;
  const uint32_t bid = near_block(blockIdx.x, gridDim.x);
  const uint32_t slices = (uint32_t)(a.P / 16) / w;
  const int64_t bh = bid / slices, h = bh % a.H, b = bh / a.H, grp = h / (a.H / a.G);
  const int64_t p = ((bid % slices) * w + wave) * 16 + c;
  const int N = (int)a.N;
  const int64_t row = b * a.L;

  f32x4_t D[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nn = 16 * j + 4 * g + r;
      D[j][r] = a.dfinal && column && nn < N ? a.dfinal[(bh * N + nn) * a.P + p] : 0.f;
    }

  for (int64_t win = ws.nw - 1; win >= 0; --win) {
    const int64_t t0 = win * kC, bhw = bh * ws.nw + win;
    const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC);
    Cuts cuts = {0, 0};
    if constexpr (VL) cuts = window_cuts(a.seq_idx, Wanted{}, row, t0, a.L, lane);
    {
      float* out = reinterpret_cast<float*>(a.ws + ws.D) + bhw * N * a.P + p;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int nn = 16 * j + 4 * g + r;
          if (column && nn < N) out[nn * a.P] = D[j][r];
        }
    }
    const char* fr = a.ws + ws.up_r + bhw * kTriBytes;
    const char* fp = a.ws + ws.up_p + bhw * kTriBytes;
    int end = n;
    while (end > 0) {
      const int begin = VL ? piece_begin(cuts.piece, end) : 0;
      const T* kb = static_cast<const T*>(a.k) + (row + t0) * a.rows.k + grp * N;
      const T* qb = static_cast<const T*>(a.q) + (row + t0) * a.rows.q + grp * N;
      if (!column) {
        const float* gates = reinterpret_cast<const float*>(reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw);
        const int st = tid - 64 * w, sn = 256 - 64 * w;
        Stager<M, NP, true> sg;
        sg.load(kb, (uint32_t)a.rows.k, qb, (uint32_t)a.rows.q, gates, N, n, begin, end, st, sn);
        __syncthreads();
        sg.store(kt, qt, gt, LP, kb, (uint32_t)a.rows.k, qb, (uint32_t)a.rows.q, N, n, begin, end, st, sn);
        __syncthreads();
        end = begin;
        continue;
      }
      // asked for before the rows are there, where there are registers for it (above 128 it spills)
      constexpr bool kEarly = NP < 256;
      Two rf[kTriFrags], pf[kTriFrags];
      uint32_t yq[16];
#pragma unroll
      for (int f = 0; f < kTriFrags; ++f)
        if constexpr (kEarly) {
          rf[f] = M::load(fr + f * 2048, lane);
          pf[f] = M::load(fp + f * 2048, lane);
        }
      load_column<typename M::IO>(static_cast<const T*>(a.dy) + ((row + t0) * a.H + h) * a.P, (uint32_t)(a.H * a.P), p, n,
                                  begin, end, g, yq);
      __syncthreads();
      __syncthreads();

      f32x4_t dy[4], du[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dy[i][r] = column_value<typename M::IO>(yq[4 * i + r]);
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
        for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(kEarly ? pf[up_frag(i, s)] : M::load(fp + up_frag(i, s) * 2048, lane), yb, du[i]);
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
        for (int i = 0; i < 2 * s + 2; ++i) du[i] = M::mma(kEarly ? rf[up_frag(i, s)] : M::load(fr + up_frag(i, s) * 2048, lane), xb[s], du[i]);
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
        if (column && nn < N) a.dinit[(bh * N + nn) * a.P + p] = D[j][r];
      }
  }
}

// ---------------------------------------------------------------- the same of bf16 inputs
// C column waves and C stagers, as in the forward chain, and C waves that work
// out a step ahead what the next piece adds whatever D is, P^T dy to its values
// and q^T diag(e^G) dy to D, and leave it in LDS as accumulators.  Bound by the
// column waves' latency: 2 x 2048 tokens of 32 heads, N = P = 128, 136 us, 4.2 a
// window (858 with waves that do everything; waves wait for 57% of their cycles
// and the matrix units are busy 8%).
template <int NP, int C>
struct ReverseLds {
  static constexpr int kPitch = NP + 24;  // rows as the products read them begin in different banks
  static constexpr int kRows = kC * kPitch * 2;
  static constexpr int kX = (NP / 16 + 4) * 1024;
  static constexpr int k = 0, r = k + kRows, g = r + kTriBytes, half = g + 5 * kC * 4;
  static constexpr int q = 2 * half, x = q + 2 * kRows, total = x + 2 * C * kX;
};

template <int NP, int C, bool VL>
__global__ __launch_bounds__(chain_threads(C), C) void delta_reverse_bf16_kernel(DeltaArgs a, DeltaWs ws) {
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

  auto gates = [&](const Pieces& s) {
    return reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bh * ws.nw + s.win;
  };
  if (wave >= first_stager(C)) {
    // ---- stager.  Step j: piece j + 1 for the column waves, q of piece j + 2
    const int ht = tid - 64 * first_stager(C);
    RowTile<NP, NH> kt, qt;
    TriTile<NH> rt;
    GateTile<NH> gt;
    const uint32_t krow = (uint32_t)a.rows.k, qrow = (uint32_t)a.rows.q;
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + row * a.rows.k + grp * N;
    const uint16_t* qb = static_cast<const uint16_t*>(a.q) + row * a.rows.q + grp * N;
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
    ask(pc);
    ask_q(pc);
    put(pc, 0);
    put_q(pc, 0);
    Pieces n1 = pc;  // whose k, R and gates are under way
    n1.step_back();
    Pieces n2 = n1;  // whose q is
    if (n1.valid_back()) {
      ask_q(n1);
      ask(n1);
      n2.step_back();
    }
    __syncthreads();
    if (n1.valid_back()) put_q(n1, 1);
    if (n1.valid_back() && n2.valid_back()) ask_q(n2);
    __syncthreads();
    for (int j = 0; pc.valid_back(); ++j) {
      if (n1.valid_back()) put(n1, (j + 1) & 1);
      if (n2.valid_back()) put_q(n2, j & 1);
      pc = n1;
      n1 = n2;
      if (n2.valid_back()) {
        ask(n1);
        n2.step_back();
        if (n2.valid_back()) ask_q(n2);
      }
      __syncthreads();
    }
    return;
  }
  if (wave >= 2 * C) return;
  if (wave >= C) {
    // ---- a step ahead of the column waves: pc is the piece worked out
    const uint32_t yrow = (uint32_t)(a.H * a.P);
    Column dy;
    f32x4_t qin[4];
    Two pf[kTriFrags];
    auto ask = [&](const Pieces& s) {
      dy.load(static_cast<const uint16_t*>(a.dy) + ((row + s.win * kC) * a.H + h) * a.P, yrow, 4 * g * yrow + p, s.n);
#pragma unroll
      for (int i = 0; i < 4; ++i) qin[i] = *reinterpret_cast<const f32x4_t*>(gates(s)->qin + 16 * i + 4 * g);
    };
    auto ask_p = [&](const Pieces& s) {
      const char* fp = a.ws + ws.up_p + (bh * ws.nw + s.win) * kTriBytes;
#pragma unroll
      for (int f = 0; f < kTriFrags; ++f) pf[f] = M::load(fp + f * 2048, lane);
    };
    ask(pc);
    ask_p(pc);
    __syncthreads();
    for (int half = 0;; half ^= 1) {
      const uint16_t* ql = reinterpret_cast<const uint16_t*>(lds + Lay::q + half * Lay::kRows);
      char* x = lds + Lay::x + (half * C + wave % C) * Lay::kX;
      One yb[2], qT[2][NT];
      Two wb[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float v[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 2 * t + e / 4, r = e % 4, tok = 16 * i + 4 * g + r;
          const bool on = !VL || (tok >= pc.begin && tok < pc.end);
          v[e] = on ? dy.get(i, r) : 0.f;
          w[e] = on ? qin[i][r] * v[e] : 0.f;
        }
        yb[t] = M::one(v);
        wb[t] = M::two(w);
#pragma unroll
        for (int j = 0; j < NT; ++j) qT[t][j] = M::transposed(ql + 32 * t * LP + 16 * j, LP, lane);
      }
      __builtin_amdgcn_sched_barrier(0);
      Pieces nx = pc;
      nx.step_back();
      if (nx.valid_back()) ask(nx);
      f32x4_t Y[NT], py[4];
#pragma unroll
      for (int j = 0; j < NT; ++j) Y[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) py[i] = Y[0];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int j = 0; j < NT; ++j) Y[j] = M::mma(qT[t][j], wb[t].lo, Y[j]);
#pragma unroll
        for (int j = 0; j < NT; ++j) Y[j] = M::mma(qT[t][j], wb[t].hi, Y[j]);
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
      if (nx.valid_back()) ask_p(nx);
      pc = nx;
      __syncthreads();
      if (!pc.valid_back()) break;
    }
    __syncthreads();  // the column waves' last step
    return;
  }

  // ---- column wave
  __builtin_amdgcn_s_setprio(3);
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
// The products over value columns go a slice of 64 columns at a time, every
// operand of the slice asked for before the one in front is worked out; the 64 x
// 64 matrices are rounded once a block and shared by its eight waves.  Bound by
// issue and LDS: 2 x 2048 tokens of 32 heads, N = P = 128, 250 us, 145 of them in
// the slices; its traffic (S, D and w, du in fp32) alone is about 110.

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
  __device__ __forceinline__ DeltaB::One dy(int t, int col) const { return DeltaB::row8(p + t * kPitch + col); }
  __device__ __forceinline__ DeltaB::Two two(int plane, int t, int col) const {
    DeltaB::Two x;
    x.hi = DeltaB::row8(p + plane * kPlane + t * kPitch + col);
    x.lo = DeltaB::row8(p + (plane + 1) * kPlane + t * kPitch + col);
    return x;
  }
  __device__ __forceinline__ DeltaB::Two u(int t, int col) const { return two(1, t, col); }
  __device__ __forceinline__ DeltaB::Two dw(int t, int col) const { return two(3, t, col); }
};
struct GradTileF {
  static constexpr int kPitch = 68, kPlane = kC * kPitch;
  float* p;  // dy, u, dw
  __device__ __forceinline__ explicit GradTileF(char* lds) : p(reinterpret_cast<float*>(lds)) {}
  static constexpr size_t bytes() { return (size_t)3 * kPlane * 4; }
  __device__ __forceinline__ void put8(int t, int col, const float* dy, const float* u, const float* dw) {
    float* q = p + t * kPitch + col;
    Lds<OpF32>::store8(q, dy);
    Lds<OpF32>::store8(q + kPlane, u);
    Lds<OpF32>::store8(q + 2 * kPlane, dw);
  }
  __device__ __forceinline__ DeltaF::One dy(int t, int col) const { return DeltaF::row8(p + t * kPitch + col); }
  __device__ __forceinline__ DeltaF::Two u(int t, int col) const { return DeltaF::row8(p + kPlane + t * kPitch + col); }
  __device__ __forceinline__ DeltaF::Two dw(int t, int col) const {
    return DeltaF::row8(p + 2 * kPlane + t * kPitch + col);
  }
};
template <> struct GradTile<DeltaF> : GradTileF { using GradTileF::GradTileF; };
template <> struct GradTile<DeltaW> : GradTileF { using GradTileF::GradTileF; };
// The token-by-token matrices as left operands: M1 lower, M2 upper triangular, M3 whole.
constexpr int kGradFrags = 2 * kTriFrags + 8;
template <class M, int WV>
constexpr size_t grad_lds() {
  const size_t tile = GradTile<M>::bytes(), tri = (size_t)3 * kC * kTP * 4;
  return (tile > tri ? tile : tri) + kGradFrags * 2048 + kC * 8 + (size_t)(7 + 3 * WV + 2 + 1) * kC * 4 + 16 * 4;
}

// Sum over the 16 lanes of a group, in every lane.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// WV waves; a wave takes NTW 16-row tiles of the state (dq and dk columns) for
// all 64 tokens, and 16 rows of the token-by-token matrices: of both where four
// waves share them, of dQK (the first four) or dKK (the others) where eight do,
// which leaves each the registers for two waves a SIMD.
template <class M, int WV, int NTW, bool VL>
__global__ __launch_bounds__(64 * WV, 2) void delta_grad_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename M::IO::type T;
  typedef typename M::One One;
  typedef typename M::Two Two;
  constexpr uint32_t es = sizeof(T);
  constexpr int kParts = WV == 4 ? 2 : 1, kCols = 64 / WV;  // matrices a wave; columns a thread stages
  extern __shared__ __align__(16) char lds[];
  constexpr size_t kBig = GradTile<M>::bytes() > (size_t)3 * kC * kTP * 4 ? GradTile<M>::bytes() : (size_t)3 * kC * kTP * 4;
  GradTile<M> tile(lds);
  float(*M1)[kTP] = reinterpret_cast<float(*)[kTP]>(lds);
  float(*M2)[kTP] = M1 + kC;
  float(*M3)[kTP] = M2 + kC;
  char* frags = lds + kBig;
  double* sG = reinterpret_cast<double*>(frags + kGradFrags * 2048);
  float* gt = reinterpret_cast<float*>(sG + kC);
  const float *sBeta = gt, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC, *sRk = gt + 5 * kC, *sRq = gt + 6 * kC;
  float(*rowS)[kC] = reinterpret_cast<float(*)[kC]>(gt + 7 * kC);  // by wave
  float(*colD)[kC] = rowS + WV;
  float(*colZ)[kC] = colD + WV;
  float(*rowZ)[kC] = colZ + WV;  // by matrix
  float* sDb = reinterpret_cast<float*>(rowZ + 2);
  float* sSD = sDb + kC;  // by wave

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4, rt = wave & 3;  // rt: the row tile of the matrices
  auto which = [&](int part) { return WV == 4 ? part : wave >> 2; };  // 0: dQK, 1: dKK
  const uint32_t bid = near_block(blockIdx.x, gridDim.x), H = (uint32_t)a.H, nw = (uint32_t)ws.nw;
  const int64_t h = bid % H, win = bid / H % nw, b = bid / H / nw;
  const int64_t row = b * a.L, t0 = win * kC, bhw = (b * a.H + h) * ws.nw + win;
  const int64_t grp = (uint32_t)h / (H / (uint32_t)a.G);
  const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC), N = (int)a.N, P = (int)a.P;
  Cuts cuts = {0, 0};
  if constexpr (VL) cuts = Pieces::uniform(reinterpret_cast<const Cuts*>(a.ws + ws.cuts)[b * ws.nw + win]);
  const DeltaGates* gates = reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw;
  for (int i = tid; i < 7 * kC / 4; i += 64 * WV)
    reinterpret_cast<f32x4_t*>(gt)[i] = reinterpret_cast<const f32x4_t*>(gates)[i];
  if (tid < kC) sG[tid] = gates->G[tid];
  const __amdgpu_buffer_rsrc_t wr = rows_of(reinterpret_cast<const float*>(a.ws + ws.w) + bhw * kC * P, kC * P * 4);
  const __amdgpu_buffer_rsrc_t ur = rows_of(reinterpret_cast<const float*>(a.ws + ws.du) + bhw * kC * P, kC * P * 4);
  const float* wsS = reinterpret_cast<const float*>(a.ws + ws.S) + bhw * N * P;
  const float* wsD = reinterpret_cast<const float*>(a.ws + ws.D) + bhw * N * P;
  const uint32_t krow = (uint32_t)a.rows.k * es, qrow = (uint32_t)a.rows.q * es, yrow = (uint32_t)(a.H * a.P) * es;
  const __amdgpu_buffer_rsrc_t kr =
      rows_of(static_cast<const T*>(a.k) + (row + t0) * a.rows.k + grp * N, (uint32_t)n * krow);
  const __amdgpu_buffer_rsrc_t qr =
      rows_of(static_cast<const T*>(a.q) + (row + t0) * a.rows.q + grp * N, (uint32_t)n * qrow);
  const __amdgpu_buffer_rsrc_t yr =
      rows_of(static_cast<const T*>(a.dy) + ((row + t0) * a.H + h) * P, (uint32_t)n * yrow);
  auto f4 = [](const __amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t s) {
    return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, s, 0));
  };
  auto input = [](uint32_t v) { return es == 2 ? bf16_bits_to_f32(v) : __uint_as_float(v); };
  float sumA = 0.f, sumB = 0.f;  // of dA and ddt_bias, in wave 0
  const f32x4_t zero4 = {0.f, 0.f, 0.f, 0.f};

  // PARTS: a piece of a window of several
  auto piece = [&](auto parts, const int begin, const int end) {
    constexpr bool PARTS = decltype(parts)::value;
    // only a row's first piece begins with a state, only its last one hands one on
    const bool first = begin == 0, last = end == n;
    const __amdgpu_buffer_rsrc_t Sr = rows_of(wsS, first ? N * P * 4 : 0), Dr = rows_of(wsD, last ? N * P * 4 : 0);
    f32x4_t qS[NTW][4], wS[NTW][4], uD[NTW][4], dX[kParts][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int q = 0; q < kParts; ++q) dX[q][i] = zero4;
#pragma unroll
      for (int m = 0; m < NTW; ++m) qS[m][i] = wS[m][i] = uD[m][i] = zero4;
    }
    float sd = 0.f, db = 0.f;
    for (int p0 = 0; p0 < P; p0 += 64) {
      // all of a slice's operands are asked for together
      f32x4_t sv[2][NTW][2], dv[2][NTW][2], w[kCols / 4], du[kCols / 4], dy[kCols / 4];
      {
        const int t = tid / WV, col = p0 + tid % WV * kCols;
        const uint32_t off = col < P ? (t * P + col) * 4 : kNowhere, yoff = col < P ? t * yrow + col * es : kNowhere;
#pragma unroll
        for (int e = 0; e < kCols / 4; ++e) {
          w[e] = f4(wr, off, 16 * e);
          du[e] = f4(ur, off, 16 * e);
          if (es == 4 || e < kCols / 8) dy[e] = f4(yr, yoff, 16 * e);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int col = p0 + 32 * s + 8 * g;
        const uint32_t off = col < P ? ((16 * wave + c) * P + col) * 4 : kNowhere;
#pragma unroll
        for (int m = 0; m < NTW; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sv[s][m][e] = f4(Sr, off, 16 * WV * m * P * 4 + 16 * e);
            dv[s][m][e] = f4(Dr, off, 16 * WV * m * P * 4 + 16 * e);
          }
      }
      __syncthreads();
      {
        const int t = tid / WV, col = tid % WV * kCols;
        const bool on = !PARTS || (t >= begin && t < end);
        const float beta = sBeta[t];
#pragma unroll
        for (int e = 0; e < kCols / 8; ++e) {
          float wv[8], uv[8], yv[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            wv[k] = w[2 * e + k / 4][k % 4];
            uv[k] = du[2 * e + k / 4][k % 4];
            if constexpr (es == 4) {
              yv[k] = dy[2 * e + k / 4][k % 4];
            } else {
              const uint32_t two = __float_as_uint(dy[e][k / 2]);
              yv[k] = __uint_as_float(k % 2 ? two & 0xffff0000u : two << 16);
            }
            if constexpr (PARTS) {
              wv[k] = on ? wv[k] : 0.f;
              uv[k] = on ? uv[k] : 0.f;
              yv[k] = on ? yv[k] : 0.f;
            }
            db = fmaf(wv[k], uv[k], db);
            wv[k] *= beta;
            uv[k] *= beta;
            if constexpr (PARTS) {  // another piece's b may be NaN
              wv[k] = on ? wv[k] : 0.f;
              uv[k] = on ? uv[k] : 0.f;
            }
          }
          tile.put8(t, col + 8 * e, yv, wv, uv);
        }
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (p0 + 32 * s >= P) break;
        const int col = 32 * s + 8 * g;
        Two sf[NTW], df[NTW];
#pragma unroll
        for (int m = 0; m < NTW; ++m) {
          float x[8], z[8];
          slots(sv[s][m][0], sv[s][m][1], x);
          slots(dv[s][m][0], dv[s][m][1], z);
#pragma unroll
          for (int k = 0; k < 8; ++k) sd = fmaf(x[k], z[k], sd);
          sf[m] = M::two(x);
          df[m] = M::two(z);
        }
        const One ym = tile.dy(16 * rt + c, col);
        const Two wm = tile.dw(16 * rt + c, col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const One ya = tile.dy(16 * i + c, col);
          const Two ua = tile.u(16 * i + c, col), wa = tile.dw(16 * i + c, col);
#pragma unroll
          for (int m = 0; m < NTW; ++m) {
            qS[m][i] = M::mma(ya, sf[m], qS[m][i]);
            wS[m][i] = M::mma(wa, sf[m], wS[m][i]);
            uD[m][i] = M::mma(ua, df[m], uD[m][i]);
          }
          if (i > rt) continue;
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            if (which(q) == 0) dX[q][i] = M::mma(ym, ua, dX[q][i]);
            else dX[q][i] = M::mma(wm, ua, dX[q][i]);
          }
        }
      }
    }
    // q and k of the wave's columns, 16 tokens a lane, for what follows the matrices
    uint32_t kv[NTW][16], qv[NTW][16];
#pragma unroll
    for (int m = 0; m < NTW; ++m) {
      const uint32_t nn = 16 * (wave + WV * m) + c;
      const uint32_t ko = (int)nn < N ? 4 * g * krow + nn * es : kNowhere, qo = (int)nn < N ? 4 * g * qrow + nn * es : kNowhere;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t t = Column::row(e);
        if constexpr (es == 2) {
          kv[m][e] = __builtin_amdgcn_raw_buffer_load_b16(kr, ko, t * krow, 0);
          qv[m][e] = __builtin_amdgcn_raw_buffer_load_b16(qr, qo, t * qrow, 0);
        } else {
          kv[m][e] = __builtin_amdgcn_raw_buffer_load_b32(kr, ko, t * krow, 0);
          qv[m][e] = __builtin_amdgcn_raw_buffer_load_b32(qr, qo, t * qrow, 0);
        }
      }
    }
    // Gram products of rows 16 rt ..
    f32x4_t gm[kParts][4];
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) gm[q][j] = zero4;
    for (int s0 = 0; 32 * s0 < N; s0 += 2) {
      One kf[4][2], xa[kParts][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t col = 32 * (s0 + s) + 8 * g;
        const uint32_t ko = (int)col < N ? c * krow + col * es : kNowhere, qo = (int)col < N ? c * qrow + col * es : kNowhere;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          xa[q][s] = which(q) == 0 ? M::rows8(qr, qo, 16 * rt * qrow) : M::rows8(kr, ko, 16 * rt * krow);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= rt) kf[j][s] = M::rows8(kr, ko, 16 * j * krow);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j > rt) continue;
#pragma unroll
          for (int q = 0; q < kParts; ++q) gm[q][j] = M::mma(xa[q][s], kf[j][s], gm[q][j]);
        }
    }
#pragma unroll
    for (int o = 1; o < WV; o <<= 1) db += __shfl_xor(db, o, 64);
    if (tid % WV == 0) sDb[tid / WV] = db;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sd += __shfl_xor(sd, o, 64);
    if (lane == 0) sSD[wave] = sd;
    __syncthreads();  // the tile's place is the matrices' from here
    {
      const int tw = 16 * rt + 4 * g;
      double Gt[4];
      float rkt[4], rqt[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) Gt[r] = sG[tw + r];
      load_vec<IoF32, 4>(sRk + tw, rkt);
      load_vec<IoF32, 4>(sRq + tw, rqt);
      float cz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        float rz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = 16 * j + c;
          const double Gs = sG[s];
          const float rks = sRk[s];
          f32x4_t v;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = tw + r;
            const bool on = j <= rt && s >= begin && s <= t && t < end, below = on && s < t;
            v[r] = fast_exp2((float)(Gt[r] - Gs)) * dX[q][j][r];
            const float x = v[r] * rks;  // of s's unit key
            const float z = below ? x * (which(q) == 0 ? rqt[r] : -rkt[r]) * gm[q][j][r] : 0.f;
            rz[r] += z;
            cz[j] += z;
            if (which(q) == 0) {
              M1[t][s] = on ? x : 0.f;
              M2[t][s] = on ? v[r] * rqt[r] : 0.f;
            } else {
              if (j < rt || (j == rt && s <= t)) M3[t][s] = below ? -x : 0.f;
              v[r] = below ? -v[r] * rkt[r] : 0.f;
            }
          }
          if (which(q) == 1) {
            if (j < rt) {
              *reinterpret_cast<f32x4_t*>(&M3[s][tw]) = v;
            } else if (j == rt) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (s < tw + r) M3[s][tw + r] = v[r];
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float z = sum16(rz[r]);
          if (c == 0) rowZ[which(q)][tw + r] = z;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cz[j] += __shfl_xor(cz[j], 16, 64);
        cz[j] += __shfl_xor(cz[j], 32, 64);
        if (g == 0) colZ[wave][16 * j + c] = cz[j];
      }
    }
    __syncthreads();
    // the matrices as operands, each rounded by one wave
    for (int f = wave; f < kGradFrags; f += WV) {
      const bool up = f >= kTriFrags && f < 2 * kTriFrags;
      float v[8];
      if (up) {  // columns 16 i .. of M2, rows 32 s ..
        const int u = f - kTriFrags, i = u < 4 ? u / 2 : u - 2, s = u < 4 ? u % 2 : 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = M2[32 * s + 16 * (e / 4) + 4 * g + e % 4][16 * i + c];
      } else {  // rows 16 i .. of M1 or M3, columns 32 s ..
        const int l = f - 2 * kTriFrags;
        const bool m3 = l >= 0;
        const int i = m3 ? l / 2 : f < 2 ? f : 2 + (f - 2) / 2, s = m3 ? l % 2 : f < 2 ? 0 : (f - 2) % 2;
        const float* q = m3 ? &M3[16 * i + c][32 * s + 4 * g] : &M1[16 * i + c][32 * s + 4 * g];
        load_vec<IoF32, 4>(q, v);
        load_vec<IoF32, 4>(q + 16, v + 4);
      }
      M::store(frags + f * 2048, lane, M::two(v));
    }
    // dq and dk of the wave's columns
    One kb[NTW][2], qb[NTW][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * i + 4 * g;
      float in[4], ko[4], rk[4], rq[4], rs[4], cd[4];
      load_vec<IoF32, 4>(sIn + t, in);
      load_vec<IoF32, 4>(sKout + t, ko);
      load_vec<IoF32, 4>(sRk + t, rk);
      load_vec<IoF32, 4>(sRq + t, rq);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        rs[r] = cd[r] = 0.f;
        const bool on = !PARTS || (t + r >= begin && t + r < end);
        const float rest = ko[r] / rk[r];
#pragma unroll
        for (int m = 0; m < NTW; ++m) {
          if (PARTS && !on) kv[m][4 * i + r] = qv[m][4 * i + r] = 0;
          const float k = input(kv[m][4 * i + r]), q = input(qv[m][4 * i + r]);
          const float x = in[r] * qS[m][i][r], y = in[r] * wS[m][i][r], z = uD[m][i][r];
          rs[r] += (rq[r] * q) * x - (rk[r] * k) * y;
          cd[r] = fmaf(ko[r] * k, z, cd[r]);
          qS[m][i][r] = x;
          wS[m][i][r] = rest * z - y;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = sum16(rs[r]), y = sum16(cd[r]);
        if (c == 0) {
          rowS[wave][t + r] = x;
          colD[wave][t + r] = y;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < NTW; ++m)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = input(kv[m][8 * s + e]);
          y[e] = input(qv[m][8 * s + e]);
        }
        kb[m][s] = M::one(x);
        qb[m][s] = M::one(y);
      }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (2 * s <= i) {
          const Two f = M::load(frags + low_frag(i, s) * 2048, lane);
#pragma unroll
          for (int m = 0; m < NTW; ++m) qS[m][i] = M::mma(f, kb[m][s], qS[m][i]);
        }
        if (i < 2 * s + 2) {
          const Two f = M::load(frags + (kTriFrags + up_frag(i, s)) * 2048, lane);
#pragma unroll
          for (int m = 0; m < NTW; ++m) wS[m][i] = M::mma(f, qb[m][s], wS[m][i]);
        }
        const Two f = M::load(frags + (2 * kTriFrags + 2 * i + s) * 2048, lane);
#pragma unroll
        for (int m = 0; m < NTW; ++m) wS[m][i] = M::mma(f, kb[m][s], wS[m][i]);
      }
    const __amdgpu_buffer_rsrc_t dqr = rows_of(reinterpret_cast<float*>(a.ws + ws.dq) + bhw * kC * N, kC * N * 4);
    const __amdgpu_buffer_rsrc_t dkr = rows_of(reinterpret_cast<float*>(a.ws + ws.dk) + bhw * kC * N, kC * N * 4);
#pragma unroll
    for (int m = 0; m < NTW; ++m) {
      const uint32_t nn = 16 * (wave + WV * m) + c;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int t = (int)Column::row(e) + 4 * g;
        const bool on = (int)nn < N && (!PARTS || (t >= begin && t < end));
        const uint32_t off = on ? (4 * g * N + nn) * 4 : kNowhere;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(qS[m][e / 4][e % 4]), dqr, off, Column::row(e) * N * 4, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(wS[m][e / 4][e % 4]), dkr, off, Column::row(e) * N * 4, 0);
      }
    }
    __syncthreads();
    if (wave == 0) {
      const bool on = lane >= begin && lane < end;
      auto waves = [&](float(*q)[kC]) {
        float v = q[0][lane];
#pragma unroll
        for (int k = 1; k < WV; ++k) v += q[k][lane];
        return v;
      };
      double x = on ? (double)(rowZ[0][lane] + rowZ[1][lane]) - waves(colZ) + waves(rowS) : 0.0;
      double y = on ? (double)waves(colD) : 0.0;
      const double mine = y;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double ox = __shfl_down(x, off, 64), oy = __shfl_up(y, off, 64);
        if (lane + off < 64) x += ox;
        if (lane >= off) y += oy;
      }
      float whole = sSD[0];
#pragma unroll
      for (int k = 1; k < WV; ++k) whole += sSD[k];
      whole = first && last ? sIn[end - 1] * whole : 0.f;
      float dg = (float)(x + (y - mine) + (double)whole);
      if (VL && lane == begin && (cuts.fresh >> begin & 1)) dg = 0.f;  // nothing comes in
      float pa = 0.f, pb = 0.f;
      if (on) {
        const int64_t t = row + t0 + lane;
        float raw = M::IO::get(static_cast<const T*>(a.dt)[t * a.rows.dt + h]);
        const float be = M::IO::get(static_cast<const T*>(a.beta)[t * a.rows.beta + h]);
        if (a.dt_bias) raw += a.dt_bias[h];
        const float step = a.softplus ? softplus2(raw * kLog2e) * kLn2 : raw;
        float d = dg * a.A[h];
        if (a.softplus) d *= sigmoid(raw);
        pa = dg * step;
        pb = d;
        static_cast<T*>(a.ddt)[t * a.grows.dt + h] = M::IO::put(d);
        float e = sDb[lane];
        if (a.sigmoid) e *= sBeta[lane] * sigmoid(-be);  // near b = 1 the difference 1 - b has few bits
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
  };
  if (!VL || cuts.piece == 0) {
    piece(std::false_type(), 0, n);
  } else {
    for (int begin = 0, end; begin < n; begin = end) {
      end = piece_end(cuts.piece, begin, n);
      piece(std::true_type(), begin, end);
    }
  }
  if (tid == 0) {
    float* part = reinterpret_cast<float*>(a.ws + ws.part) + 2 * ((b * ws.nw + win) * a.H + h);
    part[0] = sumA;
    part[1] = sumB;
  }
}

// ---------------------------------------------------------------- heads of a group together, unit length
// W lanes of four columns a (token, key group); blockIdx.y: q or k.  Bound by
// memory: the heads' fp32 shares, read once (2 x 2048 tokens of 32 heads over 16,
// N = 128: 36 us, 4.6 TB/s).
template <class IO, int W>
__global__ __launch_bounds__(256) void delta_finish_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename IO::type T;
  const int l = threadIdx.x % W;
  const uint32_t i = blockIdx.x * (256 / W) + threadIdx.x / W, G = (uint32_t)a.G;
  if (i >= (uint64_t)(a.B * a.L * a.G)) return;
  const uint32_t grp = i % G, t = i / G, b = t / (uint32_t)a.L, tl = t % (uint32_t)a.L;
  const bool isk = blockIdx.y;
  const int N = (int)a.N, rep = (int)(a.H / a.G);
  const bool on = 4 * l < N;
  const T* x = static_cast<const T*>(isk ? a.k : a.q) + (int64_t)t * (isk ? a.rows.k : a.rows.q) + grp * N + 4 * l;
  T* out = static_cast<T*>(isk ? a.dk : a.dq) + (int64_t)t * (isk ? a.grows.k : a.grows.q) + grp * N + 4 * l;
  // heads of a group are nw windows of 64 rows apart
  const float* d = reinterpret_cast<const float*>(a.ws + (isk ? ws.dk : ws.dq)) +
                   ((((int64_t)b * a.H + (int64_t)grp * rep) * ws.nw + tl / kC) * kC + tl % kC) * N + 4 * l;
  const int64_t step = ws.nw * kC * N;
  float xv[4] = {0.f, 0.f, 0.f, 0.f};
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    load_vec<IO, 4>(x, xv);
#pragma unroll 4
    for (int r = 0; r < rep; ++r) v += *reinterpret_cast<const f32x4_t*>(d + r * step);
  }
  if (!isk) v *= a.scale;
  float ss = 0.f, dot = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ss = fmaf(xv[e], xv[e], ss);
    dot = fmaf(xv[e], v[e], dot);
  }
  float rn = 1.f, back = 0.f;
  if (a.qk_norm) {
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      ss += __shfl_xor(ss, o, 64);
      dot += __shfl_xor(dot, o, 64);
    }
    rn = 1.f / sqrtf(ss + kQkEps);
    back = dot * rn * rn;
  }
  if (!on) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = rn * (v[e] - xv[e] * back);
  if ((reinterpret_cast<uintptr_t>(out) & (4 * sizeof(T) - 1)) == 0) {
    float o[4] = {v[0], v[1], v[2], v[3]};
    store_vec<IO, 4>(out, o);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = IO::put(v[e]);
  }
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
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * (a.P / 16 / chain_columns(a.P)))), dim3(256), lds, s, a, ws);
  return hipGetLastError();
}
template <int NP, int C, bool VL>
static hipError_t reverse_bf16(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_reverse_bf16_kernel<NP, C, VL>;
  const size_t lds = ReverseLds<NP, C>::total;
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * (a.P / 16 / C))), dim3(chain_threads(C)), lds, s, a, ws);
  return hipGetLastError();
}
template <class M, int NP, bool VL>
static hipError_t reverse_at(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  if constexpr (std::is_same<M, DeltaB>::value && NP <= 128)
    return a.P % 32 == 0 ? reverse_bf16<NP, 2, VL>(a, ws, s) : reverse_bf16<NP, 1, VL>(a, ws, s);
  else
    return reverse<M, NP, VL>(a, ws, s);
}
template <class M, int WV, int NTW, bool VL>
static hipError_t grad(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_grad_kernel<M, WV, NTW, VL>;
  const size_t lds = grad_lds<M, WV>();
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * ws.nw * a.H)), dim3(64 * WV), lds, s, a, ws);
  return hipGetLastError();
}
template <class M, bool VL>
static hipError_t back_of(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  hipError_t e = a.N <= 32    ? reverse_at<M, 32, VL>(a, ws, s)
                 : a.N <= 64  ? reverse_at<M, 64, VL>(a, ws, s)
                 : a.N <= 128 ? reverse_at<M, 128, VL>(a, ws, s)
                              : reverse_at<M, 256, VL>(a, ws, s);
  if (e != hipSuccess) return e;
  e = a.N <= 64    ? grad<M, 4, 1, VL>(a, ws, s)
      : a.N <= 128 ? grad<M, 8, 1, VL>(a, ws, s)
                   : grad<M, 8, 2, VL>(a, ws, s);
  if (e != hipSuccess) return e;
  const int64_t units = a.B * a.L * a.G;
  if (a.N <= 64)
    hipLaunchKernelGGL((delta_finish_kernel<typename M::IO, 16>), dim3((unsigned)((units + 15) / 16), 2), dim3(256), 0, s, a, ws);
  else if (a.N <= 128)
    hipLaunchKernelGGL((delta_finish_kernel<typename M::IO, 32>), dim3((unsigned)((units + 7) / 8), 2), dim3(256), 0, s, a, ws);
  else
    hipLaunchKernelGGL((delta_finish_kernel<typename M::IO, 64>), dim3((unsigned)((units + 3) / 4), 2), dim3(256), 0, s, a, ws);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(delta_param_kernel, dim3((unsigned)a.H), dim3(256), 0, s, a, ws);
  return hipGetLastError();
}

template <class M>
static hipError_t back_as(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  return a.seq_idx ? back_of<M, true>(a, ws, s) : back_of<M, false>(a, ws, s);
}
hipError_t launch_delta_backward(const DeltaArgs& a, bool bf16, hipStream_t s) {
  const DeltaWs ws = delta_ws(a.B, a.L, a.H, a.N, a.P, true);
  hipError_t e = launch_delta_prepare(a, ws, true, bf16, s);
  if (e == hipSuccess) e = launch_delta_chain(a, ws, true, bf16, s);
  if (e != hipSuccess) return e;
  return !bf16 ? back_as<DeltaF>(a, ws, s) : a.f32_products ? back_as<DeltaW>(a, ws, s) : back_as<DeltaB>(a, ws, s);
}

}  // namespace ssd
