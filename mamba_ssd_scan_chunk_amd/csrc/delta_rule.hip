// delta_rule.hip -- the gated delta rule: prompts and single tokens.  The
// formulas and the operands' types are in delta_rule.hpp.
//
// A prompt takes two launches (long rows of few heads four, see
// delta_segments).  delta_prepare_kernel, one block a (window, head), leaves
// what needs no state: the triangular operands R and P, laid out as the chain's
// fragments, and the scalars of the rows.  The chain walks the windows in
// order.  A column wave owns 16 value columns of a head, whose
// state it holds in accumulators, and nothing passes between waves: every
// product of the chain contracts over what are rows of the one before (state
// rows, tokens), and an accumulator's rows are the contraction slots of the
// next operand.  Only k, q (from LDS, shared by a block's waves), R and P
// (from the workspace) are read as left operands.
#include "delta_rule.hpp"

namespace ssd {

// ---------------------------------------------------------------- preparation
constexpr int kTP = kC + 4;  // pitch of the 64 x 64 fp32 tiles in LDS
constexpr int kMP = 20;      // of a 16 x 16 one
constexpr int kPrepLds = kC * kTP * 4 + 4 * 16 * kMP * 4 + kC * 8 + 5 * kC * 4;

__device__ __forceinline__ f32x4_t mma4(const float4& a, const f32x4_t& b, f32x4_t c) {
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b[2], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b[3], c, 0, 0, 0);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

__device__ __forceinline__ Wanted wanted_states(const DeltaArgs& a, const DeltaWs& ws) {
  if (a.nseq <= 0) return {nullptr, nullptr};
  return {reinterpret_cast<const int*>(a.ws + ws.wanted), reinterpret_cast<const int*>(a.ws + ws.wanted_next)};
}

// e b where e is not zero: an entry between pieces stays zero whatever b is.
__device__ __forceinline__ float times(float e, float b) { return e != 0.f ? e * b : 0.f; }

// Four waves.  Wave i takes the Gram products of rows 16 i .. (BACK: of columns
// 16 i ..), so that its accumulators are P's (P^T's) fragments as they are,
// then column block i of R: with T = I + E diag(b) in blocks of 16,
//     R_ij = T_ii^-1 (-E_ij - sum_{j <= k < i} (E b)_ik R_kj),  T_ii^-1 = I + R_ii diag(b),
// the diagonal blocks by substitution, a lane a column, the others by fp32
// matrix instructions; R takes E's place in LDS.  Entries between pieces are
// set, not multiplied, to zero, so that no value of one sequence meets
// another's.  Bound by the latency of its few dependent parts: all of a
// wave's loads (of 128 key columns) are asked for together, and one matrix in
// LDS leaves five blocks a compute unit.  2 x 8192 tokens of 32 heads, bf16, N =
// 128: 117 us; for the gradients of 2 x 2048: 49; a lone block takes some 17.
template <class M, int NP, bool BACK, bool VL>
__global__ __launch_bounds__(256, 2) void delta_prepare_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename M::IO::type T;
  typedef typename M::One One;
  extern __shared__ __align__(16) char lds[];
  float(*E)[kTP] = reinterpret_cast<float(*)[kTP]>(lds);
  float(*R)[kTP] = E;
  float(*Md)[16][kMP] = reinterpret_cast<float(*)[16][kMP]>(E + kC);
  double* sG = reinterpret_cast<double*>(Md + 4);
  float* sBeta = reinterpret_cast<float*>(sG + kC);
  float* sIn = sBeta + kC;
  float* sOut = sIn + kC;
  float* sRk = sOut + kC;
  float* sRq = sRk + kC;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t bid = near_block(blockIdx.x, gridDim.x), H = (uint32_t)a.H, nw = (uint32_t)ws.nw;
  const int64_t h = bid % H, win = bid / H % nw, b = bid / H / nw;
  const int64_t row = b * a.L, t0 = win * kC, bhw = (b * a.H + h) * ws.nw + win;
  const int64_t grp = (uint32_t)h / (H / (uint32_t)a.G);
  const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC), N = (int)a.N;

  // the gates' inputs, a token a lane of wave 0
  float raw = 0.f, beta = 0.f;
  if (wave == 0) {
    const int64_t t = row + t0 + min(lane, n - 1);
    raw = M::IO::get(static_cast<const T*>(a.dt)[t * a.rows.dt + h]);
    beta = M::IO::get(static_cast<const T*>(a.beta)[t * a.rows.beta + h]);
  }
  // Gram products: kk[j], pq[j] of tiles (wave, j), the columns the wave's own
  // tokens (BACK: (j, wave), j >= wave)
  const T* kbase = static_cast<const T*>(a.k) + (row + t0) * a.rows.k + grp * N;
  const T* qbase = static_cast<const T*>(a.q) + (row + t0) * a.rows.q + grp * N;
  f32x4_t kk[4], pq[4], qq = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = pq[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int SL = NP / 32 < 4 ? NP / 32 : 4;
#pragma unroll
  for (int s0 = 0; s0 < NP / 32; s0 += SL) {
    One kf[4][SL], qf[BACK ? 4 : 1][SL], mine[SL];
    constexpr uint32_t es = sizeof(T);
    const uint32_t krow = (uint32_t)a.rows.k * es, qrow = (uint32_t)a.rows.q * es;
    const __amdgpu_buffer_rsrc_t kr = rows_of(kbase, (uint32_t)n * krow), qr = rows_of(qbase, (uint32_t)n * qrow);
    auto load = [&](const __amdgpu_buffer_rsrc_t r, uint32_t stride, int tile, int s) {
      const uint32_t col = 32 * s + 8 * g;
      return M::rows8(r, (int)col < N ? c * stride + col * es : kNowhere, 16 * tile * stride);
    };
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      mine[s] = load(qr, qrow, wave, s0 + s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BACK ? j < wave : j > wave) continue;
        kf[j][s] = load(kr, krow, j, s0 + s);
        if constexpr (BACK) qf[j][s] = load(qr, qrow, j, s0 + s);
      }
    }
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      One own = kf[0][s];
#pragma unroll
      for (int j = 1; j < 4; ++j)
        if (j == wave) own = kf[j][s];
      qq = M::mma(mine[s], mine[s], qq);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BACK ? j < wave : j > wave) continue;
        kk[j] = M::mma(kf[j][s], own, kk[j]);
        if constexpr (BACK) pq[j] = M::mma(qf[j][s], own, pq[j]);
        else pq[j] = M::mma(kf[j][s], mine[s], pq[j]);
      }
    }
  }
  Cuts both = {0, 0};
  if constexpr (VL) {
    both = window_cuts(a.seq_idx, BACK ? Wanted{} : wanted_states(a, ws), row, t0, a.L, lane);
    if (h == 0 && threadIdx.x == 0) reinterpret_cast<Cuts*>(a.ws + ws.cuts)[b * ws.nw + win] = both;
  }
  const uint64_t cuts = both.piece;
  auto same = [&](int t, int s) { return !VL || piece_of(cuts, t) == piece_of(cuts, s); };

  if (wave == 0) {
    const bool in = lane < n;
    if (a.dt_bias) raw += a.dt_bias[h];
    const float step = a.softplus ? softplus2(raw * kLog2e) * kLn2 : raw;
    float gv = step * a.A[h];
    if (gv < -1e5f) gv = -1e5f;  // e^gv is 0 well before; sums stay finite
    if (a.sigmoid) beta = sigmoid(beta);
    if (!in) gv = beta = 0.f;
    const int begin = VL ? piece_begin(cuts, lane + 1) : 0;
    const int end = VL ? piece_end(cuts, begin, n) : n;
    // in units of ln 2, and in 64 bits: differences of far tokens keep all of an exponent's bits
    double G = (double)gv * 1.4426950408889634;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_up(G, off, 64);
      if (lane - off >= begin) G += o;
    }
    const double last = __shfl(G, end - 1, 64);
    sG[lane] = G;
    sBeta[lane] = beta;
    sIn[lane] = in ? fast_exp2((float)G) : 0.f;
    sOut[lane] = in ? fast_exp2((float)(last - G)) : 0.f;
  }
  // lengths from the diagonals
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (c != 4 * g + r) continue;
    float k2 = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) k2 = j == wave ? kk[j][r] : k2;
    sRk[16 * wave + c] = a.qk_norm ? 1.f / sqrtf(k2 + kQkEps) : 1.f;
    sRq[16 * wave + c] = (a.qk_norm ? 1.f / sqrtf(qq[r] + kQkEps) : 1.f) * a.scale;
  }
  __syncthreads();
  {
    const int y = 16 * wave + c;
    const double Gy = sG[y];
    const float ry = sRk[y], qy = sRq[y];
    double Gx[4][4];
    float rx[4][4], qx[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = 16 * j + 4 * g;
#pragma unroll
      for (int r = 0; r < 4; ++r) Gx[j][r] = sG[x + r];
      load_vec<IoF32, 4>(sRk + x, rx[j]);
      if constexpr (BACK) load_vec<IoF32, 4>(sRq + x, qx[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool there = BACK ? j >= wave : j <= wave;  // on and below the diagonal
      f32x4_t e4;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int x = 16 * j + 4 * g + r, t = BACK ? x : y, s = BACK ? y : x;
        const bool on = there && s <= t && t < n && same(t, s);
        const float rel = fast_exp2((float)(BACK ? Gx[j][r] - Gy : Gy - Gx[j][r])) * (BACK ? ry : rx[j][r]);
        const float p = rel * (BACK ? qx[j][r] : qy) * pq[j][r];
        const float e = rel * (BACK ? rx[j][r] : ry) * kk[j][r];
        pq[j][r] = on ? p : 0.f;
        e4[r] = on && s < t ? e : 0.f;
        if constexpr (BACK) E[t][s] = e4[r];
      }
      if constexpr (!BACK) *reinterpret_cast<f32x4_t*>(&E[y][16 * j + 4 * g]) = e4;
    }
  }
  if (wave == 0) {
    const float in = sIn[lane];
    DeltaGates* gates = reinterpret_cast<DeltaGates*>(a.ws + ws.gates) + bhw;
    gates->beta[lane] = sBeta[lane];
    gates->kin[lane] = in * sRk[lane];
    gates->qin[lane] = in * sRq[lane];
    gates->kout[lane] = sOut[lane] * sRk[lane];
    gates->in[lane] = in;
    if constexpr (BACK) {
      gates->rk[lane] = sRk[lane];
      gates->rq[lane] = sRq[lane];
      gates->G[lane] = sG[lane];
    }
  }
  // P's fragments: lane (c, g), slots 4t + r, contraction index 32 s + 16 t + 4 g + r
  {
    char* out = a.ws + (BACK ? ws.up_p : ws.low_p) + bhw * kTriBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (BACK ? wave >= 2 * s + 2 : 2 * s > wave) continue;
      float v[8];
      slots(pq[2 * s], pq[2 * s + 1], v);
      M::store(out + (BACK ? up_frag(wave, s) : low_frag(wave, s)) * 2048, lane, M::two(v));
    }
  }
  __syncthreads();
  f32x4_t col[4];
  {
    const int o = 16 * wave;
    float r[16], eb[16];
    const float beta = sBeta[o + c];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      r[i] = -E[o + i][o + c];
      eb[i] = times(r[i], beta);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      r[i] = c < i && same(o + i, o + c) ? r[i] : 0.f;
#pragma unroll
      for (int k = i + 1; k < 16; ++k) r[k] = fmaf(lane_value(eb[k], i), r[i], r[k]);
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool on = c < i && same(o + i, o + c);
        R[o + i][o + c] = r[i];
        Md[wave][i][c] = i == c ? 1.f : on ? r[i] * beta : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      col[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (i == wave) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = r[e];
#pragma unroll
          for (int k = 1; k < 4; ++k) v = g == k ? r[4 * k + e] : v;
          col[i][e] = v;
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= wave) continue;
    f32x4_t acc;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = -E[16 * i + 4 * g + r][16 * wave + c];
#pragma unroll
    for (int k = 0; k < i; ++k) {
      if (k < wave) continue;
      const float4 e = *reinterpret_cast<const float4*>(&E[16 * i + c][16 * k + 4 * g]);
      const float4 be = *reinterpret_cast<const float4*>(sBeta + 16 * k + 4 * g);
      const float4 m = make_float4(-times(e.x, be.x), -times(e.y, be.y), -times(e.z, be.z), -times(e.w, be.w));
      acc = mma4(m, col[k], acc);
    }
    // a row that holds no number stays so, and does not reach the rows in front of it
    f32x4_t num;
#pragma unroll
    for (int r = 0; r < 4; ++r) num[r] = fabsf(acc[r]) < __builtin_huge_valf() ? acc[r] : 0.f;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    col[i] = mma4(*reinterpret_cast<const float4*>(&Md[i][c][4 * g]), num, zero);
#pragma unroll
    for (int r = 0; r < 4; ++r) col[i][r] += acc[r] - num[r];
  }
  // what lies between pieces may hold another sequence's NaN by now
  if constexpr (VL) {
#pragma unroll
    for (int i = 1; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) col[i][r] = same(16 * i + 4 * g + r, 16 * wave + c) ? col[i][r] : 0.f;
  }
  if constexpr (BACK) {
    char* out = a.ws + ws.up_r + bhw * kTriBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (wave >= 2 * s + 2) continue;
      float v[8];
      slots(col[2 * s], col[2 * s + 1], v);
      M::store(out + up_frag(wave, s) * 2048, lane, M::two(v));
    }
  }
  __syncthreads();  // E is done with
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= wave) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) R[16 * i + 4 * g + r][16 * wave + c] = col[i][r];
  }
  __syncthreads();
  char* low_r = a.ws + ws.low_r + bhw * kTriBytes;
  for (int f = wave; f < kTriFrags; f += 4) {
    const int i = f < 2 ? f : 2 + (f - 2) / 2, s = f < 2 ? 0 : (f - 2) % 2;
    const float* p = &R[16 * i + c][32 * s + 4 * g];
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 16);
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    M::store(low_r + f * 2048, lane, M::two(v));
  }
}

// ---------------------------------------------------------------- tokens whose state is asked for
__global__ __launch_bounds__(256) void delta_wanted_clear_kernel(int* of, int64_t n) {
  const int64_t i = (int64_t)flat_block() * 256 + threadIdx.x;
  if (i < n) of[i] = -1;
}
// The order of a token's list is whatever the exchanges make it: all of it gets the same state.
__global__ __launch_bounds__(256) void delta_wanted_kernel(int* of, int* next, int64_t n, const int64_t* last, int64_t nseq) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < nseq && last[i] >= 0 && last[i] < n) next[i] = atomicExch(of + last[i], (int)i);
}

// ---------------------------------------------------------------- the chain
template <class M, int NP>
constexpr int chain_pitch() { return NP + 16 / (int)sizeof(typename M::IO::type); }
template <class M, int NP, bool SAVE>
constexpr size_t chain_lds() {
  return (size_t)(SAVE ? 1 : 2) * kC * chain_pitch<M, NP>() * sizeof(typename M::IO::type) + 5 * kC * 4;
}

// fp32 products, and bf16 inputs of more than 128 key columns, whose state fills a
// wave's registers.  Of four waves one or two hold columns, the others bring the
// next piece's k, q and gates.  SAVE: for the gradients, the state in front of
// every window and w instead of y.  Bound by the length of the chain, about 6 us a
// window of fp32 (2 x 777 tokens, N = 48, P = 80: 76 us; 157 where every wave had
// columns and staged for itself).
template <class M, int NP, bool VL, bool SAVE>
__global__ __launch_bounds__(256) void delta_chain_kernel(DeltaArgs a, DeltaWs ws) {
  typedef typename M::IO::type T;
  typedef typename M::Two Two;
  constexpr int NT = NP / 16, KS = NP / 32, LP = chain_pitch<M, NP>();
  extern __shared__ __align__(16) char lds[];
  T* kt = reinterpret_cast<T*>(lds);
  T* qt = kt + (SAVE ? 0 : kC * LP);
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
  const Wanted wanted = VL && !SAVE ? wanted_states(a, ws) : Wanted{};

  f32x4_t S[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nn = 16 * j + 4 * g + r;
      S[j][r] = a.h0 && column && nn < N ? a.h0[(bh * N + nn) * a.P + p] : 0.f;
    }

  for (int64_t win = 0; win < ws.nw; ++win) {
    const int64_t t0 = win * kC, bhw = bh * ws.nw + win;
    const int n = (int)(a.L - t0 < kC ? a.L - t0 : kC);
    Cuts cuts = {0, 0};
    if constexpr (VL) {
      cuts = window_cuts(a.seq_idx, wanted, row, t0, a.L, lane);
      if (cuts.fresh & 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) S[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
    if constexpr (SAVE) {
      float* out = reinterpret_cast<float*>(a.ws + ws.S) + bhw * N * a.P + p;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int nn = 16 * j + 4 * g + r;
          if (column && nn < N) out[nn * a.P] = S[j][r];
        }
    }
    const char* fr = a.ws + ws.low_r + bhw * kTriBytes;
    const char* fp = a.ws + ws.low_p + bhw * kTriBytes;
    int begin = 0;
    while (begin < n) {
      const int end = VL ? piece_end(cuts.piece, begin, n) : n;
      if (VL && begin > 0 && (cuts.fresh >> begin & 1)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) S[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      const T* kb = static_cast<const T*>(a.k) + (row + t0) * a.rows.k + grp * N;
      const T* qb = static_cast<const T*>(a.q) + (row + t0) * a.rows.q + grp * N;
      if (!column) {
        const float* gates = reinterpret_cast<const float*>(reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw);
        const int st = tid - 64 * w, sn = 256 - 64 * w;
        Stager<M, NP, !SAVE> sg;
        sg.load(kb, (uint32_t)a.rows.k, qb, (uint32_t)a.rows.q, gates, N, n, begin, end, st, sn);
        __syncthreads();
        sg.store(kt, qt, gt, LP, kb, (uint32_t)a.rows.k, qb, (uint32_t)a.rows.q, N, n, begin, end, st, sn);
        __syncthreads();
        begin = end;
        continue;
      }
      // asked for before the rows are there, where there are registers for it (above 128 it spills)
      constexpr bool kEarly = NP < 256;
      Two rf[kTriFrags];
      uint32_t vq[16];
#pragma unroll
      for (int f = 0; f < kTriFrags; ++f)
        if constexpr (kEarly) rf[f] = M::load(fr + f * 2048, lane);
      load_column<typename M::IO>(static_cast<const T*>(a.v) + (row + t0) * a.rows.v + h * a.P, (uint32_t)a.rows.v, p, n,
                                  begin, end, g, vq);
      __syncthreads();
      __syncthreads();

      f32x4_t X[4], Q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) X[i] = Q[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float v[8];
        slots(S[2 * s], S[2 * s + 1], v);
        const Two sb = M::two(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const T* kp = kt + (16 * i + c) * LP + 32 * s + 4 * g;
          X[i] = M::mma(lds_4x2<M>(kp, kp + 16), sb, X[i]);
          if constexpr (!SAVE) {
            const T* qp = qt + (16 * i + c) * LP + 32 * s + 4 * g;
            Q[i] = M::mma(lds_4x2<M>(qp, qp + 16), sb, Q[i]);
          }
        }
      }
      // X = v - e^G k S
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 kin = *reinterpret_cast<const float4*>(sKin + 16 * i + 4 * g);
        const float4 qin = *reinterpret_cast<const float4*>(sQin + 16 * i + 4 * g);
        const float ki[4] = {kin.x, kin.y, kin.z, kin.w}, qi[4] = {qin.x, qin.y, qin.z, qin.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = column_value<typename M::IO>(vq[4 * i + r]);
          X[i][r] = v - ki[r] * X[i][r];
          Q[i][r] *= qi[r];
        }
      }
      // w = X + R (b X); u = b w
      float be[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(sBeta + 16 * i + 4 * g);
        be[i][0] = q.x; be[i][1] = q.y; be[i][2] = q.z; be[i][3] = q.w;
      }
      f32x4_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) u[i][r] = be[i][r] * X[i][r];
      if constexpr (!SAVE) keep_causal<M>(u, X, g);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8];
        slots(u[2 * s], u[2 * s + 1], v);
        const Two xb = M::two(v);
#pragma unroll
        for (int i = 2 * s; i < 4; ++i) X[i] = M::mma(kEarly ? rf[low_frag(i, s)] : M::load(fr + low_frag(i, s) * 2048, lane), xb, X[i]);
      }
      if constexpr (SAVE) {
        float* out = reinterpret_cast<float*>(a.ws + ws.w) + bhw * kC * a.P + p;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * g + r;
            if (t >= begin && t < end) out[t * a.P] = X[i][r];
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          u[i][r] = !VL || (t >= begin && t < end) ? be[i][r] * X[i][r] : 0.f;
        }
      float whole = sIn[end - 1];
      if constexpr (!SAVE) {
        if (keep_causal<M>(u, Q, g)) whole = __builtin_nanf("");
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float v[8];
          slots(u[2 * s], u[2 * s + 1], v);
          const Two ub = M::two(v);
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) Q[i] = M::mma(M::load(fp + low_frag(i, s) * 2048, lane), ub, Q[i]);
        }
        T* yp = static_cast<T*>(a.y) + ((row + t0) * a.H + h) * a.P + p;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * g + r;
            if (t >= begin && t < end) yp[t * a.H * a.P] = M::IO::put(Q[i][r]);
          }
      }
      // S = e^G_end S + k^T (e^{G_end - G} u)
#pragma unroll
      for (int j = 0; j < NT; ++j) S[j] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = u[2 * s + e / 4][e % 4] * sKout[32 * s + 16 * (e / 4) + 4 * g + e % 4];
        const Two ub = M::two(v);
#pragma unroll
        for (int j = 0; j < NT; ++j) S[j] = M::mma(M::transposed(kt + 32 * s * LP + 16 * j, LP, lane), ub, S[j]);
      }
      if constexpr (VL) {
        for (int s = wanted.first(row + t0 + end - 1); s >= 0; s = wanted.after(s)) {
          float* out = a.seq_states + (s * a.H + h) * N * a.P + p;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int nn = 16 * j + 4 * g + r;
              if (column && nn < N) out[nn * a.P] = S[j][r];
            }
        }
      }
      begin = end;
    }
  }
  if (!SAVE && a.hfin) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int nn = 16 * j + 4 * g + r;
        if (column && nn < N) a.hfin[(bh * N + nn) * a.P + p] = S[j][r];
      }
  }
}

// ---------------------------------------------------------------- the chain of bf16 inputs
// C column waves, C stagers and C output waves, a block a compute unit.  A step
// takes a piece: the column waves correct its values and update their state,
// which is the chain's length; the stagers put the next piece's operands, asked
// for a step before, into the other half of LDS; the output waves work out the
// piece before, from the operands (state, u) that the column waves left in LDS.
// Two column waves a block: with one, k and q are staged twice as often; four
// leave half of the chip idle at 64 heads of 128 columns.  Bound by the column
// waves' latency, 2.2 us a window of which their own products, roundings and LDS
// reads take 1.75; the matrix units are busy 8 to 18%.  2 x 8192 tokens of 32
// heads, N = P = 128: 280 us (one kernel of waves that stage for themselves 2370),
// the whole call 1.0 TB/s of its bytes.  Looking at the last state for what is no
// number (mend_outputs) costs 1 to 2 us a call; looking at every piece's values in
// its column and output waves cost 6 of these, and 13 of 180 in packed rows.
template <int NP, int C>
struct ChainLds {
  static constexpr int kPitch = NP + 24;  // rows as the products read them begin in different banks
  static constexpr int kRows = kC * kPitch * 2;
  static constexpr int kX = (NP / 32 + 2) * 2048;  // operands of a column wave: state and u
  static constexpr int k = 0, r = k + kRows, g = r + kTriBytes, half = g + 5 * kC * 4;
  static constexpr int q = 2 * half, x = q + 2 * kRows, total = x + 2 * C * kX;
};

// Where a wave's columns came to hold no number, it walks their pieces once more,
// by itself, and writes the outputs of the piece in which a column did so: the NaN
// or infinity has reached those in front of it (keep_causal).  Later ones hold no
// number by their state, and every state and other output is right already.
// Operands come straight from memory, some ten times slower.  `lost`: the lane's
// column ends so; without packed sequences all is done once each such has been met.
template <int NP, bool VL>
__device__ __forceinline__ void mend_outputs(const DeltaArgs& a, const DeltaWs& ws, Pieces pc, f32x4_t* S, bool lost,
                                             int64_t bh, uint32_t p, int lane) {
  typedef DeltaB M;
  typedef DeltaB::One One;
  typedef DeltaB::Two Two;
  constexpr int NT = NP / 16, KS = NP / 32;
  const int c = lane & 15, g = lane >> 4, N = (int)a.N;
  const int64_t h = bh % a.H, row = bh / a.H * a.L, grp = h / (a.H / a.G);
  const uint32_t krow = (uint32_t)a.rows.k, qrow = (uint32_t)a.rows.q, yrow = (uint32_t)(a.H * a.P);
  for (; pc.valid() && (VL || __ballot(lost) != 0); pc.step()) {
    const int begin = pc.begin, end = pc.end, n = pc.n;
    const int64_t t0 = row + pc.win * kC, bhw = bh * ws.nw + pc.win;
    const DeltaGates* gates = reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw;
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + t0 * a.rows.k + grp * N;
    const uint16_t* qb = static_cast<const uint16_t*>(a.q) + t0 * a.rows.q + grp * N;
    if (VL && pc.fresh()) {
#pragma unroll
      for (int j = 0; j < NT; ++j) S[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    auto in_piece = [&](int t) { return t >= begin && t < end; };
    // rows of the window times the state
    auto times_state = [&](const uint16_t* base, uint32_t stride, f32x4_t* out) {
      const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float v[8];
        slots(S[2 * s], S[2 * s + 1], v);
        const Two sb = M::two(v);
        const int col = 32 * s + 4 * g;
        const uint32_t off = (c * stride + col) * 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto lo = __builtin_amdgcn_raw_buffer_load_b64(r, col < N ? off : kNowhere, 16 * i * stride * 2, 0);
          const auto hi = __builtin_amdgcn_raw_buffer_load_b64(r, col + 16 < N ? off + 32 : kNowhere, 16 * i * stride * 2, 0);
          One f;
          f.v = make_uint4(lo[0], lo[1], hi[0], hi[1]);
          out[i] = M::mma(f, sb, out[i]);
        }
        __builtin_amdgcn_sched_barrier(0);  // a few loads at a time: for registers, not time
      }
    };
    f32x4_t X[4], u[4];
    auto triangle = [&](size_t at, f32x4_t* y) {
      const char* f = a.ws + at + bhw * kTriBytes;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v[8];
        slots(u[2 * s], u[2 * s + 1], v);
        const Two ub = M::two(v);
#pragma unroll
        for (int i = 2 * s; i < 4; ++i) y[i] = M::mma(M::load(f + low_frag(i, s) * 2048, lane), ub, y[i]);
      }
    };
    auto strengthen = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          u[i][r] = in_piece(t) ? gates->beta[t] * X[i][r] : 0.f;
        }
    };
    times_state(kb, krow, X);
    uint32_t q[16];
    load_column<IoBF16>(static_cast<const uint16_t*>(a.v) + t0 * a.rows.v + h * a.P, (uint32_t)a.rows.v, p, n, begin, end, g, q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * g + r;
        X[i][r] = in_piece(t) ? fmaf(-gates->kin[t], X[i][r], bf16_bits_to_f32(q[4 * i + r])) : 0.f;
      }
    strengthen();
    keep_causal<M>(u, X, g);
    triangle(ws.low_r, X);
    strengthen();
    if (!all_numbers<M>(u)) {
      times_state(qb, qrow, X);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) X[i][r] *= gates->qin[16 * i + 4 * g + r];
      const bool met = keep_causal<M>(u, X, g);
      triangle(ws.low_p, X);
      const __amdgpu_buffer_rsrc_t yr =
          rows_of(static_cast<uint16_t*>(a.y) + (t0 * a.H + h) * a.P, (uint32_t)n * yrow * 2);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t t = Column::row(e) + 4 * g;
        __builtin_amdgcn_raw_buffer_store_b16(IoBF16::put(X[e / 4][e % 4]), yr,
                                              met && in_piece((int)t) ? (t * yrow + p) * 2 : kNowhere, 0, 0);
      }
      if (met) {
        lost = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[j][r] = __builtin_nanf("");
      }
    }
    const float whole = gates->in[end - 1];
    Two ub[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 32 * s + 16 * (e / 4) + 4 * g + e % 4;
        v[e] = in_piece(t) ? u[2 * s + e / 4][e % 4] * gates->kout[t] : 0.f;
      }
      ub[s] = M::two(v);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      S[j] *= whole;
      load_column<IoBF16>(kb, krow, min(16 * j, N - 16) + c, n, begin, end, g, q);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t* w = q + 8 * s;
        One f;
        f.v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        S[j] = M::mma(f, ub[s], S[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Rows too long and too few to fill the chip are cut into stretches, walked side
// by side in two passes.  A stretch maps the state in front of it to M S + R:
// kStretch walks it from the unit matrix (N more columns, without values) and
// from zero, delta_enter_kernel joins the stretches' maps in order, and kOut
// then walks each from the state that enters it.
enum ChainMode { kOut, kSave, kStretch };
template <int NP, int C, bool VL, ChainMode MODE>
__global__ __launch_bounds__(MODE == kOut ? chain_threads(C) : 128 * C, C) void delta_chain_bf16_kernel(DeltaArgs a, DeltaWs ws) {
  typedef DeltaB M;
  typedef DeltaB::One One;
  typedef DeltaB::Two Two;
  typedef ChainLds<NP, C> Lay;
  constexpr int NT = NP / 16, KS = NP / 32, LP = Lay::kPitch, NH = 64 * C;
  constexpr bool SAVE = MODE == kSave, OUT = MODE == kOut;
  extern __shared__ __align__(16) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t bid = near_block(blockIdx.x, gridDim.x);
  const int N = (int)a.N;
  const uint32_t slices = (uint32_t)((MODE == kStretch ? a.N + a.P : a.P) / 16) / C;
  const uint32_t segs = MODE == kOut ? (uint32_t)ws.segs : MODE == kStretch ? (uint32_t)ws.segs - 1 : 1;
  const int64_t seg = bid / slices % segs, bh = bid / slices / segs, h = bh % a.H, b = bh / a.H, grp = h / (a.H / a.G);
  uint32_t p = ((bid % slices) * C + wave % C) * 16 + c;
  // kStretch: columns of the unit matrix, then those of the values
  const bool unit = MODE == kStretch && __builtin_amdgcn_readfirstlane(((bid % slices) * C + wave % C) * 16) < N;
  if (MODE == kStretch && !unit) p -= N;
  const uint32_t P = (uint32_t)a.P;
  const int64_t row = b * a.L;
  const Wanted wanted = VL && OUT ? wanted_states(a, ws) : Wanted{};
  Pieces pc;
  const int64_t w0 = MODE == kSave ? 0 : seg * ws.seg_wins;
  auto first_piece = [&] {
    pc.first(VL ? reinterpret_cast<const Cuts*>(a.ws + ws.cuts) + b * ws.nw : nullptr, w0,
             MODE == kSave || w0 + ws.seg_wins > ws.nw ? ws.nw : w0 + ws.seg_wins, a.L);
  };
  first_piece();

  constexpr int SG = OUT ? first_stager(C) : C;
  if (wave >= SG) {
    // ---- stager: pc is the piece the column waves take, n1 the next
    const int ht = tid - 64 * SG;
    RowTile<NP, NH> kt, qt;
    TriTile<NH> rt;
    GateTile<NH> gt;
    const uint32_t krow = (uint32_t)a.rows.k, qrow = (uint32_t)a.rows.q;
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + row * a.rows.k + grp * N;
    const uint16_t* qb = static_cast<const uint16_t*>(a.q) + row * a.rows.q + grp * N;
    auto ask = [&](const Pieces& s) {
      const int64_t bhw = bh * ws.nw + s.win;
      kt.load(kb + s.win * kC * a.rows.k, krow, N, s.n, ht);
      rt.load(a.ws + ws.low_r + bhw * kTriBytes, ht);
      gt.load(reinterpret_cast<const DeltaGates*>(a.ws + ws.gates) + bhw, ht);
    };
    auto put = [&](const Pieces& s, int half) {
      char* o = lds + half * Lay::half;
      kt.template store<VL>(reinterpret_cast<uint16_t*>(o + Lay::k), LP, s.begin, s.end, ht);
      rt.store(o + Lay::r, ht);
      gt.template store<VL>(reinterpret_cast<float*>(o + Lay::g), s.begin, s.end, ht);
    };
    ask(pc);
    put(pc, 0);
    Pieces n1 = pc;
    n1.step();
    if (n1.valid()) ask(n1);
    if (OUT) qt.load(qb + pc.win * kC * a.rows.q, qrow, N, pc.n, ht);
    __syncthreads();
    for (int j = 0; pc.valid(); ++j) {
      if (n1.valid()) put(n1, (j + 1) & 1);
      if (OUT) qt.template store<VL>(reinterpret_cast<uint16_t*>(lds + Lay::q + (j & 1) * Lay::kRows), LP, pc.begin, pc.end, ht);
      pc = n1;
      if (n1.valid()) {
        if (OUT) qt.load(qb + n1.win * kC * a.rows.q, qrow, N, n1.n, ht);
        n1.step();
        if (n1.valid()) ask(n1);
      }
      __syncthreads();
    }
    if (OUT) __syncthreads();  // the outputs'
    return;
  }
  if (wave >= 2 * C) return;
  if (OUT && wave >= C) {
    // ---- output wave: pc is the piece the column waves take, the one before is worked out
    const uint32_t yrow = (uint32_t)(a.H * a.P);
    Two pf[kTriFrags];
    f32x4_t qin[4];
    int64_t t0 = 0;
    int begin = 0, end = 0, n = 0;
    __syncthreads();
    for (int j = 0;; ++j) {
      if (j > 0) {
        const char* x = lds + Lay::x + (((j - 1) & 1) * C + wave % C) * Lay::kX;
        const uint16_t* ql = reinterpret_cast<const uint16_t*>(lds + Lay::q + ((j - 1) & 1) * Lay::kRows);
        f32x4_t y[4], u[4];
        Two sb[KS];
        One qf[KS][4];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          sb[s] = M::load(x + s * 2048, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint16_t* qp = ql + (16 * i + c) * LP + 32 * s + 4 * g;
            qf[s][i] = lds_4x2<M>(qp, qp + 16);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          u[i] = *reinterpret_cast<const f32x4_t*>(x + KS * 2048 + i * 1024 + 16 * lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = M::mma(qf[s][i], sb[s].lo, y[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = M::mma(qf[s][i], sb[s].hi, y[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= qin[i];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float v[8];
          slots(u[2 * s], u[2 * s + 1], v);
          const Two ub = M::two(v);
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) y[i] = M::mma(pf[low_frag(i, s)].hi, ub.lo, y[i]);
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) y[i] = M::mma(pf[low_frag(i, s)].lo, ub.hi, y[i]);
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) y[i] = M::mma(pf[low_frag(i, s)].hi, ub.hi, y[i]);
        }
        Column::put<VL>(static_cast<uint16_t*>(a.y) + ((row + t0) * a.H + h) * a.P, yrow, 4 * g * yrow + p, n, y, begin,
                        end, g);
      }
      if (!pc.valid()) break;
      // kept for the next step, when piece j is worked out
      const char* fp = a.ws + ws.low_p + (bh * ws.nw + pc.win) * kTriBytes;
#pragma unroll
      for (int f = 0; f < kTriFrags; ++f) pf[f] = M::load(fp + f * 2048, lane);
      const float* sq = reinterpret_cast<const float*>(lds + (j & 1) * Lay::half + Lay::g) + 2 * kC;
#pragma unroll
      for (int i = 0; i < 4; ++i) qin[i] = *reinterpret_cast<const f32x4_t*>(sq + 16 * i + 4 * g);
      t0 = pc.win * kC;
      n = pc.n;
      begin = pc.begin;
      end = pc.end;
      pc.step();
      __syncthreads();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // a column wave may write them again
    __syncthreads();
    return;
  }

  // ---- column wave
  __builtin_amdgcn_s_setprio(3);
  f32x4_t S[NT];
  const float* from = a.h0 ? a.h0 + bh * N * a.P : nullptr;
  if (MODE == kOut && segs > 1) from = reinterpret_cast<const float*>(a.ws + ws.enter) + (bh * segs + seg) * N * a.P;
  auto enter = [&](f32x4_t* s) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int nn = 16 * j + 4 * g + r;
        if (MODE == kStretch) s[j][r] = unit && nn == (int)p ? 1.f : 0.f;
        else s[j][r] = from && nn < N ? from[nn * a.P + p] : 0.f;
      }
  };
  enter(S);
  const uint32_t vrow = (uint32_t)a.rows.v, voff = 4 * g * vrow + p;
  const uint16_t* vb = static_cast<const uint16_t*>(a.v) + row * a.rows.v + h * a.P;
  // of the lane's column: a token that is no number leaves none in its state, to the end of its sequence
  auto numbers = [&] {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) sum += (fabsf(S[j][0]) + fabsf(S[j][1])) + (fabsf(S[j][2]) + fabsf(S[j][3]));
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    return sum < M::kMost;
  };
  bool again = false;
  Column vn;
  vn.load(vb + pc.win * kC * a.rows.v, vrow, voff, unit ? 0 : pc.n);
  __syncthreads();
  for (int step = 0; pc.valid(); ++step) {
    const int begin = pc.begin, end = pc.end;
    const int64_t win = pc.win, bhw = bh * ws.nw + win;
    const char* in = lds + (step & 1) * Lay::half;
    const uint16_t* kt = reinterpret_cast<const uint16_t*>(in + Lay::k);
    const float* gt = reinterpret_cast<const float*>(in + Lay::g);
    const float *sBeta = gt, *sKin = gt + kC, *sKout = gt + 3 * kC, *sIn = gt + 4 * kC;
    char* x = lds + Lay::x + ((step & 1) * C + wave) * Lay::kX;
    if (VL && pc.fresh()) {
      if (OUT) again |= __ballot(!numbers()) != 0;
#pragma unroll
      for (int j = 0; j < NT; ++j) S[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // The wave has its SIMD to itself: what a product needs from LDS is asked for
    // well before, k and R ahead of the state's rounding, k^T ahead of R's product.
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
    if (SAVE && begin == 0)
      put_state<NT>(reinterpret_cast<float*>(a.ws + ws.S) + bhw * N * a.P, N, P, 4 * g * P + p, S);
    f32x4_t X[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) X[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float v[8];
      slots(S[2 * s], S[2 * s + 1], v);
      const Two sb = M::two(v);
      if constexpr (OUT) M::store(x + s * 2048, lane, sb);
#pragma unroll
      for (int i = 0; i < 4; ++i) X[i] = M::mma(kf[s][i], sb.lo, X[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) X[i] = M::mma(kf[s][i], sb.hi, X[i]);
      if (s == 0) {
#pragma unroll
        for (int f = 0; f < kTriFrags; ++f) rf[f] = M::load(in + Lay::r + f * 2048, lane);
      }
    }
    // the state's rounding between the products: a product occupies the matrix unit for four issues
#pragma unroll
    for (int e = 0; e < 8 * KS; ++e) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
    }
    float ki[4][4], be[4][4], ko[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_vec<IoF32, 4>(sKin + 16 * i + 4 * g, ki[i]);
      load_vec<IoF32, 4>(sBeta + 16 * i + 4 * g, be[i]);
      load_vec<IoF32, 4>(sKout + 16 * i + 4 * g, ko[i]);
    }
    const float whole = sIn[end - 1];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) kT[s][j] = M::transposed(kt + 32 * s * LP + 16 * j, LP, lane);
    __builtin_amdgcn_sched_barrier(0);
    // X = v - e^G k S; in packed rows the others' values are left out (what is behind the row reads as zero)
    f32x4_t bx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * g + r;
        const float v = !VL || (t >= begin && t < end) ? vn.get(i, r) : 0.f;
        X[i][r] = fmaf(-ki[i][r], X[i][r], v);
        bx[i][r] = be[i][r] * X[i][r];
      }
    pc.step();
    if (pc.valid()) vn.load(vb + pc.win * kC * a.rows.v, vrow, voff, unit ? 0 : pc.n);
    // w = X + R (b X); u = b w
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = bx[2 * s + e / 4][e % 4];
      const Two xb = M::two(v);
#pragma unroll
      for (int i = 2 * s; i < 4; ++i) X[i] = M::mma(rf[low_frag(i, s)].hi, xb.lo, X[i]);
#pragma unroll
      for (int i = 2 * s; i < 4; ++i) X[i] = M::mma(rf[low_frag(i, s)].lo, xb.hi, X[i]);
#pragma unroll
      for (int i = 2 * s; i < 4; ++i) X[i] = M::mma(rf[low_frag(i, s)].hi, xb.hi, X[i]);
    }
    if constexpr (SAVE)
      Column::put<VL>(reinterpret_cast<float*>(a.ws + ws.w) + bhw * kC * a.P, P, 4 * g * P + p, kC, X, begin, end, g);
#pragma unroll
    for (int j = 0; j < NT; ++j) S[j] *= whole;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int t4 = 0; t4 < 2; ++t4) {
        const int i = 2 * s + t4;
        f32x4_t u;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * i + 4 * g + r;
          u[r] = !VL || (t >= begin && t < end) ? be[i][r] * X[i][r] : 0.f;
          v[4 * t4 + r] = u[r] * ko[i][r];
        }
        if constexpr (OUT) *reinterpret_cast<f32x4_t*>(x + KS * 2048 + i * 1024 + 16 * lane) = u;
      }
      const Two ub = M::two(v);
#pragma unroll
      for (int j = 0; j < NT; ++j) S[j] = M::mma(kT[s][j], ub.lo, S[j]);
#pragma unroll
      for (int j = 0; j < NT; ++j) S[j] = M::mma(kT[s][j], ub.hi, S[j]);
    }
    if constexpr (VL) {
      for (int s = wanted.first(row + win * kC + end - 1); s >= 0; s = wanted.after(s))
        put_state<NT>(a.seq_states + (s * a.H + h) * N * a.P, N, P, 4 * g * P + p, S);
    }
    __syncthreads();
  }
  if constexpr (OUT) {
    __syncthreads();  // the outputs are written
    const bool lost = !numbers();
    again |= __ballot(lost) != 0;
    f32x4_t S0[NT];
    if (__builtin_expect(again, 0)) enter(S0);  // before the last state may take its place
    if (a.hfin && seg == segs - 1) put_state<NT>(a.hfin + bh * N * a.P, N, P, 4 * g * P + p, S);
    if (__builtin_expect(again, 0)) {
      first_piece();
      mend_outputs<NP, VL>(a, ws, pc, S0, lost, bh, p, lane);
    }
  }
  if constexpr (MODE == kStretch) {
    const uint32_t cols = (uint32_t)N + P;
    put_state<NT>(reinterpret_cast<float*>(a.ws + ws.trans) + (bh * segs + seg) * N * cols, N, cols,
                  4 * g * cols + (unit ? p : N + p), S);
  }
}

// The states that enter the stretches of a row: S' = M S + R, a block 16 columns
// and a wave 32 rows of them, so that the next stretch's map is asked for while
// one is multiplied; the waves meet once a stretch, for S as operands.  Where a
// sequence begins in the stretch it is R alone, and M is not multiplied: its
// zeros would make NaN of what the sequence before left.  3 us a stretch; one
// wave for all rows, which read each map only when its turn came, took 6.
template <int NP>
__global__ __launch_bounds__(2 * NP) void delta_enter_kernel(DeltaArgs a, DeltaWs ws) {
  typedef DeltaB M;
  constexpr int KS = NP / 32;
  __shared__ M::Two sS[2][KS][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4, N = (int)a.N;
  const uint32_t P = (uint32_t)a.P, cols = N + P, tiles = P / 16;
  const int64_t bh = blockIdx.x / tiles;
  const uint32_t p = blockIdx.x % tiles * 16 + c;
  const Cuts* list = a.seq_idx ? reinterpret_cast<const Cuts*>(a.ws + ws.cuts) + bh / a.H * ws.nw : nullptr;
  f32x4_t S[2], R[2], x[2][KS][2];
  bool begins = false;
  auto ask = [&](int64_t seg) {
    if (list) {
      bool any = false;
      const int64_t to = min((seg + 1) * ws.seg_wins, ws.nw);
      for (int64_t w = seg * ws.seg_wins + lane; w < to; w += 64) any |= list[w].fresh != 0;
      begins = __ballot(any) != 0;
    }
    const float* m = reinterpret_cast<const float*>(a.ws + ws.trans) + (bh * (ws.segs - 1) + seg) * N * cols;
    const __amdgpu_buffer_rsrc_t r = rows_of(m, (uint32_t)N * cols * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t base = (32 * wave + 16 * i) * cols * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        R[i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (4 * g * cols + N + p) * 4, base + e * cols * 4, 0));
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int col = 32 * s + 16 * t + 4 * g;
          x[i][s][t] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                       r, col < N ? (c * cols + col) * 4 : kNowhere, base, 0));
        }
    }
  };
  ask(0);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nn = 32 * wave + 16 * i + 4 * g + r;
      S[i][r] = a.h0 && nn < N ? a.h0[(bh * N + nn) * a.P + p] : 0.f;
    }
  for (int64_t seg = 0;; ++seg) {
    float* out = reinterpret_cast<float*>(a.ws + ws.enter) + (bh * ws.segs + seg) * N * P;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int nn = 32 * wave + 16 * i + 4 * g + r;
        if (nn < N) out[nn * P + p] = S[i][r];
      }
    if (seg == ws.segs - 1) break;
    float v[8];
    slots(S[0], S[1], v);
    sS[seg & 1][wave][lane] = M::two(v);
    M::Two map[2][KS];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      S[i] = R[i];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        slots(x[i][s][0], x[i][s][1], v);
        map[i][s] = M::two(v);
      }
    }
    const bool only = begins;
    if (seg + 1 < ws.segs - 1) ask(seg + 1);
    __syncthreads();  // a wave writes the other half next, and meets the others before this one again
    if (only) continue;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const M::Two sb = sS[seg & 1][s][lane];
#pragma unroll
      for (int i = 0; i < 2; ++i) S[i] = M::mma(map[i][s], sb, S[i]);
    }
  }
}

// ---------------------------------------------------------------- one token
// A block takes 64 value columns of a (row, head): 16 threads of four columns
// by 16 state rows, whose up to 16 rows a thread are all asked for first.
// Bound by the state, read and written once: k^T h and q^T h are summed
// together, for y = a q^T h + (q.k) u.  64 streams of 32 heads, N = P = 128: 52 us
// for 268 MB, 5.1 TB/s, the rate of a copy.
constexpr int kStepCols = 64, kStepRows = (int)kDeltaMaxDim / 16;
template <class IO>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs a, const float* state, float* state_out) {
  typedef typename IO::type T;
  __shared__ float sk[kDeltaMaxDim], sq[kDeltaMaxDim];
  __shared__ float red[3][4];
  __shared__ float4 part[2][4][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cg = tid & 15, rg = tid >> 4;
  const uint32_t slices = (uint32_t)((a.P + kStepCols - 1) / kStepCols);
  const uint32_t bid = flat_block();
  const int64_t bh = bid / slices;
  if (bh >= a.B * a.H) return;
  const int64_t h = bh % a.H, b = bh / a.H, grp = h / (a.H / a.G);
  const int N = (int)a.N;
  const int64_t p = (int64_t)(bid % slices) * kStepCols + 4 * cg;
  const bool on = p < a.P;
  const float4* st = reinterpret_cast<const float4*>(state + bh * N * a.P + p);
  float4 s[kStepRows];
#pragma unroll
  for (int u = 0; u < kStepRows; ++u) {
    const int nn = rg + 16 * u;
    s[u] = on && nn < N ? st[nn * (a.P / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float kv = tid < N ? IO::get(static_cast<const T*>(a.k)[b * a.rows.k + grp * N + tid]) : 0.f;
  const float qv = tid < N ? IO::get(static_cast<const T*>(a.q)[b * a.rows.q + grp * N + tid]) : 0.f;
  float raw = IO::get(static_cast<const T*>(a.dt)[b * a.rows.dt + h]);
  if (a.dt_bias) raw += a.dt_bias[h];
  const float decay = expf((a.softplus ? softplus2(raw * kLog2e) * kLn2 : raw) * a.A[h]);
  float beta = IO::get(static_cast<const T*>(a.beta)[b * a.rows.beta + h]);
  if (a.sigmoid) beta = sigmoid(beta);
  sk[tid] = kv;
  sq[tid] = qv;
  float k2 = kv * kv, q2 = qv * qv, qk = kv * qv;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    k2 += __shfl_xor(k2, o, 64);
    q2 += __shfl_xor(q2, o, 64);
    qk += __shfl_xor(qk, o, 64);
  }
  if (lane == 0) {
    red[0][wave] = k2;
    red[1][wave] = q2;
    red[2][wave] = qk;
  }
  __syncthreads();
  auto total = [&](const float* r) { return (r[0] + r[1]) + (r[2] + r[3]); };
  const float rk = a.qk_norm ? 1.f / sqrtf(total(red[0]) + kQkEps) : 1.f;
  const float rq = (a.qk_norm ? 1.f / sqrtf(total(red[1]) + kQkEps) : 1.f) * a.scale;
  qk = total(red[2]) * rk * rq;
  float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
#pragma unroll
  for (int u = 0; u < kStepRows; ++u) {
    const int nn = rg + 16 * u;
    if (nn >= N) break;
    const float kn = sk[nn], qn = sq[nn];
    ks.x = fmaf(kn, s[u].x, ks.x); ks.y = fmaf(kn, s[u].y, ks.y);
    ks.z = fmaf(kn, s[u].z, ks.z); ks.w = fmaf(kn, s[u].w, ks.w);
    qs.x = fmaf(qn, s[u].x, qs.x); qs.y = fmaf(qn, s[u].y, qs.y);
    qs.z = fmaf(qn, s[u].z, qs.z); qs.w = fmaf(qn, s[u].w, qs.w);
  }
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) {
    ks.x += __shfl_xor(ks.x, o, 64); ks.y += __shfl_xor(ks.y, o, 64);
    ks.z += __shfl_xor(ks.z, o, 64); ks.w += __shfl_xor(ks.w, o, 64);
    qs.x += __shfl_xor(qs.x, o, 64); qs.y += __shfl_xor(qs.y, o, 64);
    qs.z += __shfl_xor(qs.z, o, 64); qs.w += __shfl_xor(qs.w, o, 64);
  }
  if (lane < 16) {
    part[0][wave][cg] = ks;
    part[1][wave][cg] = qs;
  }
  __syncthreads();
  auto sum4 = [&](const float4(*q)[16]) {
    float4 o = q[0][cg];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 e = q[w][cg];
      o.x += e.x; o.y += e.y; o.z += e.z; o.w += e.w;
    }
    return o;
  };
  if (!on) return;
  ks = sum4(part[0]);
  qs = sum4(part[1]);
  float v[4], u[4];
  load_vec<IO, 1>(static_cast<const T*>(a.v) + b * a.rows.v + h * a.P + p, v);
#pragma unroll
  for (int e = 1; e < 4; ++e) v[e] = IO::get((static_cast<const T*>(a.v) + b * a.rows.v + h * a.P + p)[e]);
  const float kse[4] = {ks.x, ks.y, ks.z, ks.w}, qse[4] = {qs.x, qs.y, qs.z, qs.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = beta * (v[e] - decay * rk * kse[e]);
  if (rg == 0) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf(decay * rq, qse[e], qk * u[e]);
    store_vec<IO, 4>(static_cast<T*>(a.y) + bh * a.P + p, y);
  }
  float4* so = reinterpret_cast<float4*>(state_out + bh * N * a.P + p);
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    const int nn = rg + 16 * r;
    if (nn >= N) break;
    const float kn = rk * sk[nn];
    so[nn * (a.P / 4)] = make_float4(fmaf(decay, s[r].x, kn * u[0]), fmaf(decay, s[r].y, kn * u[1]),
                                     fmaf(decay, s[r].z, kn * u[2]), fmaf(decay, s[r].w, kn * u[3]));
  }
}

// ---------------------------------------------------------------- launches
int64_t delta_segments(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P, bool bf16);
int64_t delta_stretch_room(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P);
static DeltaWs forward_ws(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P, bool bf16) {
  return delta_ws(B, L, H, N, P, false, delta_segments(B, L, H, N, P, bf16), delta_stretch_room(B, L, H, N, P));
}
size_t delta_forward_ws_bytes(int64_t B, int64_t L, int64_t H, int64_t G, int64_t N, int64_t P) {
  return forward_ws(B, L, H, N, P, true).total;
}

template <class M, int NP, bool BACK>
static hipError_t prepare(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  const bool vl = a.seq_idx || (!BACK && a.nseq > 0);
  auto kern = vl ? delta_prepare_kernel<M, NP, BACK, true> : delta_prepare_kernel<M, NP, BACK, false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * ws.nw * a.H)), dim3(256), kPrepLds, s, a, ws);
  return hipGetLastError();
}
template <class M, bool BACK>
static hipError_t prepare_at(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  return a.N <= 64    ? prepare<M, 64, BACK>(a, ws, s)
         : a.N <= 128 ? prepare<M, 128, BACK>(a, ws, s)
                      : prepare<M, 256, BACK>(a, ws, s);
}
template <class M>
static hipError_t prepare_of(const DeltaArgs& a, const DeltaWs& ws, bool back, hipStream_t s) {
  return back ? prepare_at<M, true>(a, ws, s) : prepare_at<M, false>(a, ws, s);
}
hipError_t launch_delta_prepare(const DeltaArgs& a, const DeltaWs& ws, bool back, bool bf16, hipStream_t s) {
  return !bf16            ? prepare_of<DeltaF>(a, ws, back, s)
         : a.f32_products ? prepare_of<DeltaW>(a, ws, back, s)
                          : prepare_of<DeltaB>(a, ws, back, s);
}

template <class M, int NP, bool VL, bool SAVE>
static hipError_t chain(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_chain_kernel<M, NP, VL, SAVE>;
  const size_t lds = chain_lds<M, NP, SAVE>();
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * (a.P / 16 / chain_columns(a.P)))), dim3(256), lds, s, a, ws);
  return hipGetLastError();
}
template <int NP, int C, bool VL, ChainMode MODE>
static hipError_t chain_bf16(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  auto kern = delta_chain_bf16_kernel<NP, C, VL, MODE>;
  const size_t lds = MODE == kOut ? ChainLds<NP, C>::total : ChainLds<NP, C>::q;
  hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const int64_t cols = MODE == kStretch ? a.N + a.P : a.P, segs = MODE == kOut ? ws.segs : MODE == kStretch ? ws.segs - 1 : 1;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.B * a.H * segs * (cols / 16 / C))), dim3(MODE == kOut ? chain_threads(C) : 128 * C),
                     lds, s, a, ws);
  return hipGetLastError();
}
template <int NP, bool VL, ChainMode MODE>
static hipError_t chain_bf16_as(const DeltaArgs& a, const DeltaWs& ws, hipStream_t s) {
  const int64_t cols = MODE == kStretch ? a.N + a.P : a.P;
  return cols % 32 == 0 ? chain_bf16<NP, 2, VL, MODE>(a, ws, s) : chain_bf16<NP, 1, VL, MODE>(a, ws, s);
}
template <int NP, bool VL>
static hipError_t chain_bf16_of(const DeltaArgs& a, const DeltaWs& ws, bool save, hipStream_t s) {
  if (save) return chain_bf16_as<NP, VL, kSave>(a, ws, s);
  if (ws.segs > 1) {
    hipError_t e = chain_bf16_as<NP, VL, kStretch>(a, ws, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(delta_enter_kernel<NP>, dim3((unsigned)(a.B * a.H * (a.P / 16))), dim3(2 * NP), 0, s, a, ws);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return chain_bf16_as<NP, VL, kOut>(a, ws, s);
}
template <int NP>
static hipError_t chain_bf16_at(const DeltaArgs& a, const DeltaWs& ws, bool save, hipStream_t s) {
  const bool vl = a.seq_idx || (!save && a.nseq > 0);
  return vl ? chain_bf16_of<NP, true>(a, ws, save, s) : chain_bf16_of<NP, false>(a, ws, save, s);
}
// Stretches of a row: as many as leave each compute unit a block (of 32 columns)
// and each stretch eight windows; from three on the second pass pays.  Only the
// bf16 chain of up to 128 key columns has them.  Calls of one row, N = P = 128,
// without stretches and with them, us: 2048 tokens of 8 heads 75 and 59, 8192 of
// 2 heads 254 and 87, of 20 heads (three stretches) 280 and 247; two stretches
// take what one does.  Stretches of four windows: 1024 tokens of 8 heads 44 and 54.
constexpr int64_t kSegWins = 8, kSegMost = 128;  // windows a stretch at least, key columns at most
static int64_t head_blocks(int64_t P) { return P % 32 == 0 ? P / 32 : P / 16; }
int64_t delta_segments(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P, bool bf16) {
  if (!bf16 || N > kSegMost) return 1;
  const int64_t nw = (L + kDeltaC - 1) / kDeltaC;
  int64_t segs = device_cu_count() / (B * H * head_blocks(P));
  if (segs > nw / kSegWins) segs = nw / kSegWins;
  if (segs < 3) return 1;
  return (nw + (nw + segs - 1) / segs - 1) / ((nw + segs - 1) / segs);  // none of them empty
}
// Stretches that the workspace has room for: no call has more, and no call of
// more rows, tokens or heads has room for fewer, so that a workspace serves every
// smaller prompt too.  At most one a compute unit: 25 MB.
int64_t delta_stretch_room(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P) {
  if (N > kSegMost) return 0;
  const int64_t all = B * H * ((L + kDeltaC - 1) / kDeltaC / kSegWins), most = device_cu_count() / head_blocks(P);
  return all < most ? all : most;
}
template <class M, int NP>
static hipError_t chain_of(const DeltaArgs& a, const DeltaWs& ws, bool save, hipStream_t s) {
  const bool vl = a.seq_idx || (!save && a.nseq > 0);
  if (save) return vl ? chain<M, NP, true, true>(a, ws, s) : chain<M, NP, false, true>(a, ws, s);
  return vl ? chain<M, NP, true, false>(a, ws, s) : chain<M, NP, false, false>(a, ws, s);
}
template <class M>
static hipError_t chain_at(const DeltaArgs& a, const DeltaWs& ws, bool save, hipStream_t s) {
  if (a.N <= 32) return chain_of<M, 32>(a, ws, save, s);
  if (a.N <= 64) return chain_of<M, 64>(a, ws, save, s);
  if (a.N <= 128) return chain_of<M, 128>(a, ws, save, s);
  return chain_of<M, 256>(a, ws, save, s);
}
hipError_t launch_delta_chain(const DeltaArgs& a, const DeltaWs& ws, bool save, bool bf16, hipStream_t s) {
  if (!bf16) return chain_at<DeltaF>(a, ws, save, s);
  if (a.f32_products) return chain_at<DeltaW>(a, ws, save, s);
  if (a.N <= 32) return chain_bf16_at<32>(a, ws, save, s);
  if (a.N <= 64) return chain_bf16_at<64>(a, ws, save, s);
  if (a.N <= 128) return chain_bf16_at<128>(a, ws, save, s);
  return chain_of<DeltaB, 256>(a, ws, save, s);  // two halves of LDS do not hold 256 key columns
}

hipError_t launch_delta_forward(const DeltaArgs& a, bool bf16, hipStream_t s) {
  const DeltaWs ws = forward_ws(a.B, a.L, a.H, a.N, a.P, bf16 && !a.f32_products);
  if (a.nseq > 0) {
    int* of = reinterpret_cast<int*>(a.ws + ws.wanted);
    hipLaunchKernelGGL(delta_wanted_clear_kernel, flat_grid((a.B * a.L + 255) / 256), dim3(256), 0, s, of, a.B * a.L);
    hipLaunchKernelGGL(delta_wanted_kernel, dim3((unsigned)((a.nseq + 255) / 256)), dim3(256), 0, s, of,
                       reinterpret_cast<int*>(a.ws + ws.wanted_next), a.B * a.L, a.seq_last, a.nseq);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const hipError_t e = launch_delta_prepare(a, ws, false, bf16, s);
  return e != hipSuccess ? e : launch_delta_chain(a, ws, false, bf16, s);
}

hipError_t launch_delta_step(const DeltaArgs& a, const float* state, float* state_out, bool bf16, hipStream_t s) {
  auto kern = bf16 ? delta_step_kernel<IoBF16> : delta_step_kernel<IoF32>;
  hipLaunchKernelGGL(kern, flat_grid(a.B * a.H * ((a.P + kStepCols - 1) / kStepCols)), dim3(256), 0, s, a, state,
                     state_out);
  return hipGetLastError();
}

}  // namespace ssd
