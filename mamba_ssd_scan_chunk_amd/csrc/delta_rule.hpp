// delta_rule.hpp -- what the gated delta rule's kernels share.
//
// Per head, with unit (or raw) keys k_t, queries q_t (scaled), decays a_t =
// e^{g_t} and writing strengths b_t, the state h (N x P) follows
//     h~ = a_t h_{t-1},  u_t = b_t (v_t - k_t^T h~),  h_t = h~ + k_t u_t^T,
//     y_t = q_t^T h_t.
// Tokens are taken in windows of 64, a window in pieces of one sequence (one
// piece unless sequences are packed).  With G the running sum of g in a piece,
// S the state in front of it and
//     E_ts = e^{G_t - G_s} k_t.k_s (s < t),   P_ts = e^{G_t - G_s} q_t.k_s (s <= t),
//     R = -(I + E diag(b))^{-1} E             (strictly lower triangular)
// a piece is a few products:
//     X = v - diag(e^G) k S,   w = X + R (b X),   u = b w,
//     y = diag(e^G) q S + P u,   S' = e^{G_end} S + k^T diag(e^{G_end - G}) u.
// R in place of (I + b E)^{-1} b keeps b = 0 exact here and in the gradients.
//
// Matrix operands.  bf16 inputs enter as they are; what is computed (states,
// corrected values, R, P) enters as the sum of two bf16 values, 16 bits, and
// every sum and the states themselves are fp32, so that states are 2 to 3e-6 and
// sums over tokens up to 6e-6 from the 64-bit values, where one bf16 operand would
// be 2^-9 off.  fp32 products (1 to 2e-7) have an eighth of the rate; a caller who
// wants them asks for them (DeltaW) or passes fp32 inputs.
// Unit length goes into the fp32 scalars of a row, never into rounded rows.
// fp32 inputs use the fp32 matrix instructions throughout.
#pragma once

#include <type_traits>

#include "delta_launch.hpp"
#include "layer_device.hpp"

namespace ssd {

constexpr float kQkEps = 1e-6f;
constexpr int kC = (int)kDeltaC;

// Rows of a window through a buffer descriptor: a lane's offset in one register,
// the row's in a scalar, and rows behind the window's n read as zero and are not
// written.  64 rows stay below 2^32 bytes (rows below 2^23 elements).
constexpr uint32_t kNowhere = 0xfffffff0u;  // a lane's offset that is behind every window
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));  // copied as a value, where uint4 is a struct

// One: an operand of inputs.  Two: of computed values.
struct DeltaB {
  static constexpr float kMost = 3.3961775e38f;  // computed values from here on are infinite as bf16
  typedef IoBF16 IO;
  typedef OpBF16::Frag One;
  struct Two { One hi, lo; };
  __device__ __forceinline__ static Two two(const float* s) {
    Two t;
    t.hi = OpBF16::from_f32(s);
    uint32_t w[4] = {t.hi.v.x, t.hi.v.y, t.hi.v.z, t.hi.v.w};
    float d[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      asm("" : "+v"(w[e]));  // the pair as it is, not each value rounded again
      d[2 * e] = s[2 * e] - __uint_as_float(w[e] << 16);
      d[2 * e + 1] = s[2 * e + 1] - __uint_as_float(w[e] & 0xffff0000u);
    }
    t.lo = OpBF16::from_f32(d);
    return t;
  }
  __device__ __forceinline__ static One one(const float* s) { return OpBF16::from_f32(s); }
  __device__ __forceinline__ static f32x4_t mma(const One& a, const One& b, f32x4_t c) { return OpBF16::mma(a, b, c); }
  __device__ __forceinline__ static f32x4_t mma(const One& a, const Two& b, f32x4_t c) {
    return OpBF16::mma(a, b.hi, OpBF16::mma(a, b.lo, c));
  }
  __device__ __forceinline__ static f32x4_t mma(const Two& a, const One& b, f32x4_t c) {
    return OpBF16::mma(a.hi, b, OpBF16::mma(a.lo, b, c));
  }
  __device__ __forceinline__ static f32x4_t mma(const Two& a, const Two& b, f32x4_t c) {
    return OpBF16::mma(a.hi, b.hi, OpBF16::mma(a.lo, b.hi, OpBF16::mma(a.hi, b.lo, c)));
  }
  // 2 KB a fragment in memory: 16 bytes a lane, twice
  __device__ __forceinline__ static Two load(const char* p, int lane) {
    Two t;
    t.hi.v = *reinterpret_cast<const uint4*>(p + 16 * lane);
    t.lo.v = *reinterpret_cast<const uint4*>(p + 1024 + 16 * lane);
    return t;
  }
  __device__ __forceinline__ static void store(char* p, int lane, const Two& t) {
    *reinterpret_cast<uint4*>(p + 16 * lane) = t.hi.v;
    *reinterpret_cast<uint4*>(p + 1024 + 16 * lane) = t.lo.v;
  }
  // eight consecutive inputs
  __device__ __forceinline__ static One row8(const uint16_t* p) {
    One f;
    f.v = *reinterpret_cast<const uint4*>(p);
    return f;
  }
  // the same by byte offsets of a lane and of a row
  __device__ __forceinline__ static One rows8(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t row) {
    One f;
    f.v = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, row, 0));
    return f;
  }
  // rows of a tile in LDS as the transposed operand: lane (i, g) gets, as slots
  // 4t + r, tile[16t + 4g + r][i]
  __device__ __forceinline__ static One transposed(const uint16_t* tile, int pitch, int lane) {
    return lds_frag_tr(tile, pitch, lane);
  }
};
// fp32 products: of fp32 inputs, and of bf16 ones where the caller asks for them.
struct Fp32Products {
  static constexpr float kMost = __builtin_huge_valf();
  typedef OpF32::Frag One;
  typedef OpF32::Frag Two;
  __device__ __forceinline__ static Two two(const float* s) { return OpF32::from_f32(s); }
  __device__ __forceinline__ static One one(const float* s) { return OpF32::from_f32(s); }
  __device__ __forceinline__ static f32x4_t mma(const One& a, const One& b, f32x4_t c) { return OpF32::mma(a, b, c); }
  __device__ __forceinline__ static Two load(const char* p, int lane) {
    Two t;
    t.lo = *reinterpret_cast<const float4*>(p + 16 * lane);
    t.hi = *reinterpret_cast<const float4*>(p + 1024 + 16 * lane);
    return t;
  }
  __device__ __forceinline__ static void store(char* p, int lane, const Two& t) {
    *reinterpret_cast<float4*>(p + 16 * lane) = t.lo;
    *reinterpret_cast<float4*>(p + 1024 + 16 * lane) = t.hi;
  }
  __device__ __forceinline__ static One row8(const float* p) { return Lds<OpF32>::load8(p); }
};
struct DeltaF : Fp32Products {
  typedef IoF32 IO;
  __device__ __forceinline__ static One rows8(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t row) {
    One f;
    f.lo = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, row, 0));
    f.hi = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, row + 16, 0));
    return f;
  }
  __device__ __forceinline__ static One transposed(const float* tile, int pitch, int lane) {
    const float* p = tile + 4 * (lane >> 4) * pitch + (lane & 15);
    One f;
    f.lo = make_float4(p[0], p[pitch], p[2 * pitch], p[3 * pitch]);
    p += 16 * pitch;
    f.hi = make_float4(p[0], p[pitch], p[2 * pitch], p[3 * pitch]);
    return f;
  }
};
struct DeltaW : Fp32Products {
  typedef IoBF16 IO;
  __device__ __forceinline__ static One wide(const uint4& v) {
    One f;
    f.lo = make_float4(bf16_bits_to_f32(v.x & 0xffffu), __uint_as_float(v.x & 0xffff0000u),
                       bf16_bits_to_f32(v.y & 0xffffu), __uint_as_float(v.y & 0xffff0000u));
    f.hi = make_float4(bf16_bits_to_f32(v.z & 0xffffu), __uint_as_float(v.z & 0xffff0000u),
                       bf16_bits_to_f32(v.w & 0xffffu), __uint_as_float(v.w & 0xffff0000u));
    return f;
  }
  __device__ __forceinline__ static One rows8(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t row) {
    return wide(DeltaB::rows8(r, lane, row).v);
  }
  __device__ __forceinline__ static One transposed(const uint16_t* tile, int pitch, int lane) {
    return wide(DeltaB::transposed(tile, pitch, lane).v);
  }
};
// Slots 0..3 of p0, 4..7 of p1.
template <class M>
__device__ __forceinline__ typename M::One lds_4x2(const typename M::IO::type* p0, const typename M::IO::type* p1) {
  if constexpr (std::is_same<M, DeltaW>::value) return M::wide(Lds<OpBF16>::load4x2(p0, p1).v);
  else if constexpr (sizeof(typename M::IO::type) == 2) return Lds<OpBF16>::load4x2(p0, p1);
  else return Lds<OpF32>::load4x2(p0, p1);
}

// ---- what the preparation leaves for a (row, head, window) ----
struct DeltaGates {
  float beta[kC];
  float kin[kC];   // e^G |k|^-1
  float qin[kC];   // e^G |q|^-1 scale
  float kout[kC];  // e^{G_end - G} |k|^-1
  float in[kC];    // e^G
  float rk[kC], rq[kC];  // |k|^-1, |q|^-1 scale
  double G[kC];    // in units of ln 2
};
// Triangular 64 x 64 operands: 6 of 8 fragments, those of row tile i and
// 32-column step s that are not all zero.
constexpr int kTriFrags = 6;
constexpr int kTriBytes = kTriFrags * 2048;
// lower triangular: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1)
__host__ __device__ constexpr int low_frag(int i, int s) { return i < 2 ? i : 2 + 2 * (i - 2) + s; }
// its transpose, upper triangular: (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
__host__ __device__ constexpr int up_frag(int i, int s) { return i < 2 ? 2 * i + s : 2 + i; }

// ---- tokens whose state is asked for ----
// The first asked-for state of every token of the batch (-1: none), and of a
// state the next one after the same token: a token goes straight to its states,
// however many there are.  Null `of`: none are asked for.
struct Wanted {
  const int *of, *next;
  __device__ __forceinline__ int first(int64_t token) const {
    return of ? __builtin_amdgcn_readfirstlane(of[token]) : -1;
  }
  __device__ __forceinline__ int after(int s) const { return __builtin_amdgcn_readfirstlane(next[s]); }
};

// ---- pieces of a window ----
// Bits of the tokens t > 0 of a window at which a piece begins: another
// sequence, or behind a token whose state is asked for; `fresh`: where a
// sequence begins, t = 0 included (not at a row's start).
struct Cuts {
  uint64_t piece, fresh;
};
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
         ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32);
}
// Every lane of a wave calls this; row: the batch's first token, t0 the window's.
__device__ __forceinline__ Cuts window_cuts(const int* seq_idx, const Wanted& wanted, int64_t row, int64_t t0, int64_t L,
                                            int lane) {
  const int64_t t = t0 + lane;
  bool fresh = false, mark = false;
  if (t < L && t > 0) {
    if (seq_idx) fresh = seq_idx[row + t] != seq_idx[row + t - 1];
    if (wanted.of) mark = wanted.of[row + t - 1] >= 0;
  }
  Cuts c;
  c.fresh = uniform64(__ballot(fresh));
  c.piece = (c.fresh | uniform64(__ballot(mark))) & ~uint64_t(1);
  return c;
}
// The piece's number of token t.
__device__ __forceinline__ int piece_of(uint64_t cuts, int t) { return __popcll(cuts & (~uint64_t(0) >> (63 - t))); }
// The end of the piece that begins at a, in a window of n tokens.
__device__ __forceinline__ int piece_end(uint64_t cuts, int a, int n) {
  const uint64_t later = a >= 63 ? 0 : cuts >> (a + 1);
  return later ? min(n, a + 1 + (int)__builtin_ctzll(later)) : n;
}
// The beginning of the piece that ends before e.
__device__ __forceinline__ int piece_begin(uint64_t cuts, int e) {
  const uint64_t before = cuts & (~uint64_t(0) >> (64 - e));
  return before ? 63 - (int)__builtin_clzll(before) : 0;
}

// The pieces of a row in order.  The windows' cuts come from the preparation,
// the next one's asked for while one is walked.
struct Pieces {
  int64_t win, nw, L;
  const Cuts* list;  // of the row, or null: a piece a window
  Cuts cuts, next;
  int begin, end, n;
  __device__ __forceinline__ Cuts at(int64_t w) const {
    const Cuts none = {0, 0};
    return list && w >= 0 && w < nw ? list[w] : none;
  }
  // waited for and put into scalars where it is taken over
  __device__ __forceinline__ static Cuts uniform(const Cuts& c) { return {uniform64(c.piece), uniform64(c.fresh)}; }
  __device__ __forceinline__ int tokens() const { return (int)(L - win * kC < kC ? L - win * kC : kC); }
  // windows from .. to - 1
  __device__ __forceinline__ void first(const Cuts* l, int64_t from, int64_t to, int64_t len) {
    list = l;
    nw = to;
    L = len;
    win = from;
    cuts = uniform(at(from));
    next = at(from + 1);
    begin = 0;
    n = tokens();
    end = piece_end(cuts.piece, 0, n);
  }
  __device__ __forceinline__ bool valid() const { return win < nw; }
  __device__ __forceinline__ void step() {
    if (end < n) {
      begin = end;
    } else {
      ++win;
      cuts = uniform(next);
      next = at(win + 1);
      begin = 0;
      n = tokens();
    }
    end = piece_end(cuts.piece, begin, n);
  }
  // back to front
  __device__ __forceinline__ void last(const Cuts* l, int64_t windows, int64_t len) {
    list = l;
    nw = windows;
    L = len;
    win = nw - 1;
    cuts = uniform(at(win));
    next = at(win - 1);
    end = n = tokens();
    begin = piece_begin(cuts.piece, end);
  }
  __device__ __forceinline__ bool valid_back() const { return win >= 0; }
  __device__ __forceinline__ void step_back() {
    if (begin > 0) {
      end = begin;
    } else {
      --win;
      cuts = uniform(next);
      next = at(win - 1);
      end = n = kC;
    }
    begin = piece_begin(cuts.piece, end);
  }
  __device__ __forceinline__ bool fresh() const { return cuts.fresh >> begin & 1; }
};

// Eight slots of two accumulator tiles.
__device__ __forceinline__ void slots(const f32x4_t& lo, const f32x4_t& hi, float* o) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    o[r] = lo[r];
    o[4 + r] = hi[r];
  }
}

// ---- causality of values that are not numbers ----
// A product over tokens multiplies every token's value, those behind a row with
// zeros, and zero times a NaN or infinity is NaN.  So that a token reaches no
// earlier one, its values and all behind it in the column are taken out of such
// an operand and put in where a row only adds.  v: of tokens 16 i + 4 g + r.
template <class M>
__device__ __forceinline__ bool all_numbers(const f32x4_t* v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s += (fabsf(v[i][0]) + fabsf(v[i][1])) + (fabsf(v[i][2]) + fabsf(v[i][3]));
  return __builtin_expect(__ballot(!(s < M::kMost)) == 0, 1);
}
// Of the lane's column, the first token whose value cannot be an operand (kC:
// none).  Whole-register masks here and below: compares would hold two scalars
// each and push a chain's own out.
template <class M>
__device__ __forceinline__ int first_bad(const f32x4_t* v, int g) {
  int first = kC;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      int good = ((int)(__float_as_uint(v[i][r]) & 0x7fffffffu) - (int)__builtin_bit_cast(uint32_t, M::kMost)) >> 31;
      asm("" : "+v"(good));
      first = min(first, 16 * i + 4 * g + r + (good & kC));
    }
  first = min(first, __shfl_xor(first, 16, 64));
  return min(first, __shfl_xor(first, 32, 64));
}
// Values from token `first` on become `to`.
__device__ __forceinline__ void set_from(f32x4_t* v, int first, int g, float to) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      int on = (16 * i + 4 * g + r - first) >> 31;
      asm("" : "+v"(on));
      v[i][r] = __int_as_float((__float_as_int(v[i][r]) & on) | (__float_as_int(to) & ~on));
    }
}
// Makes v an operand and x, which the product is added to, NaN where v is none.
// Returns whether the lane's column has such a token.
template <class M>
__device__ __forceinline__ bool keep_causal(f32x4_t* v, f32x4_t* x, int g) {
  if (all_numbers<M>(v)) return false;
  const int first = first_bad<M>(v, g);
  set_from(x, first, g, __builtin_nanf(""));
  set_from(v, first, g, 0.f);
  return first < kC;
}

// ---- staging by a chain's helper waves ----
// The six fragments of a triangular operand.
template <int NTHR>
struct TriTile {
  static constexpr int NV = kTriBytes / 16 / NTHR;
  u32x4v q[NV];
  __device__ __forceinline__ void load(const char* p, int tid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = reinterpret_cast<const u32x4v*>(p)[tid + i * NTHR];
  }
  __device__ __forceinline__ void store(char* p, int tid) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) reinterpret_cast<u32x4v*>(p)[tid + i * NTHR] = q[i];
  }
};
// 64 rows of NP bf16 values (N of them there).
template <int NP, int NTHR>
struct RowTile {
  static constexpr int kPer = NP / 8, kRows = NTHR / kPer > 0 ? NTHR / kPer : 1, NV = kC * kPer / NTHR;
  static_assert(NTHR % kPer == 0 && kC % kRows == 0, "whole rows at a time");
  u32x4v q[NV];
  // the window's first row, rows `stride` apart
  __device__ __forceinline__ void load(const uint16_t* base, uint32_t stride, int N, int n, int tid) {
    const uint32_t col = tid % kPer * 8;
    const uint32_t off = (int)col < N ? (tid / kPer * stride + col) * 2 : kNowhere;
    const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * 2);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      q[i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, off, i * kRows * stride * 2, 0));
  }
  // PARTS: rows outside [begin, end) as zero
  template <bool PARTS>
  __device__ __forceinline__ void store(uint16_t* tile, int pitch, int begin, int end, int tid) const {
    const int t = tid / kPer, col = tid % kPer * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ti = t + i * kRows;
      u32x4v v = q[i];
      if constexpr (PARTS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ti >= begin && ti < end ? v[e] : 0u;
      }
      *reinterpret_cast<u32x4v*>(tile + ti * pitch + col) = v;
    }
  }
};
// The rows and gates of one piece for the general chains, brought by the waves
// of a block that hold no columns: asked for while the others work on the piece
// before, put when they are done.  Rows outside [begin, end) are zero.
template <class M, int NP, bool Q>
struct Stager {
  typedef typename M::IO::type T;
  static constexpr int V = M::IO::kVec, kPer = NP / V, es = 16 / V;
  static constexpr int kEach = kC * kPer / 128;    // of one tile, for the least number of threads
  static constexpr bool kAhead = NP < 256;          // else eight at a time when they are put, which spills less
  u32x4v k[kAhead ? kEach : 1], q[kAhead && Q ? kEach : 1];
  float gate[3];

  static __device__ __forceinline__ u32x4v ask(__amdgpu_buffer_rsrc_t r, int i, uint32_t stride, int N, int begin, int end) {
    const int t = i / kPer, col = i % kPer * V;
    const bool on = t >= begin && t < end && col < N;
    return __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, on ? (t * stride + col) * es : kNowhere, 0, 0));
  }
  static __device__ __forceinline__ void put(T* tile, int pitch, int i, u32x4v v) {
    if (i < kC * kPer) *reinterpret_cast<u32x4v*>(tile + i / kPer * pitch + i % kPer * V) = v;
  }
  static __device__ __forceinline__ void all(T* tile, int pitch, const T* base, uint32_t stride, int N, int n, int begin,
                                             int end, int tid, int nthr) {
    const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * es);
    for (int i0 = tid; i0 < kC * kPer; i0 += 8 * nthr) {
      u32x4v v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ask(r, i0 + e * nthr, stride, N, begin, end);
#pragma unroll
      for (int e = 0; e < 8; ++e) put(tile, pitch, i0 + e * nthr, v[e]);
    }
  }
  __device__ __forceinline__ void load(const T* kb, uint32_t ks, const T* qb, uint32_t qs, const float* gates, int N, int n,
                                       int begin, int end, int tid, int nthr) {
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      const int i = tid + e * nthr;
      gate[e] = i < 5 * kC && i % kC >= begin && i % kC < end ? gates[i] : 0.f;
    }
    if constexpr (kAhead) {
      const __amdgpu_buffer_rsrc_t rk = rows_of(kb, (uint32_t)n * ks * es);
#pragma unroll
      for (int e = 0; e < kEach; ++e) k[e] = ask(rk, tid + e * nthr, ks, N, begin, end);
      if constexpr (Q) {
        const __amdgpu_buffer_rsrc_t rq = rows_of(qb, (uint32_t)n * qs * es);
#pragma unroll
        for (int e = 0; e < kEach; ++e) q[e] = ask(rq, tid + e * nthr, qs, N, begin, end);
      }
    }
  }
  __device__ __forceinline__ void store(T* kt, T* qt, float* gt, int pitch, const T* kb, uint32_t ks, const T* qb, uint32_t qs,
                                        int N, int n, int begin, int end, int tid, int nthr) {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (tid + e * nthr < 5 * kC) gt[tid + e * nthr] = gate[e];
    if constexpr (kAhead) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) put(kt, pitch, tid + e * nthr, k[e]);
      if constexpr (Q) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) put(qt, pitch, tid + e * nthr, q[e]);
      }
    } else {
      all(kt, pitch, kb, ks, N, n, begin, end, tid, nthr);
      if constexpr (Q) all(qt, pitch, qb, qs, N, n, begin, end, tid, nthr);
    }
  }
};
// A lane's 16 tokens of one column of any type, zero outside [begin, end).
template <class IO>
__device__ __forceinline__ void load_column(const typename IO::type* base, uint32_t stride, uint32_t col, int n, int begin,
                                            int end, int g, uint32_t* q) {
  constexpr int es = sizeof(typename IO::type);
  const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * es);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int t = 16 * (e / 4) + 4 * g + e % 4;
    const uint32_t off = t >= begin && t < end ? (t * stride + col) * es : kNowhere;
    if constexpr (es == 2) q[e] = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else q[e] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
}
template <class IO>
__device__ __forceinline__ float column_value(uint32_t v) {
  return sizeof(typename IO::type) == 2 ? bf16_bits_to_f32(v) : __uint_as_float(v);
}
// Five gates of 64 tokens, zero outside [begin, end) (behind the row's end they are zero as prepared).
template <int NTHR>
struct GateTile {
  static constexpr int kAll = 5 * kC / 4, NV = (kAll + NTHR - 1) / NTHR;
  f32x4_t q[NV];
  __device__ __forceinline__ void load(const DeltaGates* g, int tid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = reinterpret_cast<const f32x4_t*>(g)[min(tid + i * NTHR, kAll - 1)];
  }
  template <bool PARTS>
  __device__ __forceinline__ void store(float* p, int begin, int end, int tid) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = tid + i * NTHR, t = 4 * e % kC;
      f32x4_t v = q[i];
      if constexpr (PARTS) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = t + r >= begin && t + r < end ? v[r] : 0.f;
      }
      if (e < kAll) reinterpret_cast<f32x4_t*>(p)[e] = v;
    }
  }
};
// A lane's 16 tokens (rows 16 i + 4 g + r) of one column, at lane offset
// (4 g stride + column) elements.
struct Column {
  uint32_t q[16];  // a register each: packed in pairs they would be waited for where they are asked for
  __device__ __forceinline__ static uint32_t row(int e) { return 16 * (e / 4) + e % 4; }
  __device__ __forceinline__ void load(const uint16_t* base, uint32_t stride, uint32_t off, int n) {
    const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * 2);
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = __builtin_amdgcn_raw_buffer_load_b16(r, off * 2, row(e) * stride * 2, 0);
  }
  __device__ __forceinline__ float get(int i, int r) const { return bf16_bits_to_f32(q[4 * i + r]); }
  template <bool PARTS>
  __device__ __forceinline__ static void put(uint16_t* base, uint32_t stride, uint32_t off, int n, const f32x4_t* v,
                                             int begin, int end, int g) {
    const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * 2);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int t = (int)row(e) + 4 * g;
      __builtin_amdgcn_raw_buffer_store_b16(IoBF16::put(v[e / 4][e % 4]), r,
                                            !PARTS || (t >= begin && t < end) ? off * 2 : kNowhere, row(e) * stride * 2, 0);
    }
  }
  template <bool PARTS>
  __device__ __forceinline__ static void put(float* base, uint32_t stride, uint32_t off, int n, const f32x4_t* v,
                                             int begin, int end, int g) {
    const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)n * stride * 4);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int t = (int)row(e) + 4 * g;
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e / 4][e % 4]), r,
                                            !PARTS || (t >= begin && t < end) ? off * 4 : kNowhere, row(e) * stride * 4, 0);
    }
  }
};
// A state's accumulators into [N, P] fp32 (N rows of them), lane offset (4 g P + column).
template <int NT>
__device__ __forceinline__ void put_state(float* base, int N, uint32_t P, uint32_t off, const f32x4_t* S) {
  const __amdgpu_buffer_rsrc_t r = rows_of(base, (uint32_t)N * P * 4);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[j][e]), r, off * 4, (16 * j + e) * P * 4, 0);
}

// Waves of a block go to the four SIMDs in turn.  Column waves keep theirs to
// themselves: of two and two others, the stagers are the seventh and eighth wave
// and share the others' SIMDs, and the two between end at once.
__host__ __device__ constexpr int first_stager(int C) { return C == 2 ? 6 : 2; }
__host__ __device__ constexpr int chain_threads(int C) { return 64 * (first_stager(C) + C); }

// Neighbouring blocks (slices of a head, heads of a group) on one XCD's L2.
__device__ __forceinline__ uint32_t near_block(uint32_t bid, uint32_t n) {
  return n % 8 == 0 ? (bid & 7u) * (n >> 3) + (bid >> 3) : bid;
}

// ---- the workspace ----
struct DeltaWs {
  int64_t nw;        // windows a row
  size_t gates, cuts, low_r, low_p, up_r, up_p, wanted, wanted_next, trans, enter, S, D, w, du, dq, dk, part, total;
  int64_t segs, seg_wins;  // stretches of a row that are walked side by side, and their windows
};
// segs, room: see delta_segments() and delta_stretch_room().
inline DeltaWs delta_ws(int64_t B, int64_t L, int64_t H, int64_t N, int64_t P, bool back, int64_t segs = 1, int64_t room = 0) {
  DeltaWs o = {};
  o.nw = (L + kDeltaC - 1) / kDeltaC;
  const size_t bhw = (size_t)(B * H * o.nw);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  o.gates = take(bhw * sizeof(DeltaGates));
  o.cuts = take((size_t)(B * o.nw) * 16);
  o.low_r = take(bhw * kTriBytes);
  if (!back) {
    o.low_p = take(bhw * kTriBytes);
    o.wanted = take((size_t)(B * L) * 4);
    o.wanted_next = take((size_t)kDeltaMaxStates * 4);
    o.segs = segs;
    o.seg_wins = (o.nw + segs - 1) / segs;
    o.trans = take((size_t)(room * N * (N + P)) * 4);
    o.enter = take((size_t)(room * N * P) * 4);
  } else {
    o.up_r = take(bhw * kTriBytes);
    o.up_p = take(bhw * kTriBytes);
    o.S = take(bhw * N * P * 4);
    o.D = take(bhw * N * P * 4);
    o.w = take(bhw * kDeltaC * P * 4);
    o.du = take(bhw * kDeltaC * P * 4);
    o.dq = take(bhw * kDeltaC * N * 4);
    o.dk = take(bhw * kDeltaC * N * 4);
    o.part = take(bhw * 2 * 4);
  }
  o.total = at;
  return o;
}

// Launches shared by the forward and the gradients (delta_rule.hip).
hipError_t launch_delta_prepare(const DeltaArgs& a, const DeltaWs& ws, bool back, bool bf16, hipStream_t s);
hipError_t launch_delta_chain(const DeltaArgs& a, const DeltaWs& ws, bool save, bool bf16, hipStream_t s);
// Column waves of a block of the general chains, of four waves; the others stage.
__host__ __device__ inline int chain_columns(int64_t P) { return P / 16 % 2 == 0 ? 2 : 1; }

}  // namespace ssd
