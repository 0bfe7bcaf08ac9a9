// selective_scan.hpp -- what the selective scan's forward and backward kernels
// share: the split of the work over waves, and the packed form of B, C and A
// that their inner loops read.
#pragma once

#include <type_traits>

#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace ssd {

constexpr int kScanT = 16;  // tokens held in registers at a time (a tile)

struct ScanGrid {
  int64_t Q, nc;     // tokens a chunk (a multiple of kScanT), chunks
  int64_t ncb;       // blocks of 64 channels per group
  int64_t ntile;     // tiles of a row
};

struct ScanWs {
  float* carry;      // [B,nc,N,D] states
  float* sdt;        // [B,nc,D] summed time steps of a chunk (since its last restart)
  int* cut;          // [B,nc] whether a sequence starts inside the chunk
  float* adj;        // backward: [B,nc,N,D] adjoint states
  float* bc;         // [B,G,ntile,N][kEntry] fp32, and one entry more
  float* at;         // [N,D] A
  uint32_t* starts;  // [B,ntile] bit i: token i of the tile begins another sequence
  float* tstate;     // backward: [B,ntile,N,D] states entering each tile, from a zero chunk start
  float* tsdt;       // backward: [B,ntile,D] time steps summed up to the tile (since the last restart)
};

struct ScanBlock {
  int64_t b, c, grp, cb, d0, dend, t0, t1;
};

// Grid (G * ncb, chunks, B), a wave a block: consecutive blocks take
// neighbouring channels of the same tokens, which share their rows of B and C.
__device__ __forceinline__ ScanBlock scan_block(const ScanGrid& g, const ScanArgs& a) {
  ScanBlock k;
  const int64_t gd = a.D / a.G;
  k.grp = blockIdx.x / (unsigned)g.ncb;
  k.cb = blockIdx.x % (unsigned)g.ncb;
  k.d0 = k.grp * gd + k.cb * 64;
  k.dend = (k.grp + 1) * gd;
  k.c = blockIdx.y;
  k.b = blockIdx.z;
  k.t0 = k.c * g.Q;
  k.t1 = k.t0 + g.Q < a.L ? k.t0 + g.Q : a.L;
  return k;
}

// B and C of one state over the 16 tokens of a tile, in two halves.  They are
// the same for all lanes (channels), so they are read by scalar loads of 64
// bytes and feed the vector ALU as scalar operands.  Scalar loads return out
// of order and can only be waited for all together: `settle` makes the half in
// hand arrive before the next one is asked for, whose latency then hides
// behind the arithmetic of this one (and of the SIMD's other waves).
typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
constexpr int kHalf = kScanT / 2;
constexpr int kEntry = 2 * kScanT;  // floats of a state's [B0-7 | C0-7 | B8-15 | C8-15]
template <bool WANT_C>
struct BCHalf {
  typedef std::conditional_t<WANT_C, f32x16_t, f32x8_t> vec;
  vec v;
  __device__ __forceinline__ void load(const float* p) {
    v = *(const __attribute__((address_space(4))) vec*)(uintptr_t)p;
  }
  __device__ __forceinline__ void settle() { asm volatile("" : "+s"(v)); }
  __device__ __forceinline__ float b(int i) const { return v[i]; }
  __device__ __forceinline__ float c(int i) const { return v[kHalf + i]; }
};

template <bool WANT_C>
struct BCPair {
  BCHalf<WANT_C> lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo.load(p);
    hi.load(p + kScanT);
  }
  __device__ __forceinline__ void settle() {
    lo.settle();
    hi.settle();
  }
  __device__ __forceinline__ float b(int i) const { return i < kHalf ? lo.b(i) : hi.b(i - kHalf); }
  __device__ __forceinline__ float c(int i) const { return i < kHalf ? lo.c(i) : hi.c(i - kHalf); }
};

// Lines that coming loads will need, asked for early, one a lane, and held until
// `settle`.  A tile's entries miss its die's L2 when first read, and the states
// would wait for theirs one after another: 2 x 8192 tokens of 5120 channels
// 565 us without, 491 with; 1 x 4 tokens of 1058 channels, 32 states, 31 and 20.
struct Touch {
  float v;
  // the entries (128 bytes) of N states, the first 64 of them
  __device__ __forceinline__ void entries(const float* p, int N, int lane) {
    v = p[(lane < N ? lane : N - 1) * kEntry];
  }
  __device__ __forceinline__ void settle() { asm volatile("" : : "v"(v)); }
};

// Rows 0..N-1 of [N, D], a channel a lane, to or from LDS, 16 rows' loads at a
// time (N is a multiple of 4; past it the last row again).
__device__ __forceinline__ void rows_to_lds(float* dst, const float* src, int64_t D, int N) {
  for (int n0 = 0; n0 < N; n0 += 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = src[(n0 + i < N ? n0 + i : N - 1) * D];
#pragma unroll
    for (int i = 0; i < 16; ++i) dst[(n0 + i < N ? n0 + i : N - 1) * 64] = v[i];
  }
}

// Tokens of the tile at t0 (uniform, kept in 32 bits).
__device__ __forceinline__ int tile_tokens(const ScanBlock& k, int64_t t0) {
  return __builtin_amdgcn_readfirstlane((int)(k.t1 - t0 < kScanT ? k.t1 - t0 : kScanT));
}

// The waves of a SIMD have equal work, but its arbiter prefers the oldest: left
// alone they finish one after the other, the last ones with nobody to fill
// their stalls.  Each lowers its priority after 1/2, 3/4 and 7/8 of its tiles,
// so that the ones behind catch up there and all end within an eighth of each
// other.
__device__ __forceinline__ void pace(int64_t done, int64_t all) {
  if (done * 2 < all) __builtin_amdgcn_s_setprio(3);
  else if (done * 4 < all * 3) __builtin_amdgcn_s_setprio(2);
  else if (done * 8 < all * 7) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

// Raw elements of a tile, one channel a lane: buffer loads from the tile's
// first row, the token's row as the scalar offset (the last token's again past
// the tile's nt tokens), `off` the lane's byte offset in a row.
template <class IO>
struct RawTile {
  typename IO::type v[kScanT];
  __device__ __forceinline__ void load(const typename IO::type* base, int64_t row, int64_t t0, int nt, int off) {
    constexpr int es = sizeof(typename IO::type);
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<typename IO::type*>(base + t0 * row), 0, 0x7fffffff, 0x00027000);
    const int step = (int)row * es;
    if (nt == kScanT) {
      int so = 0;
#pragma unroll
      for (int i = 0; i < kScanT; ++i) {
        v[i] = load1(r, off, so);
        so += step;
        asm volatile("" : "+s"(so));  // one running offset, not sixteen multiples kept in registers
      }
    } else {
#pragma unroll
      for (int i = 0, so = 0; i < kScanT; ++i, so += i < nt ? step : 0) v[i] = load1(r, off, so);
    }
  }
  __device__ __forceinline__ static typename IO::type load1(__amdgpu_buffer_rsrc_t r, int off, int so) {
    if constexpr (IO::kVec == 8) return __builtin_amdgcn_raw_buffer_load_b16(r, off, so, 0);
    else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, so, 0));
  }
  __device__ __forceinline__ float at(int i) const { return IO::get(v[i]); }
};
// The same for storing.
template <class IO>
__device__ __forceinline__ void store_tile(typename IO::type* base, int64_t row, int64_t t0, int nt, int off,
                                           const float (&v)[kScanT]) {
  constexpr int es = sizeof(typename IO::type);
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(base + t0 * row, 0, 0x7fffffff, 0x00027000);
  const int step = (int)row * es;
  auto put = [&](int i, int so) {
    if constexpr (es == 2) __builtin_amdgcn_raw_buffer_store_b16(IO::put(v[i]), r, off, so, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), r, off, so, 0);
  };
  int so = 0;
  if (nt == kScanT) {
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      put(i, so);
      so += step;
      asm volatile("" : "+s"(so));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScanT; ++i) {
      if (i < nt) put(i, so);
      so += step;
      asm volatile("" : "+s"(so));
    }
  }
}

// Time steps of a tile from the raw projections, in units of ln 2: the decay is
// then exp2(dt A), and the softplus log2(1 + 2^w) needs no scaling but that of
// its argument.  Packed B is scaled by ln 2 in exchange.  Zero past the tile's
// tokens, where the decay is then 1.  `bias` is in the same units.
template <class IO>
__device__ __forceinline__ void time_steps(const RawTile<IO>& raw, float bias, bool plus, int nt, float (&dt)[kScanT]) {
#pragma unroll
  for (int i = 0; i < kScanT; ++i) dt[i] = fmaf(raw.at(i), kLog2e, bias);
  if (plus) {
#pragma unroll
    for (int i = 0; i < kScanT; ++i) dt[i] = softplus2(dt[i]);
  }
  if (nt < kScanT) {
#pragma unroll
    for (int i = 0; i < kScanT; ++i)
      if (i >= nt) dt[i] = 0.f;
  }
}

// Floats of the packed B and C (the entry more is what the last prefetch reads).
inline int64_t scan_bc_floats(int64_t B, int64_t G, int64_t ntile, int64_t N) { return (B * G * ntile * N + 1) * kEntry; }

// Fills ws.bc, ws.at and (packed sequences) ws.starts.
hipError_t launch_scan_pack(const ScanArgs& a, const ScanGrid& g, const ScanWs& ws, bool bf16, hipStream_t s);

// Carries ws.carry and, where there is one, ws.adj from chunk to chunk.
hipError_t launch_scan_carry(const ScanArgs& a, const ScanGrid& g, const ScanWs& ws, hipStream_t s);

}  // namespace ssd
