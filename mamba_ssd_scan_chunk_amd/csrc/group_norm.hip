// group_norm.hip -- norm of groups of a token's channels with an activation,
// its gradients, and activations in 8 bits.
//
// Per row and group of S = D / G columns, with act(z) = z / (1 + e^-z):
//     r = x,  or x act(z)  (gate first)
//     xh = (r - mean) rstd,  rstd = 1 / sqrt(mean((r - mean)^2) + eps)  (rms: mean = 0)
//     y = xh w + bias,  times act(z) (gate behind),  or act of itself (silu)
// Backward, with dy' the gradient of xh w + bias and v = dy' w:
//     dr = rstd (v - mean(v) - xh mean(v xh)),  dw = sum dy' xh,  dbias = sum dy'
// (rms: without mean(v)), from x and z as they were or from their 8 bits.
//
// Bound by memory: a thread holds 8 K consecutive columns' groups of 8 in
// registers between their one read and one write, a group is 2 to 64 lanes of
// a wave, or a block of 256 or 1024 threads past 2048 columns.  Loads and stores are of 8
// columns wherever a group begins; the hardware takes them at any element.
// 16384 x 5120 bf16 in groups of 64 with a gate out of rows of 10576: 110 us, 4.65
// TB/s (a copy: 5.0); gradients of 8192 x 4096 in groups of 128 from 8 bits: 61
// us, 4.5 TB/s, 5 of them the sum of dw (191 before a row's loads were asked for
// while the one in front is worked out).  8 bits of 16384 x 5376 out of rows of
// 10576: 56 us, 4.8 TB/s; back, 8192 x 1792: 9.6 us, 4.6 TB/s.
//
// 8 bits: 64 values share a bf16 scale, the least that times 127 reaches their
// largest magnitude, and are its nearest whole multiples, ties to even.  With
// so few bits in the scale and at most 24 in x a quotient is either a tie
// exactly or away from it by half a unit in its last place at least, so one
// correctly rounded division decides it.
#include "group_launch.hpp"
#include "layer_device.hpp"

namespace ssd {

// ---------------------------------------------------------------- 8 columns at any element
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

template <class IO>
__device__ __forceinline__ void get8(const typename IO::type* p, int left, float* o) {
  if (left >= 8) {
    if constexpr (sizeof(typename IO::type) == 2) {
      const u32x4_any q = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[2 * e] = __uint_as_float(q[e] << 16);
        o[2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
      }
    } else {
      const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = a[e];
        o[4 + e] = b[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = e < left ? IO::get(p[e]) : 0.f;
  }
}
template <class IO>
__device__ __forceinline__ void put8(typename IO::type* p, int left, const float* v) {
  if (left >= 8) {
    if constexpr (sizeof(typename IO::type) == 2) {
      u32x4_any q;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<u32x4_any*>(p) = q;
    } else {
      f32x4_any a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = v[e];
        b[e] = v[4 + e];
      }
      *reinterpret_cast<f32x4_any*>(p) = a;
      *reinterpret_cast<f32x4_any*>(p + 4) = b;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = IO::put(v[e]);
  }
}
// 8 bits at column col of a row of D: they lie in one or two blocks of a scale.
__device__ __forceinline__ void get8_kept(const int8_t* q, const uint16_t* scale, int64_t row, int col, int D, int left,
                                          float* o) {
  const int64_t nb = (D + (int)kPackBlock - 1) / (int)kPackBlock;
  const uint16_t* sc = scale + row * nb;
  const int8_t* p = q + row * D + col;
  if (left <= 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    return;
  }
  const int b0 = col / (int)kPackBlock, b1 = min(col + 7, D - 1) / (int)kPackBlock;
  const float s0 = bf16_bits_to_f32(sc[b0]), s1 = bf16_bits_to_f32(sc[b1]);
  const int cut = (b0 + 1) * (int)kPackBlock - col;  // elements of the first block
  int8_t v[8];
  if (left >= 8) {
    const u32x2_any w = *reinterpret_cast<const u32x2_any*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : (int8_t)0;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = e < left ? (float)v[e] * (e < cut ? s0 : s1) : 0.f;
}

// Sum over the T threads of a group (T > 64: the block).
template <int T>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int o = 1; o < (T < 64 ? T : 64); o <<= 1) v += __shfl_xor(v, o, 64);
  if constexpr (T > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < T / 64; ++k) v += red[k];
  }
  return v;
}

// Column in the group of chunk k of a thread (lane l of T): chunks of a group's
// threads lie side by side.
template <int T>
__device__ __forceinline__ int chunk_col(int k, int l) { return 8 * (k * T + l); }

// Threads of a block: groups of a block's threads and more take one each.
constexpr int group_block(int T) { return T > 256 ? T : 256; }

template <class IO, int T, int K>
__global__ __launch_bounds__(group_block(T)) void group_norm_forward_kernel(GroupNormArgs a) {
  typedef typename IO::type E;
  __shared__ float red[16];
  const int l = threadIdx.x % T;
  const uint32_t gi = (uint32_t)flat_block() * (group_block(T) / T) + threadIdx.x / T;
  const uint32_t G = (uint32_t)a.G;
  const int S = (int)(a.D / a.G);
  const uint32_t row = gi / G, grp = gi - row * G;
  const bool on = row < (uint64_t)a.rows;  // whole blocks where T > 64
  const float inv = 1.f / (float)S;
  const E* x = static_cast<const E*>(a.x) + (int64_t)row * a.D + (int64_t)grp * S;
  const E* z = static_cast<const E*>(a.z) + (int64_t)row * a.z_row + (int64_t)grp * S;
  float v[K][8], zv[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = chunk_col<T>(k, l), left = on ? S - c : 0;
    get8<IO>(x + c, left, v[k]);
    if (a.z) get8<IO>(z + c, left, zv[k]);
  }
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (a.z) {
#pragma unroll
      for (int e = 0; e < 8; ++e) zv[k][e] *= sigmoid(zv[k][e]);
    }
    if (a.gate_first) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] *= zv[k][e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += v[k][e];
  }
  float mean = 0.f;
  if (!a.rms) mean = group_sum<T>(sum, red) * inv;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = chunk_col<T>(k, l) + e < S ? v[k][e] - mean : 0.f;
      v[k][e] = d;
      ss = fmaf(d, d, ss);
    }
  const float rstd = 1.f / sqrtf(group_sum<T>(ss, red) * inv + a.eps);
  if (!on) return;
  if (l == 0) {
    a.rstd[gi] = rstd;
    if (!a.rms) a.mean[gi] = mean;
  }
  const int64_t w0 = a.shared ? 0 : (int64_t)grp * S;
  E* y = static_cast<E*>(a.y) + (int64_t)row * a.D + (int64_t)grp * S;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = chunk_col<T>(k, l), left = S - c;
    float w[8], b[8];
    get8<IoF32>(a.w + w0 + c, left, w);
    if (a.bias) get8<IoF32>(a.bias + w0 + c, left, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float o = v[k][e] * rstd * w[e];
      if (a.bias) o += b[e];
      if (a.z && !a.gate_first) o *= zv[k][e];
      if (a.silu) o *= sigmoid(o);
      v[k][e] = o;
    }
    put8<IO>(y + c, left, v[k]);
  }
}

// Lanes of a row side by side, a block's from blockIdx.x on; rows from
// blockIdx.y on in steps.  A thread keeps its columns, and dw and dbias of them
// in registers.
struct GroupWalk {
  int lanes;      // of a row: G T
  int per_block;  // of them in a block
  int slots;      // rows a block takes at once
  int col_blocks;
  int row_blocks;
};

// What a row's eight columns are in memory, held so until they are widened: the
// next row's are asked for before this one is worked out.
template <class IO, bool KEPT>
struct GroupRaw {
  typedef typename IO::type E;
  static constexpr int kW = sizeof(E) * 2;  // 4-byte words of 8 elements
  uint32_t dy[kW], x[KEPT ? 2 : kW], z[KEPT ? 2 : kW];
  uint16_t s[4];  // KEPT: scales of x and z at the first and the last column
  template <int W>
  __device__ __forceinline__ static void words(const void* p, uint32_t* o) {
    if constexpr (W == 2) {
      const u32x2_any q = *static_cast<const u32x2_any*>(p);
      o[0] = q[0]; o[1] = q[1];
    } else {
#pragma unroll
      for (int k = 0; k < W; k += 4) {
        const u32x4_any q = static_cast<const u32x4_any*>(p)[k / 4];
        o[k] = q[0]; o[k + 1] = q[1]; o[k + 2] = q[2]; o[k + 3] = q[3];
      }
    }
  }
  __device__ __forceinline__ void load(const GroupNormArgs& a, int64_t row, int col) {
    words<kW>(static_cast<const E*>(a.dy) + row * a.D + col, dy);
    if constexpr (KEPT) {
      const int64_t nb = (a.D + kPackBlock - 1) / kPackBlock, b0 = row * nb + col / (int)kPackBlock,
                    b1 = row * nb + (col + 7) / (int)kPackBlock;
      words<2>(static_cast<const int8_t*>(a.x) + row * a.D + col, x);
      s[0] = a.xs[b0];
      s[1] = a.xs[b1];
      if (a.z) {
        words<2>(static_cast<const int8_t*>(a.z) + row * a.D + col, z);
        s[2] = a.zs[b0];
        s[3] = a.zs[b1];
      }
    } else {
      words<kW>(static_cast<const E*>(a.x) + row * a.D + col, x);
      if (a.z) words<kW>(static_cast<const E*>(a.z) + row * a.z_row + col, z);
    }
  }
  __device__ __forceinline__ static void widen(const uint32_t* w, float* o) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (sizeof(E) == 2) o[e] = __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
      else o[e] = __uint_as_float(w[e]);
    }
  }
  __device__ __forceinline__ static void widen8(const uint32_t* w, uint16_t s0, uint16_t s1, int cut, float* o) {
    const float f0 = bf16_bits_to_f32(s0), f1 = bf16_bits_to_f32(s1);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (float)(int8_t)(w[e / 4] >> (8 * (e % 4))) * (e < cut ? f0 : f1);
  }
  __device__ __forceinline__ void get(int col, bool gate, float* dyv, float* xv, float* zv) const {
    widen(dy, dyv);
    if constexpr (KEPT) {
      const int cut = (int)kPackBlock - col % (int)kPackBlock;
      widen8(x, s[0], s[1], cut, xv);
      if (gate) widen8(z, s[2], s[3], cut, zv);
    } else {
      widen(x, xv);
      if (gate) widen(z, zv);
    }
  }
};

// FULL: groups of whole eights.
template <class IO, int T, int K, bool KEPT, bool FULL>
__global__ __launch_bounds__(group_block(T)) void group_norm_backward_kernel(GroupNormArgs a, GroupWalk w) {
  typedef typename IO::type E;
  constexpr int BT = group_block(T);
  __shared__ float red[16];
  extern __shared__ float sums[];  // shared weights: a block's dw and dbias by thread
  const int slot = threadIdx.x / w.per_block, in = threadIdx.x % w.per_block;
  const int lane = blockIdx.x * w.per_block + in;
  const int S = (int)(a.D / a.G), D = (int)a.D;
  const int grp = lane / T, l = lane % T;
  const bool live = slot < w.slots && lane < w.lanes;
  const float inv = 1.f / (float)S;
  float wv[K][8], bv[K][8], dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = chunk_col<T>(k, l), left = live ? S - c : 0;
    const int64_t w0 = (a.shared ? 0 : (int64_t)grp * S) + c;
    get8<IoF32>(a.w + w0, left, wv[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) bv[k][e] = dw[k][e] = db[k][e] = 0.f;
    if (a.bias) get8<IoF32>(a.bias + w0, left, bv[k]);
  }
  // FULL: threads past the group's end, or the row's lanes, read its last columns instead
  GroupRaw<IO, KEPT> raw[FULL ? K : 1];
  float rn = 0.f, mn = 0.f;
  auto ask = [&](int64_t r0) {
    const int64_t r = r0 + slot < a.rows ? r0 + slot : a.rows - 1;
    const int gq = live ? grp : 0;
    rn = a.rstd[r * a.G + gq];
    mn = a.rms ? 0.f : a.mean[r * a.G + gq];
    if constexpr (FULL) {
#pragma unroll
      for (int k = 0; k < K; ++k) raw[k].load(a, r, gq * S + min(chunk_col<T>(k, l), S - 8));
    }
  };
  const int64_t step = (int64_t)w.row_blocks * w.slots;
  ask((int64_t)blockIdx.y * w.slots);
  for (int64_t r0 = (int64_t)blockIdx.y * w.slots; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + slot;
    const bool on = live && row < a.rows;
    const float rstd = rn, mean = mn;
    float x[K][8], z[K][8], dy[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = chunk_col<T>(k, l), left = on ? S - c : 0, col = grp * S + c;
      if constexpr (FULL) {
        raw[k].get((live ? grp : 0) * S + min(c, S - 8), a.z != nullptr, dy[k], x[k], z[k]);
        if (left <= 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dy[k][e] = 0.f;
        }
      } else {
        get8<IO>(static_cast<const E*>(a.dy) + row * D + col, left, dy[k]);
        if constexpr (KEPT) {
          get8_kept(static_cast<const int8_t*>(a.x), a.xs, row, col, D, left, x[k]);
          if (a.z) get8_kept(static_cast<const int8_t*>(a.z), a.zs, row, col, D, left, z[k]);
        } else {
          get8<IO>(static_cast<const E*>(a.x) + row * D + col, left, x[k]);
          if (a.z) get8<IO>(static_cast<const E*>(a.z) + row * a.z_row + col, left, z[k]);
        }
      }
    }
    if (r0 + step < a.rows) ask(r0 + step);
    float s1 = 0.f, s2 = 0.f;
    float xh[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = chunk_col<T>(k, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool has = on && c + e < S;
        float g = dy[k][e], r = x[k][e];
        float sg = 0.f, act = 0.f;
        if (a.z) {
          sg = sigmoid(z[k][e]);
          act = z[k][e] * sg;
        }
        if (a.gate_first) r *= act;
        const float h = has ? (r - mean) * rstd : 0.f;
        const float pre = fmaf(h, wv[k][e], bv[k][e]);
        if (a.z && !a.gate_first) {
          x[k][e] = g * pre * dsilu(z[k][e], sg);  // dz
          g = has ? g * act : 0.f;
        }
        if (a.silu) g *= dsilu(pre, sigmoid(pre));
        dw[k][e] = fmaf(g, h, dw[k][e]);
        db[k][e] += g;
        const float v = g * wv[k][e];
        s1 += v;
        s2 = fmaf(v, h, s2);
        xh[k][e] = h;
        dy[k][e] = v;
      }
    }
    const float m2 = group_sum<T>(s2, red) * inv;
    const float m1 = a.rms ? 0.f : group_sum<T>(s1, red) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = chunk_col<T>(k, l), left = on ? S - c : 0, col = grp * S + c;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float d = rstd * (dy[k][e] - m1 - xh[k][e] * m2);
        if (a.gate_first) {
          const float sg = sigmoid(z[k][e]);
          x[k][e] = d * x[k][e] * dsilu(z[k][e], sg);
          d *= z[k][e] * sg;
        }
        o[e] = d;
      }
      if (FULL ? left > 0 : true) {
        const int take = FULL ? 8 : left;
        put8<IO>(static_cast<E*>(a.dx) + row * D + col, take, o);
        if (a.z) put8<IO>(static_cast<E*>(a.dz) + row * a.dz_row + col, take, x[k]);
      }
    }
  }
  if constexpr (T < BT) {
    if (a.shared) {
      // the block's groups and rows have the same columns: one sum of them a block
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p && !a.db) break;
        float* out = a.ws + ((int64_t)p * w.row_blocks * w.col_blocks + (int64_t)blockIdx.y * w.col_blocks + blockIdx.x) * S;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < 8; ++e) sums[e * BT + threadIdx.x] = live ? (p ? db[k][e] : dw[k][e]) : 0.f;
          __syncthreads();
          // thread i adds element i / T of lane i % T over the block's BT / T of them
          for (int i = threadIdx.x; i < 8 * T; i += BT) {
            const int e = i / T, ll = i % T;
            float v = 0.f;
            for (int q = 0; q < BT / T; ++q) v += sums[e * BT + q * T + ll];
            const int c = chunk_col<T>(k, ll) + e;
            if (c < S) out[c] = v;
          }
        }
      }
      return;
    }
  }
  // a partial sum of every column by row block and slot, [.. , G, S] twice
  if (!live) return;
  const int64_t part = ((int64_t)blockIdx.y * w.slots + slot) * D + (int64_t)grp * S;
  float* pw = a.ws + part;
  float* pb = pw + (int64_t)w.row_blocks * w.slots * D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = chunk_col<T>(k, l);
    put8<IoF32>(pw + c, S - c, dw[k]);
    if (a.db) put8<IoF32>(pb + c, S - c, db[k]);
  }
}

// 64 columns a block of `cols`; blockIdx.y: dw or dbias.
// `rows` partial sums of each.
__global__ __launch_bounds__(kColsumThreads) void group_norm_param_kernel(GroupNormArgs a, int cols, int64_t rows) {
  __shared__ float lds[kColsumThreads];
  const int lane = threadIdx.x & 63;
  const int c = blockIdx.x * 64 + lane;
  const float* p = a.ws + (blockIdx.y ? rows * cols : 0) + min(c, cols - 1);
  const float s = column_sum(p, rows, cols, lds);
  if (threadIdx.x < 64 && c < cols) (blockIdx.y ? a.db : a.dw)[c] = s;
}

// ---------------------------------------------------------------- 8 bits
template <class IO>
__global__ __launch_bounds__(256) void pack8_kernel(int64_t rows, int D, const typename IO::type* x, int64_t x_row,
                                                    int8_t* q, uint16_t* scale) {
  const int nb = (D + (int)kPackBlock - 1) / (int)kPackBlock;
  const int64_t i = (int64_t)flat_block() * 32 + (threadIdx.x >> 3);  // a block of 64 values, 8 lanes
  const int64_t row = i / nb;
  const int blk = (int)(i - row * nb), col = blk * (int)kPackBlock + 8 * (threadIdx.x & 7);
  const bool on = row < rows;
  const int left = on ? D - col : 0;
  float v[8];
  get8<IO>(x + row * x_row + col, left, v);
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o, 64));
  uint32_t sb;
  const bool bad = most >= 0x7f800000u;  // an infinity or NaN among them: all come back as NaN
  if (bad) {
    sb = 0x7fc0u;
  } else {
    const float m = __uint_as_float(most);
    sb = f32_to_bf16_bits(m / 127.f);
    if (bf16_bits_to_f32(sb) * 127.f < m) ++sb;
  }
  const float s = bf16_bits_to_f32(sb);
  uint32_t w[2] = {0, 0};
  if (!bad && s > 0.f) {
    const float inv = 1.f / s;
    const bool far = s < 1e-35f;  // 1 / s near the largest value: divide
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // x inv, then its remainder's share: the correctly rounded quotient
      float t = v[e] * inv;
      t = far ? v[e] / s : fmaf(fmaf(-t, s, v[e]), inv, t);
      w[e / 4] |= ((uint32_t)(int)rintf(t) & 0xffu) << (8 * (e % 4));
    }
  }
  if (!on) return;
  if ((threadIdx.x & 7) == 0) scale[i] = (uint16_t)sb;
  int8_t* o = q + row * D + col;
  if (left >= 8) {
    u32x2_any p;
    p[0] = w[0];
    p[1] = w[1];
    *reinterpret_cast<u32x2_any*>(o) = p;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) o[e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

template <class IO>
__global__ __launch_bounds__(256) void unpack8_kernel(int64_t rows, int D, const int8_t* q, const uint16_t* scale,
                                                      typename IO::type* x, int64_t x_row) {
  const int nb = (D + (int)kPackBlock - 1) / (int)kPackBlock;
  const int64_t i = (int64_t)flat_block() * 32 + (threadIdx.x >> 3);
  const int64_t row = i / nb;
  const int col = (int)(i - row * nb) * (int)kPackBlock + 8 * (threadIdx.x & 7);
  if (row >= rows) return;
  float v[8];
  get8_kept(q, scale, row, col, D, D - col, v);
  put8<IO>(x + row * x_row + col, D - col, v);
}

// ---------------------------------------------------------------- launches
// Threads of a group: the fewest whose 8 columns each cover it, at most a wave
// (then K times 8), past 2048 columns a block.
static int group_threads(int64_t S) {
  if (S > 2048) return S > 4096 ? 1024 : 256;
  int t = 2;
  while (t < 64 && 8 * t < S) t *= 2;
  return t;
}
static GroupWalk group_walk(int64_t rows, int64_t G, int T) {
  GroupWalk w;
  w.lanes = (int)(G * T);
  const int block = group_block(T);
  w.per_block = w.lanes < block ? w.lanes : block;
  w.slots = block / w.per_block;
  w.col_blocks = (w.lanes + block - 1) / block;
  // three blocks a compute unit are there at once
  int64_t rb = (int64_t)device_cu_count() * (block > 256 ? 1 : 3) / w.col_blocks;
  const int64_t most = (rows + w.slots - 1) / w.slots;
  if (rb > most) rb = most;
  w.row_blocks = (int)(rb < 1 ? 1 : rb > 65535 ? 65535 : rb);
  return w;
}
size_t group_norm_backward_ws_bytes(int64_t rows, int64_t D, int64_t G) {
  const GroupWalk w = group_walk(rows, G, group_threads(D / G));
  return (size_t)w.row_blocks * w.slots * D * 2 * 4;
}

template <class IO, int T, int K>
static hipError_t forward(const GroupNormArgs& a, hipStream_t s) {
  const int64_t per = group_block(T) / T;
  hipLaunchKernelGGL((group_norm_forward_kernel<IO, T, K>), flat_grid((a.rows * a.G + per - 1) / per),
                     dim3(group_block(T)), 0, s, a);
  return hipGetLastError();
}
template <class IO, int T, int K, bool KEPT, bool FULL>
static hipError_t backward_as(const GroupNormArgs& a, const GroupWalk& w, hipStream_t s) {
  constexpr int BT = group_block(T);
  const size_t lds = T < BT && a.shared ? (size_t)8 * BT * 4 : 0;
  hipLaunchKernelGGL((group_norm_backward_kernel<IO, T, K, KEPT, FULL>),
                     dim3((unsigned)w.col_blocks, (unsigned)w.row_blocks), dim3(BT), lds, s, a, w);
  return hipGetLastError();
}
template <class IO, int T, int K>
static hipError_t backward(const GroupNormArgs& a, hipStream_t s) {
  const GroupWalk w = group_walk(a.rows, a.G, T);
  const bool full = a.D / a.G % 8 == 0;
  hipError_t e;
  if (a.xs) e = full ? backward_as<IO, T, K, true, true>(a, w, s) : backward_as<IO, T, K, true, false>(a, w, s);
  else e = full ? backward_as<IO, T, K, false, true>(a, w, s) : backward_as<IO, T, K, false, false>(a, w, s);
  if (e != hipSuccess) return e;
  const int cols = (int)(a.shared ? a.D / a.G : a.D);
  int64_t rows = (int64_t)w.row_blocks * w.slots;
  if (a.shared) rows = T < group_block(T) ? (int64_t)w.row_blocks * w.col_blocks : rows * a.G;
  hipLaunchKernelGGL(group_norm_param_kernel, dim3((unsigned)((cols + 63) / 64), a.db ? 2 : 1), dim3(kColsumThreads), 0,
                     s, a, cols, rows);
  return hipGetLastError();
}
#define SSD_GROUP_CASES(f)                          \
  const int64_t S = a.D / a.G;                      \
  switch (group_threads(S)) {                       \
    case 2: return f<IO, 2, 1>(a, s);               \
    case 4: return f<IO, 4, 1>(a, s);               \
    case 8: return f<IO, 8, 1>(a, s);               \
    case 16: return f<IO, 16, 1>(a, s);             \
    case 32: return f<IO, 32, 1>(a, s);             \
    case 64:                                        \
      if (S <= 512) return f<IO, 64, 1>(a, s);      \
      return S <= 1024 ? f<IO, 64, 2>(a, s) : f<IO, 64, 4>(a, s); \
    case 256: return f<IO, 256, 2>(a, s);           \
    default: return f<IO, 1024, 2>(a, s);           \
  }
template <class IO>
static hipError_t forward_of(const GroupNormArgs& a, hipStream_t s) { SSD_GROUP_CASES(forward) }
template <class IO>
static hipError_t backward_of(const GroupNormArgs& a, hipStream_t s) { SSD_GROUP_CASES(backward) }
#undef SSD_GROUP_CASES

hipError_t launch_group_norm_forward(const GroupNormArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? forward_of<IoBF16>(a, s) : forward_of<IoF32>(a, s);
}
hipError_t launch_group_norm_backward(const GroupNormArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? backward_of<IoBF16>(a, s) : backward_of<IoF32>(a, s);
}

hipError_t launch_pack8(int64_t rows, int64_t D, const void* x, int64_t x_row, bool bf16, int8_t* q, uint16_t* scale,
                        hipStream_t s) {
  const dim3 grid = flat_grid((rows * ((D + kPackBlock - 1) / kPackBlock) + 31) / 32);
  if (bf16) hipLaunchKernelGGL(pack8_kernel<IoBF16>, grid, dim3(256), 0, s, rows, (int)D, static_cast<const uint16_t*>(x), x_row, q, scale);
  else hipLaunchKernelGGL(pack8_kernel<IoF32>, grid, dim3(256), 0, s, rows, (int)D, static_cast<const float*>(x), x_row, q, scale);
  return hipGetLastError();
}
hipError_t launch_unpack8(int64_t rows, int64_t D, const int8_t* q, const uint16_t* scale, void* x, int64_t x_row,
                          bool bf16, hipStream_t s) {
  const dim3 grid = flat_grid((rows * ((D + kPackBlock - 1) / kPackBlock) + 31) / 32);
  if (bf16) hipLaunchKernelGGL(unpack8_kernel<IoBF16>, grid, dim3(256), 0, s, rows, (int)D, q, scale, static_cast<uint16_t*>(x), x_row);
  else hipLaunchKernelGGL(unpack8_kernel<IoF32>, grid, dim3(256), 0, s, rows, (int)D, q, scale, static_cast<float*>(x), x_row);
  return hipGetLastError();
}

}  // namespace ssd
