// api_checks.hpp -- argument checks shared by the C ABI layers of the layer
// operators (layer_api.cpp) and of the delta rule and what goes with it
// (delta_api.cpp).  Host only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "ssd.h"

namespace ssd {
namespace api {

constexpr int64_t k31 = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 46;  // far below where byte offsets leave 64 bits

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool a16(const void* p) { return aligned(p, 16); }  // true for NULL

inline ssd_status check_dtype(ssd_dtype t) { return (t == SSD_F32 || t == SSD_BF16) ? SSD_OK : SSD_ERR_DTYPE; }
inline ssd_status from_hip(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }
inline uintptr_t elem(ssd_dtype t) { return t == SSD_BF16 ? 2 : 4; }

#define SSD_TRY(expr)              \
  do {                             \
    const ssd_status st_ = (expr); \
    if (st_ != SSD_OK) return st_; \
  } while (0)

// A product of positive sizes, or SSD_ERR_UNSUPPORTED past `most`.
inline ssd_status product(std::initializer_list<int64_t> f, int64_t most) {
  int64_t p = 1;
  for (int64_t v : f) {
    if (v > most / p) return SSD_ERR_UNSUPPORTED;
    p *= v;
  }
  return SSD_OK;
}

// A row stride: 0 stands for `dense`; shorter rows than the channels overlap.
// Up to 16 rows of a sequence are addressed by 32-bit byte offsets from the first.
inline bool row_too_long(int64_t seqlen, int64_t row) { return seqlen > 1 && row >= int64_t(1) << 25; }

inline ssd_status row_stride(int64_t given, int64_t dense, int64_t batch, int64_t seqlen, int64_t* out) {
  if (given == 0) given = dense;
  if (given < dense) return SSD_ERR_SHAPE;
  SSD_TRY(product({batch, seqlen, given}, kMaxElems));
  if (row_too_long(seqlen, given)) return SSD_ERR_UNSUPPORTED;
  *out = given;
  return SSD_OK;
}

// The state after a row goes to memory of its own: other blocks still read the
// one before it.
inline ssd_status check_states(const void* initial, const void* final) {
  return final && final == initial ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

constexpr int64_t kMaxSeqStates = 65535;
inline ssd_status check_seq_list(int64_t nseq, const int64_t* last, const void* states) {
  if (nseq < 0) return SSD_ERR_SHAPE;
  if (nseq > kMaxSeqStates) return SSD_ERR_UNSUPPORTED;
  if (nseq > 0 && (!last || !states)) return SSD_ERR_NULL;
  if (nseq > 0 && (!a16(last) || !a16(states))) return SSD_ERR_ALIGN;
  return SSD_OK;
}

}  // namespace api
}  // namespace ssd
