// group_api.cpp -- the C ABI of the group norm and of activations in 8 bits
// declared in include/ssd.h: argument validation on the host before any HIP
// call, then the launch.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include "api_checks.hpp"
#include "group_launch.hpp"

using namespace ssd::api;

namespace {

ssd_status check_group(int64_t rows, int64_t dim, int64_t groups) {
  if (rows <= 0 || dim <= 0 || groups <= 0 || dim % groups != 0) return SSD_ERR_SHAPE;
  if (dim / groups > ssd::kGroupNormMaxSize || dim > int64_t(1) << 24) return SSD_ERR_UNSUPPORTED;
  return product({rows, groups}, k31 - 1);
}

// A gate behind the norm and SiLU of its own output exclude each other.
ssd_status check_group_flags(int flags, const void* z) {
  if (flags & ~(SSD_GROUP_RMS | SSD_GROUP_GATE_FIRST | SSD_GROUP_SILU | SSD_GROUP_SHARED)) return SSD_ERR_UNSUPPORTED;
  if ((flags & SSD_GROUP_GATE_FIRST) && !z) return SSD_ERR_NULL;
  if ((flags & SSD_GROUP_SILU) && z && !(flags & SSD_GROUP_GATE_FIRST)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd::GroupNormArgs group_args(int64_t rows, int64_t dim, int64_t groups, int flags) {
  ssd::GroupNormArgs a = {};
  a.rows = rows;
  a.D = dim;
  a.G = groups;
  a.rms = flags & SSD_GROUP_RMS;
  a.gate_first = flags & SSD_GROUP_GATE_FIRST;
  a.silu = flags & SSD_GROUP_SILU;
  a.shared = flags & SSD_GROUP_SHARED;
  return a;
}

ssd_status check_pack(int64_t rows, int64_t dim, int64_t x_row, int64_t* row) {
  if (rows <= 0 || dim <= 0) return SSD_ERR_SHAPE;
  if (rows >= k31 || dim > int64_t(1) << 24) return SSD_ERR_UNSUPPORTED;
  // 32 blocks of 64 values a launch's block, fewer than 2^32 of those
  SSD_TRY(product({rows, (dim - 1) / ssd::kPackBlock + 1}, (int64_t(1) << 36) - 1));
  return row_stride(x_row, dim, 1, rows, row);
}

}  // namespace

extern "C" {

ssd_status ssd_group_norm(int64_t rows, int64_t dim, int64_t groups, const void* x, ssd_dtype in, const void* z,
                          int64_t z_row, const float* w, const float* bias, float eps, int flags, void* y, float* mean,
                          float* rstd, void* stream) {
  SSD_TRY(check_group(rows, dim, groups));
  SSD_TRY(check_dtype(in));
  SSD_TRY(check_group_flags(flags, z));
  if (!x || !w || !y || !rstd || (!(flags & SSD_GROUP_RMS) && !mean)) return SSD_ERR_NULL;
  ssd::GroupNormArgs a = group_args(rows, dim, groups, flags);
  if (z) SSD_TRY(row_stride(z_row, dim, 1, rows, &a.z_row));
  if (!a16(x) || !aligned(z, elem(in)) || !a16(w) || !a16(bias) || !a16(y) || !a16(mean) || !a16(rstd))
    return SSD_ERR_ALIGN;
  a.eps = eps;
  a.x = x;
  a.z = z;
  a.w = w;
  a.bias = bias;
  a.y = y;
  a.mean = a.rms ? nullptr : mean;
  a.rstd = rstd;
  return from_hip(ssd::launch_group_norm_forward(a, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_group_norm_backward_workspace_bytes(int64_t rows, int64_t dim, int64_t groups) {
  if (check_group(rows, dim, groups) != SSD_OK) return 0;
  return ssd::group_norm_backward_ws_bytes(rows, dim, groups);
}

ssd_status ssd_group_norm_backward(int64_t rows, int64_t dim, int64_t groups, const void* dy, ssd_dtype in,
                                   const void* x, const void* x_scale, const void* z, int64_t z_row,
                                   const void* z_scale, const float* w, const float* bias, const float* mean,
                                   const float* rstd, int flags, void* dx, void* dz, int64_t dz_row, float* dw,
                                   float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  SSD_TRY(check_group(rows, dim, groups));
  SSD_TRY(check_dtype(in));
  SSD_TRY(check_group_flags(flags, z));
  if (!dy || !x || !w || !rstd || (!(flags & SSD_GROUP_RMS) && !mean) || !dx || !dw || (z && !dz)) return SSD_ERR_NULL;
  if (z && (x_scale != nullptr) != (z_scale != nullptr)) return SSD_ERR_NULL;
  ssd::GroupNormArgs a = group_args(rows, dim, groups, flags);
  if (z) {
    if (x_scale && z_row != 0 && z_row != dim) return SSD_ERR_SHAPE;
    SSD_TRY(row_stride(z_row, dim, 1, rows, &a.z_row));
    SSD_TRY(row_stride(dz_row, dim, 1, rows, &a.dz_row));
  }
  if (!workspace || workspace_bytes < ssd_group_norm_backward_workspace_bytes(rows, dim, groups))
    return SSD_ERR_WORKSPACE;
  const uintptr_t e = elem(in);
  if (!a16(dy) || (x_scale ? !aligned(x_scale, 2) || !aligned(z_scale, 2) : !a16(x) || !aligned(z, e)) || !a16(w) ||
      !a16(bias) || !a16(mean) || !a16(rstd) || !a16(dx) || !aligned(dz, e) || !a16(dw) || !a16(dbias) ||
      !a16(workspace))
    return SSD_ERR_ALIGN;
  a.x = x;
  a.z = z;
  a.xs = static_cast<const uint16_t*>(x_scale);
  a.zs = static_cast<const uint16_t*>(z_scale);
  a.w = w;
  a.bias = bias;
  a.mean = a.rms ? nullptr : const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dx = dx;
  a.dz = z ? dz : nullptr;
  a.dw = dw;
  a.db = dbias;
  a.ws = static_cast<float*>(workspace);
  return from_hip(ssd::launch_group_norm_backward(a, in == SSD_BF16, (hipStream_t)stream));
}

ssd_status ssd_pack8(int64_t rows, int64_t dim, const void* x, int64_t x_row, ssd_dtype in, int8_t* q, void* scale,
                     void* stream) {
  int64_t row = 0;
  SSD_TRY(check_pack(rows, dim, x_row, &row));
  SSD_TRY(check_dtype(in));
  if (!x || !q || !scale) return SSD_ERR_NULL;
  if (!aligned(x, elem(in)) || !aligned(scale, 2)) return SSD_ERR_ALIGN;
  return from_hip(ssd::launch_pack8(rows, dim, x, row, in == SSD_BF16, q, static_cast<uint16_t*>(scale),
                                    (hipStream_t)stream));
}

ssd_status ssd_unpack8(int64_t rows, int64_t dim, const int8_t* q, const void* scale, void* x, int64_t x_row,
                       ssd_dtype in, void* stream) {
  int64_t row = 0;
  SSD_TRY(check_pack(rows, dim, x_row, &row));
  SSD_TRY(check_dtype(in));
  if (!x || !q || !scale) return SSD_ERR_NULL;
  if (!aligned(x, elem(in)) || !aligned(scale, 2)) return SSD_ERR_ALIGN;
  return from_hip(ssd::launch_unpack8(rows, dim, q, static_cast<const uint16_t*>(scale), x, row, in == SSD_BF16,
                                      (hipStream_t)stream));
}

}  // extern "C"
