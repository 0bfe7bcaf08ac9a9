// layer_api.cpp -- the C ABI of the layer operators (causal convolution,
// selective scan, layer norm) declared in include/ssd.h: argument validation
// on the host before any HIP call, then the launch.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include "api_checks.hpp"
#include "layer_launch.hpp"

using namespace ssd::api;

namespace {

// ---- convolution ----
ssd_status check_conv(const ssd_conv_shape* s, bool step) {
  if (!s) return SSD_ERR_NULL;
  if (s->batch <= 0 || s->seqlen <= 0 || s->channels <= 0 || s->width <= 0) return SSD_ERR_SHAPE;
  if (step && s->seqlen != 1) return SSD_ERR_SHAPE;
  if (s->width < 2 || s->width > 4) return SSD_ERR_UNSUPPORTED;
  SSD_TRY(product({s->batch, s->seqlen, s->channels}, kMaxElems));
  if (row_too_long(s->seqlen, s->channels)) return SSD_ERR_UNSUPPORTED;
  SSD_TRY(product({s->channels, s->width + 1}, int64_t(1) << 37));  // 512 GiB of partial sums
  // waves (64 channels and at least 8 tokens each) in 31 bits
  return product({s->batch, (s->seqlen - 1) / 8 + 1, (s->channels - 1) / 64 + 1}, k31 - 1);
}

ssd::ConvArgs conv_args(const ssd_conv_shape* s) {
  ssd::ConvArgs a = {};
  a.B = s->batch;
  a.L = s->seqlen;
  a.D = s->channels;
  a.W = (int)s->width;
  return a;
}

// ---- selective scan ----
ssd_status check_scan(const ssd_scan_shape* s, bool step) {
  if (!s) return SSD_ERR_NULL;
  if (s->batch <= 0 || s->seqlen <= 0 || s->channels <= 0 || s->dstate <= 0 || s->ngroups <= 0) return SSD_ERR_SHAPE;
  if (step && s->seqlen != 1) return SSD_ERR_SHAPE;
  if (s->channels % s->ngroups != 0) return SSD_ERR_SHAPE;
  if (!ssd::scan_dstate_supported(s->dstate)) return SSD_ERR_UNSUPPORTED;
  // grid limits: twice the batches and the 16-token chunks in 16-bit dimensions, channel blocks in 31 bits
  if (s->batch > 32767 || (s->seqlen - 1) / 16 + 1 > 65535 || s->channels >= k31) return SSD_ERR_UNSUPPORTED;
  SSD_TRY(product({s->batch, s->seqlen, s->channels}, kMaxElems));
  SSD_TRY(product({s->batch, s->seqlen, s->ngroups, s->dstate}, (int64_t(1) << 36)));
  if (row_too_long(s->seqlen, s->channels) || row_too_long(s->seqlen, s->ngroups * s->dstate)) return SSD_ERR_UNSUPPORTED;
  // blocks of 64 threads, one a group's 64 channels, along one dimension of a launch: below 2^32 threads
  if (s->ngroups * ((s->channels / s->ngroups - 1) / 64 + 1) >= int64_t(1) << 26) return SSD_ERR_UNSUPPORTED;
  // a block a tile of a group in 31 bits, beside the few for A and the starts
  SSD_TRY(product({s->batch, (s->seqlen - 1) / 16 + 1, s->ngroups}, int64_t(1) << 30));
  // 512 GiB of states; (dstate + 2) channels / 64 blocks in 32 bits
  return product({s->batch, s->dstate, s->channels}, (int64_t(1) << 37));
}

ssd_status scan_rows(const ssd_scan_shape* s, const ssd_scan_rows* r, ssd_dtype in, ssd::ScanRows* o) {
  const ssd_scan_rows none = {0, 0, 0, 0, 0};
  if (!r) r = &none;
  const int64_t D = s->channels, gn = s->ngroups * s->dstate;
  SSD_TRY(row_stride(r->u, D, s->batch, s->seqlen, &o->u));
  SSD_TRY(row_stride(r->dt, D, s->batch, s->seqlen, &o->dt));
  SSD_TRY(row_stride(r->Bm, gn, s->batch, s->seqlen, &o->b));
  SSD_TRY(row_stride(r->Cm, gn, s->batch, s->seqlen, &o->c));
  SSD_TRY(row_stride(r->z, D, s->batch, s->seqlen, &o->z));
  // B and C are read in 4-byte units
  if (in == SSD_BF16 && (o->b % 2 != 0 || o->c % 2 != 0)) return SSD_ERR_ALIGN;
  return SSD_OK;
}

ssd_status scan_inputs(const ssd_scan_shape* s, const ssd_scan_rows* rows, const void* u, const void* dt,
                       const float* A, const void* Bm, const void* Cm, const float* Dskip, const void* z,
                       const float* dt_bias, int softplus, ssd_dtype in, ssd::ScanArgs* a) {
  SSD_TRY(check_dtype(in));
  if (!u || !dt || !A || !Bm || !Cm) return SSD_ERR_NULL;
  SSD_TRY(scan_rows(s, rows, in, &a->rows));
  const uintptr_t e = elem(in);
  if (!aligned(u, e) || !aligned(dt, e) || !aligned(z, e) || !aligned(Bm, 4) || !aligned(Cm, 4) || !a16(A) ||
      !a16(Dskip) || !a16(dt_bias))
    return SSD_ERR_ALIGN;
  a->B = s->batch;
  a->L = s->seqlen;
  a->D = s->channels;
  a->N = s->dstate;
  a->G = s->ngroups;
  a->softplus = softplus != 0;
  a->u = u;
  a->dt = dt;
  a->Bm = Bm;
  a->Cm = Cm;
  a->z = z;
  a->A = A;
  a->D_skip = Dskip;
  a->dt_bias = dt_bias;
  return SSD_OK;
}

// ---- norm ----
ssd_status check_norm(int64_t rows, int64_t dim) {
  if (rows <= 0 || dim <= 0) return SSD_ERR_SHAPE;
  if (dim > ssd::kNormMaxDim || rows >= k31) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_causal_conv(const ssd_conv_shape* shape, const void* x, int64_t x_row, const float* w,
                           const float* bias, ssd_dtype in, int silu, const void* initial_state,
                           const int32_t* seq_idx, void* y, void* final_state, int64_t nseq,
                           const int64_t* seq_last, void* seq_states, void* stream) {
  SSD_TRY(check_conv(shape, false));
  SSD_TRY(check_dtype(in));
  if (!x || !w || !y) return SSD_ERR_NULL;
  ssd::ConvArgs a = conv_args(shape);
  SSD_TRY(row_stride(x_row, a.D, a.B, a.L, &a.x_row));
  SSD_TRY(check_seq_list(nseq, seq_last, seq_states));
  if (!aligned(x, elem(in)) || !a16(w) || !a16(bias) || !a16(initial_state) || !a16(seq_idx) || !a16(y) ||
      !a16(final_state))
    return SSD_ERR_ALIGN;
  SSD_TRY(check_states(initial_state, final_state));
  a.silu = silu != 0;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.init = initial_state;
  a.seq_idx = seq_idx;
  a.y = y;
  a.final_state = final_state;
  a.nseq = nseq;
  a.seq_last = seq_last;
  a.seq_states = seq_states;
  return from_hip(ssd::launch_conv_forward(a, in == SSD_BF16, (hipStream_t)stream));
}

ssd_status ssd_causal_conv_step(const ssd_conv_shape* shape, const void* x, int64_t x_row, const void* state,
                                const float* w, const float* bias, ssd_dtype in, int silu, void* state_out, void* y,
                                void* stream) {
  SSD_TRY(check_conv(shape, true));
  SSD_TRY(check_dtype(in));
  if (!x || !state || !w || !state_out || !y) return SSD_ERR_NULL;
  ssd::ConvArgs a = conv_args(shape);
  SSD_TRY(row_stride(x_row, a.D, a.B, 1, &a.x_row));
  if (!aligned(x, elem(in)) || !a16(state) || !a16(w) || !a16(bias) || !a16(state_out) || !a16(y)) return SSD_ERR_ALIGN;
  a.silu = silu != 0;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.y = y;
  return from_hip(ssd::launch_conv_step(a, state, state_out, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_causal_conv_backward_workspace_bytes(const ssd_conv_shape* shape) {
  if (check_conv(shape, false) != SSD_OK) return 0;
  return ssd::conv_backward_ws_bytes(shape->batch, shape->seqlen, shape->channels, (int)shape->width);
}

ssd_status ssd_causal_conv_backward(const ssd_conv_shape* shape, const void* x, int64_t x_row, const float* w,
                                    const float* bias, ssd_dtype in, int silu, const void* initial_state,
                                    const int32_t* seq_idx, const void* dy, const void* dfinal, void* dx,
                                    int64_t dx_row, float* dw, float* dbias, void* dinitial, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  SSD_TRY(check_conv(shape, false));
  SSD_TRY(check_dtype(in));
  if (!x || !w || !dy || !dx || !dw) return SSD_ERR_NULL;
  ssd::ConvArgs a = conv_args(shape);
  SSD_TRY(row_stride(x_row, a.D, a.B, a.L, &a.x_row));
  SSD_TRY(row_stride(dx_row, a.D, a.B, a.L, &a.dx_row));
  if (!workspace || workspace_bytes < ssd_causal_conv_backward_workspace_bytes(shape)) return SSD_ERR_WORKSPACE;
  if (!aligned(x, elem(in)) || !aligned(dx, elem(in)) || !a16(w) || !a16(bias) || !a16(initial_state) ||
      !a16(seq_idx) || !a16(dy) || !a16(dfinal) || !a16(dw) || !a16(dbias) || !a16(dinitial) || !a16(workspace))
    return SSD_ERR_ALIGN;
  a.silu = silu != 0;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.init = initial_state;
  a.seq_idx = seq_idx;
  a.dy = dy;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dinit = dinitial;
  a.ws = static_cast<float*>(workspace);
  return from_hip(ssd::launch_conv_backward(a, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_selective_scan_workspace_bytes(const ssd_scan_shape* s) {
  if (check_scan(s, false) != SSD_OK) return 0;
  return ssd::scan_forward_ws_bytes(s->batch, s->seqlen, s->channels, s->dstate, s->ngroups);
}

ssd_status ssd_selective_scan(const ssd_scan_shape* shape, const ssd_scan_rows* rows, const void* u, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, int softplus, ssd_dtype in, const float* initial_states,
                              const int32_t* seq_idx, void* y, float* final_states, int64_t nseq,
                              const int64_t* seq_last, float* seq_states, void* workspace, size_t workspace_bytes,
                              void* stream) {
  ssd::ScanArgs a = {};
  SSD_TRY(check_scan(shape, false));
  SSD_TRY(scan_inputs(shape, rows, u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, in, &a));
  if (!y) return SSD_ERR_NULL;
  SSD_TRY(check_seq_list(nseq, seq_last, seq_states));
  const size_t need = ssd_selective_scan_workspace_bytes(shape);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  if (!a16(initial_states) || !a16(seq_idx) || !a16(y) || !a16(final_states) || !a16(workspace)) return SSD_ERR_ALIGN;
  SSD_TRY(check_states(initial_states, final_states));
  a.seq_idx = seq_idx;
  a.h0 = initial_states;
  a.y = y;
  a.hfin = final_states;
  a.nseq = nseq;
  a.seq_last = seq_last;
  a.seq_states = seq_states;
  a.ws = workspace;
  return from_hip(ssd::launch_scan_forward(a, in == SSD_BF16, (hipStream_t)stream));
}

ssd_status ssd_selective_step(const ssd_scan_shape* shape, const ssd_scan_rows* rows, const void* u, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, int softplus, ssd_dtype in, const float* state, float* state_out,
                              void* y, void* stream) {
  ssd::ScanArgs a = {};
  SSD_TRY(check_scan(shape, true));
  SSD_TRY(scan_inputs(shape, rows, u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, in, &a));
  if (!state || !state_out || !y) return SSD_ERR_NULL;
  if (!a16(state) || !a16(state_out) || !a16(y)) return SSD_ERR_ALIGN;
  a.y = y;
  return from_hip(ssd::launch_scan_step(a, state, state_out, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_selective_scan_backward_workspace_bytes(const ssd_scan_shape* s) {
  if (check_scan(s, false) != SSD_OK) return 0;
  return ssd::scan_backward_ws_bytes(s->batch, s->seqlen, s->channels, s->dstate, s->ngroups);
}

ssd_status ssd_selective_scan_backward(const ssd_scan_shape* shape, const ssd_scan_rows* rows, const void* u,
                                       const void* dt, const float* A, const void* Bm, const void* Cm,
                                       const float* Dskip, const void* z, const float* dt_bias, int softplus,
                                       ssd_dtype in, const float* initial_states, const int32_t* seq_idx,
                                       const void* dy, const float* dfinal, const ssd_scan_rows* grad_rows, void* du,
                                       void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz, float* ddt_bias,
                                       float* dinitial, void* workspace, size_t workspace_bytes, void* stream) {
  ssd::ScanArgs a = {};
  SSD_TRY(check_scan(shape, false));
  SSD_TRY(scan_inputs(shape, rows, u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, in, &a));
  if (!dy || !du || !ddt || !dA || !dB || !dC || (z && !dz)) return SSD_ERR_NULL;
  SSD_TRY(scan_rows(shape, grad_rows, SSD_F32, &a.grows));  // gradients are written an element at a time
  const size_t need = ssd_selective_scan_backward_workspace_bytes(shape);
  if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
  const uintptr_t e = elem(in);
  if (!aligned(du, e) || !aligned(ddt, e) || !aligned(dB, e) || !aligned(dC, e) || !aligned(dz, e) || !a16(dy) ||
      !a16(initial_states) || !a16(seq_idx) || !a16(dfinal) || !a16(dA) || !a16(dD) || !a16(ddt_bias) ||
      !a16(dinitial) || !a16(workspace))
    return SSD_ERR_ALIGN;
  a.seq_idx = seq_idx;
  a.h0 = initial_states;
  a.dy = dy;
  a.dfinal = dfinal;
  a.du = du;
  a.ddt = ddt;
  a.dB = dB;
  a.dC = dC;
  a.dz = dz;
  a.dA = dA;
  a.dD = dD;
  a.ddt_bias = ddt_bias;
  a.dinit = dinitial;
  a.ws = workspace;
  return from_hip(ssd::launch_scan_backward(a, in == SSD_BF16, (hipStream_t)stream));
}

ssd_status ssd_layer_norm(int64_t rows, int64_t dim, const void* x, ssd_dtype in, const void* residual,
                          ssd_dtype res_dtype, const float* w, const float* bias, float eps, int rms, void* y,
                          void* residual_out, float* mean, float* rstd, void* stream) {
  SSD_TRY(check_norm(rows, dim));
  SSD_TRY(check_dtype(in));
  SSD_TRY(check_dtype(res_dtype));
  if (!x || !w || !y || !rstd || (!rms && !mean) || (residual && !residual_out)) return SSD_ERR_NULL;
  if (!a16(x) || !a16(residual) || !a16(w) || !a16(bias) || !a16(y) || !a16(residual_out) || !a16(mean) || !a16(rstd))
    return SSD_ERR_ALIGN;
  ssd::NormArgs a = {};
  a.rows = rows;
  a.D = dim;
  a.eps = eps;
  a.rms = rms != 0;
  a.x = x;
  a.res_bf16 = res_dtype == SSD_BF16;
  a.residual = residual;
  a.residual_out = residual ? residual_out : nullptr;
  a.w = w;
  a.bias = bias;
  a.y = y;
  a.mean = rms ? nullptr : mean;
  a.rstd = rstd;
  return from_hip(ssd::launch_norm_forward(a, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_layer_norm_backward_workspace_bytes(int64_t rows, int64_t dim) {
  if (check_norm(rows, dim) != SSD_OK) return 0;
  return ssd::norm_backward_ws_bytes(rows, dim);
}

ssd_status ssd_layer_norm_backward(int64_t rows, int64_t dim, const void* dy, ssd_dtype in, const void* x,
                                   ssd_dtype x_dtype, const float* w, const float* mean, const float* rstd, int rms,
                                   const void* dresidual, void* dx, void* residual_grad, float* dw, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  SSD_TRY(check_norm(rows, dim));
  SSD_TRY(check_dtype(in));
  SSD_TRY(check_dtype(x_dtype));
  if (!dy || !x || !w || !rstd || (!rms && !mean) || !dx || !dw) return SSD_ERR_NULL;
  if (!workspace || workspace_bytes < ssd_layer_norm_backward_workspace_bytes(rows, dim)) return SSD_ERR_WORKSPACE;
  if (!a16(dy) || !a16(x) || !a16(w) || !a16(mean) || !a16(rstd) || !a16(dresidual) || !a16(dx) ||
      !a16(residual_grad) || !a16(dw) || !a16(dbias) || !a16(workspace))
    return SSD_ERR_ALIGN;
  ssd::NormArgs a = {};
  a.rows = rows;
  a.D = dim;
  a.rms = rms != 0;
  a.dy = dy;
  a.x = x;
  a.res_bf16 = x_dtype == SSD_BF16;
  a.w = w;
  a.mean = rms ? nullptr : const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dres = dresidual;
  a.dx = dx;
  a.dres_out = residual_grad;
  a.dw = dw;
  a.db = dbias;
  a.ws = static_cast<float*>(workspace);
  return from_hip(ssd::launch_norm_backward(a, in == SSD_BF16, (hipStream_t)stream));
}

}  // extern "C"
