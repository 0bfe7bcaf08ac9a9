// delta_api.cpp -- the C ABI of the gated delta rule declared in include/ssd.h:
// argument validation on the host before any HIP call, then the launch.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include "api_checks.hpp"
#include "delta_launch.hpp"

using namespace ssd::api;

namespace {

// 64 rows of up to 4 bytes an element are addressed by 32-bit byte offsets
constexpr int64_t kMaxRow = int64_t(1) << 23;

ssd_status check_delta(const ssd_delta_shape* s, bool step) {
  if (!s) return SSD_ERR_NULL;
  if (s->batch <= 0 || s->seqlen <= 0 || s->nheads <= 0 || s->headdim <= 0 || s->dstate <= 0 || s->ngroups <= 0)
    return SSD_ERR_SHAPE;
  if (step && s->seqlen != 1) return SSD_ERR_SHAPE;
  if (s->nheads % s->ngroups != 0) return SSD_ERR_SHAPE;
  if (s->dstate % 16 != 0 || s->headdim % 16 != 0 || s->dstate > ssd::kDeltaMaxDim || s->headdim > ssd::kDeltaMaxDim)
    return SSD_ERR_UNSUPPORTED;
  // a launch holds fewer than 2^32 threads in a dimension (one that asks for more runs the rest and reports
  // success): up to 512 a (row, window, head), 64 a (row, head, 16 columns), 512 a (row, head, 32 columns)
  SSD_TRY(product({s->batch, s->nheads, (s->seqlen - 1) / ssd::kDeltaC + 1}, (int64_t(1) << 23) - 1));
  SSD_TRY(product({s->batch, s->nheads}, (int64_t(1) << 22) - 1));
  SSD_TRY(product({s->batch, s->nheads, s->headdim}, (int64_t(1) << 28) - 1));
  // dense rows, of v (those of dt and beta are shorter) and of q and k
  SSD_TRY(product({s->nheads, s->headdim}, kMaxRow - 1));
  SSD_TRY(product({s->ngroups, s->dstate}, kMaxRow - 1));
  return product({s->batch, s->seqlen, s->nheads, s->headdim}, kMaxElems);
}

ssd_status delta_rows(const ssd_delta_shape* s, const ssd_delta_rows* r, ssd::DeltaRows* o) {
  const ssd_delta_rows none = {0, 0, 0, 0, 0};
  if (!r) r = &none;
  const int64_t qk = s->ngroups * s->dstate;
  for (int64_t given : {r->q, r->k, r->v, r->dt, r->beta})
    if (given >= kMaxRow) return SSD_ERR_UNSUPPORTED;
  SSD_TRY(row_stride(r->q, qk, s->batch, s->seqlen, &o->q));
  SSD_TRY(row_stride(r->k, qk, s->batch, s->seqlen, &o->k));
  SSD_TRY(row_stride(r->v, s->nheads * s->headdim, s->batch, s->seqlen, &o->v));
  SSD_TRY(row_stride(r->dt, s->nheads, s->batch, s->seqlen, &o->dt));
  return row_stride(r->beta, s->nheads, s->batch, s->seqlen, &o->beta);
}

ssd_status delta_inputs(const ssd_delta_shape* s, const ssd_delta_rows* rows, const void* q, const void* k,
                        const void* v, const void* dt, const void* beta, const float* A, const float* dt_bias,
                        int flags, float scale, ssd_dtype in, bool step, ssd::DeltaArgs* a) {
  SSD_TRY(check_dtype(in));
  if (flags & ~(SSD_DELTA_SOFTPLUS | SSD_DELTA_SIGMOID | SSD_DELTA_QK_NORM | SSD_DELTA_MMA_F32)) return SSD_ERR_UNSUPPORTED;
  if (!q || !k || !v || !dt || !beta || !A) return SSD_ERR_NULL;
  SSD_TRY(delta_rows(s, rows, &a->rows));
  const uintptr_t e = elem(in);
  // prompts read q and k 16 bytes at a time
  const uintptr_t qk = step ? e : 16;
  if (!aligned(q, qk) || !aligned(k, qk) || !aligned(v, e) || !aligned(dt, e) || !aligned(beta, e) || !a16(A) ||
      !a16(dt_bias))
    return SSD_ERR_ALIGN;
  if (!step && (a->rows.q * e % 16 != 0 || a->rows.k * e % 16 != 0)) return SSD_ERR_ALIGN;
  a->B = s->batch;
  a->L = s->seqlen;
  a->H = s->nheads;
  a->G = s->ngroups;
  a->N = s->dstate;
  a->P = s->headdim;
  a->softplus = flags & SSD_DELTA_SOFTPLUS;
  a->sigmoid = flags & SSD_DELTA_SIGMOID;
  a->qk_norm = flags & SSD_DELTA_QK_NORM;
  a->f32_products = flags & SSD_DELTA_MMA_F32;
  a->scale = scale;
  a->q = q;
  a->k = k;
  a->v = v;
  a->dt = dt;
  a->beta = beta;
  a->A = A;
  a->dt_bias = dt_bias;
  return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_delta_rule_workspace_bytes(const ssd_delta_shape* s) {
  if (check_delta(s, false) != SSD_OK) return 0;
  return ssd::delta_forward_ws_bytes(s->batch, s->seqlen, s->nheads, s->ngroups, s->dstate, s->headdim);
}

ssd_status ssd_delta_rule(const ssd_delta_shape* shape, const ssd_delta_rows* rows, const void* q, const void* k,
                          const void* v, const void* dt, const void* beta, const float* A, const float* dt_bias,
                          int flags, float scale, ssd_dtype in, const float* initial_states, const int32_t* seq_idx,
                          void* y, float* final_states, int64_t nseq, const int64_t* seq_last, float* seq_states,
                          void* workspace, size_t workspace_bytes, void* stream) {
  ssd::DeltaArgs a = {};
  SSD_TRY(check_delta(shape, false));
  SSD_TRY(delta_inputs(shape, rows, q, k, v, dt, beta, A, dt_bias, flags, scale, in, false, &a));
  if (!y) return SSD_ERR_NULL;
  SSD_TRY(check_seq_list(nseq, seq_last, seq_states));
  static_assert(ssd::kDeltaMaxStates >= kMaxSeqStates, "the workspace holds a link for every state");
  if (!workspace || workspace_bytes < ssd_delta_rule_workspace_bytes(shape)) return SSD_ERR_WORKSPACE;
  if (!a16(initial_states) || !a16(seq_idx) || !a16(y) || !a16(final_states) || !a16(workspace)) return SSD_ERR_ALIGN;
  a.h0 = initial_states;
  a.seq_idx = seq_idx;
  a.y = y;
  a.hfin = final_states;
  a.nseq = nseq;
  a.seq_last = seq_last;
  a.seq_states = seq_states;
  a.ws = static_cast<char*>(workspace);
  return from_hip(ssd::launch_delta_forward(a, in == SSD_BF16, (hipStream_t)stream));
}

ssd_status ssd_delta_step(const ssd_delta_shape* shape, const ssd_delta_rows* rows, const void* q, const void* k,
                          const void* v, const void* dt, const void* beta, const float* A, const float* dt_bias,
                          int flags, float scale, ssd_dtype in, const float* state, float* state_out, void* y,
                          void* stream) {
  ssd::DeltaArgs a = {};
  SSD_TRY(check_delta(shape, true));
  SSD_TRY(delta_inputs(shape, rows, q, k, v, dt, beta, A, dt_bias, flags, scale, in, true, &a));
  if (!state || !state_out || !y) return SSD_ERR_NULL;
  if (!a16(state) || !a16(state_out) || !a16(y)) return SSD_ERR_ALIGN;
  a.y = y;
  return from_hip(ssd::launch_delta_step(a, state, state_out, in == SSD_BF16, (hipStream_t)stream));
}

size_t ssd_delta_rule_backward_workspace_bytes(const ssd_delta_shape* s) {
  if (check_delta(s, false) != SSD_OK) return 0;
  return ssd::delta_backward_ws_bytes(s->batch, s->seqlen, s->nheads, s->ngroups, s->dstate, s->headdim);
}

ssd_status ssd_delta_rule_backward(const ssd_delta_shape* shape, const ssd_delta_rows* rows, const void* q,
                                   const void* k, const void* v, const void* dt, const void* beta, const float* A,
                                   const float* dt_bias, int flags, float scale, ssd_dtype in,
                                   const float* initial_states, const int32_t* seq_idx, const void* dy,
                                   const float* dfinal, const ssd_delta_rows* grad_rows, void* dq, void* dk, void* dv,
                                   void* ddt, void* dbeta, float* dA, float* ddt_bias, float* dinitial,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  ssd::DeltaArgs a = {};
  SSD_TRY(check_delta(shape, false));
  SSD_TRY(delta_inputs(shape, rows, q, k, v, dt, beta, A, dt_bias, flags, scale, in, false, &a));
  if (!dy || !dq || !dk || !dv || !ddt || !dbeta || !dA) return SSD_ERR_NULL;
  SSD_TRY(delta_rows(shape, grad_rows, &a.grows));
  // blocks of four waves, one a (token, key group)
  SSD_TRY(product({shape->batch, shape->seqlen, shape->ngroups}, (int64_t(1) << 25)));
  if (!workspace || workspace_bytes < ssd_delta_rule_backward_workspace_bytes(shape)) return SSD_ERR_WORKSPACE;
  const uintptr_t e = elem(in);
  if (!aligned(dq, e) || !aligned(dk, e) || !aligned(dv, e) || !aligned(ddt, e) || !aligned(dbeta, e) || !a16(dy) ||
      !a16(initial_states) || !a16(seq_idx) || !a16(dfinal) || !a16(dA) || !a16(ddt_bias) || !a16(dinitial) ||
      !a16(workspace))
    return SSD_ERR_ALIGN;
  a.h0 = initial_states;
  a.seq_idx = seq_idx;
  a.dy = dy;
  a.dfinal = dfinal;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.ddt = ddt;
  a.dbeta = dbeta;
  a.dA = dA;
  a.ddt_bias = ddt_bias;
  a.dinit = dinitial;
  a.ws = static_cast<char*>(workspace);
  return from_hip(ssd::launch_delta_backward(a, in == SSD_BF16, (hipStream_t)stream));
}

}  // extern "C"
