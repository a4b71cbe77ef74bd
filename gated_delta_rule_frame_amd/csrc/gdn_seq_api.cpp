// C-ABI entry points of the sequence operators: argument validation,
// workspace sizing and dispatch.  Host code; no HIP call is made before every
// argument has been checked.
#include <cmath>

#include "gdn_norm.h"
#include "gdn_seq_check.h"

namespace {

using namespace gdn;

gdn_status check_norm(const gdn_norm_problem* pr, gdn::NormProblem* out) {
  if (!pr) return fail(GDN_ERR_INVALID_ARGUMENT, "problem is NULL");
  if (pr->abi_version != GDN_ABI_VERSION)
    return fail(GDN_ERR_INVALID_ARGUMENT, "abi_version %d != %d", pr->abi_version, GDN_ABI_VERSION);
  for (int i = 0; i < (int)(sizeof pr->reserved / sizeof pr->reserved[0]); ++i)
    if (pr->reserved[i] != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "reserved[%d] is not zero", i);
  if (pr->dtype != GDN_F32 && pr->dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "dtype must be GDN_F32 or GDN_BF16");
  if (pr->batch < 0 || pr->spatial < 1 || pr->spatial > (1 << 30) || pr->channels < 1 || pr->channels > (1 << 24))
    return fail(GDN_ERR_INVALID_ARGUMENT, "batch must be >= 0, spatial in [1, 2^30], channels in [1, 2^24] (got %lld, %d, %d)",
                (long long)pr->batch, pr->spatial, pr->channels);
  if (pr->groups < 1 || pr->channels % pr->groups)
    return fail(GDN_ERR_INVALID_ARGUMENT, "channels (%d) must be a multiple of groups (%d)", pr->channels, pr->groups);
  if (pr->batch > (1LL << 40) / ((long long)pr->spatial * pr->channels) + 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "tensor too large (batch %lld)", (long long)pr->batch);
  if (pr->activation < GDN_ACT_NONE || pr->activation > GDN_ACT_RELU)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown activation %d", pr->activation);
  if (pr->center != 0 && pr->center != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "center must be 0 or 1 (got %d)", pr->center);
  if (!std::isfinite(pr->eps) || pr->eps < 0.f) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  out->N = pr->batch;
  out->S = pr->spatial;
  out->C = pr->channels;
  out->G = pr->groups;
  out->cg = pr->channels / pr->groups;
  out->act = pr->activation;
  out->bf16 = pr->dtype == GDN_BF16;
  out->center = pr->center != 0;
  out->eps = pr->eps;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_decode(const gdn_seq_problem* pr, const void* q, const void* k, const void* v, const float* log_gate,
                      const float* beta, float* state, const int32_t* slots, void* out, void* stream) {
  try {
    gdn::SeqProblem p;
    gdn_status s = check_seq(pr, slots != nullptr, &p);
    if (s != GDN_OK) return s;
    if (p.tokens == 0 || (slots && p.state_rows == 0)) return finish(hipSuccess);
    s = check_needed({q, k, v, log_gate, beta, state, out}, "q, k, v, log_gate, beta, state and out");
    if (s == GDN_OK) s = check_aligned({q, k, v, state, out}, {log_gate, beta, slots});
    if (s != GDN_OK) return s;
    return finish(gdn::decode_launch(p, q, k, v, log_gate, beta, state, slots, out, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_packed_workspace_size(const gdn_seq_problem* pr, int32_t gradient, size_t* bytes_out) {
  try {
    if (!bytes_out) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
    gdn::SeqProblem p;
    const gdn_status s = check_packed(pr, false, &p);
    if (s != GDN_OK) return s;
    *bytes_out = gdn::packed_space(p, gradient != 0, nullptr, nullptr);
    return finish(hipSuccess);
  } catch (...) {
    return fail(GDN_ERR_INVALID_ARGUMENT, "internal error while sizing the workspace");
  }
}

gdn_status gdn_packed_forward(const gdn_seq_problem* pr, const void* q, const void* k, const void* v, const float* log_gate,
                              const float* beta, const int32_t* cu_seqlens, const int32_t* slots, const float* initial_state,
                              void* out, float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    gdn::SeqProblem p;
    gdn_status s = check_packed(pr, slots != nullptr, &p);
    if (s != GDN_OK) return s;
    if (p.sequences == 0) return finish(hipSuccess);
    s = check_needed({cu_seqlens}, "cu_seqlens");
    if (s == GDN_OK && p.tokens > 0) s = check_needed({q, k, v, log_gate, beta, out}, "q, k, v, log_gate, beta and out");
    if (s == GDN_OK)
      s = check_aligned({q, k, v, initial_state, out, final_state, workspace}, {log_gate, beta, cu_seqlens, slots});
    if (s != GDN_OK) return s;
    s = check_workspace(gdn::packed_space(p, false, nullptr, nullptr), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    gdn::PackedTensors t = {};
    t.q = q;
    t.k = k;
    t.v = v;
    t.g = log_gate;
    t.beta = beta;
    t.cu = cu_seqlens;
    t.slots = slots;
    t.h0 = initial_state;
    t.out = out;
    t.hT = final_state;
    gdn::PackedSpace ws;
    gdn::packed_space(p, false, workspace, &ws);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = gdn::packed_prep(p, t, ws, false, st);
    if (e == hipSuccess) e = gdn::packed_scan(p, t, ws, false, st);
    return finish(e);
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_packed_backward(const gdn_seq_problem* pr, const void* q, const void* k, const void* v, const float* log_gate,
                               const float* beta, const int32_t* cu_seqlens, const float* initial_state, const void* dout,
                               const float* dfinal_state, void* dq, void* dk, void* dv, float* dlog_gate, float* dbeta,
                               float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    gdn::SeqProblem p;
    gdn_status s = check_packed(pr, false, &p);
    if (s != GDN_OK) return s;
    if (p.sequences == 0) return finish(hipSuccess);
    s = check_needed({cu_seqlens}, "cu_seqlens");
    if (s == GDN_OK && p.tokens > 0)
      s = check_needed({q, k, v, log_gate, beta, dout, dq, dk, dv, dlog_gate, dbeta},
                       "q, k, v, log_gate, beta, dout, dq, dk, dv, dlog_gate and dbeta");
    if (s == GDN_OK)
      s = check_aligned({q, k, v, initial_state, dout, dfinal_state, dq, dk, dv, dinitial_state, workspace},
                        {log_gate, beta, cu_seqlens, dlog_gate, dbeta});
    if (s == GDN_OK) s = check_workspace(gdn::packed_space(p, true, nullptr, nullptr), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    const gdn::PackedTensors t = {q, k, v, log_gate, beta, cu_seqlens, nullptr, initial_state, nullptr, nullptr,
                                  dout, dfinal_state, dq, dk, dv, dlog_gate, dbeta, dinitial_state};
    gdn::PackedSpace ws;
    gdn::packed_space(p, true, workspace, &ws);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = gdn::packed_prep(p, t, ws, true, st);
    if (e == hipSuccess) e = gdn::packed_scan(p, t, ws, true, st);
    if (e == hipSuccess) e = gdn::packed_scan_grad(p, t, ws, st);
    if (e == hipSuccess) e = gdn::packed_grads(p, t, ws, st);
    return finish(e);
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_group_norm_workspace_size(const gdn_norm_problem* pr, int32_t gradient, size_t* bytes_out) {
  try {
    if (!bytes_out) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
    gdn::NormProblem p;
    const gdn_status s = check_norm(pr, &p);
    if (s != GDN_OK) return s;
    *bytes_out = gdn::norm_workspace(p, gradient != 0);
    return finish(hipSuccess);
  } catch (...) {
    return fail(GDN_ERR_INVALID_ARGUMENT, "internal error while sizing the workspace");
  }
}

gdn_status gdn_group_norm(const gdn_norm_problem* pr, const void* x, const float* weight, const float* bias, const void* gate,
                          void* out, float* mean, float* rstd, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    gdn::NormProblem p;
    gdn_status s = check_norm(pr, &p);
    if (s != GDN_OK) return s;
    if (p.N == 0) return finish(hipSuccess);
    s = check_needed({x, out, rstd}, "x, out and rstd");
    if (s == GDN_OK) s = check_aligned({x, out, rstd, weight, bias, gate, mean, workspace}, {});
    if (s != GDN_OK) return s;
    if (p.center && !mean) return fail(GDN_ERR_INVALID_ARGUMENT, "mean must be non-NULL with center = 1");
    s = check_workspace(gdn::norm_workspace(p, false), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    return finish(gdn::norm_launch(p, x, weight, bias, gate, out, mean, rstd, workspace, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_group_norm_backward(const gdn_norm_problem* pr, const void* dout, const void* x, const float* weight,
                                   const float* bias, const void* gate, const float* mean, const float* rstd, void* dx,
                                   float* dweight, float* dbias, void* dgate, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  try {
    gdn::NormProblem p;
    gdn_status s = check_norm(pr, &p);
    if (s != GDN_OK) return s;
    if (p.N > 0) {
      s = check_needed({dout, x, rstd, dx}, "dout, x, rstd and dx");
      if (s == GDN_OK)
        s = check_aligned({dout, x, rstd, dx, weight, bias, gate, mean, dweight, dbias, dgate, workspace}, {});
      if (s != GDN_OK) return s;
      if (p.center && !mean) return fail(GDN_ERR_INVALID_ARGUMENT, "mean must be non-NULL with center = 1");
      if (!gate != !dgate) return fail(GDN_ERR_INVALID_ARGUMENT, "gate and dgate must be given together");
    } else {
      s = check_aligned({dweight, dbias}, {});
      if (s != GDN_OK) return s;
      if (!dweight && !dbias) return finish(hipSuccess);
    }
    s = check_workspace(gdn::norm_workspace(p, true), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    const gdn::NormGrad t{dout, x, weight, bias, gate, mean, rstd, dx, dgate, dweight, dbias};
    return finish(gdn::norm_grad_launch(p, t, workspace, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

}  // extern "C"
