// C-ABI entry points of linear attention and rotary positions: argument
// validation, workspace sizing and dispatch.  Host code; no HIP call is made
// before every argument has been checked.
#include <cmath>

#include "gdn_linear.h"
#include "gdn_seq_check.h"

namespace {

using namespace gdn;

gdn_status check_linear(const gdn_linear_problem* pr, bool packed, bool slots, LinearProblem* out) {
  if (!pr) return fail(GDN_ERR_INVALID_ARGUMENT, "problem is NULL");
  for (int i = 0; i < (int)(sizeof pr->reserved / sizeof pr->reserved[0]); ++i)
    if (pr->reserved[i] != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "reserved[%d] is not zero", i);
  if (pr->gate_per_head != 0 && pr->gate_per_head != 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gate_per_head must be 0 or 1 (got %d)", pr->gate_per_head);
  if (!std::isfinite(pr->scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "scale must be finite");
  const gdn_seq_problem s = {pr->abi_version, pr->heads_k, pr->heads_v, pr->d_k, pr->d_v, pr->qkv_dtype, pr->out_dtype,
                             pr->state_rows, pr->tokens, pr->q_stride, pr->k_stride, pr->v_stride, pr->sequences, {}};
  const gdn_status status = packed ? check_packed(&s, slots, out) : check_seq(&s, slots, out);
  if (status != GDN_OK) return status;
  out->scale = pr->scale;
  out->fixed = pr->gate_per_head == 1;
  return GDN_OK;
}

gdn_status check_rotary(const gdn_rotary_problem* pr, RotaryProblem* out) {
  if (!pr) return fail(GDN_ERR_INVALID_ARGUMENT, "problem is NULL");
  if (pr->abi_version != GDN_ABI_VERSION)
    return fail(GDN_ERR_INVALID_ARGUMENT, "abi_version %d != %d", pr->abi_version, GDN_ABI_VERSION);
  for (int i = 0; i < (int)(sizeof pr->reserved / sizeof pr->reserved[0]); ++i)
    if (pr->reserved[i] != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "reserved[%d] is not zero", i);
  if (pr->dtype != GDN_F32 && pr->dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "dtype must be GDN_F32 or GDN_BF16");
  if (pr->tokens < 0 || pr->tokens > (1LL << 31) - 256)
    return fail(GDN_ERR_INVALID_ARGUMENT, "tokens must be in [0, 2^31 - 256] (got %lld)", (long long)pr->tokens);
  if (pr->heads_q < 1 || pr->heads_q > 65535 || pr->heads_k < 0 || pr->heads_k > 65535)
    return fail(GDN_ERR_INVALID_ARGUMENT, "heads_q must be in [1, 65535] and heads_k in [0, 65535] (got %d, %d)",
                pr->heads_q, pr->heads_k);
  if (pr->width < 8 || pr->width > 1024 || pr->width % 8)
    return fail(GDN_ERR_INVALID_ARGUMENT, "width must be a multiple of 8 in [8, 1024] (got %d)", pr->width);
  if (pr->pairs < 1 || pr->pairs > pr->width / 2)
    return fail(GDN_ERR_INVALID_ARGUMENT, "pairs must be in [1, width / 2] (got %d of %d)", pr->pairs, pr->width);
  if (pr->layout != GDN_ROTARY_HALF && pr->layout != GDN_ROTARY_INTERLEAVED)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown layout %d", pr->layout);
  if (pr->inverse != 0 && pr->inverse != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "inverse must be 0 or 1 (got %d)", pr->inverse);
  if (pr->axes < 1 || pr->axes > 4) return fail(GDN_ERR_INVALID_ARGUMENT, "axes must be in [1, 4] (got %d)", pr->axes);
  int end = 0;
  for (int a = 0; a < 4; ++a) {
    if (pr->sections[a] < 0 || pr->sections[a] > pr->pairs - end || (a >= pr->axes && pr->sections[a] != 0))
      return fail(GDN_ERR_INVALID_ARGUMENT, "sections must be >= 0, %d in all and 0 behind the last axis", pr->pairs);
    end += pr->sections[a];
    out->ends[a] = end;
  }
  if (end != pr->pairs) return fail(GDN_ERR_INVALID_ARGUMENT, "sections must be %d in all (got %d)", pr->pairs, end);
  if (!std::isfinite(pr->magnitude)) return fail(GDN_ERR_INVALID_ARGUMENT, "magnitude must be finite");
  const long long unit = pr->dtype == GDN_BF16 ? 8 : 4;   // elements in 16 bytes
  const long long wq = (long long)pr->heads_q * pr->width, wk = (long long)pr->heads_k * pr->width;
  struct { const char* name; long long given, width; } st[] = {{"q_stride", pr->q_stride, wq}, {"k_stride", pr->k_stride, wk},
      {"q_out_stride", pr->q_out_stride, wq}, {"k_out_stride", pr->k_out_stride, wk}};
  for (const auto& s : st)
    if (s.given != 0 && (s.given < s.width || s.given % unit || s.given > (1LL << 23)))
      return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be 0 or a multiple of 16 bytes in [%lld, 2^23] elements (got %lld)",
                  s.name, s.width, s.given);
  out->bf16 = pr->dtype == GDN_BF16;
  out->tokens = pr->tokens;
  out->hq = pr->heads_q;
  out->hk = pr->heads_k;
  out->width = pr->width;
  out->pairs = pr->pairs;
  out->interleaved = pr->layout == GDN_ROTARY_INTERLEAVED;
  out->axes = pr->axes;
  out->cos_factor = pr->magnitude;
  out->sin_factor = pr->inverse ? -pr->magnitude : pr->magnitude;
  out->qs = pr->q_stride ? pr->q_stride : wq;
  out->ks = pr->k_stride ? pr->k_stride : wk;
  out->qos = pr->q_out_stride ? pr->q_out_stride : wq;
  out->kos = pr->k_out_stride ? pr->k_out_stride : wk;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_linear_decode(const gdn_linear_problem* pr, const void* q, const void* k, const void* v,
                             const float* log_gate, float* state, const int32_t* slots, void* out, void* stream) {
  try {
    LinearProblem p;
    gdn_status s = check_linear(pr, false, slots != nullptr, &p);
    if (s != GDN_OK) return s;
    if (p.tokens == 0 || (slots && p.state_rows == 0)) return finish(hipSuccess);
    s = check_needed({q, k, v, log_gate, state, out}, "q, k, v, log_gate, state and out");
    if (s == GDN_OK) s = check_aligned({q, k, v, state, out}, {log_gate, slots});
    if (s != GDN_OK) return s;
    return finish(linear_decode_launch(p, q, k, v, log_gate, state, slots, out, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_linear_workspace_size(const gdn_linear_problem* pr, int32_t gradient, size_t* bytes_out) {
  try {
    if (!bytes_out) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
    LinearProblem p;
    const gdn_status s = check_linear(pr, true, false, &p);
    if (s != GDN_OK) return s;
    *bytes_out = linear_space(p, gradient != 0, nullptr, nullptr);
    return finish(hipSuccess);
  } catch (...) {
    return fail(GDN_ERR_INVALID_ARGUMENT, "internal error while sizing the workspace");
  }
}

gdn_status gdn_linear_forward(const gdn_linear_problem* pr, const void* q, const void* k, const void* v,
                              const float* log_gate, const int32_t* cu_seqlens, const int32_t* slots,
                              const float* initial_state, void* out, float* final_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
  try {
    LinearProblem p;
    gdn_status s = check_linear(pr, true, slots != nullptr, &p);
    if (s != GDN_OK) return s;
    if (p.sequences == 0) return finish(hipSuccess);
    s = check_needed({cu_seqlens}, "cu_seqlens");
    if (s == GDN_OK && p.tokens > 0) s = check_needed({q, k, v, log_gate, out}, "q, k, v, log_gate and out");
    if (s == GDN_OK)
      s = check_aligned({q, k, v, initial_state, out, final_state, workspace}, {log_gate, cu_seqlens, slots});
    if (s == GDN_OK) s = check_workspace(linear_space(p, false, nullptr, nullptr), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    LinearTensors t = {};
    t.q = q;
    t.k = k;
    t.v = v;
    t.g = log_gate;
    t.cu = cu_seqlens;
    t.slots = slots;
    t.h0 = initial_state;
    t.out = out;
    t.hT = final_state;
    LinearSpace ws;
    linear_space(p, false, workspace, &ws);
    return finish(linear_forward_launch(p, t, ws, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_linear_backward(const gdn_linear_problem* pr, const void* q, const void* k, const void* v,
                               const float* log_gate, const int32_t* cu_seqlens, const float* initial_state,
                               const void* dout, const float* dfinal_state, void* dq, void* dk, void* dv,
                               float* dlog_gate, float* dinitial_state, void* workspace, size_t workspace_bytes,
                               void* stream) {
  try {
    LinearProblem p;
    gdn_status s = check_linear(pr, true, false, &p);
    if (s != GDN_OK) return s;
    if (p.sequences == 0 && !p.fixed) return finish(hipSuccess);
    if (p.sequences > 0) s = check_needed({cu_seqlens}, "cu_seqlens");
    if (s == GDN_OK && p.fixed) s = check_needed({log_gate, dlog_gate}, "log_gate and dlog_gate");
    if (s == GDN_OK && p.sequences > 0 && p.tokens > 0)
      s = check_needed({q, k, v, log_gate, dout, dq, dk, dv, dlog_gate}, "q, k, v, log_gate, dout, dq, dk, dv and dlog_gate");
    if (s == GDN_OK)
      s = check_aligned({q, k, v, initial_state, dout, dfinal_state, dq, dk, dv, dinitial_state, workspace},
                        {log_gate, cu_seqlens, dlog_gate});
    if (s == GDN_OK) s = check_workspace(linear_space(p, true, nullptr, nullptr), workspace, workspace_bytes);
    if (s != GDN_OK) return s;
    const LinearTensors t = {q, k, v, log_gate, cu_seqlens, nullptr, initial_state, nullptr, nullptr,
                             dout, dfinal_state, dq, dk, dv, dlog_gate, dinitial_state};
    LinearSpace ws;
    linear_space(p, true, workspace, &ws);
    return finish(linear_backward_launch(p, t, ws, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

gdn_status gdn_rotary(const gdn_rotary_problem* pr, const void* q, const void* k, const int32_t* positions,
                      const double* frequencies, void* q_out, void* k_out, void* stream) {
  try {
    RotaryProblem p;
    gdn_status s = check_rotary(pr, &p);
    if (s != GDN_OK) return s;
    if (p.tokens == 0) return finish(hipSuccess);
    if (p.hk == 0) k = k_out = nullptr;
    s = check_needed({q, positions, frequencies, q_out}, "q, positions, frequencies and q_out");
    if (s == GDN_OK && p.hk > 0) s = check_needed({k, k_out}, "k and k_out");
    if (s != GDN_OK) return s;
    for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
      if (!aligned16(x)) return fail(GDN_ERR_INVALID_ARGUMENT, "pointers of q, k and their outputs must be 16-byte aligned");
    if (!aligned4(positions) || (reinterpret_cast<uintptr_t>(frequencies) & 7u))
      return fail(GDN_ERR_INVALID_ARGUMENT, "positions must be 4-byte aligned and frequencies 8-byte aligned");
    if ((q == q_out && p.qs != p.qos) || (k && k == k_out && p.ks != p.kos))
      return fail(GDN_ERR_INVALID_ARGUMENT, "a call in place needs the same strides of q and q_out, k and k_out");
    return finish(rotary_launch(p, q, k, positions, frequencies, q_out, k_out, reinterpret_cast<hipStream_t>(stream)));
  } catch (...) {
    return fail(GDN_ERR_HIP, "internal error while enqueueing");
  }
}

}  // extern "C"
