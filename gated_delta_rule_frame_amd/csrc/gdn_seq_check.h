// Argument checks that the C-ABI layers of the sequence operators share.  Host code.
#pragma once

#include <initializer_list>

#include "gdn_seq.h"

namespace gdn {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline gdn_status check_seq(const gdn_seq_problem* pr, bool slots, SeqProblem* out) {
  if (!pr) return fail(GDN_ERR_INVALID_ARGUMENT, "problem is NULL");
  if (pr->abi_version != GDN_ABI_VERSION)
    return fail(GDN_ERR_INVALID_ARGUMENT, "abi_version %d != %d", pr->abi_version, GDN_ABI_VERSION);
  for (int i = 0; i < (int)(sizeof pr->reserved / sizeof pr->reserved[0]); ++i)
    if (pr->reserved[i] != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "reserved[%d] is not zero", i);
  if (pr->heads_k < 1 || pr->heads_v < 1 || pr->heads_v % pr->heads_k || pr->heads_v > 65535)
    return fail(GDN_ERR_INVALID_ARGUMENT, "heads_v must be a multiple of heads_k, both in [1, 65535] (got %d, %d)",
                pr->heads_v, pr->heads_k);
  if (pr->d_k < 16 || pr->d_k > 128 || pr->d_k % 16 || pr->d_v < 16 || pr->d_v > 128 || pr->d_v % 16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "d_k and d_v must be multiples of 16 in [16, 128] (got %d, %d)", pr->d_k, pr->d_v);
  if ((pr->qkv_dtype != GDN_F32 && pr->qkv_dtype != GDN_BF16) || (pr->out_dtype != GDN_F32 && pr->out_dtype != GDN_BF16))
    return fail(GDN_ERR_INVALID_ARGUMENT, "qkv_dtype/out_dtype must be GDN_F32 or GDN_BF16");
  if (pr->tokens < 0 || pr->tokens > (1LL << 31) - 256)
    return fail(GDN_ERR_INVALID_ARGUMENT, "tokens must be in [0, 2^31 - 256] (got %lld)", (long long)pr->tokens);
  if (slots && pr->state_rows < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "state_rows must be >= 0 (got %d)", pr->state_rows);
  const long long qk = (long long)pr->heads_k * pr->d_k, v = (long long)pr->heads_v * pr->d_v;
  const long long unit = pr->qkv_dtype == GDN_BF16 ? 8 : 4;   // elements in 16 bytes
  struct { const char* name; long long given, width; } st[] = {
      {"q_stride", pr->q_stride, qk}, {"k_stride", pr->k_stride, qk}, {"v_stride", pr->v_stride, v}};
  for (const auto& s : st)
    if (s.given != 0 && (s.given < s.width || s.given % unit || s.given > (1LL << 23)))
      return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be 0 or a multiple of 16 bytes in [%lld, 2^23] elements (got %lld)",
                  s.name, s.width, s.given);
  out->hk = pr->heads_k;
  out->hv = pr->heads_v;
  out->dk = pr->d_k;
  out->dv = pr->d_v;
  out->in_bf16 = pr->qkv_dtype == GDN_BF16;
  out->out_bf16 = pr->out_dtype == GDN_BF16;
  out->state_rows = pr->state_rows;
  out->tokens = pr->tokens;
  out->qs = pr->q_stride ? pr->q_stride : qk;
  out->ks = pr->k_stride ? pr->k_stride : qk;
  out->vs = pr->v_stride ? pr->v_stride : v;
  out->sequences = pr->sequences;
  return GDN_OK;
}

inline gdn_status check_packed(const gdn_seq_problem* pr, bool slots, SeqProblem* out) {
  const gdn_status s = check_seq(pr, slots, out);
  if (s != GDN_OK) return s;
  // one workgroup for 16 columns of each (sequence, value head)
  if (pr->sequences < 0 || (long long)pr->sequences * pr->heads_v > (1LL << 20))
    return fail(GDN_ERR_INVALID_ARGUMENT, "sequences must be >= 0 and sequences * heads_v at most 2^20 (got %d, %d heads)",
                pr->sequences, pr->heads_v);
  return GDN_OK;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Pointers that must be there; `wide` ones are read 16 bytes at a time.
inline gdn_status check_needed(std::initializer_list<const void*> needed, const char* names) {
  for (const void* p : needed)
    if (!p) return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be non-NULL", names);
  return GDN_OK;
}

inline gdn_status check_aligned(std::initializer_list<const void*> wide, std::initializer_list<const void*> narrow) {
  for (const void* p : wide)
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARGUMENT, "tensor and workspace pointers must be 16-byte aligned");
  for (const void* p : narrow)
    if (!aligned4(p))
      return fail(GDN_ERR_INVALID_ARGUMENT, "log_gate, beta, cu_seqlens and slots pointers must be 4-byte aligned");
  return GDN_OK;
}

inline gdn_status check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (need > 0 && (!workspace || bytes < need))
    return fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes needed, %zu given%s", need, bytes,
                workspace ? "" : " (NULL)");
  return GDN_OK;
}

inline gdn_status finish(hipError_t e) {
  if (e != hipSuccess) return fail(GDN_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
  clear_error();
  return GDN_OK;
}

}  // namespace gdn
