// Internal interface between the C-ABI layer (gdn_seq_api.cpp) and the group
// norm kernels (gdn_norm.hip).  Not installed; not part of the ABI.
#pragma once

#include "gdn_seq.h"

namespace gdn {

// A validated group norm: x [N, S, C], G groups of cg channels.
struct NormProblem {
  long long N;
  int S, C, G, cg, act;
  bool bf16, center;
  float eps;
};

// How the S > 1 kernels cut the work.  A group has `per` channel vectors; a
// workgroup has `tile` of them (whole groups, or one of `pieces` of a group), in
// `tiles` along the channels, and one of `splits` ranges of `rows` rows, `rpb`
// at a time; z workgroups walk over n.  A (n, group) has `parts` partial sums.
struct NormPlan {
  int per, tile, tiles, pieces, rpb, rows, splits, parts, threads, z;
};

// Device pointers of a gradient call (bias, gate, dgate, dweight, dbias and,
// without centring, mean may be null).
struct NormGrad {
  const void* dout;
  const void* x;
  const float* weight;
  const float* bias;
  const void* gate;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dgate;
  float* dweight;
  float* dbias;
};

size_t norm_workspace(const NormProblem& p, bool gradient);
hipError_t norm_launch(const NormProblem& p, const void* x, const float* weight, const float* bias, const void* gate, void* out,
                       float* mean, float* rstd, void* ws, hipStream_t stream);
hipError_t norm_grad_launch(const NormProblem& p, const NormGrad& t, void* ws, hipStream_t stream);

}  // namespace gdn
