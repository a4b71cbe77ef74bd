// Internal interface between the C-ABI layer of the sequence operators
// (gdn_seq_api.cpp) and their kernel launchers.  Not installed; not part of
// the ABI.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// A validated sequence problem; strides in elements, never 0.
struct SeqProblem {
  int hk, hv, dk, dv;
  bool in_bf16, out_bf16;
  int state_rows;               // bound of the slots, where they are given
  long long tokens;
  long long qs, ks, vs;
  int sequences;
};

// Grids stay below 2^31 threads; work beyond that is looped over.
constexpr long long kMaxBlocks = 1 << 21;

hipError_t decode_launch(const SeqProblem& p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, float* state, const int* slots, void* out, hipStream_t stream);

}  // namespace gdn
