// Internal interface between the C-ABI layer of linear attention and rotary
// positions (gdn_linear_api.cpp) and their kernel launchers.  Not installed; not
// part of the ABI.
#pragma once

#include "gdn_seq.h"

namespace gdn {

// A validated problem; strides in elements, never 0.
struct LinearProblem : SeqProblem {
  float scale;
  bool fixed;                   // one gate a head
};

hipError_t linear_decode_launch(const LinearProblem& p, const void* q, const void* k, const void* v, const float* g,
                                float* state, const int* slots, void* out, hipStream_t stream);

// ---------------------------------------------------------------- rotary positions

struct RotaryProblem {
  bool bf16;
  long long tokens;
  int hq, hk, width, pairs;
  bool interleaved;
  int axes;
  int ends[4];                  // first pair behind each axis
  float cos_factor, sin_factor; // the magnitude, and with the turn's sign
  long long qs, ks, qos, kos;   // strides in elements
};

hipError_t rotary_launch(const RotaryProblem& p, const void* q, const void* k, const int* positions, const double* frequencies,
                         void* q_out, void* k_out, hipStream_t stream);

}  // namespace gdn
