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

// ---------------------------------------------------------------- packed sequences

// Rows of one operand of a scan.
struct Operand {
  const char* p;
  uint32_t row;       // bytes between tokens
  int width;          // of a head, in values
  bool shared;        // by the value heads of a key head
};

// One scan, or the sums of its segments (operand a is not used then).
struct ScanArgs {
  Operand a, b, c;
  Operand d;                // DOT: rows of the same shape as the outputs'
  const float* g;
  const int* cu;
  long long tokens, slots;
  int sequences, hk, rep, L;
  bool fixed;
  float scale;
  // outputs
  char* out;
  uint32_t out_row;
  int out_bytes;            // of a value
  float* part;              // dq and dk of shared key heads: sums over value heads so far, [token][key head][J]; or null
  float* dot;               // [head][token]
  // states
  const float* from;        // of sequences, or rows of a pool; or null (zeros)
  float* to;                // or null
  const int* state_slots;   // or null
  int state_rows;
  float* between;           // states between segments [bound][head]: sums first, then states
  float* firsts;            // in place: states before a sequence's first segment, at its first bound
  float* decay;             // [slot][head]: of a segment
};

// Everything a call reads or writes besides the workspace.
struct LinearTensors {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const int* cu;
  const int* slots;
  const float* h0;
  void* out;
  float* hT;
  // gradients
  const void* dout;
  const float* dhT;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dh0;
};

struct LinearPlan {
  int L;                    // tokens of a segment
  long long slots;          // segments, at most
  long long bounds;         // between segments of one sequence, at most; 0: every sequence is one segment
};

LinearPlan linear_plan(const LinearProblem& p, bool grad);

// Workspace of a call: what is not needed is null.
struct LinearSpace {
  float* states;            // [bound][heads_v][d_k][d_v]
  float* decay;             // [slot][heads_v]
  float* firsts;            // forward: like states
  // gradients
  float* rstates;           // like states
  float* rdecay;
  float* last;              // [sequence][heads_v][d_k][d_v]: final states
  float* qdq;               // [heads_v][tokens]
  float* vdv;
  float* dq;                // shared key heads: sums so far, [tokens][heads_k][d_k]
  float* dk;
  double* dg;               // one gate a head: [slot][heads_v]
};

size_t linear_space(const LinearProblem& p, bool grad, void* base, LinearSpace* s);   // bytes; fills *s if not null

ScanArgs scan_args(const LinearProblem& p, const LinearTensors& t, const LinearPlan& plan);   // what all its scans share

hipError_t linear_forward_launch(const LinearProblem& p, const LinearTensors& t, const LinearSpace& s, hipStream_t stream);
hipError_t linear_backward_launch(const LinearProblem& p, const LinearTensors& t, const LinearSpace& s, hipStream_t stream);

// The sums of every segment's contributions to the state, and the states between segments from them (gdn_linear.hip): of the
// forward scan, and of the reversed one where it is given.
hipError_t linear_states(const ScanArgs& forward, const ScanArgs* reversed, bool bf16, hipStream_t stream);

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
