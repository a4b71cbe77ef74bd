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

// ---------------------------------------------------------------- packed sequences

constexpr int kC = 64;         // tokens of a chunk
constexpr int kTri = 8;        // fragments of a 64 x 64 matrix: [row tile 4][column half 2]

// Workspace of a packed call.  A cell is one (chunk slot, value head); chunk
// slots of sequence s start at cu[s] / 64 + s (floor), which never overlap.
// Sizes in bytes per item.
struct PackedSpace {
  uint4* t1;      // cells: T' = (I + B diag(beta))^-1, fragments x 3 terms
  uint4* p;       // cells: P (forward) or P^T (gradients), fragments x 3 terms
  float* gates;   // cells: e^G, e^(Gn - G), beta, 64 each
  uint4* kt;      // (slot, key head): K^T fragments [d_k tile][token half] x input terms
  // gradients only
  uint4* t2;      // cells: T^T with T = (I + diag(beta) B)^-1
  uint4* qt;      // as kt, of Q
  double* g;      // cells: G in units of log 2, 64
  float* e;       // cells: residuals e [strip][64 tokens][16 columns]
  float* w;       // cells: W = T^T dU, laid out like e
  float* s0;      // cells: state before the chunk [strip][d_k padded][16 columns]
  float* ds;      // cells: gradient of the state after the chunk, laid out like s0
};

struct PackedPlan {
  long long slots;     // chunk slots
  int strips;          // d_v / 16
  int dkp;             // d_k padded to 32, 64 or 128
  int terms;           // of q, k, v, dout: 1 (bf16) or 3 (fp32)
};

PackedPlan packed_plan(const SeqProblem& p);
size_t packed_space(const SeqProblem& p, bool grad, void* base, PackedSpace* s);   // bytes; fills *s if not null

// Everything a packed kernel reads or writes besides the workspace.
struct PackedTensors {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
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
  float* dbeta;
  float* dh0;
};

hipError_t packed_prep(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, bool grad, hipStream_t stream);
hipError_t packed_scan(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, bool grad, hipStream_t stream);
hipError_t packed_scan_grad(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, hipStream_t stream);
hipError_t packed_grads(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, hipStream_t stream);

}  // namespace gdn
