// Gradients of linear attention with a decay for each head: three scans over the
// same operands, then the gates' gradients from sums of theirs.
#include <cstddef>

#include "gdn_linear_scan.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr float kNoGate = -103.97207641601562f;   // exp of less rounds to 0 in fp32: it is below 2^-150, half of the smallest value

// The sums of x and y over the workgroup, in every lane; `red`: four pairs.
__device__ __forceinline__ double2 block_sum(double x, double y, double2* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    x += __shfl_xor(x, m);
    y += __shfl_xor(y, m);
  }
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = make_double2(x, y);
  __syncthreads();
  return make_double2(red[0].x + red[1].x + red[2].x + red[3].x, red[0].y + red[1].y + red[2].y + red[3].y);
}

struct GateArgs {
  const float* qdq;         // [head][token]
  const float* vdv;
  const float* states;      // [bound][head][cell]
  const float* rstates;
  const float* last;        // [sequence][head][cell]: the final states
  const float* dlast;       // their gradients, or null
  const float* h0;          // the initial states, or null
  const float* dh0;         // their gradients, or null
  float* dg;                // [token][head]
  double* sums;             // one gate a head: [slot][head]
};

// dlog_gate of a segment's tokens, D_t = <R, S> before token t, in fp64: <R, S> at the segment's end and the sums of x = q.dq -
// v.dv behind each token, both without what a token reads of itself.  The x are rounded independently (1e-7 of them), so the sums' error grows like a random walk to the
// segment's start, where it shows: the sum is not the <R, S> of that place.  What it is off by is taken back along the way, by
// the parts of the walk's variance behind each token (16384 tokens, 35 heads of 64 with a gate each, six inputs: errors of the
// gates' gradients 0.6 to 4.5e-6 without, 0.7 to 2.1e-6 with it, 2.3 to 9.1e-7 in segments of 512, 3.4e-7 to 1.7e-6 there without).  The first gate of a sequence that starts from zeros scales nothing, and one
// whose exponential is 0 in fp32 (-inf, a mask's lowest value) drops what it scales: their gradients are 0, not what the
// sums' roundings leave.
__global__ __launch_bounds__(kThreads) void linear_gates_kernel(ScanArgs s, GateArgs a, int cell) {
  __shared__ double2 red[4];
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64, hv = s.hk * s.rep;
  const uint32_t items = s.slots * hv;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int slot = item / (uint32_t)hv, h = item - slot * hv;
    Segment seg;
    if (!find_segment(s.cu, s.sequences, s.tokens, s.L, slot, &seg) || seg.n == 0) {
      if (a.sums && tid == 0) a.sums[item] = 0;
      continue;
    }
    // S and R at the segment's end and start; where one is zeros, or R is not there: null
    const float *S[2] = {nullptr, nullptr}, *R[2] = {nullptr, nullptr};
    const bool inner = seg.c < seg.count - 1;
    const size_t row = ((size_t)seg.seq * hv + h) * cell;
    if (inner || a.dlast) {
      const size_t at = inner ? (size_t)(bound_of(seg.start, seg.c, s.L) * hv + h) * cell : row;
      S[0] = (inner ? a.states : a.last) + at;
      R[0] = (inner ? a.rstates : a.dlast) + at;
    }
    if (seg.c > 0 || (a.h0 && a.dh0)) {
      const size_t at = seg.c > 0 ? (size_t)(bound_of(seg.start, seg.c - 1, s.L) * hv + h) * cell : row;
      S[1] = (seg.c > 0 ? a.states : a.h0) + at;
      R[1] = (seg.c > 0 ? a.rstates : a.dh0) + at;
    }
    const bool both = seg.c > 0 || !a.h0 || a.dh0;              // <R, S> at the start is known
    double ends[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (S[e]) {
#pragma unroll 4
        for (int i = tid * 4; i < cell; i += kThreads * 4) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(S[e] + i), y = *reinterpret_cast<const f32x4*>(R[e] + i);
#pragma unroll
          for (int r = 0; r < 4; ++r) ends[e] += (double)x[r] * y[r];
        }
      }
    const float* qdq = a.qdq + (size_t)h * s.tokens + seg.first;
    const float* vdv = a.vdv + (size_t)h * s.tokens + seg.first;
    double x = 0, var = 0;
    for (int i = tid; i < seg.n; i += kThreads) {
      const double u = qdq[i], v = vdv[i];
      x += u - v;
      var += u * u + v * v;
    }
    const double2 D = block_sum(ends[0], ends[1], red), all = block_sum(x, var, red);
    const double off = both && all.y > 0 ? (D.y - D.x - all.x) / all.y : 0;
    double carry = D.x, sum = 0;
    for (int end = seg.n; end > 0; end -= kThreads) {             // tokens end - 1 - tid
      const int i = end - 1 - tid;
      double x = 0;
      if (i >= 0) {
        const double u = qdq[i], v = vdv[i];
        x = u - v + off * (u * u + v * v);
      }
      x = prefix_sum(x);
      __syncthreads();
      if (lane == 63) red[w].x = x;
      __syncthreads();
      for (int k = 0; k < w; ++k) x += red[k].x;
      x += carry;
      carry += red[0].x + red[1].x + red[2].x + red[3].x;
      if (i >= 0) {
        const float g = s.g[s.fixed ? h : (size_t)(seg.first + i) * hv + h];
        if ((!a.h0 && seg.first + i == seg.start) || g < kNoGate) x = 0;
        if (a.sums) sum += x;
        else a.dg[(size_t)(seg.first + i) * hv + h] = (float)x;
      }
    }
    if (a.sums) {
      sum = block_sum(sum, 0, red).x;
      if (tid == 0) a.sums[item] = sum;
    }
    __syncthreads();
  }
}

// One gate a head: the sums of its segments.
__global__ __launch_bounds__(kThreads) void linear_gate_sums_kernel(const double* sums, long long slots, int hv, float* dg) {
  __shared__ double2 red[4];
  const int h = blockIdx.x;                                         // at most 65535
  double x = 0;
  for (long long i = threadIdx.x; i < slots; i += kThreads) x += sums[i * hv + h];
  x = block_sum(x, 0, red).x;
  if (threadIdx.x == 0) dg[h] = (float)x;
}

struct GradArgs {
  ScanArgs dq, dk, dv;
};

// dq, dk and dv in one launch: a unit's workgroups (of a segment and key head) one after another on one XCD, as they read the
// same rows; those that sum over value heads, the longest, first (three launches, and every value head's dq and dk summed
// afterwards: 507 us a call against 474 for 8192 tokens in 6, 16 and 32 heads of 128; fp32, 880 in 3, 148 against 89; both with
// two-term states).  That call spends 412 to 438 us here, 1.18 GB at 2.7 TB/s: operands three times, the sums over value heads in
// fp32 out and back, 61 spilled vector and 300 scalar registers; 16384 tokens of 35 heads of 64 282 to 312 us, 880 of fp32 50.
// KSK, CTK and KSV, CTV: by_width of d_k and d_v.
template <int NT, int KSK, int CTK, int KSV, int CTV>
__global__ __launch_bounds__(kScanThreads, 2) void linear_grad_kernel(GradArgs g) {
  using Q = ScanSpace<NT, KSV, CTK, true, true>;
  using K = ScanSpace<NT, KSV, CTK, true, false>;
  using V = ScanSpace<NT, KSK, CTV, true, true>;
  __shared__ union {
    Q q;
    K k;
    V v;
  } z;
  const uint32_t keys = g.dq.part ? 1 : g.dq.rep, parts = 2 * keys + g.dv.rep;
  const uint32_t blocks = scan_blocks(g.dv) / g.dv.rep * parts;
  for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    const uint32_t group = block / 8 / parts, unit = group * 8 + block % 8, part = block / 8 - group * parts;
    if (part < keys) {
      const ScanArgs s = scan_args_at(offsetof(GradArgs, dq));
      scan_item<NT, KSV, CTK, false, true, true>(s, unit, part, z.q);
    } else if (part < 2 * keys) {
      const ScanArgs s = scan_args_at(offsetof(GradArgs, dk));
      scan_item<NT, KSV, CTK, true, true, false>(s, unit, part - keys, z.k);
    } else {
      const ScanArgs s = scan_args_at(offsetof(GradArgs, dv));
      scan_item<NT, KSK, CTV, true, true, true>(s, unit, part - 2 * keys, z.v);
    }
  }
}

unsigned blocks_of(long long n) { return (unsigned)(n < 1 ? 1 : n < kMaxBlocks ? n : kMaxBlocks); }

}  // namespace

hipError_t linear_backward_launch(const LinearProblem& p, const LinearTensors& t, const LinearSpace& ws, hipStream_t stream) {
  const LinearPlan plan = linear_plan(p, true);
  const uint32_t es = p.in_bf16 ? 2 : 4;
  const Operand q = {static_cast<const char*>(t.q), (uint32_t)p.qs * es, p.dk, true};
  const Operand k = {static_cast<const char*>(t.k), (uint32_t)p.ks * es, p.dk, true};
  const Operand v = {static_cast<const char*>(t.v), (uint32_t)p.vs * es, p.dv, false};
  const Operand dout = {static_cast<const char*>(t.dout), (uint32_t)(p.hv * p.dv) * es, p.dv, false};
  ScanArgs forward = scan_args(p, t, plan), reversed = forward;
  forward.from = t.h0;
  forward.between = ws.states;
  forward.decay = ws.decay;
  reversed.from = t.dhT;
  reversed.between = ws.rstates;
  reversed.decay = ws.rdecay;
  hipError_t e = hipSuccess;
  if (p.sequences == 0) {                                         // nothing but a fixed gate's gradient, which is 0
    hipLaunchKernelGGL(linear_gate_sums_kernel, dim3(p.hv), dim3(kThreads), 0, stream, ws.dg, 0LL, p.hv, t.dg);
    return hipGetLastError();
  }
  if (plan.bounds) {
    ScanArgs f = forward, r = reversed;
    f.b = k;
    f.c = v;
    r.b = q;
    r.c = dout;
    e = linear_states(f, &r, p.in_bf16, stream);
    if (e != hipSuccess) return e;
  }
  const bool shared = p.hv > p.hk;
  GradArgs g = {forward, reversed, reversed};
  g.dq.a = dout;
  g.dq.b = v;
  g.dq.c = k;
  g.dq.d = q;
  g.dq.out = static_cast<char*>(t.dq);
  g.dq.part = shared ? ws.dq : nullptr;
  g.dq.dot = ws.qdq;
  g.dq.to = t.dhT ? ws.last : nullptr;
  g.dk.a = v;
  g.dk.b = dout;
  g.dk.c = q;
  g.dk.out = static_cast<char*>(t.dk);
  g.dk.part = shared ? ws.dk : nullptr;
  g.dv.a = k;
  g.dv.b = q;
  g.dv.c = dout;
  g.dv.d = v;
  g.dv.out = static_cast<char*>(t.dv);
  g.dv.dot = ws.vdv;
  g.dv.to = t.dh0;
  g.dq.out_bytes = g.dk.out_bytes = g.dv.out_bytes = es;
  g.dq.out_row = g.dk.out_row = (uint32_t)(p.hk * p.dk) * es;
  g.dv.out_row = (uint32_t)(p.hv * p.dv) * es;
  prof_begin(stream, GDN_KERNEL_LINEAR_SCAN);
  by_width(p.dk, [&](auto ksk, auto ctk) {
    by_width(p.dv, [&](auto ksv, auto ctv) {
      constexpr int KSK = decltype(ksk)::value, CTK = decltype(ctk)::value, KSV = decltype(ksv)::value, CTV = decltype(ctv)::value;
      const dim3 grid = scan_grid((long long)scan_blocks(g.dv) + 2LL * scan_blocks(g.dq)), threads(kScanThreads);
      if (p.in_bf16) hipLaunchKernelGGL((linear_grad_kernel<1, KSK, CTK, KSV, CTV>), grid, threads, 0, stream, g);
      else hipLaunchKernelGGL((linear_grad_kernel<3, KSK, CTK, KSV, CTV>), grid, threads, 0, stream, g);
    });
  });
  e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_LINEAR_SCAN);
  if (e != hipSuccess) return e;
  prof_begin(stream, GDN_KERNEL_LINEAR_GATES);
  const GateArgs a = {ws.qdq, ws.vdv, ws.states, ws.rstates, ws.last, t.dhT, t.h0, t.dh0, t.dg, p.fixed ? ws.dg : nullptr};
  hipLaunchKernelGGL(linear_gates_kernel, dim3(blocks_of(plan.slots * p.hv)), dim3(kThreads), 0, stream, forward, a, p.dk * p.dv);
  if (p.fixed) hipLaunchKernelGGL(linear_gate_sums_kernel, dim3(p.hv), dim3(kThreads), 0, stream, ws.dg, plan.slots, p.hv, t.dg);
  e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_LINEAR_GATES);
  return e;
}

}  // namespace gdn
