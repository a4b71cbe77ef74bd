// Gradients of linear attention with a decay for each head: three scans over the
// same operands, then the gates' gradients from sums of theirs.
#include "gdn_linear_scan.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// The sum of x over the workgroup, in every lane; `red`: four values.
__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = x;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

struct GateArgs {
  const float* qdq;         // [head][token]
  const float* vdv;
  const float* states;      // [bound][head][cell]
  const float* rstates;
  const float* last;        // [sequence][head][cell]: the final states
  const float* dlast;       // their gradients, or null
  bool from_zero;           // no initial states
  float* dg;                // [token][head]
  double* sums;             // one gate a head: [slot][head]
};

// dlog_gate of a segment's tokens: <R, S> at its end and the sums of q.dq - v.dv behind each token, in fp64.  The first
// gate of a sequence that starts from zeros scales nothing: its gradient is 0, not what the sums' roundings leave.
__global__ __launch_bounds__(kThreads) void linear_gates_kernel(ScanArgs s, GateArgs a, int cell) {
  __shared__ double red[4];
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64, hv = s.hk * s.rep;
  const uint32_t items = s.slots * hv;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int slot = item / (uint32_t)hv, h = item - slot * hv;
    Segment seg;
    if (!find_segment(s.cu, s.sequences, s.tokens, s.L, slot, &seg) || seg.n == 0) {
      if (a.sums && tid == 0) a.sums[item] = 0;
      continue;
    }
    const float *S = nullptr, *R = nullptr;
    if (seg.c < seg.count - 1) {
      const size_t at = (size_t)(bound_of(seg.start, seg.c, s.L) * hv + h) * cell;
      S = a.states + at;
      R = a.rstates + at;
    } else if (a.dlast) {
      const size_t at = ((size_t)seg.seq * hv + h) * cell;
      S = a.last + at;
      R = a.dlast + at;
    }
    double carry = 0;
    if (S) {
      for (int i = tid * 4; i < cell; i += kThreads * 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(S + i), y = *reinterpret_cast<const f32x4*>(R + i);
#pragma unroll
        for (int r = 0; r < 4; ++r) carry += (double)x[r] * y[r];
      }
    }
    carry = block_sum(carry, red);
    double sum = 0;
    for (int end = seg.n; end > 0; end -= kThreads) {             // tokens end - 1 - tid
      const int i = end - 1 - tid;
      double x = 0;
      if (i >= 0) {
        const size_t at = (size_t)h * s.tokens + seg.first + i;
        x = (double)a.qdq[at] - a.vdv[at];
      }
      x = prefix_sum(x);
      __syncthreads();
      if (lane == 63) red[w] = x;
      __syncthreads();
      for (int k = 0; k < w; ++k) x += red[k];
      x += carry;
      carry += red[0] + red[1] + red[2] + red[3];
      if (i >= 0) {
        if (a.from_zero && seg.first + i == seg.start) x = 0;
        if (a.sums) sum += x;
        else a.dg[(size_t)(seg.first + i) * hv + h] = (float)x;
      }
    }
    if (a.sums) {
      sum = block_sum(sum, red);
      if (tid == 0) a.sums[item] = sum;
    }
    __syncthreads();
  }
}

// One gate a head: the sums of its segments.
__global__ __launch_bounds__(kThreads) void linear_gate_sums_kernel(const double* sums, long long slots, int hv, float* dg) {
  __shared__ double red[4];
  const int h = blockIdx.x;                                         // at most 65535
  double x = 0;
  for (long long i = threadIdx.x; i < slots; i += kThreads) x += sums[i * hv + h];
  x = block_sum(x, red);
  if (threadIdx.x == 0) dg[h] = (float)x;
}

// Gradients of a key head: the sums of its value heads', four values a lane.
__global__ __launch_bounds__(kThreads) void linear_heads_kernel(ScanArgs s, const float* parts, void* out, int width, bool bf16) {
  const int t0 = min(max(s.cu[0], 0), (int)s.tokens), t1 = min(max(s.cu[s.sequences], t0), (int)s.tokens);
  const long long quads = (long long)(t1 - t0) * s.hk * width / 4;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < quads; i += (long long)gridDim.x * kThreads) {
    const long long e = (long long)t0 * s.hk * width + i * 4, head = e / width;     // head: of tokens * hk
    const float* p = parts + head * s.rep * width + e % width;
    f32x4 x = *reinterpret_cast<const f32x4*>(p);
    for (int r = 1; r < s.rep; ++r) x += *reinterpret_cast<const f32x4*>(p + (size_t)r * width);
    if (bf16) {
      uint32_t lo[1], hi[1];
      split2<1>(x[0], x[1], lo);
      split2<1>(x[2], x[3], hi);
      reinterpret_cast<uint2*>(out)[e / 4] = make_uint2(lo[0], hi[0]);
    } else {
      reinterpret_cast<f32x4*>(out)[e / 4] = x;
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
    ScanArgs s = forward;
    s.b = k;
    s.c = v;
    e = linear_states(s, p.in_bf16, false, stream);
    if (e != hipSuccess) return e;
    s = reversed;
    s.b = q;
    s.c = dout;
    e = linear_states(s, p.in_bf16, true, stream);
    if (e != hipSuccess) return e;
  }
  const bool shared = p.hv > p.hk;
  prof_begin(stream, GDN_KERNEL_LINEAR_SCAN);
  {
    ScanArgs s = forward;
    s.a = dout;
    s.b = v;
    s.c = k;
    s.d = q;
    s.out = shared ? reinterpret_cast<char*>(ws.dq) : static_cast<char*>(t.dq);
    s.out_bytes = shared ? 4 : es;
    s.out_row = (uint32_t)(p.hv * p.dk) * s.out_bytes;
    s.dot = ws.qdq;
    s.to = t.dhT ? ws.last : nullptr;
    e = p.in_bf16 ? scan_variant<1, 3, false, true, true>(s, stream) : scan_variant<3, 3, false, true, true>(s, stream);
  }
  if (e == hipSuccess) {
    ScanArgs s = reversed;
    s.a = k;
    s.b = q;
    s.c = dout;
    s.d = v;
    s.out = static_cast<char*>(t.dv);
    s.out_bytes = es;
    s.out_row = (uint32_t)(p.hv * p.dv) * es;
    s.dot = ws.vdv;
    s.to = t.dh0;
    e = p.in_bf16 ? scan_variant<1, 3, true, true, true>(s, stream) : scan_variant<3, 3, true, true, true>(s, stream);
  }
  if (e == hipSuccess) {
    ScanArgs s = reversed;
    s.a = v;
    s.b = dout;
    s.c = q;
    s.out = shared ? reinterpret_cast<char*>(ws.dk) : static_cast<char*>(t.dk);
    s.out_bytes = shared ? 4 : es;
    s.out_row = (uint32_t)(p.hv * p.dk) * s.out_bytes;
    e = p.in_bf16 ? scan_variant<1, 2, true, true, false>(s, stream) : scan_variant<3, 3, true, true, false>(s, stream);
  }
  prof_end(stream, GDN_KERNEL_LINEAR_SCAN);
  if (e != hipSuccess) return e;
  prof_begin(stream, GDN_KERNEL_LINEAR_GATES);
  const GateArgs a = {ws.qdq, ws.vdv, ws.states, ws.rstates, ws.last, t.dhT, t.h0 == nullptr, t.dg, p.fixed ? ws.dg : nullptr};
  hipLaunchKernelGGL(linear_gates_kernel, dim3(blocks_of(plan.slots * p.hv)), dim3(kThreads), 0, stream, forward, a, p.dk * p.dv);
  if (p.fixed) hipLaunchKernelGGL(linear_gate_sums_kernel, dim3(p.hv), dim3(kThreads), 0, stream, ws.dg, plan.slots, p.hv, t.dg);
  if (shared) {
    const dim3 grid(blocks_of((p.tokens * p.hk * p.dk / 4 + kThreads - 1) / kThreads));
    hipLaunchKernelGGL(linear_heads_kernel, grid, dim3(kThreads), 0, stream, forward, ws.dq, t.dq, p.dk, p.in_bf16);
    hipLaunchKernelGGL(linear_heads_kernel, grid, dim3(kThreads), 0, stream, forward, ws.dk, t.dk, p.dk, p.in_bf16);
  }
  e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_LINEAR_GATES);
  return e;
}

}  // namespace gdn
