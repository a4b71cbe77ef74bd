// Linear attention with a decay for each head: outputs and final states, and the
// states between segments.
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "gdn_linear_scan.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

struct SumsArgs {
  ScanArgs forward, reversed;
  int directions;
};

template <int NT, int KS, int CT>
__global__ __launch_bounds__(kScanThreads, 2) void linear_sums_kernel(SumsArgs a) {
  __shared__ ScanSpace<NT, KS, CT, false, false> z;
  const uint32_t heads = a.forward.rep, parts = heads * a.directions, blocks = scan_blocks(a.forward) * a.directions;
  for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    const uint32_t group = block / 8 / parts, unit = group * 8 + block % 8, part = block / 8 - group * parts;
    if (part < heads) {
      const ScanArgs s = scan_args_at(offsetof(SumsArgs, forward));
      scan_item<NT, KS, CT, false, false, false>(s, unit, part, z);
    } else {
      const ScanArgs s = scan_args_at(offsetof(SumsArgs, reversed));
      scan_item<NT, KS, CT, true, false, false>(s, unit, part - heads, z);
    }
  }
}

// The states between the segments of a sequence from their sums, V times four elements of the state a lane: forward S <- e^G S +
// sum from the initial state, reversed R <- e^G R + sum from the final state's gradient.
template <bool REV, int V>
__device__ __forceinline__ void chain(const ScanArgs& s, int cell, int part, int seq, int h) {
  const int hv = s.hk * s.rep;
  const bool in_place = s.from && s.from == s.to;
  int a, b;
  seq_bounds(s.cu, seq, s.tokens, &a, &b);
  int each;
  const int count = segments_of(b - a, s.L, &each);
  if (count < 2) return;
  long long row = seq;
  if (s.state_slots) {
    row = s.state_slots[seq];
    if (row < 0 || row >= s.state_rows) row = -1;
    else if (in_place) {
      bool earlier;
      int next;
      same_slot(s.state_slots, s.sequences, seq, &earlier, &next);
      if (earlier || next < s.sequences) return;
    }
  }
  const int e = (part * V * kThreads + threadIdx.x) * 4;
  constexpr int kNext = kThreads * 4;
  if (V == 1 && e >= cell) return;                                // V = 2: cell is a multiple of what a workgroup has
  const long long slot = a / (uint32_t)s.L + seq;
  const long long b0 = bound_of(a, 0, s.L);
  float* at = s.between + (size_t)(b0 * hv + h) * cell + e;
  const size_t step = (size_t)hv * cell;
  f32x4 S[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    S[v] = s.from && row >= 0 ? *reinterpret_cast<const f32x4*>(s.from + ((size_t)row * hv + h) * cell + e + v * kNext) : zero4();
    if (!REV && in_place) *reinterpret_cast<f32x4*>(s.firsts + (size_t)(b0 * hv + h) * cell + e + v * kNext) = S[v];
  }
  // Two bounds at once: more cost instructions and registers where sequences have few (8191 tokens in 13, sums and states 40.5 us
  // at 2, 42 at 8, 48 at 16, 55 at 24), and gain nothing along 21 of them
  constexpr int kAhead = 2;
  for (int i0 = 0; i0 < count - 1; i0 += kAhead) {
    f32x4 u[kAhead][V];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = REV ? count - 2 - i0 - i : i0 + i;            // bound k, between segments k and k + 1
      if (i0 + i < count - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) u[i][v] = *reinterpret_cast<const f32x4*>(at + k * step + v * kNext);
        d[i] = s.decay[(slot + (REV ? k + 1 : k)) * hv + h];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = REV ? count - 2 - i0 - i : i0 + i;
      if (i0 + i < count - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          S[v] = d[i] * S[v] + u[i][v];
          *reinterpret_cast<f32x4*>(at + k * step + v * kNext) = S[v];
        }
      }
    }
  }
}

template <int V>
__global__ __launch_bounds__(kThreads) void linear_chain_kernel(ScanArgs f, ScanArgs r, int directions, int cell, int parts) {
  const uint32_t hv = f.hk * f.rep, each = f.sequences * hv * parts;       // at most 2^20 * 16
  for (uint32_t item = blockIdx.x; item < each * directions; item += gridDim.x) {
    const bool reversed = item >= each;
    const uint32_t i = reversed ? item - each : item, pair = i / (uint32_t)parts;
    const int part = i - pair * parts, seq = pair / hv, h = pair - seq * hv;
    if (reversed) chain<true, V>(r, cell, part, seq, h);
    else chain<false, V>(f, cell, part, seq, h);
  }
}

size_t carve(char** at, char* base, size_t* bytes, size_t n) {
  const size_t from = align_up(*bytes, 256);
  *at = base ? base + from : nullptr;
  *bytes = from + n;
  return n;
}

}  // namespace

// Segments.  A scan's workgroup takes about as long beside another on its CU as alone, and every segment costs the bytes of
// a state, four times, and a start of some chunks' time: so there are about as many (segment, head) pairs as workgroups run at
// once (LDS and registers: two a CU, three where no width is above 64, forward and bf16), with half a segment more for each
// sequence's last one, or twice as many and so on where the sequences alone are that many.  Prompts of 8191 tokens in 13,
// 32 heads of 128: 188 us at 256 tokens a segment, 170 at 512, 157 at 768, 167 at 1024, 152 to 159 as here; gradients of 8192 in 6:
// 608, 538, 565, 583, 505; one document of 32768, 35 heads of 64: 281 at 512, 280 at 1024, 264 at 1536, 287 at 2048, 346 at 4096,
// 243 as here.  One workgroup alone takes 7 us for a chunk of 64 tokens, which bounds short calls: 880 tokens in 3 of fp32, 20 heads
// of 112 (gradients): 94 us at 128 tokens a segment, 121 at 256, 128 at 512; but up to 384 tokens the two launches more cost more
// (203 tokens: 20 us in one, 30 at 128).  Heads are counted by the value: where many share a key head, whose workgroups sum them
// one after another in the gradients, there are too few of those (8000 tokens, 32 heads of 64: 191 us with as many key heads, 230
// with 16, 383 with 4, 1122 with one).
// The errors of gates' gradients grow with a segment (linear_gates_kernel), those of one gate a head twice over: their
// segments end at 1536 and 512 tokens (16384 tokens, 35 heads of 64 with a gate each: 409 us at 512, 394 at 1536).
LinearPlan linear_plan(const LinearProblem& p, bool grad) {
  const bool wide = p.dk > 64 || p.dv > 64;
  const double at_once = 256.0 * (wide || grad || !p.in_bf16 ? 2 : 3), each = at_once / p.hv, half = 0.5 * p.sequences;
  const double wanted = p.sequences <= 1 ? std::fmax(1.0, std::floor(each))
                                         : (std::floor(half / each + 0.5) + 1) * each - half;
  double tokens = (double)p.tokens / wanted * (p.sequences <= 1 ? 1.0 : 1.03);
  tokens = tokens < 128 ? 128 : tokens;
  if (grad && tokens > (p.fixed ? 512 : 1536)) tokens = p.fixed ? 512 : 1536;
  long long L = tokens < (double)p.tokens ? ((long long)std::ceil(tokens) + 63) / 64 * 64 : p.tokens;
  if (p.tokens <= 384 || L >= p.tokens) L = (p.tokens + 64) / 64 * 64;       // one segment, and none behind it
  LinearPlan plan;
  plan.L = (int)L;
  plan.slots = p.tokens / L + p.sequences;
  plan.bounds = p.tokens / L;
  return plan;
}

size_t linear_space(const LinearProblem& p, bool grad, void* base, LinearSpace* s) {
  LinearSpace none;
  LinearSpace& o = s ? *s : none;
  o = {};
  char* at = nullptr;
  size_t bytes = 0;
  const LinearPlan plan = linear_plan(p, grad);
  const auto take = [&](auto** to, size_t n) {
    if (n == 0) return;
    carve(&at, static_cast<char*>(base), &bytes, n * sizeof **to);
    *to = reinterpret_cast<std::remove_reference_t<decltype(*to)>>(at);
  };
  const size_t cell = (size_t)p.dk * p.dv, states = (size_t)plan.bounds * p.hv * cell;
  const size_t segments = plan.bounds ? (size_t)plan.slots * p.hv : 0;
  take(&o.states, states);
  take(&o.decay, segments);
  if (!grad) {
    take(&o.firsts, states);
    return bytes;
  }
  take(&o.rstates, states);
  take(&o.rdecay, segments);
  take(&o.last, (size_t)p.sequences * p.hv * cell);
  take(&o.qdq, (size_t)p.tokens * p.hv);
  take(&o.vdv, (size_t)p.tokens * p.hv);
  if (p.hv > p.hk) {
    take(&o.dq, (size_t)p.tokens * p.hk * p.dk);
    take(&o.dk, (size_t)p.tokens * p.hk * p.dk);
  }
  if (p.fixed) take(&o.dg, (size_t)plan.slots * p.hv);
  return bytes;
}

hipError_t linear_states(const ScanArgs& forward, const ScanArgs* reversed, bool bf16, hipStream_t stream) {
  const int directions = reversed ? 2 : 1;
  const ScanArgs& r = reversed ? *reversed : forward;
  const SumsArgs a = {forward, r, directions};
  prof_begin(stream, GDN_KERNEL_LINEAR_STATES);
  by_width(forward.b.width, [&](auto ks, auto) {
    by_width(forward.c.width, [&](auto, auto ct) {
      constexpr int KS = decltype(ks)::value, CT = decltype(ct)::value;
      const dim3 grid = scan_grid((long long)scan_blocks(forward) * directions), threads(kScanThreads);
      if (bf16) hipLaunchKernelGGL((linear_sums_kernel<1, KS, CT>), grid, threads, 0, stream, a);
      else hipLaunchKernelGGL((linear_sums_kernel<3, KS, CT>), grid, threads, 0, stream, a);
    });
  });
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) {
    // Two vectors a lane where that divides a state and there are more workgroups than run at once: 8191 tokens in 13, 32 heads of
    // 128: 38 us with the sums against 42; but 35 heads of 64 in one sequence 88 against 84.
    const int cell = forward.b.width * forward.c.width, parts = (cell + kThreads * 4 - 1) / (kThreads * 4);
    const long long items = (long long)forward.sequences * forward.hk * forward.rep * parts * directions;
    if (items > 2048 && cell % (kThreads * 8) == 0)
      hipLaunchKernelGGL(linear_chain_kernel<2>, scan_grid(items / 2), dim3(kThreads), 0, stream, forward, r, directions, cell, parts / 2);
    else
      hipLaunchKernelGGL(linear_chain_kernel<1>, scan_grid(items), dim3(kThreads), 0, stream, forward, r, directions, cell, parts);
    e = hipGetLastError();
  }
  prof_end(stream, GDN_KERNEL_LINEAR_STATES);
  return e;
}

ScanArgs scan_args(const LinearProblem& p, const LinearTensors& t, const LinearPlan& plan) {
  ScanArgs s = {};
  s.g = t.g;
  s.cu = t.cu;
  s.tokens = p.tokens;
  s.slots = plan.slots;
  s.sequences = p.sequences;
  s.hk = p.hk;
  s.rep = p.hv / p.hk;
  s.L = plan.L;
  s.fixed = p.fixed;
  s.scale = p.scale;
  return s;
}

hipError_t linear_forward_launch(const LinearProblem& p, const LinearTensors& t, const LinearSpace& ws, hipStream_t stream) {
  const LinearPlan plan = linear_plan(p, false);
  const uint32_t es = p.in_bf16 ? 2 : 4;
  ScanArgs s = scan_args(p, t, plan);
  s.a = {static_cast<const char*>(t.q), (uint32_t)p.qs * es, p.dk, true};
  s.b = {static_cast<const char*>(t.k), (uint32_t)p.ks * es, p.dk, true};
  s.c = {static_cast<const char*>(t.v), (uint32_t)p.vs * es, p.dv, false};
  s.out = static_cast<char*>(t.out);
  s.out_bytes = p.out_bf16 ? 2 : 4;
  s.out_row = (uint32_t)p.hv * p.dv * s.out_bytes;
  s.from = t.h0;
  s.to = t.hT;
  s.state_slots = t.slots;
  s.state_rows = p.state_rows;
  s.between = ws.states;
  s.firsts = ws.firsts;
  s.decay = ws.decay;
  if (plan.bounds) {
    const hipError_t e = linear_states(s, nullptr, p.in_bf16, stream);
    if (e != hipSuccess) return e;
  }
  prof_begin(stream, GDN_KERNEL_LINEAR_SCAN);
  by_width(p.dk, [&](auto ks, auto) {
    by_width(p.dv, [&](auto, auto ct) {
      constexpr int KS = decltype(ks)::value, CT = decltype(ct)::value;
      const dim3 grid = scan_grid(scan_blocks(s)), threads(kScanThreads);
      if (p.in_bf16) hipLaunchKernelGGL((linear_scan_kernel<1, KS, CT>), grid, threads, 0, stream, s);
      else hipLaunchKernelGGL((linear_scan_kernel<3, KS, CT>), grid, threads, 0, stream, s);
    });
  });
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_LINEAR_SCAN);
  return e;
}

}  // namespace gdn
