// One token of the gated delta rule for each row of a serving batch.
//
// With a = exp(g) and the state S (d_k x d_v, fp32) of the row's slot:
//     u = beta (v - a S^T k),   S <- a S + k u^T,   o = S^T q = a S_old^T q + (q.k) u
// so one pass over S_old gives both products (S^T k and S^T q), and S is read
// once and written once: 8 d_k d_v bytes for 7 d_k d_v flops, bound by HBM.
//
// Work split: the columns of S evolve independently, so a workgroup takes W
// columns of one (row, value head).  A thread holds R rows x 4 columns in
// registers (one 16-byte load each, all in flight at once); the sums over rows
// go through lane shuffles, then one LDS exchange between the four wavefronts.
#include "gdn_common.h"
#include "gdn_seq.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <bool BF16IN, int W>
__global__ __launch_bounds__(kThreads) void decode_kernel(
    const void* __restrict__ q, const void* __restrict__ k, const void* __restrict__ v, const float* __restrict__ g,
    const float* __restrict__ beta, float* state, const int* __restrict__ slots, void* __restrict__ out, SeqProblem p) {
  constexpr int L = W / 4;               // lanes along a state row
  constexpr int RG = kThreads / L;       // rows of the state held at once
  constexpr int R = (128 + RG - 1) / RG; // state rows of a thread
  __shared__ float red[4][2 * W + 1];
  __shared__ int earlier, next;
  const int tid = threadIdx.x, wave = tid / 64;
  const int rg = tid / L, c = (tid % L) * 4;
  const int strips = (p.dv + W - 1) / W;
  const int h = blockIdx.x / strips, col = (blockIdx.x % strips) * W + c;
  const bool live = col < p.dv;          // d_v is a multiple of 16: four columns are in or out together
  const int kh = h / (p.hv / p.hk);

  for (long long first = blockIdx.y; first < p.tokens; first += gridDim.y) {
    const int slot = slots ? slots[first] : (int)first;
    if (slots && (slot < 0 || slot >= p.state_rows)) continue;   // padding (uniform over the workgroup)
    float* S = state + ((size_t)slot * p.hv + h) * p.dk * p.dv;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = rg + RG * i;
      s[i] = live && r < p.dk ? *reinterpret_cast<const float4*>(S + (size_t)r * p.dv + col) : make_float4(0, 0, 0, 0);
    }
    long long row = first;
    if (slots) {
      // rows of the same slot belong to the workgroup of the first of them
      __syncthreads();
      if (tid == 0) { earlier = 0; next = 0x7fffffff; }
      __syncthreads();
      for (long long i = tid; i < p.tokens; i += kThreads)
        if (slots[i] == slot) {
          if (i < row) earlier = 1;
          else if (i > row) atomicMin(&next, (int)i);
        }
      __syncthreads();
      if (earlier) continue;
    }
    for (;;) {
      const float a = expf(g[(size_t)row * p.hv + h]), b = beta[(size_t)row * p.hv + h];
      float kr[R], acc[9];
#pragma unroll
      for (int j = 0; j < 9; ++j) acc[j] = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = rg + RG * i;
        const bool in = r < p.dk;
        kr[i] = in ? load_scalar<BF16IN>(k, (size_t)row * p.ks + kh * p.dk + r) : 0.f;
        const float qr = in ? load_scalar<BF16IN>(q, (size_t)row * p.qs + kh * p.dk + r) : 0.f;
        acc[0] = fmaf(kr[i], s[i].x, acc[0]);
        acc[1] = fmaf(kr[i], s[i].y, acc[1]);
        acc[2] = fmaf(kr[i], s[i].z, acc[2]);
        acc[3] = fmaf(kr[i], s[i].w, acc[3]);
        acc[4] = fmaf(qr, s[i].x, acc[4]);
        acc[5] = fmaf(qr, s[i].y, acc[5]);
        acc[6] = fmaf(qr, s[i].z, acc[6]);
        acc[7] = fmaf(qr, s[i].w, acc[7]);
        acc[8] = fmaf(qr, kr[i], acc[8]);
      }
#pragma unroll
      for (int m = L; m < 64; m <<= 1)
#pragma unroll
        for (int j = 0; j < 9; ++j) acc[j] += __shfl_xor(acc[j], m);
      __syncthreads();                   // the previous row's sums have been read
      if (tid % 64 < L) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          red[wave][c + j] = acc[j];
          red[wave][W + c + j] = acc[4 + j];
        }
        if (tid % 64 == 0) red[wave][2 * W] = acc[8];
      }
      __syncthreads();
      const float qk = red[0][2 * W] + red[1][2 * W] + red[2][2 * W] + red[3][2 * W];
      float u[4], o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float ks = red[0][c + j] + red[1][c + j] + red[2][c + j] + red[3][c + j];
        const float qs = red[0][W + c + j] + red[1][W + c + j] + red[2][W + c + j] + red[3][W + c + j];
        const float vj = live ? load_scalar<BF16IN>(v, (size_t)row * p.vs + (size_t)h * p.dv + col + j) : 0.f;
        u[j] = b * (vj - a * ks);
        o[j] = fmaf(a, qs, qk * u[j]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[i].x = fmaf(a, s[i].x, kr[i] * u[0]);
        s[i].y = fmaf(a, s[i].y, kr[i] * u[1]);
        s[i].z = fmaf(a, s[i].z, kr[i] * u[2]);
        s[i].w = fmaf(a, s[i].w, kr[i] * u[3]);
      }
      if (live && rg == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store_scalar(out, ((size_t)row * p.hv + h) * p.dv + col + j, o[j], p.out_bf16);
      }
      if (!slots || next == 0x7fffffff) break;
      // the next row of this slot, if any (rare: its search costs a pass over the slots)
      const int from = next;
      __syncthreads();
      if (tid == 0) next = 0x7fffffff;
      __syncthreads();
      row = from;
      for (long long i = row + 1 + tid; i < p.tokens; i += kThreads)
        if (slots[i] == slot) atomicMin(&next, (int)i);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = rg + RG * i;
      if (live && r < p.dk) *reinterpret_cast<float4*>(S + (size_t)r * p.dv + col) = s[i];
    }
  }
}

template <bool BF16IN, int W>
void go(const SeqProblem& p, const void* q, const void* k, const void* v, const float* g, const float* beta, float* state,
        const int* slots, void* out, hipStream_t stream) {
  const int x = (p.dv + W - 1) / W * p.hv;
  long long y = kMaxBlocks / x;
  y = y < 1 ? 1 : y > 65535 ? 65535 : y;
  if (y > p.tokens) y = p.tokens;
  hipLaunchKernelGGL((decode_kernel<BF16IN, W>), dim3(x, (unsigned)y), dim3(kThreads), 0, stream, q, k, v, g, beta, state,
                     slots, out, p);
}

}  // namespace

hipError_t decode_launch(const SeqProblem& p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, float* state, const int* slots, void* out, hipStream_t stream) {
  prof_begin(stream, GDN_KERNEL_DECODE);
  // 64 columns a workgroup: 440 rows x 32 heads x 128^2 407 us (4.55 TB/s; a copy of its size reaches 4.7), against 449 at 32
  // (128-byte pieces of the rows), 417 at 128 (a register more for every row held) and 650 at 16; 48 rows 43.5, 45.8, 45.2 and
  // 69.7.  Narrower values leave less than half of 64 columns' lanes idle at 32.
  auto launch = p.in_bf16 ? (p.dv > 32 ? go<true, 64> : go<true, 32>) : (p.dv > 32 ? go<false, 64> : go<false, 32>);
  launch(p, q, k, v, g, beta, state, slots, out, stream);
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_DECODE);
  return e;
}

}  // namespace gdn
