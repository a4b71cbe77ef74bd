// Rotary positions of queries and keys, and their gradients (the same turns with
// the other sign).
//
// Pair (x, y) at the angle a = p f:  (x cos a - y sin a, x sin a + y cos a) m.
// An angle is shared by all heads of a token, so a workgroup forms the factors of
// its tokens' angles once, in LDS, and turns every head of q and k by them: each
// value is read once and written once, bound by HBM.  106480 tokens of 40 heads of
// 112, bf16: 350 to 414 us, 4.6 to 5.4 TB/s (a copy of that size reaches 5.1);
// 16384 of 48 heads of 128: 85 to 92; 48 tokens: 4.6, one workgroup's latency.
//
// Angles.  p f is formed and reduced to a quarter turn in fp64 with the products'
// rounding errors carried along (a far position times a frequency near 1 has no
// digits left in fp32, and at 2^31 only 22 in fp64); its sine and cosine are
// the Taylor polynomials of degree 9 and 10 on [-pi/4, pi/4], whose first terms
// left out are below 2e-9.
#include "gdn_common.h"
#include "gdn_linear.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// (cos a, sin a) of the angle p f.
__device__ __forceinline__ float2 turn_of(int p, double f) {
#pragma clang fp contract(off)     // the rounding errors are of the products as written
  constexpr double kTurn = 0.15915494309189535, kRest = -9.839338337591243e-18;   // 1 / (2 pi) and what its rounding leaves out
  const double F = f * kTurn, rest = fma(f, kTurn, -F) + f * kRest;
  const double t = p * F, e = fma((double)p, F, -t) + p * rest;          // turns, and what their rounding leaves out
  const double u = 4.0 * ((t - floor(t)) + e), k = rint(u);              // quarter turns in [0, 4]
  const float a = (float)((u - k) * 1.57079632679489661923), z = a * a;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);                      // 1/9!, -1/7!
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(a * z, s, a);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);                      // -1/10!, 1/8!
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const int n = (int)k;
  const float x = n & 1 ? s : c, y = n & 1 ? c : s;
  return make_float2(n == 1 || n == 2 ? -x : x, n == 2 || n == 3 ? -y : y);
}

template <bool BF16>
struct Vec {                                   // 16 bytes of values
  static constexpr int N = BF16 ? 8 : 4;
  float x[N];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (16 / N));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        x[j] = __uint_as_float(w[j]);
      }
    }
  }
  __device__ __forceinline__ void store(void* p, size_t i) const {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) w[j] = f32_to_bf16_bits(x[2 * j]) | (uint32_t)f32_to_bf16_bits(x[2 * j + 1]) << 16;
      else w[j] = __float_as_uint(x[j]);
    }
    *reinterpret_cast<uint4*>(static_cast<char*>(p) + i * (16 / N)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// LAYOUT 0: halves with whole vectors of pairs (pairs a multiple of 16 bytes' values); 1: neighbours; 2: halves, pair by pair (16384
// tokens of 48 heads of 128, bf16: 120 components turned 234 us, 128 in LAYOUT 0 78; fp32, 126 turned 242, 120 in LAYOUT 0 162).
template <bool BF16, int LAYOUT, int TT>
__global__ __launch_bounds__(kThreads) void rotary_kernel(
    const void* q, const void* k, const int* __restrict__ positions, const double* __restrict__ frequencies, void* qo,
    void* ko, RotaryProblem p) {
  constexpr int N = Vec<BF16>::N;
  extern __shared__ float2 turns[];            // [token][pair]: the factors of x and y
  const int tid = threadIdx.x;
  // work items of a head: turned vectors first (halves: two vectors an item), then those that are copied
  const int turned = LAYOUT == 0 ? p.pairs / N : LAYOUT == 1 ? (2 * p.pairs + N - 1) / N : p.pairs;
  const int rest = LAYOUT == 2 ? p.width - 2 * p.pairs : (p.width - (LAYOUT == 0 ? 2 * p.pairs : turned * N)) / N;
  const int items = turned + (qo == q && (ko == k || p.hk == 0) ? 0 : rest);
  const int heads = p.hq + p.hk;
  for (long long first = (long long)blockIdx.x * TT; first < p.tokens; first += (long long)gridDim.x * TT) {
    __syncthreads();                           // the previous tokens' factors have been read
    const int n = (int)min((long long)TT, p.tokens - first);
    for (int i = tid; i < n * p.pairs; i += kThreads) {
      const int t = i / p.pairs, pair = i - t * p.pairs;
      int axis = 0;
#pragma unroll
      for (int a = 0; a < 3; ++a) axis += a + 1 < p.axes && pair >= p.ends[a];
      const float2 w = turn_of(positions[(size_t)(first + t) * p.axes + axis], frequencies[pair]);
      turns[i] = make_float2(w.x * p.cos_factor, w.y * p.sin_factor);
    }
    __syncthreads();
    for (int i = tid; i < n * heads * items; i += kThreads) {
      const int row = i / items, item = i - row * items;
      const int t = row / heads, h = row - t * heads;
      const bool key = h >= p.hq;
      const void* in = key ? k : q;
      void* out = key ? ko : qo;
      const size_t hw = (size_t)(key ? h - p.hq : h) * p.width;
      const size_t from = (size_t)(first + t) * (key ? p.ks : p.qs) + hw, to = (size_t)(first + t) * (key ? p.kos : p.qos) + hw;
      const float2* w = turns + t * p.pairs;
      if constexpr (LAYOUT == 2) {
        if (item < turned) {
          const float x = load_scalar<BF16>(in, from + item), y = load_scalar<BF16>(in, from + item + p.pairs);
          const float2 c = w[item];
          store_scalar(out, to + item, x * c.x - y * c.y, BF16);
          store_scalar(out, to + item + p.pairs, x * c.y + y * c.x, BF16);
        } else {
          const size_t j = 2 * p.pairs + item - turned;
          if constexpr (BF16) static_cast<uint16_t*>(out)[to + j] = static_cast<const uint16_t*>(in)[from + j];
          else static_cast<float*>(out)[to + j] = static_cast<const float*>(in)[from + j];
        }
      } else if (item >= turned) {
        const size_t j = (LAYOUT == 0 ? 2 * p.pairs : turned * N) + (size_t)(item - turned) * N;
        *reinterpret_cast<uint4*>(static_cast<char*>(out) + (to + j) * (16 / N)) =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(in) + (from + j) * (16 / N));
      } else if constexpr (LAYOUT == 0) {
        Vec<BF16> x, y, u, v;
        x.load(in, from + item * N);
        y.load(in, from + p.pairs + item * N);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float2 c = w[item * N + j];
          u.x[j] = x.x[j] * c.x - y.x[j] * c.y;
          v.x[j] = x.x[j] * c.y + y.x[j] * c.x;
        }
        u.store(out, to + item * N);
        v.store(out, to + p.pairs + item * N);
      } else {
        Vec<BF16> x, u;
        x.load(in, from + item * N);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const int pair = item * (N / 2) + j;
          if (pair < p.pairs) {
            const float2 c = w[pair];
            u.x[2 * j] = x.x[2 * j] * c.x - x.x[2 * j + 1] * c.y;
            u.x[2 * j + 1] = x.x[2 * j] * c.y + x.x[2 * j + 1] * c.x;
          } else {
            u.x[2 * j] = x.x[2 * j];
            u.x[2 * j + 1] = x.x[2 * j + 1];
          }
        }
        u.store(out, to + item * N);
      }
    }
  }
}

template <bool BF16, int LAYOUT>
void go(const RotaryProblem& p, const void* q, const void* k, const int* positions, const double* frequencies, void* qo,
        void* ko, hipStream_t stream) {
  const auto launch = [&](auto kernel, int tt) {
    const long long blocks = (p.tokens + tt - 1) / tt;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(kThreads),
                       (size_t)tt * p.pairs * sizeof(float2), stream, q, k, positions, frequencies, qo, ko, p);
  };
  // Four tokens a workgroup where there are enough of them to fill the card, so that a wavefront has several angles and more
  // loads in flight: 106480 tokens of 40 heads of 112 414 us at one, 381 at two, 371 at four, 385 at eight; 8192 of 10 heads of 64
  // 14.6, 12.6, 9.8, 9.8; 4096 of 48 heads of 128 20.6, 20.4, 20.7, 23.3; but 2048 14.5, 13.1, 15.0, 19.9 and 48 6.3, 8.0, 10.2, 16.0.
  // Four tokens of narrow rows leave most lanes idle: a million of 2 heads of 16 255 us, 0.5 TB/s; 250000 of 3 heads of 64 80, 2.4.
  if (p.tokens >= 4096) launch(rotary_kernel<BF16, LAYOUT, 4>, 4);
  else launch(rotary_kernel<BF16, LAYOUT, 1>, 1);
}

}  // namespace

hipError_t rotary_launch(const RotaryProblem& p, const void* q, const void* k, const int* positions, const double* frequencies,
                         void* q_out, void* k_out, hipStream_t stream) {
  prof_begin(stream, GDN_KERNEL_ROTARY);
  const int layout = p.interleaved ? 1 : p.pairs % (p.bf16 ? 8 : 4) == 0 ? 0 : 2;
  auto launch = p.bf16 ? (layout == 0 ? go<true, 0> : layout == 1 ? go<true, 1> : go<true, 2>)
                       : (layout == 0 ? go<false, 0> : layout == 1 ? go<false, 1> : go<false, 2>);
  launch(p, q, k, positions, frequencies, q_out, k_out, stream);
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_ROTARY);
  return e;
}

}  // namespace gdn
