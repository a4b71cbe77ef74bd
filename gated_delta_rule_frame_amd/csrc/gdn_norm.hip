// Group norm with an activation or an activated gate, channels last, and its
// gradients.
//
// For x [N, S, C] with C split into G groups of cg = C / G channels, every
// (n, group) has one mean and one deviation over its S cg values:
//     h = (x - mean) rstd,  u = weight h + bias,  y = act(u)  or  u act(gate)
// and, with du the gradient of u and dh = weight du,
//     dx = rstd (dh - mean(dh) - h mean(dh h)),  dweight = sum du h,  dbias = sum du
// (without centring: mean = 0, no mean(dh) term).  All of it is a few flops
// per element, so HBM bounds it: the floor is each tensor read or written once.
//
// Two ways, by S:
//   S = 1 (the norm of each token's heads): a group is cg neighbouring values.
//     L lanes (a power of two, or a whole workgroup) keep a group in registers,
//     so everything is read once; a workgroup stays on its channels and walks
//     over the rows, so weights stay in registers and the sums of dweight and
//     dbias over its rows need no exchange.
//   S > 1: the S x C values of one n are contiguous and a group is a column
//     band of them.  A first kernel walks over the rows with one thread per
//     channel vector and leaves sums for each (n, part, channel vector or
//     channel); a small kernel joins them; a last one reads the inputs again and
//     writes the result.
// Sums are fp32: a group's second moment is taken about its mean (S = 1) or
// about each thread's first value and joined pairwise with counts, so a mean
// far from zero does not cancel.  No atomics: results are the same every run.
#include "gdn_common.h"
#include "gdn_norm.h"

namespace gdn {
namespace {

constexpr int kT = 256;       // threads of the S = 1 kernels
constexpr int kTF = 512;      // most threads of the S > 1 kernels

template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void* p, size_t i, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = load_scalar<BF16>(p, i);
  } else if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  } else {
    const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(void* p, size_t i, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    store_scalar(p, i, x[0], BF16);
  } else if constexpr (BF16) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x[2 * j], x[2 * j + 1]}, b2));   // round to nearest even
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(a[0], a[1], a[2], a[3]);
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// 1 / (1 + e^-u) with the hardware's 2^x and 1 / x (1 ulp each): with expf and an
// IEEE division the vector units, not memory, bounded the kernels (a 121 x 880 x
// 2240 bf16 frame norm with SiLU: 360 us for the pass that writes, 2.7 TB/s).
// The product -u log2(e) keeps its rounding error as a first-order factor, so
// the exponent's size costs no accuracy; above 2^126 the result is 0.
__device__ __forceinline__ float sigmoid(float u) {
  const float t = fminf(-1.44269504f * u, 126.f);
  const float lo = fmaf(-1.44269504f, u, -t) - 1.92596299e-8f * u;      // log2(e) = 1.44269504 + 1.926e-8
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_amdgcn_rcpf(1.f + fmaf(e, t < 126.f ? 0.69314718f * lo : 0.f, e));
}

__device__ __forceinline__ float act(int a, float u) {
  switch (a) {
    case GDN_ACT_SILU: return u * sigmoid(u);
    case GDN_ACT_GELU: return 0.5f * u * (1.f + erff(u * 0.70710678f));
    case GDN_ACT_RELU: return u < 0.f ? 0.f : u;
    default: return u;
  }
}

// Value and slope of the activation.
__device__ __forceinline__ float2 act_slope(int a, float u) {
  switch (a) {
    case GDN_ACT_SILU: {
      const float s = sigmoid(u);
      return make_float2(u * s, s * (1.f + u * (1.f - s)));
    }
    case GDN_ACT_GELU: {
      const float c = 0.5f * (1.f + erff(u * 0.70710678f));
      return make_float2(u * c, c + u * 0.39894228f * expf(-0.5f * u * u));
    }
    case GDN_ACT_RELU: return make_float2(u < 0.f ? 0.f : u, u > 0.f ? 1.f : 0.f);
    default: return make_float2(u, 1.f);
  }
}

// Gradient of u (returned) and of the gate (dz) from that of y.
template <bool GATE>
__device__ __forceinline__ float grad_u(int a, float dy, float u, float z, float* dz) {
  const float2 f = act_slope(a, GATE ? z : u);
  if constexpr (GATE) {
    *dz = dy * u * f.y;
    return dy * f.x;
  }
  return dy * f.y;
}

// Sum over the L lanes of a group; L a power of two up to 64, or kT.
__device__ __forceinline__ float lane_sum(float x, int L, float* lds) {
  for (int m = L < 64 ? L >> 1 : 32; m; m >>= 1) x += __shfl_xor(x, m);
  if (L > 64) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
    __syncthreads();
    x = lds[0] + lds[1] + lds[2] + lds[3];
  }
  return x;
}

// ---------------------------------------------------------------- S = 1

template <bool BF16, int VEC, int NV, bool GATE>
__global__ __launch_bounds__(kT) void norm_rows_kernel(
    const void* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const void* __restrict__ gate, void* __restrict__ out, float* __restrict__ mean, float* __restrict__ rstd,
    NormProblem p, int L) {
  __shared__ float lds[4];
  const int per = kT / L, lane = threadIdx.x % L;
  const int grp = blockIdx.x * per + threadIdx.x / L;
  const int cvs = p.cg / VEC;
  const bool on = grp < p.G;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int cv = lane + L * j;
      const bool in = on && cv < cvs;
      const int c = grp * p.cg + cv * VEC + e;
      w[j][e] = in && weight ? weight[c] : 1.f;
      b[j][e] = in && bias ? bias[c] : 0.f;
    }
  const float inv = 1.f / (float)p.cg;
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    float v[NV][VEC], s = 0.f;
    const size_t base = (size_t)n * p.C + (size_t)grp * p.cg;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (on && cv < cvs) {
        load_vec<BF16, VEC>(x, base + (size_t)cv * VEC, v[j]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += v[j][e];
      }
    }
    float m = 0.f;
    if (p.center) m = lane_sum(s, L, lds) * inv;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on && lane + L * j < cvs)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(v[j][e] - m, v[j][e] - m, s);
    const float r = 1.f / sqrtf(lane_sum(s, L, lds) * inv + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      float z[VEC];
      if constexpr (GATE) load_vec<BF16, VEC>(gate, base + (size_t)cv * VEC, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = fmaf((v[j][e] - m) * r, w[j][e], b[j][e]);
        v[j][e] = GATE ? u * act(p.act, z[e]) : act(p.act, u);
      }
      store_vec<BF16, VEC>(out, base + (size_t)cv * VEC, v[j]);
    }
    if (on && lane == 0) {
      if (mean) mean[(size_t)n * p.G + grp] = m;
      rstd[(size_t)n * p.G + grp] = r;
    }
  }
}

// dx, dgate, and for each workgroup row block the sums of du h and du per channel:
// part [gridDim.y][2][C].
template <bool BF16, int VEC, int NV, bool GATE>
__global__ __launch_bounds__(kT) void norm_rows_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ bias, const void* __restrict__ gate, const float* __restrict__ mean,
    const float* __restrict__ rstd, void* __restrict__ dx, void* __restrict__ dgate, float* __restrict__ part,
    NormProblem p, int L) {
  __shared__ float lds[4];
  const int per = kT / L, lane = threadIdx.x % L;
  const int grp = blockIdx.x * per + threadIdx.x / L;
  const int cvs = p.cg / VEC;
  const bool on = grp < p.G;
  float w[NV][VEC], b[NV][VEC], sw[NV][VEC], sb[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int cv = lane + L * j;
      const bool in = on && cv < cvs;
      const int c = grp * p.cg + cv * VEC + e;
      w[j][e] = in && weight ? weight[c] : 1.f;
      b[j][e] = in && bias ? bias[c] : 0.f;
      sw[j][e] = sb[j][e] = 0.f;
    }
  const float inv = 1.f / (float)p.cg;
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    const size_t base = (size_t)n * p.C + (size_t)grp * p.cg;
    const float m = on && p.center ? mean[(size_t)n * p.G + grp] : 0.f;
    const float r = on ? rstd[(size_t)n * p.G + grp] : 0.f;
    float h[NV][VEC], d[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      float z[VEC], dz[VEC];
      load_vec<BF16, VEC>(x, base + (size_t)cv * VEC, h[j]);
      load_vec<BF16, VEC>(dout, base + (size_t)cv * VEC, d[j]);
      if constexpr (GATE) load_vec<BF16, VEC>(gate, base + (size_t)cv * VEC, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[j][e] = (h[j][e] - m) * r;
        const float du = grad_u<GATE>(p.act, d[j][e], fmaf(h[j][e], w[j][e], b[j][e]), GATE ? z[e] : 0.f, &dz[e]);
        sw[j][e] = fmaf(du, h[j][e], sw[j][e]);
        sb[j][e] += du;
        d[j][e] = du * w[j][e];
        s1 += d[j][e];
        s2 = fmaf(d[j][e], h[j][e], s2);
      }
      if constexpr (GATE) store_vec<BF16, VEC>(dgate, base + (size_t)cv * VEC, dz);
    }
    s1 = p.center ? lane_sum(s1, L, lds) * inv : 0.f;
    s2 = lane_sum(s2, L, lds) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[j][e] = r * (d[j][e] - s1 - h[j][e] * s2);
      store_vec<BF16, VEC>(dx, base + (size_t)cv * VEC, d[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      float* o = part + (size_t)blockIdx.y * 2 * p.C + grp * p.cg + cv * VEC + e;
      o[0] = sw[j][e];
      o[p.C] = sb[j][e];
    }
}

// ---------------------------------------------------------------- S > 1

// The place of a thread of the S > 1 kernels: one channel vector, every
// rpb-th row of the part's rows.
struct Place {
  int cv, first, last, step, part;
  bool on;
};

__device__ __forceinline__ Place place(const NormProblem& p, const NormPlan& f) {
  Place t;
  const int tid = threadIdx.x, off = tid / f.tile;
  t.cv = blockIdx.x * f.tile + tid % f.tile;
  t.on = off < f.rpb && t.cv < f.cvs;
  t.first = blockIdx.y * f.rows + off;
  t.last = min((blockIdx.y + 1) * f.rows, p.S);
  t.step = f.rpb;
  t.part = blockIdx.y * f.rpb + off;
  return t;
}

// Sum and second moment about the mean of each thread's values:
// part [N][parts][cvs] pairs.
template <bool BF16, int VEC>
__global__ __launch_bounds__(kTF) void norm_stats_kernel(const void* __restrict__ x, float2* __restrict__ part, NormProblem p,
                                                         NormPlan f) {
  const Place t = place(p, f);
  if (!t.on) return;
  for (long long n = blockIdx.z; n < p.N; n += gridDim.z) {
    const size_t base = (size_t)n * p.S * p.C + (size_t)t.cv * VEC;
    float s = 0.f, s2 = 0.f, shift = 0.f;
    int rows = 0;
    float v[VEC];
    if (t.first < t.last && p.center) {
      load_vec<BF16, VEC>(x, base + (size_t)t.first * p.C, v);
      shift = v[0];
    }
#pragma unroll 4
    for (int i = t.first; i < t.last; i += t.step, ++rows) {
      load_vec<BF16, VEC>(x, base + (size_t)i * p.C, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = v[e] - shift;
        s += d;
        s2 = fmaf(d, d, s2);
      }
    }
    float2 r = make_float2(0.f, s2);
    if (p.center && rows) {
      const float d = s / (float)(rows * VEC);
      const float about = s2 - s * d;
      r = make_float2(shift + d, about < 0.f ? 0.f : about);   // NaN stays NaN
    }
    part[((size_t)n * f.parts + t.part) * f.cvs + t.cv] = r;
  }
}

// Joins two sets of values given as (count, mean, second moment about it).
__device__ __forceinline__ void join(float& n, float& m, float& q, float n2, float m2, float q2) {
  const float t = n + n2;
  if (n2 == 0.f) return;
  if (n == 0.f) { n = n2; m = m2; q = q2; return; }
  const float d = m2 - m, w = n2 / t;
  m = fmaf(d, w, m);
  q += q2 + d * d * n * w;
  n = t;
}

// One wavefront per (n, group): joins the threads' sums into mean and 1 / deviation.
__global__ __launch_bounds__(64) void norm_stats_join_kernel(const float2* __restrict__ part, float* __restrict__ mean,
                                                             float* __restrict__ rstd, NormProblem p, NormPlan f, int vec) {
  const int per = f.cvs / p.G, grp = blockIdx.x;
  const long long items = (long long)f.parts * per;
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    float c = 0.f, m = 0.f, q = 0.f;
    for (long long i = threadIdx.x; i < items; i += 64) {
      const int k = (int)(i / per), split = k / f.rpb;
      const int first = split * f.rows + k % f.rpb, last = min((split + 1) * f.rows, p.S);
      const float cnt = first < last ? (float)(((last - first + f.rpb - 1) / f.rpb) * vec) : 0.f;
      const float2 a = part[((size_t)n * f.parts + k) * f.cvs + (size_t)grp * per + i % per];
      if (p.center) join(c, m, q, cnt, a.x, a.y);
      else q += a.y;
    }
    for (int s = 32; s; s >>= 1) {
      const float c2 = __shfl_down(c, s), m2 = __shfl_down(m, s), q2 = __shfl_down(q, s);
      if (p.center) join(c, m, q, c2, m2, q2);
      else q += q2;
    }
    if (threadIdx.x == 0) {
      if (mean) mean[(size_t)n * p.G + grp] = m;
      rstd[(size_t)n * p.G + grp] = 1.f / sqrtf(q / ((float)p.S * (float)p.cg) + p.eps);
    }
  }
}

template <bool BF16, int VEC, bool GATE>
__global__ __launch_bounds__(kTF) void norm_apply_kernel(const void* __restrict__ x, const float* __restrict__ weight,
                                                         const float* __restrict__ bias, const void* __restrict__ gate,
                                                         void* __restrict__ out, const float* __restrict__ mean,
                                                         const float* __restrict__ rstd, NormProblem p, NormPlan f) {
  const Place t = place(p, f);
  if (!t.on) return;
  float w[VEC], b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    w[e] = weight ? weight[t.cv * VEC + e] : 1.f;
    b[e] = bias ? bias[t.cv * VEC + e] : 0.f;
  }
  const int grp = t.cv * VEC / p.cg;
  // from the last n to the first: the pass before went upwards, and its last rows are still in the cache
  for (long long n = p.N - 1 - blockIdx.z; n >= 0; n -= gridDim.z) {
    const size_t base = (size_t)n * p.S * p.C + (size_t)t.cv * VEC;
    const float m = p.center ? mean[(size_t)n * p.G + grp] : 0.f, r = rstd[(size_t)n * p.G + grp];
#pragma unroll 4
    for (int i = t.first; i < t.last; i += t.step) {
      float v[VEC], z[VEC];
      load_vec<BF16, VEC>(x, base + (size_t)i * p.C, v);
      if constexpr (GATE) load_vec<BF16, VEC>(gate, base + (size_t)i * p.C, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = fmaf((v[e] - m) * r, w[e], b[e]);
        v[e] = GATE ? u * act(p.act, z[e]) : act(p.act, u);
      }
      store_vec<BF16, VEC>(out, base + (size_t)i * p.C, v);
    }
  }
}

// FINAL false: dgate, and sums over each thread's rows of du h and du per
// channel, part [N][parts][2][C].  FINAL true: dx, with the group's sums of
// dh and dh h in sums [N][G].
template <bool BF16, int VEC, bool GATE, bool FINAL>
__global__ __launch_bounds__(kTF) void norm_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ bias, const void* __restrict__ gate, const float* __restrict__ mean,
    const float* __restrict__ rstd, void* __restrict__ dx, void* __restrict__ dgate, float* __restrict__ part,
    const float2* __restrict__ sums, NormProblem p, NormPlan f) {
  const Place t = place(p, f);
  if (!t.on) return;
  float w[VEC], b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    w[e] = weight ? weight[t.cv * VEC + e] : 1.f;
    b[e] = bias ? bias[t.cv * VEC + e] : 0.f;
  }
  const int grp = t.cv * VEC / p.cg;
  const float inv = 1.f / ((float)p.S * (float)p.cg);
  for (long long z = blockIdx.z; z < p.N; z += gridDim.z) {
    const long long n = FINAL ? p.N - 1 - z : z;   // the second pass backwards, as in norm_apply_kernel
    const size_t base = (size_t)n * p.S * p.C + (size_t)t.cv * VEC;
    const float m = p.center ? mean[(size_t)n * p.G + grp] : 0.f, r = rstd[(size_t)n * p.G + grp];
    float sw[VEC] = {}, sb[VEC] = {};
    float s1 = 0.f, s2 = 0.f;
    if constexpr (FINAL) {
      const float2 s = sums[(size_t)n * p.G + grp];
      s1 = p.center ? s.x * inv : 0.f;
      s2 = s.y * inv;
    }
#pragma unroll 4
    for (int i = t.first; i < t.last; i += t.step) {
      float v[VEC], d[VEC], z[VEC], dz[VEC];
      load_vec<BF16, VEC>(x, base + (size_t)i * p.C, v);
      load_vec<BF16, VEC>(dout, base + (size_t)i * p.C, d);
      if constexpr (GATE) load_vec<BF16, VEC>(gate, base + (size_t)i * p.C, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float h = (v[e] - m) * r;
        const float du = grad_u<GATE>(p.act, d[e], fmaf(h, w[e], b[e]), GATE ? z[e] : 0.f, &dz[e]);
        if constexpr (FINAL) {
          v[e] = r * (du * w[e] - s1 - h * s2);
        } else {
          sw[e] = fmaf(du, h, sw[e]);
          sb[e] += du;
        }
      }
      if constexpr (FINAL) store_vec<BF16, VEC>(dx, base + (size_t)i * p.C, v);
      else if constexpr (GATE) store_vec<BF16, VEC>(dgate, base + (size_t)i * p.C, dz);
    }
    if constexpr (!FINAL) {
      float* o = part + ((size_t)n * f.parts + t.part) * 2 * p.C + (size_t)t.cv * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        o[e] = sw[e];
        o[p.C + e] = sb[e];
      }
    }
  }
}

// One workgroup per (n, group): sums of dh = weight du and of dh h.
__global__ __launch_bounds__(256) void norm_grad_join_kernel(const float* __restrict__ part, const float* __restrict__ weight,
                                                             float2* __restrict__ sums, NormProblem p, NormPlan f) {
  __shared__ float lds[2][4];
  const int grp = blockIdx.x;
  // a thread stays on one channel and walks over the parts
  const int wide = p.cg < 256 ? p.cg : 256, rows = 256 / wide;
  const int c0 = threadIdx.x % wide, r0 = threadIdx.x / wide;
  for (long long n = blockIdx.y; n < p.N; n += gridDim.y) {
    float s1 = 0.f, s2 = 0.f;
    if (r0 < rows)
      for (int c = c0; c < p.cg; c += wide) {
        const float w = weight ? weight[grp * p.cg + c] : 1.f;
        const float* o = part + (size_t)n * f.parts * 2 * p.C + grp * p.cg + c;
        float a = 0.f, b = 0.f;
#pragma unroll 8
        for (int k = r0; k < f.parts; k += rows) {
          a += o[(size_t)k * 2 * p.C + p.C];
          b += o[(size_t)k * 2 * p.C];
        }
        s1 = fmaf(w, a, s1);
        s2 = fmaf(w, b, s2);
      }
    for (int s = 32; s; s >>= 1) {
      s1 += __shfl_xor(s1, s);
      s2 += __shfl_xor(s2, s);
    }
    __syncthreads();
    if (threadIdx.x % 64 == 0) {
      lds[0][threadIdx.x / 64] = s1;
      lds[1][threadIdx.x / 64] = s2;
    }
    __syncthreads();
    if (threadIdx.x == 0)
      sums[(size_t)n * p.G + grp] = make_float2(lds[0][0] + lds[0][1] + lds[0][2] + lds[0][3],
                                                lds[1][0] + lds[1][1] + lds[1][2] + lds[1][3]);
  }
}

// Sums of part [rows][2][C] over the rows: 16 channels of one of the two per workgroup.
__global__ __launch_bounds__(256) void norm_weight_grad_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                               float* __restrict__ dbias, long long rows, int C) {
  __shared__ float lds[16][17];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int c = blockIdx.x * 16 + threadIdx.x % 16, rg = threadIdx.x / 16;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (long long r = rg; r < rows; r += 16) s += part[(r * 2 + blockIdx.y) * C + c];
  }
  lds[rg][threadIdx.x % 16] = s;
  __syncthreads();
  if (rg == 0 && c < C) {
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += lds[i][threadIdx.x];
    out[c] = t;
  }
}

// ---------------------------------------------------------------- host

int vec_of(const NormProblem& p) {
  const int v = p.bf16 ? 8 : 4;
  return p.cg % v == 0 ? v : 1;
}

// Lanes of a group on the S = 1 way and vectors per lane (0: the group is too
// wide for the registers of one workgroup).
void rows_shape(const NormProblem& p, int* L, int* NV) {
  const int cvs = p.cg / vec_of(p);
  int l = 1;
  while (l < 64 && l < cvs) l *= 2;
  if (cvs > 64) l = kT;
  const int need = (cvs + l - 1) / l;
  *L = l;
  *NV = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 0;
}

bool by_rows(const NormProblem& p) {
  int L, NV;
  rows_shape(p, &L, &NV);
  return p.S == 1 && NV > 0;
}

dim3 rows_grid(const NormProblem& p, int L, bool gradient) {
  const int per = kT / L, x = (p.G + per - 1) / per;
  // the gradient leaves one row of sums per workgroup row: a few rounds over the 256 CUs; the forward
  // kernel only amortises its weights
  long long y = ((gradient ? 2048 : 8192) + x - 1) / x;
  y = y < 1 ? 1 : y > 65535 ? 65535 : y;
  if (y > p.N) y = p.N;
  return dim3(x, (unsigned)y);
}

NormPlan plan(const NormProblem& p) {
  NormPlan f;
  f.cvs = p.C / vec_of(p);
  const int tiles = (f.cvs + kTF - 1) / kTF;
  f.tile = (f.cvs + tiles - 1) / tiles;
  f.tiles = tiles;
  f.rpb = kTF / f.tile;
  if (f.rpb > p.S) f.rpb = p.S;
  // parts of the rows: about 2048 workgroups in all, at least 8 rows a thread
  long long want = 2048 / ((long long)tiles * (p.N < 2048 ? p.N : 2048));
  long long most = p.S / (8LL * f.rpb);
  long long splits = want < most ? want : most;
  if (splits < 1) splits = 1;
  if (splits > 4096) splits = 4096;
  f.rows = (int)((p.S + splits - 1) / splits);
  f.splits = (p.S + f.rows - 1) / f.rows;
  f.parts = f.splits * f.rpb;
  f.threads = (f.tile * f.rpb + 63) / 64 * 64;
  return f;
}

int loop_dim(long long n, long long others) {
  long long y = kMaxBlocks / 4 / others;   // up to 512 threads a workgroup
  y = y < 1 ? 1 : y > 65535 ? 65535 : y;
  return (int)(n < y ? n : y);
}

template <bool BF16, int VEC, bool GATE>
hipError_t forward_v(const NormProblem& p, const void* x, const float* weight, const float* bias, const void* gate, void* out,
                     float* mean, float* rstd, void* ws, hipStream_t st) {
  if (by_rows(p)) {
    int L, NV;
    rows_shape(p, &L, &NV);
    const dim3 grid = rows_grid(p, L, false);
#define GDN_ROWS(V)                                                                                                      \
  case V:                                                                                                                \
    hipLaunchKernelGGL((norm_rows_kernel<BF16, VEC, V, GATE>), grid, dim3(kT), 0, st, x, weight, bias, gate, out, mean, \
                       rstd, p, L);                                                                                      \
    break;
    switch (NV) { GDN_ROWS(1) GDN_ROWS(2) GDN_ROWS(4) GDN_ROWS(8) }
#undef GDN_ROWS
    return hipGetLastError();
  }
  const NormPlan f = plan(p);
  float2* part = static_cast<float2*>(ws);
  const long long xy = (long long)f.tiles * f.splits;
  const dim3 grid(f.tiles, f.splits, loop_dim(p.N, xy)), small(p.G, loop_dim(p.N, p.G));
  hipLaunchKernelGGL((norm_stats_kernel<BF16, VEC>), grid, dim3(f.threads), 0, st, x, part, p, f);
  hipLaunchKernelGGL(norm_stats_join_kernel, small, dim3(64), 0, st, part, mean, rstd, p, f, VEC);
  hipLaunchKernelGGL((norm_apply_kernel<BF16, VEC, GATE>), grid, dim3(f.threads), 0, st, x, weight, bias, gate, out, mean, rstd,
                     p, f);
  return hipGetLastError();
}

template <bool BF16, int VEC, bool GATE>
hipError_t backward_v(const NormProblem& p, const NormGrad& t, void* ws, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  long long rows = 0;
  if (p.N > 0 && by_rows(p)) {
    int L, NV;
    rows_shape(p, &L, &NV);
    const dim3 grid = rows_grid(p, L, true);
    rows = grid.y;
#define GDN_ROWS(V)                                                                                                       \
  case V:                                                                                                                 \
    hipLaunchKernelGGL((norm_rows_grad_kernel<BF16, VEC, V, GATE>), grid, dim3(kT), 0, st, t.dout, t.x, t.weight, t.bias, \
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, p, L);                                                \
    break;
    switch (NV) { GDN_ROWS(1) GDN_ROWS(2) GDN_ROWS(4) GDN_ROWS(8) }
#undef GDN_ROWS
  } else if (p.N > 0) {
    const NormPlan f = plan(p);
    rows = p.N * f.parts;
    float2* sums = reinterpret_cast<float2*>(part + (size_t)rows * 2 * p.C);
    const long long xy = (long long)f.tiles * f.splits;
    const dim3 grid(f.tiles, f.splits, loop_dim(p.N, xy)), small(p.G, loop_dim(p.N, p.G));
    hipLaunchKernelGGL((norm_grad_kernel<BF16, VEC, GATE, false>), grid, dim3(f.threads), 0, st, t.dout, t.x, t.weight, t.bias,
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, sums, p, f);
    hipLaunchKernelGGL(norm_grad_join_kernel, small, dim3(256), 0, st, part, t.weight, sums, p, f);
    hipLaunchKernelGGL((norm_grad_kernel<BF16, VEC, GATE, true>), grid, dim3(f.threads), 0, st, t.dout, t.x, t.weight, t.bias,
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, sums, p, f);
  }
  if (t.dweight || t.dbias)
    hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((p.C + 15) / 16, 2), dim3(256), 0, st, part, t.dweight, t.dbias, rows, p.C);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace(const NormProblem& p, bool gradient) {
  if (p.N == 0) return 0;
  if (by_rows(p)) {
    int L, NV;
    rows_shape(p, &L, &NV);
    return gradient ? (size_t)rows_grid(p, L, true).y * 2 * p.C * sizeof(float) : 0;
  }
  const NormPlan f = plan(p);
  const size_t rows = (size_t)p.N * f.parts;
  return gradient ? (rows * 2 * p.C + (size_t)p.N * p.G * 2) * sizeof(float) : rows * f.cvs * sizeof(float2);
}

hipError_t norm_launch(const NormProblem& p, const void* x, const float* weight, const float* bias, const void* gate, void* out,
                       float* mean, float* rstd, void* ws, hipStream_t st) {
  prof_begin(st, GDN_KERNEL_NORM);
  const bool vec = vec_of(p) > 1;
  auto f = p.bf16 ? (vec ? (gate ? forward_v<true, 8, true> : forward_v<true, 8, false>)
                         : (gate ? forward_v<true, 1, true> : forward_v<true, 1, false>))
                  : (vec ? (gate ? forward_v<false, 4, true> : forward_v<false, 4, false>)
                         : (gate ? forward_v<false, 1, true> : forward_v<false, 1, false>));
  const hipError_t e = f(p, x, weight, bias, gate, out, mean, rstd, ws, st);
  prof_end(st, GDN_KERNEL_NORM);
  return e;
}

hipError_t norm_grad_launch(const NormProblem& p, const NormGrad& t, void* ws, hipStream_t st) {
  prof_begin(st, GDN_KERNEL_NORM_GRAD);
  const bool vec = vec_of(p) > 1;
  auto f = p.bf16 ? (vec ? (t.gate ? backward_v<true, 8, true> : backward_v<true, 8, false>)
                         : (t.gate ? backward_v<true, 1, true> : backward_v<true, 1, false>))
                  : (vec ? (t.gate ? backward_v<false, 4, true> : backward_v<false, 4, false>)
                         : (t.gate ? backward_v<false, 1, true> : backward_v<false, 1, false>));
  const hipError_t e = f(p, t, ws, st);
  prof_end(st, GDN_KERNEL_NORM_GRAD);
  return e;
}

}  // namespace gdn
