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
// Three ways, by the size of a group:
//   S = 1 (the norm of each token's heads): a group is cg neighbouring values.
//     L lanes (a power of two, or a whole workgroup) keep a group in registers,
//     so everything is read once; a workgroup stays on its channels and walks
//     over the rows, so weights stay in registers and the sums of dweight and
//     dbias over its rows need no exchange.
//   S > 1, and the S x cg values (a band of the S x C of one n) fit the registers
//     of at most 512 lanes: the same, with lanes over rows and channels.  One
//     launch, one read (20000 x 4 x 512 bf16 in 32 groups 69 us against 233 the
//     third way, 8 x 64 x 512 in 8: 6.8 against 16, their gradients 96 against 211
//     and 13 against 26).
//   Otherwise a first kernel walks over the rows with one thread per channel
//     vector and leaves each workgroup's sums for its groups; a small kernel
//     joins them; a last one reads the inputs again and writes the result.
// Sums are fp32: a group's second moment is taken about its mean (in registers) or
// about each thread's first value and joined pairwise with counts, so a mean
// far from zero does not cancel.  No atomics: results are the same every run.
#include <cfloat>

#include "gdn_common.h"
#include "gdn_norm.h"

namespace gdn {
namespace {

constexpr int kT = 256;       // threads of the S = 1 kernels
constexpr int kTF = 512;      // most threads of the S > 1 kernels

// A vector as it lies in memory, so that one can be fetched ahead in few registers.
template <bool BF16, int VEC>
struct RawVec {
  uint4 v;
};
template <>
struct RawVec<true, 1> {
  uint16_t v;
};
template <>
struct RawVec<false, 1> {
  float v;
};

template <bool BF16, int VEC>
__device__ __forceinline__ RawVec<BF16, VEC> fetch_vec(const void* p, size_t i) {
  RawVec<BF16, VEC> r;
  r.v = *reinterpret_cast<const decltype(r.v)*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
  return r;
}

template <bool BF16, int VEC>
__device__ __forceinline__ void unpack(const RawVec<BF16, VEC>& r, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (BF16) x[0] = bf16_bits_to_f32(r.v);
    else x[0] = r.v;
  } else {
    const uint32_t a[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        x[2 * j] = __uint_as_float(a[j] << 16);
        x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
      } else {
        x[j] = __uint_as_float(a[j]);
      }
    }
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void* p, size_t i, float (&x)[VEC]) {
  unpack<BF16, VEC>(fetch_vec<BF16, VEC>(p, i), x);
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
// The product -u log2(e) keeps its rounding error as a factor close to 1, so the
// exponent's size costs no accuracy; that factor is made from u held to a range
// where it is finite.  The result is 0 below -89, 1 at the other end and NaN for NaN.
__device__ __forceinline__ float held(float u) { return __builtin_amdgcn_fmed3f(u, -100.f, 100.f); }

__device__ __forceinline__ float sigmoid(float u) {
  const float c = held(u), t = -1.44269504f * c;
  const float lo = fmaf(-1.44269504f, c, -t) - 1.92596299e-8f * c;      // log2(e) = 1.44269504 + 1.926e-8
  const float e = __builtin_amdgcn_exp2f(-1.44269504f * u);
  return __builtin_amdgcn_rcpf(fmaf(e, fmaf(0.69314718f, lo, 1.f), 1.f));
}

// u cut off where the normal distribution's density is 0 and its integral 0 or 1,
// so that 0 times an infinity is not asked for; NaN stays NaN.
__device__ __forceinline__ float gelu_range(float u) {
  const float lo = u < -40.f ? -40.f : u;
  return lo > 40.f ? 40.f : lo;
}

// At -inf value and slope are their limits 0, at +inf inf and 1.
__device__ __forceinline__ float act(int a, float u) {
  switch (a) {
    case GDN_ACT_SILU: return fmaxf(u, -FLT_MAX) * sigmoid(u);    // -inf 0; NaN is in the second factor
    case GDN_ACT_GELU: return 0.5f * (u < -40.f ? -40.f : u) * (1.f + erff(u * 0.70710678f));
    case GDN_ACT_RELU: return u < 0.f ? 0.f : u;
    default: return u;
  }
}

template <int VEC>
__device__ __forceinline__ void act_all(int a, float (&u)[VEC]) {
  switch (a) {
    case GDN_ACT_SILU:
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = act(GDN_ACT_SILU, u[e]);
      break;
    case GDN_ACT_GELU:
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = act(GDN_ACT_GELU, u[e]);
      break;
    case GDN_ACT_RELU:
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = act(GDN_ACT_RELU, u[e]);
      break;
    default: break;
  }
}

// Value and slope of the activation.
__device__ __forceinline__ float2 act_slope(int a, float u) {
  switch (a) {
    case GDN_ACT_SILU: {
      const float s = sigmoid(u);
      return make_float2(fmaxf(u, -FLT_MAX) * s, s * (1.f + held(u) * (1.f - s)));
    }
    case GDN_ACT_GELU: {
      const float c = 0.5f * (1.f + erff(u * 0.70710678f)), r = gelu_range(u);
      return make_float2((u < -40.f ? -40.f : u) * c, c + r * 0.39894228f * expf(-0.5f * r * r));
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

// The same for a vector of them, dy in place.
template <bool GATE, int VEC>
__device__ __forceinline__ void grad_all(int a, float (&dy)[VEC], const float (&u)[VEC], const float (&z)[VEC], float (&dz)[VEC]) {
  const auto each = [&](int act) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) dy[e] = grad_u<GATE>(act, dy[e], u[e], z[e], &dz[e]);
  };
  switch (a) {
    case GDN_ACT_SILU: each(GDN_ACT_SILU); break;
    case GDN_ACT_GELU: each(GDN_ACT_GELU); break;
    case GDN_ACT_RELU: each(GDN_ACT_RELU); break;
    default: each(GDN_ACT_NONE); break;
  }
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

// Where a thread of the S = 1 kernels works: one group, and rows first, first +
// step, ...  A workgroup holds kT / L groups: of one row, or all groups of
// several rows where a row has fewer.
struct RowPlace {
  int grp;
  bool on;
  long long first, step;
};

__device__ __forceinline__ RowPlace row_place(const NormProblem& p, int L) {
  const int slots = kT / L, slot = threadIdx.x / L;
  RowPlace t;
  if (p.G >= slots) {
    t.grp = blockIdx.x * slots + slot;
    t.on = t.grp < p.G;
    t.first = blockIdx.y;
    t.step = gridDim.y;
  } else {
    const int rows = slots / p.G, r = slot / p.G;
    t.grp = slot % p.G;
    t.on = r < rows;
    t.first = t.on ? (long long)blockIdx.y * rows + r : p.N;
    t.step = (long long)gridDim.y * rows;
  }
  return t;
}

template <bool BF16, int VEC, int NV, bool GATE>
__global__ __launch_bounds__(kT) void norm_rows_kernel(
    const void* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const void* __restrict__ gate, void* __restrict__ out, float* __restrict__ mean, float* __restrict__ rstd,
    NormProblem p, int L) {
  __shared__ float lds[4];
  const int lane = threadIdx.x % L;
  const RowPlace t = row_place(p, L);
  const int grp = t.grp, cvs = p.cg / VEC;
  const bool on = t.on;
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
  // the next row's values are fetched before this one's sums
  RawVec<BF16, VEC> rx[NV], rz[GATE ? NV : 1];
  auto fetch = [&](long long n) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      const size_t at = (size_t)n * p.C + (size_t)grp * p.cg + (size_t)cv * VEC;
      rx[j] = fetch_vec<BF16, VEC>(x, at);
      if constexpr (GATE) rz[j] = fetch_vec<BF16, VEC>(gate, at);
    }
  };
  if (t.first < p.N) fetch(t.first);
  for (long long n = t.first; n < p.N; n += t.step) {
    float v[NV][VEC], z[GATE ? NV : 1][VEC], s = 0.f;
    const size_t base = (size_t)n * p.C + (size_t)grp * p.cg;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack<BF16, VEC>(rx[j], v[j]);
      if constexpr (GATE) unpack<BF16, VEC>(rz[j], z[j]);
    }
    if (n + t.step < p.N) fetch(n + t.step);
    if (p.center) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on && lane + L * j < cvs)
#pragma unroll
          for (int e = 0; e < VEC; ++e) s += v[j][e];
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
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = fmaf((v[j][e] - m) * r, w[j][e], b[j][e]);
        v[j][e] = GATE ? u * act(p.act, z[GATE ? j : 0][e]) : act(p.act, u);
      }
      store_vec<BF16, VEC>(out, base + (size_t)cv * VEC, v[j]);
    }
    if (on && lane == 0) {
      if (mean) mean[(size_t)n * p.G + grp] = m;
      rstd[(size_t)n * p.G + grp] = r;
    }
  }
}

// dx, dgate, and for each of the rows walked at once the sums of du h and du per
// channel: part [rows at once][2][C].
template <bool BF16, int VEC, int NV, bool GATE>
__global__ __launch_bounds__(kT) void norm_rows_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ bias, const void* __restrict__ gate, const float* __restrict__ mean,
    const float* __restrict__ rstd, void* __restrict__ dx, void* __restrict__ dgate, float* __restrict__ part,
    NormProblem p, int L) {
  __shared__ float lds[4];
  const int lane = threadIdx.x % L;
  const RowPlace t = row_place(p, L);
  const int grp = t.grp, cvs = p.cg / VEC;
  const bool on = t.on;
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
  // the next row's values are fetched before this one's sums
  RawVec<BF16, VEC> rx[NV], rd[NV], rz[GATE ? NV : 1];
  float nm = 0.f, nr = 0.f;
  auto fetch = [&](long long n) {
    nm = on && p.center ? mean[(size_t)n * p.G + grp] : 0.f;
    nr = on ? rstd[(size_t)n * p.G + grp] : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      const size_t at = (size_t)n * p.C + (size_t)grp * p.cg + (size_t)cv * VEC;
      rx[j] = fetch_vec<BF16, VEC>(x, at);
      rd[j] = fetch_vec<BF16, VEC>(dout, at);
      if constexpr (GATE) rz[j] = fetch_vec<BF16, VEC>(gate, at);
    }
  };
  if (t.first < p.N) fetch(t.first);
  for (long long n = t.first; n < p.N; n += t.step) {
    const size_t base = (size_t)n * p.C + (size_t)grp * p.cg;
    const float m = nm, r = nr;
    float h[NV][VEC], d[NV][VEC], zz[GATE ? NV : 1][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack<BF16, VEC>(rx[j], h[j]);
      unpack<BF16, VEC>(rd[j], d[j]);
      if constexpr (GATE) unpack<BF16, VEC>(rz[j], zz[j]);
    }
    if (n + t.step < p.N) fetch(n + t.step);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int cv = lane + L * j;
      if (!(on && cv < cvs)) continue;
      float dz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[j][e] = (h[j][e] - m) * r;
        const float du =
            grad_u<GATE>(p.act, d[j][e], fmaf(h[j][e], w[j][e], b[j][e]), GATE ? zz[GATE ? j : 0][e] : 0.f, &dz[e]);
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
      float* o = part + (size_t)t.first * 2 * p.C + grp * p.cg + cv * VEC + e;
      o[0] = sw[j][e];
      o[p.C] = sb[j][e];
    }
}

// ---------------------------------------------------------------- S > 1

// The place of a thread of the S > 1 kernels: one channel vector, every rpb-th
// row of the part's rows.  A workgroup has whole groups, or a piece of one.
struct Place {
  int cv, grp, first, last, step, off;
  bool on;
};

__device__ __forceinline__ Place place(const NormProblem& p, const NormPlan& f) {
  Place t;
  const int tid = threadIdx.x, c = tid % f.tile;
  t.off = tid / f.tile;
  if (f.pieces == 1) {
    t.cv = blockIdx.x * f.tile + c;
    t.grp = t.cv / f.per;
    t.on = t.off < f.rpb && t.grp < p.G;
  } else {
    const int in = blockIdx.x % f.pieces * f.tile + c;
    t.grp = blockIdx.x / f.pieces;
    t.cv = t.grp * f.per + in;
    t.on = t.off < f.rpb && in < f.per;
  }
  t.first = blockIdx.y * f.rows + t.off;
  t.last = min((blockIdx.y + 1) * f.rows, p.S);
  t.step = f.rpb;
  return t;
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

// The groups of a workgroup and its threads of one: a wavefront sums each group's
// values, left by thread in LDS.  `each(entry)` adds a thread's, `done(group)`
// is called with the wavefront's lanes' sums.
template <typename Each, typename Done>
__device__ __forceinline__ void by_group(const NormProblem& p, const NormPlan& f, Each each, Done done) {
  const int groups = f.pieces == 1 ? f.tile / f.per : 1, wide = f.pieces == 1 ? f.per : f.tile;
  const int first = f.pieces == 1 ? blockIdx.x * groups : blockIdx.x / f.pieces;
  for (int g = threadIdx.x / 64; g < groups && first + g < p.G; g += blockDim.x / 64) {
    for (int i = threadIdx.x % 64; i < wide * f.rpb; i += 64) each(i / wide * f.tile + g * wide + i % wide);
    done(first + g);
  }
}

// Count, sum and second moment of a workgroup's values of each group:
// part [N][splits * pieces][G].
template <bool BF16, int VEC>
__global__ __launch_bounds__(kTF) void norm_stats_kernel(const void* __restrict__ x, float4* __restrict__ part, NormProblem p,
                                                         NormPlan f) {
  __shared__ float lds[3][kTF];
  const Place t = place(p, f);
  for (long long n = blockIdx.z; n < p.N; n += gridDim.z) {
    const size_t base = (size_t)n * p.S * p.C + (size_t)t.cv * VEC;
    float s = 0.f, s2 = 0.f, shift = 0.f;
    int rows = 0;
    float v[VEC];
    if (t.on && t.first < t.last && p.center) {
      load_vec<BF16, VEC>(x, base + (size_t)t.first * p.C, v);
      shift = v[0];
    }
    if (t.on)
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
    float c = (float)(rows * VEC), m = 0.f, q = s2;
    if (p.center && rows) {
      const float d = s / c, about = s2 - s * d;
      m = shift + d;
      q = about < 0.f ? 0.f : about;                   // NaN stays NaN
    }
    __syncthreads();                                   // the previous n has been summed
    lds[0][threadIdx.x] = c;
    lds[1][threadIdx.x] = m;
    lds[2][threadIdx.x] = q;
    __syncthreads();
    c = m = q = 0.f;
    by_group(p, f,
             [&](int i) {
               if (p.center) join(c, m, q, lds[0][i], lds[1][i], lds[2][i]);
               else q += lds[2][i];
             },
             [&](int grp) {
               for (int k = 32; k; k >>= 1) {
                 const float c2 = __shfl_down(c, k), m2 = __shfl_down(m, k), q2 = __shfl_down(q, k);
                 if (p.center) join(c, m, q, c2, m2, q2);
                 else q += q2;
               }
               const int piece = f.pieces == 1 ? 0 : blockIdx.x % f.pieces;
               if (threadIdx.x % 64 == 0)
                 part[((size_t)n * f.parts + blockIdx.y * f.pieces + piece) * p.G + grp] = make_float4(c, m, q, 0.f);
               c = m = q = 0.f;
             });
  }
}

// The parts of each (n, group) joined into mean and 1 / deviation, by `lanes`
// neighbouring lanes (a power of two).
__global__ __launch_bounds__(256) void norm_stats_join_kernel(const float4* __restrict__ part, float* __restrict__ mean,
                                                              float* __restrict__ rstd, NormProblem p, NormPlan f, int lanes) {
  const int lane = threadIdx.x % lanes, per = 256 / lanes;
  const long long pairs = p.N * p.G;
  for (long long i = blockIdx.x * (long long)per + threadIdx.x / lanes; i < pairs; i += (long long)gridDim.x * per) {
    const long long n = i / p.G;
    const int grp = (int)(i % p.G);
    float c = 0.f, m = 0.f, q = 0.f;
    for (int k = lane; k < f.parts; k += lanes) {
      const float4 a = part[((size_t)n * f.parts + k) * p.G + grp];
      if (p.center) join(c, m, q, a.x, a.y, a.z);
      else q += a.z;
    }
    for (int k = lanes / 2; k; k >>= 1) {
      const float c2 = __shfl_xor(c, k), m2 = __shfl_xor(m, k), q2 = __shfl_xor(q, k);
      if (p.center) {
        // both sides of an exchange join in the same order
        if (lane & k) {
          float a = c2, b = m2, d = q2;
          join(a, b, d, c, m, q);
          c = a; m = b; q = d;
        } else {
          join(c, m, q, c2, m2, q2);
        }
      } else {
        q += q2;
      }
    }
    if (lane == 0) {
      if (mean) mean[i] = m;
      rstd[i] = 1.f / sqrtf(q / ((float)p.S * (float)p.cg) + p.eps);
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
  const int grp = t.grp;
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

// FINAL false: dgate, the workgroup's sums of dh and dh h of each group, psum
// [N][splits * pieces][G], and its sums over all its rows of du h and du per
// channel, part [gridDim.z][splits][2][C].  FINAL true: dx, with the
// group's sums in sums [N][G].
template <bool BF16, int VEC, bool GATE, bool FINAL>
__global__ __launch_bounds__(kTF, 4) void norm_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ weight,
    const float* __restrict__ bias, const void* __restrict__ gate, const float* __restrict__ mean,
    const float* __restrict__ rstd, void* __restrict__ dx, void* __restrict__ dgate, float* __restrict__ part,
    float2* __restrict__ psum, const float2* __restrict__ sums, NormProblem p, NormPlan f) {
  constexpr int kUnroll = FINAL ? 4 : 2;            // rows in flight: the sums take registers too
  __shared__ float2 lds[FINAL ? 1 : kTF];
  const Place t = place(p, f);
  if (FINAL && !t.on) return;
  float w[VEC], b[VEC], sw[VEC] = {}, sb[VEC] = {};
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    w[e] = weight && t.on ? weight[t.cv * VEC + e] : 1.f;
    b[e] = bias && t.on ? bias[t.cv * VEC + e] : 0.f;
  }
  const float inv = 1.f / ((float)p.S * (float)p.cg);
  for (long long z = blockIdx.z; z < p.N; z += gridDim.z) {
    const long long n = FINAL ? p.N - 1 - z : z;   // the second pass backwards, as in norm_apply_kernel
    const size_t base = (size_t)n * p.S * p.C + (size_t)t.cv * VEC;
    const float m = t.on && p.center ? mean[(size_t)n * p.G + t.grp] : 0.f, r = t.on ? rstd[(size_t)n * p.G + t.grp] : 0.f;
    float s1 = 0.f, s2 = 0.f;
    if constexpr (FINAL) {
      const float2 s = sums[(size_t)n * p.G + t.grp];
      s1 = p.center ? s.x * inv : 0.f;
      s2 = s.y * inv;
    }
    if (t.on)
#pragma unroll kUnroll
      for (int i = t.first; i < t.last; i += t.step) {
        float v[VEC], d[VEC], z4[VEC], dz[VEC];
        load_vec<BF16, VEC>(x, base + (size_t)i * p.C, v);
        load_vec<BF16, VEC>(dout, base + (size_t)i * p.C, d);
        if constexpr (GATE) load_vec<BF16, VEC>(gate, base + (size_t)i * p.C, z4);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float h = (v[e] - m) * r;
          const float du = grad_u<GATE>(p.act, d[e], fmaf(h, w[e], b[e]), GATE ? z4[e] : 0.f, &dz[e]);
          if constexpr (FINAL) {
            v[e] = r * (du * w[e] - s1 - h * s2);
          } else {
            sw[e] = fmaf(du, h, sw[e]);
            sb[e] += du;
            s1 = fmaf(du, w[e], s1);
            s2 = fmaf(du * w[e], h, s2);
          }
        }
        if constexpr (FINAL) store_vec<BF16, VEC>(dx, base + (size_t)i * p.C, v);
        else if constexpr (GATE) store_vec<BF16, VEC>(dgate, base + (size_t)i * p.C, dz);
      }
    if constexpr (!FINAL) {
      __syncthreads();                                 // the previous n has been summed
      lds[threadIdx.x] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.f;
      by_group(p, f,
               [&](int i) {
                 s1 += lds[i].x;
                 s2 += lds[i].y;
               },
               [&](int grp) {
                 for (int k = 32; k; k >>= 1) {
                   s1 += __shfl_xor(s1, k);
                   s2 += __shfl_xor(s2, k);
                 }
                 const int piece = f.pieces == 1 ? 0 : blockIdx.x % f.pieces;
                 if (threadIdx.x % 64 == 0)
                   psum[((size_t)n * f.parts + blockIdx.y * f.pieces + piece) * p.G + grp] = make_float2(s1, s2);
                 s1 = s2 = 0.f;
               });
    }
  }
  if constexpr (!FINAL) {
    // over the rpb rows at a time, through LDS
    float* o = part + ((size_t)blockIdx.z * f.splits + blockIdx.y) * 2 * p.C + (size_t)t.cv * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      __syncthreads();
      lds[threadIdx.x] = make_float2(sw[e], sb[e]);
      __syncthreads();
      if (t.on && t.off == 0) {
        float a = sw[e], c = sb[e];
        for (int k = 1; k < f.rpb; ++k) {
          a += lds[threadIdx.x + k * f.tile].x;
          c += lds[threadIdx.x + k * f.tile].y;
        }
        o[e] = a;
        o[p.C + e] = c;
      }
    }
  }
}

// The parts of each (n, group)'s sums added up, by `lanes` neighbouring lanes.
__global__ __launch_bounds__(256) void norm_grad_join_kernel(const float2* __restrict__ psum, float2* __restrict__ sums,
                                                             NormProblem p, NormPlan f, int lanes) {
  const int lane = threadIdx.x % lanes, per = 256 / lanes;
  const long long pairs = p.N * p.G;
  for (long long i = blockIdx.x * (long long)per + threadIdx.x / lanes; i < pairs; i += (long long)gridDim.x * per) {
    const float2* at = psum + (size_t)(i / p.G) * f.parts * p.G + i % p.G;
    float s1 = 0.f, s2 = 0.f;
    for (int k = lane; k < f.parts; k += lanes) {
      s1 += at[(size_t)k * p.G].x;
      s2 += at[(size_t)k * p.G].y;
    }
    for (int k = lanes / 2; k; k >>= 1) {
      s1 += __shfl_xor(s1, k);
      s2 += __shfl_xor(s2, k);
    }
    if (lane == 0) sums[i] = make_float2(s1, s2);
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

// ---------------------------------------------------------------- S > 1, bands

// Where a thread of the band kernels works.  L lanes (a power of two up to 64, or
// all T of a workgroup) hold the S x cg values of an (n, group): rpb rows at
// once, one vector a lane, rows row0, row0 + rpb, ...  A workgroup holds T / L
// groups of one n, or all groups of several n where there are fewer, and walks
// over n.  Workgroups go to the eight XCDs in turn: neighbouring bands, which
// share cache lines, get ids of equal remainder, so that one L2 serves them.
struct Band {
  int grp, cv, row0, rpb;
  bool on, valid;                   // has a group; the workgroup has work
  long long first, step;
};

template <int T>
__device__ __forceinline__ Band band_place(const NormProblem& p, int L, int vec, int X, int Y) {
  const int slots = T / L, slot = threadIdx.x / L, l = threadIdx.x % L, cvs = p.cg / vec;
  const unsigned total = (unsigned)X * Y, share = (total + 7) / 8, at = blockIdx.x % 8 * share + blockIdx.x / 8;
  const int bx = at % X, by = at / X;
  Band t;
  t.valid = at < total && blockIdx.x / 8 < share;
  t.rpb = L / cvs;
  t.row0 = l / cvs;
  t.cv = l % cvs;
  if (p.G >= slots) {
    t.grp = bx * slots + slot;
    t.on = t.grp < p.G;
    t.first = by;
    t.step = Y;
  } else {
    const int rows = slots / p.G, r = slot / p.G;
    t.grp = slot % p.G;
    t.on = r < rows;
    t.first = (long long)by * rows + r;
    t.step = (long long)Y * rows;
  }
  t.on = t.on && t.row0 < t.rpb;
  return t;
}

// Sums of two values over a band's lanes.
template <int T>
__device__ __forceinline__ float2 band_sum(float a, float b, int L, float2* lds) {
  for (int m = L < 64 ? L >> 1 : 32; m; m >>= 1) {
    a += __shfl_xor(a, m);
    b += __shfl_xor(b, m);
  }
  if (L > 64) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      a += lds[i].x;
      b += lds[i].y;
    }
  }
  return make_float2(a, b);
}

// Hides where a fetched vector came from: the values unpacked from it are not
// kept in registers from one use to the next.
template <bool BF16, int VEC>
__device__ __forceinline__ void forget(RawVec<BF16, VEC>& v) {
  if constexpr (VEC == 1) asm volatile("" : "+v"(v.v));
  else asm volatile("" : "+v"(v.v.x), "+v"(v.v.y), "+v"(v.v.z), "+v"(v.v.w));
}

constexpr int kTurn = 5;            // passes (vectors of a lane) of one turn of the output loop

// The activation is a switch over some code for each, of which a copy for every
// pass would take registers and instruction cache: the output loop handles kTurn
// passes a turn and moves the next ones' vectors down.  NV = 10 leaves two
// workgroups of 512 on a CU.  More does not pay: a 121 x 880 x 2240 frame norm in
// 20 groups, a band in 15 passes of 1024 lanes, 390 us (in 25 of 512, with
// spills, 482) against 324 by reading twice, because loads, sums and stores of
// the one band that a CU holds follow one another.
template <bool BF16, int VEC, int NV, bool GATE, int T>
__global__ __launch_bounds__(T, 4) void norm_band_kernel(
    const void* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias, const void* __restrict__ gate,
    void* __restrict__ out, float* __restrict__ mean, float* __restrict__ rstd, NormProblem p, int L, int X, int Y) {
  constexpr uint32_t es = BF16 ? 2 : 4;
  __shared__ float2 lds[T / 64];
  const Band t = band_place<T>(p, L, VEC, X, Y);
  if (!t.valid) return;
  const float inv = 1.f / ((float)p.S * (float)p.cg);
  int full = p.S / t.rpb;                              // passes in which every lane has a row; one more has some
  const int passes = (p.S + t.rpb - 1) / t.rpb;
  const bool part = t.on && t.row0 + full * t.rpb < p.S;
  const auto has = [&](int j) { return j < full ? t.on : j == full && part; };
  // bytes from the first value of an n; lanes without a row read one that exists, and add nothing
  const uint32_t off0 = t.on ? (uint32_t)(min(t.row0, p.S - 1) * p.C + t.grp * p.cg + t.cv * VEC) * es : 0;
  const uint32_t step = (uint32_t)(t.rpb * p.C) * es;
  for (long long n = t.first; n < p.N; n += t.step) {
    const size_t base = (size_t)n * p.S * p.C * es;
    const char* xn = static_cast<const char*>(x) + base;
    RawVec<BF16, VEC> v[NV];
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int j0 = 0; j0 < NV; j0 += kTurn)
      if (j0 < passes)
#pragma unroll
        for (int j = j0; j < j0 + kTurn; ++j)
          if (NV > kTurn || j < passes) v[j] = fetch_vec<BF16, VEC>(xn + (has(j) ? off0 + j * step : off0), 0);
    float m = 0.f;
    if (p.center) {
      asm volatile("" : "+s"(full));                   // the passes' masks are made anew, not kept in registers
#pragma unroll
      for (int j0 = 0; j0 < NV; j0 += kTurn)
        if (j0 < passes)
#pragma unroll
          for (int j = j0; j < j0 + kTurn; ++j) {
            if (NV == kTurn && j >= passes) continue;
            float a[VEC], y = 0.f;
            unpack<BF16, VEC>(v[j], a);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y += a[e];
            s += has(j) ? y : 0.f;
          }
      m = band_sum<T>(s, 0.f, L, lds).x * inv;
      s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) forget(v[j]);
    }
    asm volatile("" : "+s"(full));
#pragma unroll
    for (int j0 = 0; j0 < NV; j0 += kTurn)
      if (j0 < passes)
#pragma unroll
        for (int j = j0; j < j0 + kTurn; ++j) {
          if (NV == kTurn && j >= passes) continue;
          float a[VEC], y = 0.f, y2 = 0.f;
          unpack<BF16, VEC>(v[j], a);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float d = a[e] - m;
            y += d;
            y2 = fmaf(d, d, y2);
          }
          s += has(j) ? y : 0.f;
          q += has(j) ? y2 : 0.f;
        }
    asm volatile("" : "+s"(full));
    const float2 sums = band_sum<T>(s, q, L, lds);
    q = sums.y;
    if (p.center) {
      // what the mean's rounding left
      const float d = sums.x * inv;
      m += d;
      q = fmaf(-d, sums.x, q);
      q = q < 0.f ? 0.f : q;                           // NaN stays NaN
    }
    const float r = 1.f / sqrtf(q * inv + p.eps);
    if (!t.on) continue;
    if (t.row0 == 0 && t.cv == 0) {
      const size_t i = (size_t)n * p.G + t.grp;
      if (mean) mean[i] = m;
      rstd[i] = r;
    }
    float w[VEC], b[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[e] = weight ? weight[t.grp * p.cg + t.cv * VEC + e] : 1.f;
      b[e] = bias ? bias[t.grp * p.cg + t.cv * VEC + e] : 0.f;
    }
    char* on = static_cast<char*>(out) + base;
    const char* zn = static_cast<const char*>(gate) + base;
    uint32_t off = off0;
#pragma unroll 1
    for (int j0 = 0; j0 < passes; j0 += kTurn) {
#pragma unroll
      for (int j = 0; j < kTurn; ++j) {
        if (j0 + j >= passes) continue;
        const bool is = has(j0 + j);
        float a[VEC], z[VEC];
        forget(v[j]);
        unpack<BF16, VEC>(v[j], a);
        if constexpr (GATE) load_vec<BF16, VEC>(zn + (is ? off : off0), 0, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[e] = fmaf((a[e] - m) * r, w[e], b[e]);
        if constexpr (GATE) {
          act_all<VEC>(p.act, z);
#pragma unroll
          for (int e = 0; e < VEC; ++e) a[e] *= z[e];
        } else {
          act_all<VEC>(p.act, a);
        }
        if (is) store_vec<BF16, VEC>(on + off, 0, a);
        off += step;
        __builtin_amdgcn_sched_barrier(0);             // one pass's temporaries at a time
      }
#pragma unroll
      for (int j = 0; j + kTurn < NV; ++j) v[j] = v[j + kTurn];
    }
  }
}

// Gradients: x and dout in registers.  dweight and dbias: the sums of a lane over
// its n, joined over the lanes of the same channels, part [n held at once by all
// workgroups][2][C].
template <bool BF16, int VEC, bool GATE, int T>
__global__ __launch_bounds__(T, T == kT ? 3 : 2) void norm_band_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const void* __restrict__ gate, const float* __restrict__ mean, const float* __restrict__ rstd, void* __restrict__ dx,
    void* __restrict__ dgate, float* __restrict__ parts, NormProblem p, int L, int X, int Y) {
  constexpr uint32_t es = BF16 ? 2 : 4;
  __shared__ float2 lds[T];
  const Band t = band_place<T>(p, L, VEC, X, Y);
  if (!t.valid) return;
  const float inv = 1.f / ((float)p.S * (float)p.cg);
  const int full = p.S / t.rpb, passes = (p.S + t.rpb - 1) / t.rpb;
  const bool part = t.on && t.row0 + full * t.rpb < p.S;
  const auto has = [&](int j) { return j < full ? t.on : j == full && part; };
  const int c0 = t.on ? t.grp * p.cg + t.cv * VEC : 0;
  const uint32_t off0 = t.on ? (uint32_t)(min(t.row0, p.S - 1) * p.C + c0) * es : 0;
  const uint32_t step = (uint32_t)(t.rpb * p.C) * es;
  float w[VEC], b[VEC], sw[VEC], sb[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    w[e] = weight ? weight[c0 + e] : 1.f;
    b[e] = bias ? bias[c0 + e] : 0.f;
    sw[e] = sb[e] = 0.f;
  }
  for (long long n = t.first; n < p.N; n += t.step) {
    const size_t base = (size_t)n * p.S * p.C * es, at = (size_t)n * p.G + (t.on ? t.grp : 0);
    const char *xn = static_cast<const char*>(x) + base, *yn = static_cast<const char*>(dout) + base;
    const char* zn = static_cast<const char*>(gate) + base;
    RawVec<BF16, VEC> v[kTurn], g[kTurn];
#pragma unroll
    for (int j = 0; j < kTurn; ++j)
      if (j < passes) {
        const uint32_t off = has(j) ? off0 + j * step : off0;
        v[j] = fetch_vec<BF16, VEC>(xn + off, 0);
        g[j] = fetch_vec<BF16, VEC>(yn + off, 0);
      }
    const float m = p.center ? mean[at] : 0.f, r = rstd[at];
    float s1 = 0.f, s2 = 0.f;
    // h, du and dz of a pass
    const auto pass = [&](int j, float (&h)[VEC], float (&du)[VEC], float (&dz)[VEC]) {
      float u[VEC], z[VEC] = {};
      forget(v[j]);
      forget(g[j]);
      unpack<BF16, VEC>(v[j], h);
      unpack<BF16, VEC>(g[j], du);
      if constexpr (GATE) load_vec<BF16, VEC>(zn + (has(j) ? off0 + j * step : off0), 0, z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[e] = (h[e] - m) * r;
        u[e] = fmaf(h[e], w[e], b[e]);
      }
      grad_all<GATE, VEC>(p.act, du, u, z, dz);
    };
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if (j >= passes) continue;
      float h[VEC], du[VEC], dz[VEC];
      pass(j, h, du, dz);
      const bool is = has(j);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float y = is ? du[e] : 0.f, k = is ? h[e] : 0.f;   // of another row: NaN there stays there
        sw[e] = fmaf(y, k, sw[e]);
        sb[e] += y;
        s1 = fmaf(y, w[e], s1);
        s2 = fmaf(y * w[e], k, s2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const float2 sums = band_sum<T>(s1, s2, L, lds);
    s1 = p.center ? sums.x * inv : 0.f;
    s2 = sums.y * inv;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if (j >= passes) continue;
      float h[VEC], du[VEC], dz[VEC];
      pass(j, h, du, dz);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = r * (du[e] * w[e] - s1 - h[e] * s2);
      if (has(j)) {
        const size_t off = base + off0 + j * step;
        store_vec<BF16, VEC>(static_cast<char*>(dx) + off, 0, h);
        if constexpr (GATE) store_vec<BF16, VEC>(static_cast<char*>(dgate) + off, 0, dz);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  float* o = parts + (size_t)t.first * 2 * p.C + c0;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    __syncthreads();
    lds[threadIdx.x] = make_float2(sw[e], sb[e]);
    __syncthreads();
    if (t.on && t.row0 == 0) {
      float a = 0.f, c = 0.f;
      for (int k = 0; k < t.rpb; ++k) {
        a += lds[threadIdx.x + k * (p.cg / VEC)].x;
        c += lds[threadIdx.x + k * (p.cg / VEC)].y;
      }
      o[e] = a;
      o[p.C + e] = c;
    }
  }
}

// ---------------------------------------------------------------- host

int vec_of(const NormProblem& p) {
  const int v = p.bf16 ? 8 : 4;
  return p.cg % v == 0 ? v : 1;
}

// Lanes of a group on the S = 1 way and vectors per lane (0: the group is too
// wide for the registers of one workgroup; the gradient of 8 bf16 vectors a lane spills
// 26 of them, with a gate 105).  A wavefront has a group alone,
// without an exchange through LDS, up to 16 values a lane (32 take the
// gradient kernel's registers to one wavefront a SIMD: 16384 rows of one group
// of 2048 bf16 278 us against 76 by a workgroup).
void rows_shape(const NormProblem& p, int* L, int* NV) {
  const int vec = vec_of(p), cvs = p.cg / vec;
  int l = 1;
  while (l < 64 && l < cvs) l *= 2;
  if (cvs > 64 * (vec == 1 ? 8 : 16 / vec)) l = kT;
  const int need = (cvs + l - 1) / l;
  *L = l;
  *NV = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 0;
}

bool by_rows(const NormProblem& p) {
  int L, NV;
  rows_shape(p, &L, &NV);
  return p.S == 1 && NV > 0;
}

// About 2048 workgroups, a few rounds over the 256 CUs: each loads its weights
// once, and in the gradient leaves its rows' sums.  *rows: rows walked at once.
dim3 rows_grid(const NormProblem& p, int L, long long* rows) {
  const int slots = kT / L, x = p.G >= slots ? (p.G + slots - 1) / slots : 1, at_once = p.G >= slots ? 1 : slots / p.G;
  long long y = (2048 + x - 1) / x;
  const long long most = (p.N + at_once - 1) / at_once;
  if (y > most) y = most;
  if (rows) *rows = y * at_once;
  return dim3(x, (unsigned)y);
}

NormPlan plan(const NormProblem& p) {
  NormPlan f;
  f.per = p.cg / vec_of(p);
  if (f.per <= kTF) {
    int groups = kTF / f.per < p.G ? kTF / f.per : p.G;
    f.tiles = (p.G + groups - 1) / groups;
    groups = (p.G + f.tiles - 1) / f.tiles;
    f.tile = groups * f.per;
    f.pieces = 1;
  } else {
    f.pieces = (f.per + kTF - 1) / kTF;
    f.tile = (f.per + f.pieces - 1) / f.pieces;
    f.tiles = p.G * f.pieces;
  }
  f.rpb = kTF / f.tile;
  if (f.rpb > p.S) f.rpb = p.S;
  // splits of the rows: about 2048 workgroups in all, at least 4 rows a thread
  const long long want = 2048 / ((long long)f.tiles * (p.N < 2048 ? p.N : 2048)), most = p.S / (4LL * f.rpb);
  long long splits = want < most ? want : most;
  if (splits < 1) splits = 1;
  f.rows = (int)((p.S + splits - 1) / splits);
  f.splits = (p.S + f.rows - 1) / f.rows;
  f.parts = f.splits * f.pieces;
  f.threads = (f.tile * f.rpb + 63) / 64 * 64;
  // workgroups over n: all of them, or about 2048 in all that walk over n
  long long z = 2048 / ((long long)f.tiles * f.splits);
  f.z = (int)(z < 1 ? 1 : z < p.N ? z : p.N);
  return f;
}

// Lanes of an (n, group) on the band way, the fewest that hold it; returns the
// passes its kernel has registers for, or 0 where the band does not fit (the
// gradient keeps two tensors, so half as much).
int band_shape(const NormProblem& p, bool grad, int* L) {
  const int cvs = p.cg / vec_of(p);
  if ((long long)p.S * p.C * (p.bf16 ? 2 : 4) >= 1LL << 31) return 0;     // offsets within an n have 32 bits
  for (int l = 8; l <= kTF; l *= l == 64 ? 4 : 2) {
    const int most = l == kTF && !grad ? 2 * kTurn : kTurn, rpb = l / cvs;
    if (rpb == 0 || (p.S + rpb - 1) / rpb > most) continue;
    *L = l;
    return most;
  }
  return 0;
}

// Workgroups: X over the groups, Y over n; the gradient's about 2048 in all, each
// of which walks over several n and leaves one set of sums.  *rows: n held at once.
dim3 band_grid(const NormProblem& p, bool grad, int L, int* X, int* Y, long long* rows) {
  const int slots = (L < kTF ? kT : kTF) / L, at_once = p.G >= slots ? 1 : slots / p.G;
  *X = p.G >= slots ? (p.G + slots - 1) / slots : 1;
  const long long all = (p.N + at_once - 1) / at_once, most = (grad ? 2048 : kMaxBlocks) / *X;
  const long long y = most < 1 ? 1 : most < all ? most : all, walk = (all + y - 1) / y;
  *Y = (int)((all + walk - 1) / walk);                 // as few as the longest walk allows
  *rows = (long long)*Y * at_once;
  return dim3(((unsigned)*X * *Y + 7) / 8 * 8);
}

// Lanes that join a (n, group)'s parts, and the workgroups of that.
int join_lanes(const NormPlan& f) {
  int l = 1;
  while (l < 64 && l < f.parts) l *= 2;
  return l;
}

unsigned join_grid(const NormProblem& p, int lanes) {
  const long long b = (p.N * p.G + 256 / lanes - 1) / (256 / lanes);
  return (unsigned)(b < kMaxBlocks ? b : kMaxBlocks);
}

template <bool BF16, int VEC, bool GATE>
hipError_t forward_v(const NormProblem& p, const void* x, const float* weight, const float* bias, const void* gate, void* out,
                     float* mean, float* rstd, void* ws, hipStream_t st) {
  if (by_rows(p)) {
    int L, NV;
    rows_shape(p, &L, &NV);
    const dim3 grid = rows_grid(p, L, nullptr);
#define GDN_ROWS(V)                                                                                                      \
  case V:                                                                                                                \
    hipLaunchKernelGGL((norm_rows_kernel<BF16, VEC, V, GATE>), grid, dim3(kT), 0, st, x, weight, bias, gate, out, mean, \
                       rstd, p, L);                                                                                      \
    break;
    switch (NV) { GDN_ROWS(1) GDN_ROWS(2) GDN_ROWS(4) GDN_ROWS(8) }
#undef GDN_ROWS
    return hipGetLastError();
  }
  int L, X, Y;
  if (const int passes = band_shape(p, false, &L)) {
    long long rows;
    const dim3 grid = band_grid(p, false, L, &X, &Y, &rows);
    const auto f = passes == kTurn && L < kTF ? norm_band_kernel<BF16, VEC, kTurn, GATE, kT> : norm_band_kernel<BF16, VEC, 2 * kTurn, GATE, kTF>;
    hipLaunchKernelGGL(f, grid, dim3(L < kTF ? kT : kTF), 0, st, x, weight, bias, gate, out, mean, rstd, p, L, X, Y);
    return hipGetLastError();
  }
  const NormPlan f = plan(p);
  float4* part = static_cast<float4*>(ws);
  const dim3 grid(f.tiles, f.splits, f.z);
  const int lanes = join_lanes(f);
  hipLaunchKernelGGL((norm_stats_kernel<BF16, VEC>), grid, dim3(f.threads), 0, st, x, part, p, f);
  hipLaunchKernelGGL(norm_stats_join_kernel, dim3(join_grid(p, lanes)), dim3(256), 0, st, part, mean, rstd, p, f, lanes);
  hipLaunchKernelGGL((norm_apply_kernel<BF16, VEC, GATE>), grid, dim3(f.threads), 0, st, x, weight, bias, gate, out, mean, rstd,
                     p, f);
  return hipGetLastError();
}

template <bool BF16, int VEC, bool GATE>
hipError_t backward_v(const NormProblem& p, const NormGrad& t, void* ws, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  long long rows = 0;
  int L, X, Y;
  if (p.N > 0 && by_rows(p)) {
    int L, NV;
    rows_shape(p, &L, &NV);
    const dim3 grid = rows_grid(p, L, &rows);
#define GDN_ROWS(V)                                                                                                       \
  case V:                                                                                                                 \
    hipLaunchKernelGGL((norm_rows_grad_kernel<BF16, VEC, V, GATE>), grid, dim3(kT), 0, st, t.dout, t.x, t.weight, t.bias, \
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, p, L);                                                \
    break;
    switch (NV) { GDN_ROWS(1) GDN_ROWS(2) GDN_ROWS(4) GDN_ROWS(8) }
#undef GDN_ROWS
  } else if (p.N > 0 && band_shape(p, true, &L)) {
    const dim3 grid = band_grid(p, true, L, &X, &Y, &rows);
    const auto f = L < kTF ? norm_band_grad_kernel<BF16, VEC, GATE, kT> : norm_band_grad_kernel<BF16, VEC, GATE, kTF>;
    hipLaunchKernelGGL(f, grid, dim3(L < kTF ? kT : kTF), 0, st, t.dout, t.x, t.weight, t.bias, t.gate, t.mean, t.rstd, t.dx,
                       t.dgate, part, p, L, X, Y);
  } else if (p.N > 0) {
    const NormPlan f = plan(p);
    rows = (long long)f.z * f.splits;
    float2* psum = reinterpret_cast<float2*>(part + (size_t)rows * 2 * p.C);
    float2* sums = psum + (size_t)p.N * f.parts * p.G;
    const dim3 grid(f.tiles, f.splits, f.z);
    const int lanes = join_lanes(f);
    hipLaunchKernelGGL((norm_grad_kernel<BF16, VEC, GATE, false>), grid, dim3(f.threads), 0, st, t.dout, t.x, t.weight, t.bias,
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, psum, sums, p, f);
    hipLaunchKernelGGL(norm_grad_join_kernel, dim3(join_grid(p, lanes)), dim3(256), 0, st, psum, sums, p, f, lanes);
    hipLaunchKernelGGL((norm_grad_kernel<BF16, VEC, GATE, true>), grid, dim3(f.threads), 0, st, t.dout, t.x, t.weight, t.bias,
                       t.gate, t.mean, t.rstd, t.dx, t.dgate, part, psum, sums, p, f);
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
    long long rows;
    rows_shape(p, &L, &NV);
    rows_grid(p, L, &rows);
    return gradient ? (size_t)rows * 2 * p.C * sizeof(float) : 0;
  }
  int L, X, Y;
  if (band_shape(p, gradient, &L)) {
    long long rows;
    band_grid(p, gradient, L, &X, &Y, &rows);
    return gradient ? (size_t)rows * 2 * p.C * sizeof(float) : 0;
  }
  const NormPlan f = plan(p);
  const size_t sums = (size_t)p.N * f.parts * p.G;
  return gradient ? (size_t)f.z * f.splits * 2 * p.C * sizeof(float) + (sums + (size_t)p.N * p.G) * sizeof(float2)
                  : sums * sizeof(float4);
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
