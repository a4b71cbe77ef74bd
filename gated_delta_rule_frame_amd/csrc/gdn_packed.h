// Shared parts of the packed gated delta rule kernels (gdn_packed.hip,
// gdn_packed_grad.hip): precision and tile layouts (the workspace: gdn_seq.h).
//
// Precision.  Matrix products run on the bf16 MFMA with fp32 accumulation.  An
// operand that is given in bf16 is one term; an fp32 one (states, residuals,
// triangular inverses, fp32 inputs) is split into three bf16 terms, x = x0 + x1 +
// x2 exactly to 24 bits, and a product of two split operands sums the six term
// products i + j <= 2; what is left out is below 2^-24 of the product.  Two terms
// would leave 4e-6 to 7e-6 relative error in states and gate gradients (a float64
// emulation of the kernels); three leave 1e-7, that of fp32 arithmetic, without
// the range limit of fp16 operands.  The bf16 MFMA with six terms still has 2.7
// times the rate of the fp32 MFMA.
//
// Fragments.  Operand convention as in gdn_mfma.h: for a 16 x 32 tile lane l holds
// row l % 16, columns 8 (l / 16) .. + 8, as one 16-byte vector.  Matrices that a
// later kernel multiplies are stored fragment by fragment, 64 x 16 bytes each, so
// that a load is one contiguous KB.
#pragma once

#include "gdn_common.h"
#include "gdn_mfma.h"
#include "gdn_seq.h"

namespace gdn {

// ---------------------------------------------------------------- device

typedef bf16x8_t frag_t;

template <int N>
struct Frag {
  frag_t t[N];
};

__device__ __forceinline__ frag_t as_frag(uint4 v) { return __builtin_bit_cast(frag_t, v); }
__device__ __forceinline__ uint4 as_bits(frag_t v) { return __builtin_bit_cast(uint4, v); }

__device__ __forceinline__ f32x4 mfma(frag_t a, frag_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += a b over the term pairs that matter.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 c) {
#pragma unroll
  for (int s = (NA < 3 ? NA : 3) + (NB < 3 ? NB : 3) - 2; s >= 0; --s) {   // smallest terms first
    if (s > 2) continue;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = mfma(a.t[i], b.t[s - i], c);
  }
  return c;
}

// c[s] += the products of terms i + j = s, for s = 0, 1, 2: three chains of
// dependent MFMAs instead of one.
template <int NA, int NB>
__device__ __forceinline__ void mma_by_term(const Frag<NA>& a, const Frag<NB>& b, f32x4 (&c)[3]) {
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c[s] = mfma(a.t[i], b.t[s - i], c[s]);
}

template <int N, int M>
__device__ __forceinline__ Frag<N> first_terms(const Frag<M>& f) {
  Frag<N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.t[i] = f.t[i];
  return o;
}

// x as the sum of N bf16 values, largest first.
template <int N>
__device__ __forceinline__ void split(float x, bh (&o)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    o[i] = f2bh(x);
    x -= bh2f(o[i]);
  }
}

template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&x)[8]) {
  Frag<N> f;
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f.t[i][j] = static_cast<__bf16>(r[j]);
      if (i + 1 < N) r[j] -= static_cast<float>(f.t[i][j]);
    }
  return f;
}

template <int N>
__device__ __forceinline__ Frag<N> zero_frag() {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(make_uint4(0, 0, 0, 0));
  return f;
}

// Eight consecutive fp32 values as a fragment.
template <int N>
__device__ __forceinline__ Frag<N> frag_f32(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return split8<N>(x);
}

// Eight consecutive input values (bf16 for one term, fp32 for three).
template <int NT>
__device__ __forceinline__ Frag<NT> frag_in(const void* p, size_t i) {
  if constexpr (NT == 1) {
    Frag<1> f;
    f.t[0] = as_frag(*reinterpret_cast<const uint4*>(static_cast<const bh*>(p) + i));
    return f;
  } else {
    return frag_f32<3>(static_cast<const float*>(p) + i);
  }
}

// Element at a 32-bit byte offset from a uniform base (one scalar pair and one
// vector register of address).
template <typename T>
__device__ __forceinline__ T at_byte(const void* base, uint32_t off) {
  return *reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// One input value as it lies in memory, and its value.
template <int NT>
struct RawIn {
  using type = uint16_t;
};
template <>
struct RawIn<3> {
  using type = float;
};
__device__ __forceinline__ float raw_value(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ float raw_value(float x) { return x; }

// Eight consecutive input values as they lie in memory, split where they are used.
template <int NT>
struct RawFrag {
  uint4 a, b;                       // fp32: two vectors
};
template <>
struct RawFrag<1> {
  uint4 a;
};

template <int NT>
__device__ __forceinline__ RawFrag<NT> zero_raw() {
  RawFrag<NT> r;
  r.a = make_uint4(0, 0, 0, 0);
  if constexpr (NT == 3) r.b = r.a;
  return r;
}

template <int NT>
__device__ __forceinline__ RawFrag<NT> raw_at(const void* base, uint32_t off) {
  RawFrag<NT> r;
  r.a = at_byte<uint4>(base, off);
  if constexpr (NT == 3) r.b = at_byte<uint4>(base, off + 16);
  return r;
}

template <int NT>
__device__ __forceinline__ Frag<NT> frag_of(const RawFrag<NT>& r) {
  if constexpr (NT == 1) {
    Frag<1> f;
    f.t[0] = as_frag(r.a);
    return f;
  } else {
    const float x[8] = {__uint_as_float(r.a.x), __uint_as_float(r.a.y), __uint_as_float(r.a.z), __uint_as_float(r.a.w),
                        __uint_as_float(r.b.x), __uint_as_float(r.b.y), __uint_as_float(r.b.z), __uint_as_float(r.b.w)};
    return split8<3>(x);
  }
}

template <int NT>
__device__ __forceinline__ float elem_in(const void* p, size_t i) {
  return load_scalar<NT == 1>(p, i);
}

// The first N of a stored fragment's LD terms.
template <int N, int LD = N>
__device__ __forceinline__ Frag<N> load_frag(const uint4* p, int frag, int lane) {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(p[((size_t)frag * LD + i) * 64 + lane]);
  return f;
}

template <int N>
__device__ __forceinline__ void store_frag(uint4* p, int frag, int lane, const Frag<N>& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) p[((size_t)frag * N + i) * 64 + lane] = as_bits(f.t[i]);
}

constexpr int kTok = 72;    // row stride (bf16) of a 16 x 64 operand tile in LDS

// Writes four consecutive rows of a column as N terms: tile[term][column][row].
template <int N, int LD>
__device__ __forceinline__ void put(bh* tile, int plane, int column, int row, const float (&x)[4]) {
  bh b[4][N];
#pragma unroll
  for (int r = 0; r < 4; ++r) split<N>(x[r], b[r]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint2 v;
    v.x = b[0][i] | (uint32_t)b[1][i] << 16;
    v.y = b[2][i] | (uint32_t)b[3][i] << 16;
    *reinterpret_cast<uint2*>(tile + i * plane + column * LD + row) = v;
  }
}

template <int LD>
__device__ __forceinline__ void put3(bh* tile, int plane, int column, int row, const float (&x)[4]) {
  put<3, LD>(tile, plane, column, row, x);
}

template <int N, int LD>
__device__ __forceinline__ Frag<N> get(const bh* tile, int plane, int column, int row) {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(*reinterpret_cast<const uint4*>(tile + i * plane + column * LD + row));
  return f;
}

// Tokens [start, end) of sequence s.  Bounds that do not fit the packed rows
// are clamped to them, so no value of cu reads or writes out of range.
__device__ __forceinline__ void seq_bounds(const int* cu, int s, long long tokens, int* start, int* end) {
  const int n = (int)tokens;
  const int a = min(max(cu[s], 0), n);
  *start = a;
  *end = min(max(cu[s + 1], a), n);
}

// The (sequence, head) and strip of a scan's workgroup.  Workgroups go to the
// eight XCDs in turn, so the strips of one (sequence, head), which read the same
// operands, get ids of equal remainder mod 8 that follow one another: they run
// at the same time on one XCD and share its L2.  The grid has the number of
// (sequence, head) pairs rounded up to 8, times the strips.
__device__ __forceinline__ void strip_of(int block, int strips, int* sh, int* strip) {
  const int i = block / 8;
  *sh = i / strips * 8 + block % 8;
  *strip = i % strips;
}

// The sequence and chunk of a chunk slot; false for a slot without tokens.
__device__ __forceinline__ bool find_chunk(const int* cu, int sequences, long long tokens, long long slot, int* seq, int* first,
                                           int* n) {
  int lo = 0, hi = sequences - 1;
  const int t = (int)tokens;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (min(max(cu[mid], 0), t) / kC + (long long)mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  int a, b;
  seq_bounds(cu, lo, tokens, &a, &b);
  const long long c = slot - (a / kC + (long long)lo);
  *seq = lo;
  if (c < 0 || c * kC >= b - a) return false;
  *first = a + (int)c * kC;
  *n = min(kC, b - *first);
  return true;
}

}  // namespace gdn
