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

// 2^x in one instruction (1 ulp; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

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

// Two values as the sums of N bf16 values each, largest first, packed by term:
// one conversion, two unpackings and two subtractions for a term of a pair.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&o)[N]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x, y}, b2));   // round to nearest even
    if (i + 1 < N) {
      x -= __uint_as_float(o[i] << 16);
      y -= __uint_as_float(o[i] & 0xffff0000u);
    }
  }
}

template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&x)[8]) {
  uint32_t o[4][N];
#pragma unroll
  for (int j = 0; j < 4; ++j) split2<N>(x[2 * j], x[2 * j + 1], o[j]);
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(make_uint4(o[0][i], o[1][i], o[2][i], o[3][i]));
  return f;
}

// Eight consecutive fp32 values as a fragment.
template <int N>
__device__ __forceinline__ Frag<N> frag_f32(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return split8<N>(x);
}

// Buffer addressing: `bytes` from a uniform base, per-lane 32-bit offsets.  The
// hardware returns 0 for loads and drops stores behind the end, so rows behind a
// sequence's end and columns behind d_k (their lanes' offsets are kNowhere) need
// no branches: a branch around a load would make every wait for a younger load
// wait for it too.
typedef __amdgpu_buffer_rsrc_t buf_t;
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ buf_t buf(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ uint4 buf_load16(buf_t b, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}

// Bytes that a chunk's rows span: min(n, 64) rows of `width`, `stride` apart.
__device__ __forceinline__ uint32_t span(int n, uint32_t stride, uint32_t width) {
  return n > 0 ? (uint32_t)(min(n, kC) - 1) * stride + width : 0;
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

// Four input values to and from LDS.
template <int NT>
__device__ __forceinline__ void put_values(typename RawIn<NT>::type* to, const typename RawIn<NT>::type (&x)[4]) {
  if constexpr (NT == 1)
    *reinterpret_cast<uint2*>(to) = make_uint2(x[0] | (uint32_t)x[1] << 16, x[2] | (uint32_t)x[3] << 16);
  else
    *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
}

template <int NT>
__device__ __forceinline__ void get_values(const typename RawIn<NT>::type* from, float (&x)[4]) {
  if constexpr (NT == 1) {
    const uint2 v = *reinterpret_cast<const uint2*>(from);
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    const float4 v = *reinterpret_cast<const float4*>(from);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
}

__device__ __forceinline__ void floats(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}

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
__device__ __forceinline__ RawFrag<NT> raw_at(buf_t b, uint32_t off) {
  RawFrag<NT> r;
  r.a = buf_load16(b, off);
  if constexpr (NT == 3) r.b = buf_load16(b, off + 16);
  return r;
}

template <int NT>
__device__ __forceinline__ typename RawIn<NT>::type value_at(buf_t b, uint32_t off) {
  if constexpr (NT == 1) return __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0);
  else return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}

// Stores x as bf16 (two bytes) or fp32 (four).
template <int BYTES>
__device__ __forceinline__ void store_at(buf_t b, uint32_t off, float x) {
  if constexpr (BYTES == 2) __builtin_amdgcn_raw_buffer_store_b16(f2bh(x), b, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), b, off, 0, 0);
}

// A fragment of N terms whose lane has its place at `off`.
template <int N>
__device__ __forceinline__ Frag<N> frag_at(buf_t b, uint32_t off) {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(buf_load16(b, off + i * 1024));
  return f;
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

// A stored fragment of N terms.
template <int N>
__device__ __forceinline__ Frag<N> load_frag(const uint4* p, int frag, int lane) {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(p[((size_t)frag * N + i) * 64 + lane]);
  return f;
}

template <int N>
__device__ __forceinline__ void store_frag(uint4* p, int frag, int lane, const Frag<N>& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) p[((size_t)frag * N + i) * 64 + lane] = as_bits(f.t[i]);
}

// Operand tiles in LDS: 16 columns of K rows (K a multiple of 32) as N terms, in
// fragment order, [term][K / 32][lane][8]: a fragment is read as 64 contiguous
// vectors, and the four rows of a column that an accumulator lane holds are half
// a vector, so a wavefront's write is contiguous too.  (Row-major tiles with a
// padded stride lost half of the LDS cycles to bank conflicts.)

// Elements from the tile's start to the lane that holds rows row .. row + 3 of a
// column (row a multiple of 4).
__device__ __forceinline__ int put_place(int column, int row) {
  return ((row / 32 * 4 + row % 32 / 8) * 16 + column) * 8 + row % 8;
}

// Writes four consecutive rows of a column; `to` points at their place.
template <int N, int K>
__device__ __forceinline__ void put(bh* to, const float (&x)[4]) {
  uint32_t lo[N], hi[N];
  split2<N>(x[0], x[1], lo);
  split2<N>(x[2], x[3], hi);
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<uint2*>(to + i * K * 16) = make_uint2(lo[i], hi[i]);
}

// Rows 32 ks .. of the tile; `from` points at the lane's vector of its first fragment.
template <int N, int K>
__device__ __forceinline__ Frag<N> get(const bh* from, int ks) {
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.t[i] = as_frag(*reinterpret_cast<const uint4*>(from + i * K * 16 + ks * 512));
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

// The r-th sequence by length, longest first, in each wavefront for itself.  A
// scan's workgroup lasts as long as its sequence, and where there are several
// rounds of workgroups a long one that starts last leaves the card idle
// (13 prompts of 35 to 1881 tokens, 32 heads of 128: scan 270 us in the order
// given, 232 so; 6 training sequences of 762 to 2716: forward scan 241 and 193,
// reverse scan 322 and 259).
// More than 64 sequences even out by themselves and keep their order.
__device__ __forceinline__ int by_length(const int* cu, int sequences, long long tokens, int r) {
  if (sequences == 1 || sequences > 64) return r;
  const int lane = threadIdx.x % 64;
  int a = 0, b = 0, rank = 0;
  if (lane < sequences) seq_bounds(cu, lane, tokens, &a, &b);
  const int length = b - a;
  for (int i = 0; i < sequences; ++i) {
    const int other = __builtin_amdgcn_readlane(length, i);
    rank += other > length || (other == length && i < lane);
  }
  return __ffsll(__ballot(lane < sequences && rank == r)) - 1;
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
