// Linear attention with a decay for each head over packed sequences, chunked, and
// its gradients: the scan that the calls share.
//
// One scan serves all of them.  For operands A, B (width I) and C (width J), the
// cumulative log-gate G of a chunk and a state S (I x J):
//     forward:   out_x = s (e^{G_x} A_x S + sum_{y <= x} e^{G_x - G_y} (A_x.B_y) C_y)
//                S    <- e^{G_n} S + sum_y e^{G_n - G_y} B_y C_y^T
//     reversed:  out_x = e^{G_n - G_x} A_x S + s sum_{y >= x} e^{G_y - G_x} (A_x.B_y) C_y
//                S    <- e^{G_n} S + s sum_y e^{G_y} B_y C_y^T
//     outputs    forward  (A, B, C) = (q, k, v),  S from the initial state
//     dq         forward  (dout, v, k),  S transposed
//     dv         reversed (k, q, dout),  S from the final state's gradient
//     dk         reversed (v, dout, q),  S transposed
// so a gradient costs three scans over the same operands, and dlog_gate follows
// from sums: q.dq and v.dv of a token are its place in the outputs and in the
// writes, dlog_gate_t = <R, S> at the segment's end + sum_{s >= t} (q_s.dq_s -
// v_s.dv_s), with the gradient R of the state there.  What a token reads of its own
// write, scale (q.k)(do.v), is in both and would drown what strong decays leave of
// the others, so the dot products are formed without it: P goes into its product
// without its diagonal, which joins the outputs afterwards (8192 tokens of 16 and 32
// heads of 128: 403 -> 425 us; a gate of -16 for all tokens of a head: relative
// error of its gradient 190 -> 2e-5).
//
// Segments.  Sequences are cut into segments of L tokens that run in parallel:
// a first launch sums what each segment adds to the state (its last line above
// alone), a second one chains these sums into the states between segments, and
// the scan starts every segment from its own.
//
// A chunk.  Four wavefronts of 16 or 32 columns of the state each, which stay in
// accumulators: the rows of an accumulator tile are the rows of an operand, so that
// A S takes the state from the registers it is summed in.  A, B and C pass through
// LDS once (the next chunk's are in flight meanwhile); P = A B^T, gated and split,
// passes through LDS to the wavefronts' columns.  fp32 values are three bf16 terms,
// products six of the nine term products.  What bounds it: with d = 128 and bf16
// a wavefront has 240 matrix instructions of 16 clocks a chunk.  A chunk takes 6.9 us
// for a workgroup alone on a CU and 9.6 for two (16 sequences of 2048 tokens, 32
// heads: 338 us), of which the matrix instructions would take 4.5 at 1.7 GHz: the rest
// is the splitting of the state and of P, of which a matrix instruction hides two
// instructions, and the waits at the chunk's three barriers.  8191 tokens of 32 heads
// in segments: 113 to 120 us, 2.5 TB/s; 32768 of 35 heads of 64: 159 to 201, 3 to 3.8.
#pragma once

#include <type_traits>

#include "gdn_linear.h"
#include "gdn_packed.h"

namespace gdn {

// ---------------------------------------------------------------- device

constexpr int kScanThreads = 256;
// bf16 terms of the states and of P where they meet A and C, whatever the outputs' type: with three a bf16 output is the fp32
// output rounded once.  Two (2^-17 of a product) sent 0.23 % of a call's bf16 values to another neighbour than the plain fp32 form
// has, against 0.02 %, for 99 us of the forward scan's 115 (8191 tokens of 32 heads of 128) and 385 of the gradients' 389.
constexpr int kTerms = 3;
constexpr int kAtOnce = 512;                   // workgroups of a scan that run at once, at least

// Gates below this are this: e^-10000 is 0 in fp32, and G stays finite for -inf.
constexpr float kLowestGate = -10000.f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef s16x4 __attribute__((address_space(3)))* lds_s16x4;

// Operand tiles in LDS: rows (tokens) of U units of 16 bytes (8 bf16 values), unit
// u of row r at place u ^ swizzle(r).  Row fragments (16 rows, the same unit) and
// transposed ones (4 rows, 16 columns) both touch every bank once.
template <int U>
__device__ __forceinline__ uint32_t swizzle(uint32_t r) {
  if constexpr (U == 16) return (r & 3) << 2 | (r >> 2 & 3);
  else if constexpr (U == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
  else return r >> 2 & 3;
}

// Rows row0 .. + 15, columns 32 ks + 8 (lane / 16) .. + 8: lane l has row l % 16.
template <int NT, int U, int CH>
__device__ __forceinline__ Frag<NT> row_frag(const char* tile, int row0, int ks, uint32_t lane) {
  const uint32_t r = lane % 16;
  const uint32_t at = row0 * U * 16 + r * U * 16 + ((ks * 4 + lane / 16) ^ swizzle<U>(r)) * 16;
  Frag<NT> f;
#pragma unroll
  for (int i = 0; i < NT; ++i) f.t[i] = as_frag(*reinterpret_cast<const uint4*>(tile + i * CH * U * 16 + at));
  return f;
}

// The transpose: lane l has column l % 16 of a tile whose columns are four pieces of
// four, rows 32 k2 + 8 (l / 16) .. + 8.  `unit`, `sub`: where piece l % 4 lies in a row.
template <int NT, int U, int CH>
__device__ __forceinline__ Frag<NT> column_frag(const char* tile, int k2, uint32_t unit, uint32_t sub, uint32_t lane) {
  const uint32_t r0 = 8 * (lane / 16) + lane % 16 / 4;
  Frag<NT> f;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    s16x4 h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t r = r0 + 4 * j;
      const char* at = tile + (i * CH + 32 * k2) * U * 16 + (r * U * 16 + (unit ^ swizzle<U>(r)) * 16 + sub);
      h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at);
    }
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    f.t[i] = __builtin_bit_cast(frag_t, (s16x8)__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return f;
}

// A chunk's rows of one operand on their way into LDS.
template <int NT, int U, int CH, int TH>
struct Stage {                                  // TH: threads
  static constexpr int N = (CH * U + TH - 1) / TH;
  uint4 r[N][NT == 1 ? 1 : 2];

  static constexpr uint32_t step = TH / U;          // rows from one vector of a thread to its next: a multiple of 16

  __device__ __forceinline__ void load(buf_t b, uint32_t stride, int width, uint32_t tid) {
    constexpr uint32_t es = NT == 1 ? 2 : 4;
    asm volatile("" : "+v"(tid));                    // offsets are made here and not kept in registers through the chunk
    const uint32_t row = tid / U, u = tid % U;
    const bool in = (CH * U % TH == 0 || tid < CH * U) && (int)u * 8 < width;
    uint32_t off = in ? row * stride + u * 8 * es : kNowhere;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r[i][0] = buf_load16(b, off);
      if constexpr (NT == 3) r[i][1] = buf_load16(b, off + 16);
      off += step * stride;                          // behind kNowhere it stays there: 64 rows span less than 2^31 bytes
    }
  }

  __device__ __forceinline__ void store(char* tile, uint32_t tid) const {
    asm volatile("" : "+v"(tid));
    const uint32_t row = tid / U, u = tid % U;
    char* to = tile + row * U * 16 + (u ^ swizzle<U>(row)) * 16;
    if (CH * U % TH && tid >= CH * U) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (NT == 1) {
        *reinterpret_cast<uint4*>(to + i * step * U * 16) = r[i][0];
      } else {
        RawFrag<3> raw;
        raw.a = r[i][0];
        raw.b = r[i][1];
        const Frag<3> f = frag_of<3>(raw);
#pragma unroll
        for (int t = 0; t < 3; ++t) *reinterpret_cast<uint4*>(to + (i * step + t * CH) * U * 16) = as_bits(f.t[t]);
      }
    }
  }
};

// Keeps loads from LDS a step ahead of the products that use them: nothing is scheduled across.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// N (4 or 8) consecutive input values.
template <int NT, int N>
struct Values {
  uint32_t b[NT == 1 ? N / 2 : N];
  __device__ __forceinline__ void load(buf_t from, uint32_t off) {
    if constexpr (NT == 1 && N == 4) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(from, off, 0, 0));
      b[0] = v[0];
      b[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < (int)(sizeof b / 16); ++i) {
        const uint4 v = buf_load16(from, off + 16 * i);
        b[4 * i] = v.x;
        b[4 * i + 1] = v.y;
        b[4 * i + 2] = v.z;
        b[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (NT == 1) return __uint_as_float(i % 2 ? b[i / 2] & 0xffff0000u : b[i / 2] << 16);
    else return __uint_as_float(b[i]);
  }
};

// The sum of x over the lanes up to this one, by shifts in rows of 16 lanes and
// broadcasts of their last lanes (lane shuffles through LDS take several times as long).
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_before(double x) {      // 0 where no lane is
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 v = __builtin_bit_cast(i32x2, x);
  return __builtin_bit_cast(double, i32x2{__builtin_amdgcn_update_dpp(0, v[0], CTRL, ROWS, 0xf, false),
                                          __builtin_amdgcn_update_dpp(0, v[1], CTRL, ROWS, 0xf, false)});
}

__device__ __forceinline__ double prefix_sum(double x) {
  x += lanes_before<0x111, 0xf>(x);    // row_shr:1, 2, 4, 8
  x += lanes_before<0x112, 0xf>(x);
  x += lanes_before<0x114, 0xf>(x);
  x += lanes_before<0x118, 0xf>(x);
  x += lanes_before<0x142, 0xa>(x);    // row_bcast:15 into rows 1 and 3
  x += lanes_before<0x143, 0xc>(x);    // row_bcast:31 into rows 2 and 3
  return x;
}

__device__ __forceinline__ double last_lane(double x) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 v = __builtin_bit_cast(i32x2, x);
  return __builtin_bit_cast(double, i32x2{__builtin_amdgcn_readlane(v[0], 63), __builtin_amdgcn_readlane(v[1], 63)});
}

// A segment of a sequence.  Those of sequence s, which starts at token a, have the slots a / L + s (rounded down) and on.
struct Segment {
  int slot;
  int seq, c, count;        // segment c of `count` of this sequence
  int first, n;             // its tokens
  int start, length;        // those of the sequence
};

// Segments of a sequence, as many as its length needs at most L tokens each, and their length: equal ones of whole chunks, so
// that the workgroups of a launch end together (the last may be shorter).
__device__ __forceinline__ int segments_of(int tokens, int L, int* length) {
  const uint32_t chunks = ((uint32_t)tokens + kC - 1) / kC, wanted = ((uint32_t)tokens + L - 1) / (uint32_t)L;
  if (wanted == 0) {
    *length = kC;
    return 0;
  }
  const uint32_t each = (chunks + wanted - 1) / wanted;
  *length = each * kC;
  return (chunks + each - 1) / each;
}

// Segment c of sequence seq, tokens a .. b; false where there is none.
__device__ __forceinline__ bool set_segment(int seq, int c, int a, int b, int L, Segment* s) {
  int each;
  const int count = max(1, segments_of(b - a, L, &each));   // an empty sequence has one of no tokens
  if (c < 0 || c >= count) return false;
  s->seq = __builtin_amdgcn_readfirstlane(seq);
  s->c = __builtin_amdgcn_readfirstlane(c);
  s->start = __builtin_amdgcn_readfirstlane(a);
  s->count = __builtin_amdgcn_readfirstlane(count);
  s->length = __builtin_amdgcn_readfirstlane(b - a);
  s->first = s->start + s->c * __builtin_amdgcn_readfirstlane(each);
  s->n = __builtin_amdgcn_readfirstlane(min(each, b - s->first));
  s->slot = __builtin_amdgcn_readfirstlane((int)(a / (uint32_t)L) + seq + c);
  return true;
}

__device__ __forceinline__ bool find_segment(const int* cu, int sequences, long long tokens, int L, int slot, Segment* s) {
  // A wavefront looks at 64 sequences at once: one load where there are no more than that, and few otherwise.
  const int t = (int)tokens, lane = threadIdx.x % 64;
  int lo = 0, width = sequences, a, b;
  for (;;) {
    const int step = (width + 63) / 64, at = lo + lane * step;
    const bool in = lane * (long long)step < width;
    const int first = in ? min(max(cu[at], 0), t) : 0, end = in ? cu[at + 1] : 0;
    const int before = __popcll(__ballot(in && first / (uint32_t)L + at <= (uint32_t)slot));
    const int k = max(before - 1, 0);
    lo += k * step;
    if (step == 1) {
      a = __builtin_amdgcn_readlane(first, k);
      b = min(max(__builtin_amdgcn_readlane(end, k), a), t);
      break;
    }
    width = min(step, width - k * step);
  }
  return set_segment(lo, slot - (int)(a / (uint32_t)L + lo), a, b, L, s);
}

// The segment that a scan's workgroups take `at`-th: where they are more than run at once the longest first, so that the last
// to start are short ones (13 prompts of 35 to 1881 tokens, 32 heads of 128: states 47 -> 39 us, scan 122 -> 120; the order itself
// costs a workgroup a microsecond, and 6 training sequences of 762 to 2716 have 464 -> 490 us with it).  More than 64 sequences even out by themselves and keep their order.
__device__ __forceinline__ bool find_in_order(const int* cu, int sequences, long long tokens, int L, bool several, int at,
                                              Segment* s) {
  if (!several || sequences == 1 || sequences > 64) return find_segment(cu, sequences, tokens, L, at, s);
  const int lane = threadIdx.x % 64;
  int a = 0, b = 0, each = 0, count = 0, before = 0;
  if (lane < sequences) {
    seq_bounds(cu, lane, tokens, &a, &b);
    count = max(1, segments_of(b - a, L, &each));
  }
  for (int i = 0; i < sequences; ++i) {
    const int other = __builtin_amdgcn_readlane(each, i), n = __builtin_amdgcn_readlane(count, i);
    before += other > each || (other == each && i < lane) ? n : 0;
  }
  const uint64_t it = __ballot(lane < sequences && at >= before && at < before + count);
  if (it == 0) return false;
  const int k = __ffsll((unsigned long long)it) - 1;
  return set_segment(k, at - __builtin_amdgcn_readlane(before, k), __builtin_amdgcn_readlane(a, k), __builtin_amdgcn_readlane(b, k), L, s);
}

// Place of the state between segments c and c + 1 of a sequence that starts at `start`: a sequence of n tokens has at most
// n / L of them (rounded down), so the next one's places are behind.
__device__ __forceinline__ long long bound_of(int start, int c, int L) { return start / (uint32_t)L + c; }

// Whether an earlier sequence uses this slot, and the next one that does (or `sequences`).  Every wavefront for itself.
__device__ __forceinline__ void same_slot(const int* slots, int sequences, int seq, bool* earlier, int* next) {
  const int lane = threadIdx.x % 64, slot = slots[seq];
  int before = 0, after = sequences;
  for (int i = lane; i < sequences; i += 64)
    if (slots[i] == slot) {
      before |= i < seq;
      if (i > seq && i < after) after = i;
    }
  *earlier = __ballot(before) != 0;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) after = min(after, __shfl_xor(after, m));
  *next = __builtin_amdgcn_readfirstlane(after);
}

// A state element (i, j) lies at i * si + j * sj.
template <int KS, int CT>
struct State {
  f32x4 t[KS * 2][CT];                          // rows 32 ks + 8 lg + 4 half + r of column 16 or 32 w + ...

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < KS * 2; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) t[i][j] = zero4();
  }
  // From or to [rows][columns] in memory, or its transpose (TR).  What is behind either width is zero, or dropped: its lanes'
  // offsets are kNowhere, and the scalar offsets of the others stay inside.
  template <bool LOAD, bool TR>
  __device__ __forceinline__ void move(float* p, int rows, int columns, int w, uint32_t lane) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    asm volatile("" : "+v"(lane));               // offsets are made here and not kept in registers through the chunks
    const uint32_t lr = lane % 16, lg = lane / 16;
    const buf_t b = buf(p, (uint32_t)rows * columns * 4);
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      const uint32_t col = CT == 2 ? 32 * w + 8 * (lr / 4) + 4 * j + lr % 4 : 16 * w + lr;
      const uint32_t base = TR ? (uint32_t)(col * rows + 8 * lg) * 4 : (uint32_t)(8 * lg * columns + col) * 4;
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) {
        const uint32_t at = (int)col < columns && (int)(32 * (i / 2) + 8 * lg) < rows ? base : kNowhere;
        const int row = 32 * (i / 2) + 4 * (i % 2);
        if constexpr (TR) {
          if constexpr (LOAD) t[i][j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at, row * 4, 0));
          else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, t[i][j]), b, at, row * 4, 0);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int to = (row + r) * columns * 4;
            if constexpr (LOAD) t[i][j][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, at, to, 0));
            else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(t[i][j][r]), b, at, to, 0);
          }
        }
      }
    }
  }
};

// What a scan keeps in LDS.
template <int NT, int KS, int CT, bool OUT, bool DOT>
struct ScanSpace {
  static constexpr int NW = kScanThreads / 64;
  static constexpr int CH = NT == 1 ? 64 : 32, RT = CH / 16, K2 = CH / 32;   // tokens of a chunk, in tiles of 16 and 32
  static constexpr int U = KS * 4, UC = NW * CT * 2;                         // 16-byte units of a row of A and B, and of C
  static constexpr int GR = NT == 1 ? 4 : 2;                                 // chunks whose gates are there at once
  alignas(16) char As[OUT ? NT * CH * U * 16 : 16];
  alignas(16) char Bs[NT * CH * U * 16];
  alignas(16) char Cs[NT * CH * UC * 16];
  alignas(16) bh P[OUT ? RT * K2 * kTerms * 512 : 8];
  alignas(16) float Gh[GR][CH];                // G = Gh + Gl to 48 bits: its differences have the accuracy of fp32
  alignas(16) float Gl[GR][CH];
  alignas(16) float fo[GR][CH];
  alignas(16) float fs[GR][CH];
  float all[GR];
  float red[DOT ? NW : 1][DOT ? CH : 1];
  float own[DOT ? CH : 1];                     // P's diagonal
  double totals[OUT ? 1 : NW];
};

// The arguments of one of a kernel's scans, read where that scan begins: those of all of them at once do not fit the scalar
// registers.  They lie `offset` bytes behind the kernel's first argument.
__device__ __forceinline__ ScanArgs scan_args_at(uint32_t offset) {
  auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr() + offset;
  asm volatile("" : "+s"(p));
  return *(const ScanArgs*)(const char*)p;
}

// Workgroups of a scan: one for each (segment, value head), or (segment, key head) where the heads' outputs are summed.
__host__ __device__ inline uint32_t scan_blocks(const ScanArgs& s) {
  return (uint32_t)(s.slots * s.hk + 7) / 8 * 8 * (s.part ? 1 : s.rep);
}

// One workgroup's scan.  Units of the same remainder mod 8 run on one XCD: `unit` is a (slot, key head), `part` one of its value
// heads (all of them, one after another, where their outputs are summed).
template <int NT, int KS, int CT, bool REV, bool OUT, bool DOT>
__device__ __forceinline__ void scan_item(const ScanArgs& s, uint32_t unit, int part, ScanSpace<NT, KS, CT, OUT, DOT>& z) {
  using Z = ScanSpace<NT, KS, CT, OUT, DOT>;
  constexpr int TH = kScanThreads, NW = Z::NW, CH = Z::CH, RT = Z::RT, K2 = Z::K2, U = Z::U, UC = Z::UC, GR = Z::GR;
  constexpr int es = NT == 1 ? 2 : 4;
  constexpr bool TR = OUT && REV != DOT;       // dq and dk: states are [J][I] in memory, and shared heads' outputs are summed
  auto& As = z.As;
  auto& Bs = z.Bs;
  auto& Cs = z.Cs;
  auto& P = z.P;
  auto& Gh = z.Gh;
  auto& Gl = z.Gl;
  auto& fo = z.fo;
  auto& fs = z.fs;
  auto& all = z.all;
  auto& red = z.red;
  auto& own = z.own;
  const uint32_t tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid / 64);
  uint32_t lane = tid % 64;
  const int I = s.b.width, J = s.c.width, hv = s.hk * s.rep;
  if (unit >= (uint32_t)(s.slots * s.hk)) return;
  const uint32_t order = unit / (uint32_t)s.hk;
  const int kh = unit - order * s.hk;
  const bool summed = TR && s.part;
    Segment seg;
    if (!find_in_order(s.cu, s.sequences, s.tokens, s.L, s.slots * hv > kAtOnce, order, &seg)) return;
    const size_t cell = (size_t)I * J;
    const bool in_place = s.from && s.from == s.to;
    bool keep = true;                           // the state after the last segment
    int next = s.sequences;
    long long row = seg.seq;
    if (s.state_slots) {
      row = s.state_slots[seg.seq];
      if (row < 0 || row >= s.state_rows) row = -1;
      else {
        bool earlier;
        same_slot(s.state_slots, s.sequences, seg.seq, &earlier, &next);
        if (!in_place) {
          keep = next == s.sequences;
          next = s.sequences;
        } else if (earlier || (next < s.sequences && (!OUT || seg.c > 0))) {
          return;                               // the first of them runs them all, one after another
        }
      }
    }
    if constexpr (!OUT) {
      if (REV ? seg.c == 0 : seg.c == seg.count - 1) return;
    }
    for (int r = summed ? 0 : part; r < (summed ? s.rep : part + 1); ++r) {
    const int h = kh * s.rep + r;
    State<KS, CT> S;
    double total = 0;                           // of the gates of the wavefront's chunks
    if constexpr (!OUT) {
      S.zero();
    } else {
      float* p = const_cast<float*>(s.from);
      const bool inner = REV ? seg.c < seg.count - 1 : seg.c > 0;
      if (inner) p = s.between + (size_t)(bound_of(seg.start, REV ? seg.c : seg.c - 1, s.L) * hv + h) * cell;
      else if (in_place && seg.count > 1 && next == s.sequences) p = s.firsts + (size_t)(bound_of(seg.start, 0, s.L) * hv + h) * cell;
      else if (p && row >= 0) p += ((size_t)row * hv + h) * cell;
      else p = nullptr;
      if (p) S.template move<true, TR>(p, I, J, w, lane);
      else S.zero();
    }
    const bool serial = next < s.sequences;     // in place, with others that name this slot behind it
    int seq = seg.seq, first = seg.first, n = serial ? seg.length : seg.n;
    for (;;) {
      const int chunks = (n + CH - 1) / CH;
      Stage<NT, U, CH, TH> ra, rb;
      Stage<NT, UC, CH, TH> rc;
      float gate = 0.f;
      // operands (bits: a, b, c) of the i-th chunk in the scan's order; behind the last: nothing
      auto fetch = [&](int i, int which) {
        const int k = i < chunks ? (REV ? chunks - 1 - i : i) : 0, t0 = first + k * CH;
        const int m = i < chunks ? min(CH, n - k * CH) : 0;
        auto rows = [&](const Operand& o) {
          return buf(o.p + (size_t)t0 * o.row + (size_t)(o.shared ? kh : h) * o.width * es,
                     m > 0 ? (uint32_t)(m - 1) * o.row + o.width * es : 0);
        };
        if constexpr (OUT) {
          if (which & 1) ra.load(rows(s.a), s.a.row, I, tid);
        }
        if (which & 2) rb.load(rows(s.b), s.b.row, I, tid);
        if (which & 4) rc.load(rows(s.c), s.c.row, J, tid);
      };
      // GR chunks at a time, the wavefront's one of them: its gates, loaded long before, then their sums and factors.
      auto fetch_gates = [&](int i) {
        const int k = i < chunks ? (REV ? chunks - 1 - i : i) : 0, t0 = first + k * CH;
        const int m = i < chunks ? min(CH, n - k * CH) : 0;
        gate = (int)lane < m ? s.g[s.fixed ? h : (size_t)(t0 + lane) * hv + h] : 0.f;
      };
      auto gates = [&] {
        gate = gate < kLowestGate ? kLowestGate : gate;
        const double G = prefix_sum(gate * 1.4426950408889634);         // in units of log 2
        const double Gn = last_lane(G);
        const float up = exp2_of((float)G), down = exp2_of((float)(Gn - G));
        const float hi = (float)G;
        if (lane < CH) {
          Gh[w][lane] = hi;
          Gl[w][lane] = (float)(G - hi);
          fo[w][lane] = REV ? down : s.scale * up;
          fs[w][lane] = REV ? s.scale * up : down;
        }
        if (lane == 0) all[w] = exp2_of((float)Gn);
        total += Gn;
      };
      auto dot_of = [&] {                       // a token's sum over the columns
        float x = red[0][tid];
#pragma unroll
        for (int j = 1; j < NW; ++j) x += red[j][tid];
        return x;
      };
      if (w < GR) fetch_gates(w);
      fetch(0, 7);
      for (int i = 0; i < chunks; ++i) {
        const int k = REV ? chunks - 1 - i : i, at = i % GR;
        const int t0 = first + k * CH, m = min(CH, n - k * CH);
        asm volatile("" : "+v"(lane));         // addresses in LDS are made in each chunk and not kept in registers
        const uint32_t lr = lane % 16, lg = lane / 16;
        __syncthreads();                        // the previous tiles and gates have been read
        if constexpr (OUT) ra.store(As, tid);
        rb.store(Bs, tid);
        if constexpr (!OUT) rc.store(Cs, tid);
        if (at == 0 && w < GR) {
          gates();
          fetch_gates(i + GR + w);
        }
        if constexpr (DOT) {
          if (i && tid < CH) {
            const int b0 = REV ? t0 + CH : t0 - CH;
            if (b0 + (int)tid < first + n) s.dot[(size_t)h * s.tokens + b0 + tid] = dot_of();
          }
        }
        __syncthreads();

        f32x4 o[RT][CT];
        if constexpr (OUT) {
          fetch(i + 1, 3);
          rc.store(Cs, tid);
          // P: rows x of A, y of B; a lane holds four y of one x, which is half a vector of P's fragment.  Its blocks above the
          // diagonal that share a fragment with one below are formed too, as zeros: three blocks a wavefront (one of four with
          // chunks of 32).  Their gates run between the products of the state's part, out = A S, whose operands are read and
          // split a step ahead.
          constexpr int T = RT == 4 ? 3 : 1;
          int tx[T], ty[T];
          f32x4 d[T];
#pragma unroll
          for (int t = 0; t < T; ++t) {
            if constexpr (RT == 4) {
              tx[t] = w < 2 || t == 0 ? 2 + (w & 1) : w & 1;
              ty[t] = w < 2 ? t : t == 0 ? 3 : t - 1;
            } else {
              tx[t] = w / 2;
              ty[t] = w % 2;
            }
            if constexpr (REV) {
              tx[t] = RT - 1 - tx[t];
              ty[t] = RT - 1 - ty[t];
            }
            d[t] = zero4();
          }
          Frag<NT> fa[2][T], fb[2][T], af[2][RT];
          const auto blocks_at = [&](int ks) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
              fb[ks % 2][t] = row_frag<NT, U, CH>(Bs, 16 * ty[t], ks, lane);
              fa[ks % 2][t] = row_frag<NT, U, CH>(As, 16 * tx[t], ks, lane);
            }
          };
          const auto rows_at = [&](int ks) {
#pragma unroll
            for (int x = 0; x < RT; ++x) af[ks % 2][x] = row_frag<NT, U, CH>(As, 16 * x, ks, lane);
          };
          const auto terms_of = [&](int ks, int j) {
            const f32x4 u = S.t[2 * ks][j], v = S.t[2 * ks + 1][j];
            const float e[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
            return split8<kTerms>(e);
          };
          blocks_at(0);
          fence();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS) blocks_at(ks + 1);
            else rows_at(0);
            fence();
#pragma unroll
            for (int t = 0; t < T; ++t) d[t] = mma<NT, NT>(fb[ks % 2][t], fa[ks % 2][t], d[t]);
            fence();
          }
          fetch(i + 1, 4);
          float hx, lx;
          f32x4 hy, ly;
          const auto gates_at = [&](int t) {
            const uint32_t x = 16 * tx[t] + lr, y = 16 * ty[t] + 4 * lg;
            hx = Gh[at][x];
            lx = Gl[at][x];
            hy = *reinterpret_cast<const f32x4*>(&Gh[at][y]);
            ly = *reinterpret_cast<const f32x4*>(&Gl[at][y]);
          };
          const auto gate_block = [&](int t) {
            const uint32_t x = 16 * tx[t] + lr, y = 16 * ty[t] + 4 * lg;
            float p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float e = REV ? (hy[r] - hx) + (ly[r] - lx) : (hx - hy[r]) + (lx - ly[r]);
              // The exponent carries the mask: no branch around the exponential.  Outputs mask the product too, which may be of a
              // later key that is not finite; gradients, which such a key spoils anyhow, do not (it costs them registers, 10 %).
              const bool in = REV ? y + r >= x + DOT : y + r + DOT <= x;
              p[r] = s.scale * exp2_of(in ? e : -INFINITY) * (in || REV || DOT ? d[t][r] : 0.f);
              if constexpr (DOT) {
                if (y + r == x) own[x] = s.scale * d[t][r];
              }
            }
            uint32_t p0[kTerms], p1[kTerms];
            split2<kTerms>(p[0], p[1], p0);
            split2<kTerms>(p[2], p[3], p1);
            bh* to = P + (tx[t] * K2 + ty[t] / 2) * kTerms * 512 + (((ty[t] & 1) * 2 + lg / 2) * 16 + lr) * 8 + (lg & 1) * 4;
#pragma unroll
            for (int i2 = 0; i2 < kTerms; ++i2) *reinterpret_cast<uint2*>(to + i2 * 512) = make_uint2(p0[i2], p1[i2]);
          };
#pragma unroll
          for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int j = 0; j < CT; ++j) o[x][j] = zero4();
          Frag<kTerms> sf[2];
          sf[0] = terms_of(0, 0);
          gates_at(0);
          constexpr int N = KS * CT, every = N > T ? N / T : 1;         // steps, and steps between P's blocks
#pragma unroll
          for (int n = 0; n < KS * CT; ++n) {
            const int ks = n / CT, j = n % CT;
            if (j == 0 && ks + 1 < KS) rows_at(ks + 1);
            if (n + 1 < KS * CT) sf[(n + 1) % 2] = terms_of((n + 1) / CT, (n + 1) % CT);
            fence();
#pragma unroll
            for (int x = 0; x < RT; ++x) o[x][j] = mma<kTerms, NT>(sf[n % 2], af[ks % 2][x], o[x][j]);
            // T blocks over the KS * CT steps
#pragma unroll
            for (int t = 0; t < T; ++t)
              if (n == (N >= T ? t * every : 0)) {
                gate_block(t);
                if (t + 1 < T) gates_at(t + 1);
              }
            fence();
          }
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            const float f = fo[at][16 * x + lr];
#pragma unroll
            for (int j = 0; j < CT; ++j) o[x][j] *= f;
          }
          __syncthreads();                      // P and C are there
        } else {
          fetch(i + 1, 6);
        }
        // Columns of C, as they are and, times the decay up to the chunk's end, as they go into the state: formed between the
        // products of P C and of the state's update, whose operands are read a step ahead.
        Frag<NT> cf[K2][CT], bf[3];
        Frag<kTerms> pf[2];
        Frag<3> vf[2][CT];
        float decays[2][8];
        const uint32_t piece = lane % 4;
        const auto decays_at = [&](int k2) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<f32x4*>(&decays[k2 % 2][4 * e]) = *reinterpret_cast<const f32x4*>(&fs[at][32 * k2 + 8 * lg + 4 * e]);
        };
        const auto columns_of = [&](int k2, int j, int pair) {        // values 2 pair, 2 pair + 1 of the eight
          float x[2] = {0.f, 0.f};
#pragma unroll
          for (int t = NT - 1; t >= 0; --t) {
            const uint4 b = as_bits(cf[k2][j].t[t]);
            const uint32_t word = pair == 0 ? b.x : pair == 1 ? b.y : pair == 2 ? b.z : b.w;
            x[0] += __uint_as_float(word << 16);
            x[1] += __uint_as_float(word & 0xffff0000u);
          }
          uint32_t v[3];
          split2<3>(x[0] * decays[k2 % 2][2 * pair], x[1] * decays[k2 % 2][2 * pair + 1], v);
#pragma unroll
          for (int t = 0; t < 3; ++t) {
            uint4 b = as_bits(vf[k2 % 2][j].t[t]);
            (pair == 0 ? b.x : pair == 1 ? b.y : pair == 2 ? b.z : b.w) = v[t];
            vf[k2 % 2][j].t[t] = as_frag(b);
          }
        };
        // P's fragments in turn: tokens 16 x .., by 32 k2 ..
        constexpr int PN = RT == 4 ? 6 : 2;
        const auto p_x = [](int n) { return RT == 4 ? (REV ? (n < 4 ? n / 2 : n - 2) : (n < 2 ? n : n / 2 + 1)) : n; };
        const auto p_k2 = [](int n) { return RT == 4 ? (REV ? (n < 4 ? n % 2 : 1) : (n < 2 ? 0 : n % 2)) : 0; };
        const auto p_at = [&](int n) {
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
            pf[n % 2].t[t] = as_frag(*reinterpret_cast<const uint4*>(P + ((p_x(n) * K2 + p_k2(n)) * kTerms + t) * 512 + lane * 8));
        };
        const auto b_at = [&](int n) {          // step n: rows of tile n % (2 KS), tokens of half n / (2 KS)
          const int i2 = n % (2 * KS);
          bf[n % 3] = column_frag<NT, U, CH>(Bs, n / (2 * KS), 4 * (i2 / 2) + piece, 8 * (i2 % 2), lane);
        };
#pragma unroll
        for (int k2 = 0; k2 < K2; ++k2)
#pragma unroll
          for (int j = 0; j < CT; ++j)
            cf[k2][j] = column_frag<NT, UC, CH>(Cs, k2, CT == 2 ? 4 * w + piece : 2 * w + piece / 2, CT == 2 ? 8 * j : piece % 2 * 8, lane);
        decays_at(0);
        // Shared heads: the sums so far in fp32, and the last head's go out
        const bool last = !summed || r == s.rep - 1;
        char* const out = last ? s.out : reinterpret_cast<char*>(s.part);
        const uint32_t part_row = (uint32_t)(s.hk * J) * 4, out_row = last ? s.out_row : part_row, ob = last ? s.out_bytes : 4;
        const uint32_t col = CT == 2 ? 32 * w + 8 * lg : 16 * w + 4 * lg;
        // What the outputs of 16 tokens need: their rows of d, and the sums so far
        Values<3, 4 * CT> sums[TR ? 2 : 1];
        Values<NT, 4 * CT> drow[DOT ? 2 : 1];
        const auto out_at = [&](int x) {
          if constexpr (DOT) {
            const buf_t from = buf(s.d.p + (size_t)t0 * s.d.row + (size_t)(s.d.shared ? kh : h) * J * es, (uint32_t)(m - 1) * s.d.row + J * es);
            drow[x % 2].load(from, (int)col < J ? (16 * x + lr) * s.d.row + col * es : kNowhere);
          }
          if constexpr (TR) {
            if (summed && r > 0) {
              const buf_t from = buf(reinterpret_cast<char*>(s.part) + (size_t)t0 * part_row + (size_t)kh * J * 4, (uint32_t)(m - 1) * part_row + J * 4);
              sums[x % 2].load(from, (int)col < J ? (16 * x + lr) * part_row + col * 4 : kNowhere);
            }
          }
        };
        const auto rows_out = [&](int x) {        // outputs of 16 tokens
          const buf_t to = buf(out + (size_t)t0 * out_row + (size_t)(summed ? kh : h) * J * ob, (uint32_t)(m - 1) * out_row + J * ob);
          float v[4 * CT];
#pragma unroll
          for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * j + e] = o[x][j][e];
          float f;                                // P's diagonal and the token's row of C
          uint32_t c[NT][2 * CT];
          if constexpr (DOT) {
            const uint32_t row = 16 * x + lr, unit = CT == 2 ? 4 * w + lg : 2 * w + lg / 2;
            const char* const from = Cs + row * UC * 16 + (unit ^ swizzle<UC>(row)) * 16 + (CT == 2 ? 0 : lg % 2 * 8);
            f = own[row];
#pragma unroll
            for (int t = 0; t < NT; ++t) __builtin_memcpy(c[t], __builtin_assume_aligned(from + t * CH * UC * 16, 8 * CT), 8 * CT);
          }
          if constexpr (DOT) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4 * CT; ++e) sum = fmaf(v[e], drow[x % 2].value(e), sum);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lg == 0) red[w][16 * x + lr] = sum;
          }
          if constexpr (DOT) {                    // what the token has of itself, behind its dot product
#pragma unroll
            for (int t = NT - 1; t >= 0; --t)
#pragma unroll
              for (int e = 0; e < 4 * CT; ++e)
                v[e] = fmaf(f, __uint_as_float(e % 2 ? c[t][e / 2] & 0xffff0000u : c[t][e / 2] << 16), v[e]);
          }
          if constexpr (TR) {
            if (summed && r > 0) {
#pragma unroll
              for (int e = 0; e < 4 * CT; ++e) v[e] += sums[x % 2].value(e);
            }
          }
          const uint32_t off = (int)col < J ? (16 * x + lr) * out_row + col * ob : kNowhere;
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
          if (ob == 2) {
            uint32_t b[2 * CT];
#pragma unroll
            for (int e = 0; e < 2 * CT; ++e) {
              uint32_t one[1];
              split2<1>(v[2 * e], v[2 * e + 1], one);
              b[e] = one[0];
            }
            if constexpr (CT == 2) __builtin_amdgcn_raw_buffer_store_b128(u32x4{b[0], b[1], b[2], b[3]}, to, off, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b64(u32x2{b[0], b[1]}, to, off, 0, 0);
          } else {
#pragma unroll
            for (int j = 0; j < CT; ++j)
              __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                           __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])},
                                                     to, off + 16 * j, 0, 0);
          }
        };
        const float decay = all[at];
        if constexpr (OUT) {
          p_at(0);
          fence();
#pragma unroll
          for (int n = 0; n < PN; ++n) {
            if (n + 1 < PN) p_at(n + 1);
            else b_at(0);
            if (n + 1 == PN) b_at(1);
            fence();
#pragma unroll
            for (int j = 0; j < CT; ++j) o[p_x(n)][j] = mma<NT, kTerms>(cf[p_k2(n)][j], pf[n % 2], o[p_x(n)][j]);
#pragma unroll
            for (int c = n * 4 * CT / PN; c < (n + 1) * 4 * CT / PN; ++c) columns_of(0, c / 4, c % 4);
            fence();
          }
        } else {
          b_at(0);
          b_at(1);
#pragma unroll
          for (int n = 0; n < 4 * CT; ++n) columns_of(0, n / 4, n % 4);
        }
        if constexpr (OUT) {
          out_at(0);
          out_at(1);
        }
#pragma unroll
        for (int n = 0; n < K2 * 2 * KS; ++n) {
          const int i2 = n % (2 * KS), k2 = n / (2 * KS);
          if (n + 2 < K2 * 2 * KS) b_at(n + 2);
          if (i2 == 0 && k2 + 1 < K2) decays_at(k2 + 1);
          if (k2 == 0) {
#pragma unroll
            for (int j = 0; j < CT; ++j) S.t[i2][j] *= decay;
          }
          fence();
#pragma unroll
          for (int j = 0; j < CT; ++j) S.t[i2][j] = mma<NT, 3>(bf[n % 3], vf[k2 % 2][j], S.t[i2][j]);
          if (k2 + 1 < K2) {
#pragma unroll
            for (int c = i2 * 4 * CT / (2 * KS); c < (i2 + 1) * 4 * CT / (2 * KS); ++c) columns_of(k2 + 1, c / 4, c % 4);
          }
          if constexpr (OUT) {
            constexpr int N = K2 * 2 * KS;                             // outputs in the later steps
#pragma unroll
            for (int x = 0; x < RT; ++x)
              if (n == N - 1 - (RT - 1 - x) * (N * 3 / (4 * RT))) {
                rows_out(x);
                if (x + 2 < RT) out_at(x + 2);
              }
          }
          fence();
        }
      }
      if constexpr (DOT) {
        __syncthreads();
        const int b0 = REV ? first : first + (chunks - 1) * CH;
        if (chunks > 0 && tid < CH && b0 + (int)tid < first + n)
          s.dot[(size_t)h * s.tokens + b0 + tid] = dot_of();
      }
      if (!serial || next >= s.sequences) break;
      seq = next;
      bool earlier;
      same_slot(s.state_slots, s.sequences, seq, &earlier, &next);
      int a, b;
      seq_bounds(s.cu, seq, s.tokens, &a, &b);
      first = __builtin_amdgcn_readfirstlane(a);
      n = __builtin_amdgcn_readfirstlane(b - a);
    }
    if constexpr (!OUT) {
      S.template move<false, TR>(s.between + (size_t)(bound_of(seg.start, REV ? seg.c - 1 : seg.c, s.L) * hv + h) * cell, I, J,
                                 w, lane);
      if (lane == 0) z.totals[w] = total;
      __syncthreads();
      if (tid == 0) s.decay[(size_t)seg.slot * hv + h] = exp2_of((float)(z.totals[0] + z.totals[1] + z.totals[2] + z.totals[3]));
    } else if (s.to && keep && row >= 0 && (serial || (REV ? seg.c == 0 : seg.c == seg.count - 1))) {
      S.template move<false, TR>(s.to + ((size_t)row * hv + h) * cell, I, J, w, lane);
    }
    }
}

template <int NT, int KS, int CT>
__global__ __launch_bounds__(kScanThreads, 2) void linear_scan_kernel(ScanArgs s) {
  __shared__ ScanSpace<NT, KS, CT, true, false> z;
  const uint32_t blocks = scan_blocks(s);
  for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    const uint32_t group = block / 8 / (uint32_t)s.rep;
    scan_item<NT, KS, CT, false, true, false>(s, group * 8 + block % 8, block / 8 - group * s.rep, z);
  }
}

// ---------------------------------------------------------------- host

// Calls f with the steps of 32 rows and the column tiles of a wavefront that widths up to 32, 64 and 128 take, as types.
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
void by_width(int width, F f) {
  if (width <= 32) f(Int<1>(), Int<1>());
  else if (width <= 64) f(Int<2>(), Int<1>());
  else f(Int<4>(), Int<2>());
}

inline dim3 scan_grid(long long blocks) { return dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)); }

}  // namespace gdn
