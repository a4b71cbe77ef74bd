// The gated delta rule over packed sequences, chunked: chunk preparation and
// the forward scan.
//
// Per chunk of 64 tokens and value head, with the cumulative log-gate G, E_ij =
// e^(G_i - G_j) for i >= j (every exponent <= 0 on the documented domain; G is
// summed in fp64, so strong gates cost no accuracy) and the state S0 before it:
//     B_ij = E_ij k_i.k_j (i > j),  T' = (I + B diag(beta))^-1,  P_ij = E_ij q_i.k_j (i >= j)
//     e = T' (V - e^G K S0),  U = beta e
//     O = e^G Q S0 + P U,     S1 = e^Gn S0 + K^T (e^(Gn - G) U)
// prep_kernel forms T', P and the gate factors of every chunk in parallel;
// scan_kernel runs the chunks of a sequence in order.  The columns of the state
// (of V, e, U, O) evolve independently, so a workgroup carries 16 of them.
#include "gdn_packed.h"

namespace gdn {
namespace {

constexpr int kLd = 68;     // row stride (floats) of a 64 x 64 fp32 tile in LDS

// Gates below this are this: e^-10000 is 0 in fp32, and G stays finite for -inf.
constexpr float kLowestGate = -10000.f;

// Four accumulator values of rows (k) row0 .. row0 + 3 of a column, as three terms
// into stored fragments [column tile][row half]: the same places as in an LDS tile.
__device__ __forceinline__ void store_quad(uint4* frags, int tile, int column, int row, const float (&x)[4]) {
  uint32_t lo[3], hi[3];
  split2<3>(x[0], x[1], lo);
  split2<3>(x[2], x[3], hi);
  bh* to = reinterpret_cast<bh*>(frags + (size_t)(tile * 2 + row / 32) * 3 * 64) + put_place(column, row % 32);
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(to + i * 512) = make_uint2(lo[i], hi[i]);
}

// One workgroup per cell; wavefront w has rows (tokens) 16 w .. of the 64 x 64
// matrices.  Accumulators hold four rows of a column, which is half a vector of
// the transposed matrix's fragment; so the products are taken in the order that
// makes each result leave its registers as it is stored.  What it reads and
// writes bounds it: 32768 tokens of 35 heads of 64 274 us, some 67 KB a cell, 4.4
// TB/s.  Of the 128 registers that four workgroups a CU leave a lane, d_k above
// 64 spills 10.
template <int NT, int DKP, bool GRAD>
__global__ __launch_bounds__(256, NT == 1 && !GRAD ? 4 : 2) void packed_prep_kernel(SeqProblem p, PackedTensors t, PackedSpace ws, long long slots, int heads) {
  constexpr int NM = GRAD ? 2 : 1, KS = DKP / 32;
  constexpr uint32_t es = NT == 1 ? 2 : 4;
  __shared__ double Gb[2][kC];
  __shared__ float bb[2][kC];
  __shared__ __align__(16) float A[NM][kC][kLd];
  __shared__ __align__(16) float T[NM][kC][kLd];
  const int tid = threadIdx.x, lane = tid % 64, w = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lr = lane % 16, lg = lane / 16;
  const int rep = p.hv / p.hk;
  const int share = GRAD ? heads : 1;                 // value heads of a workgroup
  const int parts = p.hv / share;
  const long long items = slots * parts;
  const uint32_t ks_b = (uint32_t)p.ks * es, qs_b = (uint32_t)p.qs * es;

  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int h0 = (int)(item % parts) * share, kh = h0 / rep;
    const long long slot = item / parts;
    int seq, first, n;
    if (!find_chunk(t.cu, p.sequences, p.tokens, slot, &seq, &first, &n)) continue;   // uniform over the workgroup
    first = __builtin_amdgcn_readfirstlane(first);
    n = __builtin_amdgcn_readfirstlane(n);
    const buf_t kb = buf(static_cast<const char*>(t.k) + ((size_t)first * p.ks + kh * p.dk) * es, span(n, ks_b, p.dk * es));
    const buf_t qb = buf(static_cast<const char*>(t.q) + ((size_t)first * p.qs + kh * p.dk) * es, span(n, qs_b, p.dk * es));
    auto row_frag = [&](buf_t base, uint32_t stride, int tile, int ks) {
      const int c = ks * 32 + lg * 8;
      return frag_of<NT>(raw_at<NT>(base, c < p.dk ? (tile * 16 + lr) * stride + c * es : kNowhere));
    };
    auto gates_of = [&](int h) {                        // by one wavefront, into the buffers of the head's turn
      const size_t at = (size_t)(first + lane) * p.hv + h;
      float g = lane < n ? t.g[at] : 0.f;
      g = g < kLowestGate ? kLowestGate : g;
      double G = g * 1.4426950408889634;              // in units of log 2: exp2 of the differences
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(G, m);
        if (lane >= m) G += o;
      }
      Gb[(h - h0) & 1][lane] = G;
      bb[(h - h0) & 1][lane] = lane < n ? t.beta[at] : 0.f;
    };
    __syncthreads();                                  // the previous cell's tiles have been read
    if (w == 0) gates_of(h0);
    // K K^T as (rows w, columns j); Q K^T the same way for P^T, or as (rows j, columns w) for P
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero4();
    uint4* ktp = ws.kt + ((size_t)slot * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
    uint4* qtp = ws.qt + ((size_t)slot * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
    // Rows of an operand fragment to fragments of its transpose: a product with the identity, exact for each bf16 term.
    auto transpose = [&](const Frag<NT>& f, uint4* to, int ks) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = lg * 8 + j == half * 16 + lr ? 1.f : 0.f;
        const Frag<1> one = split8<1>(e);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const f32x4 d = mfma(f.t[i], one.t[0], zero4());
          uint32_t v[2][1];
          split2<1>(d[0], d[1], v[0]);
          split2<1>(d[2], d[3], v[1]);
          const int row = 16 * w + 4 * lg;
          bh* o = reinterpret_cast<bh*>(to + ((size_t)((ks * 2 + half) * 2 + row / 32) * NT + i) * 64) + put_place(lr, row % 32);
          *reinterpret_cast<uint2*>(o) = make_uint2(v[0][0], v[1][0]);
        }
      }
    };
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<NT> ak = row_frag(kb, ks_b, w, ks), aq = row_frag(qb, qs_b, w, ks);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          const Frag<NT> b = j == w ? ak : row_frag(kb, ks_b, j, ks);
          kk[j] = mma<NT, NT>(ak, b, kk[j]);
          qk[j] = GRAD ? mma<NT, NT>(aq, b, qk[j]) : mma<NT, NT>(b, aq, qk[j]);
        }
      if (h0 % rep == 0) {
        transpose(ak, ktp, ks);
        if constexpr (GRAD) transpose(aq, qtp, ks);
      }
    }
    for (int h = h0; h < h0 + share; ++h) {
      const long long cell = GRAD ? slot * p.hv + h : item;
      const double* Gs = Gb[(h - h0) & 1];
      const float* bs = bb[(h - h0) & 1];
      __syncthreads();                                // the gates are there, the previous head's tiles have been read
      if (w == 3 && h + 1 < h0 + share) gates_of(h + 1);
      {
        uint4* pp = ws.p + (size_t)cell * kTri * 3 * 64;
        double Gr[4];
        float br[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          Gr[r] = Gs[16 * w + 4 * lg + r];
          br[r] = bs[16 * w + 4 * lg + r];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j <= w) {
            const int c = 16 * j + lr;
            const double Gc = Gs[c];
            const float bc = bs[c];
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int i = 16 * w + 4 * lg + r;
              const float E = i >= c ? exp2_of((float)(Gr[r] - Gc)) : 0.f;
              const float b = i > c ? E * kk[j][r] : 0.f;
              A[0][i][c] = b * bc;
              if constexpr (GRAD) {
                A[NM - 1][i][c] = b * br[r];
                x[r] = E * qk[j][r];
              } else {
                // qk[j] holds rows 16 j + 4 lg + r of K and the row 16 w + lr of Q
                const int pi = 16 * w + lr, pj = 16 * j + 4 * lg + r;
                x[r] = pi >= pj ? exp2_of((float)(Gs[pi] - Gs[pj])) * qk[j][r] : 0.f;
              }
            }
            if constexpr (GRAD) store_quad(pp, j, lr, 16 * w + 4 * lg, x);                // P^T: row tile j, rows i
            else store_quad(pp, w, lr, 16 * j + 4 * lg, x);                               // P: row tile w, columns j
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              T[0][16 * w + 4 * lg + r][16 * j + lr] = 0.f;
              if constexpr (GRAD) T[NM - 1][16 * w + 4 * lg + r][16 * j + lr] = 0.f;
            }
            // the fragments on the diagonal's block row hold a block above it
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            if (j / 2 == w / 2) {
              if constexpr (GRAD) store_quad(pp, j, lr, 16 * w + 4 * lg, z);
              else store_quad(pp, w, lr, 16 * j + 4 * lg, z);
            }
          }
        }
      }
      __syncthreads();
      // (I + A)^-1: the 16 x 16 diagonal blocks by substitution, lane c a column
      {
        const int m = GRAD ? lg & 1 : 0, o = 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s = i == lr ? 1.f : 0.f;
#pragma unroll
          for (int j4 = 0; j4 < i; j4 += 4) {
            const float4 a = *reinterpret_cast<const float4*>(&A[m][o + i][o + j4]);
            s = fmaf(-a.x, x[j4], s);
            if (j4 + 1 < i) s = fmaf(-a.y, x[j4 + 1], s);
            if (j4 + 2 < i) s = fmaf(-a.z, x[j4 + 2], s);
            if (j4 + 3 < i) s = fmaf(-a.w, x[j4 + 3], s);
          }
          x[i] = s;
        }
        if (lg < NM) {
#pragma unroll
          for (int i = 0; i < 16; ++i) T[m][o + i][o + lr] = x[i];
        }
      }
      // then the blocks below the diagonal, T_ij = -T_ii sum_k A_ik T_kj, by distance from it
#pragma unroll
      for (int d = 1; d < 4; ++d) {
        __syncthreads();
        if (w < 4 - d) {
          const int bi = w + d, bj = w;
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            f32x4 x = zero4(), y = zero4();
#pragma unroll
            for (int k = 0; k < d; ++k) {
              // any order of k that both operands share gives the product: 4 lg + s
              const float4 a = *reinterpret_cast<const float4*>(&A[m][16 * bi + lr][16 * (bj + k) + 4 * lg]);
              const float* b = &T[m][16 * (bj + k) + 4 * lg][16 * bj + lr];
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b[0], x, 0, 0, 0);
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b[kLd], x, 0, 0, 0);
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b[2 * kLd], x, 0, 0, 0);
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b[3 * kLd], x, 0, 0, 0);
            }
            const float4 a = *reinterpret_cast<const float4*>(&T[m][16 * bi + lr][16 * bi + 4 * lg]);
            const float at[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(at[r], x[r], y, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) T[m][16 * bi + 4 * lg + r][16 * bj + lr] = -y[r];
          }
        }
      }
      __syncthreads();
      // out as fragments: of T' the column halves up to the diagonal, of T^T those from it on
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int f = w * 2 + ks;
        if (ks <= w / 2)
          store_frag<3>(ws.t1 + (size_t)cell * kTri * 3 * 64, f, lane, frag_f32<3>(&T[0][16 * w + lr][32 * ks + 8 * lg]));
        if constexpr (GRAD)
          if (ks >= w / 2) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = T[NM - 1][32 * ks + 8 * lg + j][16 * w + lr];
            store_frag<3>(ws.t2 + (size_t)cell * kTri * 3 * 64, f, lane, split8<3>(x));
          }
      }
      if (tid < kC) {
        float* o = ws.gates + (size_t)cell * 3 * kC;
        o[tid] = exp2_of((float)Gs[tid]);
        o[kC + tid] = exp2_of((float)(Gs[kC - 1] - Gs[tid]));
        o[2 * kC + tid] = bs[tid];
        if constexpr (GRAD) ws.g[(size_t)cell * kC + tid] = Gs[tid];
      }
    }
  }
}

// Sequences of one state row belong to the workgroup (of T threads) of the first of
// them: whether seq is that one, and in *next the one after it, or 2^31 - 1.
template <int T>
__device__ __forceinline__ bool first_of_slot(const int* slots, int sequences, int seq, int slot, int* earlier, int* next) {
  if (threadIdx.x == 0) {
    *earlier = 0;
    *next = 0x7fffffff;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < sequences; i += T)
    if (slots[i] == slot) {
      if (i < seq) *earlier = 1;
      else if (i > seq) atomicMin(next, i);
    }
  __syncthreads();
  return !*earlier;
}

// That next one, and in *next the one after it.
template <int T>
__device__ __forceinline__ int next_of_slot(const int* slots, int sequences, int slot, int* next) {
  __syncthreads();
  const int seq = *next;
  __syncthreads();
  if (threadIdx.x == 0) *next = 0x7fffffff;
  __syncthreads();
  for (int i = seq + 1 + threadIdx.x; i < sequences; i += T)
    if (slots[i] == slot) atomicMin(next, i);
  __syncthreads();
  return seq;
}

// The scan.  A step's chain of dependent work is
//     N = V - e^G K S0   |   e = T' N, U, e^(Gn-G) U   |   S1   |
// with a barrier (|) wherever a product's result becomes the next one's operand
// through LDS.  One wavefront issues an instruction every four clocks at best, so
// a step lasts as long as the instructions on this chain and little else: eight
// wavefronts share the work such that the chain is short.  Wavefronts 0 - 3 (rows
// 16 w .. of the chunk) run the first two phases; 4 - 7 have the output's
// products, which fill the waits, and (all eight at d_k > 64) the rows of the
// state.  Loads are issued SETS steps ahead, into registers that have just been
// used.  One sequence of 32768 tokens, 35 heads of 64: 512 steps in 848 us, 1.66 us
// a step, on 140 CUs (some 4000 with four wavefronts, row-major LDS tiles and loads
// of the step's own operands).  fp32 at d_k above 64 spills 21 or 22 registers with
// one strip (256 strips of 16 chunks 71 us against 42 of bf16).
//
// OB: bytes of an output element (2: bf16, 4: fp32), or 0: no outputs, but e and
// the state before each chunk are left in the workspace for the gradients.  The
// output's products take three terms whatever its type: with two, 3 to 5% faster
// (13 prompts of 8191 tokens, 32 heads of 128, the call 289 us against 303; 32768
// tokens, 35 heads of 64 1088 against 1120), three in a thousand bf16 outputs
// are the neighbour of what the fp32 result rounds to.
//
// NS: strips of 16 columns of a workgroup.  One where every strip can have a CU
// to itself (256 strips of 16 chunks, bf16: 42 us against 55 in pairs at d_k = d_v
// = 128, 31 against 37 at 64, 29 against 36 at 32): only the step's own length counts, loads run two steps ahead.  Two
// where there are more: the operands come through a CU's L1 once for both, which is
// what bounds a full CU, and a step's waits have twice the products to fill them;
// loads run one step ahead (384 strips 54 us against 73, 38 against 55, 39 against 53).
template <int NT, int DKP, int OB, int NS>
__global__ __launch_bounds__(512, 2) void packed_scan_kernel(SeqProblem p, PackedTensors t, PackedSpace ws) {
  constexpr int PT = OB ? 3 : 0;                      // terms of the output products
  constexpr int SETS = NS == 1 ? 2 : 1;               // operand sets in registers: steps that loads run ahead
  constexpr int KS = DKP / 32;                        // steps over d_k
  constexpr int SP = 16 * DKP, TP = 16 * kC;   // elements of a term's tile
  constexpr uint32_t es = NT == 1 ? 2 : 4;            // bytes of an input element
  constexpr uint32_t os = OB;                         // of an output element
  __shared__ __align__(16) bh Sl[NS][3 * SP];
  __shared__ __align__(16) bh Nl[NS][3 * TP];
  __shared__ __align__(16) bh Ul[NS][(PT ? PT : 1) * TP];
  __shared__ __align__(16) bh Dl[NS][3 * TP];
  __shared__ __align__(16) typename RawIn<NT>::type Vl[NS][TP];
  __shared__ int earlier, next;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lr = lane % 16, lg = lane / 16;
  const int strips = p.dv / 16;
  int sh, strip;                                      // strips strip .. + NS; the last one of the last workgroup may not exist
  strip_of(blockIdx.x, (strips + NS - 1) / NS, &sh, &strip);
  strip *= NS;
  if (sh >= p.sequences * p.hv) return;
  const int h = sh % p.hv, kh = h / (p.hv / p.hk);
  const int col = strip * 16 + lr;
  const auto there = [&](int i) { return NS == 1 || strip + i < strips; };
  const int w = wave & 3;                             // row tile of the chunk
  const bool first_half = wave < 4;
  const int srow = DKP > 64 ? wave : wave - 4;        // row tile of the state, if it has one
  const bool has_state = srow >= 0 && srow < DKP / 16;
  int seq = NS == 1 ? sh / p.hv : by_length(t.cu, p.sequences, p.tokens, sh / p.hv);   // NS = 1: all start at once
  const int slot_of = t.slots ? t.slots[seq] : seq;
  const bool kept = !t.slots || (slot_of >= 0 && slot_of < p.state_rows);
  if (t.slots && kept && !first_of_slot<512>(t.slots, p.sequences, seq, slot_of, &earlier, &next)) return;
  const size_t state = ((size_t)slot_of * p.hv + h) * p.dk * p.dv;
  const int row0 = 16 * w + 4 * lg;                   // of this lane's four accumulator rows
  const int krow = 16 * w + lr;                       // of its operand rows
  const int st0 = srow * 16 + 4 * lg;                 // of its four state rows
  const int tok_place = put_place(lr, row0), st_place = put_place(lr, has_state ? st0 : 0);
  int vector_zero = 0;
  asm volatile("" : "+v"(vector_zero));               // a scalar load would be waited for with the LDS traffic
  // per chunk, in elements of each workspace array
  const size_t tri = (size_t)kTri * 3 * 64, tr = (size_t)(DKP / 16) * 2 * NT * 64;

  for (;;) {
    int start, end;
    seq_bounds(t.cu, seq, p.tokens, &start, &end);
    start = __builtin_amdgcn_readfirstlane(start);
    end = __builtin_amdgcn_readfirstlane(end);
    const size_t slot = start / kC + (size_t)seq;
    f32x4 S[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      S[i] = zero4();
      if (has_state) {
        if (t.h0 && kept && there(i))
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (st0 + r < p.dk) S[i][r] = t.h0[state + (size_t)(st0 + r) * p.dv + col + 16 * i];
        const float x[4] = {S[i][0], S[i][1], S[i][2], S[i][3]};
        put<3, DKP>(Sl[i] + st_place, x);
      }
    }
    const int last = (end - start + kC - 1) / kC - 1;
    // Loads behind the last chunk return 0.
    auto rows_of = [&](int c) { return end - start - c * kC; };
    // The state's share of a step, by the wavefronts that have rows of it:
    Frag<NT> kt[SETS][2];
    float eGn[SETS];
    const uint32_t kt_off = ((uint32_t)srow * 2 * NT * 64 + lane) * 16;
    auto load_state = [&](int c, int set) {
      const bool is = c <= last;
      const buf_t kb = buf(ws.kt + ((slot + c) * p.hk + kh) * tr, is && has_state ? (uint32_t)tr * 16 : 0);
      const buf_t gb = buf(ws.gates + ((slot + c) * p.hv + h) * 3 * kC, is ? kC * 4 : 0);
      eGn[set] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(gb, (kC - 1) * 4 + vector_zero, 0, 0));
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) kt[set][ks] = frag_at<NT>(kb, kt_off + ks * NT * 1024);
    };
    auto step_state = [&](int c, int set) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if constexpr (PT == 0) {
          const buf_t sb = buf(ws.s0 + (((slot + c) * p.hv + h) * strips + strip + i) * DKP * 16,
                               has_state && there(i) ? DKP * 16 * 4 : 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) store_at<4>(sb, ((st0 + r) * 16 + lr) * 4, S[i][r]);
        }
        f32x4 a[3];
        a[0] = S[i] * eGn[set];
        a[1] = a[2] = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) mma_by_term<NT, 3>(kt[set][ks], get<3, kC>(Dl[i] + lane * 8, ks), a);
        S[i] = a[0] + (a[1] + a[2]);
        const float x[4] = {S[i][0], S[i][1], S[i][2], S[i][3]};
        if (has_state) put<3, DKP>(Sl[i] + st_place, x);
      }
      load_state(c + SETS, set);
    };
    uint32_t col_off[KS];                             // of this lane's columns of K and Q
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) col_off[ks] = ks * 32 + lg * 8 < p.dk ? (ks * 32 + lg * 8) * es : kNowhere;
    const uint32_t dk_b = p.dk * es, dv_b = p.dv * es;
    // of this lane's fragments in a lower triangle; there are none to the right of the diagonal
    uint32_t tri_off[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) tri_off[ks] = ks <= w / 2 ? ((uint32_t)(w * 2 + ks) * 3 * 64 + lane) * 16 : kNowhere;
    if (last < 0) {
      // nothing to scan: the state stays as it is
    } else if (first_half) {
      const uint32_t ks_b = (uint32_t)p.ks * es;
      RawFrag<NT> k[SETS][KS];
      uint4 eG[SETS], eD[SETS], be[SETS];
      Frag<3> t1[SETS][2];
      auto load = [&](int c, int set) {
        const int n = rows_of(c);
        const buf_t kb = buf(static_cast<const char*>(t.k) + ((size_t)(start + c * kC) * p.ks + kh * p.dk) * es, span(n, ks_b, dk_b));
        const size_t cl = (slot + c) * p.hv + h;
        const buf_t tb = buf(ws.t1 + cl * tri, n > 0 ? (uint32_t)tri * 16 : 0);
        const buf_t gb = buf(ws.gates + cl * 3 * kC, n > 0 ? 3 * kC * 4 : 0);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) k[set][ks] = raw_at<NT>(kb, krow * ks_b + col_off[ks]);
        eG[set] = buf_load16(gb, row0 * 4);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) t1[set][ks] = frag_at<3>(tb, tri_off[ks]);
        eD[set] = buf_load16(gb, (kC + row0) * 4);
        be[set] = buf_load16(gb, (2 * kC + row0) * 4);
      };
      load(0, 0);
      load_state(0, 0);
      if constexpr (SETS == 2) {
        load(1, 1);
        load_state(1, 1);
      }
      __syncthreads();
      auto step = [&](int c, int set) {
        if constexpr (SETS == 2) __builtin_amdgcn_s_setprio(3);
        float eg[4], ed[4], bt[4];
        f32x4 e[NS];
        floats(eG[set], eg);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          f32x4 a[3];
#pragma unroll
          for (int j = 0; j < 3; ++j) a[j] = zero4();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) mma_by_term<NT, 3>(frag_of<NT>(k[set][ks]), get<3, DKP>(Sl[i] + lane * 8, ks), a);
          float x[4];
          get_values<NT>(Vl[i] + (w * 64 + lane) * 4, x);
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = fmaf(-eg[r], (a[2][r] + a[1][r]) + a[0][r], x[r]);
          put<3, kC>(Nl[i] + tok_place, x);
        }
        __syncthreads();
        floats(eD[set], ed);
        floats(be[set], bt);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          f32x4 a[3];
#pragma unroll
          for (int j = 0; j < 3; ++j) a[j] = zero4();
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) mma_by_term<3, 3>(t1[set][ks], get<3, kC>(Nl[i] + lane * 8, ks), a);
          e[i] = (a[2] + a[1]) + a[0];
          float x[4], ud[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = bt[r] * e[i][r];
            ud[r] = ed[r] * x[r];
          }
          put<3, kC>(Dl[i] + tok_place, ud);
          if constexpr (PT > 0) put<PT, kC>(Ul[i] + tok_place, x);
        }
        __syncthreads();
        if constexpr (DKP > 64) step_state(c, set);
        if constexpr (SETS == 2) __builtin_amdgcn_s_setprio(0);
        load(c + SETS, set);
        if constexpr (PT == 0)
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const buf_t eb = buf(ws.e + (((slot + c) * p.hv + h) * strips + strip + i) * kC * 16, there(i) ? kC * 16 * 4 : 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) store_at<4>(eb, ((row0 + r) * 16 + lr) * 4, e[i][r]);
          }
        __syncthreads();
      };
      for (int c = 0; c <= last; c += SETS) {
        step(c, 0);
        if constexpr (SETS == 2)
          if (c < last) step(c + 1, 1);
      }
    } else {
      const uint32_t qs_b = (uint32_t)p.qs * es, vs_b = (uint32_t)p.vs * es, os_b = (uint32_t)(p.hv * p.dv) * os;
      RawFrag<NT> q[SETS][KS];
      typename RawIn<NT>::type v[NS][4];
      uint4 eG[SETS];
      Frag<PT ? PT : 1> pf[SETS][2];
      auto load = [&](int c, int set) {
        if constexpr (PT > 0) {
          const int n = rows_of(c);
          const size_t first = start + (size_t)c * kC;
          const buf_t qb = buf(static_cast<const char*>(t.q) + (first * p.qs + kh * p.dk) * es, span(n, qs_b, dk_b));
          const buf_t gb = buf(ws.gates + ((slot + c) * p.hv + h) * 3 * kC, n > 0 ? kC * 4 : 0);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) q[set][ks] = raw_at<NT>(qb, krow * qs_b + col_off[ks]);
          eG[set] = buf_load16(gb, row0 * 4);
        }
      };
      auto load_v = [&](int c) {
        const buf_t vb = buf(static_cast<const char*>(t.v) + ((start + (size_t)c * kC) * p.vs + h * p.dv) * es,
                             span(rows_of(c), vs_b, dv_b));
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[i][r] = value_at<NT>(vb, there(i) ? (row0 + r) * vs_b + (col + 16 * i) * es : kNowhere);
      };
      auto load_p = [&](int c, int set) {
        if constexpr (PT > 0) {
          const buf_t pb = buf(ws.p + ((slot + c) * p.hv + h) * tri, c <= last ? (uint32_t)tri * 16 : 0);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) pf[set][ks] = frag_at<PT>(pb, tri_off[ks]);
        }
      };
      // a chunk's V goes into LDS a step ahead, as columns of four rows for the first half
      load_v(0);
      load(0, 0);
      load_p(0, 0);
      load_state(0, 0);
      auto put_v = [&]() {
#pragma unroll
        for (int i = 0; i < NS; ++i) put_values<NT>(Vl[i] + (w * 64 + lane) * 4, v[i]);
      };
      put_v();
      load_v(1);
      if constexpr (SETS == 2) {
        load(1, 1);
        load_p(1, 1);
        load_state(1, 1);
      }
      __syncthreads();
      f32x4 o[NS];
      // P U of chunk c and its store, beside the next step's first phase
      auto finish = [&](int c, int set) {
        if constexpr (PT > 0) {
          const buf_t ob = buf(static_cast<char*>(t.out) + ((start + (size_t)c * kC) * p.hv + h) * p.dv * os,
                               span(rows_of(c), os_b, p.dv * os));
#pragma unroll
          for (int i = 0; i < NS; ++i) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) o[i] = mma<PT, PT>(pf[set][ks], get<PT, kC>(Ul[i] + lane * 8, ks), o[i]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              store_at<os>(ob, there(i) ? (row0 + r) * os_b + (col + 16 * i) * os : kNowhere, o[i][r]);
          }
          load_p(c + SETS, set);
        }
      };
      auto step = [&](int c, int set) {
        if constexpr (PT > 0)
          if (c > 0) finish(c - 1, SETS == 2 ? set ^ 1 : 0);
        __syncthreads();
        put_v();
        load_v(c + 2);
        if constexpr (PT > 0) {
          float eg[4];
          floats(eG[set], eg);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            o[i] = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
              o[i] = mma<NT, PT>(frag_of<NT>(q[set][ks]), get<PT, DKP>(Sl[i] + lane * 8, ks), o[i]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[i][r] *= eg[r];
          }
        }
        load(c + SETS, set);
        __syncthreads();
        if constexpr (SETS == 2) __builtin_amdgcn_s_setprio(3);
        step_state(c, set);
        if constexpr (SETS == 2) __builtin_amdgcn_s_setprio(0);
        __syncthreads();
      };
      step(0, 0);
      for (int c = 1; c <= last; c += SETS) {
        step(c, SETS - 1);
        if constexpr (SETS == 2)
          if (c < last) step(c + 1, 0);
      }
      if (SETS == 2 && (last & 1)) finish(last, SETS - 1);
      else finish(last, 0);
    }
    if (t.hT && kept && has_state)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (st0 + r < p.dk && there(i)) t.hT[state + (size_t)(st0 + r) * p.dv + col + 16 * i] = S[i][r];
    if (!t.slots || !kept || next == 0x7fffffff) break;
    seq = next_of_slot<512>(t.slots, p.sequences, slot_of, &next);
  }
}

// The scan where there are more pairs of strips than CUs, bf16: then what counts
// is the work of all CUs, not the length of a step, and four wavefronts that each
// do every part of it, for two strips, leave two workgroups on a CU to fill each
// other's waits.  K and Q share the state's operand reads, a lane's rows of V
// need no staging.  13 prompts of 8191 tokens, 32 heads of 128: 202 us against
// 258 by the eight wavefronts above in pairs; equal strips of 16 chunks at d_k =
// d_v = 128, 64, 32: 768 of them 89, 67, 96 against 103, 73, 102; 2048 196, 203, 253
// against 235, 204, 247; but 512 of them 61, 48, 50 against 55, 40, 49.  The rule
// counts strips, since the lengths are on the GPU: one long prompt among many short
// ones runs its chain with this kernel's longer step.  fp32 operands take the
// registers of both workgroups (2048 strips 398 against 372), so they stay with
// the kernel above.
template <int DKP, int OB>
__global__ __launch_bounds__(256, 2) void packed_scan_pairs_kernel(SeqProblem p, PackedTensors t, PackedSpace ws) {
  constexpr int PT = OB ? 3 : 0;                      // terms of the output products
  constexpr int NT = 1, NS = 2, KS = DKP / 32, MT = DKP >= 64 ? DKP / 64 : 1;
  constexpr int SP = 16 * DKP, TP = 16 * kC;          // elements of a term's tile
  constexpr uint32_t es = 2;                          // bytes of an input element
  constexpr uint32_t os = OB;                         // of an output element
  __shared__ __align__(16) bh Sl[NS][3 * SP];
  __shared__ __align__(16) bh Nl[NS][3 * TP];
  __shared__ __align__(16) bh Ul[NS][(PT ? PT : 1) * TP];
  __shared__ __align__(16) bh Dl[NS][3 * TP];
  __shared__ int earlier, next;
  const int tid = threadIdx.x, lane = tid % 64, w = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lr = lane % 16, lg = lane / 16;
  const int strips = p.dv / 16;
  int sh, strip;                                      // strips strip, strip + 1; the second of the last pair may not exist
  strip_of(blockIdx.x, (strips + 1) / 2, &sh, &strip);
  strip *= NS;
  if (sh >= p.sequences * p.hv) return;
  const int h = sh % p.hv, kh = h / (p.hv / p.hk);
  const int col = strip * 16 + lr;
  const auto there = [&](int i) { return strip + i < strips; };
  const bool srows = DKP >= 64 || w < DKP / 16;       // has rows of the state
  int seq = by_length(t.cu, p.sequences, p.tokens, sh / p.hv);
  const int slot_of = t.slots ? t.slots[seq] : seq;
  const bool kept = !t.slots || (slot_of >= 0 && slot_of < p.state_rows);
  if (t.slots && kept && !first_of_slot<256>(t.slots, p.sequences, seq, slot_of, &earlier, &next)) return;
  const size_t state = ((size_t)slot_of * p.hv + h) * p.dk * p.dv;
  const int row0 = 16 * w + 4 * lg;                   // of this lane's four accumulator rows
  const int krow = 16 * w + lr;                       // of its operand rows
  const int tok_place = put_place(lr, row0);
  int vector_zero = 0;
  asm volatile("" : "+v"(vector_zero));               // a scalar load would be waited for with the LDS traffic
  const size_t tri = (size_t)kTri * 3 * 64, tr = (size_t)(DKP / 16) * 2 * NT * 64;
  const uint32_t ks_b = (uint32_t)p.ks * es, qs_b = (uint32_t)p.qs * es, vs_b = (uint32_t)p.vs * es;
  const uint32_t dk_b = p.dk * es, dv_b = p.dv * es, os_b = (uint32_t)(p.hv * p.dv) * os;
  uint32_t col_off[KS], tri_off[2];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) col_off[ks] = ks * 32 + lg * 8 < p.dk ? (ks * 32 + lg * 8) * es : kNowhere;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) tri_off[ks] = ks <= w / 2 ? ((uint32_t)(w * 2 + ks) * 3 * 64 + lane) * 16 : kNowhere;

  for (;;) {
    int start, end;
    seq_bounds(t.cu, seq, p.tokens, &start, &end);
    start = __builtin_amdgcn_readfirstlane(start);
    end = __builtin_amdgcn_readfirstlane(end);
    const size_t slot = start / kC + (size_t)seq;
    const int last = (end - start + kC - 1) / kC - 1;
    f32x4 S[NS][MT];
    auto put_state = [&](int i) {
      if (srows)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float x[4] = {S[i][m][0], S[i][m][1], S[i][m][2], S[i][m][3]};
          put<3, DKP>(Sl[i] + put_place(lr, (w * MT + m) * 16 + 4 * lg), x);
        }
    };
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = (w * MT + m) * 16 + 4 * lg + r;
          S[i][m][r] = t.h0 && kept && there(i) && row < p.dk ? t.h0[state + (size_t)row * p.dv + col + 16 * i] : 0.f;
        }
      put_state(i);
    }
    // Loads behind the last chunk return 0.
    auto rows_of = [&](int c) { return end - start - c * kC; };
    RawFrag<NT> k[KS], q[KS];
    typename RawIn<NT>::type v[NS][4];
    uint4 eG, eD, be;
    Frag<3> t1[2];
    Frag<PT ? PT : 1> pf[2];
    Frag<NT> kt[MT][2];
    float eGn;
    auto load_rows = [&](int c) {
      const int n = rows_of(c);
      const size_t first = start + (size_t)c * kC;
      const buf_t kb = buf(static_cast<const char*>(t.k) + (first * p.ks + kh * p.dk) * es, span(n, ks_b, dk_b));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) k[ks] = raw_at<NT>(kb, krow * ks_b + col_off[ks]);
      if constexpr (PT > 0) {
        const buf_t qb = buf(static_cast<const char*>(t.q) + (first * p.qs + kh * p.dk) * es, span(n, qs_b, dk_b));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = raw_at<NT>(qb, krow * qs_b + col_off[ks]);
      }
      const buf_t vb = buf(static_cast<const char*>(t.v) + (first * p.vs + h * p.dv) * es, span(n, vs_b, dv_b));
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[i][r] = value_at<NT>(vb, there(i) ? (row0 + r) * vs_b + (col + 16 * i) * es : kNowhere);
      eG = buf_load16(buf(ws.gates + ((slot + c) * p.hv + h) * 3 * kC, n > 0 ? kC * 4 : 0), row0 * 4);
    };
    auto load_inverse = [&](int c) {
      const size_t cl = (slot + c) * p.hv + h;
      const buf_t tb = buf(ws.t1 + cl * tri, c <= last ? (uint32_t)tri * 16 : 0);
      const buf_t gb = buf(ws.gates + cl * 3 * kC, c <= last ? 3 * kC * 4 : 0);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) t1[ks] = frag_at<3>(tb, tri_off[ks]);
      eD = buf_load16(gb, (kC + row0) * 4);
      be = buf_load16(gb, (2 * kC + row0) * 4);
      eGn = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(gb, (kC - 1) * 4 + vector_zero, 0, 0));
    };
    auto load_state = [&](int c) {
      const buf_t kb = buf(ws.kt + ((slot + c) * p.hk + kh) * tr, c <= last && srows ? (uint32_t)tr * 16 : 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) kt[m][ks] = frag_at<NT>(kb, (((w * MT + m) * 2 + ks) * NT * 64 + lane) * 16);
      if constexpr (PT > 0) {
        const buf_t pb = buf(ws.p + ((slot + c) * p.hv + h) * tri, c <= last ? (uint32_t)tri * 16 : 0);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) pf[ks] = frag_at<PT>(pb, tri_off[ks]);
      }
    };
    load_rows(0);
    load_inverse(0);
    load_state(0);
    __syncthreads();
    for (int c = 0; c <= last; ++c) {
      const size_t cl = (slot + c) * p.hv + h;
      f32x4 o[NS];
      {
        float eg[4];
        floats(eG, eg);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          f32x4 a[3];
#pragma unroll
          for (int j = 0; j < 3; ++j) a[j] = zero4();
          o[i] = zero4();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const Frag<3> sf = get<3, DKP>(Sl[i] + lane * 8, ks);
            mma_by_term<NT, 3>(frag_of<NT>(k[ks]), sf, a);
            if constexpr (PT > 0) o[i] = mma<NT, PT>(frag_of<NT>(q[ks]), sf, o[i]);
          }
          float x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = fmaf(-eg[r], (a[2][r] + a[1][r]) + a[0][r], raw_value(v[i][r]));
            o[i][r] *= eg[r];
          }
          put<3, kC>(Nl[i] + tok_place, x);
        }
      }
      load_rows(c + 1);
      __syncthreads();
      {
        float ed[4], bt[4];
        floats(eD, ed);
        floats(be, bt);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          f32x4 a[3];
#pragma unroll
          for (int j = 0; j < 3; ++j) a[j] = zero4();
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            if (ks <= w / 2) mma_by_term<3, 3>(t1[ks], get<3, kC>(Nl[i] + lane * 8, ks), a);
          const f32x4 e = (a[2] + a[1]) + a[0];
          float x[4], ud[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = bt[r] * e[r];
            ud[r] = ed[r] * x[r];
          }
          put<3, kC>(Dl[i] + tok_place, ud);
          if constexpr (PT > 0) {
            put<PT, kC>(Ul[i] + tok_place, x);
          } else {
            const buf_t eb = buf(ws.e + (cl * strips + strip + i) * kC * 16, there(i) ? kC * 16 * 4 : 0);
            const buf_t sb = buf(ws.s0 + (cl * strips + strip + i) * DKP * 16, there(i) && srows ? DKP * 16 * 4 : 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) store_at<4>(eb, ((row0 + r) * 16 + lr) * 4, e[r]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int r = 0; r < 4; ++r) store_at<4>(sb, (((w * MT + m) * 16 + 4 * lg + r) * 16 + lr) * 4, S[i][m][r]);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) S[i][m] = S[i][m] * eGn;
        }
      }
      load_inverse(c + 1);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (srows) {
          Frag<3> df[2];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) df[ks] = get<3, kC>(Dl[i] + lane * 8, ks);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4 a[3];
            a[0] = S[i][m];
            a[1] = a[2] = zero4();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) mma_by_term<NT, 3>(kt[m][ks], df[ks], a);
            S[i][m] = a[0] + (a[1] + a[2]);
          }
        }
        put_state(i);
      }
      if constexpr (PT > 0) {
        const buf_t ob = buf(static_cast<char*>(t.out) + ((start + (size_t)c * kC) * p.hv + h) * p.dv * os,
                             span(rows_of(c), os_b, p.dv * os));
#pragma unroll
        for (int i = 0; i < NS; ++i) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            if (ks <= w / 2) o[i] = mma<PT, PT>(pf[ks], get<PT, kC>(Ul[i] + lane * 8, ks), o[i]);
#pragma unroll
          for (int r = 0; r < 4; ++r) store_at<os>(ob, there(i) ? (row0 + r) * os_b + (col + 16 * i) * os : kNowhere, o[i][r]);
        }
      }
      load_state(c + 1);
      __syncthreads();
    }
    if (t.hT && kept && srows)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = (w * MT + m) * 16 + 4 * lg + r;
            if (row < p.dk && there(i)) t.hT[state + (size_t)row * p.dv + col + 16 * i] = S[i][m][r];
          }
    if (!t.slots || !kept || next == 0x7fffffff) break;
    seq = next_of_slot<256>(t.slots, p.sequences, slot_of, &next);
  }
}

}  // namespace

PackedPlan packed_plan(const SeqProblem& p) {
  PackedPlan f;
  f.slots = p.tokens / kC + p.sequences;
  f.strips = p.dv / 16;
  f.dkp = p.dk <= 32 ? 32 : p.dk <= 64 ? 64 : 128;
  f.terms = p.in_bf16 ? 1 : 3;
  return f;
}

size_t packed_space(const SeqProblem& p, bool grad, void* base, PackedSpace* s) {
  const PackedPlan f = packed_plan(p);
  const size_t cells = (size_t)f.slots * p.hv, rows = (size_t)f.slots * p.hk;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = base ? static_cast<char*>(base) + at : nullptr;
    at += align_up(bytes, 256);
    return q;
  };
  const size_t tri = (size_t)kTri * 3 * 64 * sizeof(uint4), tr = (size_t)f.dkp / 16 * 2 * f.terms * 64 * sizeof(uint4);
  PackedSpace o = {};
  o.t1 = reinterpret_cast<uint4*>(take(cells * tri));
  o.p = reinterpret_cast<uint4*>(take(cells * tri));
  o.gates = reinterpret_cast<float*>(take(cells * 3 * kC * sizeof(float)));
  o.kt = reinterpret_cast<uint4*>(take(rows * tr));
  if (grad) {
    const size_t tok = (size_t)f.strips * kC * 16 * sizeof(float), st = (size_t)f.strips * f.dkp * 16 * sizeof(float);
    o.t2 = reinterpret_cast<uint4*>(take(cells * tri));
    o.qt = reinterpret_cast<uint4*>(take(rows * tr));
    o.g = reinterpret_cast<double*>(take(cells * kC * sizeof(double)));
    o.e = reinterpret_cast<float*>(take(cells * tok));
    o.w = reinterpret_cast<float*>(take(cells * tok));
    o.s0 = reinterpret_cast<float*>(take(cells * st));
    o.ds = reinterpret_cast<float*>(take(cells * st));
  }
  if (s) *s = o;
  return at;
}

hipError_t packed_prep(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, bool grad, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  // Value heads of a workgroup: in the gradients all of a key head, whose products
  // they share, where that leaves each CU four workgroups (8192 tokens, 16 and 32
  // heads of 128: 116 us against 148).  In the forward call those products' registers
  // cost half of the wavefronts or spill (122 against 104).
  const int share = grad && f.slots * p.hk >= 1024 ? p.hv / p.hk : 1;
  const long long items = f.slots * (p.hv / share);
  const dim3 grid((unsigned)(items < kMaxBlocks ? items : kMaxBlocks));
  prof_begin(stream, GDN_KERNEL_PACKED_PREP);
#define GDN_PREP(NT, D)                                                                                                          \
  if (f.terms == NT && f.dkp == D) {                                                                                             \
    if (grad) hipLaunchKernelGGL((packed_prep_kernel<NT, D, true>), grid, dim3(256), 0, stream, p, t, s, f.slots, share);        \
    else hipLaunchKernelGGL((packed_prep_kernel<NT, D, false>), grid, dim3(256), 0, stream, p, t, s, f.slots, share);            \
  }
  GDN_PREP(1, 32) GDN_PREP(1, 64) GDN_PREP(1, 128) GDN_PREP(3, 32) GDN_PREP(3, 64) GDN_PREP(3, 128)
#undef GDN_PREP
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_PREP);
  return e;
}

hipError_t packed_scan(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, bool grad, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  const unsigned heads = (p.sequences * p.hv + 7) / 8 * 8;
  const long long strips = (long long)p.sequences * p.hv * f.strips;
  const bool pairs = f.strips > 1 && strips > 256;     // more strips than CUs
  const bool four = pairs && strips > 512 && f.terms == 1;   // more pairs than CUs
  const dim3 grid(heads * (pairs ? (f.strips + 1) / 2 : f.strips));
  prof_begin(stream, GDN_KERNEL_PACKED_SCAN);
#define GDN_SCAN2(NT, D, OB)                                                                                         \
  if (four) hipLaunchKernelGGL((packed_scan_pairs_kernel<D, OB>), grid, dim3(256), 0, stream, p, t, s);              \
  else if (pairs) hipLaunchKernelGGL((packed_scan_kernel<NT, D, OB, 2>), grid, dim3(512), 0, stream, p, t, s);       \
  else hipLaunchKernelGGL((packed_scan_kernel<NT, D, OB, 1>), grid, dim3(512), 0, stream, p, t, s);
#define GDN_SCAN(NT, D)                      \
  if (f.terms == NT && f.dkp == D) {         \
    if (grad) { GDN_SCAN2(NT, D, 0) }        \
    else if (p.out_bf16) { GDN_SCAN2(NT, D, 2) } \
    else { GDN_SCAN2(NT, D, 4) }             \
  }
  GDN_SCAN(1, 32) GDN_SCAN(1, 64) GDN_SCAN(1, 128) GDN_SCAN(3, 32) GDN_SCAN(3, 64) GDN_SCAN(3, 128)
#undef GDN_SCAN
#undef GDN_SCAN2
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_SCAN);
  return e;
}

}  // namespace gdn
