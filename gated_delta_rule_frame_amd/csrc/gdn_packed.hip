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

template <int NT, int DKP, bool GRAD>
__global__ __launch_bounds__(256) void packed_prep_kernel(SeqProblem p, PackedTensors t, PackedSpace ws, long long slots) {
  constexpr int NM = GRAD ? 2 : 1;
  __shared__ double Gs[kC];
  __shared__ float bs[kC];
  __shared__ __align__(16) float A[NM][kC][kLd];
  __shared__ __align__(16) float T[NM][kC][kLd];
  __shared__ __align__(16) float P[kC][kLd];
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64;
  const int lr = lane % 16, lg = lane / 16;
  const int rep = p.hv / p.hk;
  const long long cells = slots * p.hv;

  for (long long cell = blockIdx.x; cell < cells; cell += gridDim.x) {
    const int h = (int)(cell % p.hv), kh = h / rep;
    const long long slot = cell / p.hv;
    int seq, first, n;
    if (!find_chunk(t.cu, p.sequences, p.tokens, slot, &seq, &first, &n)) continue;   // uniform over the workgroup
    __syncthreads();
    if (w == 0) {
      const size_t at = (size_t)(first + lane) * p.hv + h;
      float g = lane < n ? t.g[at] : 0.f;
      g = g < kLowestGate ? kLowestGate : g;
      double G = g;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(G, m);
        if (lane >= m) G += o;
      }
      Gs[lane] = G;
      bs[lane] = lane < n ? t.beta[at] : 0.f;
    }
    // Gram tiles: wavefront w has rows 16 w .. + 16
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero4();
    const char* kbase = static_cast<const char*>(t.k);
    const char* qbase = static_cast<const char*>(t.q);
    auto row_frag = [&](const char* base, long long stride, int tile, int ks) {
      const int row = tile * 16 + lr, c = ks * 32 + lg * 8;
      if (row < n && c < p.dk) return frag_in<NT>(base, (size_t)(first + row) * stride + kh * p.dk + c);
      return zero_frag<NT>();
    };
#pragma unroll
    for (int ks = 0; ks < DKP / 32; ++ks) {
      const Frag<NT> ak = row_frag(kbase, p.ks, w, ks), aq = row_frag(qbase, p.qs, w, ks);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          const Frag<NT> b = j == w ? ak : row_frag(kbase, p.ks, j, ks);
          kk[j] = mma<NT, NT>(ak, b, kk[j]);
          qk[j] = mma<NT, NT>(aq, b, qk[j]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * lg + r, c = 16 * j + lr;
        const float E = i >= c ? expf((float)(Gs[i] - Gs[c])) : 0.f;
        const float b = i > c ? E * kk[j][r] : 0.f;
        A[0][i][c] = b * bs[c];
        if constexpr (GRAD) A[NM - 1][i][c] = b * bs[i];
        P[i][c] = i >= c ? E * qk[j][r] : 0.f;
        if (j > w) {
          T[0][i][c] = 0.f;
          if constexpr (GRAD) T[NM - 1][i][c] = 0.f;
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
        for (int j = 0; j < i; ++j) s = fmaf(-A[m][o + i][o + j], x[j], s);
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
          for (int k = bj; k < bi; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s)
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(A[m][16 * bi + lr][16 * k + 4 * s + lg],
                                                       T[m][16 * k + 4 * s + lg][16 * bj + lr], x, 0, 0, 0);
          // x holds rows 4 lg + r: any order of k that both operands share gives the product
#pragma unroll
          for (int r = 0; r < 4; ++r)
            y = __builtin_amdgcn_mfma_f32_16x16x4f32(T[m][16 * bi + lr][16 * bi + 4 * lg + r], x[r], y, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) T[m][16 * bi + 4 * lg + r][16 * bj + lr] = -y[r];
        }
      }
    }
    __syncthreads();
    // out as fragments: row tile w; of the lower triangles only the column halves that hold any of it, of the transposed ones
    // likewise
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int f = w * 2 + ks;
      if (ks <= w / 2) {
        store_frag<3>(ws.t1 + (size_t)cell * kTri * 3 * 64, f, lane, frag_f32<3>(&T[0][16 * w + lr][32 * ks + 8 * lg]));
        if constexpr (!GRAD)
          store_frag<3>(ws.p + (size_t)cell * kTri * 3 * 64, f, lane, frag_f32<3>(&P[16 * w + lr][32 * ks + 8 * lg]));
      }
      if constexpr (GRAD)
        if (ks >= w / 2) {
          float x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = T[NM - 1][32 * ks + 8 * lg + j][16 * w + lr];
            y[j] = P[32 * ks + 8 * lg + j][16 * w + lr];
          }
          store_frag<3>(ws.t2 + (size_t)cell * kTri * 3 * 64, f, lane, split8<3>(x));
          store_frag<3>(ws.p + (size_t)cell * kTri * 3 * 64, f, lane, split8<3>(y));
        }
    }
    if (tid < kC) {
      float* o = ws.gates + (size_t)cell * 3 * kC;
      o[tid] = expf((float)Gs[tid]);
      o[kC + tid] = expf((float)(Gs[kC - 1] - Gs[tid]));
      o[2 * kC + tid] = bs[tid];
      if constexpr (GRAD) ws.g[(size_t)cell * kC + tid] = Gs[tid];
    }
    if (h % rep == 0) {
      const size_t at = ((size_t)slot * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
      auto column_frag = [&](const void* base, long long stride, int mt, int ks) {
        const int c = mt * 16 + lr;
        Frag<NT> f;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int row = ks * 32 + lg * 8 + j;
          x[j] = c < p.dk && row < n ? elem_in<NT>(base, (size_t)(first + row) * stride + kh * p.dk + c) : 0.f;
        }
        f = split8<NT>(x);
        return f;
      };
      for (int f = w; f < DKP / 16 * 2; f += 4) {
        store_frag<NT>(ws.kt + at, f, lane, column_frag(t.k, p.ks, f / 2, f % 2));
        if constexpr (GRAD) store_frag<NT>(ws.qt + at, f, lane, column_frag(t.q, p.qs, f / 2, f % 2));
      }
    }
  }
}

// What a chunk's step reads from memory, as each phase of the step needs it.
// A phase's registers are loaded for the next chunk as soon as the phase has
// used them, so every load has a whole step to arrive.
template <int NT, int DKP, int PT>
struct ChunkIn {
  static constexpr int KS = DKP / 32, MT = DKP >= 64 ? DKP / 64 : 1;
  RawFrag<NT> k[KS], q[PT ? KS : 1];   // rows of K and Q
  typename RawIn<NT>::type v[4];
  float4 eG;
  Frag<3> t1[2];                    // T' and the gates of the rows
  float4 eD, beta;
  Frag<NT> kt[MT][2];               // K^T
  float eGn;
  Frag<PT ? PT : 1> p[2];           // P
};

// PT: terms of the output products (2 for a bf16 output, whose rounding is 2^9
// times the third term; 3 for fp32), or 0: no outputs, but e and the state
// before each chunk are left in the workspace for the gradients.
template <int NT, int DKP, int PT>
__global__ __launch_bounds__(256, NT == 1 ? 2 : 1) void packed_scan_kernel(SeqProblem p, PackedTensors t, PackedSpace ws) {
  using In = ChunkIn<NT, DKP, PT>;
  constexpr int KS = In::KS;                          // steps over d_k
  constexpr int MT = In::MT;                          // state row tiles of a wavefront
  constexpr int SLD = DKP + 8, SP = 16 * SLD, TP = 16 * kTok;
  __shared__ __align__(16) bh Sl[3 * SP];
  __shared__ __align__(16) bh Nl[3 * TP];
  __shared__ __align__(16) bh Ul[(PT ? PT : 1) * TP];
  __shared__ __align__(16) bh Dl[3 * TP];
  __shared__ int earlier, next;
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64;
  const int lr = lane % 16, lg = lane / 16;
  int sh, strip;
  strip_of(blockIdx.x, p.dv / 16, &sh, &strip);
  if (sh >= p.sequences * p.hv) return;
  const int h = sh % p.hv, kh = h / (p.hv / p.hk);
  const int col = strip * 16 + lr;
  const int strips = p.dv / 16;
  const bool srows = DKP >= 64 || w < DKP / 16;
  int seq = sh / p.hv;
  const int slot_of = t.slots ? t.slots[seq] : seq;
  const bool kept = !t.slots || (slot_of >= 0 && slot_of < p.state_rows);
  if (t.slots && kept) {
    // sequences of the same state row belong to the workgroup of the first of them
    if (tid == 0) { earlier = 0; next = 0x7fffffff; }
    __syncthreads();
    for (int i = tid; i < p.sequences; i += 256)
      if (t.slots[i] == slot_of) {
        if (i < seq) earlier = 1;
        else if (i > seq) atomicMin(&next, i);
      }
    __syncthreads();
    if (earlier) return;
  }
  const size_t state = ((size_t)slot_of * p.hv + h) * p.dk * p.dv;
  const int row0 = 16 * w + 4 * lg;                   // of this lane's four accumulator rows
  const int krow = 16 * w + lr;                       // of its operand rows

  for (;;) {
    int start, end;
    seq_bounds(t.cu, seq, p.tokens, &start, &end);
    start = __builtin_amdgcn_readfirstlane(start);
    end = __builtin_amdgcn_readfirstlane(end);
    const long long slot0 = start / kC + (long long)seq;
    f32x4 S[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = (w * MT + m) * 16 + 4 * lg + r;
        S[m][r] = t.h0 && kept && row < p.dk ? t.h0[state + (size_t)row * p.dv + col] : 0.f;
      }
    auto put_state = [&]() {
      if (srows)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float x[4] = {S[m][0], S[m][1], S[m][2], S[m][3]};
          put3<SLD>(Sl, SP, lr, (w * MT + m) * 16 + 4 * lg, x);
        }
    };
    In in;
    // columns behind d_k are never loaded and stay zero
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      in.k[ks] = zero_raw<NT>();
      if constexpr (PT > 0) in.q[ks] = zero_raw<NT>();
    }
    constexpr uint32_t es = NT == 1 ? 2 : 4;          // bytes of an input element
    // Rows behind the sequence's end take its last row instead: their beta is 0 and their outputs are not stored.
    auto load_rows = [&](int first, size_t cell) {
      const int n = end - first;
      const char* kb = static_cast<const char*>(t.k) + ((size_t)first * p.ks + kh * p.dk) * es;
      const char* qb = static_cast<const char*>(t.q) + ((size_t)first * p.qs + kh * p.dk) * es;
      const char* vb = static_cast<const char*>(t.v) + ((size_t)first * p.vs + h * p.dv) * es;
      const uint32_t row = min(krow, n - 1);
      const uint32_t ko = row * ((uint32_t)p.ks * es) + lg * 8 * es, qo = row * ((uint32_t)p.qs * es) + lg * 8 * es;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        if (ks * 32 + lg * 8 < p.dk) {
          in.k[ks] = raw_at<NT>(kb, ko + ks * 32 * es);
          if constexpr (PT > 0) in.q[ks] = raw_at<NT>(qb, qo + ks * 32 * es);
        }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        in.v[r] = at_byte<typename RawIn<NT>::type>(vb, (uint32_t)min(row0 + r, n - 1) * ((uint32_t)p.vs * es) + col * es);
      in.eG = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + row0);
    };
    auto load_inverse = [&](size_t cell) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= w / 2) in.t1[ks] = load_frag<3>(ws.t1 + cell * kTri * 3 * 64, w * 2 + ks, lane);
      in.eD = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + kC + row0);
      in.beta = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + 2 * kC + row0);
    };
    int vector_zero = 0;
    asm volatile("" : "+v"(vector_zero));             // a scalar load would be waited for with the LDS traffic
    auto load_state = [&](size_t cell, long long slot) {
      if (srows) {
        const uint4* kt = ws.kt + ((size_t)slot * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) in.kt[m][ks] = load_frag<NT>(kt, (w * MT + m) * 2 + ks, lane);
      }
      in.eGn = ws.gates[cell * 3 * kC + kC - 1 + vector_zero];
      if constexpr (PT > 0)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= w / 2) in.p[ks] = load_frag<PT, 3>(ws.p + cell * kTri * 3 * 64, w * 2 + ks, lane);
    };
    put_state();
    if (start < end) {
      const size_t cell = (size_t)slot0 * p.hv + h;
      load_rows(start, cell);
      load_inverse(cell);
      load_state(cell, slot0);
    }
    __syncthreads();
    long long slot = slot0;
    for (int first = start; first < end; first += kC) {
      const int n = min(kC, end - first);
      const bool more = first + kC < end;
      const size_t cell = (size_t)slot * p.hv + h;
      if (more) ++slot;                               // the last chunk's loads are repeated instead
      const int nfirst = more ? first + kC : first;
      const size_t ncell = (size_t)slot * p.hv + h;
      f32x4 kS[3], qS = zero4();
#pragma unroll
      for (int i = 0; i < 3; ++i) kS[i] = zero4();
      Frag<3> b[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) b[ks] = get<3, SLD>(Sl, SP, lr, ks * 32 + lg * 8);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) mma_by_term<NT, 3>(frag_of<NT>(in.k[ks]), b[ks], kS);
      float x[4];
      const float eg[4] = {in.eG.x, in.eG.y, in.eG.z, in.eG.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = fmaf(-eg[r], (kS[2][r] + kS[1][r]) + kS[0][r], row0 + r < n ? raw_value(in.v[r]) : 0.f);
      put3<kTok>(Nl, TP, lr, row0, x);
      if constexpr (PT > 0) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qS = mma<NT, PT>(frag_of<NT>(in.q[ks]), first_terms<PT>(b[ks]), qS);
#pragma unroll
        for (int r = 0; r < 4; ++r) qS[r] *= eg[r];
      }
      load_rows(nfirst, ncell);
      __syncthreads();
      f32x4 eT[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) eT[i] = zero4();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= w / 2) mma_by_term<3, 3>(in.t1[ks], get<3, kTok>(Nl, TP, lr, ks * 32 + lg * 8), eT);
      const f32x4 e = (eT[2] + eT[1]) + eT[0];
      const float ed[4] = {in.eD.x, in.eD.y, in.eD.z, in.eD.w}, bt[4] = {in.beta.x, in.beta.y, in.beta.z, in.beta.w};
      float u[4], ud[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        u[r] = bt[r] * e[r];
        ud[r] = ed[r] * u[r];
      }
      put3<kTok>(Dl, TP, lr, row0, ud);
      if constexpr (PT > 0) put<PT, kTok>(Ul, TP, lr, row0, u);
      load_inverse(ncell);
      if constexpr (PT == 0) {
        float* eo = ws.e + (cell * strips + strip) * kC * 16;
        float* so = ws.s0 + (cell * strips + strip) * DKP * 16;
#pragma unroll
        for (int r = 0; r < 4; ++r) eo[(row0 + r) * 16 + lr] = e[r];
        if (srows)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) so[((w * MT + m) * 16 + 4 * lg + r) * 16 + lr] = S[m][r];
      }
      __syncthreads();
      if (srows) {
        Frag<3> d[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) d[ks] = get<3, kTok>(Dl, TP, lr, ks * 32 + lg * 8);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 a[3];
          a[0] = S[m] * in.eGn;
          a[1] = a[2] = zero4();
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) mma_by_term<NT, 3>(in.kt[m][ks], d[ks], a);
          S[m] = a[0] + (a[1] + a[2]);
        }
      }
      put_state();
      if constexpr (PT > 0) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= w / 2) qS = mma<PT, PT>(in.p[ks], get<PT, kTok>(Ul, TP, lr, ks * 32 + lg * 8), qS);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row0 + r < n) {
            constexpr uint32_t os = PT == 2 ? 2 : 4;
            char* ob = static_cast<char*>(t.out) + ((size_t)first * p.hv + h) * p.dv * os;
            const uint32_t oo = (uint32_t)(row0 + r) * ((uint32_t)(p.hv * p.dv) * os) + col * os;
            if constexpr (PT == 2) *reinterpret_cast<bh*>(ob + oo) = f2bh(qS[r]);
            else *reinterpret_cast<float*>(ob + oo) = qS[r];
          }
      }
      load_state(ncell, slot);
      __syncthreads();
    }
    if (t.hT && kept && srows)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = (w * MT + m) * 16 + 4 * lg + r;
          if (row < p.dk) t.hT[state + (size_t)row * p.dv + col] = S[m][r];
        }
    if (!t.slots || !kept || next == 0x7fffffff) break;
    // the next sequence of this state row (rare)
    seq = next;
    __syncthreads();
    if (tid == 0) next = 0x7fffffff;
    __syncthreads();
    for (int i = seq + 1 + tid; i < p.sequences; i += 256)
      if (t.slots[i] == slot_of) atomicMin(&next, i);
    __syncthreads();
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
  const long long cells = f.slots * p.hv;
  const dim3 grid((unsigned)(cells < kMaxBlocks ? cells : kMaxBlocks));
  prof_begin(stream, GDN_KERNEL_PACKED_PREP);
#define GDN_PREP(NT, D)                                                                                                          \
  if (f.terms == NT && f.dkp == D) {                                                                                             \
    if (grad) hipLaunchKernelGGL((packed_prep_kernel<NT, D, true>), grid, dim3(256), 0, stream, p, t, s, f.slots);               \
    else hipLaunchKernelGGL((packed_prep_kernel<NT, D, false>), grid, dim3(256), 0, stream, p, t, s, f.slots);                   \
  }
  GDN_PREP(1, 32) GDN_PREP(1, 64) GDN_PREP(1, 128) GDN_PREP(3, 32) GDN_PREP(3, 64) GDN_PREP(3, 128)
#undef GDN_PREP
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_PREP);
  return e;
}

hipError_t packed_scan(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, bool grad, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  const int padded = (p.sequences * p.hv + 7) / 8 * 8;
  const dim3 grid((unsigned)padded * f.strips);
  prof_begin(stream, GDN_KERNEL_PACKED_SCAN);
#define GDN_SCAN(NT, D)                                                                                                          \
  if (f.terms == NT && f.dkp == D) {                                                                                             \
    if (grad) hipLaunchKernelGGL((packed_scan_kernel<NT, D, 0>), grid, dim3(256), 0, stream, p, t, s);                   \
    else if (p.out_bf16) hipLaunchKernelGGL((packed_scan_kernel<NT, D, 2>), grid, dim3(256), 0, stream, p, t, s);        \
    else hipLaunchKernelGGL((packed_scan_kernel<NT, D, 3>), grid, dim3(256), 0, stream, p, t, s);                        \
  }
  GDN_SCAN(1, 32) GDN_SCAN(1, 64) GDN_SCAN(1, 128) GDN_SCAN(3, 32) GDN_SCAN(3, 64) GDN_SCAN(3, 128)
#undef GDN_SCAN
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_SCAN);
  return e;
}

}  // namespace gdn
