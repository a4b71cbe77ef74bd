// Gradients of the packed gated delta rule.
//
// With the forward quantities of a chunk (gdn_packed.hip: B, P, E, G, e, U =
// beta e, S0), T = (I + diag(beta) B)^-1, and the gradients dO of its outputs and
// dS1 of the state after it:
//     dU = P^T dO + e^(Gn - G) K dS1,  W = T^T dU,  dN = beta W
//     dV = dN,  dbeta = W.e (per token)
//     dS0 = e^Gn dS1 + Q^T (e^G dO) - K^T (e^G dN)
//     D = E o (dO U^T),  M = -E o (dN U^T) below the diagonal
//     dQ = e^G dO S0^T + D K
//     rows = M K - e^G dN S0^T,  tail = e^(Gn - G) U dS1^T
//     cols = D^T Q + M^T K + tail,  dK = rows + cols
//     dG = q.dq + k.rows - k.cols per token; the last token's G also gets
//     sum k.tail + e^Gn <S0, dS1>;  dlog_gate = sums of dG from each token on.
// The T and T' forms need no division by beta, so beta = 0 is an ordinary value.
//
// Four launches: the preparation and the forward scan of gdn_packed.hip (which
// leave e and S0 of every chunk), scan_grad (the chunks in reverse order, 16
// columns of the state a workgroup, leaving W and dS1), and grads (every chunk
// and key head in parallel; it loops over the value heads that share the key
// head, so dq and dk are summed in one order).  No atomics.
#include "gdn_packed.h"

namespace gdn {
namespace {

constexpr int kLd = 68;     // row stride (floats) of a 64 x 64 fp32 tile in LDS

// What a chunk's step reads, by phase; loaded for the next chunk as soon as a
// phase has used it, as in the forward scan.
template <int NT, int DKP, int NS>
struct GradIn {
  static constexpr int KS = DKP / 32, MT = DKP >= 64 ? DKP / 64 : 1;
  typename RawIn<NT>::type dout[NS][4]; // of the chunk after the one whose step runs
  float4 deG;
  RawFrag<NT> k[KS];                // rows of K
  Frag<3> p[2];                     // P^T
  Frag<NT> qt[MT][2];               // Q^T
  float4 eD;
  float eGn;
  Frag<3> t2[2];                    // T^T
  float4 eG, beta;
  Frag<NT> kt[MT][2];               // K^T
};

// NS: strips of 16 columns of a workgroup.  One where all of them are resident at
// once, two to a CU; two where there are more: operands are fetched once for both
// (16 chunks, bf16: 2048 strips 250 us against 357 at d_k = d_v = 128, 225 against 285
// at 64, 257 against 286 at 32; 512 strips of equal lengths 71 against 86, but 420
// of three unequal sequences 32 against 27, since the longest sequence's steps are
// what lasts).  Eight wavefronts in two roles as in the forward scan gave 305 and 79.
template <int NT, int DKP, int NS>
__global__ __launch_bounds__(256, NT == 1 ? 2 : 1) void packed_scan_grad_kernel(SeqProblem p, PackedTensors t, PackedSpace ws) {
  using In = GradIn<NT, DKP, NS>;
  constexpr int KS = In::KS;
  constexpr int MT = In::MT;
  constexpr int SP = 16 * DKP, TP = 16 * kC;   // elements of a term's tile
  __shared__ __align__(16) bh Sl[NS][3 * SP];           // dS
  __shared__ __align__(16) bh Ol[NS][NT * TP];          // dO
  __shared__ __align__(16) bh Xl[NS][3 * TP];           // e^G dO
  __shared__ __align__(16) bh Ul[NS][3 * TP];           // dU
  __shared__ __align__(16) bh Yl[NS][3 * TP];           // -e^G dN
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64;
  const int lr = lane % 16, lg = lane / 16;
  int sh, strip;
  strip_of(blockIdx.x, (p.dv / 16 + NS - 1) / NS, &sh, &strip);
  strip *= NS;                                      // strips strip .. + NS; the last one of the last workgroup may not exist
  if (sh >= p.sequences * p.hv) return;
  const int h = sh % p.hv, kh = h / (p.hv / p.hk);
  const int seq = NS == 1 ? sh / p.hv : by_length(t.cu, p.sequences, p.tokens, sh / p.hv);   // NS = 1: all start at once
  const int col = strip * 16 + lr;
  const int strips = p.dv / 16;
  const auto there = [&](int i) { return NS == 1 || strip + i < strips; };
  const bool srows = DKP >= 64 || w < DKP / 16;
  const size_t state = ((size_t)seq * p.hv + h) * p.dk * p.dv;
  int start, end;
  seq_bounds(t.cu, seq, p.tokens, &start, &end);
  start = __builtin_amdgcn_readfirstlane(start);
  end = __builtin_amdgcn_readfirstlane(end);
  const long long slot0 = start / kC + (long long)seq;
  const int row0 = 16 * w + 4 * lg, krow = 16 * w + lr;
  const int tok_place = put_place(lr, row0);
  auto cell_of = [&](int c) { return (size_t)(slot0 + c) * p.hv + h; };

  f32x4 S[NS][MT];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = (w * MT + m) * 16 + 4 * lg + r;
        S[i][m][r] = t.dhT && row < p.dk && there(i) ? t.dhT[state + (size_t)row * p.dv + col + 16 * i] : 0.f;
      }
  auto put_state = [&](int i) {
    if (srows)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float x[4] = {S[i][m][0], S[i][m][1], S[i][m][2], S[i][m][3]};
        put<3, DKP>(Sl[i] + put_place(lr, (w * MT + m) * 16 + 4 * lg), x);
      }
  };
  In in;
  constexpr uint32_t es = NT == 1 ? 2 : 4;           // bytes of an input element
  const uint32_t ostride = (uint32_t)(p.hv * p.dv) * es;
  auto load_dout = [&](int c) {
    const int first = start + c * kC, n = end - first;
    const buf_t ob = buf(static_cast<const char*>(t.dout) + ((size_t)first * p.hv + h) * p.dv * es, span(n, ostride, p.dv * es));
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        in.dout[i][r] = value_at<NT>(ob, there(i) ? (row0 + r) * ostride + (col + 16 * i) * es : kNowhere);
    in.deG = *reinterpret_cast<const float4*>(ws.gates + cell_of(c) * 3 * kC + row0);
  };
  // chunk c's four tokens of this lane, plain and times e^G, as operand columns
  auto put_dout = [&]() {
    const float eg[4] = {in.deG.x, in.deG.y, in.deG.z, in.deG.w};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = raw_value(in.dout[i][r]);
        y[r] = eg[r] * x[r];
      }
      put<NT, kC>(Ol[i] + tok_place, x);
      put<3, kC>(Xl[i] + tok_place, y);
    }
  };
  int vector_zero = 0;
  asm volatile("" : "+v"(vector_zero));             // a scalar load would be waited for with the LDS traffic
  auto load_first = [&](int c) {
    const int first = start + c * kC, n = end - first;
    const size_t cell = cell_of(c);
    const uint32_t ks_b = (uint32_t)p.ks * es;
    const buf_t kb = buf(static_cast<const char*>(t.k) + ((size_t)first * p.ks + kh * p.dk) * es, span(n, ks_b, p.dk * es));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      in.k[ks] = raw_at<NT>(kb, ks * 32 + lg * 8 < p.dk ? krow * ks_b + (ks * 32 + lg * 8) * es : kNowhere);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) in.p[ks] = load_frag<3>(ws.p + cell * kTri * 3 * 64, w * 2 + ks, lane);
    if (srows) {
      const uint4* qt = ws.qt + ((size_t)(slot0 + c) * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) in.qt[m][ks] = load_frag<NT>(qt, (w * MT + m) * 2 + ks, lane);
    }
    in.eD = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + kC + row0);
    in.eGn = ws.gates[cell * 3 * kC + kC - 1 + vector_zero];
  };
  auto load_second = [&](int c) {
    const size_t cell = cell_of(c);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) in.t2[ks] = load_frag<3>(ws.t2 + cell * kTri * 3 * 64, w * 2 + ks, lane);
    in.eG = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + row0);
    in.beta = *reinterpret_cast<const float4*>(ws.gates + cell * 3 * kC + 2 * kC + row0);
  };
  auto load_third = [&](int c) {
    if (srows) {
      const uint4* kt = ws.kt + ((size_t)(slot0 + c) * p.hk + kh) * (DKP / 16) * 2 * NT * 64;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) in.kt[m][ks] = load_frag<NT>(kt, (w * MT + m) * 2 + ks, lane);
    }
  };
  const int last = (end - start + kC - 1) / kC - 1;
  if (last >= 0) {
    load_dout(last);
    put_dout();
    load_dout(last ? last - 1 : 0);
    load_first(last);
    load_second(last);
    load_third(last);
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) put_state(i);
  __syncthreads();
  for (int c = last; c >= 0; --c) {
    const int first = start + c * kC, n = min(kC, end - first);
    const size_t cell = cell_of(c);
    const int next = c ? c - 1 : 0, after = c > 1 ? c - 2 : 0;   // the first chunks' loads are repeated instead
    {
      const float ed[4] = {in.eD.x, in.eD.y, in.eD.z, in.eD.w};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        f32x4 a[3], u = zero4();
#pragma unroll
        for (int j = 0; j < 3; ++j) a[j] = zero4();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) mma_by_term<NT, 3>(frag_of<NT>(in.k[ks]), get<3, DKP>(Sl[i] + lane * 8, ks), a);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks >= w / 2) u = mma<3, NT>(in.p[ks], get<NT, kC>(Ol[i] + lane * 8, ks), u);
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = fmaf(ed[r], (a[2][r] + a[1][r]) + a[0][r], u[r]);
        put<3, kC>(Ul[i] + tok_place, x);
      }
    }
    if (srows) {
      // Q^T (e^G dO) needs nothing of this step: it fills the wait for the barrier
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const buf_t sb = buf(ws.ds + (cell * strips + strip + i) * DKP * 16, there(i) ? DKP * 16 * 4 : 0);
        Frag<3> xf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xf[ks] = get<3, kC>(Xl[i] + lane * 8, ks);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int r = 0; r < 4; ++r) store_at<4>(sb, (((w * MT + m) * 16 + 4 * lg + r) * 16 + lr) * 4, S[i][m][r]);
          S[i][m] = S[i][m] * in.eGn;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) S[i][m] = mma<NT, 3>(in.qt[m][ks], xf[ks], S[i][m]);
        }
      }
    }
    load_first(next);
    __syncthreads();
    {
      const float eg[4] = {in.eG.x, in.eG.y, in.eG.z, in.eG.w}, bt[4] = {in.beta.x, in.beta.y, in.beta.z, in.beta.w};
      const buf_t vb = buf(static_cast<char*>(t.dv) + ((size_t)first * p.hv + h) * p.dv * es, span(n, ostride, p.dv * es));
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        f32x4 a[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) a[j] = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks >= w / 2) mma_by_term<3, 3>(in.t2[ks], get<3, kC>(Ul[i] + lane * 8, ks), a);
        const f32x4 W = (a[2] + a[1]) + a[0];
        const buf_t wb = buf(ws.w + (cell * strips + strip + i) * kC * 16, there(i) ? kC * 16 * 4 : 0);
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = -eg[r] * (bt[r] * W[r]);
        put<3, kC>(Yl[i] + tok_place, y);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          store_at<4>(wb, ((row0 + r) * 16 + lr) * 4, W[r]);
          store_at<es>(vb, there(i) ? (row0 + r) * ostride + (col + 16 * i) * es : kNowhere, bt[r] * W[r]);
        }
      }
    }
    put_dout();                                      // the next chunk's: this one's have been read
    load_dout(after);
    load_second(next);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if (srows) {
        Frag<3> yf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) yf[ks] = get<3, kC>(Yl[i] + lane * 8, ks);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 b[3];
          b[0] = S[i][m];
          b[1] = b[2] = zero4();
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) mma_by_term<NT, 3>(in.kt[m][ks], yf[ks], b);
          S[i][m] = b[0] + (b[1] + b[2]);
        }
      }
      put_state(i);
    }
    load_third(next);
    __syncthreads();
  }
  if (t.dh0 && srows)
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = (w * MT + m) * 16 + 4 * lg + r;
          if (row < p.dk && there(i)) t.dh0[state + (size_t)row * p.dv + col + 16 * i] = S[i][m][r];
        }
}

// Sum over a wavefront's 64 lanes.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

// One workgroup per chunk and key head.  Nearly all of it is products over d_v
// (dO, W and e with S0 and dS1) on split operands, 690 MFMAs a row tile at 128 x
// 128, so the work is to keep those fed: 32 columns of d_v at a time, every
// operand that several wavefronts read is split once, by one wavefront, into an
// LDS buffer (two in turn, one barrier a step), its fp32 values fetched a step
// ahead.  Wavefronts w and w + 4 have row tile w and each half of the columns of
// d_k; the first four also have the 64 x 64 product D, the second M.
//
// Measured (8192 tokens, 16 key and 32 value heads of 128, bf16): 503 us, 31 us a
// chunk and value head on each CU, of which its 270 KB take 14 at the rate of a
// large copy and the MFMAs 7: one workgroup has a CU's registers and LDS, so its
// phases follow one another.  It spills 38 registers itself (14 at fp32 and d_k =
// 64, 141 above), which make most of the 249 MB that it writes; its outputs are 70.
// Sixteen wavefronts of 128 registers: 584 us; four of 512: 738 (105 spilled);
// eight that stay and fetch the next chunk's first operands ahead: 590 (81).
template <int NT, int DKP>
__global__ __launch_bounds__(512, 2) void packed_grads_kernel(SeqProblem p, PackedTensors t, PackedSpace ws, long long slots) {
  constexpr int NTI = DKP / 16, HT = NTI / 2;        // column tiles of d_k, and of a wavefront
  constexpr int KH = (HT + 1) / 2;                   // fragments of 32 columns that cover the latter
  constexpr uint32_t es = NT == 1 ? 2 : 4;
  constexpr int kFrag = 3 * 512;                     // bf16 values of a split fragment
  constexpr int kBuf = (8 + 2 * NTI) * kFrag;        // W, e: four tiles each; S0, dS1: NTI each
  __shared__ __align__(16) bh lds[2 * kBuf];
  __shared__ double Gs[kC];
  __shared__ float bs[kC], egs[kC], eds[kC], dGs[2][kC], part[16];   // beta, e^G, e^(Gn - G)
  float (*Dl)[kLd] = reinterpret_cast<float (*)[kLd]>(lds);            // D and M, when the buffers are done with
  float (*Ml)[kLd] = reinterpret_cast<float (*)[kLd]>(lds) + kC;
  static_assert(2 * kBuf * sizeof(bh) >= 2 * kC * kLd * sizeof(float), "D and M fit");
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lr = lane % 16, lg = lane / 16, w = wave & 3, half = wave >> 2;
  const int rep = p.hv / p.hk, strips = p.dv / 16, VS = (strips + 1) / 2;
  const long long items = slots * p.hk;
  const int row0 = 16 * w + 4 * lg, arow = 16 * w + lr;
  const uint32_t ks_b = (uint32_t)p.ks * es, qs_b = (uint32_t)p.qs * es, os_b = (uint32_t)(p.hv * p.dv) * es;
  const uint32_t dk_b = (uint32_t)p.dk * es, gs_b = (uint32_t)(p.hk * p.dk) * es;

  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int kh = (int)(item % p.hk);
    const long long slot = item / p.hk;
    int seq, first, n;
    if (!find_chunk(t.cu, p.sequences, p.tokens, slot, &seq, &first, &n)) continue;   // uniform over the workgroup
    first = __builtin_amdgcn_readfirstlane(first);
    n = __builtin_amdgcn_readfirstlane(n);
    const buf_t kb = buf(static_cast<const char*>(t.k) + ((size_t)first * p.ks + kh * p.dk) * es, span(n, ks_b, dk_b));
    const buf_t qb = buf(static_cast<const char*>(t.q) + ((size_t)first * p.qs + kh * p.dk) * es, span(n, qs_b, dk_b));
    const uint32_t tr = NTI * 2 * NT * 64;
    const buf_t ktb = buf(ws.kt + ((size_t)slot * p.hk + kh) * tr, tr * 16);
    const buf_t qtb = buf(ws.qt + ((size_t)slot * p.hk + kh) * tr, tr * 16);
    f32x4 gq[HT], gk[HT];
#pragma unroll
    for (int j = 0; j < HT; ++j) gq[j] = gk[j] = zero4();
    RawFrag<NT> rk[KH], rq[KH];
    // as accumulators hold them: a product with the identity, exact
    auto as_rows = [&](const RawFrag<NT> (&f)[KH], int j) {
      float one[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) one[i] = lg * 8 + i == (half * HT + j) % 2 * 16 + lr ? 1.f : 0.f;
      return mma<NT, 1>(frag_of<NT>(f[HT == 1 ? 0 : j / 2]), split8<1>(one), zero4());
    };
    // this lane's eight values of columns 32 vs .. of a row of e, W (64 rows) or S0, dS1 (DKP rows); behind the last strip
    // there is nothing
    uint4 we[2][2], sd[2][2];
    RawFrag<NT> dof;
    const uint32_t tok_b = strips * kC * 16 * 4, st_b = strips * DKP * 16 * 4;
    auto fetch = [&](int h, int vs) {
      const size_t cell = (size_t)slot * p.hv + h;
      const buf_t eb = buf(ws.e + cell * strips * kC * 16, tok_b), wb = buf(ws.w + cell * strips * kC * 16, tok_b);
      const buf_t sb = buf(ws.s0 + cell * strips * DKP * 16, st_b), db = buf(ws.ds + cell * strips * DKP * 16, st_b);
      const buf_t ob = buf(static_cast<const char*>(t.dout) + ((size_t)first * p.hv + h) * p.dv * es, span(n, os_b, p.dv * es));
      const int strip = vs * 2 + lg / 2, c8 = lg % 2 * 8;
      const uint32_t nowhere = strip < strips ? 0 : kNowhere;
      if (half == 0) {
        const uint32_t o = ((strip * kC + arow) * 16 + c8) * 4 | nowhere;
        we[0][0] = buf_load16(wb, o);
        we[0][1] = buf_load16(wb, o + 16);
        we[1][0] = buf_load16(eb, o);
        we[1][1] = buf_load16(eb, o + 16);
      }
      if (NTI == 8 || wave < NTI) {
        const uint32_t o = ((strip * DKP + wave * 16 + lr) * 16 + c8) * 4 | nowhere;
        sd[0][0] = buf_load16(sb, o);
        sd[0][1] = buf_load16(sb, o + 16);
        sd[1][0] = buf_load16(db, o);
        sd[1][1] = buf_load16(db, o + 16);
      }
      dof = raw_at<NT>(ob, arow * os_b + (strip * 16 + c8) * es | nowhere);
    };

    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
      const size_t cell = (size_t)slot * p.hv + h;
      auto eight = [&](const uint4 (&v)[2], float (&x)[8]) {
        const uint32_t a[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(a[j]);
      };
      auto put_frag = [&](bh* to, const float (&x)[8]) {
        const Frag<3> f = split8<3>(x);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(to + i * 512 + lane * 8) = as_bits(f.t[i]);
      };
      auto get_frag = [&](const bh* from) {
        Frag<3> f;
#pragma unroll
        for (int i = 0; i < 3; ++i) f.t[i] = as_frag(*reinterpret_cast<const uint4*>(from + i * 512 + lane * 8));
        return f;
      };
      fetch(h, 0);
      __syncthreads();                               // the previous head has read the tiles and gates
      if (tid < kC) {
        const float* gates = ws.gates + cell * 3 * kC;
        Gs[tid] = ws.g[cell * kC + tid];
        egs[tid] = gates[tid];
        eds[tid] = gates[kC + tid];
        bs[tid] = gates[2 * kC + tid];
      }
      f32x4 dq[HT], rw[HT], cl[HT], Z[4];             // Z: dO e^T in the first half, W e^T in the second
#pragma unroll
      for (int j = 0; j < HT; ++j) dq[j] = rw[j] = cl[j] = zero4();
#pragma unroll
      for (int j = 0; j < 4; ++j) Z[j] = zero4();
      float dbeta = 0.f, dot = 0.f;                  // of token arow over this lane's columns; of <S0, dS1>
      for (int vs = 0; vs < VS; ++vs) {
        bh* buf0 = lds + (vs & 1) * kBuf;
        if (half == 0) {
          float x[8], y[8];
          eight(we[0], x);
          eight(we[1], y);
#pragma unroll
          for (int j = 0; j < 8; ++j) dbeta = fmaf(x[j], y[j], dbeta);
          put_frag(buf0 + w * kFrag, x);
          put_frag(buf0 + (4 + w) * kFrag, y);
        }
        if (NTI == 8 || wave < NTI) {
          float x[8], y[8];
          eight(sd[0], x);
          eight(sd[1], y);
#pragma unroll
          for (int j = 0; j < 8; ++j) dot = fmaf(x[j], y[j], dot);
          put_frag(buf0 + (8 + wave) * kFrag, x);
          put_frag(buf0 + (8 + NTI + wave) * kFrag, y);
        }
        const Frag<NT> ao = frag_of<NT>(dof);
        if (vs + 1 < VS) fetch(h, vs + 1);
        __syncthreads();
        const Frag<3> aw = get_frag(buf0 + w * kFrag), ae = get_frag(buf0 + (4 + w) * kFrag);
#pragma unroll
        for (int j = 0; j < HT; ++j) {
          const int tile = half * HT + j;
          const Frag<3> s = get_frag(buf0 + (8 + tile) * kFrag), d = get_frag(buf0 + (8 + NTI + tile) * kFrag);
          dq[j] = mma<NT, 3>(ao, s, dq[j]);
          rw[j] = mma<3, 3>(aw, s, rw[j]);
          cl[j] = mma<3, 3>(ae, d, cl[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= w) {
            const Frag<3> b = get_frag(buf0 + (4 + j) * kFrag);
            if (half == 0) Z[j] = mma<NT, 3>(ao, b, Z[j]);
            else Z[j] = mma<3, 3>(aw, b, Z[j]);
          }
      }
      if (half == 0) {
        dbeta += __shfl_xor(dbeta, 16);
        dbeta += __shfl_xor(dbeta, 32);
        if (lg == 0 && arow < n) t.dbeta[(size_t)(first + arow) * p.hv + h] = dbeta;
      }
      // rows of K and Q in this wavefront's columns
#pragma unroll
      for (int j = 0; j < KH; ++j) {
        const int c = (half * HT / 2 + j) * 32 + lg * 8;
        const uint32_t nowhere = c < p.dk ? 0 : kNowhere;
        rk[j] = raw_at<NT>(kb, arow * ks_b + c * es | nowhere);
        rq[j] = raw_at<NT>(qb, arow * qs_b + c * es | nowhere);
      }
      // K^T and Q^T for what follows, on their way over the next barriers
      Frag<NT> kf[2][HT], qf[2][HT];
      auto fetch_transposed = [&](int ks) {
#pragma unroll
        for (int j = 0; j < HT; ++j) {
          const uint32_t o = (((half * HT + j) * 2 + ks) * NT * 64 + lane) * 16;
          kf[ks][j] = frag_at<NT>(ktb, o);
          qf[ks][j] = frag_at<NT>(qtb, o);
        }
      };
      if constexpr (NT == 1) fetch_transposed(0);
      float tails = 0.f;
#pragma unroll
      for (int j = 0; j < HT; ++j) {
        const f32x4 kd = as_rows(rk, j);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = row0 + r;
          dq[j][r] *= egs[i];
          rw[j][r] *= -bs[i] * egs[i];
          cl[j][r] *= bs[i] * eds[i];
          tails = fmaf(kd[r], cl[j][r], tails);
        }
      }
      tails = wave_sum(tails);
      dot = wave_sum(dot);
      __syncthreads();                               // the last buffers have been read
      if (lane == 0) {
        part[wave] = tails;
        part[8 + wave] = dot;
      }
      {
        float (*to)[kLd] = half == 0 ? Dl : Ml;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 16 * j + lr;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = row0 + r;
            const float E = i >= c + half ? exp2_of((float)(Gs[i] - Gs[c])) * bs[c] : 0.f;   // M: below the diagonal
            to[i][c] = j <= w ? (half == 0 ? E : -E * bs[i]) * Z[j][r] : 0.f;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int k8 = ks * 32 + lg * 8;
        if (NT == 3 || ks == 1) fetch_transposed(ks);
        if (ks <= w / 2) {
          const Frag<3> ad = frag_f32<3>(&Dl[arow][k8]), am = frag_f32<3>(&Ml[arow][k8]);
#pragma unroll
          for (int j = 0; j < HT; ++j) {
            dq[j] = mma<3, NT>(ad, kf[ks][j], dq[j]);
            rw[j] = mma<3, NT>(am, kf[ks][j], rw[j]);
          }
        }
        if (ks >= w / 2) {
          float x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = Dl[k8 + j][arow];
            y[j] = Ml[k8 + j][arow];
          }
          const Frag<3> bd = split8<3>(x), bm = split8<3>(y);
#pragma unroll
          for (int j = 0; j < HT; ++j) {
            cl[j] = mma<3, NT>(bd, qf[ks][j], cl[j]);
            cl[j] = mma<3, NT>(bm, kf[ks][j], cl[j]);
          }
        }
      }
      float sum[4] = {};
#pragma unroll
      for (int j = 0; j < HT; ++j) {
        const f32x4 kd = as_rows(rk, j), qd = as_rows(rq, j);
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += qd[r] * dq[j][r] + kd[r] * (rw[j][r] - cl[j][r]);
        gq[j] += dq[j];
        gk[j] += rw[j] + cl[j];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) sum[r] += __shfl_xor(sum[r], m);
        if (lr == 0) dGs[half][row0 + r] = sum[r];
      }
      __syncthreads();
      if (wave == 0) {
        // the chunk's last G is every padded row's too, so its share can sit in row 63
        double s = (double)dGs[0][lane] + dGs[1][lane];
        if (lane == kC - 1) {
          double tail = 0.0, states = 0.0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            tail += part[i];
            states += part[8 + i];
          }
          s += tail + (double)egs[kC - 1] * states;
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
          const double o = __shfl_down(s, m);
          if (lane + m < 64) s += o;
        }
        if (lane < n) t.dg[(size_t)(first + lane) * p.hv + h] = (float)s;
      }
    }
    const buf_t dqb = buf(static_cast<char*>(t.dq) + ((size_t)first * p.hk + kh) * p.dk * es, span(n, gs_b, dk_b));
    const buf_t dkb = buf(static_cast<char*>(t.dk) + ((size_t)first * p.hk + kh) * p.dk * es, span(n, gs_b, dk_b));
#pragma unroll
    for (int j = 0; j < HT; ++j) {
      const int c = (half * HT + j) * 16 + lr;
      const uint32_t nowhere = c < p.dk ? 0 : kNowhere;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        store_at<es>(dqb, (row0 + r) * gs_b + c * es | nowhere, gq[j][r]);
        store_at<es>(dkb, (row0 + r) * gs_b + c * es | nowhere, gk[j][r]);
      }
    }
  }
}

}  // namespace

hipError_t packed_scan_grad(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  const unsigned heads = (p.sequences * p.hv + 7) / 8 * 8;
  const bool pairs = f.strips > 1 && (long long)p.sequences * p.hv * f.strips > 512;   // more than two strips a CU
  const dim3 grid(heads * (pairs ? (f.strips + 1) / 2 : f.strips));
  prof_begin(stream, GDN_KERNEL_PACKED_SCAN_GRAD);
#define GDN_SCAN(NT, D)                                                                                            \
  if (f.terms == NT && f.dkp == D) {                                                                               \
    if (pairs) hipLaunchKernelGGL((packed_scan_grad_kernel<NT, D, 2>), grid, dim3(256), 0, stream, p, t, s);       \
    else hipLaunchKernelGGL((packed_scan_grad_kernel<NT, D, 1>), grid, dim3(256), 0, stream, p, t, s);             \
  }
  GDN_SCAN(1, 32) GDN_SCAN(1, 64) GDN_SCAN(1, 128) GDN_SCAN(3, 32) GDN_SCAN(3, 64) GDN_SCAN(3, 128)
#undef GDN_SCAN
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_SCAN_GRAD);
  return e;
}

hipError_t packed_grads(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  const long long items = f.slots * p.hk;
  const dim3 grid((unsigned)(items < kMaxBlocks ? items : kMaxBlocks));
  prof_begin(stream, GDN_KERNEL_PACKED_GRADS);
#define GDN_GRADS(NT, D) \
  if (f.terms == NT && f.dkp == D) hipLaunchKernelGGL((packed_grads_kernel<NT, D>), grid, dim3(512), 0, stream, p, t, s, f.slots);
  GDN_GRADS(1, 32) GDN_GRADS(1, 64) GDN_GRADS(1, 128) GDN_GRADS(3, 32) GDN_GRADS(3, 64) GDN_GRADS(3, 128)
#undef GDN_GRADS
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_GRADS);
  return e;
}

}  // namespace gdn
