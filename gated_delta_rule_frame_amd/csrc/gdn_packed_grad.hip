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
template <int NT, int DKP>
struct GradIn {
  static constexpr int KS = DKP / 32, MT = DKP >= 64 ? DKP / 64 : 1;
  typename RawIn<NT>::type dout[4]; // of the chunk after the one whose step runs
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

template <int NT, int DKP>
__global__ __launch_bounds__(256, NT == 1 ? 2 : 1) void packed_scan_grad_kernel(SeqProblem p, PackedTensors t, PackedSpace ws) {
  using In = GradIn<NT, DKP>;
  constexpr int KS = In::KS;
  constexpr int MT = In::MT;
  constexpr int SP = 16 * DKP, TP = 16 * kC;   // elements of a term's tile
  __shared__ __align__(16) bh Sl[3 * SP];           // dS
  __shared__ __align__(16) bh Ol[NT * TP];          // dO
  __shared__ __align__(16) bh Xl[3 * TP];           // e^G dO
  __shared__ __align__(16) bh Ul[3 * TP];           // dU
  __shared__ __align__(16) bh Yl[3 * TP];           // -e^G dN
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64;
  const int lr = lane % 16, lg = lane / 16;
  int sh, strip;
  strip_of(blockIdx.x, p.dv / 16, &sh, &strip);
  if (sh >= p.sequences * p.hv) return;
  const int h = sh % p.hv, kh = h / (p.hv / p.hk), seq = sh / p.hv;
  const int col = strip * 16 + lr;
  const int strips = p.dv / 16;
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

  f32x4 S[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = (w * MT + m) * 16 + 4 * lg + r;
      S[m][r] = t.dhT && row < p.dk ? t.dhT[state + (size_t)row * p.dv + col] : 0.f;
    }
  auto put_state = [&]() {
    if (srows)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float x[4] = {S[m][0], S[m][1], S[m][2], S[m][3]};
        put<3, DKP>(Sl + put_place(lr, (w * MT + m) * 16 + 4 * lg), x);
      }
  };
  In in;
  constexpr uint32_t es = NT == 1 ? 2 : 4;           // bytes of an input element
  const uint32_t ostride = (uint32_t)(p.hv * p.dv) * es;
  auto load_dout = [&](int c) {
    const int first = start + c * kC, n = end - first;
    const buf_t ob = buf(static_cast<const char*>(t.dout) + ((size_t)first * p.hv + h) * p.dv * es, span(n, ostride, p.dv * es));
#pragma unroll
    for (int r = 0; r < 4; ++r) in.dout[r] = value_at<NT>(ob, (row0 + r) * ostride + col * es);
    in.deG = *reinterpret_cast<const float4*>(ws.gates + cell_of(c) * 3 * kC + row0);
  };
  // chunk c's four tokens of this lane, plain and times e^G, as operand columns
  auto put_dout = [&]() {
    const float eg[4] = {in.deG.x, in.deG.y, in.deG.z, in.deG.w};
    float x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = raw_value(in.dout[r]);
      y[r] = eg[r] * x[r];
    }
    put<NT, kC>(Ol + tok_place, x);
    put<3, kC>(Xl + tok_place, y);
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
  put_state();
  __syncthreads();
  for (int c = last; c >= 0; --c) {
    const int first = start + c * kC, n = min(kC, end - first);
    const size_t cell = cell_of(c);
    const int next = c ? c - 1 : 0, after = c > 1 ? c - 2 : 0;   // the first chunks' loads are repeated instead
    f32x4 a[3], u = zero4();
#pragma unroll
    for (int i = 0; i < 3; ++i) a[i] = zero4();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mma_by_term<NT, 3>(frag_of<NT>(in.k[ks]), get<3, DKP>(Sl + lane * 8, ks), a);
    const float ed[4] = {in.eD.x, in.eD.y, in.eD.z, in.eD.w};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) u = mma<3, NT>(in.p[ks], get<NT, kC>(Ol + lane * 8, ks), u);
    {
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = fmaf(ed[r], (a[2][r] + a[1][r]) + a[0][r], u[r]);
      put<3, kC>(Ul + tok_place, x);
    }
    if (srows) {
      // Q^T (e^G dO) needs nothing of this step: it fills the wait for the barrier
      float* so = ws.ds + (cell * strips + strip) * DKP * 16;
      Frag<3> xf[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) xf[ks] = get<3, kC>(Xl + lane * 8, ks);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int r = 0; r < 4; ++r) so[((w * MT + m) * 16 + 4 * lg + r) * 16 + lr] = S[m][r];
        S[m] = S[m] * in.eGn;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) S[m] = mma<NT, 3>(in.qt[m][ks], xf[ks], S[m]);
      }
    }
    load_first(next);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) a[i] = zero4();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) mma_by_term<3, 3>(in.t2[ks], get<3, kC>(Ul + lane * 8, ks), a);
    {
      const f32x4 W = (a[2] + a[1]) + a[0];
      const float eg[4] = {in.eG.x, in.eG.y, in.eG.z, in.eG.w}, bt[4] = {in.beta.x, in.beta.y, in.beta.z, in.beta.w};
      float* wo = ws.w + (cell * strips + strip) * kC * 16;
      const buf_t vb = buf(static_cast<char*>(t.dv) + ((size_t)first * p.hv + h) * p.dv * es, span(n, ostride, p.dv * es));
      float y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = -eg[r] * (bt[r] * W[r]);
      put<3, kC>(Yl + tok_place, y);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        wo[(row0 + r) * 16 + lr] = W[r];
        store_at<es>(vb, (row0 + r) * ostride + col * es, bt[r] * W[r]);
      }
    }
    put_dout();                                      // the next chunk's: this one's have been read
    load_dout(after);
    load_second(next);
    __syncthreads();
    if (srows) {
      Frag<3> yf[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) yf[ks] = get<3, kC>(Yl + lane * 8, ks);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 b[3];
        b[0] = S[m];
        b[1] = b[2] = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) mma_by_term<NT, 3>(in.kt[m][ks], yf[ks], b);
        S[m] = b[0] + (b[1] + b[2]);
      }
    }
    put_state();
    load_third(next);
    __syncthreads();
  }
  if (t.dh0 && srows)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = (w * MT + m) * 16 + 4 * lg + r;
        if (row < p.dk) t.dh0[state + (size_t)row * p.dv + col] = S[m][r];
      }
}

// Sum over a wavefront's 64 lanes.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

template <int NT, int DKP>
__global__ __launch_bounds__(256, 1) void packed_grads_kernel(SeqProblem p, PackedTensors t, PackedSpace ws, long long slots) {
  constexpr int NTI = DKP / 16;                      // column tiles of d_k
  __shared__ __align__(16) float Dl[kC][kLd];        // D = E o (dO U^T)
  __shared__ __align__(16) float Ml[kC][kLd];        // M
  __shared__ double Gs[kC];
  __shared__ float bs[kC], dGs[kC], part[8];
  const int tid = threadIdx.x, lane = tid % 64, w = tid / 64;
  const int lr = lane % 16, lg = lane / 16;
  const int rep = p.hv / p.hk, strips = p.dv / 16, VS = (strips + 1) / 2;
  const long long items = slots * p.hk;

  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int kh = (int)(item % p.hk);
    const long long slot = item / p.hk;
    int seq, first, n;
    if (!find_chunk(t.cu, p.sequences, p.tokens, slot, &seq, &first, &n)) continue;   // uniform over the workgroup
    const int row0 = 16 * w + 4 * lg, arow = 16 * w + lr;
    const size_t at = ((size_t)slot * p.hk + kh) * NTI * 2 * NT * 64;
    const uint4* kt = ws.kt + at;
    const uint4* qt = ws.qt + at;
    f32x4 gq[NTI], gk[NTI];
#pragma unroll
    for (int j = 0; j < NTI; ++j) gq[j] = gk[j] = zero4();

    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
      const size_t cell = (size_t)slot * p.hv + h;
      const float* gates = ws.gates + cell * 3 * kC;
      const float* ec = ws.e + cell * strips * kC * 16;
      const float* wc = ws.w + cell * strips * kC * 16;
      const float* sc = ws.s0 + cell * strips * DKP * 16;
      const float* dc = ws.ds + cell * strips * DKP * 16;
      __syncthreads();                               // the previous head has read the tiles
      if (tid < kC) {
        Gs[tid] = ws.g[cell * kC + tid];
        bs[tid] = gates[2 * kC + tid];
      }
      f32x4 dq[NTI], rw[NTI], cl[NTI], D[4], X[4];
#pragma unroll
      for (int j = 0; j < NTI; ++j) dq[j] = rw[j] = cl[j] = zero4();
#pragma unroll
      for (int j = 0; j < 4; ++j) D[j] = X[j] = zero4();
      float dbeta = 0.f;                             // of token arow, this lane's columns
      // products over d_v, 32 columns (two strips) at a time
      for (int vs = 0; vs < VS; ++vs) {
        const int strip = vs * 2 + lg / 2, c8 = lg % 2 * 8;
        const bool in = strip < strips;
        auto tile = [&](const float* base, int rows, int row) {   // [strip][rows][16]
          return in ? frag_f32<3>(base + ((size_t)strip * rows + row) * 16 + c8) : zero_frag<3>();
        };
        const Frag<NT> ao = in && arow < n
            ? frag_in<NT>(t.dout, ((size_t)(first + arow) * p.hv + h) * p.dv + strip * 16 + c8) : zero_frag<NT>();
        const Frag<3> aw = tile(wc, kC, arow), ae = tile(ec, kC, arow);
        if (in) {
          const float* a = wc + ((size_t)strip * kC + arow) * 16 + c8;
          const float* b = ec + ((size_t)strip * kC + arow) * 16 + c8;
#pragma unroll
          for (int j = 0; j < 8; ++j) dbeta = fmaf(a[j], b[j], dbeta);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= w) {
            const Frag<3> b = j == w ? ae : tile(ec, kC, 16 * j + lr);
            D[j] = mma<NT, 3>(ao, b, D[j]);
            X[j] = mma<3, 3>(aw, b, X[j]);
          }
#pragma unroll
        for (int j = 0; j < NTI; ++j) {
          const Frag<3> s = tile(sc, DKP, 16 * j + lr);
          dq[j] = mma<NT, 3>(ao, s, dq[j]);
          rw[j] = mma<3, 3>(aw, s, rw[j]);
          cl[j] = mma<3, 3>(ae, tile(dc, DKP, 16 * j + lr), cl[j]);
        }
      }
      dbeta += __shfl_xor(dbeta, 16);
      dbeta += __shfl_xor(dbeta, 32);
      if (lg == 0 && arow < n) t.dbeta[(size_t)(first + arow) * p.hv + h] = dbeta;
      __syncthreads();                               // Gs, bs
      float tails = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = row0 + r;
        const float eg = gates[i], ed = gates[kC + i], b = bs[i];
        const bool in = i < n;
#pragma unroll
        for (int j = 0; j < NTI; ++j) {
          dq[j][r] *= eg;
          rw[j][r] *= -b * eg;
          cl[j][r] *= b * ed;
          const int c = 16 * j + lr;
          if (in && c < p.dk) tails = fmaf(elem_in<NT>(t.k, (size_t)(first + i) * p.ks + kh * p.dk + c), cl[j][r], tails);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 16 * j + lr;
          const float E = i >= c ? exp2_of((float)(Gs[i] - Gs[c])) * bs[c] : 0.f;
          Dl[i][c] = E * D[j][r];
          Ml[i][c] = i > c ? -E * b * X[j][r] : 0.f;
        }
      }
      // <S0, dS1>: the workgroup's threads over the cell
      float dot = 0.f;
      for (int i = tid; i < strips * DKP * 4; i += 256) {
        const float4 a = reinterpret_cast<const float4*>(sc)[i], b = reinterpret_cast<const float4*>(dc)[i];
        dot += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
      }
      tails = wave_sum(tails);
      dot = wave_sum(dot);
      if (lane == 0) {
        part[w] = tails;
        part[4 + w] = dot;
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int k8 = ks * 32 + lg * 8;
        Frag<3> ad, am, bd, bm;
        if (ks <= w / 2) {
          ad = frag_f32<3>(&Dl[arow][k8]);
          am = frag_f32<3>(&Ml[arow][k8]);
        }
        if (ks >= w / 2) {
          float x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = Dl[k8 + j][arow];
            y[j] = Ml[k8 + j][arow];
          }
          bd = split8<3>(x);
          bm = split8<3>(y);
        }
#pragma unroll
        for (int j = 0; j < NTI; ++j) {
          const Frag<NT> kf = load_frag<NT>(kt, j * 2 + ks, lane);
          if (ks <= w / 2) {
            dq[j] = mma<3, NT>(ad, kf, dq[j]);
            rw[j] = mma<3, NT>(am, kf, rw[j]);
          }
          if (ks >= w / 2) {
            cl[j] = mma<3, NT>(bd, load_frag<NT>(qt, j * 2 + ks, lane), cl[j]);
            cl[j] = mma<3, NT>(bm, kf, cl[j]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = row0 + r;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NTI; ++j) {
          const int c = 16 * j + lr;
          const bool in = i < n && c < p.dk;
          const float q = in ? elem_in<NT>(t.q, (size_t)(first + i) * p.qs + kh * p.dk + c) : 0.f;
          const float k = in ? elem_in<NT>(t.k, (size_t)(first + i) * p.ks + kh * p.dk + c) : 0.f;
          s += q * dq[j][r] + k * (rw[j][r] - cl[j][r]);
          gq[j][r] += dq[j][r];
          gk[j][r] += rw[j][r] + cl[j][r];
        }
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) s += __shfl_xor(s, m);
        if (lr == 0) dGs[i] = s;
      }
      __syncthreads();
      if (w == 0) {
        // the chunk's last G is every padded row's too, so its share can sit in row 63
        double s = dGs[lane];
        if (lane == kC - 1)
          s += (double)(part[0] + part[1] + part[2] + part[3]) + (double)gates[kC - 1] * (part[4] + part[5] + part[6] + part[7]);
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
          const double o = __shfl_down(s, m);
          if (lane + m < 64) s += o;
        }
        if (lane < n) t.dg[(size_t)(first + lane) * p.hv + h] = (float)s;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < NTI; ++j) {
        const int c = 16 * j + lr;
        if (row0 + r < n && c < p.dk) {
          const size_t o = ((size_t)(first + row0 + r) * p.hk + kh) * p.dk + c;
          store_scalar(t.dq, o, gq[j][r], NT == 1);
          store_scalar(t.dk, o, gk[j][r], NT == 1);
        }
      }
  }
}

}  // namespace

hipError_t packed_scan_grad(const SeqProblem& p, const PackedTensors& t, const PackedSpace& s, hipStream_t stream) {
  const PackedPlan f = packed_plan(p);
  const int padded = (p.sequences * p.hv + 7) / 8 * 8;
  const dim3 grid((unsigned)padded * f.strips);
  prof_begin(stream, GDN_KERNEL_PACKED_SCAN_GRAD);
#define GDN_SCAN(NT, D) \
  if (f.terms == NT && f.dkp == D) hipLaunchKernelGGL((packed_scan_grad_kernel<NT, D>), grid, dim3(256), 0, stream, p, t, s);
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
  if (f.terms == NT && f.dkp == D) hipLaunchKernelGGL((packed_grads_kernel<NT, D>), grid, dim3(256), 0, stream, p, t, s, f.slots);
  GDN_GRADS(1, 32) GDN_GRADS(1, 64) GDN_GRADS(1, 128) GDN_GRADS(3, 32) GDN_GRADS(3, 64) GDN_GRADS(3, 128)
#undef GDN_GRADS
  const hipError_t e = hipGetLastError();
  prof_end(stream, GDN_KERNEL_PACKED_GRADS);
  return e;
}

}  // namespace gdn
