// Chunked gated delta rule with a scalar gate: intra-chunk kernel and forward
// scan. Formulas, layouts and the rounding rule are in kda_gdn.h.
//
//   gdn_intra_kernel  one workgroup per (chunk, group of value heads of a q/k
//                     head): q k^T and k k^T once on the matrix cores for the
//                     whole group, then per value head the gate, the FP32
//                     solve for M, and M, P and the row factors written out.
//   gdn_scan_kernel   one wave per 16 columns of one (sequence, value head)
//                     state, walking the chunks in order; S stays in the
//                     wave's accumulators.
#include "kda_gdn.h"

namespace kda {

// ------------------------------------------------------------------ intra
constexpr int kGdnAS = kC + 4;  // row stride of the FP32 A and P in LDS

template <typename T, int K, bool BWD>
__global__ void __launch_bounds__(256)
gdn_intra_kernel(const T* __restrict__ q, const T* __restrict__ k, GdnGate gate,
                 const T* __restrict__ beta, const int32_t* __restrict__ cu,
                 const int* __restrict__ table, int N, int T_, int H, int HV, int hpw, int l2,
                 float scale, float* __restrict__ ws_scal, T* __restrict__ ws_fwd,
                 T* __restrict__ ws_bwd) {
  constexpr int NK = K / 32;
  __shared__ __attribute__((aligned(16))) float sA[kC * kGdnAS];
  __shared__ __attribute__((aligned(16))) float sP[kC * kGdnAS];
  __shared__ double sG[kC];
  __shared__ __attribute__((aligned(16))) float sB[kC], sRq[kC], sRk[kC];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nh = HV / hpw;
  const int j = blockIdx.x / nh, hv0 = (blockIdx.x % nh) * hpw, h = hv0 / (HV / H);
  const ChunkGeo geo = chunk_geo(j, cu, table, N, T_);
  if (!geo.ok) return;
  const int L = geo.L;

  // k k^T and q k^T: row tile I = wave, column tiles J <= I (rows past L repeat
  // row L - 1; their entries are dropped below)
  Op8<T> kf[NK], qf[NK];
  {
    const int64_t off = ((geo.t0 + min(16 * wave + l16, L - 1)) * H + h) * K + 8 * g;
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      ld_op(kf[s], k + off + 32 * s);
      ld_op(qf[s], q + off + 32 * s);
    }
  }
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int J = 0; J < 4; ++J) {
    kk[J] = qk[J] = zero4();
    if (J > wave) continue;
    Op8<T> kj[NK];
    const int64_t off = ((geo.t0 + min(16 * J + l16, L - 1)) * H + h) * K + 8 * g;
#pragma unroll
    for (int s = 0; s < NK; ++s) ld_op(kj[s], k + off + 32 * s);
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      kk[J] = mma8(kf[s], kj[s], kk[J]);
      qk[J] = mma8(qf[s], kj[s], qk[J]);
    }
  }
  {
    float nk = 0.f, nq = 0.f;
    if (l2) {
#pragma unroll
      for (int s = 0; s < NK; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = op_get(kf[s], i), b = op_get(qf[s], i);
          nk = fmaf(a, a, nk);
          nq = fmaf(b, b, nq);
        }
      nk += __shfl_xor(nk, 16);
      nq += __shfl_xor(nq, 16);
      nk += __shfl_xor(nk, 32);
      nq += __shfl_xor(nq, 32);
    }
    if (g == 0) {
      sRk[16 * wave + l16] = l2 ? l2norm_inv(nk) : 1.f;
      sRq[16 * wave + l16] = l2 ? l2norm_inv(nq) : 1.f;
    }
  }

  for (int hh = 0; hh < hpw; ++hh) {
    const int hv = hv0 + hh;
    const size_t ch = (size_t)j * HV + hv;
    __syncthreads();  // row norms written; the previous head's reads done
    // gate sums in double: differences G_i - G_j stay exact to FP32 for any gate
    if (wave == 0) {
      float gn = 0.f, b = 0.f;
      if (lane < L) {
        const int64_t at = (geo.t0 + lane) * HV + hv;
        float xb, sc;
        gn = gdn_gate(gate, at, hv, &xb, &sc);
        b = to_f32(beta[at]);
      }
      double G = (double)gn * 1.4426950408889634074;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(G, d);
        if (lane >= d) G += y;
      }
      const double Gl = __shfl(G, L - 1);
      sG[lane] = G;
      sB[lane] = b;
      float* sc = ws_scal + ch * (kGdnScal * kC);
      const float rk = sRk[lane], rq = sRq[lane], eg = ex2((float)G);
      const bool ok = lane < L;
      sc[kSk * kC + lane] = ok ? eg * rk : 0.f;
      sc[kSq * kC + lane] = ok ? eg * rq * scale : 0.f;
      sc[kSe * kC + lane] = ok ? ex2((float)(Gl - G)) * rk : 0.f;
      sc[kSb * kC + lane] = b;
      if constexpr (BWD) {
        if (!ok) sc[kSp * kC + lane] = 0.f;
        reinterpret_cast<double*>(sc + kSG * kC)[lane] = G;
        sc[kSrq * kC + lane] = rq;
        sc[kSrk * kC + lane] = rk;
      }
      sc[kSl * kC + lane] = ex2((float)Gl);
    }
    __syncthreads();
#pragma unroll
    for (int J = 0; J < 4; ++J) {
      if (J > wave && (J != wave + 1 || (wave & 1))) continue;  // tiles no fragment covers
      const int jj = 16 * J + l16;
      const double gj = sG[jj];
      const float rkj = sRk[jj];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * wave + 4 * g + e;
        float a = 0.f, p = 0.f;
        if (i >= jj && i < L) {
          const float d = ex2((float)(sG[i] - gj)) * rkj;
          a = i > jj ? kk[J][e] * d * sRk[i] : 0.f;
          p = qk[J][e] * d * sRq[i] * scale;
          if (BWD && i == jj) {
            ws_scal[ch * (kGdnScal * kC) + kSp * kC + i] = p;
            p = 0.f;
          }
        }
        sA[i * kGdnAS + jj] = a;
        sP[i * kGdnAS + jj] = p;
      }
    }
    __syncthreads();

    // M = (I + Abar diag b)^-1 Abar in place. Diagonal 16 x 16 blocks by
    // forward substitution, wave d, lane = column:
    //   m_i = a_i - sum_{n < i} a_in b_n m_n
    if (lane < 16) {
      const int d = wave;
      float x[16], bb[16];
#pragma unroll
      for (int n = 0; n < 16; n += 4) lds4(sB + 16 * d + n, bb + n);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float row[16];
#pragma unroll
        for (int n = 0; n < 16; n += 4) lds4(sA + (16 * d + i) * kGdnAS + 16 * d + n, row + n);
        float s = sA[(16 * d + i) * kGdnAS + 16 * d + lane];
#pragma unroll
        for (int n = 0; n < i; ++n) s = fmaf(-row[n], bb[n] * x[n], s);
        x[i] = s;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sA[(16 * d + i) * kGdnAS + 16 * d + lane] = x[i];
    }
    __syncthreads();
    // block rows, wave J owns block column J: X = Abar_IJ - sum_{J <= N < I} Abar_IN (b M_NJ),
    // M_IJ = X - M_II (b X), on the FP32 matrix cores (an accumulator tile is the
    // next product's operand over its rows)
    {
      f32x4 col[4];
#pragma unroll
      for (int J = 0; J < 3; ++J) {
        if (J != wave) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) col[J][e] = sA[(16 * J + 4 * g + e) * kGdnAS + 16 * J + l16];
#pragma unroll
        for (int I = J + 1; I < 4; ++I) {
          f32x4 x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = sA[(16 * I + 4 * g + e) * kGdnAS + 16 * J + l16];
#pragma unroll
          for (int n = J; n < I; ++n) {
            float a4[4], b4[4];
            lds4(sA + (16 * I + l16) * kGdnAS + 16 * n + 4 * g, a4);
            lds4(sB + 16 * n + 4 * g, b4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x = __builtin_amdgcn_mfma_f32_16x16x4f32(-a4[e] * b4[e], col[n][e], x, 0, 0, 0);
          }
          float a4[4], b4[4];
          lds4(sA + (16 * I + l16) * kGdnAS + 16 * I + 4 * g, a4);
          lds4(sB + 16 * I + 4 * g, b4);
          f32x4 y = x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y = __builtin_amdgcn_mfma_f32_16x16x4f32(-a4[e] * b4[e], x[e], y, 0, 0, 0);
          col[I] = y;
        }
      }
      __syncthreads();  // every read of A is done
#pragma unroll
      for (int J = 0; J < 3; ++J) {
        if (J != wave) continue;
#pragma unroll
        for (int I = J + 1; I < 4; ++I)
#pragma unroll
          for (int e = 0; e < 4; ++e) sA[(16 * I + 4 * g + e) * kGdnAS + 16 * J + l16] = col[I][e];
      }
      __syncthreads();
    }

    // fragments: item f holds 8 entries of one lane of one fragment
    T* fw = ws_fwd + ch * (BWD ? GdnWs<T>::bwd : GdnWs<T>::fwd);
    T* bw = BWD ? ws_bwd + ch * GdnWs<T>::bwd : nullptr;
    auto put = [&](T* hi, T* lo, const float* x) {
      if constexpr (sizeof(T) == 2) {
        bf16x8 a, b;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = (bf16)x[i];
          b[i] = (bf16)(x[i] - (float)a[i]);
        }
        *reinterpret_cast<bf16x8*>(hi) = a;
        if (lo) *reinterpret_cast<bf16x8*>(lo) = b;
      } else {
        *reinterpret_cast<float4*>(hi) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(hi + 4) = make_float4(x[4], x[5], x[6], x[7]);
      }
    };
    constexpr int PT = GdnWs<T>::kParts;
    for (int f = tid; f < 6 * 64; f += 256) {
      const int fi = f >> 6, ln = f & 63, t = fi < 2 ? fi : (fi + 2) >> 1, s = fi < 2 ? 0 : fi & 1;
      const int row = perm_row(t, ln & 15), col = 32 * s + 8 * (ln >> 4);
      float x[8];
      lds4(sA + row * kGdnAS + col, x);
      lds4(sA + row * kGdnAS + col + 4, x + 4);
      put(fw + f * 8, PT == 2 ? fw + kTriElems + f * 8 : nullptr, x);
      lds4(sP + row * kGdnAS + col, x);
      lds4(sP + row * kGdnAS + col + 4, x + 4);
      put(fw + PT * kTriElems + f * 8, BWD && PT == 2 ? fw + (PT + 1) * kTriElems + f * 8 : nullptr, x);
    }
    if constexpr (BWD) {
      for (int f = tid; f < 6 * 64; f += 256) {
        const int fi = f >> 6, ln = f & 63, t = fi < 4 ? fi >> 1 : fi - 2, s = fi < 4 ? fi & 1 : 1;
        const int row = perm_row(t, ln & 15), col = 32 * s + 8 * (ln >> 4);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = sA[(col + i) * kGdnAS + row];
        put(bw + f * 8, PT == 2 ? bw + kTriElems + f * 8 : nullptr, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = sP[(col + i) * kGdnAS + row];
        put(bw + PT * kTriElems + f * 8, PT == 2 ? bw + (PT + 1) * kTriElems + f * 8 : nullptr, x);
      }
    }
  }
}

// ------------------------------------------------------------------ scan
// One wave owns 16 columns of S for the whole sequence: K / 16 accumulator
// tiles. Every product of a chunk step takes an accumulator result of the same
// wave as its right operand, so the recurrence crosses no barrier and no LDS;
// LDS only carries the left operands (k, q, M, P, shared by the NW waves),
// fetched a chunk ahead where two buffers fit. The one barrier per chunk
// orders those buffers.
template <typename T, int K, bool BWD>
struct GdnScanLds {
  static constexpr size_t tok = TokTile<T, K>::bytes;
  static constexpr size_t tri = (BWD ? GdnWs<T>::bwd : GdnWs<T>::fwd) * sizeof(T);
  static constexpr size_t oQ = tok;
  static constexpr size_t oM = 2 * tok;       // M, P
  static constexpr size_t oS = oM + tri;      // row factors: 0..3, or for BWD 0..7
  static constexpr int scal = (BWD ? 8 : 4) * kC * (int)sizeof(float);
  static constexpr size_t buf = oS + scal;
  static constexpr int nbuf = sizeof(T) == 2 ? 2 : 1;
  static constexpr size_t total = nbuf * buf;
};

// BWD: the backward's run over the forward. S0 and Y are kept; no output, but
// (bf16) dO comes in and o' is formed in full precision, both its products
// split, for the tokens' scalars of the gate's gradient (P is strictly lower).
template <typename T, int K, int V, int NW, bool BWD>
__global__ void __launch_bounds__(NW * 64)
gdn_scan_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const float* h0, const int32_t* __restrict__ cu, const int* __restrict__ table, int N,
                int T_, int H, int HV, const float* __restrict__ ws_scal,
                const T* __restrict__ ws_frag, int write_final, T* __restrict__ o, float* ht,
                const T* __restrict__ dO, const float* __restrict__ dht, T* __restrict__ ws_S0,
                T* __restrict__ ws_Y, float* __restrict__ ws_tok, float* __restrict__ ws_end) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using Lds = GdnScanLds<T, K, BWD>;
  using TT = TokTile<T, K>;
  constexpr int NK = K / 32, RT = K / 16, BV = 16 * NW, NVB = V / BV, PT = GdnWs<T>::kParts;
  constexpr bool kOut = !BWD || GdnWs<T>::kScanGate;  // o is formed
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // 1-D grid in groups of 8 chains x NVB column blocks: the blocks of a chain
  // are 8 apart, so they run on one XCD and share its L2 for k, q, M and P
  const int grp = blockIdx.x / (8 * NVB), in = blockIdx.x % (8 * NVB);
  const int64_t chain = (int64_t)grp * 8 + in % 8;
  if (chain >= (int64_t)N * HV) return;
  const int n = cu ? table[2 + N + (int)(chain / HV)] : (int)(chain / HV);
  const int hv = (int)(chain % HV), h = hv / (HV / H);
  const int col0 = (in / 8) * BV + 16 * wave;
  int64_t bos;
  int len;
  seq_range(cu, n, T_, &bos, &len);
  const size_t st = ((size_t)n * HV + hv) * (size_t)K * V;
  if (len <= 0) {
    // empty slot: bitwise passthrough of the state (or +0.0 without one)
    if constexpr (BWD) return;
    if (!write_final || (h0 == ht && h0 != nullptr)) return;
    for (int e = lane; e < K * 16; e += 64) {
      const size_t off = st + (size_t)(e >> 4) * V + col0 + (e & 15);
      reinterpret_cast<uint32_t*>(ht)[off] = h0 ? reinterpret_cast<const uint32_t*>(h0)[off] : 0u;
    }
    return;
  }
  const int nc = (len + kC - 1) / kC;
  const int64_t c0 = cu ? table[1 + n] : (int64_t)n * ((T_ + kC - 1) / kC);

  auto fetch = [&](int c, char* b) {
    const size_t ch = (size_t)(c0 + c) * HV + hv;
    const int64_t row = ((bos + (int64_t)c * kC) * H + h) * K;
    const int L = min(kC, len - c * kC);
    dma_tok_tile<T, K, NW>(b, k + row, (int64_t)H * K, L, wave);
    dma_tok_tile<T, K, NW>(b + Lds::oQ, q + row, (int64_t)H * K, L, wave);
    dma_flat<(int)Lds::tri, NW>(b + Lds::oM, ws_frag + ch * (Lds::tri / sizeof(T)), wave);
    dma_flat<Lds::scal, NW>(b + Lds::oS, ws_scal + ch * (kGdnScal * kC), wave);
  };
  TileRaw<T> vr[4], dr[4];
  float gl;
  auto fetch_v = [&](int c) {
    const int L = min(kC, len - c * kC);
    const int64_t at = ((bos + (int64_t)c * kC) * HV + hv) * V;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      tile_ld(vr[t], v + at, (int64_t)HV * V, perm_row4(t, g), col0, L);
      if constexpr (BWD && GdnWs<T>::kScanGate)
        tile_ld(dr[t], dO + at, (int64_t)HV * V, perm_row4(t, g), col0, L);
    }
    gl = ws_scal[((size_t)(c0 + c) * HV + hv) * (kGdnScal * kC) + kSl * kC];
  };

  f32x4 S[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[r][e] = h0 ? h0[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] : 0.f;

  fetch(0, smem);
  fetch_v(0);
  for (int c = 0; c < nc; ++c) {
    const char* b = smem + (Lds::nbuf == 2 ? (c & 1) * Lds::buf : 0);
    lds_dma_wait();
    __syncthreads();  // this chunk's operands are in LDS; the other buffer is no longer read
    if (Lds::nbuf == 2 && c + 1 < nc) fetch(c + 1, smem + ((c + 1) & 1) * Lds::buf);
    const float* sf = reinterpret_cast<const float*>(b + Lds::oS);
    const T* sM = reinterpret_cast<const T*>(b + Lds::oM);
    const T* sP = sM + PT * kTriElems;
    const size_t ch = (size_t)(c0 + c) * HV + hv;
    const int L = min(kC, len - c * kC);
    f32x4 x[4], dot[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = tile_get(vr[t]);
      if constexpr (BWD && GdnWs<T>::kScanGate) dot[t] = tile_get(dr[t]);
    }
    const float el = gl;
    if (c + 1 < nc) fetch_v(c + 1);

    if constexpr (BWD) {
#pragma unroll
      for (int r = 0; r < RT; ++r) tile_st(ws_S0 + ch * K * V, V, perm_row4(r, g), col0, K, S[r]);
    }
    // k S0 (split: it feeds the state) and q S0
    f32x4 ks[4], qs[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) ks[t] = qs[t] = zero4();
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      Op8s<T> sb;
      make_op(sb, S[2 * s], S[2 * s + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op8<T> a;
        TT::rows(a, b, t, s);
        ks[t] = mma8s(a, sb, ks[t]);
        if constexpr (kOut) {
          TT::rows(a, b + Lds::oQ, t, s);
          qs[t] = BWD ? mma8s(a, sb, qs[t]) : mma8h(a, sb, qs[t]);
        }
      }
    }
    // R = v - e^G k S0, then Y = R - M (b R)
    f32x4 bb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float f[4], w[4];
      lds4(sf + kSk * kC + perm_row4(t, g), f);
      lds4(sf + kSb * kC + perm_row4(t, g), w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ks[t][e] *= f[e];
        x[t][e] -= ks[t][e];
        bb[t][e] = w[e];
      }
    }
    {
      Op8s<T> rb[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4 a0, a1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a0[e] = -bb[2 * s][e] * x[2 * s][e];
          a1[e] = -bb[2 * s + 1][e] * x[2 * s + 1][e];
        }
        make_op(rb[s], a0, a1);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4 m = zero4();
#pragma unroll
        for (int s = 0; s <= (t >> 1); ++s) {
          Op8<T> a;
          if constexpr (sizeof(T) == 2) {
            ld_op(a, sM + kTriElems + frag_low(t, s) * kFragElems + lane * 8);
            m = mma8h(a, rb[s], m);
          }
          ld_op(a, sM + frag_low(t, s) * kFragElems + lane * 8);
          m = mma8s(a, rb[s], m);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[t][e] += m[e];
          ks[t][e] -= m[e];  // v - Y, without v
        }
      }
    }
    if constexpr (BWD) {
#pragma unroll
      for (int t = 0; t < 4; ++t) tile_st(ws_Y + ch * kC * V, V, perm_row4(t, g), col0, kC, x[t]);
    }
    // Delta = b Y; O = e^G q~ S0 + P Delta
    Op8s<T> eb[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 d[2], ed[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * s + i;
        float f[4];
        lds4(sf + kSe * kC + perm_row4(t, g), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[i][e] = bb[t][e] * x[t][e];
          ed[i][e] = f[e] * d[i][e];
        }
      }
      make_op(eb[s], ed[0], ed[1]);
      if constexpr (kOut) {
        Op8s<T> db;  // split: with S0 and P rounded as well, hi alone left o at 1.65x its rounding error
        make_op(db, d[0], d[1]);
        if (s == 0) {
  #pragma unroll
          for (int t = 0; t < 4; ++t) {
            float f[4];
            lds4(sf + kSq * kC + perm_row4(t, g), f);
  #pragma unroll
            for (int e = 0; e < 4; ++e) qs[t][e] *= f[e];
          }
        }
  #pragma unroll
        for (int t = 2 * s; t < 4; ++t) {
          Op8<T> a;
          if constexpr (BWD && PT == 2) {
            ld_op(a, sP + kTriElems + frag_low(t, s) * kFragElems + lane * 8);
            qs[t] = mma8h(a, db, qs[t]);
          }
          ld_op(a, sP + frag_low(t, s) * kFragElems + lane * 8);
          qs[t] = mma8s(a, db, qs[t]);
        }
      }
    }
    // S1 = e^{G_last} S0 + K^T (e^{G_last - G} Delta)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] *= el;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Op8<T> a;
        TT::cols(a, b, r, s);
        S[r] = mma8s(a, eb[s], S[r]);
      }
    }
    if constexpr (BWD && GdnWs<T>::kScanGate) {
      float* tk = ws_tok + (ch * (V / 16) + (col0 >> 4)) * kC;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float f[4], y[4];
        lds4(sf + kSp * kC + perm_row4(t, g), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = row16_sum(dot[t][e] * (qs[t][e] - f[e] * bb[t][e] * ks[t][e]));
        if (l16 == 0) *reinterpret_cast<float4*>(tk + perm_row4(t, g)) = make_float4(y[0], y[1], y[2], y[3]);
      }
    } else if constexpr (!BWD) {
      T* ob = o + ((bos + (int64_t)c * kC) * HV + hv) * V;
#pragma unroll
      for (int t = 0; t < 4; ++t) tile_st(ob, (int64_t)HV * V, perm_row4(t, g), col0, L, qs[t]);
    }
    if (Lds::nbuf == 1 && c + 1 < nc) {
      __syncthreads();  // every wave is done with the only buffer
      fetch(c + 1, smem);
    }
  }
  if constexpr (BWD) {
    if (GdnWs<T>::kScanGate && dht) {
      float y = 0.f;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y = fmaf(S[r][e], dht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16], y);
      y = row16_sum(y);
      y += __shfl_xor(y, 16);
      y += __shfl_xor(y, 32);
      if (lane == 0) ws_end[((size_t)n * HV + hv) * (V / 16) + (col0 >> 4)] = y;
    }
  } else if (write_final) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] = S[r][e];
  }
}

template <typename F>
static hipError_t set_lds(F* f, size_t bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                             (int)bytes);
}

struct GdnCall {
  const void *q, *k, *v, *beta;
  GdnGate gate;
  int l2;
  const float* h0;
  const int32_t* cu;
  void* o;
  float* ht;          // null: no final state
  const void* dO;     // backward's run only
  const float* dht;
};

template <typename T, int K, int V, int NW, bool BWD>
static hipError_t scan_t(const kda_dims& d, const GdnCall& c, const GdnLayout<T>& w, hipStream_t s) {
  constexpr size_t lds = GdnScanLds<T, K, BWD>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  hipError_t e = set_lds(&gdn_scan_kernel<T, K, V, NW, BWD>, lds);
  if (e != hipSuccess) return e;
  const int64_t chains = (int64_t)d.N * d.HV;
  hipLaunchKernelGGL((gdn_scan_kernel<T, K, V, NW, BWD>), dim3(scan_grid(chains, V, 16 * NW)), dim3(64 * NW),
                     lds, s, (const T*)c.q, (const T*)c.k, (const T*)c.v, c.h0, c.cu, w.table, d.N, d.T, d.H,
                     d.HV, w.scal, w.frag, c.ht != nullptr, (T*)c.o, c.ht, (const T*)c.dO, c.dht, w.S0, w.Y,
                     w.tok, w.end);
  return hipGetLastError();
}

template <typename T, int K, int V, bool BWD>
static hipError_t gdn_fwd_kv(const kda_dims& d, const GdnCall& c, void* ws, hipStream_t s) {
  const bool varlen = c.cu != nullptr;
  const int64_t mc = max_chunks(d, varlen);
  const GdnLayout<T> w(d, varlen, ws, BWD);
  if (varlen) {
    hipError_t e = launch_chunk_table(c.cu, d.N, w.table, (int)mc, s);
    if (e != hipSuccess) return e;
  }
  if (mc > 0) {
    // all value heads of a q/k head in one workgroup (q k^T and k k^T formed
    // once) as long as that leaves two workgroups per compute unit
    const int grp = d.HV / d.H;
    const int hpw = mc * d.H >= 2 * (int64_t)kda_host::device_cus() ? grp : 1;
    hipLaunchKernelGGL((gdn_intra_kernel<T, K, BWD>), dim3((unsigned)(mc * (d.HV / hpw))), dim3(256), 0, s,
                       (const T*)c.q, (const T*)c.k, c.gate, (const T*)c.beta, c.cu, w.table, d.N, d.T, d.H,
                       d.HV, hpw, c.l2, 1.0f / sqrtf((float)K), w.scal, w.frag, w.fragT);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // 64 columns per workgroup while that fills the device, else 32
  const bool wide = (int64_t)d.N * d.HV * (V / 64) >= kda_host::device_cus();
  return wide ? scan_t<T, K, V, 4, BWD>(d, c, w, s) : scan_t<T, K, V, 2, BWD>(d, c, w, s);
}

template <typename T, bool BWD>
static hipError_t gdn_fwd_t(const kda_dims& d, const GdnCall& c, void* ws, hipStream_t s) {
#define KDA_GDN_FWD(K_, V_) \
  if (d.K == K_ && d.V == V_) return gdn_fwd_kv<T, K_, V_, BWD>(d, c, ws, s);
  KDA_GDN_FWD(64, 64)
  KDA_GDN_FWD(64, 128)
  KDA_GDN_FWD(128, 64)
  KDA_GDN_FWD(128, 128)
#undef KDA_GDN_FWD
  return hipErrorInvalidValue;
}

}  // namespace kda

namespace kda_host {

size_t gdn_workspace_bytes(const kda_dims& d, kda_dtype dt, int bwd) {
  size_t b = 0;
  for (int varlen = 0; varlen < 2; ++varlen)
    b = std::max(b, dt == KDA_BF16 ? kda::GdnLayout<kda::bf16>(d, varlen != 0, nullptr, bwd != 0).bytes
                                   : kda::GdnLayout<float>(d, varlen != 0, nullptr, bwd != 0).bytes);
  return b;
}

hipError_t launch_gdn_fwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                          const kda::GdnGate& gate, int l2, const void* beta, const float* h0,
                          const int32_t* cu, int write_final, void* o, float* ht, void* ws, hipStream_t s) {
  const kda::GdnCall c{q, k, v, beta, gate, l2, h0, cu, o, write_final ? ht : nullptr, nullptr, nullptr};
  return dt == KDA_BF16 ? kda::gdn_fwd_t<kda::bf16, false>(d, c, ws, s) : kda::gdn_fwd_t<float, false>(d, c, ws, s);
}

hipError_t launch_gdn_refwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                            const kda::GdnGate& gate, int l2, const void* beta, const float* h0,
                            const int32_t* cu, const void* dO, const float* dht, void* ws, hipStream_t s) {
  const kda::GdnCall c{q, k, v, beta, gate, l2, h0, cu, nullptr, nullptr, dO, dht};
  return dt == KDA_BF16 ? kda::gdn_fwd_t<kda::bf16, true>(d, c, ws, s) : kda::gdn_fwd_t<float, true>(d, c, ws, s);
}

}  // namespace kda_host
