// Chunked gated delta rule with a scalar gate: intra-chunk kernel and forward
// scan. Formulas, layouts and the rounding rule are in kda_gdn.h.
//
//   gdn_intra_kernel  one workgroup per (chunk, group of value heads of a q/k
//                     head): q k^T and k k^T once on the matrix cores for the
//                     whole group, then per value head the gate, the FP32
//                     solve for M, and M, P and the row factors written out.
//   gdn_scan_kernel   16 columns of one (sequence, value head) state per wave,
//                     walking the chunks in order; S stays in the wave's
//                     accumulators (gdn_scan32_kernel for FP32 inputs).
#include "kda_gdn.h"

namespace kda {

// ------------------------------------------------------------------ intra
constexpr int kGdnAS = kC + 4;  // row stride of the FP32 A and P in LDS

// The kernel waits more than it computes (65% of its wave cycles when every wave
// fetched its own column tiles): all of q, k, gate and beta is fetched once and
// up front, a wave's rows of k reach the others through LDS, and the registers
// are held to four workgroups a CU (three with BWD): 256 chunks x 16 heads, K
// = 128, 93 -> 66 us (BWD 130 -> 91 us), 155 MB at 2.3 TB/s.
template <typename T, int K, bool BWD>
__global__ void __launch_bounds__(256, BWD ? 3 : 4)
gdn_intra_kernel(const T* __restrict__ q, const T* __restrict__ k, GdnGate gate,
                 const T* __restrict__ beta, const int32_t* __restrict__ cu,
                 const int* __restrict__ table, int N, int T_, int H, int HV, int hpw, int l2,
                 float scale, float* __restrict__ ws_scal, T* __restrict__ ws_fwd,
                 T* __restrict__ ws_bwd) {
  constexpr int NK = K / 32;
  // A and P of a value head; before them, k's rows as operands for every wave
  constexpr int kAP = 2 * kC * kGdnAS, kKf = 4 * NK * kFragElems * (int)sizeof(T) / 4;
  __shared__ __attribute__((aligned(16))) float s_big[kAP > kKf ? kAP : kKf];
  float* sA = s_big;
  float* sP = s_big + kC * kGdnAS;
  T* sKf = reinterpret_cast<T*>(s_big);
  __shared__ double sG[kC];
  __shared__ __attribute__((aligned(16))) float sB[kC], sRq[kC], sRk[kC];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nh = HV / hpw;
  const int j = blockIdx.x / nh, hv0 = (blockIdx.x % nh) * hpw, h = hv0 / (HV / H);
  const ChunkGeo geo = chunk_geo(j, cu, table, N, T_);
  if (!geo.ok) return;
  const int L = geo.L;

  // wave 0 (which has one column tile, wave 3 has four) does the gate, lane =
  // token; a head's inputs are fetched ahead
  float gx = 0.f, gb = 0.f, ga = 0.f, gd = 0.f;
  auto fetch_gate = [&](int hv) __attribute__((always_inline)) {
    const int64_t at = (geo.t0 + min(lane, L - 1)) * HV + hv;
    gx = ld_any(gate.x, at, gate.bf);
    gb = to_f32(beta[at]);
    if (gate.A_log) ga = ld_any(gate.A_log, hv, gate.bf);
    if (gate.dt_bias) gd = ld_any(gate.dt_bias, hv, gate.bf);
  };
  if (wave == 0) fetch_gate(hv0);

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
#pragma unroll
  for (int s = 0; s < NK; ++s) {
    T* d = sKf + ((wave * NK + s) * 64 + lane) * 8;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<bf16x8*>(d) = kf[s].v;
    } else {
      *reinterpret_cast<float4*>(d) = make_float4(kf[s].v[0], kf[s].v[1], kf[s].v[2], kf[s].v[3]);
      *reinterpret_cast<float4*>(d + 4) = make_float4(kf[s].v[4], kf[s].v[5], kf[s].v[6], kf[s].v[7]);
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
  __syncthreads();
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int J = 0; J < 4; ++J) {
    kk[J] = qk[J] = zero4();
    if (J > wave) continue;
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      Op8<T> kj;
      ld_op(kj, sKf + ((J * NK + s) * 64 + lane) * 8);
      kk[J] = mma8(kf[s], kj, kk[J]);
      qk[J] = mma8(qf[s], kj, qk[J]);
    }
  }

  for (int hh = 0; hh < hpw; ++hh) {
    const int hv = hv0 + hh;
    const size_t ch = (size_t)j * HV + hv;
    if (hh > 0) __syncthreads();  // the previous head's reads done
    // gate sums in double: differences G_i - G_j stay exact to FP32 for any gate
    if (wave == 0) {
      const bool ok = lane < L;
      float gn = gx;
      if (gate.raw) gn = -(gate.A_log ? expf(ga) : 1.f) * softplus_f32(gate.dt_bias ? gx + gd : gx);
      if (!ok) gn = 0.f;
      const float b = ok ? gb : 0.f;
      if (hh + 1 < hpw) fetch_gate(hv + 1);
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
      sc[kSk * kC + lane] = ok ? eg * rk : 0.f;
      sc[kSq * kC + lane] = ok ? eg * rq * scale : 0.f;
      const float ee = ok ? ex2((float)(Gl - G)) * rk : 0.f;
      sc[kSeb * kC + lane] = ee * b;
      sc[kSb * kC + lane] = b;
      if constexpr (BWD) {
        if (!ok) sc[kSp * kC + lane] = sc[kSpd * kC + lane] = 0.f;
        sc[kSe * kC + lane] = ee;
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
            ws_scal[ch * (kGdnScal * kC) + kSpd * kC + i] = p;
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
// bf16. Two waves per 16 columns. The state wave keeps S (K / 16 accumulator
// tiles) and walks the recurrence: every product of a chunk takes an
// accumulator result of the wave itself as its right operand, so the
// recurrence crosses no LDS. The output wave follows one chunk behind: it takes
// the chunk's start state (already split for the products) and Y through LDS
// and forms O, and it issues all transfers of left operands (k, q, M, P) into
// LDS a chunk ahead. With one wave per 16 columns doing both, a chunk step was
// about 1000 instructions of one wave with nothing else on its SIMD (2.5 us of
// 3.9 us per chunk at 64 chains); the two halves of the work now run on two.
// Two barriers per chunk: at its top (operands in LDS) and after the output
// wave has taken the previous chunk's S and Y. What bounds it now is the step
// of the recurrence, 2.1 us a chunk with 32 columns per workgroup (64 chains
// of 4096 tokens, K = V = 128: 135 us) and 3.4 us with 64, where state and
// output waves share their SIMDs' issue slots (608 chains, 32768 tokens: 431 us).
//
// BWD: the backward's run over the forward. S0 and Y are kept instead of O, and
// dO comes in: o' is formed in full precision (S0 and P split as well; P is
// strictly lower) for the tokens' scalars of the gate's gradient. Two output waves
// per pair take two token tiles each, and a fourth wave stores S0 and Y: 64
// chains of 4096 tokens 207 us (with one output wave 45 us more, and 60 where it
// stores too).
template <int K, int NP, bool BWD>
struct GdnScanLds {
  static constexpr int NK = K / 32, PT = BWD ? 2 : 1;
  static constexpr uint32_t tok = TokTile<bf16, K>::bytes, tri = kTriElems * sizeof(bf16);
  static constexpr int scal = 4 * kC * (int)sizeof(float);  // state: slots 0..3, output: 3..6
  // state wave's buffer: k, M (hi, lo), row factors; output wave's: q, P, row factors
  static constexpr uint32_t sM = tok, sF = sM + 2 * tri, sbuf = sF + scal;
  static constexpr uint32_t oP = tok, oF = oP + PT * tri, obuf = oF + scal;
  static constexpr uint32_t at_o = 2 * sbuf, at_x = at_o + 2 * obuf;
  // exchange of a pair: S0 (BWD: hi, lo), Y, BWD: v - Y
  static constexpr uint32_t xS = PT * NK * 1024, xY = 4 * 1024, xbuf = xS + (BWD ? 2 : 1) * xY;
  static constexpr uint32_t total = at_x + NP * xbuf;
};

template <int K, int V, int NP, bool BWD>
__global__ void __launch_bounds__(NP * (BWD ? 256 : 128), 2)  // 2: 256 registers, none of them accumulation-only
gdn_scan_kernel(const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
                const float* h0, const int32_t* __restrict__ cu, const int* __restrict__ table, int N,
                int T_, int H, int HV, const float* __restrict__ ws_scal, const bf16* __restrict__ ws_frag,
                int write_final, bf16* __restrict__ o, float* ht, const bf16* __restrict__ dO,
                const float* __restrict__ dht, bf16* __restrict__ ws_S0, bf16* __restrict__ ws_Y,
                float* __restrict__ ws_tok, float* __restrict__ ws_end, float* __restrict__ ws_anc,
                bf16* __restrict__ ws_Yl) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using L_ = GdnScanLds<K, NP, BWD>;
  using TT = TokTile<bf16, K>;
  constexpr int NK = K / 32, RT = K / 16, BV = 16 * NP, NVB = V / BV;
  constexpr size_t kFrag = BWD ? GdnWs<bf16>::bwd : GdnWs<bf16>::fwd;
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = wave % NP, role = wave / NP;  // 0 state, 1 output (BWD: and 3), 2 store
  const bool state_wave = role == 0;
  const GdnChain ch = gdn_chain(NVB, cu, table, N, T_, H, HV);
  if (!ch.ok) return;
  const int col0 = ch.vb * BV + 16 * pair, hv = ch.hv, len = ch.len;
  const size_t st = ((size_t)ch.n * HV + hv) * (size_t)K * V;
  if (len <= 0) {
    if (!BWD && state_wave && write_final && !(h0 == ht && h0 != nullptr)) gdn_pass(h0, ht, st, K, V, col0);
    return;
  }
  const int nc = (len + kC - 1) / kC;
  auto chunk = [&](int c) { return (size_t)(ch.c0 + c) * HV + hv; };
  auto tokens = [&](int c) { return min(kC, len - c * kC); };
  auto vrow = [&](int c) { return ((ch.bos + (int64_t)c * kC) * HV + hv) * V; };
  char* xch = smem + L_::at_x + pair * L_::xbuf;

  if (state_wave) {
    f32x4 S[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[r][e] = h0 ? h0[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] : 0.f;
    TileRaw<bf16> vr[4];
    auto fetch_v = [&](int c) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) tile_ld(vr[t], v + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
    };
    fetch_v(0);
    __syncthreads();  // the first chunk's operands
    __builtin_amdgcn_s_setprio(2);  // ahead of an output wave on the same SIMD
    for (int it = 0; it < nc; ++it) {
      __syncthreads();
      if (BWD && it > 0 && it % kGdnAnchor == 0) {
        float4* a = reinterpret_cast<float4*>(ws_anc) +
                    ((gdn_anchor(ch.c0, it) * HV + hv) * (V / 16) + (col0 >> 4)) * RT * 64 + lane;
#pragma unroll
        for (int r = 0; r < RT; ++r) a[r * 64] = make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
      }
      const char* b = smem + (it & 1) * L_::sbuf;
      const bf16* sM = reinterpret_cast<const bf16*>(b + L_::sM);
      const float* sf = reinterpret_cast<const float*>(b + L_::sF);
      // Left operands are read from LDS a group ahead of the products that take
      // them (`stage` keeps the compiler from moving the reads back to their use).
      Op8<bf16> ka[NK][4];
      auto read_k = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) TT::rows(ka[s][t], b, t, s);
      };
      read_k(0);
      read_k(1);
      f32x4 x[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) x[t] = tile_get(vr[t]);
      // (from LDS: a scalar load in flight would turn every wait on LDS into a full one)
      const float el = sf[kSl * kC + lane];
      if (it + 1 < nc) fetch_v(it + 1);
      // k S0, both parts of S0: it feeds the state
      Op8s<bf16> sb[NK];
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        make_op(sb[s], S[2 * s], S[2 * s + 1]);
        S[2 * s] *= el;  // S0 is not needed again
        S[2 * s + 1] *= el;
      }
      f32x4 ks[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) ks[t] = zero4();
      Op8<bf16> ml[2][6];
      auto read_m = [&](int f) __attribute__((always_inline)) {
        ld_op(ml[0][f], sM + f * kFragElems + lane * 8);
        ld_op(ml[1][f], sM + kTriElems + f * kFragElems + lane * 8);
      };
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        stage();
        if (s + 2 < NK) {
          read_k(s + 2);
        } else {
          read_m(2 * (s + 2 - NK));
          read_m(2 * (s + 2 - NK) + 1);
        }
        stage();
        mma_rows(ka[s], sb[s], ks);
      }
      stage();
      read_m(4);
      read_m(5);
      __syncthreads();  // the output wave has taken the previous chunk's S0 and Y
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        *reinterpret_cast<bf16x8*>(xch + (s * 64 + lane) * 16) = sb[s].hi;
        if constexpr (BWD) *reinterpret_cast<bf16x8*>(xch + ((NK + s) * 64 + lane) * 16) = sb[s].lo;
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
          if constexpr (BWD) {
            ks[t][e] *= f[e];
            x[t][e] -= ks[t][e];
          } else {
            x[t][e] = fmaf(-f[e], ks[t][e], x[t][e]);
          }
          bb[t][e] = w[e];
        }
      }
      Op8s<bf16> rb[2];
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
      if constexpr (BWD) {
        f32x4 m[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) m[t] = zero4();
        mma_tri<2>(ml, rb, m);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[t][e] += m[t][e];
            ks[t][e] -= m[t][e];  // v - Y, without v
          }
          *reinterpret_cast<f32x4*>(xch + L_::xS + L_::xY + (t * 64 + lane) * 16) = ks[t];
        }
      } else {
        mma_tri<2>(ml, rb, x);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(xch + L_::xS + (t * 64 + lane) * 16) = x[t];
      // S1 = e^{G_last} S0 + K^T (e^{G_last - G} b Y)
      Op8<bf16> kc[RT][2];
      auto read_kc = [&](int r) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s) TT::cols(kc[r][s], b, r, s);
      };
      read_kc(0);
      read_kc(1);
      Op8s<bf16> eb[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4 ed[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 2 * s + i;
          float f[4];
          lds4(sf + kSeb * kC + perm_row4(t, g), f);
#pragma unroll
          for (int e = 0; e < 4; ++e) ed[i][e] = f[e] * x[t][e];
        }
        make_op(eb[s], ed[0], ed[1]);
      }
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        stage();
        if (r + 2 < RT) {
          read_kc(r + 2);
          read_kc(r + 3);
        }
        stage();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          S[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[r][s].v, eb[s].lo, S[r], 0, 0, 0);
          S[r + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[r + 1][s].v, eb[s].lo, S[r + 1], 0, 0, 0);
          S[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[r][s].v, eb[s].hi, S[r], 0, 0, 0);
          S[r + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[r + 1][s].v, eb[s].hi, S[r + 1], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();  // the output wave's last chunk
    __syncthreads();
    if constexpr (BWD) {
      if (dht) {
        float y = 0.f;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y = fmaf(S[r][e], dht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16], y);
        y = row16_sum(y);
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        if (lane == 0) ws_end[((size_t)ch.n * HV + hv) * (V / 16) + (col0 >> 4)] = y;
      }
    } else if (write_final) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] = S[r][e];
    }
    return;
  }

  if constexpr (BWD) {
    if (role == 2) {  // S0 (its high part) and Y (both parts) of the chunk behind
      __syncthreads();
      for (int it = 0; it <= nc; ++it) {
        __syncthreads();
        uint4 s0[NK];
        f32x4 x[4];
        if (it > 0) {
#pragma unroll
          for (int s = 0; s < NK; ++s) s0[s] = *reinterpret_cast<const uint4*>(xch + (s * 64 + lane) * 16);
#pragma unroll
          for (int t = 0; t < 4; ++t) x[t] = *reinterpret_cast<const f32x4*>(xch + L_::xS + (t * 64 + lane) * 16);
        }
        __syncthreads();
        if (it == 0) continue;
#pragma unroll
        for (int r = 0; r < RT; ++r)
          op_st(ws_S0 + chunk(it - 1) * K * V, r, col0 >> 4, V / 32,
                (r & 1) ? make_uint2(s0[r >> 1].z, s0[r >> 1].w) : make_uint2(s0[r >> 1].x, s0[r >> 1].y));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint2 y = pack4(x[t]);
          op_st(ws_Y + chunk(it - 1) * kC * V, t, col0 >> 4, V / 32, y);
          reinterpret_cast<uint2*>(ws_Yl)[((chunk(it - 1) * (V / 16) + (col0 >> 4)) * 4 + t) * 64 + lane] =
              make_uint2(pack2_rest(x[t][0], x[t][1], y.x), pack2_rest(x[t][2], x[t][3], y.y));
        }
      }
      return;
    }
  }

  // ---- output wave: all four token tiles, BWD tiles 0, 1 or 2, 3
  constexpr int OT = BWD ? 2 : 4, NO = BWD ? 2 * NP : NP;
  const int t0 = BWD && role == 3 ? 2 : 0, ow = BWD && role == 3 ? NP + pair : pair;
  const uint32_t lds = lds_addr(smem);
  const TokDma<bf16, K, NO> tok((uint32_t)(H * K * sizeof(bf16)), ow);
  auto fetch_s = [&](int c) __attribute__((always_inline)) {  // what the state waves read
    const uint32_t b = lds + (c & 1) * L_::sbuf;
    tok.go(b, k + ((ch.bos + (int64_t)c * kC) * H + ch.h) * K, tokens(c));
    dma_flat<2 * L_::tri, NO>(b + L_::sM, ws_frag + chunk(c) * kFrag, ow);
    dma_flat<L_::scal, NO>(b + L_::sF, ws_scal + chunk(c) * (kGdnScal * kC), ow);
  };
  auto fetch_o = [&](int c) __attribute__((always_inline)) {  // what the output waves read
    const uint32_t b = lds + L_::at_o + (c & 1) * L_::obuf;
    tok.go(b, q + ((ch.bos + (int64_t)c * kC) * H + ch.h) * K, tokens(c));
    dma_flat<L_::PT * L_::tri, NO>(b + L_::oP, ws_frag + chunk(c) * kFrag + 2 * kTriElems, ow);
    dma_flat<L_::scal, NO>(b + L_::oF, ws_scal + chunk(c) * (kGdnScal * kC) + kSb * kC, ow);
  };
  TileRaw<bf16> dr[OT];
  fetch_s(0);
  lds_dma_wait();
  __syncthreads();
  for (int it = 0; it <= nc; ++it) {
    // behind the previous round's transfers: the OT stores of chunk it - 2, a full one
    if (it >= 2) lds_dma_wait_but<OT>();
    else lds_dma_wait();
    __syncthreads();
    if constexpr (BWD) {
#pragma unroll
      for (int t = 0; t < OT; ++t)
        if (it > 0) settle(dr[t].r);
    }
    if (it + 1 < nc) fetch_s(it + 1);
    if (it < nc) fetch_o(it);
    const int c = it - 1;
    Op8s<bf16> sb[NK];
    f32x4 x[4], pred[OT], dot[OT];
    if (it > 0) {
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        sb[s].hi = *reinterpret_cast<const bf16x8*>(xch + (s * 64 + lane) * 16);
        if constexpr (BWD) sb[s].lo = *reinterpret_cast<const bf16x8*>(xch + ((NK + s) * 64 + lane) * 16);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        x[t] = *reinterpret_cast<const f32x4*>(xch + L_::xS + (t * 64 + lane) * 16);
      }
      if constexpr (BWD) {
#pragma unroll
        for (int t = 0; t < OT; ++t)
          pred[t] = *reinterpret_cast<const f32x4*>(xch + L_::xS + L_::xY + ((t0 + t) * 64 + lane) * 16);
      }
    }
    __syncthreads();
    if (it == 0) {
      if constexpr (BWD) {
#pragma unroll
        for (int t = 0; t < OT; ++t) tile_ld(dr[t], dO + vrow(0), HV * V, perm_row4(t0 + t, g), col0, tokens(0));
      }
      continue;
    }
    const char* b = smem + L_::at_o + (c & 1) * L_::obuf;
    const bf16* sP = reinterpret_cast<const bf16*>(b + L_::oP);
    const float* sf = reinterpret_cast<const float*>(b + L_::oF);  // from slot kSb on
    if constexpr (BWD) {
#pragma unroll
      for (int t = 0; t < OT; ++t) dot[t] = tile_get(dr[t]);
      if (it < nc) {
#pragma unroll
        for (int t = 0; t < OT; ++t) tile_ld(dr[t], dO + vrow(it), HV * V, perm_row4(t0 + t, g), col0, tokens(it));
      }
    }
    // O = e^G q~ S0 + P Delta, Delta = b Y
    Op8<bf16> qa[2][OT], pf[L_::PT][BWD ? 4 : 6];
    f32x4 qs[OT];
#pragma unroll
    for (int t = 0; t < OT; ++t) qs[t] = zero4();
    auto read_q = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < OT; ++t) TT::rows(qa[s & 1][t], b, t0 + t, s);
    };
    read_q(0);
    float bb[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) lds4(sf + perm_row4(t, g), bb[t]);
    Op8s<bf16> db[2];  // split: with S0 and P rounded as well, hi alone left o at 1.65x its rounding error
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 d[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = bb[2 * s + i][e] * x[2 * s + i][e];
      make_op(db[s], d[0], d[1]);
    }
    // BWD: P's fragments of the wave's tiles, [s][tile]: tiles 0, 1 have none at s = 1, and read
    // others that the branch below leaves out
    const auto frag = [&](int f) __attribute__((always_inline)) {
      return BWD ? (t0 ? 2 + 2 * (f & 1) + (f >> 1) : f & 1) : f;
    };
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      stage();
      if (s + 1 < NK) {
        read_q(s + 1);
      } else {
#pragma unroll
        for (int pt = 0; pt < L_::PT; ++pt)
#pragma unroll
          for (int f = 0; f < (BWD ? 4 : 6); ++f)
            ld_op(pf[pt][f], sP + pt * kTriElems + frag(f) * kFragElems + lane * 8);
      }
      stage();
      if constexpr (BWD) {
#pragma unroll
        for (int t = 0; t < OT; ++t) qs[t] = mma8s(qa[s & 1][t], sb[s], qs[t]);
      } else {
#pragma unroll
        for (int t = 0; t < OT; ++t) qs[t] = mma8h(qa[s & 1][t], sb[s], qs[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < OT; ++t) {
      float f[4];
      lds4(sf + (kSq - kSb) * kC + perm_row4(t0 + t, g), f);
#pragma unroll
      for (int e = 0; e < 4; ++e) qs[t][e] *= f[e];
    }
    if constexpr (BWD) {
      auto mma_p = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < OT; ++t)
          qs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[0][2 * s + t].v, db[s].lo, qs[t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < OT; ++t)
          qs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[1][2 * s + t].v, db[s].hi, qs[t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < OT; ++t)
          qs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[0][2 * s + t].v, db[s].hi, qs[t], 0, 0, 0);
      };
      if (t0) mma_p(1);
      mma_p(0);
      float* tk = ws_tok + (chunk(c) * (V / 16) + (col0 >> 4)) * kC;
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        const int row4 = perm_row4(t0 + t, g);
        float f[4], y[4], w[4];
        lds4(sf + (kSp - kSb) * kC + row4, f);
        lds4(sf + row4, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = row16_sum(dot[t][e] * (qs[t][e] - f[e] * w[e] * pred[t][e]));
        if (l16 == 0) *reinterpret_cast<float4*>(tk + row4) = make_float4(y[0], y[1], y[2], y[3]);
      }
    } else {
      mma_tri<L_::PT>(pf, db, qs);
#pragma unroll
      for (int t = 0; t < OT; ++t) tile_st(o + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c), qs[t]);
    }
  }
}

// FP32. The same step by one wave per 16 columns, on the FP32 matrix cores;
// operands need no splitting. One operand buffer (two do not fit). BWD keeps
// S0 and Y and forms no output.
template <int K, bool BWD>
struct GdnScan32Lds {
  static constexpr uint32_t tok = TokTile<float, K>::bytes, tri = kTriElems * sizeof(float);
  static constexpr uint32_t oQ = tok, oM = 2 * tok, oS = oM + 2 * tri, total = oS + 8 * kC * sizeof(float);
};

template <int K, int V, int NW, bool BWD>
__global__ void __launch_bounds__(NW * 64)
gdn_scan32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                  const float* h0, const int32_t* __restrict__ cu, const int* __restrict__ table, int N, int T_,
                  int H, int HV, const float* __restrict__ ws_scal, const float* __restrict__ ws_frag,
                  int write_final, float* __restrict__ o, float* ht, float* __restrict__ ws_S0,
                  float* __restrict__ ws_Y) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using L_ = GdnScan32Lds<K, BWD>;
  using TT = TokTile<float, K>;
  constexpr int NK = K / 32, RT = K / 16, BV = 16 * NW, NVB = V / BV;
  constexpr size_t kFrag = GdnWs<float>::fwd;
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GdnChain ch = gdn_chain(NVB, cu, table, N, T_, H, HV);
  if (!ch.ok) return;
  const int col0 = ch.vb * BV + 16 * wave, hv = ch.hv, len = ch.len;
  const size_t st = ((size_t)ch.n * HV + hv) * (size_t)K * V;
  if (len <= 0) {
    if (!BWD && write_final && !(h0 == ht && h0 != nullptr)) gdn_pass(h0, ht, st, K, V, col0);
    return;
  }
  const int nc = (len + kC - 1) / kC;
  const uint32_t lds = lds_addr(smem);
  const TokDma<float, K, NW> tok((uint32_t)(H * K * sizeof(float)), wave);
  auto fetch = [&](int c) {
    const size_t cc = (size_t)(ch.c0 + c) * HV + hv;
    const int64_t row = ((ch.bos + (int64_t)c * kC) * H + ch.h) * K;
    const int L = min(kC, len - c * kC);
    tok.go(lds, k + row, L);
    if constexpr (!BWD) tok.go(lds + L_::oQ, q + row, L);
    dma_flat<2 * L_::tri, NW>(lds + L_::oM, ws_frag + cc * kFrag, wave);
    dma_flat<8 * kC * 4, NW>(lds + L_::oS, ws_scal + cc * (kGdnScal * kC), wave);
  };
  f32x4 S[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[r][e] = h0 ? h0[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] : 0.f;
  const float* sf = reinterpret_cast<const float*>(smem + L_::oS);
  const float* sM = reinterpret_cast<const float*>(smem + L_::oM);
  const float* sP = sM + kTriElems;
  for (int c = 0; c < nc; ++c) {
    if (c > 0) __syncthreads();  // every wave is done with the buffer
    fetch(c);
    const size_t cc = (size_t)(ch.c0 + c) * HV + hv;
    const int L = min(kC, len - c * kC);
    const int64_t at = ((ch.bos + (int64_t)c * kC) * HV + hv) * V;
    f32x4 x[4], ks[4], qs[4], bb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      TileRaw<float> r;
      tile_ld(r, v + at, HV * V, perm_row4(t, g), col0, L);
      x[t] = r.r;
      ks[t] = qs[t] = zero4();
    }
    const float el = ws_scal[cc * (kGdnScal * kC) + kSl * kC];
    if constexpr (BWD) {
#pragma unroll
      for (int r = 0; r < RT; ++r) op_st(ws_S0 + cc * K * V, r, col0 >> 4, V / 32, S[r]);
    }
    lds_dma_wait();
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      Op8s<float> sb;
      make_op(sb, S[2 * s], S[2 * s + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op8<float> a;
        TT::rows(a, smem, t, s);
        ks[t] = mma8s(a, sb, ks[t]);
        if constexpr (!BWD) {
          TT::rows(a, smem + L_::oQ, t, s);
          qs[t] = mma8s(a, sb, qs[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float f[4], w[4];
      lds4(sf + kSk * kC + perm_row4(t, g), f);
      lds4(sf + kSb * kC + perm_row4(t, g), w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[t][e] = fmaf(-f[e], ks[t][e], x[t][e]);
        bb[t][e] = w[e];
      }
    }
    Op8s<float> rb[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) make_op(rb[s], -bb[2 * s] * x[2 * s], -bb[2 * s + 1] * x[2 * s + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = 0; s <= (t >> 1); ++s) {
        Op8<float> a;
        ld_op(a, sM + frag_low(t, s) * kFragElems + lane * 8);
        x[t] = mma8s(a, rb[s], x[t]);
      }
    if constexpr (BWD) {
#pragma unroll
      for (int t = 0; t < 4; ++t) op_st(ws_Y + cc * kC * V, t, col0 >> 4, V / 32, x[t]);
    }
    Op8s<float> eb[2], db[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 d[2], ed[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * s + i;
        float f[4];
        lds4(sf + kSeb * kC + perm_row4(t, g), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[i][e] = bb[t][e] * x[t][e];
          ed[i][e] = f[e] * x[t][e];
        }
      }
      make_op(eb[s], ed[0], ed[1]);
      make_op(db[s], d[0], d[1]);
    }
    if constexpr (!BWD) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float f[4];
        lds4(sf + kSq * kC + perm_row4(t, g), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) qs[t][e] *= f[e];
#pragma unroll
        for (int s = 0; s <= (t >> 1); ++s) {
          Op8<float> a;
          ld_op(a, sP + frag_low(t, s) * kFragElems + lane * 8);
          qs[t] = mma8s(a, db[s], qs[t]);
        }
        tile_st(o + at, HV * V, perm_row4(t, g), col0, L, qs[t]);
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] *= el;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Op8<float> a;
        TT::cols(a, smem, r, s);
        S[r] = mma8s(a, eb[s], S[r]);
      }
    }
  }
  if (!BWD && write_final) {
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

// bf16 in NP pairs of waves, FP32 in NP waves: 16 NP columns per workgroup
template <int K, int V, int NP, bool BWD>
static hipError_t scan_t(const kda_dims& d, const GdnCall& c, const GdnLayout<bf16>& w, hipStream_t s) {
  constexpr size_t lds = GdnScanLds<K, NP, BWD>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  hipError_t e = set_lds(&gdn_scan_kernel<K, V, NP, BWD>, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdn_scan_kernel<K, V, NP, BWD>), dim3(scan_grid((int64_t)d.N * d.HV, V, 16 * NP)),
                     dim3((BWD ? 256 : 128) * NP), lds, s, (const bf16*)c.q, (const bf16*)c.k, (const bf16*)c.v, c.h0, c.cu,
                     w.table, d.N, d.T, d.H, d.HV, w.scal, w.frag, c.ht != nullptr, (bf16*)c.o, c.ht,
                     (const bf16*)c.dO, c.dht, w.S0, w.Y, w.tokf, w.end, w.ancS, w.Yl);
  return hipGetLastError();
}
template <int K, int V, int NP, bool BWD>
static hipError_t scan_t(const kda_dims& d, const GdnCall& c, const GdnLayout<float>& w, hipStream_t s) {
  constexpr size_t lds = GdnScan32Lds<K, BWD>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  hipError_t e = set_lds(&gdn_scan32_kernel<K, V, NP, BWD>, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdn_scan32_kernel<K, V, NP, BWD>), dim3(scan_grid((int64_t)d.N * d.HV, V, 16 * NP)),
                     dim3(64 * NP), lds, s, (const float*)c.q, (const float*)c.k, (const float*)c.v, c.h0, c.cu,
                     w.table, d.N, d.T, d.H, d.HV, w.scal, w.frag, c.ht != nullptr, (float*)c.o, c.ht, w.S0, w.Y);
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
    // once) as long as that leaves two workgroups per compute unit (two value
    // heads a head: 32768 tokens x 16 heads 199 us, one workgroup each 239 us;
    // 8 chunks x 2 heads, FP32, 19 and 12 us)
    const int grp = d.HV / d.H;
    const int hpw = mc * d.H >= 2 * (int64_t)kda_host::device_cus() ? grp : 1;
    hipLaunchKernelGGL((gdn_intra_kernel<T, K, BWD>), dim3((unsigned)(mc * (d.HV / hpw))), dim3(256), 0, s,
                       (const T*)c.q, (const T*)c.k, c.gate, (const T*)c.beta, c.cu, w.table, d.N, d.T, d.H,
                       d.HV, hpw, c.l2, 1.0f / sqrtf((float)K), w.scal, w.frag, w.fragT);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // 64 columns per workgroup while that fills the device, else 32 (608 chains
  // of V = 128, 32768 tokens: 64 columns 431 us, 32 columns 575 us; 64 chains of
  // 4096 tokens: 188 and 135 us). The backward's exchange of 64 columns does
  // not fit LDS.
  const bool wide = (int64_t)d.N * d.HV * (V / 64) >= kda_host::device_cus();
  if constexpr (!BWD || sizeof(T) == 4) {
    if (wide) return scan_t<K, V, 4, BWD>(d, c, w, s);
  }
  return scan_t<K, V, 2, BWD>(d, c, w, s);
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
