// Chunked gated delta rule with a scalar gate, backward. Formulas, layouts and
// the rounding rule are in kda_gdn.h.
//
//   gdn_rev_scan_kernel   the state gradient of 16 columns of one (sequence,
//                         value head), walking the chunks backwards; writes
//                         dv, its part of the tokens' scalars, <D, Y>, and per
//                         chunk dS (at the chunk's end) and D.
//   gdn_gate_bwd_kernel   bf16: the gate's gradient and dbeta from the tokens'
//                         scalars, a workgroup per anchor.
//   gdn_local_kernel      per (chunk, q/k head): dq and dk (summed over the head's
//                         value heads) from the chunk's S0, Y, dS and D
//                         (gdn_local32_kernel for FP32 inputs, with dbeta and the
//                         gate's gradient).
//   gdn_par_kernel        dA_log and d_dt_bias from per-chunk partial sums.
//
// With dP = dO Delta^T and dE = E Delta^T (64 x 64) the gradients of k, q are
//   dq~ = e^G (dO S0^T) + (e . dP) K                          (lower triangle)
//   dk  = e^{G_last - G} (Delta dS^T) - e^G (E S0^T)
//         + (e . dP)^T q~ - (e . dE) K - (e . dE)^T K         (dE strictly lower)
// S0, Y, dS and D pass between the kernels rounded to the inputs' type: they
// feed dq and dk, which are rounded to it as well and sum over V or 64 tokens.
// dbeta = <D, Y> (and <dO, Y>, which scales a token's own part of dq and dk) is one number per token: from rounded operands its error does
// not shrink where the sum's terms cancel (5e-3 in a call of a few tokens), so
// bf16 takes it from D in FP32 and Y's two parts inside the reverse scan (252 ->
// 275 us at 64 chains of 4096 tokens).
//
// The gate's gradient comes one of two ways.
//   bf16: dg_t = <S_T, dS_T> + sum_{t <= i < T} s_i (kda_gdn.h), from FP32 values
//     inside the scans, summed in double. Formed from the rounded S0, Y, dS and D
//     instead it was off by 2e-3, and dA_log and d_dt_bias, which sum it over
//     tokens of either sign, by 1e-2 and more. A token's scalars are off by some
//     1e-6, adding up like a random walk towards T, the same for all tokens
//     before: with T the sequence's end dA_log was off by 5e-3 at 4096 tokens
//     and 4e-2 at 16384. T is therefore the next anchor: every 8 chunks the
//     forward run keeps S in FP32 and the reverse scan takes <S, dS> there (6%
//     of the workspace; 64 chains of 4096 tokens 24 us in all). Every 16 chunks is
//     12 us cheaper and left 3e-3 beside the outputs' rounding.
//   FP32: the operands are exact, the walk would not be small enough, and dg is
//     taken chunk by chunk: what the decay between tokens t - 1 and t scales is
//     the rows i >= t against S0, the columns j < t towards the chunk's end and
//     the pairs i >= t > j,
//       dg_t = e^{G_last} <S0, dS> + sum_{j < t} c_j + sum_{i >= t} (r_i + sum_{j < i} X_ij - sum_{n > i} X_ni),
//       c_j = <k_j, e^{G_last - G_j} dS Delta_j>,  r_i = <q~_i, e^G S0 dO_i> - <k_i, e^G S0 E_i>,
//       X_ij = e_ij (dP_ij q~_i.k_j - dE_ij k_i.k_j)                          (i > j);
//     pairs on one side of t cancel exactly, as both sums add the same X_ij.
#include "kda_gdn.h"

namespace kda {

// ------------------------------------------------------------------ reverse scan
// bf16. Four waves per 16 columns. The state wave keeps dS and walks
//   x = e^{G_last - G} k dS + p,  D' = x - M^T b (x + P_ii dO),  D = D' + P_ii dO,
//   dS = e^{G_last} dS + Z - (e^G k)^T b D
// with p = P^T dO (P strictly lower) and Z = (e^G q~)^T dO, which do not depend
// on dS: the ahead wave forms them a chunk early, and issues the transfers of
// left operands into LDS. The behind wave follows a chunk late with what
// leaves: dS, D and dv = b D in memory, and the columns' part of the tokens'
// scalars; a fourth forms <D, Y>. (One side wave doing all was the step's
// longest: 373 us at 64 chains; <D, Y> in the behind wave 278 us.) Two barriers
// per chunk: at its top (operands, p and Z in LDS), and after the state wave has
// taken p and Z and the others the previous chunk's dS and D'. The state waves
// share their SIMDs with the <D, Y> waves only. 64 chains of 4096 tokens, K = V
// = 128: 281 us, 4.4 us a chunk, bound by the step; splitting the ahead wave in
// two (p, Z) took 15 us more.
template <int K, int NP>
struct GdnRevLds {
  static constexpr int NK = K / 32, RT = K / 16;
  static constexpr uint32_t tok = TokTile<bf16, K>::bytes, tri = kTriElems * sizeof(bf16), scal = 1024;
  // state wave: k, M^T (hi, lo), row factors 0..3 and 8..11, twice
  static constexpr uint32_t sM = tok, sF = sM + 2 * tri, sE = sF + scal, sbuf = sE + scal;
  // side wave: q, P^T (hi, lo), row factors 3..6, twice
  static constexpr uint32_t oP = tok, oF = oP + 2 * tri, obuf = oF + scal;
  static constexpr uint32_t at_o = 2 * sbuf, at_x = at_o + 2 * obuf;
  // exchange of a pair: dS (high part), D'; p, Z
  static constexpr uint32_t xS = NK * 1024, xD = 4 * 1024, xp = 4 * 1024, xZ = RT * 1024;
  static constexpr uint32_t xbuf = xS + xD + xp + xZ;
  static constexpr uint32_t total = at_x + NP * xbuf;
};

// c += X^T b with the six fragments of a transposed triangle (frag_up order)
__device__ __forceinline__ void mma_up(const Op8<bf16> (&a)[6], const bf16x8 (&b)[2], f32x4 (&c)[4]) {
#pragma unroll
  for (int s = 1; s >= 0; --s)
#pragma unroll
    for (int t = 0; t < 2 * s + 2; ++t)
      c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[frag_up(t, s)].v, b[s], c[t], 0, 0, 0);
}

template <int K, int V, int NP>
__global__ void __launch_bounds__(NP * 256)
gdn_rev_scan_kernel(const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
                    const bf16* __restrict__ dO, const float* __restrict__ dht, const int32_t* __restrict__ cu,
                    const int* __restrict__ table, int N, int T_, int H, int HV,
                    const float* __restrict__ ws_scal, const bf16* __restrict__ ws_frag, bf16* __restrict__ dv,
                    float* __restrict__ dh0, bf16* __restrict__ ws_dS, bf16* __restrict__ ws_D,
                    float* __restrict__ ws_tok, const float* __restrict__ ws_ancS, float* __restrict__ ws_anc,
                    const bf16* __restrict__ ws_Y, const bf16* __restrict__ ws_Yl, float* __restrict__ ws_tokb) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using L_ = GdnRevLds<K, NP>;
  using TT = TokTile<bf16, K>;
  constexpr int NK = K / 32, RT = K / 16, BV = 16 * NP, NVB = V / BV;
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = wave % NP, role = wave / NP;  // 0 state, 1 ahead, 2 dbeta, 3 behind
  const GdnChain ch = gdn_chain(NVB, cu, table, N, T_, H, HV);
  if (!ch.ok) return;
  const int col0 = ch.vb * BV + 16 * pair, hv = ch.hv, len = ch.len;
  const size_t st = ((size_t)ch.n * HV + hv) * (size_t)K * V;
  if (len <= 0) {
    if (dh0 && role == 0) gdn_pass(dht, dh0, st, K, V, col0);
    return;
  }
  const int nc = (len + kC - 1) / kC;
  auto chunk = [&](int c) { return (size_t)(ch.c0 + c) * HV + hv; };
  auto tokens = [&](int c) { return min(kC, len - c * kC); };
  auto vrow = [&](int c) { return ((ch.bos + (int64_t)c * kC) * HV + hv) * V; };
  char* xch = smem + L_::at_x + pair * L_::xbuf;
  char* xp = xch + L_::xS + L_::xD;
  char* xZ = xp + L_::xp;

  if (role == 0) {
    f32x4 S[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[r][e] = dht ? dht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] : 0.f;
    TileRaw<bf16> dr[4];
    auto fetch_do = [&](int c) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) tile_ld(dr[t], dO + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
    };
    fetch_do(nc - 1);
    __syncthreads();  // the last chunk's operands
    __builtin_amdgcn_s_setprio(2);
    for (int c = nc - 1, buf = 0; c >= 0; --c, buf ^= 1) {
      __syncthreads();
      if (c + 1 < nc && (c + 1) % kGdnAnchor == 0) {  // <S, dS> before chunk c + 1
        const size_t at = (gdn_anchor(ch.c0, c + 1) * HV + hv) * (V / 16) + (col0 >> 4);
        const float4* a = reinterpret_cast<const float4*>(ws_ancS) + at * RT * 64 + lane;
        float y = 0.f;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float4 s = a[r * 64];
          y += s.x * S[r][0] + s.y * S[r][1] + s.z * S[r][2] + s.w * S[r][3];
        }
        y = row16_sum(y);
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        if (lane == 0) ws_anc[at] = y;
      }
      const char* b = smem + buf * L_::sbuf;
      const bf16* sM = reinterpret_cast<const bf16*>(b + L_::sM);
      const float* sf = reinterpret_cast<const float*>(b + L_::sF);
      const float* se = reinterpret_cast<const float*>(b + L_::sE);  // from slot kSe on
      Op8<bf16> ka[NK][4], ml[2][6];
      auto read_k = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) TT::rows(ka[s][t], b, t, s);
      };
      auto read_m = [&](int f) __attribute__((always_inline)) {
        ld_op(ml[0][f], sM + f * kFragElems + lane * 8);
        ld_op(ml[1][f], sM + kTriElems + f * kFragElems + lane * 8);
      };
      read_k(0);
      read_k(1);
      f32x4 pd[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) pd[t] = tile_get(dr[t]);
      const float el = sf[kSl * kC + lane];
      if (c > 0) fetch_do(c - 1);
      Op8s<bf16> sb[NK];
#pragma unroll
      for (int s = 0; s < NK; ++s) make_op(sb[s], S[2 * s], S[2 * s + 1]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(xZ + (r * 64 + lane) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][e] = fmaf(S[r][e], el, z[e]);
      }
      f32x4 ks[4], x[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ks[t] = zero4();
        x[t] = *reinterpret_cast<const f32x4*>(xp + (t * 64 + lane) * 16);
      }
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
      __syncthreads();  // p, Z and the previous chunk's dS, D' are taken
#pragma unroll
      for (int s = 0; s < NK; ++s) *reinterpret_cast<bf16x8*>(xch + (s * 64 + lane) * 16) = sb[s].hi;
      f32x4 bb[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float f[4], w[4], y[4];
        lds4(se + perm_row4(t, g), f);
        lds4(sf + kSb * kC + perm_row4(t, g), w);
        lds4(se + (kSpd - kSe) * kC + perm_row4(t, g), y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[t][e] = fmaf(f[e], ks[t][e], x[t][e]);
          pd[t][e] *= y[e];
          bb[t][e] = w[e];
        }
      }
      Op8s<bf16> rb[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4 a0, a1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a0[e] = -bb[2 * s][e] * (x[2 * s][e] + pd[2 * s][e]);
          a1[e] = -bb[2 * s + 1][e] * (x[2 * s + 1][e] + pd[2 * s + 1][e]);
        }
        make_op(rb[s], a0, a1);
      }
      {
        const bf16x8 hi[2] = {rb[0].hi, rb[1].hi}, lo[2] = {rb[0].lo, rb[1].lo};
        mma_up(ml[0], lo, x);
        mma_up(ml[1], hi, x);
        mma_up(ml[0], hi, x);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(xch + L_::xS + (t * 64 + lane) * 16) = x[t];
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
          lds4(sf + kSk * kC + perm_row4(t, g), f);
#pragma unroll
          for (int e = 0; e < 4; ++e) ed[i][e] = -(f[e] * bb[t][e]) * (x[t][e] + pd[t][e]);
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
    __syncthreads();  // the behind wave's last chunk
    __syncthreads();
    if (dh0) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dh0[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] = S[r][e];
    }
    return;
  }

  if (role == 1) {
    const uint32_t lds = lds_addr(smem);
    const TokDma<bf16, K, NP> tok((uint32_t)(H * K * sizeof(bf16)), pair);
    auto fetch_s = [&](int c, int buf) __attribute__((always_inline)) {
      const uint32_t b = lds + buf * L_::sbuf;
      tok.go(b, k + ((ch.bos + (int64_t)c * kC) * H + ch.h) * K, tokens(c));
      dma_flat<2 * L_::tri, NP>(b + L_::sM, ws_frag + chunk(c) * GdnWs<bf16>::bwd, pair);
      dma_flat<L_::scal, NP>(b + L_::sF, ws_scal + chunk(c) * (kGdnScal * kC), pair);
      dma_flat<L_::scal, NP>(b + L_::sE, ws_scal + chunk(c) * (kGdnScal * kC) + kSe * kC, pair);
    };
    auto fetch_o = [&](int c) __attribute__((always_inline)) {
      const uint32_t b = lds + L_::at_o + (c & 1) * L_::obuf;
      tok.go(b, q + ((ch.bos + (int64_t)c * kC) * H + ch.h) * K, tokens(c));
      dma_flat<2 * L_::tri, NP>(b + L_::oP, ws_frag + chunk(c) * GdnWs<bf16>::bwd + 2 * kTriElems, pair);
      dma_flat<L_::scal, NP>(b + L_::oF, ws_scal + chunk(c) * (kGdnScal * kC) + kSb * kC, pair);
    };
    TileRaw<bf16> dn[4];  // dO of the chunk ahead
    auto fetch_dn = [&](int c) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) tile_ld(dn[t], dO + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
    };
    auto ahead = [&](int c) __attribute__((always_inline)) {  // p and Z of chunk c into LDS
      const char* ob = smem + L_::at_o + (c & 1) * L_::obuf;
      const bf16* sP = reinterpret_cast<const bf16*>(ob + L_::oP);
      const float* of = reinterpret_cast<const float*>(ob + L_::oF);  // from slot kSb on
      Op8<bf16> pf[2][6];
#pragma unroll
      for (int f = 0; f < 6; ++f)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) ld_op(pf[pt][f], sP + pt * kTriElems + f * kFragElems + lane * 8);
      Op8<bf16> dop[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) tile_op(dop[s], dn[2 * s], dn[2 * s + 1]);
      Op8s<bf16> qb[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4 d[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = __builtin_bit_cast(uint4, dop[s].v);
          d[i] = unpack4(i ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y));
          float f[4];
          lds4(of + (kSq - kSb) * kC + perm_row4(2 * s + i, g), f);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[i][e] *= f[e];
        }
        make_op(qb[s], d[0], d[1]);
      }
      if (c > 0) fetch_dn(c - 1);
      Op8<bf16> qc[RT][2];
      auto read_qc = [&](int r) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s) TT::cols(qc[r][s], ob, r, s);
      };
      read_qc(0);
      read_qc(1);
      stage();
      f32x4 p[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) p[t] = zero4();
      const bf16x8 dd[2] = {dop[0].v, dop[1].v};
      mma_up(pf[1], dd, p);
      mma_up(pf[0], dd, p);
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(xp + (t * 64 + lane) * 16) = p[t];
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        stage();
        if (r + 2 < RT) {
          read_qc(r + 2);
          read_qc(r + 3);
        }
        stage();
        f32x4 z0 = zero4(), z1 = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          z0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qc[r][s].v, qb[s].lo, z0, 0, 0, 0);
          z1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qc[r + 1][s].v, qb[s].lo, z1, 0, 0, 0);
          z0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qc[r][s].v, qb[s].hi, z0, 0, 0, 0);
          z1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qc[r + 1][s].v, qb[s].hi, z1, 0, 0, 0);
        }
        *reinterpret_cast<f32x4*>(xZ + (r * 64 + lane) * 16) = z0;
        *reinterpret_cast<f32x4*>(xZ + ((r + 1) * 64 + lane) * 16) = z1;
      }
    };
    fetch_s(nc - 1, 0);
    fetch_o(nc - 1);
    if (nc > 1) fetch_o(nc - 2);
    fetch_dn(nc - 1);
    lds_dma_wait();
    __syncthreads();
    ahead(nc - 1);
    for (int c = nc - 1, buf = 0; c >= -1; --c, buf ^= 1) {
      lds_dma_wait();
      __syncthreads();
      if (c > 0) fetch_s(c - 1, buf ^ 1);
      if (c > 1) fetch_o(c - 2);
      __syncthreads();
      if (c > 0) ahead(c - 1);
    }
    return;
  }

  if (role == 2) {  // <D, Y> and <dO, Y> of the chunk behind
    TileRaw<bf16> db[4];
    uint2 yh[4], yl[4];
    float pw[4][4];
    auto fetch = [&](int c) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        tile_ld(db[t], dO + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
        lds4(ws_scal + chunk(c) * (kGdnScal * kC) + kSp * kC + perm_row4(t, g), pw[t]);
        yh[t] = op_tile_ld(ws_Y + chunk(c) * kC * V, t, col0 >> 4, V / 32);
        yl[t] = reinterpret_cast<const uint2*>(ws_Yl)[((chunk(c) * (V / 16) + (col0 >> 4)) * 4 + t) * 64 + lane];
      }
    };
    fetch(nc - 1);
    __syncthreads();
    for (int c = nc - 1; c >= -1; --c) {
      const int cb = c + 1;
      __syncthreads();
      f32x4 x[4], z[4];
      if (cb < nc) {
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = *reinterpret_cast<const f32x4*>(xch + L_::xS + (t * 64 + lane) * 16);
      }
      __syncthreads();
      if (cb >= nc) continue;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 dt = tile_get(db[t]), y0 = unpack4(quad_transpose(yh[t])), y1 = unpack4(yl[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = fmaf(pw[t][e], dt[e], x[t][e]);
          x[t][e] = row16_sum(fmaf(d, y0[e], d * y1[e]));
          z[t][e] = row16_sum(fmaf(dt[e], y0[e], dt[e] * y1[e]));
        }
      }
      stage();
      if (c >= 0) fetch(c);
      stage();
      float* tk = ws_tokb + (chunk(cb) * 2 * (V / 16) + (col0 >> 4)) * kC;
      if (l16 == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          *reinterpret_cast<float4*>(tk + perm_row4(t, g)) = make_float4(x[t][0], x[t][1], x[t][2], x[t][3]);
          *reinterpret_cast<float4*>(tk + (V / 16) * kC + perm_row4(t, g)) =
              make_float4(z[t][0], z[t][1], z[t][2], z[t][3]);
        }
      }
    }
    return;
  }

  // ---- behind wave
  TileRaw<bf16> vb[4], db[4];  // v and dO of the chunk behind, fetched a round early
  float bw[4][4], pw[4][4];
  auto fetch_b = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      tile_ld(vb[t], v + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
      tile_ld(db[t], dO + vrow(c), HV * V, perm_row4(t, g), col0, tokens(c));
      const float* f = ws_scal + chunk(c) * (kGdnScal * kC);
      lds4(f + kSb * kC + perm_row4(t, g), bw[t]);
      lds4(f + kSp * kC + perm_row4(t, g), pw[t]);
    }
  };
  fetch_b(nc - 1);
  __syncthreads();  // the last chunk's operands
  for (int c = nc - 1; c >= -1; --c) {
    const int cb = c + 1;  // the chunk behind
    __syncthreads();
    uint4 sh[NK];
    f32x4 x[4];
    if (cb < nc) {
#pragma unroll
      for (int s = 0; s < NK; ++s) sh[s] = *reinterpret_cast<const uint4*>(xch + (s * 64 + lane) * 16);
#pragma unroll
      for (int t = 0; t < 4; ++t) x[t] = *reinterpret_cast<const f32x4*>(xch + L_::xS + (t * 64 + lane) * 16);
    }
    __syncthreads();
    if (cb >= nc) continue;
    f32x4 dd[4];
    float4 sv[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 vt = tile_get(vb[t]), dt = tile_get(db[t]);
      float z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] = row16_sum(bw[t][e] * x[t][e] * vt[e]);
        x[t][e] = fmaf(pw[t][e], dt[e], x[t][e]);
        dd[t][e] = x[t][e] * bw[t][e];
      }
      sv[t] = make_float4(z[0], z[1], z[2], z[3]);
    }
    stage();
    if (c >= 0) fetch_b(c);
    stage();
#pragma unroll
    for (int r = 0; r < RT; ++r)
      op_st(ws_dS + chunk(cb) * K * V, r, col0 >> 4, V / 32,
            (r & 1) ? make_uint2(sh[r >> 1].z, sh[r >> 1].w) : make_uint2(sh[r >> 1].x, sh[r >> 1].y));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      op_st(ws_D + chunk(cb) * kC * V, t, col0 >> 4, V / 32, pack4(x[t]));
      tile_st(dv + vrow(cb), HV * V, perm_row4(t, g), col0, tokens(cb), dd[t]);
    }
    const size_t tk = (chunk(cb) * (V / 16) + (col0 >> 4)) * kC;
    if (l16 == 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        *reinterpret_cast<float4*>(ws_tok + tk + perm_row4(t, g)) = sv[t];
      }
    }
  }
}

// bf16: the gate's gradient and dbeta from the tokens' scalars. A workgroup takes the 8
// chunks from one anchor to the next, lane = token, wave = chunk; the sums
// towards the anchor behind them (the sequence's end for the last) are held in
// double. Grid (chain, y): y strides over a chain's anchors.
template <int V>
__global__ void __launch_bounds__(64 * kGdnAnchor)
gdn_gate_bwd_kernel(GdnGate gate, const int32_t* __restrict__ cu, const int* __restrict__ table, int T_, int HV,
                    int has_h0, int has_dht, const float* __restrict__ tokf, const float* __restrict__ tokr,
                    const float* __restrict__ tokb, const float* __restrict__ ends, const float* __restrict__ anc,
                    void* __restrict__ dgate, bf16* __restrict__ dbeta, float* __restrict__ par,
                    float* __restrict__ ws_scal) {
  constexpr int NB = V / 16;
  __shared__ double s_tot[2][kGdnAnchor];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = blockIdx.x / HV, hv = blockIdx.x % HV;
  int64_t bos = (int64_t)n * T_;
  int len = T_;
  if (cu) {
    bos = cu[n];
    len = cu[n + 1] - cu[n];
  }
  const int nc = (len + kC - 1) / kC;
  if (nc <= 0) return;
  const int64_t c0 = cu ? table[1 + n] : (int64_t)n * nc;
  for (int m = blockIdx.y, b = 0; m * kGdnAnchor < nc; m += gridDim.y, b ^= 1) {
    const int c = m * kGdnAnchor + wave, cl = min(c, nc - 1);
    const bool ok = c < nc && lane < len - c * kC;
    const size_t at = (size_t)((c0 + cl) * HV + hv) * NB * kC + lane;
    const int64_t tok = (bos + min(cl * kC + lane, len - 1)) * HV + hv;
    double s = 0.;
    float y = 0.f, p = 0.f;
    const size_t atb = (size_t)((c0 + cl) * HV + hv) * 2 * NB * kC + lane;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      s += (double)tokf[at + i * kC] - (double)tokr[at + i * kC];
      y += tokb[atb + i * kC];
      p += tokb[atb + (NB + i) * kC];
    }
    if (!ok) s = 0.;
    const bool last = (m + 1) * kGdnAnchor >= nc;
    const float* e = last ? ends + ((size_t)n * HV + hv) * NB
                          : anc + (gdn_anchor(c0, (m + 1) * kGdnAnchor) * HV + hv) * NB;
    double behind = 0.;
    if (!last || has_dht)
#pragma unroll
      for (int i = 0; i < NB; ++i) behind += (double)e[i];
    float xb, as;
    const float gn = gdn_gate(gate, tok, hv, &xb, &as);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double z = __shfl_down(s, d);
      if (lane + d < 64) s += z;
    }
    if (lane == 0) s_tot[b][wave] = s;
    __syncthreads();
#pragma unroll
    for (int w = kGdnAnchor - 1; w > 0; --w) behind += w > wave ? s_tot[b][w] : 0.;
    if (c >= nc) continue;
    // the scans are done with this slot
    ws_scal[(size_t)((c0 + c) * HV + hv) * (kGdnScal * kC) + kSpy * kC + lane] = ok ? p : 0.f;
    // before a sequence's first token there is nothing to decay without a state
    const float dg = c == 0 && lane == 0 && !has_h0 ? 0.f : (float)(s + behind);
    const float dx = gate.raw ? -dg * as * sigmoid_f32(xb) : dg;
    if (ok) {
      st_any(dgate, tok, gate.bf, dx);
      dbeta[tok] = from_f32<bf16>(y);
    }
    if (gate.A_log || gate.dt_bias) {
      float pa = ok ? dg * gn : 0.f, pb = ok ? dx : 0.f;  // dg / dA_log = g
#pragma unroll
      for (int d = 32; d; d >>= 1) {
        pa += __shfl_xor(pa, d);
        pb += __shfl_xor(pb, d);
      }
      if (lane == 0) *reinterpret_cast<float2*>(par + 2 * ((c0 + c) * HV + hv)) = make_float2(pa, pb);
    }
  }
}

// FP32: one wave per 16 columns, FP32 matrix cores, one operand buffer.
template <int K>
struct GdnRev32Lds {
  static constexpr uint32_t tok = TokTile<float, K>::bytes, tri = 2 * kTriElems * sizeof(float);
  static constexpr uint32_t oQ = tok, oM = 2 * tok, oS = oM + tri, total = oS + kGdnScal * kC * sizeof(float);
};

template <int K, int V, int NW>
__global__ void __launch_bounds__(NW * 64)
gdn_rev_scan32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ dO,
                      const float* __restrict__ dht, const int32_t* __restrict__ cu,
                      const int* __restrict__ table, int N, int T_, int H, int HV,
                      const float* __restrict__ ws_scal, const float* __restrict__ ws_frag,
                      float* __restrict__ dv, float* __restrict__ dh0, float* __restrict__ ws_dS,
                      float* __restrict__ ws_D) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using L_ = GdnRev32Lds<K>;
  using TT = TokTile<float, K>;
  constexpr int NK = K / 32, RT = K / 16, BV = 16 * NW, NVB = V / BV;
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GdnChain ch = gdn_chain(NVB, cu, table, N, T_, H, HV);
  if (!ch.ok) return;
  const int col0 = ch.vb * BV + 16 * wave, hv = ch.hv, len = ch.len;
  const size_t st = ((size_t)ch.n * HV + hv) * (size_t)K * V;
  if (len <= 0) {
    if (dh0) gdn_pass(dht, dh0, st, K, V, col0);
    return;
  }
  const int nc = (len + kC - 1) / kC;
  const uint32_t lds = lds_addr(smem);
  const TokDma<float, K, NW> tok((uint32_t)(H * K * sizeof(float)), wave);
  const float* sf = reinterpret_cast<const float*>(smem + L_::oS);
  const float* sM = reinterpret_cast<const float*>(smem + L_::oM);
  const float* sP = sM + kTriElems;
  f32x4 S[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[r][e] = dht ? dht[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] : 0.f;
  for (int c = nc - 1; c >= 0; --c) {
    if (c < nc - 1) __syncthreads();  // every wave is done with the buffer
    const size_t cc = (size_t)(ch.c0 + c) * HV + hv;
    const int64_t row = ((ch.bos + (int64_t)c * kC) * H + ch.h) * K, at = ((ch.bos + (int64_t)c * kC) * HV + hv) * V;
    const int L = min(kC, len - c * kC);
    tok.go(lds, k + row, L);
    tok.go(lds + L_::oQ, q + row, L);
    dma_flat<(int)L_::tri, NW>(lds + L_::oM, ws_frag + cc * GdnWs<float>::bwd, wave);
    dma_flat<kGdnScal * kC * 4, NW>(lds + L_::oS, ws_scal + cc * (kGdnScal * kC), wave);
    f32x4 dot[4], x[4], p[4], bb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      TileRaw<float> r;
      tile_ld(r, dO + at, HV * V, perm_row4(t, g), col0, L);
      dot[t] = r.r;
      x[t] = p[t] = zero4();
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) op_st(ws_dS + cc * K * V, r, col0 >> 4, V / 32, S[r]);
    lds_dma_wait();
    __syncthreads();
    const float el = sf[kSl * kC];
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      Op8s<float> sb;
      make_op(sb, S[2 * s], S[2 * s + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Op8<float> a;
        TT::rows(a, smem, t, s);
        x[t] = mma8s(a, sb, x[t]);
      }
    }
    Op8s<float> dop[2], rb[2], qb[2], kb[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) make_op(dop[s], dot[2 * s], dot[2 * s + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int s = (t >> 1); s < 2; ++s) {
        Op8<float> a;
        ld_op(a, sP + frag_up(t, s) * kFragElems + lane * 8);
        p[t] = mma8s(a, dop[s], p[t]);
      }
      float f[4], w[4], y[4];
      lds4(sf + kSe * kC + perm_row4(t, g), f);
      lds4(sf + kSb * kC + perm_row4(t, g), w);
      lds4(sf + kSp * kC + perm_row4(t, g), y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[t][e] = fmaf(y[e], dot[t][e], fmaf(f[e], x[t][e], p[t][e]));  // dDelta
        bb[t][e] = w[e];
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) make_op(rb[s], -bb[2 * s] * x[2 * s], -bb[2 * s + 1] * x[2 * s + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = (t >> 1); s < 2; ++s) {
        Op8<float> a;
        ld_op(a, sM + frag_up(t, s) * kFragElems + lane * 8);
        x[t] = mma8s(a, rb[s], x[t]);
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) op_st(ws_D + cc * kC * V, t, col0 >> 4, V / 32, x[t]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 eq[2], ek[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * s + i;
        float fq[4], fk[4];
        lds4(sf + kSq * kC + perm_row4(t, g), fq);
        lds4(sf + kSk * kC + perm_row4(t, g), fk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[t][e] *= bb[t][e];
          eq[i][e] = fq[e] * dot[t][e];
          ek[i][e] = -fk[e] * x[t][e];
        }
        tile_st(dv + at, HV * V, perm_row4(t, g), col0, L, x[t]);
      }
      make_op(qb[s], eq[0], eq[1]);
      make_op(kb[s], ek[0], ek[1]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] *= el;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Op8<float> a;
        TT::cols(a, smem + L_::oQ, r, s);
        S[r] = mma8s(a, qb[s], S[r]);
        TT::cols(a, smem, r, s);
        S[r] = mma8s(a, kb[s], S[r]);
      }
    }
  }
  if (dh0) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dh0[st + (size_t)(perm_row4(r, g) + e) * V + col0 + l16] = S[r][e];
  }
}

// ------------------------------------------------------------------ local gradients
// c += a b, the left operand split
__device__ __forceinline__ f32x4 mma8a(const Op8s<bf16>& a, const Op8<bf16>& b, f32x4 c) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.lo, b.v, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.hi, b.v, c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ float op_dot(const Op8<T>& a, const Op8<T>& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(op_get(a, i), op_get(b, i), s);
  return s;
}

// bf16. Eight waves: wave w and wave w + 4 own token tile w. The first four
// form what takes a token as the later of a pair (from S0, Y: dq and a part of
// dk), the others what takes it as the earlier (from dS, dO, D: the rest
// of dk). The kernel moves 180 KB for some 2 us of products, so one
// workgroup stays on a CU, walks its (chunk, head) items and keeps two sets of
// transfers into LDS going: S0, dS, k and q arrive while the 64 x 64 products
// run over Y, D and dO, and the next item's Y, D and dO while the channel tiles
// run over S0 and dS. 4096 items of K = V = 128, 720 MB: 173 us, 4.2 TB/s (305 us
// with four waves a workgroup loading their operands where they use them; 166 us
// with the pairs' factors W and Z rounded to one part, which left a call of three
// tokens 5e-3 off).
template <int K, int V>
struct GdnLocalLds {
  static constexpr uint32_t tok = TokTile<bf16, K>::bytes, st = K * V * sizeof(bf16), row = kC * V * sizeof(bf16);
  static constexpr uint32_t scal = kGdnScal * kC * sizeof(float);
  static constexpr uint32_t oQ = tok, oS = oQ + tok, odS = oS + st, oY = odS + st, oD = oY + row, oO = oD + row;
  static constexpr uint32_t oF = oO + row, total = oF + 2 * scal;
  static_assert(2 * st >= (K / 16) * 4 * 1024, "dk's exchange fits S0 and dS");
};

template <int K, int V>
__global__ void __launch_bounds__(512, 2)
gdn_local_kernel(const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ dO,
                 const int32_t* __restrict__ cu, const int* __restrict__ table, int chunks, int N, int T_, int H,
                 int HV, int l2, float scale, const float* __restrict__ ws_scal, const bf16* __restrict__ ws_S0,
                 const bf16* __restrict__ ws_Y, const bf16* __restrict__ ws_dS, const bf16* __restrict__ ws_D,
                 bf16* __restrict__ dq, bf16* __restrict__ dk) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using L_ = GdnLocalLds<K, V>;
  using TT = TokTile<bf16, K>;
  using TV = TokTile<bf16, V>;
  constexpr int NV = V / 32, RT = K / 16;
  const int w8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = w8 & 3;
  const bool later = w8 < 4;
  const int grp = HV / H;
  const char *sK = smem, *sQ = smem + L_::oQ;
  const bf16* sS0 = reinterpret_cast<const bf16*>(smem + L_::oS);
  const bf16* sdS = reinterpret_cast<const bf16*>(smem + L_::odS);
  const bf16* sY = reinterpret_cast<const bf16*>(smem + L_::oY);
  const bf16* sD = reinterpret_cast<const bf16*>(smem + L_::oD);
  const char* sO = smem + L_::oO;
  char* sx = smem + L_::oS;  // exchange of dk, once S0 and dS are read
  const uint32_t lds = lds_addr(smem);
  const TokDma<bf16, K, 8> tok((uint32_t)(H * K * sizeof(bf16)), w8);
  const TokDma<bf16, V, 8> tov((uint32_t)(HV * V * sizeof(bf16)), w8);
  const int p = wave >> 1;  // 32-token block of the wave's tokens

  // the transfers a wave issues for Y, D and dO of one value head, row factors first
  constexpr int kRowDma = 2 * (int)(L_::row / 8192) + TokDma<bf16, V, 8>::kPer;
  auto fetch_rows = [&](int64_t t0, int L, int64_t ch, int hv, int buf, int lane) __attribute__((always_inline)) {
    dma_flat<L_::scal, 8>(lds + L_::oF + buf * L_::scal, ws_scal + ch * (kGdnScal * kC), w8);
    dma_flat<L_::row, 8>(lds + L_::oY, ws_Y + ch * kC * V, w8);
    dma_flat<L_::row, 8>(lds + L_::oD, ws_D + ch * kC * V, w8);
    tov.go_lean(lds + L_::oO, dO + (t0 * HV + hv) * V, L, lane);
  };
  auto fetch_states = [&](int64_t ch) __attribute__((always_inline)) {
    dma_flat<L_::st, 8>(lds + L_::oS, ws_S0 + ch * K * V, w8);
    dma_flat<L_::st, 8>(lds + L_::odS, ws_dS + ch * K * V, w8);
  };

  const int items = (cu ? table[0] : chunks) * H;
  int it = blockIdx.x;
  if (it >= items) return;
  ChunkGeo geo = chunk_geo(it / H, cu, table, N, T_);
  fetch_rows(geo.t0, geo.L, (int64_t)(it / H) * HV + (it % H) * grp, (it % H) * grp, 0, threadIdx.x & 63);
  lds_dma_wait();
  int buf = 0;
  for (; it < items; it += gridDim.x) {
    const int j = it / H, h = it % H, L = geo.L;
    const int64_t t0 = geo.t0;
    f32x4 aq[RT], ak[RT];  // aq: the first four waves only
#pragma unroll
    for (int r = 0; r < RT; ++r) aq[r] = ak[r] = zero4();
    const int nxt = it + gridDim.x;
    if (nxt < items) geo = chunk_geo(nxt / H, cu, table, N, T_);

    for (int hh = 0; hh < grp; ++hh, buf ^= 1) {
      const int hv = h * grp + hh;
      const int64_t ch = (int64_t)j * HV + hv;
      const float* sc = reinterpret_cast<const float*>(smem + L_::oF + buf * L_::scal);
      const double* sG = reinterpret_cast<const double*>(sc + kSG * kC);
      // the lane is made anew for each round: kept over all of them, the LDS addresses made from
      // it filled the registers, and what spills waits for the transfers under way
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));
      const int g = lane >> 4, l16 = lane & 15;
      const int own = perm_row(wave, l16);  // this lane's row as an operand
      const int own4 = perm_row4(wave, g);  // first of its four accumulator rows
      __syncthreads();  // Y, D, dO and the row factors are in LDS; S0, dS, k and q are read
      if (hh == 0) {
        tok.go_lean(lds, k + (t0 * H + h) * K, L, lane);
        tok.go_lean(lds + L_::oQ, q + (t0 * H + h) * K, L, lane);
      }
      fetch_states(ch);

      // 64 x 64 parts. As rows (contraction over j): W_ij = e_ij b_j rk_j / sqrt(K) dO_i.Y_j and
      // Z_ij = - e_ij b_i b_j rk_j D_i.Y_j, from the products with Y's rows on the left, so the
      // accumulators are the operand with the wave's tokens as rows. As columns (contraction
      // over i): W'_ij = e_ij b_j rq_i / sqrt(K) dO_i.Y_j, Z'_ij = - e_ij b_i b_j rk_i D_i.Y_j.
      // dO_i.Y_i comes from the scan in FP32: a token on its own has all of dq and dk from it.
      Op8<bf16> oa[NV], ob[NV];  // own rows: dO and D; Y
      Op8s<bf16> wo[2], zo[2];  // in two parts: one number scales a pair's whole row of k or q
      const double Go = sG[own];
      const float bo = sc[kSb * kC + own], pyo = sc[kSpy * kC + own];
      if (later) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          TV::rows(oa[u], sO, wave, u, lane);
          op_ld(ob[u], sD, wave, u, NV, lane);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          f32x4 w[2], z[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) w[i] = z[i] = zero4();
          if (s <= p) {
#pragma unroll
            for (int u = 0; u < NV; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                Op8<bf16> y;
                op_ld(y, sY, 2 * s + i, u, NV, lane);
                w[i] = mma8(y, oa[u], w[i]);
                z[i] = mma8(y, ob[u], z[i]);
              }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row4 = perm_row4(2 * s + i, g);
              float b4[4], rk_[4];
              float gg[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                gg[e] = (float)(Go - sG[row4 + e]);
                settle(gg[e]);  // no branch around the read
              }
              lds4(sc + kSb * kC + row4, b4);
              lds4(sc + kSrk * kC + row4, rk_);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int o = row4 + e;  // the earlier token
                const float ej = ex2((own >= o) & (own < L) ? gg[e] : -INFINITY) * b4[e] * rk_[e];
                w[i][e] = (own == o ? pyo : w[i][e]) * (ej * scale);
                z[i][e] *= own > o ? -ej * bo : 0.f;
              }
            }
          }
          make_op(wo[s], w[0], w[1]);
          make_op(zo[s], z[0], z[1]);
          stage();
        }
      } else {
#pragma unroll
        for (int u = 0; u < NV; ++u) op_ld(oa[u], sY, wave, u, NV, lane);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          f32x4 w[2], z[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) w[i] = z[i] = zero4();
          if (s >= p) {
#pragma unroll
            for (int u = 0; u < NV; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                Op8<bf16> a, d;
                TV::rows(a, sO, 2 * s + i, u, lane);
                op_ld(d, sD, 2 * s + i, u, NV, lane);
                w[i] = mma8(a, oa[u], w[i]);
                z[i] = mma8(d, oa[u], z[i]);
              }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row4 = perm_row4(2 * s + i, g);
              float b4[4], rq_[4], rk_[4];
              float gg[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                gg[e] = (float)(Go - sG[row4 + e]);
                settle(gg[e]);  // no branch around the read
              }
              lds4(sc + kSb * kC + row4, b4);
              lds4(sc + kSrq * kC + row4, rq_);
              lds4(sc + kSrk * kC + row4, rk_);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int o = row4 + e;  // the later token
                const float ei = ex2((o >= own) & (o < L) ? -gg[e] : -INFINITY) * bo;
                w[i][e] = (own == o ? pyo : w[i][e]) * (ei * rq_[e] * scale);
                z[i][e] *= o > own ? -ei * b4[e] * rk_[e] : 0.f;
              }
            }
          }
          make_op(wo[s], w[0], w[1]);
          make_op(zo[s], z[0], z[1]);
          stage();
        }
      }
      // the next value head's rows, or the next item's
      const bool more = hh + 1 < grp;
      __syncthreads();  // Y, D and dO are read
      if (more || nxt < items) {
        const int nj = more ? j : nxt / H, nhv = more ? hv + 1 : (nxt % H) * grp;
        fetch_rows(more ? t0 : geo.t0, more ? L : geo.L, (int64_t)nj * HV + nhv, nhv, buf ^ 1, lane);
        lds_dma_wait_but<kRowDma>();
      } else {
        lds_dma_wait();
      }
      __syncthreads();  // S0, dS, k and q are in LDS

      // channel tiles (a block of pairs that none of the tile's tokens has is zero in wo and zo; a
      // branch around it costs more). fq = e^G rq / sqrt(K), fk = e^G rk, fe = e^{G_last - G} rk: gradients of
      // the normalised rows, times their own inverse norm
      float fb[4], frk[4];
      lds4(sc + kSb * kC + own4, fb);
      lds4(sc + kSrk * kC + own4, frk);
      if (later) {
        float fk[4], fq[4], frq[4];
        lds4(sc + kSk * kC + own4, fk);
        lds4(sc + kSq * kC + own4, fq);
        lds4(sc + kSrq * kC + own4, frq);
#pragma unroll
        for (int e = 0; e < 4; ++e) fk[e] *= -fb[e];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 a1 = zero4(), a2 = zero4(), tq = zero4(), tr = zero4();
#pragma unroll
          for (int s = 0; s < NV; ++s) {
            Op8<bf16> x;
            op_ld(x, sS0, r, s, NV, lane);
            a1 = mma8(oa[s], x, a1);
            a2 = mma8(ob[s], x, a2);
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            Op8<bf16> kc;
            TT::cols(kc, sK, r, s, lane);
            tq = mma8a(wo[s], kc, tq);
            tr = mma8a(zo[s], kc, tr);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            aq[r][e] += a1[e] * fq[e] + frq[e] * tq[e];
            ak[r][e] += a2[e] * fk[e] + frk[e] * tr[e];
          }
          stage();  // one tile's operands live at a time
        }
      } else {
        float fe[4];
        lds4(sc + kSe * kC + own4, fe);
#pragma unroll
        for (int e = 0; e < 4; ++e) fe[e] *= fb[e];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 a3 = zero4(), tc = zero4();
#pragma unroll
          for (int s = 0; s < NV; ++s) {
            Op8<bf16> x;
            op_ld(x, sdS, r, s, NV, lane);
            a3 = mma8(oa[s], x, a3);
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            Op8<bf16> kc, qc;
            TT::cols(kc, sK, r, s, lane);
            TT::cols(qc, sQ, r, s, lane);
            tc = mma8a(wo[s], qc, tc);
            tc = mma8a(zo[s], kc, tc);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) ak[r][e] += a3[e] * fe[e] + frk[e] * tc[e];
          stage();
        }
      }
      if (more) lds_dma_wait();
      if (!more) {
        // dk's first part to the wave with the other; then each finishes one gradient
        float rn[4];
        lds4(sc + (later ? kSrq : kSrk) * kC + own4, rn);
        lds_dma_wait();   // before the stores below, not behind them
        __syncthreads();  // S0 and dS are read
        f32x4* x = reinterpret_cast<f32x4*>(sx) + (wave * RT) * 64 + lane;
        if (later) {
#pragma unroll
          for (int r = 0; r < RT; ++r) x[r * 64] = ak[r];
        }
        __syncthreads();
        if (!later) {
          f32x4 y[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) y[r] = x[r * 64];
#pragma unroll
          for (int r = 0; r < RT; ++r) aq[r] = ak[r] + y[r];
        }
        const char* sT = later ? sQ : sK;
        // through the L2 norm: q^ = rq q, so dq = rq (dq^ - q^ <q^, dq^>); aq holds rq dq^
        if (l2) {
          float nn[4] = {0.f, 0.f, 0.f, 0.f};
          f32x4 xt[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            xt[r] = TT::tile(sT, wave, r, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) nn[e] = fmaf(xt[r][e], aq[r][e], nn[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) nn[e] = row16_sum(nn[e]) * rn[e] * rn[e];
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) aq[r][e] = fmaf(-xt[r][e], nn[e], aq[r][e]);
        }
        const int row = own4 + (l16 & 3);
        bf16* out = (later ? dq : dk) + ((t0 + row) * H + h) * K + 8 * (l16 >> 2);
        uint2 y[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) y[r] = quad_transpose(pack4(aq[r]));
        if (row < L) {
#pragma unroll
          for (int r = 0; r < RT; ++r) *reinterpret_cast<uint2*>(out + 32 * (r >> 1) + 4 * (r & 1)) = y[r];
        }
      }
    }
  }
}

// FP32. Four waves, one per token tile, operands straight from memory. With few
// chunks (8 x 2 heads, K = 64, V = 128: 65 us) the FP32 matrix cores of a few
// compute units bound it: eight waves split as above took 63 us.
template <int K, int V>
__global__ void __launch_bounds__(256)
gdn_local32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ dO, GdnGate gate,
                   const int32_t* __restrict__ cu, const int* __restrict__ table, int N, int T_, int H,
                   int HV, int l2, int has_h0, float scale, const float* __restrict__ ws_scal,
                   const float* __restrict__ ws_S0, const float* __restrict__ ws_Y, const float* __restrict__ ws_dS,
                   const float* __restrict__ ws_D, float* __restrict__ dq, float* __restrict__ dk,
                   float* __restrict__ dbeta, void* __restrict__ dgate, float* __restrict__ par) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using T = float;
  using TT = TokTile<T, K>;
  constexpr int NV = V / 32, RT = K / 16;
  __shared__ double sG[kC];
  __shared__ __attribute__((aligned(16))) float sB[kC];
  __shared__ __attribute__((aligned(16))) float sR[kC], sC[kC];
  __shared__ float sS[4], sX[kC], sXc[4][kC];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = blockIdx.x / H, h = blockIdx.x % H, grp = HV / H;
  const ChunkGeo geo = chunk_geo(j, cu, table, N, T_);
  if (!geo.ok) return;
  const int L = geo.L;
  char* sK = smem;
  char* sQ = smem + TT::bytes;
  {
    const int64_t row = (geo.t0 * H + h) * K;
    const TokDma<T, K, 4> tok((uint32_t)(H * K * sizeof(T)), wave);
    const uint32_t lds = lds_addr(smem);
    tok.go(lds, k + row, L);
    tok.go(lds + TT::bytes, q + row, L);
  }
  const int own = perm_row(wave, l16);   // this lane's row as an operand
  const int own4 = perm_row4(wave, g);   // first of its four accumulator rows
  const int p = wave >> 1;               // 32-token block of the wave's tokens
  f32x4 aq[RT], ak[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) aq[r] = ak[r] = zero4();
  f32x4 rq4, rk4;  // q and k norms of the lane's rows (scale included in neither)

  for (int hh = 0; hh < grp; ++hh) {
    const int hv = h * grp + hh;
    const size_t ch = (size_t)j * HV + hv;
    const float* sc = ws_scal + ch * (kGdnScal * kC);
    if (tid < kC) {
      sG[tid] = reinterpret_cast<const double*>(sc + kSG * kC)[tid];
      sB[tid] = sc[kSb * kC + tid];
    }
    // operands of the wave's own rows
    Op8<T> od[NV], oD[NV], oY[NV];
    const T* dOb = dO + (geo.t0 * HV + hv) * V;
    const T* Db = ws_D + ch * kC * V;
    const T* Yb = ws_Y + ch * kC * V;
#pragma unroll
    for (int s = 0; s < NV; ++s) {
      ld_op(od[s], dOb + (int64_t)min(own, L - 1) * HV * V + 32 * s + 8 * g);
      op_ld(oD[s], Db, wave, s, NV);
      op_ld(oY[s], Yb, wave, s, NV);
    }
    float fk[4], fq[4], fe[4], fb[4], frq[4], frk[4];
    lds4(sc + kSk * kC + own4, fk);
    lds4(sc + kSq * kC + own4, fq);
    lds4(sc + kSe * kC + own4, fe);
    lds4(sc + kSb * kC + own4, fb);
    lds4(sc + kSrq * kC + own4, frq);
    lds4(sc + kSrk * kC + own4, frk);
    if (hh == 0) lds_dma_wait();
    __syncthreads();  // gate sums and b (and the token tiles) are in LDS

    // dbeta_i = <D_i, Y_i>
    {
      float x = 0.f;
#pragma unroll
      for (int s = 0; s < NV; ++s) x += op_dot(oD[s], oY[s]);
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      if (g == 0 && own < L) dbeta[(geo.t0 + own) * HV + hv] = from_f32<T>(x);
    }
    // 64 x 64 parts. As rows (contraction over j): W_ij = e_ij b_j rk_j / sqrt(K) dO_i.Y_j and
    // Z_ij = - e_ij b_i b_j rk_j D_i.Y_j, from the products with Y's rows on the left, so the
    // accumulators are the operand with the wave's tokens as rows. As columns (contraction
    // over i): W'_ij = e_ij b_j rq_i / sqrt(K) dO_i.Y_j, Z'_ij = - e_ij b_i b_j rk_i D_i.Y_j.
    Op8<T> wr[2], zr[2], wc[2], zc[2];
    const double Go = sG[own];
    const float bo = sB[own], rqo = sc[kSrq * kC + own], rko = sc[kSrk * kC + own];
    float xrow = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 w[2], z[2], w2[2], z2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = z[i] = w2[i] = z2[i] = zero4();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = perm_row(2 * s + i, l16), row4 = perm_row4(2 * s + i, g);
        f32x4 qk = zero4(), kk = zero4();
        if (s <= p) {
#pragma unroll
          for (int u = 0; u < K / 32; ++u) {
            Op8<T> kj, qi, ki;
            TT::rows(kj, sK, 2 * s + i, u);
            TT::rows(qi, sQ, wave, u);
            TT::rows(ki, sK, wave, u);
            qk = mma8(kj, qi, qk);
            kk = mma8(kj, ki, kk);
          }
        }
        if (s <= p) {
#pragma unroll
          for (int u = 0; u < NV; ++u) {
            Op8<T> y;
            op_ld(y, Yb, 2 * s + i, u, NV);
            w[i] = mma8(y, od[u], w[i]);
            z[i] = mma8(y, oD[u], z[i]);
          }
        }
        if (s >= p) {
#pragma unroll
          for (int u = 0; u < NV; ++u) {
            Op8<T> a, d;
            ld_op(a, dOb + (int64_t)min(row, L - 1) * HV * V + 32 * u + 8 * g);
            op_ld(d, Db, 2 * s + i, u, NV);
            w2[i] = mma8(a, oY[u], w2[i]);
            z2[i] = mma8(d, oY[u], z2[i]);
          }
        }
        float b4[4], rq_[4], rk_[4];
        lds4(sB + row4, b4);
        lds4(sc + kSrq * kC + row4, rq_);
        lds4(sc + kSrk * kC + row4, rk_);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int o = row4 + e;  // the other token: j of w, z; i of w2, z2
          const double d = Go - sG[o];
          const float ej = own >= o && own < L ? ex2((float)d) * b4[e] * rk_[e] : 0.f;
          const float ei = o >= own && o < L ? ex2((float)-d) * bo : 0.f;
          w[i][e] *= ej * scale;
          z[i][e] = own > o ? -z[i][e] * ej * bo : 0.f;
          w2[i][e] *= ei * rq_[e] * scale;
          z2[i][e] = o > own ? -z2[i][e] * ei * b4[e] * rk_[e] : 0.f;
          const float x = own > o ? w[i][e] * rqo * qk[e] + z[i][e] * rko * kk[e] : 0.f;
          xrow += x;
          const float xc = row16_sum(x);
          if (l16 == 0) sXc[wave][o] = xc;
        }
      }
      make_op(wr[s], w[0], w[1]);
      make_op(zr[s], z[0], z[1]);
      make_op(wc[s], w2[0], w2[1]);
      make_op(zc[s], z2[0], z2[1]);
    }
    xrow += __shfl_xor(xrow, 16);
    xrow += __shfl_xor(xrow, 32);
    if (g == 0) sX[own] = xrow;
    // channel tiles
    float rr[4] = {0.f, 0.f, 0.f, 0.f}, cc[4] = {0.f, 0.f, 0.f, 0.f}, sds = 0.f;
    const T* S0b = ws_S0 + ch * K * V;
    const T* dSb = ws_dS + ch * K * V;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      f32x4 a1 = zero4(), a2 = zero4(), a3 = zero4();
#pragma unroll
      for (int s = 0; s < NV; ++s) {
        Op8<T> s0, ds;
        op_ld(s0, S0b, r, s, NV);
        op_ld(ds, dSb, r, s, NV);
        a1 = mma8(od[s], s0, a1);
        a2 = mma8(oD[s], s0, a2);
        a3 = mma8(oY[s], ds, a3);
        if ((r & 3) == wave) sds += op_dot(s0, ds);
      }
      f32x4 tq = zero4(), tr = zero4(), tc = zero4();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Op8<T> kc, qc;
        TT::cols(kc, sK, r, s);
        TT::cols(qc, sQ, r, s);
        if (s <= p) {
          tq = mma8(wr[s], kc, tq);
          tr = mma8(zr[s], kc, tr);
        }
        if (s >= p) {
          tc = mma8(wc[s], qc, tc);
          tc = mma8(zc[s], kc, tc);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // fq = e^G rq / sqrt(K), fk = e^G rk, fe = e^{G_last - G} rk: gradients of the
        // normalised rows, times their own inverse norm
        aq[r][e] += a1[e] * fq[e] + frq[e] * tq[e];
        ak[r][e] += (a3[e] * fe[e] - a2[e] * fk[e]) * fb[e] + frk[e] * (tr[e] + tc[e]);
      }
      const f32x4 qt = TT::tile(sQ, wave, r), kt = TT::tile(sK, wave, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rr[e] += qt[e] * a1[e] * fq[e] - kt[e] * a2[e] * fk[e] * fb[e];
        cc[e] += kt[e] * a3[e] * fe[e] * fb[e];
      }
      __builtin_amdgcn_sched_barrier(0);  // one tile's operands live at a time
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rr[e] = row16_sum(rr[e]);
      cc[e] = row16_sum(cc[e]);
    }
    sds = row16_sum(sds);
    sds += __shfl_xor(sds, 16);
    sds += __shfl_xor(sds, 32);
    if (l16 == 0) {
      *reinterpret_cast<float4*>(sR + own4) = make_float4(rr[0], rr[1], rr[2], rr[3]);
      *reinterpret_cast<float4*>(sC + own4) = make_float4(cc[0], cc[1], cc[2], cc[3]);
    }
    if (lane == 0) sS[wave] = sds;
    __syncthreads();
    if (wave == 0) {
      const bool ok = lane < L;
      float dg = 0.f;
      float r = 0.f, c = 0.f;
      if (ok) {
        r = sR[lane] + (sX[lane] - ((sXc[0][lane] + sXc[1][lane]) + (sXc[2][lane] + sXc[3][lane])));
        c = sC[lane];
      }
      const float c_own = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const float x = __shfl_down(r, d), y = __shfl_up(c, d);
        if (lane + d < 64) r += x;
        if (lane >= d) c += y;
      }
      dg = r + (c - c_own) + sc[kSl * kC] * ((sS[0] + sS[1]) + (sS[2] + sS[3]));
      // before a sequence's first token there is nothing to decay without a state
      if (geo.c == 0 && lane == 0 && !has_h0) dg = 0.f;
      float pa = 0.f, pb = 0.f;
      if (ok) {
        const int64_t at = (geo.t0 + lane) * HV + hv;
        float xb, as;
        const float gn = gdn_gate(gate, at, hv, &xb, &as);
        const float dx = gate.raw ? -dg * as * sigmoid_f32(xb) : dg;
        st_any(dgate, at, gate.bf, dx);
        pa = dg * gn;  // dg / dA_log = g
        pb = dx;
      }
      if (gate.A_log || gate.dt_bias) {
#pragma unroll
        for (int d = 32; d; d >>= 1) {
          pa += __shfl_xor(pa, d);
          pb += __shfl_xor(pb, d);
        }
        if (lane == 0) {
          par[2 * ch] = pa;
          par[2 * ch + 1] = pb;
        }
      }
    }
    if (hh == 0) {
      rq4 = f32x4{frq[0], frq[1], frq[2], frq[3]};
      rk4 = f32x4{frk[0], frk[1], frk[2], frk[3]};
    }
    __syncthreads();  // sG and sB are rewritten for the next value head
  }

  // through the L2 norm: q^ = rq q, so dq = rq (dq^ - q^ <q^, dq^>); aq holds rq dq^
  if (l2) {
    float nq[4] = {0.f, 0.f, 0.f, 0.f}, nk[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const f32x4 qt = TT::tile(sQ, wave, r), kt = TT::tile(sK, wave, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        nq[e] = fmaf(qt[e], aq[r][e], nq[e]);
        nk[e] = fmaf(kt[e], ak[r][e], nk[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      nq[e] = row16_sum(nq[e]) * rq4[e] * rq4[e];
      nk[e] = row16_sum(nk[e]) * rk4[e] * rk4[e];
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const f32x4 qt = TT::tile(sQ, wave, r), kt = TT::tile(sK, wave, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        aq[r][e] = fmaf(-qt[e], nq[e], aq[r][e]);
        ak[r][e] = fmaf(-kt[e], nk[e], ak[r][e]);
      }
    }
  }
  const int64_t out = (geo.t0 * H + h) * K;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int col = perm_row(r, l16);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (own4 + e < L) {
        dq[out + (int64_t)(own4 + e) * H * K + col] = aq[r][e];
        dk[out + (int64_t)(own4 + e) * H * K + col] = ak[r][e];
      }
  }
}

// dA_log[hv], d_dt_bias[hv]: the chunks' partial sums in a fixed order, in double
__global__ void __launch_bounds__(256)
gdn_par_kernel(const float* __restrict__ par, const int* __restrict__ table, int chunks, int HV, int bf,
               void* dA, void* db) {
  __shared__ double s[2][256];
  const int hv = blockIdx.x, n = table ? table[0] : chunks;
  double a = 0., b = 0.;
  for (int c = threadIdx.x; c < n; c += 256) {
    const float2 x = reinterpret_cast<const float2*>(par)[(size_t)c * HV + hv];
    a += x.x;
    b += x.y;
  }
  s[0][threadIdx.x] = a;
  s[1][threadIdx.x] = b;
  __syncthreads();
  for (int d = 128; d; d >>= 1) {
    if (threadIdx.x < d) {
      s[0][threadIdx.x] += s[0][threadIdx.x + d];
      s[1][threadIdx.x] += s[1][threadIdx.x + d];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    if (dA) st_any(dA, hv, bf, (float)s[0][0]);
    if (db) st_any(db, hv, bf, (float)s[1][0]);
  }
}

template <int K, int V, int NP>
static hipError_t rev_t(const kda_dims& d, const void* q, const void* k, const void* v, const void* dO,
                        const float* dht, const int32_t* cu, const GdnLayout<bf16>& w, void* dv, float* dh0,
                        hipStream_t s) {
  constexpr size_t lds = GdnRevLds<K, NP>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gdn_rev_scan_kernel<K, V, NP>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdn_rev_scan_kernel<K, V, NP>), dim3(scan_grid((int64_t)d.N * d.HV, V, 16 * NP)),
                     dim3(256 * NP), lds, s, (const bf16*)q, (const bf16*)k, (const bf16*)v, (const bf16*)dO, dht,
                     cu, w.table, d.N, d.T, d.H, d.HV, w.scal, w.fragT, (bf16*)dv, dh0, w.dS, w.D, w.tokr, w.ancS, w.anc, w.Y,
                     w.Yl, w.tokb);
  return hipGetLastError();
}
template <int K, int V, int NP>
static hipError_t rev_t(const kda_dims& d, const void* q, const void* k, const void* v, const void* dO,
                        const float* dht, const int32_t* cu, const GdnLayout<float>& w, void* dv, float* dh0,
                        hipStream_t s) {
  constexpr size_t lds = GdnRev32Lds<K>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gdn_rev_scan32_kernel<K, V, NP>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdn_rev_scan32_kernel<K, V, NP>), dim3(scan_grid((int64_t)d.N * d.HV, V, 16 * NP)),
                     dim3(64 * NP), lds, s, (const float*)q, (const float*)k, (const float*)dO, dht, cu, w.table,
                     d.N, d.T, d.H, d.HV, w.scal, w.fragT, (float*)dv, dh0, w.dS, w.D);
  return hipGetLastError();
}

template <int K, int V>
static hipError_t local_t(const kda_dims& d, const void* q, const void* k, const void* dO, const GdnGate& gate, int l2,
                          int has_h0, int has_dht, const int32_t* cu, const GdnLayout<bf16>& w, void* dq, void* dk,
                          void* dbeta, void* dgate, hipStream_t s) {
  const int64_t mc = max_chunks(d, cu != nullptr);
  const int64_t chains = (int64_t)d.N * d.HV, segs = (cu ? mc : mc / d.N) / kGdnAnchor + 1;
  const int64_t ny = std::min<int64_t>(segs, std::max<int64_t>(1, 4 * kda_host::device_cus() / chains));
  hipLaunchKernelGGL((gdn_gate_bwd_kernel<V>), dim3((unsigned)chains, (unsigned)ny), dim3(64 * kGdnAnchor), 0, s, gate,
                     cu, w.table, d.T, d.HV, has_h0, has_dht, w.tokf, w.tokr, w.tokb, w.end, w.anc, dgate,
                     (bf16*)dbeta, w.par, w.scal);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr size_t lds = GdnLocalLds<K, V>::total;
  static_assert(lds <= 160 * 1024, "LDS");
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gdn_local_kernel<K, V>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const int64_t wgs = std::min<int64_t>(mc * d.H, kda_host::device_cus());
  hipLaunchKernelGGL((gdn_local_kernel<K, V>), dim3((unsigned)wgs), dim3(512), lds, s, (const bf16*)q, (const bf16*)k,
                     (const bf16*)dO, cu, w.table, (int)mc, d.N, d.T, d.H, d.HV, l2, 1.0f / sqrtf((float)K), w.scal,
                     w.S0, w.Y, w.dS, w.D, (bf16*)dq, (bf16*)dk);
  return hipGetLastError();
}
template <int K, int V>
static hipError_t local_t(const kda_dims& d, const void* q, const void* k, const void* dO, const GdnGate& gate, int l2,
                          int has_h0, int, const int32_t* cu, const GdnLayout<float>& w, void* dq, void* dk,
                          void* dbeta, void* dgate, hipStream_t s) {
  constexpr size_t lds = 2 * TokTile<float, K>::bytes;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gdn_local32_kernel<K, V>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdn_local32_kernel<K, V>), dim3((unsigned)(max_chunks(d, cu != nullptr) * d.H)), dim3(256), lds,
                     s, (const float*)q, (const float*)k, (const float*)dO, gate, cu, w.table, d.N, d.T, d.H, d.HV, l2,
                     has_h0, 1.0f / sqrtf((float)K), w.scal, w.S0, w.Y, w.dS, w.D, (float*)dq, (float*)dk,
                     (float*)dbeta, dgate, w.par);
  return hipGetLastError();
}

template <typename T, int K, int V>
static hipError_t gdn_bwd_kv(const kda_dims& d, const void* q, const void* k, const void* v, const GdnGate& gate, int l2,
                             const float* h0, const int32_t* cu, const void* dO, const float* dht, void* dq,
                             void* dk, void* dv, void* dgate, void* dbeta, float* dh0, void* dA,
                             void* ddt, void* ws, hipStream_t s) {
  const int64_t mc = max_chunks(d, cu != nullptr);
  const GdnLayout<T> w(d, cu != nullptr, ws, true);
  hipError_t e = hipSuccess;
  if (d.N > 0) e = rev_t<K, V, 2>(d, q, k, v, dO, dht, cu, w, dv, dh0, s);
  if (e != hipSuccess) return e;
  if (d.N > 0 && mc > 0) {
    e = local_t<K, V>(d, q, k, dO, gate, l2, h0 != nullptr, dht != nullptr, cu, w, dq, dk, dbeta, dgate, s);
    if (e != hipSuccess) return e;
  }
  if (dA || ddt) {
    hipLaunchKernelGGL(gdn_par_kernel, dim3((unsigned)d.HV), dim3(256), 0, s, w.par,
                       cu && d.N > 0 ? w.table : (const int*)nullptr, d.N > 0 ? (int)mc : 0, d.HV, gate.bf, dA,
                       ddt);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace kda

namespace kda_host {

hipError_t launch_gdn_bwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                          const kda::GdnGate& gate, int l2, const float* h0, const int32_t* cu, const void* dO,
                          const float* dht, void* dq, void* dk, void* dv,
                          void* dgate, void* dbeta, float* dh0, void* dA, void* ddt, void* ws,
                          hipStream_t s) {
#define KDA_GDN_BWD(T_, K_, V_) \
  if (d.K == K_ && d.V == V_)   \
    return kda::gdn_bwd_kv<T_, K_, V_>(d, q, k, v, gate, l2, h0, cu, dO, dht, dq, dk, dv, dgate, dbeta, dh0, dA, ddt, ws, s);
#define KDA_GDN_BWD_ALL(T_)    \
  KDA_GDN_BWD(T_, 64, 64)      \
  KDA_GDN_BWD(T_, 64, 128)     \
  KDA_GDN_BWD(T_, 128, 64)     \
  KDA_GDN_BWD(T_, 128, 128)
  if (dt == KDA_BF16) {
    KDA_GDN_BWD_ALL(kda::bf16)
  } else {
    KDA_GDN_BWD_ALL(float)
  }
#undef KDA_GDN_BWD_ALL
#undef KDA_GDN_BWD
  return hipErrorInvalidValue;
}

}  // namespace kda_host
