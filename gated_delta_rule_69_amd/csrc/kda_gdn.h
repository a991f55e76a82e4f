#pragma once
// The gated delta rule with one decay per value head and token (scalar gate):
// shared layouts and device helpers of its chunked kernels (gfx950).
//
// Per value head, with the FP32 state S [K, V] and natural-log gate g_t,
//   S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  o_t = S_t^T q~_t,
// q~ = q / sqrt(K). For a chunk of C = 64 tokens with start state S0, inclusive
// gate sum G and e_ij = e^{G_i - G_j}:
//   Abar_ij = (k_i . k_j) e_ij  (i > j),      P_ij = (q~_i . k_j) e_ij  (i >= j)
//   M = (I + Abar diag(b))^-1 Abar            (strictly lower triangular)
//   R = V - e^G K S0,   Y = R - M (b R),      Delta = b Y
//   O = e^G (q~ S0) + P Delta,                S1 = e^{G_last} S0 + K^T (e^{G_last - G} Delta)
// (Y = (I + Abar diag b)^-1 R written with M, so a zero b_t needs no division.)
// Backward, from dS at the chunk's end:
//   dDelta = P^T dO + e^{G_last - G} (K dS),  D = dDelta - M^T (b dDelta),  dV = E = b D
//   dS0 = e^{G_last} dS + (e^G q~)^T dO - (e^G K)^T E
// The gate's gradient (bf16 inputs; FP32's way is in kda_gdn_chunk_bwd.hip): scale
// every state from token t on, and v_i and o_i for i >= t with it; nothing
// changes but the decay into t. So dg_t = <S_T, dS_T> + sum_{t <= i < T} s_i for
// any T > t with s_i = <o_i, dO_i> - <v_i, dv_i>, two scalars per
// token that the scans form in FP32. What a token adds to its own output is in
// both and is left out of both, so that every term carries the decay (and a
// strongly decaying head's small dg keeps its digits):
//   s_i = <dO_i, o'_i - P_ii b_i (v_i - Y_i)> - b_i <v_i, D'_i>,
//   o'_i = o_i - P_ii Delta_i,  D'_i = D_i - P_ii dO_i.
// A decay that is one number per row and column never enters the products: k
// and q go to the matrix cores as they are in memory (exact), the decays and
// the optional L2 norms are row factors applied to the FP32 results. That is
// what this form saves against a per-channel gate, whose decays have to be
// multiplied into the operands.
//
// Rounding. q, k, v, dO enter exactly. In bf16, a computed operand x of a
// product that feeds the state is carried as hi + lo, hi = bf16(x), lo =
// bf16(x - hi): 2 (one split operand) or 3 (two) matrix-core steps leave a
// relative error near 2^-17, so states and state gradients keep FP32 quality
// through any number of chunks. What feeds only a bf16 output takes hi alone.
#include "kda_chunk_kernels.h"

namespace kda {

// ------------------------------------------------------------------ index maps
// Row r (0..15) of 16-row tile t stands for index 32 (t / 2) + 8 (r / 4) + 4 (t % 2)
// + r % 4 (tokens and channels alike). An accumulator lane (column l16, rows
// 4g .. 4g+3) of tiles 2s and 2s+1 then holds the eight consecutive indices
// 32s + 8g .. +7 of its column, which is what the lane feeds as the operand of
// the next product's contraction block s: results chain from product to
// product in registers, and the other operand is one 16-byte read of eight
// consecutive elements.
__device__ __forceinline__ int perm_row(int t, int r) {
  return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3);
}
// first of the four consecutive indices an accumulator lane holds
__device__ __forceinline__ int perm_row4(int t, int g) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); }

// Fragments of the 64 x 64 lower-triangular M and P (rows i, contraction over
// j in blocks s of 32): tiles 0 and 1 need s = 0 only. Transposed (rows j,
// contraction over i): tiles 2 and 3 need s = 1 only. Six of eight either way.
__host__ __device__ constexpr int frag_low(int t, int s) { return t < 2 ? t : 2 * t - 2 + s; }
__host__ __device__ constexpr int frag_up(int t, int s) { return t < 2 ? 2 * t + s : t + 2; }
constexpr int kFragElems = 64 * 8;          // one fragment: [lane][8]
constexpr int kTriElems = 6 * kFragElems;   // one triangular matrix

// Row factors of a (chunk, value head), FP32 [kGdnScal][64], ordered so that what one
// reader takes is consecutive:
enum GdnScal : int {
  kSk = 0,   // e^G rk                 (rk, rq: 1, or the inverse L2 norms of k and q rows)
  kSeb = 1,  // e^{G_last - G} rk b
  kSpy = 1,  // bf16 backward, behind the scans: <dO_i, Y_i>
  kSl = 2,   // e^{G_last}, 64 times
  kSb = 3,   // b
  kSq = 4,   // e^G rq / sqrt(K)
  kSp = 5,   // from here on for the backward only: P_ii
  kSG = 6,   // G log2(e) as 64 doubles (two slots)
  kSe = 8,   // e^{G_last - G} rk
  kSrq = 9,  // rq
  kSrk = 10,  // rk
  kSpd = 11,  // P_ii again
  kGdnScal = 12  // (whole KB)
};

template <typename T>
struct GdnWs {
  static constexpr bool kScanGate = sizeof(T) == 2;  // dg from the scans' scalars
  static constexpr int kParts = sizeof(T) == 2 ? 2 : 1;  // hi + lo, or FP32
  // forward: M (kParts), P; backward: M, P, M^T, P^T (kParts each), P without its diagonal
  static constexpr size_t fwd = (size_t)kTriElems * (kParts + 1);
  static constexpr size_t bwd = (size_t)kTriElems * (2 * kParts);  // one of its two pairs
};

// ------------------------------------------------------------------ operands
// Eight consecutive contraction elements per lane: one bf16 fragment (one
// 16x16x32 step), or eight FP32 values (eight 16x16x4 steps, lane group g
// carrying element i of its eight in step i).
template <typename T>
struct Op8;
template <>
struct Op8<bf16> {
  bf16x8 v;
};
template <>
struct Op8<float> {
  float v[8];
};
// a computed operand: hi + lo for bf16
template <typename T>
struct Op8s;
template <>
struct Op8s<bf16> {
  bf16x8 hi, lo;
};
template <>
struct Op8s<float> {
  float v[8];
};

__device__ __forceinline__ f32x4 mma8(const Op8<bf16>& a, const Op8<bf16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma8(const Op8<float>& a, const Op8<float>& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}
// c + a b, b split
__device__ __forceinline__ f32x4 mma8s(const Op8<bf16>& a, const Op8s<bf16>& b, f32x4 c) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.lo, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.hi, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma8s(const Op8<float>& a, const Op8s<float>& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}
// c + a b with b's high part alone
__device__ __forceinline__ f32x4 mma8h(const Op8<bf16>& a, const Op8s<bf16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.hi, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma8h(const Op8<float>& a, const Op8s<float>& b, f32x4 c) {
  return mma8s(a, b, c);
}

// Nothing is scheduled across: reads placed before it stay before it.
__device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }
// c[t] += a[t] b for four row tiles, b split: low parts first, so that the
// four tiles' steps lie between two steps of one tile
__device__ __forceinline__ void mma_rows(const Op8<bf16> (&a)[4], const Op8s<bf16>& b, f32x4 (&c)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t].v, b.lo, c[t], 0, 0, 0);
#pragma unroll
  for (int t = 0; t < 4; ++t) c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t].v, b.hi, c[t], 0, 0, 0);
}
// c += X b with the triangular X's six fragments (frag_low order; PT parts:
// hi, then lo, whose product with b's low part is left out) and b split
template <int PT, int PX>
__device__ __forceinline__ void mma_tri(const Op8<bf16> (&a)[PX][6], const Op8s<bf16> (&b)[2], f32x4 (&c)[4]) {
  static_assert(PT <= PX, "parts");
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int t = 2 * s; t < 4; ++t)
      c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0][frag_low(t, s)].v, b[s].lo, c[t], 0, 0, 0);
    if constexpr (PT == 2) {
#pragma unroll
      for (int t = 2 * s; t < 4; ++t)
        c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[1][frag_low(t, s)].v, b[s].hi, c[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 2 * s; t < 4; ++t)
      c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0][frag_low(t, s)].v, b[s].hi, c[t], 0, 0, 0);
  }
}
// two floats as bf16 in one register (first in the low half), and their rest
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 h = {(bf16)a, (bf16)b};
  return __builtin_bit_cast(uint32_t, h);
}
// a - hi.low and b - hi.high (both exact), each in one two-term bf16 dot
// product with (-1, 0) or (0, -1). Those two sit in registers: as literals the
// compiler encodes the first like the second.
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t hi) {
  const bf16x2 h = __builtin_bit_cast(bf16x2, hi);
  uint32_t c0 = 0x0000BF80u, c1 = 0xBF800000u;
  asm("" : "+v"(c0));
  asm("" : "+v"(c1));
  return pack2(__builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, c0), a, false),
               __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, c1), b, false));
}
// two accumulator tiles (2s, 2s + 1) as the operand of contraction block s
__device__ __forceinline__ void make_op(Op8s<bf16>& o, const f32x4& t0, const f32x4& t1) {
  uint4 h, l;
  h.x = pack2(t0[0], t0[1]); h.y = pack2(t0[2], t0[3]);
  h.z = pack2(t1[0], t1[1]); h.w = pack2(t1[2], t1[3]);
  l.x = pack2_rest(t0[0], t0[1], h.x); l.y = pack2_rest(t0[2], t0[3], h.y);
  l.z = pack2_rest(t1[0], t1[1], h.z); l.w = pack2_rest(t1[2], t1[3], h.w);
  o.hi = __builtin_bit_cast(bf16x8, h);
  o.lo = __builtin_bit_cast(bf16x8, l);
}
__device__ __forceinline__ void make_op(Op8s<float>& o, const f32x4& t0, const f32x4& t1) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o.v[e] = t0[e];
    o.v[4 + e] = t1[e];
  }
}
__device__ __forceinline__ void make_op(Op8<bf16>& o, const f32x4& t0, const f32x4& t1) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o.v[e] = (bf16)t0[e];
    o.v[4 + e] = (bf16)t1[e];
  }
}
__device__ __forceinline__ void make_op(Op8<float>& o, const f32x4& t0, const f32x4& t1) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o.v[e] = t0[e];
    o.v[4 + e] = t1[e];
  }
}

// eight consecutive elements from 16-byte aligned memory
__device__ __forceinline__ void ld_op(Op8<bf16>& o, const bf16* p) {
  o.v = *reinterpret_cast<const bf16x8*>(p);
}
__device__ __forceinline__ void ld_op(Op8<float>& o, const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  o.v[0] = a.x; o.v[1] = a.y; o.v[2] = a.z; o.v[3] = a.w;
  o.v[4] = b.x; o.v[5] = b.y; o.v[6] = b.z; o.v[7] = b.w;
}
__device__ __forceinline__ float op_get(const Op8<bf16>& o, int i) { return (float)o.v[i]; }
__device__ __forceinline__ float op_get(const Op8<float>& o, int i) { return o.v[i]; }

// ------------------------------------------------------------------ 4 x 4 transposes
// Within each quad of lanes: lane a holds x[a][0..3] as four bf16 in two
// registers; afterwards it holds x[0..3][a]. Its own inverse. It turns the
// accumulator's four rows of one column into four columns of one row (one
// 8-byte access in place of four 2-byte ones), and back.
__device__ __forceinline__ uint2 quad_transpose(uint2 r) {
  const int lane = threadIdx.x & 63;
  const uint32_t t0 = __builtin_amdgcn_update_dpp(0, (int)r.x, 0xB1, 0xF, 0xF, true);  // lane ^ 1
  const uint32_t t1 = __builtin_amdgcn_update_dpp(0, (int)r.y, 0xB1, 0xF, 0xF, true);
  const uint32_t sel = (lane & 1) ? 0x03020706u : 0x05040100u;
  const uint32_t a0 = __builtin_amdgcn_perm(t0, r.x, sel), a1 = __builtin_amdgcn_perm(t1, r.y, sel);
  const uint32_t u0 = __builtin_amdgcn_update_dpp(0, (int)a0, 0x4E, 0xF, 0xF, true);  // lane ^ 2
  const uint32_t u1 = __builtin_amdgcn_update_dpp(0, (int)a1, 0x4E, 0xF, 0xF, true);
  return (lane & 2) ? make_uint2(u1, a1) : make_uint2(a0, u0);
}
__device__ __forceinline__ uint2 pack4(const f32x4& x) {
  return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}
__device__ __forceinline__ f32x4 unpack4(uint2 r) {
  return f32x4{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
               __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u)};
}

// A 16 x 16 tile between row-major memory and the accumulator layout. `row4`
// is the lane's first row (perm_row4), rows row4 .. row4 + 3, column col0 + l16;
// element (r, c) at p + r * stride + c. Rows from `rows` on are not written; as
// loads they repeat the last row (unconditional loads: under a lane-dependent
// branch each would be waited for at the branch's join), and what they feed is
// multiplied by row factors that are zero there. bf16: p 8-byte aligned, stride
// and col0 multiples of 4. p is uniform in the wave and 64 rows span less than
// 2^31 bytes (checked by the entry points), so a lane's address is a scalar
// base and a 32-bit offset.
template <typename T>
struct TileRaw;
template <>
struct TileRaw<bf16> {
  uint2 r;
};
template <>
struct TileRaw<float> {
  f32x4 r;
};
__device__ __forceinline__ void tile_ld(TileRaw<bf16>& t, const bf16* p, uint32_t stride, int row4,
                                        int col0, int rows) {
  const int l16 = threadIdx.x & 15, row = min(row4 + (l16 & 3), rows - 1);
  t.r = *reinterpret_cast<const uint2*>(p + (row * stride + col0 + 4 * (l16 >> 2)));
}
__device__ __forceinline__ void tile_ld(TileRaw<float>& t, const float* p, uint32_t stride, int row4,
                                        int col0, int rows) {
  const int l16 = threadIdx.x & 15;
#pragma unroll
  for (int e = 0; e < 4; ++e) t.r[e] = p[(uint32_t)(min(row4 + e, rows - 1) * stride + col0 + l16)];
}
__device__ __forceinline__ f32x4 tile_get(const TileRaw<bf16>& t) { return unpack4(quad_transpose(t.r)); }
__device__ __forceinline__ f32x4 tile_get(const TileRaw<float>& t) { return t.r; }
// two tiles (2s, 2s + 1) straight as the operand of contraction block s
__device__ __forceinline__ void tile_op(Op8<bf16>& o, const TileRaw<bf16>& t0, const TileRaw<bf16>& t1) {
  const uint2 a = quad_transpose(t0.r), b = quad_transpose(t1.r);
  o.v = __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
__device__ __forceinline__ void tile_op(Op8<float>& o, const TileRaw<float>& t0, const TileRaw<float>& t1) {
  make_op(o, t0.r, t1.r);
}
__device__ __forceinline__ void tile_st(bf16* p, uint32_t stride, int row4, int col0, int rows, const f32x4& x) {
  const int l16 = threadIdx.x & 15, row = row4 + (l16 & 3);
  const uint2 r = quad_transpose(pack4(x));
  if (row < rows) *reinterpret_cast<uint2*>(p + (row * stride + col0 + 4 * (l16 >> 2))) = r;
}
__device__ __forceinline__ void tile_st(float* p, uint32_t stride, int row4, int col0, int rows, const f32x4& x) {
  const int l16 = threadIdx.x & 15;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (row4 + e < rows) p[(uint32_t)((row4 + e) * stride + col0 + l16)] = x[e];
}

// A 16 x 16 tile (rows of tile r, columns 16 cb .. + 15 of a width of 32 NV)
// into memory in operand order: [r][block s of 32 columns][lane][8], so that a
// later kernel's lane reads its eight column elements of row l16 as one 16-byte
// piece and a wave 1 KB in one go, with rows or columns as the product's rows
// alike. The bf16 tile is 512 consecutive bytes. (Row by row, 32 bytes per row
// and wave, the kernels of that time took 362 us against 305, local, and 374
// against 365, reverse scan.)
__device__ __forceinline__ uint32_t op_at() {  // a lane's four elements within a bf16 tile
  const int lane = threadIdx.x & 63, g = lane >> 4, Q = (lane >> 2) & 3, q = lane & 3;
  return ((Q >> 1) * 16 + 4 * g + q) * 8 + 4 * (Q & 1);
}
__device__ __forceinline__ void op_st(bf16* p, int r, int cb, int nv, uint2 x) {  // x: packed accumulator
  *reinterpret_cast<uint2*>(p + (r * nv + (cb >> 1)) * kFragElems + (cb & 1) * (kFragElems / 2) + op_at()) =
      quad_transpose(x);
}
// a tile as op_st wrote it (quad_transpose gives the packed accumulator)
__device__ __forceinline__ uint2 op_tile_ld(const bf16* p, int r, int cb, int nv) {
  return *reinterpret_cast<const uint2*>(p + (r * nv + (cb >> 1)) * kFragElems + (cb & 1) * (kFragElems / 2) + op_at());
}
__device__ __forceinline__ void op_st(float* p, int r, int cb, int nv, const f32x4& x) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  float* d = p + (r * nv + (cb >> 1)) * kFragElems;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    d[(uint32_t)(((2 * (cb & 1) + (l16 >> 3)) * 16 + 4 * g + e) * 8 + (l16 & 7))] = x[e];
}
template <typename T>
__device__ __forceinline__ void op_ld(Op8<T>& o, const T* p, int r, int s, int nv, int lane = threadIdx.x & 63) {
  ld_op(o, p + ((r * nv + s) * 64 + lane) * 8);
}

// sum over the 16 lanes that hold one accumulator row (rotations inside the
// row: no LDS), in every lane
template <int M>
__device__ __forceinline__ float add_ror(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + M,
                                                                   0xF, 0xF, true));
}
__device__ __forceinline__ float row16_sum(float x) {
  return add_ror<8>(add_ror<4>(add_ror<2>(add_ror<1>(x))));
}

// ------------------------------------------------------------------ token tiles in LDS
// A chunk's [64][K] rows of k or q, 16-byte blocks swizzled within each row:
// block b of row r sits at b ^ swz(r). Both read patterns (16 rows of one
// block column, as in a product over channels; four consecutive rows of four
// blocks, as in a product over tokens) then spread over the banks.
template <typename T, int K>
struct TokTile {
  static constexpr int kBlocks = K * (int)sizeof(T) / 16;  // 16-byte blocks per row
  static constexpr size_t bytes = (size_t)kC * K * sizeof(T);
  static constexpr int kUnits = kC * kBlocks;
  static __device__ __forceinline__ int swz(int r) {
    return kBlocks >= 16 ? ((r & 3) << 2) | ((r >> 3) & 3) : ((r & 3) << 1) | ((r >> 3) & 1);
  }
  static __device__ __forceinline__ int at(int r, int b) { return (r * kBlocks + (b ^ swz(r))) * 16; }
  // rows perm_row(t, l16), channels 32 s + 8 g .. + 7
  static __device__ __forceinline__ void rows(Op8<T>& o, const char* s, int t, int ks, int lane = threadIdx.x & 63) {
    const int g = lane >> 4, r = perm_row(t, lane & 15);
    if constexpr (sizeof(T) == 2) {
      o.v = *reinterpret_cast<const bf16x8*>(s + at(r, 4 * ks + g));
    } else {
      const float4 a = *reinterpret_cast<const float4*>(s + at(r, 8 * ks + 2 * g));
      const float4 b = *reinterpret_cast<const float4*>(s + at(r, 8 * ks + 2 * g + 1));
      o.v[0] = a.x; o.v[1] = a.y; o.v[2] = a.z; o.v[3] = a.w;
      o.v[4] = b.x; o.v[5] = b.y; o.v[6] = b.z; o.v[7] = b.w;
    }
  }
  // channels perm_row(t, l16), tokens 32 s + 8 g .. + 7 (the transposed read:
  // ds_read_b64_tr_b16 gives lane i of 16 column i of the four rows and four
  // 8-byte blocks the 16 lanes point at)
  static __device__ __forceinline__ void cols(Op8<T>& o, const char* s, int t, int ks, int lane = threadIdx.x & 63) {
    const int g = lane >> 4, l16 = lane & 15;
    if constexpr (sizeof(T) == 2) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const int b = 4 * (t >> 1) + (l16 & 3), r0 = 32 * ks + 8 * g + (l16 >> 2);
      const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(s + at(r0, b) + 8 * (t & 1)));
      const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(s + at(r0 + 4, b) + 8 * (t & 1)));
      const uint2 a = __builtin_bit_cast(uint2, x0), c = __builtin_bit_cast(uint2, x1);
      o.v = __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, c.x, c.y));
    } else {
      const int c = perm_row(t, l16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 32 * ks + 8 * g + i;
        o.v[i] = *reinterpret_cast<const float*>(s + at(r, c >> 2) + 4 * (c & 3));
      }
    }
  }
  // accumulator-layout tile: rows perm_row4(tt, g) + e, channel perm_row(ct, l16)
  static __device__ __forceinline__ f32x4 tile(const char* s, int tt, int ct, int lane = threadIdx.x & 63) {
    const int g = lane >> 4, l16 = lane & 15;
    if constexpr (sizeof(T) == 2) {
      const int r = perm_row4(tt, g) + (l16 & 3), b = 4 * (ct >> 1) + (l16 >> 2);
      const uint2 x = *reinterpret_cast<const uint2*>(s + at(r, b) + 8 * (ct & 1));
      return unpack4(quad_transpose(x));
    } else {
      const int c = perm_row(ct, l16);
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = *reinterpret_cast<const float*>(s + at(perm_row4(tt, g) + e, c >> 2) + 4 * (c & 3));
      return x;
    }
  }
};

// ------------------------------------------------------------------ global memory -> LDS
// One wave's 1 KB: lane i's 16 bytes at base + off go to LDS byte address
// dst + 16 i (base and dst uniform in the wave) without passing through
// registers. Complete after lds_dma_wait() (and, for other waves, a barrier
// behind it). Written out rather than through the builtin because the
// compiler, which cannot tell the two buffers apart, waits for every such
// transfer before the next LDS read of any kind: the prefetch of a chunk would
// end where the chunk before it begins to read. The instruction writes no
// register.
__device__ __forceinline__ void lds_dma(const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(dst)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// The same where the wave has issued at least N other vector memory accesses
// (stores) behind its last transfer: they complete in order, so the last N may
// still be under way.
template <int N>
__device__ __forceinline__ void lds_dma_wait_but() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// Makes the compiler wait for a loaded value here. It counts only the accesses
// it knows of: behind a transfer its wait would include part of that.
__device__ __forceinline__ void settle(const uint2& x) { asm volatile("" ::"v"(x.x), "v"(x.y)); }
__device__ __forceinline__ void settle(const float& x) { asm volatile("" ::"v"(x)); }
// byte address within LDS of a __shared__ object
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  typedef __attribute__((address_space(3))) const char lchar;
  return (uint32_t)(uintptr_t)(lchar*)p;
}

// A wave's share of the transfer of token tiles (chunk rows base + r * stride
// bytes): its 16-byte units' offsets, the same for every full chunk.
template <typename T, int K, int NW>
struct TokDma {
  using TT = TokTile<T, K>;
  static constexpr int kPer = TT::kUnits / (64 * NW);
  static_assert(TT::kUnits % (64 * NW) == 0, "whole waves");
  uint32_t off[kPer], stride;
  int wave;
  // rows past `last` repeat it (their factors are zero)
  __device__ __forceinline__ uint32_t unit(int n, int last, int lane = threadIdx.x & 63) const {
    const int u = 64 * (n * NW + wave) + lane, r = u / TT::kBlocks;
    return min(r, last) * stride + 16 * ((u % TT::kBlocks) ^ TT::swz(r));
  }
  __device__ __forceinline__ TokDma(uint32_t stride_bytes, int w) : stride(stride_bytes), wave(w) {
#pragma unroll
    for (int n = 0; n < kPer; ++n) off[n] = unit(n, kC - 1);
  }
  // the same with the offsets made on the spot, where registers are short
  __device__ __forceinline__ void go_lean(uint32_t dst, const T* base, int L, int lane) const {
#pragma unroll
    for (int n = 0; n < kPer; ++n) lds_dma(base, unit(n, L - 1, lane), dst + 1024 * (n * NW + wave));
  }
  __device__ __forceinline__ void go(uint32_t dst, const T* base, int L) const {
    if (L >= kC) {
#pragma unroll
      for (int n = 0; n < kPer; ++n) lds_dma(base, off[n], dst + 1024 * (n * NW + wave));
    } else {
#pragma unroll
      for (int n = 0; n < kPer; ++n) lds_dma(base, unit(n, L - 1), dst + 1024 * (n * NW + wave));
    }
  }
};
// `BYTES` (a multiple of 1 KB) of contiguous memory
template <int BYTES, int NW>
__device__ __forceinline__ void dma_flat(uint32_t dst, const void* src, int wave) {
  static_assert(BYTES % 1024 == 0, "whole waves");
  const uint32_t lane = threadIdx.x & 63;
#pragma unroll
  for (int n = 0; n < (BYTES / 1024 + NW - 1) / NW; ++n) {
    const int i = n * NW + wave;
    if (i >= BYTES / 1024) break;
    lds_dma(reinterpret_cast<const char*>(src) + 1024 * i, 16 * lane, dst + 1024 * i);
  }
}

// ------------------------------------------------------------------ chains
// What one workgroup of a scan works on: a chain (sequence, value head) and a
// block of columns. 1-D grid in groups of 8 chains x NVB column blocks: the
// blocks of a chain are 8 apart, so they run on one XCD and share its L2 for
// k, q, M and P. Packed batches take their sequences longest first.
struct GdnChain {
  int ok, n, hv, h, vb, len;
  int64_t bos, c0;  // first token; first chunk
};
__device__ __forceinline__ GdnChain gdn_chain(int nvb, const int32_t* cu, const int* table, int N, int T_,
                                              int H, int HV) {
  GdnChain r;
  const int grp = blockIdx.x / (8 * nvb), in = blockIdx.x % (8 * nvb);
  const int64_t chain = (int64_t)grp * 8 + in % 8;
  r.ok = chain < (int64_t)N * HV;
  if (!r.ok) return r;
  r.n = cu ? table[2 + N + (int)(chain / HV)] : (int)(chain / HV);
  r.hv = (int)(chain % HV);
  r.h = r.hv / (HV / H);
  r.vb = in / 8;
  seq_range(cu, r.n, T_, &r.bos, &r.len);
  r.c0 = cu ? table[1 + r.n] : (int64_t)r.n * ((T_ + kC - 1) / kC);
  return r;
}
// empty slot: bitwise passthrough of the state (or +0.0 without one), columns col0 .. + 15
__device__ __forceinline__ void gdn_pass(const float* h0, float* ht, size_t st, int K, int V, int col0) {
  for (int e = threadIdx.x & 63; e < K * 16; e += 64) {
    const size_t off = st + (size_t)(e >> 4) * V + col0 + (e & 15);
    reinterpret_cast<uint32_t*>(ht)[off] = h0 ? reinterpret_cast<const uint32_t*>(h0)[off] : 0u;
  }
}

// ------------------------------------------------------------------ gate
struct GdnGate {
  const void* x;        // [B, T, HV]
  const void* A_log;    // [HV] or null
  const void* dt_bias;  // [HV] or null
  int bf;               // all three are bf16 (else FP32)
  int raw;              // x is the raw input (else the natural-log gate)
};
__device__ __forceinline__ float ld_any(const void* p, int64_t i, int bf) {
  return bf ? (float)reinterpret_cast<const bf16*>(p)[i] : reinterpret_cast<const float*>(p)[i];
}
__device__ __forceinline__ void st_any(void* p, int64_t i, int bf, float x) {
  if (bf) reinterpret_cast<bf16*>(p)[i] = (bf16)x;
  else reinterpret_cast<float*>(p)[i] = x;
}
// natural-log gate of flat entry i (head hv); pre-activation in *xb
__device__ __forceinline__ float gdn_gate(const GdnGate& g, int64_t i, int hv, float* xb, float* scale) {
  const float x = ld_any(g.x, i, g.bf);
  if (!g.raw) {
    *xb = x;
    *scale = 1.f;
    return x;
  }
  const float a = g.A_log ? expf(ld_any(g.A_log, hv, g.bf)) : 1.f;
  const float y = g.dt_bias ? x + ld_any(g.dt_bias, hv, g.bf) : x;
  *xb = y;
  *scale = a;
  return -a * softplus_f32(y);
}

}  // namespace kda

namespace kda_host {
size_t gdn_workspace_bytes(const kda_dims& d, kda_dtype dt, int bwd);
hipError_t launch_gdn_fwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                          const kda::GdnGate& gate, int l2, const void* beta, const float* h0,
                          const int32_t* cu, int write_final, void* o, float* ht, void* ws,
                          hipStream_t s);
// the backward's own run over the forward: fragments, states, Y and <o, dO>
hipError_t launch_gdn_refwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                            const kda::GdnGate& gate, int l2, const void* beta, const float* h0,
                            const int32_t* cu, const void* dO, const float* dht, void* ws,
                            hipStream_t s);
hipError_t launch_gdn_bwd(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                          const kda::GdnGate& gate, int l2, const float* h0, const int32_t* cu,
                          const void* dO, const float* dht, void* dq, void* dk, void* dv, void* dgate,
                          void* dbeta, float* dh0, void* dA_log, void* d_dt_bias, void* ws,
                          hipStream_t s);
hipError_t launch_gdn_recurrent(const kda_dims& d, kda_dtype dt, const void* q, const void* k,
                                const void* v, const kda::GdnGate& gate, int l2, const void* beta,
                                const float* h0, const int32_t* cu, int write_final, void* o,
                                float* ht, hipStream_t s);
}  // namespace kda_host

namespace kda {
// Workspace of a chunked call, in order: the varlen chunk table, then per
// (chunk, value head): row factors and fragments, and for the backward S0, Y,
// dS, D, the per-token scalars of each 16 columns and the gate-parameter partials.
constexpr int kGdnAnchor = 8;  // chunks between a sequence's anchors of the gate's gradient
// A chunk c of a sequence that starts at flat chunk c0 and has an anchor: its
// slot (anchors are kGdnAnchor chunks apart and a sequence's first chunk has none, so
// no two share one).
__host__ __device__ __forceinline__ size_t gdn_anchor(int64_t c0, int c) { return (size_t)((c0 + c) / kGdnAnchor); }
template <typename T>
struct GdnLayout {
  int* table;
  float* scal;   // [chunk * HV + hv][kGdnScal][64]
  T* frag;       // [..][GdnWs<T>::fwd], or for the backward [..][GdnWs<T>::bwd]: M, P
  T* fragT;      // [..][GdnWs<T>::bwd]: M^T, P^T
  T* S0;         // [..][K][V] in operand order (op_st), as the next three
  T* Y;          // [..][64][V]
  T* dS;         // [..][K][V]
  T* D;          // [..][64][V]
  T* Yl;         // bf16: Y's low part, [..][V / 16][4][64][4] as the accumulators lie
  float* tokf;   // [..][V / 16][64]: the tokens' scalars from the forward run, per 16 columns
  float* tokr;   // [..][V / 16][64]: those from the reverse scan
  float* end;    // [N * HV][V / 16]: <S_T, dS_T> of the columns
  float* tokb;   // [..][2][V / 16][64]: <D, Y>, <dO, Y>
  float* anc;    // [anchors * HV][V / 16]: <S, dS> of the columns before an anchor chunk
  float* ancS;   // [anchors * HV][V / 16][K / 16][64][4]: S there in FP32, as the accumulators lie
  float* par;    // [..][2]
  size_t bytes;
  GdnLayout(const kda_dims& d, bool varlen, void* ws, bool bwd) {
    const int64_t mc = max_chunks(d, varlen);
    const size_t n = (size_t)mc * d.HV;
    char* p = reinterpret_cast<char*>(ws);
    auto take = [&](size_t b) {
      char* r = p;
      p += align256(b);
      return r;
    };
    char* p0 = p;
    table = reinterpret_cast<int*>(take(sizeof(int) * (size_t)(2 + 2 * (size_t)d.N + mc)));
    scal = reinterpret_cast<float*>(take(n * kGdnScal * kC * sizeof(float)));
    frag = reinterpret_cast<T*>(take(n * (bwd ? GdnWs<T>::bwd : GdnWs<T>::fwd) * sizeof(T)));
    fragT = S0 = Y = dS = D = Yl = nullptr;
    tokf = tokr = tokb = end = anc = ancS = par = nullptr;
    if (bwd) {
      fragT = reinterpret_cast<T*>(take(n * GdnWs<T>::bwd * sizeof(T)));
      S0 = reinterpret_cast<T*>(take(n * d.K * d.V * sizeof(T)));
      Y = reinterpret_cast<T*>(take(n * kC * d.V * sizeof(T)));
      dS = reinterpret_cast<T*>(take(n * d.K * d.V * sizeof(T)));
      D = reinterpret_cast<T*>(take(n * kC * d.V * sizeof(T)));
      tokf = reinterpret_cast<float*>(take(n * (d.V / 16) * kC * sizeof(float)));
      tokr = reinterpret_cast<float*>(take(n * (d.V / 16) * kC * sizeof(float)));
      end = reinterpret_cast<float*>(take((size_t)d.N * d.HV * (d.V / 16) * sizeof(float)));
      if (GdnWs<T>::kScanGate) {
        Yl = reinterpret_cast<T*>(take(n * kC * d.V * sizeof(T)));
        tokb = reinterpret_cast<float*>(take(2 * n * (d.V / 16) * kC * sizeof(float)));
        const size_t na = (size_t)(mc / kGdnAnchor + 1) * d.HV;
        anc = reinterpret_cast<float*>(take(na * (d.V / 16) * sizeof(float)));
        ancS = reinterpret_cast<float*>(take(na * d.K * d.V * sizeof(float)));
      }
      par = reinterpret_cast<float*>(take(n * 2 * sizeof(float)));
    }
    bytes = (size_t)(p - p0);
  }
};
}  // namespace kda
