// Output norm of a linear-attention layer, forward and backward: RMS or layer
// norm over rows of D, optional weight and bias, optional output gate.
//   mu = mean(x) (layer; 0 for RMS),  r = 1 / sqrt(mean((x - mu)^2) + eps),  n = (x - mu) r
//   a = n w + c,   y = a act(z)       (act = silu or sigmoid; y = a without a gate)
// Backward, f = act(z): da = dy f, dz = dy a act'(z), dw = sum da n, dc = sum da,
//   dn = da w,  dx = r (dn - mean(dn) [layer] - n mean(dn n))
//
// One pass: a row is read once into registers by a group of G lanes (16 lanes
// for a head's row, a wave, or a workgroup for a hidden row), normalised there
// in FP32 (the variance from the centred values, so a large mean costs no
// digits) and written once; the kernel is bound by those bytes. Groups walk
// the rows in a grid-sized stride with the weights held in registers (262144
// gated rows of 128, bf16: 36 us, 5.5 TB/s). The
// backward keeps its column sums dw, dc in registers over all the rows a group
// sees, adds the groups of a workgroup in LDS and writes one partial row per
// workgroup; a second kernel adds those in a fixed order (no atomics: results
// repeat bit for bit). 2M gated rows of 128: 515 + 6 us, 5.2 TB/s; 8191 rows of
// 4096 without a gate: 57 + 7 us, 3.5 TB/s.
#include "kda_gdn.h"
#include "kda_norm.h"

namespace kda {

struct NormArgs {
  const void *x, *w, *b, *z, *dy;
  void *y, *dx, *dz;
  float* part;  // [workgroups][2][D]
  int64_t rows;
  const int32_t* cu;
  int N, rpt;   // with cu: rows = cu[N] * rpt
  int D, wbf, layer, act;
  float eps;
};

// VEC elements as they lie in memory
template <typename T, int VEC>
using VecRaw = std::conditional_t<VEC == 1, T, uint4>;
template <typename T, int VEC>
__device__ __forceinline__ void vec_get(float* x, const VecRaw<T, VEC>& p) {
  if constexpr (VEC == 1) {
    x[0] = to_f32(p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = __builtin_bit_cast(float4, p);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  } else {
    const f32x4 lo = unpack4(make_uint2(p.x, p.y)), hi = unpack4(make_uint2(p.z, p.w));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = lo[e];
      x[4 + e] = hi[e];
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void vec_st(T* p, const float* x) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    const uint2 lo = pack4(f32x4{x[0], x[1], x[2], x[3]}), hi = pack4(f32x4{x[4], x[5], x[6], x[7]});
    *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// Sums of NS values over the G lanes of a row group, in every lane. G = 256
// goes through LDS; `s` alternates between two halves so that one barrier per
// call suffices.
template <int G, int NS>
__device__ __forceinline__ void group_sum(float (&x)[NS], float* s, int& flip) {
#pragma unroll
  for (int d = 1; d < (G < 64 ? G : 64); d <<= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] += __shfl_xor(x[i], d);
  if constexpr (G == 256) {
    float* p = s + 8 * flip;
    flip ^= 1;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) p[4 * i + wave] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] = (p[4 * i] + p[4 * i + 1]) + (p[4 * i + 2] + p[4 * i + 3]);
  }
}

// act(z) and its derivative
__device__ __forceinline__ void gate_act(int act, float z, float* f, float* df) {
  const float sg = __builtin_amdgcn_rcpf(1.f + ex2(-z * kLog2e));
  if (act == KDA_ACT_SILU) {
    *f = z * sg;
    *df = sg * fmaf(z, 1.f - sg, 1.f);
  } else {
    *f = sg;
    *df = sg * (1.f - sg);
  }
}

template <typename T, int VEC, int G, int NU, bool BWD>
__global__ void __launch_bounds__(256)
norm_kernel(NormArgs a) {
  constexpr int GPW = 256 / G, E = VEC * NU;  // groups per workgroup, elements per lane
  __shared__ float s_sum[16];
  const int gl = threadIdx.x % G, grp = threadIdx.x / G;
  const int D = a.D;
  const int64_t rows = a.cu ? (int64_t)a.cu[a.N] * a.rpt : a.rows;
  const float inv_d = 1.f / (float)D;
  int flip = 0;
  float w[E], b[E], dw[BWD ? E : 1], db[BWD ? E : 1];
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (u * G + gl) * VEC + e;
      w[u * VEC + e] = a.w && c < D ? ld_any(a.w, c, a.wbf) : 1.f;
      b[u * VEC + e] = a.b && c < D ? ld_any(a.b, c, a.wbf) : 0.f;
      if constexpr (BWD) dw[u * VEC + e] = db[u * VEC + e] = 0.f;
    }
  using R = VecRaw<T, VEC>;
  // whole workgroups step together (the G = 256 sums hold a barrier)
  for (int64_t r0 = (int64_t)blockIdx.x * GPW; r0 < rows; r0 += (int64_t)gridDim.x * GPW) {
    const int64_t row = r0 + grp;
    const bool live = row < rows;
    // rows and columns past the end repeat the last ones: no branch around a load
    const int64_t off = min(row, rows - 1) * D;
    R rx[NU], rz[NU], ry[BWD ? NU : 1];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int64_t at = off + min((u * G + gl) * VEC, D - VEC);
      rx[u] = *reinterpret_cast<const R*>(reinterpret_cast<const T*>(a.x) + at);
      if (a.z) rz[u] = *reinterpret_cast<const R*>(reinterpret_cast<const T*>(a.z) + at);
      if constexpr (BWD) ry[u] = *reinterpret_cast<const R*>(reinterpret_cast<const T*>(a.dy) + at);
    }
    float x[E], z[E], dy[BWD ? E : 1];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const bool in = (u * G + gl) * VEC < D && live;
      vec_get<T, VEC>(x + u * VEC, rx[u]);
      if (a.z) vec_get<T, VEC>(z + u * VEC, rz[u]);
      if constexpr (BWD) vec_get<T, VEC>(dy + u * VEC, ry[u]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = u * VEC + e;
        x[i] = in ? x[i] : 0.f;
        z[i] = in && a.z ? z[i] : 0.f;
        if constexpr (BWD) dy[i] = in ? dy[i] : 0.f;
      }
    }
    if (a.layer) {
      float m[1] = {0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) m[0] += x[i];
      group_sum<G, 1>(m, s_sum, flip);
      const float mu = m[0] * inv_d;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          x[u * VEC + e] = (u * G + gl) * VEC + e < D ? x[u * VEC + e] - mu : 0.f;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) q[0] = fmaf(x[i], x[i], q[0]);
    group_sum<G, 1>(q, s_sum, flip);
    const float r = 1.f / sqrtf(q[0] * inv_d + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int c = (u * G + gl) * VEC;
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = u * VEC + e;
          float v = fmaf(x[i] * r, w[i], b[i]);
          if (a.z) {
            float f, df;
            gate_act(a.act, z[i], &f, &df);
            v *= f;
          }
          y[e] = v;
        }
        if (c < D && live) vec_st<T, VEC>(reinterpret_cast<T*>(a.y) + off + c, y);
      }
    } else {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int c = (u * G + gl) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = u * VEC + e;
          x[i] *= r;  // n
          float da = dy[i];
          if (a.z) {
            float f, df;
            gate_act(a.act, z[i], &f, &df);
            z[i] = dy[i] * fmaf(x[i], w[i], b[i]) * df;
            da *= f;
          }
          dw[i] = fmaf(da, x[i], dw[i]);
          db[i] += da;
          dy[i] = da * w[i];  // dn
          m[0] = fmaf(dy[i], x[i], m[0]);
          m[1] += dy[i];
        }
        if (a.z && c < D && live) vec_st<T, VEC>(reinterpret_cast<T*>(a.dz) + off + c, z + u * VEC);
      }
      group_sum<G, 2>(m, s_sum, flip);
      const float m1 = m[0] * inv_d, m0 = a.layer ? m[1] * inv_d : 0.f;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int c = (u * G + gl) * VEC;
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = u * VEC + e;
          y[e] = r * (dy[i] - m0 - x[i] * m1);
        }
        if (c < D && live) vec_st<T, VEC>(reinterpret_cast<T*>(a.dx) + off + c, y);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // the workgroup's groups hold the same columns: add them in order
    constexpr int NB = G * VEC;  // columns per unit round
    __shared__ float s_w[GPW > 1 ? 256 * VEC : 1], s_b[GPW > 1 ? 256 * VEC : 1];
    float* part = a.part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if constexpr (GPW > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s_w[grp * NB + gl * VEC + e] = dw[u * VEC + e];
          s_b[grp * NB + gl * VEC + e] = db[u * VEC + e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < NB; c += 256) {
          float tw = 0.f, tb = 0.f;
          for (int i = 0; i < GPW; ++i) {
            tw += s_w[i * NB + c];
            tb += s_b[i * NB + c];
          }
          if (u * NB + c < D) {
            part[u * NB + c] = tw;
            part[D + u * NB + c] = tb;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int c = (u * G + gl) * VEC + e;
          if (c < D) {
            part[c] = dw[u * VEC + e];
            part[D + c] = db[u * VEC + e];
          }
        }
      }
    }
  }
}

// dweight, dbias: the workgroups' partial rows added in a fixed order (32 rows
// apart per thread, then the 32 sums in order, in double)
__global__ void __launch_bounds__(512)
norm_reduce_kernel(const float* __restrict__ part, int wgs, int D, int wbf, void* dw, void* db) {
  __shared__ double s[2][32][17];
  const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4, c = blockIdx.x * 16 + cl;
  double a = 0., b = 0.;
  if (c < D) {
    const float* p = part + c;
    int i = rl;
    for (; i + 96 < wgs; i += 128) {
      float x[4], y[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        x[n] = p[(size_t)(i + 32 * n) * 2 * D];
        y[n] = p[(size_t)(i + 32 * n) * 2 * D + D];
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        a += x[n];
        b += y[n];
      }
    }
    for (; i < wgs; i += 32) {
      a += p[(size_t)i * 2 * D];
      b += p[(size_t)i * 2 * D + D];
    }
  }
  s[0][rl][cl] = a;
  s[1][rl][cl] = b;
  __syncthreads();
  if (rl == 0 && c < D) {
    for (int i = 1; i < 32; ++i) {
      a += s[0][i][cl];
      b += s[1][i][cl];
    }
    if (dw) st_any(dw, c, wbf, (float)a);
    if (db) st_any(db, c, wbf, (float)b);
  }
}

// Workgroups of a launch: each group of lanes gets a row, up to 8 (forward) or
// kNormBwdWgs (backward, which also writes a partial row per workgroup)
// workgroups per compute unit, after which the groups stride over the rows.
// Backward, 2M rows of 128: 3 per unit 533 us, 4 552 us, 2 567 us; where a
// workgroup holds a whole row its registers allow two: 8191 rows of 4096 with
// 2 per unit 57 + 7 us (partial rows), with 3 76 + 9 us, with 4 70 + 12 us.
constexpr int kNormBwdWgs = 3;
static int norm_wgs(int64_t rows, int gpw, bool bwd) {
  const int64_t need = (rows + gpw - 1) / gpw;
  const int64_t cap = (int64_t)kda_host::device_cus() * (bwd ? (gpw == 1 ? 2 : kNormBwdWgs) : 8);
  return (int)std::max<int64_t>(1, std::min(need, cap));
}

template <typename T, int VEC, bool BWD, typename Fn>
static hipError_t norm_pick(int D, Fn&& go) {
#define KDA_NORM_CFG(G, NU) \
  if (D <= G * NU * VEC) return go(std::integral_constant<int, G>(), std::integral_constant<int, NU>());
  if constexpr (VEC > 1) {
    KDA_NORM_CFG(16, 1)
    KDA_NORM_CFG(16, 2)
    KDA_NORM_CFG(64, 1)
    KDA_NORM_CFG(64, 2)
    KDA_NORM_CFG(256, 1)
    KDA_NORM_CFG(256, 2)
    KDA_NORM_CFG(256, 4)
    if constexpr (sizeof(T) == 4) KDA_NORM_CFG(256, 8)  // 8192 columns; bf16 has them with 4 rounds of 8
  } else {
    KDA_NORM_CFG(16, 4)
    KDA_NORM_CFG(64, 4)
    KDA_NORM_CFG(256, 4)
    KDA_NORM_CFG(256, 16)
    KDA_NORM_CFG(256, 32)
  }
#undef KDA_NORM_CFG
  return hipErrorInvalidValue;
}

template <typename T, bool BWD>
static hipError_t norm_t(NormArgs a, hipStream_t s, void* dw, void* db) {
  auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  constexpr int FV = 16 / (int)sizeof(T);
  const bool vec = a.D % FV == 0 && al(a.x) && al(a.z) && al(a.dy) && al(a.y) && al(a.dx) && al(a.dz);
  int wgs = 0;
  auto go = [&](auto vc) {
    constexpr int VEC = decltype(vc)::value;
    return norm_pick<T, VEC, BWD>(a.D, [&](auto gc, auto nc) {
      constexpr int G = decltype(gc)::value, NU = decltype(nc)::value;
      wgs = norm_wgs(a.rows, 256 / G, BWD);
      hipLaunchKernelGGL((norm_kernel<T, VEC, G, NU, BWD>), dim3(wgs), dim3(256), 0, s, a);
      return hipGetLastError();
    });
  };
  hipError_t e = vec ? go(std::integral_constant<int, FV>()) : go(std::integral_constant<int, 1>());
  if (e != hipSuccess || !BWD || !a.part) return e;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((a.D + 15) / 16), dim3(512), 0, s, a.part, wgs, a.D, a.wbf, dw, db);
  return hipGetLastError();
}

}  // namespace kda

namespace kda_host {

size_t norm_bwd_ws_bytes(int D) {
  return (size_t)device_cus() * kda::kNormBwdWgs * 2 * (size_t)D * sizeof(float);
}

hipError_t launch_norm(kda_dtype dt, int64_t rows, const kda_norm& p, const int32_t* cu, int N, int rpt,
                       const void* x, const void* z, void* y, hipStream_t s) {
  kda::NormArgs a{x, p.weight, p.bias, z, nullptr, y, nullptr, nullptr, nullptr, rows, cu, N, rpt,
                  p.D, p.param_dtype == KDA_BF16, p.kind == KDA_NORM_LAYER, p.activation, p.eps};
  return dt == KDA_BF16 ? kda::norm_t<kda::bf16, false>(a, s, nullptr, nullptr)
                        : kda::norm_t<float, false>(a, s, nullptr, nullptr);
}

hipError_t launch_norm_bwd(kda_dtype dt, int64_t rows, const kda_norm& p, const int32_t* cu, int N, int rpt,
                           const void* x, const void* z, const void* dy, void* dx, void* dz, void* dw,
                           void* db, void* ws, hipStream_t s) {
  kda::NormArgs a{x, p.weight, p.bias, z, dy, nullptr, dx, dz, (dw || db) ? (float*)ws : nullptr, rows, cu, N,
                  rpt, p.D, p.param_dtype == KDA_BF16, p.kind == KDA_NORM_LAYER, p.activation, p.eps};
  return dt == KDA_BF16 ? kda::norm_t<kda::bf16, true>(a, s, dw, db) : kda::norm_t<float, true>(a, s, dw, db);
}

}  // namespace kda_host
