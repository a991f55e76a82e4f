// Token-sequential gated delta rule with a scalar gate, FP32 compute.
//
// Per token, with the decay d = e^{g_t} and q~ = q / sqrt(K):
//   u = d S^T k,  w = d S^T q~,  delta = b (v - u),  o = w + delta (k . q~),
//   S = d S + k delta^T
// in one pass over the state, which stays in registers for the whole sequence:
// it is read once and written once, and for decode (one token per sequence)
// those two passes over HBM are the kernel's time. Waves are independent: each
// owns all K rows of a block of columns of one (sequence, value head), a lane
// RPL consecutive rows of four columns, so k and q come as vectors, the sums
// over K are RPL terms and a butterfly over the row lanes, and the decay is
// one scalar per token. 256 slots of one token, 32 value heads, K = V = 128
// (970 MB): 172 us, 5.6 TB/s; one slot: 6 us, of which the launch is most.
#include "kda_gdn.h"

namespace kda {

template <int RL>
__device__ __forceinline__ float row_lanes_sum(float x) {
#pragma unroll
  for (int d = 64 / RL; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

template <typename T, int N>
__device__ __forceinline__ void ld_vec(float* x, const T* p) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + i);
      x[i] = a.x; x[i + 1] = a.y; x[i + 2] = a.z; x[i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 a = unpack4(*reinterpret_cast<const uint2*>(p + i));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i + e] = a[e];
    }
  }
}

// K in {64, 128, 256}, V a multiple of 4, aligned operands (see launch).
template <typename T, int K, int RPL>
__global__ void __launch_bounds__(256)
gdn_recurrent_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, GdnGate gate,
                     const T* __restrict__ beta, const float* h0, const int32_t* __restrict__ cu, int T_,
                     int H, int HV, int V, int n_cb, int64_t n_tasks, int l2, float scale, int write_final,
                     T* __restrict__ o, float* ht) {
  constexpr int RL = K / RPL, CL = 64 / RL, CW = 4 * CL;
  const int lane = threadIdx.x & 63, cl = lane % CL, rl = lane / CL;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= n_tasks) return;
  const int cb = (int)(task % n_cb);
  const int64_t nh = task / n_cb;
  const int hv = (int)(nh % HV), n = (int)(nh / HV), h = hv / (HV / H);
  const int col = cb * CW + 4 * cl;
  const bool col_ok = col < V;
  int64_t bos;
  int len;
  seq_range(cu, n, T_, &bos, &len);
  const size_t st = ((size_t)n * HV + hv) * (size_t)K * V + (size_t)(rl * RPL) * V + col;
  if (len <= 0) {
    if (!write_final || (h0 == ht && h0 != nullptr) || !col_ok) return;
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
      u32x4 x = {0u, 0u, 0u, 0u};
      if (h0) x = *reinterpret_cast<const u32x4*>(h0 + st + (size_t)i * V);
      *reinterpret_cast<u32x4*>(ht + st + (size_t)i * V) = x;
    }
    return;
  }
  struct Tok {
    float k[RPL], q[RPL], v[4], d, b;
  };
  auto load = [&](int64_t t, Tok& x) {
    ld_vec<T, RPL>(x.k, k + (t * H + h) * K + rl * RPL);
    ld_vec<T, RPL>(x.q, q + (t * H + h) * K + rl * RPL);
    ld_vec<T, 4>(x.v, v + (t * HV + hv) * V + (col_ok ? col : 0));
    float xb, sc;
    x.d = expf(gdn_gate(gate, t * HV + hv, hv, &xb, &sc));
    x.b = to_f32(beta[t * HV + hv]);
  };
  f32x4 s[RPL];
#pragma unroll
  for (int i = 0; i < RPL; ++i) {
    s[i] = zero4();
    if (h0 && col_ok) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(h0 + st + (size_t)i * V));
  }
  Tok x;
  load(bos, x);
  for (int it = 0; it < len; ++it) {
    Tok y;
    if (it + 1 < len) load(bos + it + 1, y);
    f32x4 u = zero4(), w = zero4();
    float kq = 0.f, kk = 0.f, qq = 0.f;
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
      kq = fmaf(x.k[i], x.q[i], kq);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = fmaf(s[i][e], x.k[i], u[e]);
        w[e] = fmaf(s[i][e], x.q[i], w[e]);
      }
    }
    float rk = 1.f, rq = scale;
    if (l2) {
#pragma unroll
      for (int i = 0; i < RPL; ++i) {
        kk = fmaf(x.k[i], x.k[i], kk);
        qq = fmaf(x.q[i], x.q[i], qq);
      }
      rk = l2norm_inv(row_lanes_sum<RL>(kk));
      rq *= l2norm_inv(row_lanes_sum<RL>(qq));
    }
    kq = row_lanes_sum<RL>(kq) * rk * rq;
    f32x4 dl, out;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = row_lanes_sum<RL>(u[e]) * (x.d * rk);
      w[e] = row_lanes_sum<RL>(w[e]) * (x.d * rq);
      const float d = x.b * (x.v[e] - u[e]);
      out[e] = fmaf(d, kq, w[e]);
      dl[e] = d * rk;
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = fmaf(x.k[i], dl[e], s[i][e] * x.d);
    if (rl == 0 && col_ok) {
      T* p = o + ((bos + it) * HV + hv) * V + col;
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = pack4(out);
      else *reinterpret_cast<f32x4*>(p) = out;
    }
    x = y;
  }
  if (write_final && col_ok) {
#pragma unroll
    for (int i = 0; i < RPL; ++i)
      __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(ht + st + (size_t)i * V));
  }
}

// Any K <= 4 MAXR, any V, any alignment: a wave owns 16 columns, lane (rl, cl)
// rows rl, rl + 4, ... of one column.
template <typename T, int MAXR>
__global__ void __launch_bounds__(256)
gdn_recurrent_any_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                         GdnGate gate, const T* __restrict__ beta, const float* h0,
                         const int32_t* __restrict__ cu, int T_, int H, int HV, int K, int V, int n_cb,
                         int64_t n_tasks, int l2, float scale, int write_final, T* __restrict__ o, float* ht) {
  const int lane = threadIdx.x & 63, cl = lane & 15, rl = lane >> 4;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (task >= n_tasks) return;
  const int cb = (int)(task % n_cb);
  const int64_t nh = task / n_cb;
  const int hv = (int)(nh % HV), n = (int)(nh / HV), h = hv / (HV / H);
  const int col = cb * 16 + cl;
  const bool ok = col < V;
  int64_t bos;
  int len;
  seq_range(cu, n, T_, &bos, &len);
  const size_t st = ((size_t)n * HV + hv) * (size_t)K * V + col;
  if (len <= 0) {
    if (!write_final || (h0 == ht && h0 != nullptr) || !ok) return;
    for (int r = rl; r < K; r += 4)
      reinterpret_cast<uint32_t*>(ht)[st + (size_t)r * V] =
          h0 ? reinterpret_cast<const uint32_t*>(h0)[st + (size_t)r * V] : 0u;
    return;
  }
  float s[MAXR];
#pragma unroll
  for (int i = 0; i < MAXR; ++i) {
    const int r = rl + 4 * i;
    s[i] = (h0 && ok && r < K) ? h0[st + (size_t)r * V] : 0.f;
  }
  for (int it = 0; it < len; ++it) {
    const int64_t t = bos + it;
    const T* kp = k + (t * H + h) * K;
    const T* qp = q + (t * H + h) * K;
    float xb, sc;
    const float d = expf(gdn_gate(gate, t * HV + hv, hv, &xb, &sc)), b = to_f32(beta[t * HV + hv]);
    const float vv = ok ? to_f32(v[(t * HV + hv) * V + col]) : 0.f;
    float u = 0.f, w = 0.f, kq = 0.f, kk = 0.f, qq = 0.f;
#pragma unroll
    for (int i = 0; i < MAXR; ++i) {
      const int r = rl + 4 * i;
      const float kr = r < K ? to_f32(kp[r]) : 0.f, qr = r < K ? to_f32(qp[r]) : 0.f;
      u = fmaf(s[i], kr, u);
      w = fmaf(s[i], qr, w);
      kq = fmaf(kr, qr, kq);
      kk = fmaf(kr, kr, kk);
      qq = fmaf(qr, qr, qq);
    }
    float rk = 1.f, rq = scale;
    if (l2) {
      rk = l2norm_inv(row_lanes_sum<4>(kk));
      rq *= l2norm_inv(row_lanes_sum<4>(qq));
    }
    kq = row_lanes_sum<4>(kq) * rk * rq;
    u = row_lanes_sum<4>(u) * (d * rk);
    w = row_lanes_sum<4>(w) * (d * rq);
    const float dl = b * (vv - u);
    if (rl == 0 && ok) o[(t * HV + hv) * V + col] = from_f32<T>(fmaf(dl, kq, w));
#pragma unroll
    for (int i = 0; i < MAXR; ++i) {
      const int r = rl + 4 * i;
      const float kr = r < K ? to_f32(kp[r]) : 0.f;
      s[i] = fmaf(kr, dl * rk, s[i] * d);
    }
  }
  if (write_final && ok) {
#pragma unroll
    for (int i = 0; i < MAXR; ++i) {
      const int r = rl + 4 * i;
      if (r < K) ht[st + (size_t)r * V] = s[i];
    }
  }
}

template <typename T, int K, int RPL>
static hipError_t rec_vec(const kda_dims& d, const void* q, const void* k, const void* v, const GdnGate& gate,
                          int l2, const void* beta, const float* h0, const int32_t* cu, int write_final,
                          void* o, float* ht, hipStream_t s) {
  constexpr int CW = 4 * 64 / (K / RPL);
  const int n_cb = (d.V + CW - 1) / CW;
  const int64_t tasks = (int64_t)d.N * d.HV * n_cb;
  hipLaunchKernelGGL((gdn_recurrent_kernel<T, K, RPL>), dim3((unsigned)((tasks + 3) / 4)), dim3(256), 0, s,
                     (const T*)q, (const T*)k, (const T*)v, gate, (const T*)beta, h0, cu, d.T, d.H, d.HV, d.V,
                     n_cb, tasks, l2, 1.0f / sqrtf((float)K), write_final, (T*)o, ht);
  return hipGetLastError();
}
template <typename T, int MAXR>
static hipError_t rec_any(const kda_dims& d, const void* q, const void* k, const void* v, const GdnGate& gate,
                          int l2, const void* beta, const float* h0, const int32_t* cu, int write_final,
                          void* o, float* ht, hipStream_t s) {
  const int n_cb = (d.V + 15) / 16;
  const int64_t tasks = (int64_t)d.N * d.HV * n_cb;
  hipLaunchKernelGGL((gdn_recurrent_any_kernel<T, MAXR>), dim3((unsigned)((tasks + 3) / 4)), dim3(256), 0, s,
                     (const T*)q, (const T*)k, (const T*)v, gate, (const T*)beta, h0, cu, d.T, d.H, d.HV, d.K,
                     d.V, n_cb, tasks, l2, 1.0f / sqrtf((float)d.K), write_final, (T*)o, ht);
  return hipGetLastError();
}

template <typename T>
static hipError_t rec_t(const kda_dims& d, const void* q, const void* k, const void* v, const GdnGate& gate,
                        int l2, const void* beta, const float* h0, const int32_t* cu, int write_final, void* o,
                        float* ht, hipStream_t s) {
  auto al = [](const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; };
  const bool vec = (d.K == 64 || d.K == 128 || d.K == 256) && d.V % 4 == 0 && al(q, 16) && al(k, 16) &&
                   al(v, 4 * sizeof(T)) && al(o, 4 * sizeof(T)) && al(h0, 16) && al(ht, 16);
#define KDA_GDN_REC(F, A, B) return F<T, A, B>(d, q, k, v, gate, l2, beta, h0, cu, write_final, o, ht, s)
#define KDA_GDN_REC1(F, A) return F<T, A>(d, q, k, v, gate, l2, beta, h0, cu, write_final, o, ht, s)
  if (vec) {
    // 16 rows per lane while its waves give every SIMD one, else 4 rows per
    // lane: four times the waves, a quarter of the loads each (K = V = 128, 32
    // value heads, one token: 256 slots 172 us with 16 rows, 501 us with 4; one
    // slot 6.0 and 5.6 us)
    const int64_t waves = (int64_t)d.N * d.HV * ((d.V * (d.K / 16) + 255) / 256);
    const bool many = waves >= 4 * (int64_t)kda_host::device_cus();
    if (d.K == 64) {
      if (many) KDA_GDN_REC(rec_vec, 64, 16);
      KDA_GDN_REC(rec_vec, 64, 4);
    }
    if (d.K == 128) {
      if (many) KDA_GDN_REC(rec_vec, 128, 16);
      KDA_GDN_REC(rec_vec, 128, 4);
    }
    if (many) KDA_GDN_REC(rec_vec, 256, 16);
    KDA_GDN_REC(rec_vec, 256, 4);
  }
  if (d.K <= 64) KDA_GDN_REC1(rec_any, 16);
  if (d.K <= 128) KDA_GDN_REC1(rec_any, 32);
  KDA_GDN_REC1(rec_any, 64);
#undef KDA_GDN_REC
#undef KDA_GDN_REC1
}

}  // namespace kda

namespace kda_host {

hipError_t launch_gdn_recurrent(const kda_dims& d, kda_dtype dt, const void* q, const void* k, const void* v,
                                const kda::GdnGate& gate, int l2, const void* beta, const float* h0,
                                const int32_t* cu, int write_final, void* o, float* ht, hipStream_t s) {
  if (d.N == 0) return hipSuccess;
  if (dt == KDA_BF16) return kda::rec_t<kda::bf16>(d, q, k, v, gate, l2, beta, h0, cu, write_final, o, ht, s);
  return kda::rec_t<float>(d, q, k, v, gate, l2, beta, h0, cu, write_final, o, ht, s);
}

}  // namespace kda_host
