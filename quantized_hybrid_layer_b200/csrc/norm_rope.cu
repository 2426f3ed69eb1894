// qhl_qk_norm_rope: RMSNorm of every query and key head and rotate-half RoPE in
// one pass over the in-projection's rows, with q, k and v leaving in the
// cache's 16-bit type.
//
// Per head vector x of D elements:  z = x / sqrt(mean(x^2) + eps) * gamma, then
// for the leading R dimensions, with i < R / 2 and a = pos * theta^(-2 i / R):
//     out_i = z_i cos a - z_{i + R/2} sin a,   out_{i + R/2} = z_{i + R/2} cos a + z_i sin a.
//
// Bound by HBM: every element is read and written once.  One warp holds V head
// vectors of one token in registers (lane l: the four elements 4l.. of each 128,
// so every load and store is a run of whole sectors); their loads are issued
// together, and the angles, which all heads of a token share, are formed while
// they are in flight.  The partner of a rotated element comes from shared
// memory.  Angles reach pos * 1 = 262144 rad, where an f32 is 2^-6 apart: the
// product and its reduction to turns are 64-bit (a handful of instructions per
// warp), and theta^(-2 i / R) is a product of at most seven factors
// theta^(-2^(j+1) / R), one for each bit j of i, so no table is read.
#include <algorithm>

#include "launch.h"
#include "verify.cuh"

namespace qhl {

struct NormRopeArgs {
  const void* y;
  long long y_stride;
  int q_off, k_off, v_off;
  int n_rows, hq, hkv, rope;
  float eps;
  const int* pos;
  const float* gq;
  const float* gk;
  void* out[3];             // q, k, v
  long long out_stride[3];
  double power[7];          // theta^(-2^(j+1) / rope)
};

template <typename T>
struct Pack;   // four elements of T
template <>
struct Pack<float> {
  using V = float4;
  QHL_DEV static void get(V v, float (&x)[4]) { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
};
template <>
struct Pack<__half> {
  using V = uint2;
  QHL_DEV static void get(V v, float (&x)[4]) {
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&v.x)), b = __half22float2(*reinterpret_cast<__half2*>(&v.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
  QHL_DEV static V put(const float (&x)[4]) {
    __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};
template <>
struct Pack<__nv_bfloat16> {
  using V = uint2;
  QHL_DEV static void get(V v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  QHL_DEV static V put(const float (&x)[4]) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};

// A warp's task: V consecutive head vectors (q heads, then k, then v) of a row.
// J groups of 128 dimensions per vector; at D = 64 the upper half-warp idles in
// the loads of a vector (its lanes hold zeros).
template <typename SRC, typename DST, int D, int V>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int J = D > 128 ? D / 128 : 1;
  __shared__ float2 s_turn[8][D / 2];
  __shared__ __align__(16) float s_vec[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nvec = a.hq + 2 * a.hkv, per_row = (nvec + V - 1) / V;
  const long long task = (long long)blockIdx.x * 8 + warp;
  if (threadIdx.x == 0) pdl_launch();
  if (task >= (long long)a.n_rows * per_row) return;
  pdl_wait();
  const int row = (int)(task / per_row), v0 = (int)(task % per_row) * V;
  const bool on = D >= 128 || 4 * lane < D;

  const SRC* yr = static_cast<const SRC*>(a.y) + (long long)row * a.y_stride;
  typename Pack<SRC>::V raw[V][J];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int vec = v0 + u;
    const int off = vec < a.hq ? a.q_off + vec * D
                               : vec < a.hq + a.hkv ? a.k_off + (vec - a.hq) * D : a.v_off + (vec - a.hq - a.hkv) * D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      raw[u][j] = typename Pack<SRC>::V{};
      if (on && vec < nvec) raw[u][j] = __ldg(reinterpret_cast<const typename Pack<SRC>::V*>(yr + off + 128 * j) + lane);
    }
  }

  const int half = a.rope / 2;
  if (v0 < a.hq + a.hkv && half) {
    const double pos = (double)__ldg(a.pos + row);
    for (int i = lane; i < half; i += 32) {
      double f = 1.0;
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (i >> j & 1) f *= a.power[j];
      double t = pos * f * 0.15915494309189533577;   // in turns: 1 / (2 pi)
      t -= rint(t);
      float sn, cs;
      sincospif((float)(2.0 * t), &sn, &cs);
      s_turn[warp][i] = make_float2(cs, sn);
    }
  }
  __syncwarp();

#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int vec = v0 + u;
    if (vec >= nvec) return;
    const int kind = vec < a.hq ? 0 : vec < a.hq + a.hkv ? 1 : 2;
    const int head = vec - (kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv);
    float x[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) Pack<SRC>::get(raw[u][j], x[j]);
    if (kind < 2) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = __fmaf_rn(x[j][e], x[j][e], ss);
      ss = warp_sum(ss);
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.f / D), a.eps)));
      const float* gamma = kind == 0 ? a.gq : a.gk;
      if (on) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + 128 * j) + lane);
          x[j][0] *= r * g.x; x[j][1] *= r * g.y; x[j][2] *= r * g.z; x[j][3] *= r * g.w;
          if (128 * j < a.rope)
            reinterpret_cast<float4*>(s_vec[warp] + 128 * j)[lane] = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
        }
      }
      __syncwarp();
      // half is a multiple of 4: a lane's four elements lie on one side of it
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int d = 128 * j + 4 * lane;
        if (on && d < a.rope) {
          const bool low = d < half;
          const int i = low ? d : d - half;
          const float4 o = *reinterpret_cast<const float4*>(s_vec[warp] + (low ? d + half : i));
          const float p[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = s_turn[warp][i + e];
            x[j][e] = low ? x[j][e] * t.x - p[e] * t.y : x[j][e] * t.x + p[e] * t.y;
          }
        }
      }
      __syncwarp();
    }
    if (on) {
      DST* dst = static_cast<DST*>(a.out[kind]) + (long long)row * a.out_stride[kind] + head * D;
#pragma unroll
      for (int j = 0; j < J; ++j) reinterpret_cast<uint2*>(dst + 128 * j)[lane] = Pack<DST>::put(x[j]);
    }
  }
}

template <typename SRC, typename DST, int D>
static cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
  const int nvec = a.hq + 2 * a.hkv;
  // Few rows: one vector per warp, over as many SMs as there are; many: four per
  // warp, so that a warp keeps 4 KB in flight and forms the angles once (8191 rows:
  // two per warp 73.8 us, four 70.1 us, eight 92.3 us).
  const bool many = (long long)a.n_rows * nvec >= 148LL * 64 * 4;
  const long long tasks = (long long)a.n_rows * (many ? (nvec + 3) / 4 : nvec);
  const unsigned grid = (unsigned)((tasks + 7) / 8);
  return many ? launch_ex(norm_rope_kernel<SRC, DST, D, 4>, dim3(grid), dim3(256), 0, s, true, a)
              : launch_ex(norm_rope_kernel<SRC, DST, D, 1>, dim3(grid), dim3(256), 0, s, true, a);
}

template <typename SRC, typename DST>
static cudaError_t launch_norm_rope_d(int d, const NormRopeArgs& a, cudaStream_t s) {
  return d == 256 ? launch_norm_rope<SRC, DST, 256>(a, s)
                  : d == 128 ? launch_norm_rope<SRC, DST, 128>(a, s) : launch_norm_rope<SRC, DST, 64>(a, s);
}

template <typename SRC>
static cudaError_t launch_norm_rope_t(int dt, int d, const NormRopeArgs& a, cudaStream_t s) {
  return dt == QHL_F16 ? launch_norm_rope_d<SRC, __half>(d, a, s) : launch_norm_rope_d<SRC, __nv_bfloat16>(d, a, s);
}

}  // namespace qhl

using namespace qhl;

extern "C" int qhl_qk_norm_rope(int n_q_heads, int n_kv_heads, int dim, int rope_dims, double theta, float eps,
                                const void* y_dev, int y_dtype, long long y_stride, int q_off, int k_off, int v_off,
                                int n_rows, const int* pos_dev, const float* gamma_q_dev, const float* gamma_k_dev,
                                int dtype, void* q_dev, long long q_stride, void* k_dev, long long k_stride,
                                void* v_dev, long long v_stride, void* stream) {
  const char* me = "qhl_qk_norm_rope";
  if (!y_dev || !pos_dev || !gamma_q_dev || !gamma_k_dev || !q_dev || !k_dev || !v_dev)
    return verify_err(me, STAGE_E_ARG, "null pointer");
  if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads > 65536 || n_kv_heads > 65536 || n_rows < 0)
    return verify_err(me, STAGE_E_ARG, "head or row count out of range");
  if (dim != 64 && dim != 128 && dim != 256) return verify_err(me, STAGE_E_UNSUPPORTED, "dim must be 64, 128 or 256");
  if (rope_dims < 0 || rope_dims > dim || rope_dims % 8)
    return verify_err(me, STAGE_E_ARG, "rope_dims must be a multiple of 8 and at most dim");
  if (rope_dims && !(theta > 0 && std::isfinite(theta))) return verify_err(me, STAGE_E_ARG, "theta must be positive");
  if (!(eps >= 0 && std::isfinite(eps))) return verify_err(me, STAGE_E_ARG, "eps must not be negative");
  if ((y_dtype != QHL_F32 && y_dtype != QHL_F16 && y_dtype != QHL_BF16) || (dtype != QHL_F16 && dtype != QHL_BF16))
    return verify_err(me, STAGE_E_UNSUPPORTED, "y must be f32, f16 or bf16, the outputs f16 or bf16");
  const int per16 = y_dtype == QHL_F32 ? 4 : 8;
  if (!aligned16(y_dev) || !aligned16(q_dev) || !aligned16(k_dev) || !aligned16(v_dev) || !aligned16(gamma_q_dev) ||
      !aligned16(gamma_k_dev) || y_stride % per16 || q_off % per16 || k_off % per16 || v_off % per16 || q_stride % 8 ||
      k_stride % 8 || v_stride % 8)
    return verify_err(me, STAGE_E_ARG, "bases, rows and offsets must be 16-byte aligned");
  const long long qw = (long long)n_q_heads * dim, kw = (long long)n_kv_heads * dim;
  if (q_off < 0 || k_off < 0 || v_off < 0 || q_off + qw > y_stride || k_off + kw > y_stride || v_off + kw > y_stride ||
      q_stride < qw || k_stride < kw || v_stride < kw)
    return verify_err(me, STAGE_E_ARG, "a row is shorter than its heads");
  if ((long long)n_rows * (n_q_heads + 2LL * n_kv_heads) > (1LL << 33))
    return verify_err(me, STAGE_E_ARG, "too many head vectors");
  if (n_rows == 0) return 0;
  NormRopeArgs a = {};
  a.y = y_dev;
  a.y_stride = y_stride;
  a.q_off = q_off;
  a.k_off = k_off;
  a.v_off = v_off;
  a.n_rows = n_rows;
  a.hq = n_q_heads;
  a.hkv = n_kv_heads;
  a.rope = rope_dims;
  a.eps = eps;
  a.pos = pos_dev;
  a.gq = gamma_q_dev;
  a.gk = gamma_k_dev;
  a.out[0] = q_dev;
  a.out[1] = k_dev;
  a.out[2] = v_dev;
  a.out_stride[0] = q_stride;
  a.out_stride[1] = k_stride;
  a.out_stride[2] = v_stride;
  double p = rope_dims ? std::pow(theta, -2.0 / rope_dims) : 1.0;
  for (int j = 0; j < 7; ++j, p *= p) a.power[j] = p;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = y_dtype == QHL_F32   ? launch_norm_rope_t<float>(dtype, dim, a, s)
                  : y_dtype == QHL_F16 ? launch_norm_rope_t<__half>(dtype, dim, a, s)
                                       : launch_norm_rope_t<__nv_bfloat16>(dtype, dim, a, s);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}
