// qhl_qk_norm_rope: RMSNorm of every query and key head and rotate-half RoPE in
// one pass over the in-projection's rows, with q, k and v leaving in the
// cache's 16-bit type.
//
// Per head vector x of D elements:  z = x / sqrt(mean(x^2) + eps) * gamma, then
// for the leading R dimensions, with i < R / 2 and a = pos * theta^(-2 i / R):
//     out_i = z_i cos a - z_{i + R/2} sin a,   out_{i + R/2} = z_{i + R/2} cos a + z_i sin a.
//
// Bound by HBM: every element is read and written once.  A lane holds eight elements,
// so a warp holds 256 / D head vectors of one token at a time, V times; their loads
// are issued together, and the angles, which all heads of a token share, are formed
// while they are in flight.  The partner of a rotated element is in the lane where
// the whole vector is rotated, and comes from shared memory otherwise.  Angles reach pos * 1 = 262144 rad, where an f32
// is 2^-6 apart: the product and its reduction to turns are 64-bit (a handful of
// instructions per warp), and theta^(-2 i / R) is a product of at most seven factors
// theta^(-2^(j+1) / R), one for each bit j of i, so no table is read.
//
// Measured: 8191 tokens of 24 + 4 + 4 heads of 256, f32 to bf16, 72 to 76 us, 5.3 to
// 5.6 TB/s (0.81 to 0.86 of the measured copy); of 96 + 8 + 8 heads of 64 61 us, 5.8
// TB/s; from 16-bit rows 4.1 to 4.6 TB/s, bound by the instructions.  One token: 3.1
// to 3.7 us a call, a launch.
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

// A warp's task: V times NP consecutive head vectors (q heads, then k, then v) of a
// row.  Lane l has a part of vector l / LPV: the four elements 4 (l % LPV) .. of each
// half of it, so that every load and store of a warp is a run of whole sectors and
// the partner of an element that is rotated with all of its vector is in the lane.
template <typename SRC, typename DST, int D, int V>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPV = D / 8, NP = 32 / LPV;
  __shared__ __align__(16) float2 s_turn[8][D / 2];
  __shared__ __align__(16) float s_vec[8][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPV, d0 = lane % LPV * 4;
  const int nvec = a.hq + 2 * a.hkv, per_row = (nvec + V * NP - 1) / (V * NP);
  const long long task = (long long)blockIdx.x * 8 + warp;
  if (threadIdx.x == 0) pdl_launch();
  if (task >= (long long)a.n_rows * per_row) return;
  pdl_wait();
  const int row = (int)(task / per_row), v0 = (int)(task % per_row) * V * NP;

  const SRC* yr = static_cast<const SRC*>(a.y) + (long long)row * a.y_stride + d0;
  typename Pack<SRC>::V raw[V][2];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int vec = v0 + u * NP + sub;
    const int off = vec < a.hq ? a.q_off + vec * D
                               : vec < a.hq + a.hkv ? a.k_off + (vec - a.hq) * D : a.v_off + (vec - a.hq - a.hkv) * D;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      raw[u][j] = typename Pack<SRC>::V{};
      if (vec < nvec) raw[u][j] = *reinterpret_cast<const typename Pack<SRC>::V*>(yr + off + j * (D / 2));
    }
  }

  const int half = a.rope / 2;
  if (v0 < a.hq + a.hkv && half) {
    const double pos = (double)a.pos[row];
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
    const int vec = v0 + u * NP + sub;
    const int kind = vec < a.hq ? 0 : vec < a.hq + a.hkv ? 1 : 2;
    const int head = vec - (kind == 0 ? 0 : kind == 1 ? a.hq : a.hq + a.hkv);
    float x[2][4];
    Pack<SRC>::get(raw[u][0], x[0]);
    Pack<SRC>::get(raw[u][1], x[1]);
    if (v0 + u * NP < a.hq + a.hkv) {                // some vector of the warp is normalised
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __fmaf_rn(x[e >> 2][e & 3], x[e >> 2][e & 3], ss);
#pragma unroll
      for (int o = LPV / 2; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.f / D), a.eps)));
      if (kind < 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 g = *reinterpret_cast<const float4*>((kind == 0 ? a.gq : a.gk) + d0 + j * (D / 2));
          x[j][0] *= r * g.x; x[j][1] *= r * g.y; x[j][2] *= r * g.z; x[j][3] *= r * g.w;
        }
      }
      if (a.rope == D) {
        if (kind < 2) {
          const float4 t0 = *reinterpret_cast<const float4*>(&s_turn[warp][d0]), t1 = *reinterpret_cast<const float4*>(&s_turn[warp][d0 + 2]);
          const float cs[4] = {t0.x, t0.z, t1.x, t1.z}, sn[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x[0][e], o = x[1][e];
            x[0][e] = p * cs[e] - o * sn[e];
            x[1][e] = o * cs[e] + p * sn[e];
          }
        }
      } else if (half) {
        float* mine = s_vec[warp] + sub * D;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (kind < 2 && d0 + j * (D / 2) < a.rope) *reinterpret_cast<float4*>(mine + d0 + j * (D / 2)) = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
        __syncwarp();
        // half is a multiple of 4: a lane's four elements lie on one side of it
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = d0 + j * (D / 2);
          if (kind < 2 && d < a.rope) {
            const bool low = d < half;
            const int i = low ? d : d - half;
            const float4 o = *reinterpret_cast<const float4*>(mine + (low ? d + half : i));
            const float4 t0 = *reinterpret_cast<const float4*>(&s_turn[warp][i]), t1 = *reinterpret_cast<const float4*>(&s_turn[warp][i + 2]);
            const float p[4] = {o.x, o.y, o.z, o.w}, cs[4] = {t0.x, t0.z, t1.x, t1.z}, sn[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = low ? x[j][e] * cs[e] - p[e] * sn[e] : x[j][e] * cs[e] + p[e] * sn[e];
          }
        }
        __syncwarp();
      }
    }
    if (vec < nvec) {
      DST* dst = static_cast<DST*>(a.out[kind]) + (long long)row * a.out_stride[kind] + head * D + d0;
      *reinterpret_cast<uint2*>(dst) = Pack<DST>::put(x[0]);
      *reinterpret_cast<uint2*>(dst + D / 2) = Pack<DST>::put(x[1]);
    }
  }
}

template <typename SRC, typename DST, int D>
static cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
  // Few vectors, all in one wave of warps: one pass per warp (one row of 32 heads
  // 3.3 us a call, 64 rows 3.3 us; with four passes 4.1 and 4.4 us).  Many: four, so
  // that a warp has four loads per lane in flight and forms the angles once (512 rows
  // 6.0 us, 8191 rows 72.1 us; with one pass 6.7 and 88.0 us).
  constexpr int NP = 256 / D;
  const int nvec = a.hq + 2 * a.hkv, one = (nvec + NP - 1) / NP, four = (nvec + 4 * NP - 1) / (4 * NP);
  const bool few = (long long)a.n_rows * one <= 148 * 48;
  const dim3 grid((unsigned)(((long long)a.n_rows * (few ? one : four) + 7) / 8));
  return few ? launch_ex(norm_rope_kernel<SRC, DST, D, 1>, grid, dim3(256), 0, s, true, a)
             : launch_ex(norm_rope_kernel<SRC, DST, D, 4>, grid, dim3(256), 0, s, true, a);
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
