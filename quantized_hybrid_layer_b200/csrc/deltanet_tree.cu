// qhl_deltanet_tree: the gated DeltaNet state step along trees of drafted
// tokens.
//
// Per value head h (key head g = h / (Hv / Hk)), with q, k L2-normalised,
// beta = sigmoid(b), alpha = sigmoid(-a), and S_p the state of the parent:
//     S_i = alpha S_p,i + beta (v_i - alpha (S_p,i . k)) k,    o_i = S_i . q
// for every value row i of S, which change independently of one another.
//
// Bound by the snapshots: 64 KB per token and value head are written once (the
// starting state is read once; a state that a later branch starts from again is
// read back, from L2).  A CTA owns 32 value rows of one head of one tree and
// walks the tree's tokens in order; a warp keeps four rows of the last token's
// state in registers.  Where the next token starts from another state (a side
// branch), that state is requested before the current token is computed, so
// that only its products, not its load, stand in the chain of tokens.  A lane
// reads back only what it has written itself.
//
// The dot products of the four rows are reduced together: the first two
// butterfly steps halve the number of values a lane carries, so four sums take
// 6 shuffles instead of 20.  A sum's tree of additions is that of the plain
// butterfly (offsets 16, 8, 4, 2, 1), so a path's results have the same bits as
// the chained steps of qhl_deltanet_step.
#include "launch.h"
#include "verify.cuh"

namespace qhl {

constexpr int kDtBlock = 16;   // tokens whose inputs are staged together

struct DnTreeArgs {
  const float* y;
  int y_stride, Hk, Hv, n_rows, max_nodes, n_states;
  const int* q_start;
  const int* parent;
  const float* states;
  const int* index;
  float* snaps;
  float* o;
  unsigned* err;
};

// Totals over the warp of four values per lane: lane l returns the total of
// value (l >> 4 & 1) * 2 + (l >> 3 & 1).
QHL_DEV float warp_sum4(float v0, float v1, float v2, float v3, int lane) {
  const bool up = lane & 16;
  float a = __fadd_rn(up ? v2 : v0, __shfl_xor_sync(0xffffffffu, up ? v0 : v2, 16));
  float b = __fadd_rn(up ? v3 : v1, __shfl_xor_sync(0xffffffffu, up ? v1 : v3, 16));
  const bool up8 = lane & 8;
  float c = __fadd_rn(up8 ? b : a, __shfl_xor_sync(0xffffffffu, up8 ? a : b, 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c = __fadd_rn(c, __shfl_xor_sync(0xffffffffu, c, o));
  return c;
}

// A 16-byte load that stays behind this thread's earlier stores: a state row may
// have been written by the same lane some tokens ago.
QHL_DEV float4 ld_after_stores(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

__global__ void __launch_bounds__(256) dn_tree_kernel(const DnTreeArgs a) {
  __shared__ __align__(16) float sq[kDtBlock][kDnDim], sk[kDtBlock][kDnDim], sv[kDtBlock][32];
  __shared__ float sb[kDtBlock], sa[kDtBlock];
  __shared__ int sp[kMaxNodes];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x >> 2, part = blockIdx.x & 3, row0 = part * 32 + warp * 4;
  const int g = h / (a.Hv / a.Hk);
  const int off_k = a.Hk * kDnDim, off_v = 2 * off_k, off_b = off_v + a.Hv * kDnDim, off_a = off_b + a.Hv;
  const size_t state_elems = (size_t)a.Hv * kDnDim * kDnDim;
  const size_t mine = ((size_t)h * kDnDim + row0) * kDnDim + 4 * lane;   // this lane's element of row 0 of its warp

  if (tid == 0) pdl_launch();
  pdl_wait();
  int first, n;
  tree_rows(a.q_start, blockIdx.y, a.n_rows, a.max_nodes, first, n, a.err);
  if (n == 0) return;
  int idx = __ldg(a.index + blockIdx.y);
  if (idx < -1 || idx >= a.n_states) {
    if (tid == 0) atomicOr(a.err, ERR_BAD_INDEX);
    idx = -1;
  }
  for (int i = tid; i < n; i += 256) {
    int p = __ldg(a.parent + first + i);
    if (p < -2 || p >= i) {
      atomicOr(a.err, ERR_BAD_INDEX);
      p = -2;
    }
    sp[i] = p;
  }
  __syncthreads();

  auto fetch = [&](int p, float4(&X)[4]) {
    const float* src = p >= 0 ? a.snaps + (size_t)(first + p) * state_elems : a.states + (size_t)max(idx, 0) * state_elems;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      X[r] = p >= 0 || idx >= 0 ? ld_after_stores(src + mine + (size_t)r * kDnDim)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // padded tokens so far, by index (tokens of one tree: at most 128)
  uint64_t dead_lo = 0, dead_hi = 0;
  auto is_dead = [&](int i) {
    const int p = sp[i];
    if (p < 0) return p == -2;
    return ((p < 64 ? dead_lo >> p : dead_hi >> (p - 64)) & 1) != 0;
  };

  float4 S[4], N[4];
  int cur = -3;                  // whose state S holds: a token, -1 (the start) or nothing yet
  bool dead = is_dead(0);
  if (!dead) {
    fetch(sp[0], S);
    cur = sp[0];
  }
  for (int base = 0; base < n; base += kDtBlock) {
    const int m = min(kDtBlock, n - base);
    __syncthreads();
    for (int i = tid; i < m * 64; i += 256) {
      const int t = i >> 6, q4 = i & 63;
      const float* yt = a.y + (size_t)(first + base + t) * a.y_stride;
      const float4 x = __ldg(reinterpret_cast<const float4*>(yt + (q4 < 32 ? 0 : off_k) + g * kDnDim) + (q4 & 31));
      reinterpret_cast<float4*>(q4 < 32 ? sq[t] : sk[t])[q4 & 31] = x;
    }
    for (int i = tid; i < m * 32; i += 256)
      sv[i >> 5][i & 31] = __ldg(a.y + (size_t)(first + base + (i >> 5)) * a.y_stride + off_v + h * kDnDim + part * 32 + (i & 31));
    if (tid < m) {
      const float* yt = a.y + (size_t)(first + base + tid) * a.y_stride;
      sb[tid] = sigmoidf_(__ldg(yt + off_b + h));
      sa[tid] = sigmoidf_(-__ldg(yt + off_a + h));
    }
    __syncthreads();
    for (int t = warp; t < m; t += 8) {
      float4 q = reinterpret_cast<const float4*>(sq[t])[lane], k = reinterpret_cast<const float4*>(sk[t])[lane];
      const float rq = __frcp_rn(__fsqrt_rn(__fadd_rn(warp_sum(dot4(q, q)), 1e-6f)));
      const float rk = __frcp_rn(__fsqrt_rn(__fadd_rn(warp_sum(dot4(k, k)), 1e-6f)));
      reinterpret_cast<float4*>(sq[t])[lane] =
          make_float4(__fmul_rn(q.x, rq), __fmul_rn(q.y, rq), __fmul_rn(q.z, rq), __fmul_rn(q.w, rq));
      reinterpret_cast<float4*>(sk[t])[lane] =
          make_float4(__fmul_rn(k.x, rk), __fmul_rn(k.y, rk), __fmul_rn(k.z, rk), __fmul_rn(k.w, rk));
    }
    __syncthreads();

    for (int t = 0; t < m; ++t) {
      const int i = base + t;
      if (dead) (i < 64 ? dead_lo : dead_hi) |= 1ull << (i & 63);
      // the next token's start, unless it is this token's result or still in S
      const bool more = i + 1 < n;
      const bool next_dead = more && is_dead(i + 1);
      const int next = more && !next_dead ? sp[i + 1] : -3;
      const int after = dead ? cur : i;                    // whose state S holds after this token
      const bool load = next > -3 && next != after;
      if (load) fetch(next, N);
      float* op = a.o + (size_t)(first + i) * a.Hv * kDnDim + h * kDnDim + row0;
      if (!dead) {
        const float4 q = reinterpret_cast<const float4*>(sq[t])[lane], k = reinterpret_cast<const float4*>(sk[t])[lane];
        const float beta = sb[t], alpha = sa[t];
        const float ks = warp_sum4(dot4(S[0], k), dot4(S[1], k), dot4(S[2], k), dot4(S[3], k), lane);
        float* dst = a.snaps + (size_t)(first + i) * state_elems + mine;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float kS = __shfl_sync(0xffffffffu, ks, r * 8);
          const float coef = __fmul_rn(beta, __fsub_rn(sv[t][warp * 4 + r], __fmul_rn(alpha, kS)));
          S[r].x = __fmaf_rn(coef, k.x, __fmul_rn(alpha, S[r].x));
          S[r].y = __fmaf_rn(coef, k.y, __fmul_rn(alpha, S[r].y));
          S[r].z = __fmaf_rn(coef, k.z, __fmul_rn(alpha, S[r].z));
          S[r].w = __fmaf_rn(coef, k.w, __fmul_rn(alpha, S[r].w));
          *reinterpret_cast<float4*>(dst + (size_t)r * kDnDim) = S[r];
        }
        const float o = warp_sum4(dot4(S[0], q), dot4(S[1], q), dot4(S[2], q), dot4(S[3], q), lane);
        if ((lane & 7) == 0) op[lane >> 3] = o;
      } else if (lane < 4) {
        op[lane] = 0.f;
      }
      cur = after;
      if (load) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[r] = N[r];
        cur = next;
      }
      dead = next_dead;
    }
  }
}

}  // namespace qhl

using namespace qhl;

extern "C" int qhl_deltanet_tree(int Hk, int Hv, const float* y_dev, int n_rows, int n_batch, int max_nodes,
                                 const int* q_start_dev, const int* parent_dev, const float* states_dev, int n_states,
                                 const int* state_index_dev, float* snaps_dev, float* o_dev, void* stream) {
  const char* me = "qhl_deltanet_tree";
  if (!y_dev || !q_start_dev || !parent_dev || !states_dev || !state_index_dev || !snaps_dev || !o_dev)
    return verify_err(me, STAGE_E_ARG, "null pointer");
  if (Hk <= 0 || Hv <= 0 || Hv % Hk || Hv > 16384 || n_rows < 0 || n_states < 1)
    return verify_err(me, STAGE_E_ARG, "head, row or state count out of range");
  if (n_batch < 1 || n_batch > kMaxBatch || max_nodes < 1 || max_nodes > kMaxNodes)
    return verify_err(me, STAGE_E_ARG, "n_batch must be 1..2048 and max_nodes 1..128");
  if (!aligned16(y_dev) || !aligned16(states_dev) || !aligned16(snaps_dev) || !aligned16(o_dev))
    return verify_err(me, STAGE_E_ARG, "y_dev, states_dev, snaps_dev and o_dev must be 16-byte aligned");
  const int y_stride = 2 * Hk * kDnDim + Hv * kDnDim + 2 * Hv;
  if (y_stride % 4) return verify_err(me, STAGE_E_UNSUPPORTED, "row width must be a multiple of 4");
  const size_t se = (size_t)Hv * kDnDim * kDnDim;
  const float *s0 = states_dev, *s1 = states_dev + (size_t)n_states * se, *d0 = snaps_dev, *d1 = snaps_dev + (size_t)n_rows * se;
  if (s0 < d1 && d0 < s1) return verify_err(me, STAGE_E_ARG, "snaps_dev overlaps states_dev");
  if (n_rows == 0) return 0;
  DnTreeArgs a = {y_dev, y_stride, Hk, Hv, n_rows, max_nodes, n_states, q_start_dev, parent_dev, states_dev,
                  state_index_dev, snaps_dev, o_dev, nullptr};
  cudaError_t e = verify_error_word(&a.err);
  if (e != cudaSuccess) return verify_cuda_err(me, e);
  e = launch_ex(dn_tree_kernel, dim3(Hv * 4, n_batch), dim3(256), 0, static_cast<cudaStream_t>(stream), true, a);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}
