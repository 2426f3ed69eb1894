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
// walks the tree's living tokens in order; a warp keeps four rows of the last
// token's state in registers.  Where the next token starts from another state (a
// side branch), that state is requested before the current token's products, so
// that its load does not stand in the chain of tokens.  A lane reads back only
// what it has written itself.
//
// What the chain of tokens costs is the reduction of S . k over the warp.  The
// o = S . q of a token and the S . k of the next (both of the state between them)
// are reduced together: each of the first three butterfly steps halves the number
// of values a lane carries, so eight sums take 9 shuffles and 5 steps of latency
// instead of 40 and 10.  A sum's tree of additions is that of the plain butterfly
// (offsets 16, 8, 4, 2, 1), so a path's results have the same bits as the chained
// steps of qhl_deltanet_step.
//
// The inputs of 16 tokens at a time come by asynchronous copies, a block ahead (as
// loads in turn they took 3.3 us a block).  Measured: one tree of 16 tokens and 48
// heads 14.5 us for 54.5 MB (3.8 TB/s: the chain of tokens), eight ragged trees,
// 427 MB, 81 to 86 us (5.0 to 5.3 TB/s; a plain fill of 400 MB reaches 7.2 TB/s).
//
// No early start of the kernel behind this one (20.0 us against 24.3): its waiting
// CTAs, spread unevenly, would take this kernel's places.
#include <climits>

#include "launch.h"
#include "verify.cuh"

namespace qhl {

constexpr int kDtBlock = 16;   // tokens whose inputs are staged together
constexpr int kDtRows = 4;     // state rows per warp

struct DnTreeArgs {
  const float* y;
  int y_stride, Hk, Hv, n_rows, n_batch, max_nodes, n_states;
  const int* q_start;
  const int* parent;
  const float* states;
  const int* index;
  float* snaps;
  float* o;
  unsigned* err;
};

// Totals over the warp of 2 R values per lane (R = 4 or 8): lane l returns the
// total of value l / (16 / R).
template <int R>
QHL_DEV float warp_sum_of(float (&v)[2 * R], int lane) {
#pragma unroll
  for (int half = R, o = 16; o >= 1; half >>= 1, o >>= 1) {
    if (half == 0) {
      v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
      continue;
    }
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i)
      v[i] = __fadd_rn(up ? v[half + i] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[half + i], o));
  }
  return v[0];
}

// A 16-byte load that stays behind this thread's earlier stores: a state row may
// have been written by the same lane some tokens ago.
QHL_DEV float4 ld_after_stores(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// The tree of rank `rank` by number of tokens, largest first (ties in order), of at
// most 32: the CTAs of a large tree then do not start last.  A full warp calls it.
QHL_DEV int tree_by_size(const int* q_start, int n_batch, int rank) {
  const int lane = threadIdx.x & 31;
  const int size = lane < n_batch ? q_start[lane + 1] - q_start[lane] : INT_MIN;
  int before = 0;
  for (int i = 0; i < n_batch; ++i) {
    const int o = __shfl_sync(0xffffffffu, size, i);
    before += o > size || (o == size && i < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, lane < n_batch && before == rank)) - 1;
}

// One block of tokens' inputs, brought in by asynchronous copies.
template <int ROWS>
struct DtStage {
  float4 q[kDtBlock][32], k[kDtBlock][32];
  float v[kDtBlock][ROWS], b[kDtBlock], a[kDtBlock];
};

QHL_DEV void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
QHL_DEV void copy_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
QHL_DEV void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// R value rows per warp, ROWS per CTA.
template <int R, int ROWS, int PER_SM>
__global__ void __launch_bounds__(ROWS / R * 32, PER_SM) dn_tree_kernel(const DnTreeArgs a) {
  constexpr int WARPS = ROWS / R, THREADS = WARPS * 32, PARTS = kDnDim / ROWS, STEP = 16 / R;   // STEP: lanes per total
  constexpr int kStay = -4;   // the node's parent is the last living node: its state is in S
  __shared__ __align__(16) DtStage<ROWS> stage[2];
  __shared__ int sj[kMaxNodes];              // parents, then by doubling -1 (living) or -2 (padded)
  __shared__ short s_node[kMaxNodes + 1];    // the living nodes in order
  __shared__ short s_from[kMaxNodes + 1];    // where each starts: kStay, -1 (the cached state) or a node
  __shared__ unsigned s_alive[kMaxNodes / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x / PARTS, part = blockIdx.x % PARTS, row0 = part * ROWS + warp * R;
  const int g = h / (a.Hv / a.Hk);
  const int off_k = a.Hk * kDnDim, off_v = 2 * off_k, off_b = off_v + a.Hv * kDnDim, off_a = off_b + a.Hv;
  const size_t state_elems = (size_t)a.Hv * kDnDim * kDnDim;
  const size_t mine = ((size_t)h * kDnDim + row0) * kDnDim + 4 * lane;   // this lane's element of row 0 of its warp

  pdl_wait();
  int first, n;
  const int tree = a.n_batch > 1 && a.n_batch <= 32 ? tree_by_size(a.q_start, a.n_batch, blockIdx.y) : (int)blockIdx.y;
  int idx = a.index[tree];
  tree_rows(a.q_start, tree, a.n_rows, a.max_nodes, first, n, a.err);
  if (n == 0) return;

  auto stage_in = [&](DtStage<ROWS>& s, int base) {
    const int m = min(kDtBlock, n - base);
    const float* y = a.y + (size_t)(first + base) * a.y_stride;
    for (int i = tid; i < m * 64; i += THREADS) {
      const int t = i >> 6, c = i & 31;
      const bool is_k = i & 32;
      copy_async16(is_k ? &s.k[t][c] : &s.q[t][c], y + (size_t)t * a.y_stride + (is_k ? off_k : 0) + g * kDnDim + 4 * c);
    }
    for (int i = tid; i < m * ROWS; i += THREADS)
      copy_async4(&s.v[i / ROWS][i % ROWS], y + (size_t)(i / ROWS) * a.y_stride + off_v + h * kDnDim + part * ROWS + i % ROWS);
    if (tid < 2 * m) {
      const int t = tid >> 1;
      copy_async4(tid & 1 ? &s.a[t] : &s.b[t], y + (size_t)t * a.y_stride + (tid & 1 ? off_a : off_b) + h);
    }
  };
  int parent = tid < n ? a.parent[first + tid] : -2;
  stage_in(stage[0], 0);
  if (idx < -1 || idx >= a.n_states) {
    if (tid == 0) atomicOr(a.err, ERR_BAD_INDEX);
    idx = -1;
  }
  auto fetch = [&](int p, float4(&X)[R]) {
    const float* src = p >= 0 ? a.snaps + (size_t)(first + p) * state_elems : a.states + (size_t)max(idx, 0) * state_elems;
#pragma unroll
    for (int r = 0; r < R; ++r)
      X[r] = p >= 0 || idx >= 0 ? ld_after_stores(src + mine + (size_t)r * kDnDim) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 S[R], N[R];
  fetch(-1, S);                              // the first living node starts from the cached state

  // living nodes, and where their states come from
  static_assert(THREADS >= kMaxNodes, "a thread per node");
  if (tid < n && (parent < -2 || parent >= tid)) {
    atomicOr(a.err, ERR_BAD_INDEX);
    parent = -2;
  }
  bool living_node;
  if (n <= 32) {
    int j = parent;
    for (int step = 1; step < n; step <<= 1) {
      const int o = __shfl_sync(0xffffffffu, j, j & 31);
      if (j >= 0) j = o;
    }
    living_node = tid < n && j == -1;
  } else {
    if (tid < n) sj[tid] = parent;
    for (int step = 1; step < n; step <<= 1) {
      __syncthreads();
      int j = tid < n ? sj[tid] : -1;
      if (j >= 0) j = sj[j];
      __syncthreads();
      if (tid < n) sj[tid] = j;
    }
    living_node = tid < n && sj[tid] == -1;
  }
  if (warp < kMaxNodes / 32) {
    const unsigned m = __ballot_sync(0xffffffffu, living_node);
    if (lane == 0) s_alive[warp] = m;
  }
  __syncthreads();
  int living = 0;
  if (tid < kMaxNodes) {
    int before = 0, last = -1;               // living nodes before this one, and the last of them
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; ++w) {
      const unsigned m = s_alive[w], low = w < warp ? m : w == warp ? m & ((1u << lane) - 1) : 0u;
      before += __popc(low);
      if (low) last = 32 * w + 31 - __clz(low);
    }
    if (living_node) {
      s_node[before] = (short)tid;
      s_from[before] = (short)(parent == last ? kStay : parent);
    }
  }
#pragma unroll
  for (int w = 0; w < kMaxNodes / 32; ++w) living += __popc(s_alive[w]);
  if (living < n) {                          // padded nodes: their outputs are 0
    for (int i = tid; i < n * ROWS; i += THREADS) {
      const int x = i / ROWS;
      if (!(s_alive[x >> 5] >> (x & 31) & 1)) a.o[(size_t)(first + x) * a.Hv * kDnDim + h * kDnDim + part * ROWS + i % ROWS] = 0.f;
    }
  }
  if (tid == 0) {
    s_node[living] = kMaxNodes;              // behind every block
    s_from[living] = kStay;
  }

  float4 q_last = make_float4(0.f, 0.f, 0.f, 0.f);
  float* o_last = nullptr;                   // the last living node's outputs, still to be formed from S
  float* const snaps = a.snaps + (size_t)first * state_elems + mine;
  float* const out = a.o + (size_t)first * a.Hv * kDnDim + h * kDnDim + row0;
  int at = 0;
  for (int base = 0; base < n; base += kDtBlock) {
    const int m = min(kDtBlock, n - base);
    DtStage<ROWS>& s = stage[base / kDtBlock & 1];
    copy_async_wait();
    __syncthreads();
    for (int t = warp; t < m; t += WARPS) {
      float4 q = s.q[t][lane], k = s.k[t][lane];
      const float rq = __frcp_rn(__fsqrt_rn(__fadd_rn(warp_sum(dot4(q, q)), 1e-6f)));
      const float rk = __frcp_rn(__fsqrt_rn(__fadd_rn(warp_sum(dot4(k, k)), 1e-6f)));
      s.q[t][lane] = make_float4(__fmul_rn(q.x, rq), __fmul_rn(q.y, rq), __fmul_rn(q.z, rq), __fmul_rn(q.w, rq));
      s.k[t][lane] = make_float4(__fmul_rn(k.x, rk), __fmul_rn(k.y, rk), __fmul_rn(k.z, rk), __fmul_rn(k.w, rk));
      if (lane == 0) s.b[t] = sigmoidf_(s.b[t]);
      if (lane == 1) s.a[t] = sigmoidf_(-s.a[t]);
    }
    __syncthreads();
    if (base + kDtBlock < n) stage_in(stage[(base / kDtBlock + 1) & 1], base + kDtBlock);

    int i = s_node[at], from = s_from[at];
    while (i < base + m) {
      const int t = i - base;
      const float4 q = s.q[t][lane], k = s.k[t][lane];
      const float beta = s.b[t], alpha = s.a[t];
      const int next = s_node[at + 1], next_from = s_from[at + 1];
      float val[R];
#pragma unroll
      for (int r = 0; r < R; ++r) val[r] = s.v[t][warp * R + r];
      float v[2 * R];
#pragma unroll
      for (int r = 0; r < R; ++r) v[R + r] = dot4(S[r], q_last);
      if (from != kStay) {
#pragma unroll
        for (int r = 0; r < R; ++r) S[r] = N[r];
      }
      if (next_from != kStay) fetch(next_from, N);
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = dot4(S[r], k);
      const float tot = warp_sum_of<R>(v, lane);
      if (o_last && lane >= 16 && lane % STEP == 0) o_last[(lane - 16) / STEP] = tot;
      float* dst = snaps + (size_t)i * state_elems;
      const float2 alpha2 = make_float2(alpha, alpha);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float kS = __shfl_sync(0xffffffffu, tot, r * STEP);
        const float coef = __fmul_rn(beta, __fsub_rn(val[r], __fmul_rn(alpha, kS)));
        const float2 c2 = make_float2(coef, coef);   // two elements at a time, each rounded as by itself
        const float2 lo = ffma2(c2, make_float2(k.x, k.y), __fmul2_rn(alpha2, make_float2(S[r].x, S[r].y)));
        const float2 hi = ffma2(c2, make_float2(k.z, k.w), __fmul2_rn(alpha2, make_float2(S[r].z, S[r].w)));
        S[r] = make_float4(lo.x, lo.y, hi.x, hi.y);
        *reinterpret_cast<float4*>(dst + (size_t)r * kDnDim) = S[r];
      }
      q_last = q;
      o_last = out + (size_t)i * a.Hv * kDnDim;
      ++at;
      i = next;
      from = next_from;
    }
  }
  if (o_last) {
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[R + r] = dot4(S[r], q_last);
      v[r] = 0.f;
    }
    const float tot = warp_sum_of<R>(v, lane);
    if (lane >= 16 && lane % STEP == 0) o_last[(lane - 16) / STEP] = tot;
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
  DnTreeArgs a = {y_dev, y_stride, Hk, Hv, n_rows, n_batch, max_nodes, n_states, q_start_dev, parent_dev, states_dev,
                  state_index_dev, snaps_dev, o_dev, nullptr};
  cudaError_t e = verify_error_word(&a.err);
  if (e != cudaSuccess) return verify_cuda_err(me, e);
  // Few CTAs: 16 rows each, spread more evenly, with all the registers that the
  // kernel wants (one tree of 16 tokens, 48 heads: 14.2 us, with 32 rows 16.9 us).
  // Many: 32 rows and registers for three CTAs per SM (eight such trees: 79.4 us,
  // with two per SM 81.7 us, with 16 rows 84.4 us).
  const bool few = (long long)Hv * 4 * n_batch <= 2 * 148;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = few ? launch_ex(dn_tree_kernel<kDtRows, 16, 4>, dim3(Hv * 8, n_batch), dim3(128), 0, s, true, a)
          : launch_ex(dn_tree_kernel<kDtRows, 32, 3>, dim3(Hv * 4, n_batch), dim3(256), 0, s, true, a);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}
