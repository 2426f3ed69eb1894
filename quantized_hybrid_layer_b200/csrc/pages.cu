// The pages of a KV cache: free, fork, extend and commit, and the error word of
// the verify operators.
//
// The only state is the caller's: the page table, the lengths, the pages held
// and a count of holders per page.  There is no list of free pages to keep in
// step with them: a free page is one that nobody holds, and extend takes those
// of the lowest numbers by counting over refs, which makes every call's result
// a function of its inputs alone (counts change by integer atomics, whose order
// does not matter).
//
// free and fork: one CTA per request, latency-bound (a table row each).
// extend: one CTA plans (a prefix sum over the requests' needs and two passes
// over refs, 4 bytes per page), a second grid copies the shared last pages'
// committed rows; bound by those rows, read and written once.  commit: one CTA
// per (tree, layer, K or V), 16-byte moves, bound by the accepted rows.
// Measured: 96 branches of 12 sequences freed, forked and extended, 16 layers of
// 4 heads x 256: 67.3 us, 6.7 TB/s of copied rows; 2 branches of one 12.5 us, four
// launches; 8 accepted paths of up to 16 tokens 5.7 us.
// Every kernel is launched as a programmatic dependent of the one before it on
// the stream and waits for that one's end before it reads anything, which hides
// most of a launch (about 1 us of a chain of short calls).
#include <mutex>

#include "launch.h"
#include "verify.cuh"

namespace qhl {

// ------------------------------------------------------------- error word --

static __device__ unsigned g_verify_err[4];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_err_mu;
unsigned* g_err_addr[kMaxDevices] = {};
}  // namespace

cudaError_t verify_error_word(unsigned** word) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_err_mu);
  if (!g_err_addr[dev]) {
    void* p = nullptr;
    if ((e = cudaGetSymbolAddress(&p, g_verify_err)) != cudaSuccess) return e;
    g_err_addr[dev] = static_cast<unsigned*>(p);
  }
  *word = g_err_addr[dev];
  return cudaSuccess;
}

unsigned verify_take_error(int dev) {
  unsigned* p = nullptr;
  {
    std::lock_guard<std::mutex> lk(g_err_mu);
    if (dev >= 0 && dev < kMaxDevices) p = g_err_addr[dev];
  }
  unsigned w = 0;
  if (!p || cudaMemcpy(&w, p, sizeof(w), cudaMemcpyDeviceToHost) != cudaSuccess) return 0;
  if (w) cudaMemset(p, 0, sizeof(w));
  return w;
}

int check_pages(const char* me, const qhl_kv_pages* kv) {
  if (!kv) return verify_err(me, STAGE_E_ARG, "null cache");
  if (!kv->k_dev || !kv->v_dev || !kv->table_dev || !kv->len_dev || !kv->held_dev || !kv->refs_dev)
    return verify_err(me, STAGE_E_ARG, "the cache has a null pointer");
  if (kv->dtype != QHL_F16 && kv->dtype != QHL_BF16) return verify_err(me, STAGE_E_UNSUPPORTED, "the cache must be f16 or bf16");
  if (kv->dim != 64 && kv->dim != 128 && kv->dim != 256) return verify_err(me, STAGE_E_UNSUPPORTED, "dim must be 64, 128 or 256");
  const int P = kv->page_rows;
  if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256)
    return verify_err(me, STAGE_E_UNSUPPORTED, "page_rows must be 16, 32, 64, 128 or 256");
  if (kv->n_layers < 1 || kv->n_layers > 4096 || kv->n_pages < 1 || kv->n_pages > (1 << 26) || kv->kv_heads < 1 ||
      kv->kv_heads > 256 || kv->n_seqs < 1 || kv->max_pages < 1)
    return verify_err(me, STAGE_E_ARG, "a count of the cache is out of range");
  if (!aligned16(kv->k_dev) || !aligned16(kv->v_dev) || kv->stride_layer % 8 || kv->stride_page % 8 || kv->stride_head % 8 ||
      kv->stride_row % 8)
    return verify_err(me, STAGE_E_ARG, "the cache's bases must be 16-byte aligned, its strides multiples of 8");
  const long long most = 1LL << 38;   // a tensor map's strides are below 2^40 bytes
  if (kv->stride_row < kv->dim || kv->stride_row > most || kv->stride_head < kv->dim || kv->stride_head > most ||
      kv->stride_page < kv->dim || kv->stride_page > most || (kv->n_layers > 1 && kv->stride_layer < kv->dim))
    return verify_err(me, STAGE_E_ARG, "a stride of the cache is shorter than a row, or too long");
  return 0;
}

// ---------------------------------------------------------- shared helpers --

struct PagesView {
  uint8_t* k;
  uint8_t* v;
  int n_layers, n_pages, heads, rows, vshift;  // a row is 1 << vshift units of 16 bytes
  long long s_layer, s_page, s_head, s_row;    // bytes
  int n_seqs, max_pages;
  int *table, *len, *held, *refs;
  unsigned* err;
};

static PagesView view_of(const qhl_kv_pages* kv, unsigned* err) {
  PagesView p;
  p.k = static_cast<uint8_t*>(kv->k_dev);
  p.v = static_cast<uint8_t*>(kv->v_dev);
  p.n_layers = kv->n_layers;
  p.n_pages = kv->n_pages;
  p.heads = kv->kv_heads;
  p.rows = kv->page_rows;
  p.vshift = kv->dim == 256 ? 5 : kv->dim == 128 ? 4 : 3;
  p.s_layer = kv->stride_layer * 2;
  p.s_page = kv->stride_page * 2;
  p.s_head = kv->stride_head * 2;
  p.s_row = kv->stride_row * 2;
  p.n_seqs = kv->n_seqs;
  p.max_pages = kv->max_pages;
  p.table = kv->table_dev;
  p.len = kv->len_dev;
  p.held = kv->held_dev;
  p.refs = kv->refs_dev;
  p.err = err;
  return p;
}

QHL_DEV int held_of(const PagesView& p, int s) {
  const int h = p.held[s];
  if (h < 0 || h > p.max_pages) {
    atomicOr(p.err, ERR_BAD_INDEX);
    return 0;
  }
  return h;
}

// Whether seq[i] was already named by an earlier request (all threads of the
// CTA call it and get the answer).
QHL_DEV bool named_before(const int* seq, int i, int s) {
  bool dup = false;
  for (int j = threadIdx.x; j < i; j += blockDim.x) dup |= seq[j] == s;
  return __syncthreads_or(dup);
}

// -------------------------------------------------------------------- free --

__global__ void __launch_bounds__(128) pages_free_kernel(const PagesView p, const int* seq, int* status) {
  if (threadIdx.x == 0) pdl_launch();
  pdl_wait();
  const int i = blockIdx.x, s = seq[i];
  const bool dup = named_before(seq, i, s);
  if (s < 0 || s >= p.n_seqs || dup) {
    if (threadIdx.x == 0) status[i] = STAGE_E_ARG;
    return;
  }
  const int held = held_of(p, s);
  int* row = p.table + (size_t)s * p.max_pages;
  for (int j = threadIdx.x; j < held; j += 128) {
    const int page = row[j];
    if (page >= 0 && page < p.n_pages)
      atomicSub(p.refs + page, 1);
    else
      atomicOr(p.err, ERR_BAD_INDEX);
    row[j] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.held[s] = 0;
    p.len[s] = 0;
    status[i] = STAGE_OK;
  }
}

// -------------------------------------------------------------------- fork --

__global__ void __launch_bounds__(128) pages_fork_kernel(const PagesView p, int n, const int* src, const int* dst, int* status) {
  if (threadIdx.x == 0) pdl_launch();
  pdl_wait();
  const int i = blockIdx.x, s = src[i], d = dst[i];
  bool again = false;   // dst named before, or src a dst of this call
  for (int j = threadIdx.x; j < n; j += 128) {
    const int o = dst[j];
    again |= (j < i && o == d) || o == s;
  }
  again = __syncthreads_or(again);
  int rc = STAGE_OK, len = 0, pages = 0;
  if (s < 0 || s >= p.n_seqs || d < 0 || d >= p.n_seqs || again) {
    rc = STAGE_E_ARG;
  } else {
    len = p.len[s];
    pages = len > 0 ? (len - 1) / p.rows + 1 : 0;
    if (p.held[d] != 0 || p.len[d] != 0 || len < 0 || pages > held_of(p, s)) rc = STAGE_E_STATE;
  }
  __syncthreads();   // every thread has read dst's held and len
  if (rc == STAGE_OK) {
    for (int j = threadIdx.x; j < pages; j += 128) {
      const int page = p.table[(size_t)s * p.max_pages + j];
      if (page >= 0 && page < p.n_pages)
        atomicAdd(p.refs + page, 1);
      else
        atomicOr(p.err, ERR_BAD_INDEX);
      p.table[(size_t)d * p.max_pages + j] = page;
    }
    if (threadIdx.x == 0) {
      p.held[d] = pages;
      p.len[d] = len;
    }
  }
  if (threadIdx.x == 0) status[i] = rc;
}

// ------------------------------------------------------------------ extend --

// A page whose first `rows` rows of every head and layer go to another page.
struct PageCopy {
  int from, to, rows, pad;
};

// Sum of v over the threads up to this one; `total`: over all.  1024 threads.  v is at
// most 2^26 + 1, more than a pool's pages.  A sum above kScanMost comes out as some
// number of at least kScanMost: a warp's sum fits 32 bits, and so do 32 of kScanMost.
constexpr unsigned kScanMost = (1u << 27) - 1;
QHL_DEV int block_scan(int v, unsigned* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  inc = min(inc, kScanMost);
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    unsigned w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = min(w, kScanMost);
  }
  __syncthreads();
  total = warp_sums[31];
  return inc + (warp ? warp_sums[warp - 1] : 0);
}

// Requests i = thread.  A request needs `copied` (0 or 1) + `fresh` pages; the
// free page of rank f goes to the request whose range of the prefix sum holds f.
__global__ void __launch_bounds__(1024) pages_extend_kernel(const PagesView p, int n, const int* seq, const int* add, int* status,
                                                            PageCopy* copies) {
  __shared__ int s_seq[kMaxRequests], s_last[kMaxRequests], s_end[kMaxRequests], s_at[kMaxRequests], s_copied[kMaxRequests],
      s_held[kMaxRequests];
  __shared__ unsigned s_warp[32];
  const int tid = threadIdx.x, P = p.rows;
  if (tid == 0) pdl_launch();
  pdl_wait();
  const int s = tid < n ? seq[tid] : -1;
  const int more = tid < n ? add[tid] : 0;
  s_seq[tid] = s;
  __syncthreads();
  int rc = STAGE_OK, len = 0, held = 0, want = 0, last_at = 0, last = -1, refs = 0;
  if (tid < n) {
    bool dup = false;
    for (int j = 0; j < tid; ++j) dup |= s_seq[j] == s;
    if (s < 0 || s >= p.n_seqs || dup || more < 0) {
      rc = STAGE_E_ARG;
    } else {
      len = p.len[s];
      held = held_of(p, s);
      const long long rows = (long long)len + more;
      const long long pages = (rows + P - 1) / P;
      if (len < 0 || (long long)held * P < len)
        rc = STAGE_E_STATE;
      else if (pages > p.max_pages)
        rc = STAGE_E_ARG;
      else {
        want = more ? (int)pages : 0;
        last_at = len / P;
        const int* row = p.table + (size_t)s * p.max_pages;
        for (int j = last_at; j < min(held, want); ++j) {
          const int page = row[j];
          const int r = page >= 0 && page < p.n_pages ? p.refs[page] : 0;
          if (r < 1) {                       // not a page that this sequence can hold
            atomicOr(p.err, ERR_BAD_INDEX);
            rc = STAGE_E_STATE;
          } else if (j == last_at) {
            last = page;
            refs = r;
          } else if (r > 1) {
            rc = STAGE_E_STATE;
          }
        }
        if (rc != STAGE_OK) last = -1;
      }
    }
  }
  s_last[tid] = last;
  __syncthreads();
  int copied = 0, fresh = 0;
  if (tid < n && rc == STAGE_OK) {
    if (last >= 0) {
      int before = 0;                        // earlier requests that let go of this page
      for (int j = 0; j < tid; ++j) before += s_last[j] == last;
      copied = refs - before > 1;
    }
    fresh = max(0, want - held);
  }
  const int need = min(copied + fresh, p.n_pages + 1);   // the pool's size is not enough for either
  int total;
  s_end[tid] = block_scan(need, s_warp, total);
  s_at[tid] = last_at;                       // table index of the page that is copied
  s_copied[tid] = copied;
  s_held[tid] = held;
  // Free pages in all, as far as they are needed, and then their hand-out in
  // ascending order.  A thread looks at 16 consecutive pages of a sweep; a pool of
  // one sweep is read once for both.
  constexpr int kSweep = 1024 * 16;
  auto free_of = [&](long long base) {       // a bit for each free page of the thread's 16
    unsigned bits = 0;
    const long long p0 = base + tid * 16;
    int r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = p0 + j < p.n_pages ? p.refs[p0 + j] : 1;
#pragma unroll
    for (int j = 0; j < 16; ++j) bits |= (r[j] == 0 ? 1u : 0u) << j;
    return bits;
  };
  int have = 0, sweep_free = 0;
  unsigned bits = 0;
  int rank = 0;
  for (long long base = 0; base < p.n_pages && have < total; base += kSweep) {
    bits = free_of(base);
    rank = block_scan(__popc(bits), s_warp, sweep_free) - __popc(bits);
    have += sweep_free;
  }
  __syncthreads();
  if (tid < n && rc == STAGE_OK && s_end[tid] > have && (need > 0 || refs > 1)) rc = STAGE_E_OOM;
  const bool ok = tid < n && rc == STAGE_OK;
  int given = 0;
  for (long long base = 0; base < p.n_pages && given < min(have, total); base += kSweep) {
    if (p.n_pages > kSweep) {
      bits = free_of(base);
      rank = block_scan(__popc(bits), s_warp, sweep_free) - __popc(bits);
    }
    int f = given + rank;
    for (unsigned left = bits; left && f < total; left &= left - 1, ++f) {
      const int pg = (int)(base + tid * 16) + __ffs(left) - 1;
      int lo = 0, hi = n - 1;                // the first request whose range ends beyond f
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_end[mid] > f) hi = mid;
        else lo = mid + 1;
      }
      if (s_end[lo] > have) break;           // not granted, nor are those behind it
      const int at = f - (lo ? s_end[lo - 1] : 0);
      int* row = p.table + (size_t)s_seq[lo] * p.max_pages;
      if (s_copied[lo] && at == 0) {
        copies[lo] = PageCopy{s_last[lo], pg, 0, 0};
        row[s_at[lo]] = pg;
      } else {
        row[s_held[lo] + at - s_copied[lo]] = pg;
      }
      p.refs[pg] = 1;
    }
    given += sweep_free;
    if (p.n_pages > kSweep) __syncthreads();
  }
  __syncthreads();
  if (tid < n) {
    if (ok && copied) {
      atomicSub(p.refs + last, 1);
      copies[tid].rows = len % P;
    } else {
      copies[tid] = PageCopy{0, 0, 0, 0};
    }
    if (ok && fresh) p.held[s] = held + fresh;
    status[tid] = rc;
  }
}

// One CTA per (layer, K or V, head) and request.
__global__ void __launch_bounds__(128) pages_copy_kernel(const PagesView p, const PageCopy* copies) {
  if (threadIdx.x == 0) pdl_launch();
  pdl_wait();
  const PageCopy c = copies[blockIdx.y];
  const int head = blockIdx.x % p.heads, z = blockIdx.x / p.heads;
  uint8_t* base = (z & 1 ? p.v : p.k) + (long long)(z >> 1) * p.s_layer + (long long)head * p.s_head;
  const uint8_t* from = base + (long long)c.from * p.s_page;
  uint8_t* to = base + (long long)c.to * p.s_page;
  const int units = c.rows << p.vshift, mask = (1 << p.vshift) - 1;
  // eight loads in flight per thread
  for (int u0 = threadIdx.x; u0 < units; u0 += 128 * 8) {
    uint4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int u = u0 + 128 * j;
      if (u < units) x[j] = __ldcs(reinterpret_cast<const uint4*>(from + (long long)(u >> p.vshift) * p.s_row) + (u & mask));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int u = u0 + 128 * j;
      if (u < units) *(reinterpret_cast<uint4*>(to + (long long)(u >> p.vshift) * p.s_row) + (u & mask)) = x[j];
    }
  }
}

// ------------------------------------------------------------------ commit --

struct CommitArgs {
  const int* seq;
  const int* q_start;
  const int* path;
  int path_stride, n_rows;
  const int* n_accepted;
  const int* pos;
  const uint8_t* k_new;
  const uint8_t* v_new;
  long long s_layer, s_row;   // bytes
  int* status;
};

// One CTA per (tree, layer, K or V); each checks the tree's request itself, so
// that none waits for another.  len is written by one of them while others may
// read it: either value passes the same test.
__global__ void __launch_bounds__(256) pages_commit_kernel(const PagesView p, const CommitArgs a) {
  __shared__ int s_from[kMaxNodes];
  __shared__ long long s_to[kMaxNodes];   // byte offset of page and row
  __shared__ int s_arg, s_state;         // whether a thread found a bad argument, a wrong state
  const int b = blockIdx.x, tid = threadIdx.x, layer = blockIdx.y >> 1, P = p.rows;
  if (tid == 0) pdl_launch();
  pdl_wait();
  // all that does not depend on another load goes out at once
  const int s = a.seq[b], acc = a.n_accepted[b], pos = a.pos[b];
  const int node = tid < min(a.path_stride, kMaxNodes) ? a.path[(size_t)b * a.path_stride + tid] : -1;
  int first, n;
  tree_rows(a.q_start, b, a.n_rows, kMaxNodes, first, n, p.err);
  if (tid == 0) s_arg = s_state = 0;
  const bool dup = named_before(a.seq, b, s);
  int rc = STAGE_OK;
  if (s < 0 || s >= p.n_seqs || dup || acc < 0 || acc > min(a.path_stride, kMaxNodes) || pos < 0) {
    rc = STAGE_E_ARG;
  } else if (pos > *reinterpret_cast<volatile int*>(p.len + s)) {
    rc = STAGE_E_ARG;
  } else if ((long long)pos + acc > (long long)held_of(p, s) * P) {
    rc = STAGE_E_STATE;
  } else if (tid < acc) {
    const int page = p.table[(size_t)s * p.max_pages + (pos + tid) / P];
    if (node < 0 || node >= n) {
      rc = STAGE_E_ARG;
    } else if (page < 0 || page >= p.n_pages || p.refs[page] != 1) {
      rc = STAGE_E_STATE;
    } else {
      s_from[tid] = first + node;
      s_to[tid] = (long long)page * p.s_page + (long long)((pos + tid) % P) * p.s_row;
    }
  }
  if (rc == STAGE_E_ARG) s_arg = 1;
  if (rc == STAGE_E_STATE) s_state = 1;
  __syncthreads();
  rc = s_arg ? STAGE_E_ARG : s_state ? STAGE_E_STATE : STAGE_OK;
  if (blockIdx.y == 0 && tid == 0) {
    a.status[b] = rc;
    if (rc == STAGE_OK) p.len[s] = pos + acc;
  }
  if (rc != STAGE_OK) return;
  const uint8_t* src = (blockIdx.y & 1 ? a.v_new : a.k_new) + (long long)layer * a.s_layer;
  uint8_t* dst = (blockIdx.y & 1 ? p.v : p.k) + (long long)layer * p.s_layer;
  const int per_row = p.heads << p.vshift, units = acc * per_row;
  for (int u0 = tid; u0 < units; u0 += 256 * 8) {
    uint4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int u = u0 + 256 * j, r = u / per_row;
      if (u < units) x[j] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)s_from[r] * a.s_row) + (u - r * per_row));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int u = u0 + 256 * j, r = u / per_row, w = u - r * per_row, head = w >> p.vshift;
      if (u < units) *(reinterpret_cast<uint4*>(dst + s_to[r] + (long long)head * p.s_head) + (w - (head << p.vshift))) = x[j];
    }
  }
}

static int check_requests(const char* me, const qhl_kv_pages* kv, int n, bool ok) {
  int rc = check_pages(me, kv);
  if (rc) return rc;
  if (n < 1 || n > kMaxRequests) return verify_err(me, STAGE_E_ARG, "the number of requests must be 1..1024");
  return ok ? 0 : verify_err(me, STAGE_E_ARG, "null pointer");
}

static int open_pages(const char* me, const qhl_kv_pages* kv, PagesView* p) {
  unsigned* err = nullptr;
  cudaError_t e = verify_error_word(&err);
  if (e != cudaSuccess) return verify_cuda_err(me, e);
  *p = view_of(kv, err);
  return 0;
}

}  // namespace qhl

using namespace qhl;

extern "C" {

int qhl_pages_free(const qhl_kv_pages* kv, int n, const int* seq_dev, int* status_dev, void* stream) {
  const char* me = "qhl_pages_free";
  PagesView p;
  int rc = check_requests(me, kv, n, seq_dev && status_dev);
  if (!rc) rc = open_pages(me, kv, &p);
  if (rc) return rc;
  const cudaError_t e = launch_ex(pages_free_kernel, dim3(n), dim3(128), 0, static_cast<cudaStream_t>(stream), true, p, seq_dev, status_dev);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}

int qhl_pages_fork(const qhl_kv_pages* kv, int n, const int* src_dev, const int* dst_dev, int* status_dev, void* stream) {
  const char* me = "qhl_pages_fork";
  PagesView p;
  int rc = check_requests(me, kv, n, src_dev && dst_dev && status_dev);
  if (!rc) rc = open_pages(me, kv, &p);
  if (rc) return rc;
  const cudaError_t e =
      launch_ex(pages_fork_kernel, dim3(n), dim3(128), 0, static_cast<cudaStream_t>(stream), true, p, n, src_dev, dst_dev, status_dev);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}

int qhl_pages_extend(const qhl_kv_pages* kv, int n, const int* seq_dev, const int* add_dev, int* status_dev,
                     void* workspace_dev, size_t workspace_bytes, void* stream) {
  const char* me = "qhl_pages_extend";
  PagesView p;
  int rc = check_requests(me, kv, n, seq_dev && add_dev && status_dev && workspace_dev);
  if (rc) return rc;
  if (!aligned16(workspace_dev) || workspace_bytes < (size_t)n * sizeof(PageCopy))
    return verify_err(me, STAGE_E_ARG, "the workspace must be 16-byte aligned and hold 16 bytes per request");
  if ((rc = open_pages(me, kv, &p))) return rc;
  PageCopy* copies = static_cast<PageCopy*>(workspace_dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_ex(pages_extend_kernel, dim3(1), dim3(1024), 0, s, true, p, n, seq_dev, add_dev, status_dev, copies);
  if (e == cudaSuccess)
    e = launch_ex(pages_copy_kernel, dim3(p.n_layers * 2 * p.heads, n), dim3(128), 0, s, true, p, (const PageCopy*)copies);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}

int qhl_pages_commit(const qhl_kv_pages* kv, int n_batch, int n_rows, const int* seq_dev, const int* q_start_dev,
                     const int* path_dev, int path_stride, const int* n_accepted_dev, const int* pos_dev,
                     const void* k_new_dev, const void* v_new_dev, long long new_stride_layer, long long new_stride_row,
                     int* status_dev, void* stream) {
  const char* me = "qhl_pages_commit";
  PagesView p;
  int rc = check_requests(me, kv, n_batch,
                          seq_dev && q_start_dev && path_dev && n_accepted_dev && pos_dev && k_new_dev && v_new_dev && status_dev);
  if (rc) return rc;
  if (n_rows < 0 || path_stride < 1) return verify_err(me, STAGE_E_ARG, "n_rows or path_stride out of range");
  if (!aligned16(k_new_dev) || !aligned16(v_new_dev) || new_stride_layer % 8 || new_stride_row % 8 ||
      new_stride_row < (long long)kv->kv_heads * kv->dim || (kv->n_layers > 1 && new_stride_layer < new_stride_row))
    return verify_err(me, STAGE_E_ARG, "new rows must be 16-byte aligned, with strides that hold their heads");
  if ((rc = open_pages(me, kv, &p))) return rc;
  CommitArgs a = {seq_dev, q_start_dev, path_dev, path_stride, n_rows, n_accepted_dev, pos_dev,
                  static_cast<const uint8_t*>(k_new_dev), static_cast<const uint8_t*>(v_new_dev), new_stride_layer * 2,
                  new_stride_row * 2, status_dev};
  const cudaError_t e =
      launch_ex(pages_commit_kernel, dim3(n_batch, p.n_layers * 2), dim3(256), 0, static_cast<cudaStream_t>(stream), true, p, a);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}

}  // extern "C"
