// qhl_tree_attention: attention of trees of drafted tokens over a paged cache.
//
// For a query row q (token i, head j, KV head j / G) over the keys it sees:
//     s = scale * q . k,   out = sum exp(s - m) v / sum exp(s - m),   m a running maximum,
// in one pass over the keys, a tile of KT keys at a time:
//     S = Q K^T (f32 in tensor memory), p = 2^(c S - c m) with c = scale / ln 2,
//     O += p V (f32 in tensor memory), l += sum p.
// m is raised only when a tile's maximum exceeds it by more than 2^8 in p (the
// result does not depend on m), so O is seldom rescaled.  p is rounded to the
// cache's type for the product, half a step each; l adds the unrounded p.  For f16
// p is 2^6 larger, 2^14 at most, so that the weights of a long tail are not lost in
// f16's subnormal numbers.
//
// What bounds it: for few query rows the bytes of K and V, for many the products.
// Both products run on tcgen05 with M = 128 query rows: all tokens x query heads of
// one KV head, so a cache row is read once for all of them; a tree with more rows
// takes several M tiles, whose CTAs walk the same tiles side by side.  A tile of 64
// keys x 256 dimensions (128 x 128, 128 x 64) is one 32 KB (16 KB) slot of a 192 KB
// ring filled by TMA.  Q lies in tensor memory, which frees 64 KB of shared memory
// for that ring (four slots instead of six: 214 us instead of 189 us for 4 trees of
// 16 tokens over 65536 rows), and so does p, over the S it came from, as the A
// operand of the second product.
//
// Measured (B200, passes one after another; 6543 GB/s and 1624 TFLOP/s are the
// measured peaks): 16 tokens of 24 heads over 262001 rows 193 us, 5.6 TB/s; 32 single
// tokens over 16384 rows each 336 us, 6.4 TB/s; 24 trees of 12 tokens over 16384 rows
// at 128 dimensions 288 us, 5.6 TB/s (253 us after a pause); 64 tokens over 4 x 65536
// rows 460 us, 0.90 PFLOP/s (395 us after a pause), where the power cap holds the
// clock at 1.5 to 1.65 GHz and a tile of 64 keys takes about 1700 cycles (S: 16 MMAs
// of N = 64 that cost as much as N = 128 would; a second S of 128 columns does not fit
// beside O and Q).
//
// Work split: the CTAs take equal runs of key tiles (see "planning"), from lengths
// that they read on the device, so one captured graph serves every length.  What is
// split leaves (O, m, l) in the workspace and a second kernel joins it in the order
// of the runs, so results do not depend on timing.
//
// Roles of a CTA (one per SM): warps 0-7 softmax (warp w: the 32 rows of lane
// quarter w % 4 and half w / 4 of the keys; O's columns are halved the same way),
// warp 8 TMA, warp 9 issues S, warp 10 issues O, warp 11 ancestor masks and the
// tiles that need care.  Rows of V that nobody may see (beyond the sequence, beyond
// the tree, in pages of garbage) are zeroed in shared memory, since 0 * NaN is
// NaN; a drafted V row's infinities and NaN are taken out the same way and put
// back, at the end, into the rows of the tokens that see them.
#include <algorithm>
#include <mutex>

#include "launch.h"
#include "tc5_f16.cuh"
#include "verify.cuh"

namespace qhl {

// ------------------------------------------------------------------- shapes --

constexpr int kTaThreads = 384;
constexpr uint32_t kTaWait = 1u << 22;   // tries of a wait before it is given up (seconds)
constexpr int kTaRows = 128;          // rows of an M tile
constexpr int kTaOwnPlan = 256;       // trees up to which every CTA plans for itself
constexpr int kTaStart = 2;           // tiles' time that an item's start and end take

template <int DIM>
struct TaShape {
  static constexpr int KT = DIM == 256 ? 64 : 128;     // keys per tile
  static constexpr int CH = DIM / 64;                  // 128-byte chunks of a row
  static constexpr int SLOT = KT * DIM * 2;            // bytes of a ring slot
  static constexpr int NS = DIM == 64 ? 12 : 6;        // 192 KB in flight or in use
  static constexpr int SMEM = 1024 + NS * SLOT;        // 1024: room to align the swizzle atoms
  // tensor-memory columns: O, Q (two elements a column), S of even and odd tiles
  static constexpr uint32_t S0 = 256, Q0 = DIM == 256 ? 384 : DIM;
};

// One tree as the plan sees it.
struct TaSeq {
  int row0, n, seq, ctx;
  int tiles;         // key tiles, of the cache and of the drafts
  int nm;            // M tiles per KV head
  int base;          // its first unit of work
  int pad;
};

// The whole plan, for the join and for large batches.
struct TaHead {
  int units;
  int runs;          // none of them empty
  int heads, tiles;  // KV heads and M tiles of a group of CTAs
};
constexpr long long kTaMostUnits = 1LL << 30;

struct TaArgs {
  CUtensorMap k, v;            // cache pages
  CUtensorMap kn, vn;          // drafted rows
  int box, dbox;               // rows per TMA box of a page / of drafted rows
  int box_shift, page_shift;   // log2 of box and of the rows of a page
  int n_pages, max_pages, n_seqs;
  int Hkv, G, n_rows, n_batch, max_nodes;
  const int* table;
  const int* len;
  const int* seq;
  const int* q_start;
  const int* parent;
  const void* q;
  long long q_stride;
  const void* v_new;
  long long new_stride;
  void* out;
  long long out_stride;
  float* lse;
  float c;                     // scale / ln 2
  TaHead* head;
  TaSeq* seqs;
  float2* pml;                 // per partial row: c m, l
  float* po;                   // per slot: O as [DIM / 4][slot_rows] float4
  int slot_rows;               // partial rows of a slot: an M tile's, or all there can be
  int grid;
  unsigned* err;
};

// ------------------------------------------------------------------ planning --
//
// The CTAs take equal runs of the work, so that all end together whatever the
// lengths.  Work is counted in key tiles, with kTaStart more for an item's start
// and end.  A group of CTAs shares a run: CTA j of it takes KV head and M tile j of
// the same keys, so that rows that lie together in memory (the heads of a page,
// the tiles that several M tiles need) are read at the same time, which HBM and L2
// reward (4 heads, 4 x 65536 rows: 166 us with a run per CTA, 160 us in groups).
// A segment is the key tiles of a tree for one group of heads; segments stand one
// after the other.
//   heads: the KV heads of a group, the most that divide the heads and leave at
//     most 5% of the CTAs without a group.
//   M tiles: as many as the largest tree has, unless that wastes more than 15% of
//     the CTAs' time (trees of very different sizes); then an M tile is a segment.
// A segment that spans several runs is joined afterwards.  A CTA has at most two
// partial items: one that goes on from the run before (slot 0) and one that the
// next run goes on with (slot 1).

QHL_DEV int ta_segments(const TaSeq& s, const TaHead& h, int Hkv) { return Hkv / h.heads * (h.tiles > 1 ? 1 : s.nm); }
QHL_DEV int ta_units(const TaSeq& s) { return s.tiles ? s.tiles + kTaStart : 0; }
// First unit of run r, and the run that has unit u: the first units % runs runs
// have one more.
QHL_DEV int ta_run_start(const TaHead& h, int r) { return h.units / h.runs * r + min(r, h.units % h.runs); }
QHL_DEV int ta_run_of(const TaHead& h, int u) {
  const int q = h.units / h.runs, rem = h.units % h.runs, more = rem * (q + 1);
  return u < more ? u / (q + 1) : rem + (u - more) / q;
}

// Tree b, its lengths checked.
template <int KT>
QHL_DEV TaSeq ta_seq(const TaArgs& a, int b) {
  TaSeq s;
  s.seq = a.seq[b];
  tree_rows(a.q_start, b, a.n_rows, a.max_nodes, s.row0, s.n, a.err);
  s.ctx = 0;
  if (s.seq < 0 || s.seq >= a.n_seqs) {
    atomicOr(a.err, ERR_BAD_INDEX);
    s.seq = 0;
  } else {
    s.ctx = a.len[s.seq];
    if (s.ctx < 0 || s.ctx > kTaMostUnits || s.ctx > ((long long)a.max_pages << a.page_shift)) {
      atomicOr(a.err, ERR_BAD_INDEX);
      s.ctx = 0;
    }
  }
  s.tiles = s.n ? (s.ctx + KT - 1) / KT + (s.n + KT - 1) / KT : 0;
  s.nm = (s.n * a.G + kTaRows - 1) / kTaRows;
  s.base = s.pad = 0;
  return s;
}

// Sums over a CTA of NW warps: every thread's v before it, and the total.
template <int NW>
QHL_DEV long long ta_scan(long long v, long long* scratch, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < warp) before += scratch[i];
    total += scratch[i];
  }
  return before + inc - v;
}

// The groups, from the units with an M tile per segment (`alone`) and with all of
// a tree's (`together`), over all KV heads.  A full warp calls it.
QHL_DEV TaHead ta_head(const TaArgs& a, long long alone, long long together, int nm) {
  TaHead h;
  const int groups = nm ? a.grid / nm : 0;
  const bool shared = nm > 1 && groups > 0 && together * a.grid * 20 <= alone * groups * 23;
  h.tiles = shared ? nm : 1;
  int best = 1;
  for (int x = (threadIdx.x & 31) + 1; x <= a.Hkv; x += 32)
    if (a.Hkv % x == 0 && a.grid / (x * h.tiles) * (x * h.tiles) * 20 >= a.grid * 19) best = x;
  h.heads = __reduce_max_sync(0xffffffffu, best);
  long long units = (shared ? together : alone) / h.heads;
  if (units > kTaMostUnits) {                        // lengths that no cache can have
    atomicOr(a.err, ERR_BAD_INDEX);
    units = 0;
  }
  h.units = (int)units;
  h.runs = min(a.grid / (h.heads * h.tiles), h.units);
  return h;
}

// The plan of at most 32 trees, by one warp: lane b gets tree b.
template <int KT>
QHL_DEV TaHead ta_plan_warp(const TaArgs& a, TaSeq& s) {
  const int lane = threadIdx.x & 31;
  s = TaSeq{};
  if (lane < a.n_batch) s = ta_seq<KT>(a, lane);
  // 32 of the most still fit 32 bits; a tree beyond it counts as too many units
  constexpr long long kMost = kTaMostUnits / 32;
  const long long mine64 = (long long)a.Hkv * ta_units(s) * s.nm;
  const bool fits = __all_sync(0xffffffffu, mine64 <= kMost);
  const int alone = __reduce_add_sync(0xffffffffu, (int)min(mine64, kMost));
  const int together = __reduce_add_sync(0xffffffffu, (int)min((long long)a.Hkv * ta_units(s), kMost));
  const TaHead h = ta_head(a, fits ? alone : 2 * kTaMostUnits * a.Hkv, fits ? together : 2 * kTaMostUnits * a.Hkv, __reduce_max_sync(0xffffffffu, s.nm));
  if (a.n_batch > 1) {
    const int mine = h.units ? ta_segments(s, h, a.Hkv) * ta_units(s) : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    s.base = inc - mine;
  }
  return h;
}

// The plan, by all threads of a CTA of NW warps: every tree to `out`, with its
// first unit.  Trees are taken 32 NW at a time.
template <int KT, int NW>
QHL_DEV TaHead ta_plan(const TaArgs& a, TaSeq* out, long long* scratch) {
  const int tid = threadIdx.x;
  long long alone = 0, together = 0;
  int nm = 0;
  for (int b = tid; b < a.n_batch; b += 32 * NW) {
    const TaSeq s = ta_seq<KT>(a, b);
    out[b] = s;
    alone += (long long)a.Hkv * s.nm * ta_units(s);
    together += (long long)a.Hkv * ta_units(s);
    nm = max(nm, s.nm);
  }
  long long all_alone, all_together, total;
  ta_scan<NW>(alone, scratch, all_alone);
  ta_scan<NW>(together, scratch, all_together);
  nm = __reduce_max_sync(0xffffffffu, nm);
  __syncthreads();
  if ((tid & 31) == 0) scratch[tid >> 5] = nm;
  __syncthreads();
  for (int i = 0; i < NW; ++i) nm = max(nm, (int)scratch[i]);
  const TaHead h = ta_head(a, all_alone, all_together, nm);
  long long base = 0;
  for (int b0 = 0; b0 < a.n_batch; b0 += 32 * NW) {
    const int b = b0 + tid;
    const long long mine = h.units && b < a.n_batch ? (long long)ta_segments(out[b], h, a.Hkv) * ta_units(out[b]) : 0;
    const long long at = base + ta_scan<NW>(mine, scratch, total);
    if (b < a.n_batch) out[b].base = (int)at;
    base += total;
  }
  __syncthreads();
  return h;
}

// The plan of a large batch.
template <int DIM>
__global__ void __launch_bounds__(512) tree_plan_kernel(const __grid_constant__ TaArgs a) {
  __shared__ long long s_scratch[16];
  if (threadIdx.x == 0) pdl_launch();
  pdl_wait();
  const TaHead h = ta_plan<TaShape<DIM>::KT, 16>(a, a.seqs, s_scratch);
  if (threadIdx.x == 0) *a.head = h;
}

// ---------------------------------------------------------------- attention --

template <bool BF16>
QHL_DEV uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
QHL_DEV bool non_finite16(uint32_t h) {
  return BF16 ? (h & 0x7f80u) == 0x7f80u : (h & 0x7c00u) == 0x7c00u;
}
template <bool BF16>
QHL_DEV float widen16(uint32_t h) {
  return BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
}

// A wait names a phase by its parity, so a waiter must not be two phases away
// from it.  The softmax warps wait for the product with V only when they rescale
// and at an item's end; pv_done is kept per tile parity for them: when S of tile
// T is there, the product of tile T - 2, issued before it, is complete.  A slot of V
// is empty when the product and warp 11, which looks at every tile, are done with it.
struct TaBars {
  uint64_t full[12], empty[12], vok[12];
  uint64_t q_ready, s_full[2], p_ready[2], pv_done[2], mask_full, mask_empty;
};

// The plan as a CTA holds it; `seq` only for small batches.
struct TaOwnPlan {
  TaSeq seq[kTaOwnPlan];
  long long scratch[kTaThreads / 32];
  TaHead head;
  // the CTA's run: units u .. end - 1, from unit x of segment seg of tree b on; its
  // head and M tile within the group; segments of a tree per M tile of its own
  int u, end, b, seg, x, hd, mt, head_groups;
};

// What the roles know of an item.
struct TaItem {
  TaSeq s;
  int t0, t1, h, mt, nct;      // nct: cache tiles
  QHL_DEV bool whole() const { return t0 == 0 && t1 == s.tiles; }
};

// The CTA's run, but for where it starts; one thread calls it.
QHL_DEV void ta_set_run(const TaArgs& a, const TaHead& h, TaOwnPlan& p) {
  const int per = h.heads * h.tiles, run = (int)blockIdx.x / per, j = (int)blockIdx.x - run * per;
  p.head = h;
  p.hd = j / h.tiles;
  p.mt = j - p.hd * h.tiles;
  p.head_groups = a.Hkv / h.heads;
  p.u = run < h.runs ? ta_run_start(h, run) : 0;
  p.end = run < h.runs ? ta_run_start(h, run + 1) : 0;
  p.b = p.seg = p.x = 0;
}
// Where it starts, from the tree that has its first unit.
QHL_DEV void ta_set_start(TaOwnPlan& p, int b, const TaSeq& s, int u) {
  const int units = ta_units(s), at = u - s.base;
  p.b = b;
  p.seg = at / units;
  p.x = at - p.seg * units;
}

// The items of a CTA, in order.
template <int DIM>
struct TaCursor {
  int u, end, b, seg, x;

  QHL_DEV explicit TaCursor(const TaOwnPlan& p) : u(p.u), end(p.end), b(p.b), seg(p.seg), x(p.x) {}
  QHL_DEV bool next(const TaArgs& a, const TaOwnPlan& p, TaItem& w) {
    const bool shared = p.head.tiles > 1;
    while (u < end) {
      if (a.n_batch <= kTaOwnPlan) {
        w.s = p.seq[b];
      } else {
        const int4* s = reinterpret_cast<const int4*>(a.seqs + b);
        const int4 s0 = __ldcg(s), s1 = __ldcg(s + 1);
        w.s = TaSeq{s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, 0};
      }
      const int units = ta_units(w.s);
      if (units == 0 || seg >= p.head_groups * (shared ? 1 : w.s.nm)) {   // no segments, or behind the last
        ++b;
        seg = x = 0;
        continue;
      }
      const int y = min(units, x + (end - u)), group = shared || w.s.nm == 1 ? seg : seg / w.s.nm;
      w.t0 = max(0, x - kTaStart);
      w.t1 = max(0, y - kTaStart);
      w.h = group * p.head.heads + p.hd;
      w.mt = shared ? p.mt : seg - group * w.s.nm;
      w.nct = (w.s.ctx + TaShape<DIM>::KT - 1) / TaShape<DIM>::KT;
      u += y - x;
      x = y;
      if (y == units) {
        ++seg;
        x = 0;
      }
      if (w.t1 > w.t0 && w.mt < w.s.nm) return true;
    }
    return false;
  }
};

// Every CTA's plan (all threads).  CTA 0 of a small batch leaves it for the join.
template <int DIM>
QHL_DEV void ta_own_plan(const TaArgs& a, TaOwnPlan& p) {
  constexpr int KT = TaShape<DIM>::KT;
  const int tid = threadIdx.x;
  if (a.n_batch <= 32) {
    if (tid < 32) {
      TaSeq s;
      const TaHead h = ta_plan_warp<KT>(a, s);
      if (tid < a.n_batch) {
        p.seq[tid] = s;
        if (blockIdx.x == 0) a.seqs[tid] = s;
      }
      if (tid == 0) {
        ta_set_run(a, h, p);
        if (blockIdx.x == 0) *a.head = h;
      }
      __syncwarp();
      const int u = p.u;
      if (p.end > u && s.base <= u && u < s.base + ta_segments(s, h, a.Hkv) * ta_units(s)) ta_set_start(p, tid, s, u);
    }
    __syncthreads();
    return;
  }
  const bool own = a.n_batch <= kTaOwnPlan;
  if (own) {
    const TaHead h = ta_plan<KT, kTaThreads / 32>(a, p.seq, p.scratch);
    if (tid == 0) ta_set_run(a, h, p);
    if (blockIdx.x == 0) {
      if (tid == 0) *a.head = h;
      if (tid < a.n_batch) a.seqs[tid] = p.seq[tid];
    }
  } else if (tid == 0) {
    const int4 h = __ldcg(reinterpret_cast<const int4*>(a.head));
    ta_set_run(a, TaHead{h.x, h.y, h.z, h.w}, p);
  }
  __syncthreads();
  const TaHead h = p.head;
  const int u = p.u;
  for (int b = tid; p.end > u && b < a.n_batch; b += kTaThreads) {
    const TaSeq s = own ? p.seq[b] : a.seqs[b];
    if (s.base <= u && u < s.base + ta_segments(s, h, a.Hkv) * ta_units(s)) ta_set_start(p, b, s, u);
  }
  __syncthreads();
}

// Partial row of row r of an M tile's part that CTA `cta` computed; `on`: the part
// goes on from the CTA before.
QHL_DEV long long ta_slot(const TaArgs& a, int cta, bool on, int r) { return ((long long)cta * 2 + (on ? 0 : 1)) * a.slot_rows + r; }

// Rows of V that the product of a tile needs: its keys, up to a multiple of 16.
template <int KT>
QHL_DEV int ta_keys(const TaItem& w, int tile) {
  return tile >= w.nct ? min(KT, w.s.n - (tile - w.nct) * KT) : min(KT, w.s.ctx - tile * KT);
}

template <int DIM, bool BF16>
__global__ void __launch_bounds__(kTaThreads, 1) tree_attn_kernel(const __grid_constant__ TaArgs a) {
  using Sh = TaShape<DIM>;
  constexpr int KT = Sh::KT, CH = Sh::CH, NS = Sh::NS, HK = KT / 2;
  constexpr float kUp = BF16 ? 0.f : 6.f;            // p is 2^kUp larger than its softmax numerator
  static_assert(NS % 2 == 0, "K has the even slots, V the odd ones");
  extern __shared__ uint8_t smem_raw[];
  __shared__ TaBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(16) uint4 s_anc[kMaxNodes];   // per token: the tokens it sees, a bit each
  __shared__ int s_jump[kMaxNodes];
  __shared__ unsigned s_bad[4];                      // tokens whose V row holds an infinity or NaN
  __shared__ int s_gone;                             // whether the TMA warp has met a page that does not exist
  __shared__ float s_max[2][2][kTaRows], s_sum[2][kTaRows];
  __shared__ __align__(16) TaOwnPlan s_plan;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto bar = [](const uint64_t& b) { return smem_u32(&b); };

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(bars.full[i]), 1);
      mbar_init(bar(bars.empty[i]), i & 1 ? 2 : 1);  // V's: the product and warp 11
      mbar_init(bar(bars.vok[i]), 1);
    }
    s_gone = 0;
    mbar_init(bar(bars.q_ready), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.s_full[i]), 1);
      mbar_init(bar(bars.p_ready[i]), 8);
      mbar_init(bar(bars.pv_done[i]), 1);
    }
    mbar_init(bar(bars.mask_full), 1);
    mbar_init(bar(bars.mask_empty), 8);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&s_tmem, 512);
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&a.k);
    tma_prefetch_map(&a.v);
    tma_prefetch_map(&a.kn);
    tma_prefetch_map(&a.vn);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_wait();
  ta_own_plan<DIM>(a, s_plan);
  TaCursor<DIM> cursor(s_plan);
  TaItem item;
  // Every wait is bounded; a role that gave one up stops (ok = false) once those
  // it shares a named barrier with know it too.
  bool ok = true;
  auto wait_warp = [&](const uint64_t& b, uint32_t parity) {   // the same answer in every lane
    return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, a.err, kTaWait)) != 0;
  };

  if (warp == 8) {
    // ---------------------------------------------------------------- TMA --
    // Where a page is less than a tile, a tile takes several copies, which the lanes
    // issue together.  K: one per (page, chunk), so that the chunks of all pages are
    // KT rows apart in the slot (the product's N runs over the rows of all pages).
    // V: one per page, whose chunks follow one another (the product takes 16 rows at
    // a time, which lie in one page); a small copy costs as much as a large one, and
    // with pages of 16 rows the copies are what bounds a tile.
    uint32_t r = 0;
    const int pchunks = a.box == KT ? 1 : CH, dchunks = a.dbox == KT ? 1 : CH;
    const int pbox = lane / pchunks, pchunk = lane % pchunks, boxes_per_tile = KT >> a.box_shift;
    while (ok && cursor.next(a, s_plan, item)) {
      const TaItem w = item;
      const int* row = a.table + (size_t)w.s.seq * a.max_pages;
      // page numbers of this item's boxes, 32 at a time, one batch ahead
      const int box_end = (w.s.ctx + a.box - 1) >> a.box_shift;
      auto page_of = [&](int j) {
        int pg = -1;
        if (j < box_end) {
          pg = row[j >> (a.page_shift - a.box_shift)];
          if (pg < 0 || pg >= a.n_pages) {
            atomicOr(a.err, ERR_BAD_INDEX);
            pg = a.n_pages;                          // beyond the tensor: the copy fills zeros
            s_gone = 1;                              // and the softmax warps, before they see the tile's S, learn of it
          }
        }
        return pg;
      };
      int ids_at = w.t0 * boxes_per_tile, ids = page_of(ids_at + lane), ids_next = page_of(ids_at + 32 + lane);
      for (int tile = w.t0; ok && tile < w.t1; ++tile) {
        const bool draft = tile >= w.nct;
        const int b0 = tile * boxes_per_tile;
        int nb = 1;
        if (!draft) {
          nb = min(boxes_per_tile, box_end - b0);
          if (b0 - ids_at >= 32) {                   // 32 is a multiple of a tile's boxes
            ids = ids_next;
            ids_at += 32;
            ids_next = page_of(ids_at + 32 + lane);
          }
        }
        const uint32_t bytes = (uint32_t)(draft ? a.dbox : nb << a.box_shift) * DIM * 2;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t s = r % NS, ph = r / NS & 1;
          ++r;
          ok = wait_warp(bars.empty[s], ph ^ 1);     // its last contents are used
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(bars.full[s]), bytes);
          __syncwarp();
          const uint32_t dst = ring + s * Sh::SLOT;
          if (draft) {
            if (lane < dchunks) tma_load_5d(dst + lane * (KT * 128), kv ? &a.vn : &a.kn, bar(bars.full[s]), w.s.row0 + (tile - w.nct) * KT, lane, w.h, 0);
          } else {
            const int box = kv ? lane : pbox, c = kv ? 0 : pchunk;
            const int pg = __shfl_sync(0xffffffffu, ids, (b0 - ids_at + box) & 31);
            const int rr = (b0 + box) << a.box_shift & ((1 << a.page_shift) - 1);
            const uint32_t off = kv ? (uint32_t)(box << a.box_shift) * (DIM * 2) : (uint32_t)(box << a.box_shift) * 128u + (uint32_t)c * (KT * 128);
            if (box < nb) tma_load_5d(dst + off, kv ? &a.v : &a.k, bar(bars.full[s]), rr, c, w.h, pg);
          }
        }
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------- S = Q K^T --
    // The two products have an issuer each: a wait that is over still takes some
    // 250 cycles under load, and one thread's waits for both left the tensor core
    // idle for 40% of a tile (2400 cycles instead of 1450 at 256 dimensions).
    // The whole warp walks the tiles, with values that the compiler knows to be the
    // same in all lanes, and one lane issues: the descriptors then stay in uniform
    // registers (from one lane's own loop a product took 1.2 x as long to issue).
    constexpr uint32_t id = idesc_f16(BF16, false, kTaRows, KT);
    uint32_t slot = 0, phase = 0, T = 0, it = 0;
    for (; ok && cursor.next(a, s_plan, item); ++it) {
      const int n = __shfl_sync(0xffffffffu, item.t1 - item.t0, 0);
      if (!(ok = wait_warp(bars.q_ready, it & 1))) break;
      for (int i = 0; i < n; ++i, ++T) {
        const uint32_t b = T & 1;
        if (!(ok = wait_warp(bars.full[slot], phase))) break;
        // p of the tile before last, which lies in this S, is used
        if (T >= 2 && !(ok = wait_warp(bars.pv_done[b], (T >> 1 & 1) ^ 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = smem_desc_sw128(ring + slot * Sh::SLOT, 16);
#pragma unroll
          for (int k = 0; k < DIM / 16; ++k)
            mma_f16_ts(tmem + Sh::S0 + b * KT, tmem + Sh::Q0 + k * 8, kd + (uint64_t)((k / 4) * (KT * 128) + (k % 4) * 32 >> 4), id, k != 0);
          tc_commit(&bars.s_full[b]);
          tc_commit(&bars.empty[slot]);
        }
        __syncwarp();
        slot += 2;                                   // K has the even slots
        if (slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ O += p V --
    constexpr uint32_t id = idesc_f16(BF16, true, kTaRows, DIM);
    uint32_t slot = 1, phase = 0, T = 0, vok_phase = 0;
    while (ok && cursor.next(a, s_plan, item)) {
      const int t0 = __shfl_sync(0xffffffffu, item.t0, 0), t1 = __shfl_sync(0xffffffffu, item.t1, 0);
      const int nct = __shfl_sync(0xffffffffu, item.nct, 0), ctx = __shfl_sync(0xffffffffu, item.s.ctx, 0);
      const int nodes = __shfl_sync(0xffffffffu, item.s.n, 0);
      for (int tile = t0; tile < t1; ++tile, ++T) {
        const uint32_t b = T & 1;
        const int keys = tile >= nct ? min(KT, nodes - (tile - nct) * KT) : min(KT, ctx - tile * KT);
        if (!(ok = wait_warp(bars.full[slot], phase))) break;
        if (tile >= nct || keys < KT) {
          if (!(ok = wait_warp(bars.vok[slot], vok_phase >> slot & 1))) break;
          vok_phase ^= 1u << slot;
        }
        if (!(ok = wait_warp(bars.p_ready[b], T >> 1 & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t p = tmem + Sh::S0 + b * KT;
          // chunks are a page's (or a tile's) rows apart, pages follow one another
          const int shift = tile >= nct ? (KT == 64 ? 6 : 7) : a.box_shift, rows = 1 << shift;
          const uint64_t vd = smem_desc_sw128(ring + slot * Sh::SLOT, rows * 128);
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            const int off = (16 * k >> shift << shift) * (DIM * 2) + (16 * k & (rows - 1)) * 128;
            if (16 * k < keys) mma_f16_ts(tmem, p + k * 8, vd + (uint64_t)(off >> 4), id, tile != t0 || k);
          }
          tc_commit(&bars.pv_done[b]);
          tc_commit(&bars.empty[slot]);
        }
        __syncwarp();
        slot += 2;
        if (slot > NS) {
          slot = 1;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 11) {
    // ------------------------------------------- masks, tiles that need care --
    uint32_t r = 1, it = 0;
    for (; ok && cursor.next(a, s_plan, item); ++it) {
      const TaItem w = item;
      const int n = w.s.n;
      if (it && !(ok = wait_warp(bars.mask_empty, (it - 1) & 1))) break;
      if (lane < 4) s_bad[lane] = 0;
      // ancestors by doubling: after k rounds those up to 2^k steps away; a jump
      // ends at -1 (the cached sequence) or -2 (padded: nothing is seen)
      for (int x = lane; x < n; x += 32) {
        int p = a.parent[w.s.row0 + x];
        if (p < -2 || p >= x) {
          atomicOr(a.err, ERR_BAD_INDEX);
          p = -2;
        }
        s_jump[x] = p;
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = x >> 5 == j ? 1u << (x & 31) : 0u;
        s_anc[x] = make_uint4(m[0], m[1], m[2], m[3]);
      }
      __syncwarp();
      for (int step = 1; step < n; step <<= 1) {
        uint4 m[4];
        int jp[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = lane + 32 * u;
          jp[u] = -1;
          if (x < n) {
            m[u] = s_anc[x];
            jp[u] = s_jump[x];
            if (jp[u] >= 0) {
              const uint4 o = s_anc[jp[u]];
              m[u] = make_uint4(m[u].x | o.x, m[u].y | o.y, m[u].z | o.z, m[u].w | o.w);
              jp[u] = s_jump[jp[u]];
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (lane + 32 * u < n) {
            s_anc[lane + 32 * u] = m[u];
            s_jump[lane + 32 * u] = jp[u];
          }
        __syncwarp();
      }
      for (int x = lane; x < n; x += 32)
        if (s_jump[x] == -2) s_anc[x] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.mask_full));

      for (int tile = w.t0; ok && tile < w.t1; ++tile, r += 2) {
        // every tile's V is waited for, and its slot is filled again only once this warp
        // has been there, so that the wait's parity is that of its phase
        const bool draft = tile >= w.nct;
        const uint32_t s = r % NS;
        const int keys = ta_keys<KT>(w, tile);
        if (!(ok = wait_warp(bars.full[s], r / NS & 1))) break;
        if (!draft && keys == KT) {
          if (lane == 0) mbar_arrive(bar(bars.empty[s]));
          continue;
        }
        uint8_t* base = smem_raw + (ring + s * Sh::SLOT - smem_u32(smem_raw));
        // Rows up to the multiple of 16 that the product reads.  Units of 16 bytes;
        // the swizzle permutes the units of a row only.
        const int end = (keys + 15) & ~15, begin = draft ? 0 : keys;
#pragma unroll 1
        for (int ch = 0; ch < CH; ++ch) {
          // row 0 of the chunk, as if the rows of the last page (or the tile) began at 0
          const int shift = draft ? (KT == 64 ? 6 : 7) : a.box_shift, page0 = begin >> shift << shift;
          uint4* p = reinterpret_cast<uint4*>(base + page0 * (DIM * 2) + (ch << shift) * 128 - page0 * 128);
#pragma unroll 4
          for (int u = begin * 8 + lane; u < keys * 8; u += 32) {
            uint4 x = p[u];
            uint32_t* y = reinterpret_cast<uint32_t*>(&x);
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (non_finite16<BF16>(y[e])) { y[e] &= 0xffff0000u; bad = true; }
              if (non_finite16<BF16>(y[e] >> 16)) { y[e] &= 0xffffu; bad = true; }
            }
            if (bad) {
              p[u] = x;
              const int node = (tile - w.nct) * KT + u / 8;
              atomicOr(&s_bad[node >> 5], 1u << (node & 31));
            }
          }
          for (int u = keys * 8 + lane; u < end * 8; u += 32) p[u] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bars.vok[s]));
          mbar_arrive(bar(bars.empty[s]));
        }
      }
    }
  } else {
    // ------------------------------------------------------------- softmax --
    const int qd = warp & 3, hf = warp >> 2, row = qd * 32 + lane;
    const uint32_t lanes = (uint32_t)(qd * 32) << 16;
    const float c = a.c, thr = 8.f / c;
    uint32_t T = 0, it = 0;
    for (; cursor.next(a, s_plan, item); ++it) {
      const TaItem w = item;
      const int qr = w.mt * kTaRows + row, node = qr / a.G, g = qr - node * a.G;   // the thread's token and query head
      const bool valid = node < w.s.n;
      const bool active = __any_sync(0xffffffffu, valid);
      // Q to tensor memory: the tile's last S is complete, so nothing reads it now
      if (active) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (long long)(w.s.row0 + node) * a.q_stride +
                                                          (w.h * a.G + g) * DIM + hf * (DIM / 2));
#pragma unroll
        for (int j = 0; j < DIM / 64; ++j) {         // 32 elements, 16 columns
          uint4 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = valid ? src[4 * j + e] : make_uint4(0, 0, 0, 0);
          tmem_st16(tmem + lanes + Sh::Q0 + hf * (DIM / 4) + 16 * j, reinterpret_cast<const uint32_t*>(x));
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.q_ready));
      ok = wait_warp(bars.mask_full, it & 1);
      uint4 anc = make_uint4(0, 0, 0, 0);
      if (valid) anc = s_anc[node];
      const bool alive = (anc.x | anc.y | anc.z | anc.w) != 0;
      float m = -INFINITY, l = 0.f;
      const int full = w.s.ctx / KT;                 // tiles of the cache that have all their keys
      bool stop = false;

      for (int tile = w.t0; tile < w.t1; ++tile, ++T) {
        const uint32_t b = T & 1;
        if (ok) ok = wait_warp(bars.s_full[b], T >> 1 & 1);
        if (!active && !ok) {
          stop = true;
          break;
        }
        if (active) {
          tc_fence_after();
          const uint32_t sb = tmem + lanes + Sh::S0 + b * KT;
          const int gone = s_gone;
          uint32_t sv[HK / 32][32];
#pragma unroll
          for (int j = 0; j < HK / 32; ++j) tmem_ld32(sb + hf * HK + 32 * j, sv[j]);
          tmem_ld_wait();
          if (tile >= full || gone) {                // perhaps not a tile of keys that all are seen
            if (tile >= w.nct) {
              const int w0 = (tile - w.nct) * (KT / 32) + hf * (HK / 32);
#pragma unroll
              for (int j = 0; j < HK / 32; ++j) {
                const int wi = w0 + j;
                const uint32_t bits = wi == 0 ? anc.x : wi == 1 ? anc.y : wi == 2 ? anc.z : anc.w;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(bits >> e & 1)) sv[j][e] = 0xff800000u;
              }
            } else {
              const int lim = w.s.ctx - tile * KT - hf * HK;
#pragma unroll
              for (int e = 0; e < HK; ++e)
                if (e >= lim) sv[e / 32][e % 32] = 0xff800000u;
              if (gone) {                            // pages have at least 16 rows
                const int* row = a.table + (size_t)w.s.seq * a.max_pages;
#pragma unroll
                for (int e = 0; e < HK; e += 16) {
                  const int key = tile * KT + hf * HK + e, pg = key < w.s.ctx ? row[key >> a.page_shift] : 0;
                  if (pg < 0 || pg >= a.n_pages) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) sv[(e + i) / 32][(e + i) % 32] = 0xff800000u;
                  }
                }
              }
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < HK / 32; ++j)
#pragma unroll
            for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(sv[j][e]));
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          s_max[b][hf][row] = top;
          ok = bar_and(1 + qd, 64, ok);
          if (!ok) {
            stop = true;
            break;
          }
          top = fmaxf(top, s_max[b][hf ^ 1][row]);

          if (tile == w.t0) {
            m = top;
          } else {
            const bool raise = top > m + thr;
            if (__any_sync(0xffffffffu, raise)) {
              ok = wait_warp(bars.pv_done[(T - 1) & 1], (T - 1) >> 1 & 1);
              tc_fence_after();
              const float al = raise ? ex2((m - top) * c) : 1.f;
              if (raise) m = top;
              l *= al;
#pragma unroll 1
              for (int j = 0; j < DIM / 64; ++j) {
                uint32_t o[32];
                const uint32_t oc = tmem + lanes + hf * (DIM / 2) + 32 * j;
                tmem_ld32(oc, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st32(oc, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : m * c - kUp;
          const float2 c2 = make_float2(c, c), ms2 = make_float2(-ms, -ms);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < HK / 32; ++j) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = ffma2(make_float2(__uint_as_float(sv[j][e]), __uint_as_float(sv[j][e + 1])), c2, ms2);
              const float2 y = make_float2(ex2(x.x), ex2(x.y));
              sum[e >> 1 & 1] = __fadd2_rn(sum[e >> 1 & 1], y);
              pk[e / 2] = pack2<BF16>(y.x, y.y);
            }
            tmem_st16(sb + hf * (KT / 4) + 16 * j, pk);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.p_ready[b]));
      }
      if (stop) break;

      // ------------------------------------------------------ the item's end --
      if (ok) ok = wait_warp(bars.pv_done[(T - 1) & 1], (T - 1) >> 1 & 1);
      if (!active && !ok) break;
      if (active) {
        tc_fence_after();
        s_sum[hf][row] = l;
        ok = bar_and(1 + qd, 64, ok);
        if (!ok) break;
        l += s_sum[hf ^ 1][row];
        if (!alive) {                                // padded: whatever was summed, nothing was seen
          m = -INFINITY;
          l = 0.f;
        }
        const bool whole = w.whole();
        const long long slot = ta_slot(a, blockIdx.x, w.t0 > 0, row);
        const float inv = l > 0.f || l != l ? __frcp_rn(l) : 0.f;
        const bool none = l == 0.f;                  // nothing seen: 0, whatever the tiles held
        uint32_t bad[4];
        const uint32_t see[4] = {anc.x, anc.y, anc.z, anc.w};
        bool any_bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bad[j] = w.t1 > w.nct ? s_bad[j] & see[j] : 0u;
          any_bad |= bad[j] != 0;
        }
        uint8_t* orow = static_cast<uint8_t*>(a.out) + ((long long)(w.s.row0 + node) * a.out_stride + (w.h * a.G + g) * DIM + hf * (DIM / 2)) * 2;
        float4* prow = reinterpret_cast<float4*>(a.po) + ta_slot(a, blockIdx.x, w.t0 > 0, 0) * (DIM / 4) + row;   // [DIM / 4][slot_rows]
#pragma unroll 1
        for (int j = 0; j < DIM / 64; ++j) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tmem + lanes + hf * (DIM / 2) + 32 * j, o);
          tmem_ld_wait();
          if (!valid) continue;
          if (any_bad) {
            // drafted V values that are not finite, seen with a positive weight
            for (int x = 0; x < w.s.n; ++x) {
              const int word = x >> 5;
              const uint32_t bw = word == 0 ? bad[0] : word == 1 ? bad[1] : word == 2 ? bad[2] : bad[3];
              const int dt = x / KT + w.nct;
              if (!(bw >> (x & 31) & 1) || dt < w.t0 || dt >= w.t1) continue;
              const uint16_t* vr = static_cast<const uint16_t*>(a.v_new) + (long long)(w.s.row0 + x) * a.new_stride + w.h * DIM + hf * (DIM / 2) + 32 * j;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t h = vr[e];
                if (non_finite16<BF16>(h)) o[e] = __float_as_uint(__uint_as_float(o[e]) + widen16<BF16>(h));
              }
            }
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 x;
              uint32_t* y = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
              for (int z = 0; z < 4; ++z)
                y[z] = none ? 0u : pack2<BF16>(__uint_as_float(o[e + 2 * z]) * inv, __uint_as_float(o[e + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(orow + (32 * j + e) * 2) = x;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(prow + (long long)(hf * (DIM / 8) + 8 * j + e / 4) * a.slot_rows) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (valid && hf == 0) {
          const float mc = m == -INFINITY ? -INFINITY : m * c - kUp;
          if (!whole)
            a.pml[slot] = make_float2(mc, l);
          else if (a.lse)
            a.lse[(long long)(w.s.row0 + node) * (a.Hkv * a.G) + w.h * a.G + g] =
                none ? -INFINITY : (mc + log2f(l)) * 0.69314718055994530942f;
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.mask_empty));
    }
  }
  // The join's CTAs come only now: waiting beside this one they slowed it by 10%.
  if (tid == 0) pdl_launch();
  if (!ok) drain_inflight_copies();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------------- join --

// A thread per four values of O; blocks of 256 / W values, each summed by W threads
// over every W-th part (W = 4 where there are few values), whose sums meet as
// (0 + 1) + (2 + 3).  The parts of an item lie as [DIM / 4][slot_rows] float4, so
// that both this kernel and the item's end move whole sectors; the loads of U parts
// go out together, the weights by a running maximum.
constexpr long long kJoinFew = 148LL * 1024;   // values (of four) up to which W = 4

template <int DIM, bool BF16, int W>
__global__ void __launch_bounds__(256, W > 1 ? 3 : 5) tree_join_kernel(const __grid_constant__ TaArgs a) {
  constexpr int U = W > 1 ? 8 : 4, V = 256 / W;
  __shared__ float4 s_o[W > 1 ? 256 : 1];
  __shared__ float2 s_ml[W > 1 ? 256 : 1];
  const int tid = threadIdx.x, part = tid / V, x = blockIdx.x * V + tid % V;
  const int b = blockIdx.z, h = blockIdx.y % a.Hkv, mt = blockIdx.y / a.Hkv;
  if (tid == 0) pdl_launch();
  pdl_wait();
  const int4* sp = reinterpret_cast<const int4*>(a.seqs + b);
  const int4 s0 = __ldcg(sp), s1 = __ldcg(sp + 1), h0 = __ldcg(reinterpret_cast<const int4*>(a.head));
  const TaHead head{h0.x, h0.y, h0.z, h0.w};
  if (mt >= s1.y || s1.x == 0 || head.units == 0) return;
  const int seg = head.tiles > 1 ? h / head.heads : h / head.heads * s1.y + mt;
  const int u0 = s1.z + seg * (s1.x + kTaStart);
  const int r0 = ta_run_of(head, u0 + kTaStart), chunks = ta_run_of(head, u0 + s1.x + kTaStart - 1) - r0 + 1;
  if (chunks <= 1) return;
  const int per = head.heads * head.tiles, cta0 = r0 * per + h % head.heads * head.tiles + (head.tiles > 1 ? mt : 0);
  const int cg = x / a.slot_rows, r = x - cg * a.slot_rows, qr = mt * kTaRows + r, node = qr / a.G, g = qr - node * a.G;
  const bool mine = cg < DIM / 4 && node < s0.y;

  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, sum = 0.f;
  if (mine) {
    for (int j0 = part; j0 < chunks; j0 += U * W) {
      float2 ml[U];
      float4 y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * W;
        const long long slot = ta_slot(a, cta0 + j * per, j > 0, 0);
        ml[u] = make_float2(0.f, 0.f);
        if (j < chunks) {
          ml[u] = __ldcg(a.pml + slot + r);
          y[u] = __ldcg(reinterpret_cast<const float4*>(a.po) + slot * (DIM / 4) + x);
        }
      }
      float now = top;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ml[u].y != 0.f) now = fmaxf(now, ml[u].x);   // a part that saw nothing does not count; NaN does
      const float al = sum != 0.f ? ex2(top - now) : 0.f;
      top = now;
      if (al != 1.f) {
        sum *= al;
        o = sum != 0.f ? make_float4(o.x * al, o.y * al, o.z * al, o.w * al) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ml[u].y != 0.f) {
          const float w = ex2(ml[u].x - now);
          if (w != 0.f || ml[u].y != ml[u].y) {      // a NaN counts whatever its weight
            sum = fmaf(w, ml[u].y, sum);
            o.x = fmaf(w, y[u].x, o.x);
            o.y = fmaf(w, y[u].y, o.y);
            o.z = fmaf(w, y[u].z, o.z);
            o.w = fmaf(w, y[u].w, o.w);
          }
        }
    }
  }
  if constexpr (W > 1) {
    s_o[tid] = o;
    s_ml[tid] = make_float2(top, sum);
    __syncthreads();
    if (part) return;
    float2 ml[W];
    float w[W];
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      ml[i] = s_ml[i * V + tid];
      if (ml[i].y != 0.f) top = fmaxf(top, ml[i].x);
    }
    float4 y[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      w[i] = ml[i].y != 0.f ? ex2(ml[i].x - top) : 0.f;
      const bool use = w[i] != 0.f || ml[i].y != ml[i].y;
      ml[i].y = use ? ml[i].y * w[i] : 0.f;
      const float4 z = s_o[i * V + tid];
      y[i] = use ? make_float4(z.x * w[i], z.y * w[i], z.z * w[i], z.w * w[i]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    sum = (ml[0].y + ml[1].y) + (ml[2].y + ml[3].y);
    o = make_float4((y[0].x + y[1].x) + (y[2].x + y[3].x), (y[0].y + y[1].y) + (y[2].y + y[3].y), (y[0].z + y[1].z) + (y[2].z + y[3].z),
                    (y[0].w + y[1].w) + (y[2].w + y[3].w));
  }
  if (!mine) return;
  const float inv = sum > 0.f || sum != sum ? __frcp_rn(sum) : 0.f;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + (long long)(s0.x + node) * a.out_stride + (h * a.G + g) * DIM + 4 * cg;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  if (cg == 0 && a.lse)
    a.lse[(long long)(s0.x + node) * (a.Hkv * a.G) + h * a.G + g] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// --------------------------------------------------------------------- host --

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct TaDevice {
  int sms = 0;
  bool ready = false;
};
std::mutex g_ta_mu;
TaDevice g_ta[64];
EncodeFn g_encode = nullptr;

// The full shared-memory carveout for every kernel of the chain: an SM that has
// another split must drain before a CTA of tree_attn_kernel starts there.
template <typename K>
cudaError_t full_carveout(K k) {
  return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}
template <int DIM, bool BF16>
cudaError_t ta_attributes() {
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<DIM, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, TaShape<DIM>::SMEM);
  if (e == cudaSuccess) e = full_carveout(tree_attn_kernel<DIM, BF16>);
  if (e == cudaSuccess) e = full_carveout(tree_join_kernel<DIM, BF16, 1>);
  if (e == cudaSuccess) e = full_carveout(tree_join_kernel<DIM, BF16, 4>);
  if (e == cudaSuccess) e = full_carveout(tree_plan_kernel<DIM>);
  return e;
}

// SM count and kernel attributes of the current device; the driver's encoder.
cudaError_t ta_device(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_ta_mu);
  TaDevice& d = g_ta[dev];
  if (!g_encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if ((e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q)) != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeFn>(f);
  }
  if (!d.ready) {
    if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = ta_attributes<64, false>()) != cudaSuccess || (e = ta_attributes<64, true>()) != cudaSuccess ||
        (e = ta_attributes<128, false>()) != cudaSuccess || (e = ta_attributes<128, true>()) != cudaSuccess ||
        (e = ta_attributes<256, false>()) != cudaSuccess || (e = ta_attributes<256, true>()) != cudaSuccess)
      return e;
    d.ready = true;
  }
  *sms = std::min(d.sms, 256);
  return cudaSuccess;
}

// A map of rank 5 whose innermost axis is the 64 elements of a 128-byte chunk;
// strides (of the other four axes) in elements.
bool encode(CUtensorMap* m, bool bf16, const void* base, const long long (&dims)[4], const long long (&strides)[4],
            const int (&box)[4]) {
  cuuint64_t gd[5] = {64, 0, 0, 0, 0}, gs[4];
  cuuint32_t bx[5] = {64, 0, 0, 0, 0}, es[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 4; ++i) {
    gd[i + 1] = (cuuint64_t)dims[i];
    gs[i] = (cuuint64_t)strides[i] * 2;
    bx[i + 1] = (cuuint32_t)box[i];
  }
  return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(base), gd, gs, bx,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct TaLayout {
  size_t seqs, pml, po, total;
  int slot_rows;
};

TaLayout ta_layout(int dim, int G, int n_batch, int max_nodes, int grid) {
  TaLayout l;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.slot_rows = std::min(kTaRows, max_nodes * G);
  const size_t rows = (size_t)grid * 2 * l.slot_rows;
  l.seqs = 256;
  l.pml = l.seqs + up(sizeof(TaSeq) * (size_t)n_batch);
  l.po = l.pml + up(8 * rows);
  l.total = l.po + up(4 * rows * dim);
  return l;
}

// Shape checks shared by the call and its workspace query.
int ta_check(const char* me, const qhl_kv_pages* kv, int Hq, int n_rows, int n_batch, int max_nodes) {
  const int rc = check_pages(me, kv);
  if (rc) return rc;
  if (Hq < 1 || Hq % kv->kv_heads || Hq / kv->kv_heads > kTaRows)
    return verify_err(me, STAGE_E_ARG, "n_q_heads must be a multiple of kv_heads, at most 128 of them each");
  if (n_rows < 0 || n_batch < 1 || n_batch > kMaxBatch || max_nodes < 1 || max_nodes > kMaxNodes)
    return verify_err(me, STAGE_E_ARG, "n_rows, n_batch (1..2048) or max_nodes (1..128) out of range");
  if ((long long)n_batch * kv->kv_heads * (Hq / kv->kv_heads) * max_nodes > 1LL << 26)
    return verify_err(me, STAGE_E_ARG, "too many query rows");
  return 0;
}

template <int DIM, bool BF16>
cudaError_t ta_launch(const TaArgs& a, cudaStream_t s) {
  // each kernel waits for the one before it on the stream before it reads anything
  cudaError_t e = cudaSuccess;
  if (a.n_batch > kTaOwnPlan) e = launch_ex(tree_plan_kernel<DIM>, dim3(1), dim3(512), 0, s, true, a);
  if (e == cudaSuccess) e = launch_ex(tree_attn_kernel<DIM, BF16>, dim3(a.grid), dim3(kTaThreads), TaShape<DIM>::SMEM, s, true, a);
  if (e != cudaSuccess) return e;
  const int nm = (a.max_nodes * a.G + kTaRows - 1) / kTaRows;
  const long long values = (long long)a.slot_rows * (DIM / 4) * nm * a.Hkv * a.n_batch;
  const int v = a.slot_rows * (DIM / 4);
  const dim3 heads(0, a.Hkv * nm, a.n_batch);
  if (values <= kJoinFew) return launch_ex(tree_join_kernel<DIM, BF16, 4>, dim3((v + 63) / 64, heads.y, heads.z), dim3(256), 0, s, true, a);
  return launch_ex(tree_join_kernel<DIM, BF16, 1>, dim3((v + 255) / 256, heads.y, heads.z), dim3(256), 0, s, true, a);
}

}  // namespace

}  // namespace qhl

using namespace qhl;

extern "C" {

size_t qhl_tree_attention_workspace(const qhl_kv_pages* kv, int n_q_heads, int n_rows, int n_batch, int max_nodes) {
  const char* me = "qhl_tree_attention_workspace";
  if (ta_check(me, kv, n_q_heads, n_rows, n_batch, max_nodes)) return 0;
  int sms = 0;
  const cudaError_t e = ta_device(&sms);
  if (e != cudaSuccess) {
    verify_cuda_err(me, e);
    return 0;
  }
  return ta_layout(kv->dim, n_q_heads / kv->kv_heads, n_batch, max_nodes, sms).total;
}

int qhl_tree_attention(const qhl_kv_pages* kv, int layer, int n_q_heads, int n_rows, int n_batch, int max_nodes,
                       const int* seq_dev, const int* q_start_dev, const int* parent_dev, const void* q_dev,
                       long long q_stride, const void* k_new_dev, const void* v_new_dev, long long new_stride,
                       void* out_dev, long long out_stride, float* lse_dev, float scale, void* workspace_dev,
                       size_t workspace_bytes, void* stream) {
  const char* me = "qhl_tree_attention";
  int rc = ta_check(me, kv, n_q_heads, n_rows, n_batch, max_nodes);
  if (rc) return rc;
  if (!seq_dev || !q_start_dev || !parent_dev || !q_dev || !k_new_dev || !v_new_dev || !out_dev || !workspace_dev)
    return verify_err(me, STAGE_E_ARG, "null pointer");
  if (layer < 0 || layer >= kv->n_layers) return verify_err(me, STAGE_E_ARG, "layer out of range");
  if (!(scale > 0) || !std::isfinite(scale)) return verify_err(me, STAGE_E_ARG, "scale must be positive");
  const long long qw = (long long)n_q_heads * kv->dim, kw = (long long)kv->kv_heads * kv->dim, most = 1LL << 38;
  if (!aligned16(q_dev) || !aligned16(k_new_dev) || !aligned16(v_new_dev) || !aligned16(out_dev) || !aligned16(workspace_dev) ||
      q_stride % 8 || new_stride % 8 || out_stride % 8)
    return verify_err(me, STAGE_E_ARG, "bases must be 16-byte aligned and strides multiples of 8");
  if (q_stride < qw || out_stride < qw || new_stride < kw || q_stride > most || new_stride > most || out_stride > most)
    return verify_err(me, STAGE_E_ARG, "a row stride is shorter than its heads, or too long");
  if (n_rows == 0) return 0;

  TaArgs a = {};
  cudaError_t e = ta_device(&a.grid);
  if (e == cudaSuccess) e = verify_error_word(&a.err);
  if (e != cudaSuccess) return verify_cuda_err(me, e);
  const int dim = kv->dim, G = n_q_heads / kv->kv_heads, KT = dim == 256 ? 64 : 128, CH = dim / 64, P = kv->page_rows;
  const bool bf16 = kv->dtype == QHL_BF16;
  const TaLayout l = ta_layout(dim, G, n_batch, max_nodes, a.grid);
  if (workspace_bytes < l.total)
    return verify_err(me, STAGE_E_ARG, "the workspace needs " + std::to_string(l.total) + " bytes");
  a.box = std::min(P, KT);
  a.dbox = std::min(KT, (max_nodes + 7) / 8 * 8);
  const uint16_t* kb = static_cast<const uint16_t*>(kv->k_dev) + (long long)layer * kv->stride_layer;
  const uint16_t* vb = static_cast<const uint16_t*>(kv->v_dev) + (long long)layer * kv->stride_layer;
  const long long pd[4] = {P, CH, kv->kv_heads, kv->n_pages}, ps[4] = {kv->stride_row, 64, kv->stride_head, kv->stride_page};
  const int kb4[4] = {a.box, a.box == KT ? CH : 1, 1, 1}, vb4[4] = {a.box, CH, 1, 1};
  const long long nd[4] = {n_rows, CH, kv->kv_heads, 1}, ns[4] = {new_stride, 64, dim, 64};
  const int nb[4] = {a.dbox, a.dbox == KT ? CH : 1, 1, 1};
  const bool fine = encode(&a.k, bf16, kb, pd, ps, kb4) && encode(&a.v, bf16, vb, pd, ps, vb4) && encode(&a.kn, bf16, k_new_dev, nd, ns, nb) &&
              encode(&a.vn, bf16, v_new_dev, nd, ns, nb);
  if (!fine) return verify_err(me, STAGE_E_UNSUPPORTED, "the driver refused a tensor map for these strides");
  auto log2i = [](int x) { int n = 0; while (1 << n < x) ++n; return n; };
  a.box_shift = log2i(a.box);
  a.page_shift = log2i(P);
  a.n_pages = kv->n_pages;
  a.max_pages = kv->max_pages;
  a.n_seqs = kv->n_seqs;
  a.Hkv = kv->kv_heads;
  a.G = G;
  a.n_rows = n_rows;
  a.n_batch = n_batch;
  a.max_nodes = max_nodes;
  a.table = kv->table_dev;
  a.len = kv->len_dev;
  a.seq = seq_dev;
  a.q_start = q_start_dev;
  a.parent = parent_dev;
  a.q = q_dev;
  a.q_stride = q_stride;
  a.v_new = v_new_dev;
  a.new_stride = new_stride;
  a.out = out_dev;
  a.out_stride = out_stride;
  a.lse = lse_dev;
  a.c = scale * 1.44269504088896340736f;
  uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
  a.head = reinterpret_cast<TaHead*>(ws);
  a.seqs = reinterpret_cast<TaSeq*>(ws + l.seqs);
  a.slot_rows = l.slot_rows;
  a.pml = reinterpret_cast<float2*>(ws + l.pml);
  a.po = reinterpret_cast<float*>(ws + l.po);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dim == 256)
    e = bf16 ? ta_launch<256, true>(a, s) : ta_launch<256, false>(a, s);
  else if (dim == 128)
    e = bf16 ? ta_launch<128, true>(a, s) : ta_launch<128, false>(a, s);
  else
    e = bf16 ? ta_launch<64, true>(a, s) : ta_launch<64, false>(a, s);
  return e == cudaSuccess ? 0 : verify_cuda_err(me, e);
}

}  // extern "C"
