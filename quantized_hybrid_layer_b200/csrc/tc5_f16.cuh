// The 16-bit floating-point form of the fifth-generation tensor core
// (tcgen05.mma kind::f16, f32 accumulators), tiled TMA loads, and their
// descriptors.  tc5.cuh has the allocation, ordering and commit primitives.
#pragma once

#include <cuda.h>

#include "tc5.cuh"

namespace qhl {

// ---- shared-memory matrix descriptors, 128-byte swizzle ---------------------
// Tiles are stored as rows of 128 bytes (64 elements), 8 rows to a 1024-byte
// swizzle atom, as a TMA load with CU_TENSOR_MAP_SWIZZLE_128B writes them (the
// 16-byte unit u of row r sits at unit u ^ (r % 8)).  Bits as in tc5.cuh, with
// swizzle mode 2 (128 bytes) in bits 61-63.
//   K-major (rows = M or N index, 128 bytes of K): sbo = 1024 to the next 8 rows;
//     a step of 16 elements along K advances the start address by 32 bytes.
//   MN-major (rows = K index, 128 bytes of N): sbo = 1024 to the next 8 of K, lbo
//     to the next 64 of N; a step of 16 along K advances it by 2048 bytes.
QHL_DEV uint64_t smem_desc_sw128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// ---- instruction descriptor of kind::f16 -----------------------------------
// D f32 (bits 4-5 = 1), A and B both f16 (0) or both bf16 (1) (bits 7-9 and
// 10-12), B's major order (bit 16: 1 = N), N >> 3 (bits 17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool b_mn_major, int m, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (=|+=) A * B^T over K = 16, A in tensor memory (row m in lane m, two
// elements of K to a column), B in shared memory.  Asynchronous, issued by one
// thread; completion through tc_commit.
QHL_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// ---- TMEM -> registers, 32 consecutive columns of the thread's lane ----------
QHL_DEV void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// registers -> TMEM, 16 consecutive columns of the thread's lane
QHL_DEV void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---- tiled TMA loads into this CTA's shared memory ---------------------------
// The innermost coordinate is always 0, so every copy starts on the tensor's
// (16-byte aligned) row.
QHL_DEV void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
QHL_DEV void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// One lane of a converged warp.
QHL_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p)
      :
      : "memory");
  return p != 0;
}

// 2^x by the hardware's approximation (relative error below 2^-22; 0 at -inf).
QHL_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace qhl
