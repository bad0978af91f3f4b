// PTX of the serving kernels beside what ptx.cuh has: conversions of 8-bit
// terms, words of shared memory, and single-CTA MMAs several a statement.
#pragma once

#include "ptx.cuh"

namespace mla {

// f16 pairs (the low half holds the first): from floats, their difference and
// sum, their E5M2 codes (two bytes), all rounded to nearest even, and each added
// to a float.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fadd_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void add_f16x2(float& lo, float& hi, uint32_t a) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
      : "+f"(lo), "+f"(hi) : "r"(a));
}
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(a));
  return r;
}

// Two E4M3 codes (low 16 bits) to floats, exactly.
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t pair) {
  float2 f;
  asm("{\n\t.reg .b16 in, l, h;\n\t.reg .b32 hx;\n\t"
      "cvt.u16.u32 in, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 hx, in;\n\t"
      "mov.b32 {l, h}, hx;\n\t"
      "cvt.f32.f16 %0, l;\n\t"
      "cvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y) : "r"(pair));
  return f;
}

// idesc_e4m3 with the format codes of A and B (0: E4M3, 1: E5M2), which need not
// be alike, and B MN-major.
__host__ __device__ constexpr uint32_t idesc_8bit(int M, int N, int a_format, int b_format, bool b_mn) {
  return idesc_e4m3(M, N) | ((uint32_t)a_format << 7) | ((uint32_t)b_format << 10) | ((b_mn ? 1u : 0u) << 16);
}

// A word of shared memory.
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A box of a tensor map into L2.
__device__ __forceinline__ void tma_prefetch_l2_2d(const void* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// Arrives on a barrier of the cluster and expects `bytes` on it (relaxed: the barrier only counts bytes).
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes)
               : "memory");
}

// The single-CTA forms (cta_group::1, M = 128) from one elected lane of a
// converged warp, some consecutive K steps a statement: the lane is elected and
// branched to once, and the operands move by constants (descriptors count 16
// bytes).  One statement an MMA takes a third more code, and the instruction
// cache paces kernels whose roles all run unrolled.
//   ts4: A in TMEM, 8 columns a step, B 32 bytes a step
//   ss4: A and B 32 bytes a step
#define MLA_ELECT(body) "{\n\t.reg .pred e, p, q;\n\t.reg .b64 x, y;\n\t.reg .b32 a;\n\t"          \
                        "elect.sync _|e, 0xffffffff;\n\t@!e bra DONE%=;\n\t"                       \
                        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t" body "DONE%=:\n\t}"
#define MLA_TS(kind, acols, badd, acc)                                                          \
  "add.u32 a, %1, " acols ";\n\tadd.u64 x, %2, " badd ";\n\t"                                   \
  "tcgen05.mma.cta_group::1.kind::" kind " [%0], [a], x, %3, " acc ";\n\t"
#define MLA_SS(kind, aadd, badd, idesc, acc)                                                    \
  "add.u64 x, %1, " aadd ";\n\tadd.u64 y, %2, " badd ";\n\t"                                    \
  "tcgen05.mma.cta_group::1.kind::" kind " [%0], x, y, " idesc ", " acc ";\n\t"
__device__ __forceinline__ void mma_ts4_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(MLA_ELECT(MLA_TS("f16", "0", "0", "p") MLA_TS("f16", "8", "2", "q") MLA_TS("f16", "16", "4", "q")
                             MLA_TS("f16", "24", "6", "q"))::"r"(d_tmem),
               "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
__device__ __forceinline__ void mma_ss4_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(MLA_ELECT(MLA_SS("f16", "0", "0", "%3", "p") MLA_SS("f16", "2", "2", "%3", "q")
                             MLA_SS("f16", "4", "4", "%3", "q") MLA_SS("f16", "6", "6", "%3", "q"))::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
// Two 8-bit terms of A, the second 128 TMEM columns on, against the same B.
__device__ __forceinline__ void mma_ts4x2_8bit_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                     uint32_t accumulate) {
  asm volatile(MLA_ELECT(MLA_TS("f8f6f4", "0", "0", "p") MLA_TS("f8f6f4", "128", "0", "q")
                             MLA_TS("f8f6f4", "8", "2", "q") MLA_TS("f8f6f4", "136", "2", "q")
                             MLA_TS("f8f6f4", "16", "4", "q") MLA_TS("f8f6f4", "144", "4", "q")
                             MLA_TS("f8f6f4", "24", "6", "q") MLA_TS("f8f6f4", "152", "6", "q"))::"r"(d_tmem),
               "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
// Two K steps with B MN-major (2048 bytes a step of 16 rows).
__device__ __forceinline__ void mma_ss2_mn_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(MLA_ELECT(MLA_SS("f16", "0", "0", "%3", "p") MLA_SS("f16", "2", "128", "%3", "q"))::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
// Two K steps of two 8-bit terms of A, the second 16 KB on, with B MN-major
// (4096 bytes a step of 32 rows).
__device__ __forceinline__ void mma_ss2x2_mn_8bit_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                        uint32_t accumulate) {
  asm volatile(MLA_ELECT(MLA_SS("f8f6f4", "0", "0", "%3", "p") MLA_SS("f8f6f4", "1024", "0", "%3", "q")
                             MLA_SS("f8f6f4", "2", "256", "%3", "q") MLA_SS("f8f6f4", "1026", "256", "%3", "q"))::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}
#undef MLA_ELECT
#undef MLA_TS
#undef MLA_SS
// Completion of the CTA's MMAs issued so far: on a barrier of this CTA, or on
// the barrier at the same offset in every CTA of the cluster that `mask` names.
__device__ __forceinline__ void mma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_commit_mc_elect(uint32_t bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(mask)
      : "memory");
}

}  // namespace mla
