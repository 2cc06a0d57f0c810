// tcgen05 (5th-generation tensor core) helpers shared by the kernels that
// issue MMAs from shared-memory operands into tensor memory: the operand
// descriptor of a K-major tile in the 128-byte swizzled layout, the
// instruction descriptor of a bf16 x bf16 -> fp32 MMA, the MMA and commit,
// the thread-sync fences and tensor-memory loads / stores (inline PTX).
#pragma once

#include <cuda.h>

#include "s2_common.cuh"

namespace s2 {

// Shared-memory matrix descriptor: K-major operand, 128-byte swizzle, rows of
// 128 bytes in 8-row (1024-byte) atoms.
S2_DEV uint64_t smem_desc_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)1 << 16;             // leading byte offset (unused for swizzled K-major)
  d |= (uint64_t)(1024 >> 4) << 32;   // stride byte offset: 8 rows x 128 B
  d |= (uint64_t)1 << 46;             // descriptor version (sm_100 family)
  d |= (uint64_t)2 << 61;             // 128-byte swizzle
  return d;
}

// Instruction descriptor: kind::f16, bf16 A and B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

S2_DEV void umma_bf16(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(tmem_d), "l"(a), "l"(b), "r"(idesc), "r"(accum) : "memory");
}
S2_DEV void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(smem_u32(bar)) : "memory");
}
S2_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
S2_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

S2_DEV void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 consecutive 32-bit columns of this thread's tensor-memory lane (one
// load, one wait).
S2_DEV void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 consecutive 32-bit columns of this thread's tensor-memory lane into
// ``taddr`` (warp w owns lanes 32w..32w+31), then wait for the store.
S2_DEV void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
      :: "r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
         "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
         "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Block-scaled MMA (kind::mxf8f6f4): e2m1 A and e4m3 B, both K-major in
// shared memory (e2m1: 16 values in 8 of each 16 bytes), one power-of-two scale
// (ue8m0) per row and 32 k, fp32 D.  One instruction covers 32 k; the byte of
// the scale columns' words that it takes is ``sf`` for both operands.
__host__ __device__ constexpr uint32_t idesc_e2m1_e4m3(int m, int n, int sf) {
  return ((uint32_t)sf << 4) | (5u << 7) | (0u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 4) << 24) | ((uint32_t)sf << 29);
}
// Descriptors by their low words, address / 16 (the high words are constants):
// operands in 128-byte swizzled rows, scales without a swizzle, eight rows of
// 16 bytes after eight.
S2_DEV uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) & 0x3FFF; }
constexpr uint32_t kDescHiSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHiScales = (128 >> 4) | (1u << 14);
S2_DEV void umma_mxf8f6f4(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t tmem_sfa,
                          uint32_t tmem_sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 x, {%1, %7};\n\tmov.b64 y, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], x, y, %3, [%4], [%5], p;\n\t}"
      :: "r"(tmem_d), "r"(a), "r"(b), "r"(idesc), "r"(tmem_sfa), "r"(tmem_sfb), "r"(accum), "r"(kDescHiSw128)
      : "memory");
}
// A scale tile (32 rows of 16 bytes, contiguous) from shared memory into four
// tensor-memory columns, repeated in each quarter of the lanes.
S2_DEV void tmem_cp_scales(uint32_t taddr, uint32_t scales) {
  asm volatile(
      "{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], x;\n\t}"
      :: "r"(taddr), "r"(scales), "r"(kDescHiScales) : "memory");
}

// One lane of a converged warp, chosen such that the compiler knows that it is
// one: the operands of products and copies then go to uniform registers as they
// are, where a branch by lane number has each of them moved there in a loop over
// lanes.
S2_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// 2-D tiled TMA load of the box at (x = column, y = row) of `map` into shared
// memory, completing on `bar` (the _hint form carries an L2 cache policy).
S2_DEV void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y),
         "r"(smem_u32(bar))
      : "memory");
}
S2_DEV void tma_load_2d_hint(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                             uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y),
         "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

// Byte offset of the 16-byte unit ``c`` (0..7) of row ``r`` in a K-major tile
// of 128-byte rows in the 128-byte swizzled layout (the layout the TMA
// engine writes with 128-byte swizzle): 8-row atoms of 1,024 bytes, the unit
// index XORed with the row's index within its atom.  The tile must start on
// a 1,024-byte boundary.
S2_DEV uint32_t sw128_offset(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// Thread-block cluster: barrier over all CTAs of the cluster (release /
// acquire: shared-memory writes before it are visible to the partners'
// distributed-shared-memory reads after it), and a load from partner CTA
// ``rank``'s shared memory at the address ``local`` has in this CTA.
S2_DEV void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
S2_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
S2_DEV float ld_dsmem_f32(const float* local, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra));
  return v;
}
// Four consecutive floats (16-byte aligned) from partner CTA ``rank``.
S2_DEV float4 ld_dsmem_f32x4(const float* local, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(ra));
  return v;
}

}  // namespace s2
