// tc05.cuh - fifth-generation tensor core helpers (sm_103a), inline PTX:
// tensor memory allocation, tcgen05.mma of bf16 operands with fp32
// accumulators, tensor memory loads and stores, tiled TMA loads.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace cas {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---------------------------------------------------------------- tensor memory
// Warp-wide; the base address lands in shared memory. Columns: a power of two, 32..512.
__device__ __forceinline__ void tm_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tm_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Loads complete; the registers of one load pass through, so that no use of them moves before the wait.
__device__ __forceinline__ void tm_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: register j of a lane is column addr + j of
// its row. The address holds the lane in its upper and the column in its lower
// 16 bits; warp w of a warpgroup reaches lanes 32 (w % 4) to 32 (w % 4) + 31.
__device__ __forceinline__ void tm_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// ---------------------------------------------------------------- matrix products
// Instruction descriptor of kind::f16 with bf16 operands and fp32 accumulators:
// D type at bit 4, A and B types at 7 and 10, B transposed (N contiguous) at
// 16, N / 8 at 17, M / 16 at 24.
constexpr uint32_t tc_idesc_bf16(int M, int N, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_n_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Shared-memory operand in 128-byte swizzled atoms of 8 rows x 128 bytes (as a
// TMA load with 128B swizzle writes them; the tile 1024-byte aligned). K-major:
// rows are M or N, 1024 bytes between atoms of 8 rows. MN-major: rows are K,
// 1024 bytes between atoms of 8 k, `lead` bytes between atoms of 64 n. The lower
// half of a descriptor (address and lead) as a function of both; the upper half
// (stride 1024, version 1, 128-byte swizzle) is a constant.
constexpr uint32_t kTcDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t tc_desc_lo(uint32_t smem_addr, uint32_t lead) {
  return ((smem_addr & 0x3FFFF) >> 4) | (lead >> 4) << 16;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// A whole product of depth 128 (eight steps of 16) in one block: the warp is
// converged and one elected lane runs it, so that the descriptors stay in
// uniform registers and an instruction costs few issue slots of the SM
// sub-partition that the issuing warp shares with softmax warps (with eight
// separate statements in one thread: 1600 instead of 1190 clocks for two
// products while the softmax runs, 1024 by themselves).
#define CAS_MMA_SS(P, OFF)                                                                              \
  " add.u32 ta, %1, " #OFF ";\n add.u32 tb, %2, " #OFF ";\n mov.b64 da, {ta, %3};\n mov.b64 db, {tb, %3};\n" \
  " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " P ";\n"
// D = A B^T, A [128][128] and B [128][128] bf16, both K-major in halves of 64 k that are 16 KB apart.
__device__ __forceinline__ void tc_product_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile("{\n .reg .pred t, f;\n .reg .b32 ta, tb;\n .reg .b64 da, db;\n setp.eq.u32 t, 0, 0;\n"
               " setp.ne.u32 f, 0, 0;\n" CAS_MMA_SS("f", 0) CAS_MMA_SS("t", 2) CAS_MMA_SS("t", 4) CAS_MMA_SS("t", 6)
                   CAS_MMA_SS("t", 1024) CAS_MMA_SS("t", 1026) CAS_MMA_SS("t", 1028) CAS_MMA_SS("t", 1030) "}\n" ::"r"(d),
               "r"(a), "r"(b), "r"(kTcDescHi), "r"(idesc)
               : "memory");
}
#define CAS_MMA_TS(P, AO, BO)                                                                       \
  " add.u32 ta, %1, " #AO ";\n add.u32 tb, %2, " #BO ";\n mov.b64 db, {tb, %3};\n"                    \
  " tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, " P ";\n"
// D (+)= A B, A [128][128] bf16 pairs in 64 columns of tensor memory, B [128 k][128] bf16 MN-major.
__device__ __forceinline__ void tc_product_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile("{\n .reg .pred t, f;\n .reg .b32 ta, tb;\n .reg .b64 db;\n setp.eq.u32 t, 0, 0;\n"
               " setp.ne.u32 f, %5, 0;\n" CAS_MMA_TS("f", 0, 0) CAS_MMA_TS("t", 8, 128) CAS_MMA_TS("t", 16, 256)
                   CAS_MMA_TS("t", 24, 384) CAS_MMA_TS("t", 32, 512) CAS_MMA_TS("t", 40, 640) CAS_MMA_TS("t", 48, 768)
                       CAS_MMA_TS("t", 56, 896) "}\n" ::"r"(d),
               "r"(a), "r"(b), "r"(kTcDescHi), "r"(idesc), "r"(add)
               : "memory");
}
// The barrier completes when the tcgen05 operations that this thread issued so far have.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------- barriers and TMA
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// generic shared-memory writes before it are seen by the tensor cores and TMA after it
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 4-D tile load; coordinates innermost first, x0 * element size a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x0, int x1, int x2, int x3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x0), "r"(x1), "r"(x2), "r"(x3)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x0, int x1, int x2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x0), "r"(x1), "r"(x2)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------- arithmetic
// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// the largest of three; NaN loses
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace cas
