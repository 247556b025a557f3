// Inline PTX for the 5th-generation tensor cores on sm_103a: tensor memory,
// block-scaled products with operands in shared memory, and the tiled TMA
// load that pads 4-bit codes out to 8-bit containers.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"

namespace ep {

// One lane of a converged warp, the same each time. Instructions whose
// operands must be uniform over the warp (products, copies, their barriers)
// are issued under this by a warp that runs its loop as a whole: inside a
// branch on the thread index each of them cost 84 cycles to issue, under this
// the products' own 51 (at 64 columns and fewer) to 96 (at 192).
__device__ __forceinline__ bool elect_one() {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A value that every lane holds, known to the compiler as such.
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// mbar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, unsigned parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// The 128 threads of barrier 1 meet: whether all of them go on. A thread whose
// wait has run out may not leave alone, since the others meet there again.
__device__ __forceinline__ bool all_agree(bool ok) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Registers of a warpgroup's threads, taken from or given back to what the
// block was launched with (all four warps call it).
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Whether the phase has completed, without waiting: non-zero. The answer takes
// about 100 cycles, so a loop that has other work asks a turn ahead (raw, and
// mbar_wait_asked when it needs to know) instead of standing still.
__device__ __forceinline__ unsigned mbar_ask(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok;
}

// By a whole warp: waits for the phase unless `asked` says it has completed.
__device__ __forceinline__ bool mbar_wait_asked(unsigned asked, uint64_t* bar, unsigned parity, int32_t* status) {
  return __all_sync(0xffffffffu, asked != 0) || mbar_wait_warp(bar, parity, status);
}

// ---- tensor memory ---------------------------------------------------------
// Whole warp; the column count is a power of two >= 32. The base address
// appears at *slot (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, unsigned columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t base, unsigned columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Eight columns of this thread's lane (warp w of a warpgroup: lanes 32 w ..).
// (Straight into v: a copy of a register would read it before the wait.)
__device__ __forceinline__ void tmem_load8(float (&v)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}

// 32 columns of it.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

// What tmem_load8 asked for has arrived in v (and in w). Each register is an operand:
// what reads one that is not may be moved in front of the wait.
__device__ __forceinline__ void tmem_wait_load(float (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]),
                 "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_load(float (&v)[8], float (&w)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]),
                 "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(w[0]), "+f"(w[1]),
                 "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]),
                 "+f"(w[7])
               :
               : "memory");
}

// ---- shared-memory matrix descriptors ----------------------------------------
// Rows of 128 bytes in the 128-byte swizzle (16-byte piece c of row r lies at
// piece c ^ (r % 8)), groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_rows128(uint32_t addr) {
  return (static_cast<uint64_t>(addr) >> 4 & 0x3FFF) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}

// The transposed operand: rows of 128 bytes along the outputs, one row an
// input, in the same swizzle; groups of eight inputs lie 1024 bytes apart,
// groups of 128 outputs `apart` bytes.
__device__ __forceinline__ uint64_t desc_inputs128(uint32_t addr, uint32_t apart) {
  return (static_cast<uint64_t>(addr) >> 4 & 0x3FFF) | static_cast<uint64_t>(apart >> 4) << 16 |
         uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// Rows of 16 bytes one after the other (the scale factors' 32 x 128 bits).
__device__ __forceinline__ uint64_t desc_rows16(uint32_t addr) {
  return (static_cast<uint64_t>(addr) >> 4 & 0x3FFF) | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}

// 32 rows of 128 bits from shared memory into four columns, the same in each
// of the four 32-lane quarters: one scale byte a row for four steps of 32.
__device__ __forceinline__ void tmem_copy_scales(uint32_t column, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(column), "l"(desc) : "memory");
}

// ---- block-scaled product ------------------------------------------------------
// D[128, N] (+)= A[128, 32] B[N, 32]^T, A in E2M1, B in E4M3, a UE8M0 scale for
// each row of either. The instruction descriptor: B's scale byte at bit 4, A's
// type (5: E2M1) at 7, B's type (0: E4M3) at 10, N / 8 at 17, UE8M0 scales at
// 23, M / 16 at 24, A's scale byte at 29.
__device__ __forceinline__ uint32_t idesc_e2m1_e4m3(int n) {
  return 5u << 7 | static_cast<uint32_t>(n / 8) << 17 | 1u << 23 | (128u / 16u) << 24;
}
__device__ __forceinline__ uint32_t idesc_scale_byte(uint32_t idesc, unsigned byte) {
  return idesc | byte << 4 | byte << 29;
}

__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                           uint32_t sb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// ---- product of 8-bit operands ---------------------------------------------------
// D[M, N] (+)= A[M, 32] B[N, 32]^T, both E4M3, fp32 sums. The instruction
// descriptor: fp32 sums (1) at bit 4, the operands' types (0: E4M3) at 7 and 10,
// B transposed at 16, N / 8 at 17, M / 16 at 24.
__device__ __forceinline__ uint32_t idesc_e4m3(unsigned m, unsigned n, bool b_transposed) {
  return 1u << 4 | (b_transposed ? 1u << 16 : 0u) | n / 8 << 17 | m / 16 << 24;
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// Arrive on an mbarrier once every product and copy issued so far by this
// thread has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// ---- tensor maps (host) ----------------------------------------------------------
// cuTensorMapEncodeTiled, asked of the driver once (launch_cache.cu); null on failure.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();

// A tensor map on its way to where loads look for it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tiled TMA load --------------------------------------------------------------
__device__ __forceinline__ void tma_load_2d(void* smem_dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace ep
