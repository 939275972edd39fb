// tensor_core.cuh -- thin wrappers over the 5th-generation tensor core PTX of
// sm_103a (tcgen05) that the latent attention uses: tensor memory allocation,
// shared-memory and instruction descriptors, the bf16 and e4m3 / e5m2 matrix
// instructions with fp32 accumulators in tensor memory, their completion on an
// mbarrier, loads and stores of tensor memory, and the copies that feed them.
#pragma once

#include <cstdint>

#include "mla_device.cuh"

namespace mla {
// Arrives n times.
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// mbar_try_wait without suspending the thread.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; "
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

namespace tc {

// Tensor memory: `cols` columns (a power of two >= 32) of 128 lanes x 32 bits;
// the base address is written to shared memory.  One whole warp calls these.
__device__ __forceinline__ void alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
               : "memory");
}

// Order tensor-memory accesses around a synchronisation between threads.
__device__ __forceinline__ void fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Make this thread's view of shared memory (ordinary stores, its own or ones it
// has synchronised with) visible to the tensor core's reads.
__device__ __forceinline__ void fence_smem_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory operand with the 128-byte swizzle: rows of 128 bytes whose
// 16-byte units are permuted by XOR with the row number mod 8, in groups of 8
// rows (1024 bytes, 1024-byte aligned).
//   K-major (a row holds 64 consecutive k of one m or n): sbo = bytes from one
//     group of 8 rows to the next; lbo unused.
//   MN-major (a row holds 64 consecutive m of one k): sbo = bytes from one group
//     of 8 k to the next, lbo = bytes from one run of 64 m to the next.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, M x N tile, A MN-major or K-major, B
// K-major.  fa / fb: 1 for bf16 (mma_bf16); 0 for e4m3, 1 for e5m2 (mma_fp8).
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, bool a_mn, int fa, int fb) {
  return (1u << 4) | ((uint32_t)fa << 7) | ((uint32_t)fb << 10) | (a_mn ? 1u << 15 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}

// D[tmem] (+)= A * B for one k step of 16.  The whole (converged) warp runs these
// two statements and `lane` holds in the one lane that issues: without a branch
// around them, descriptors that are the same in all lanes are computed in uniform
// registers, where the instruction wants them.
__device__ __forceinline__ void mma_bf16(bool lane, uint32_t d, uint64_t a, uint64_t b,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %4, 0; setp.ne.u32 q, %5, 0;\n"
      "  @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(lane ? 1u : 0u)
      : "memory");
}
// The same for fp8 operands (of either format each): one k step of 32.
__device__ __forceinline__ void mma_fp8(bool lane, uint32_t d, uint64_t a, uint64_t b,
                                        uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %4, 0; setp.ne.u32 q, %5, 0;\n"
      "  @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(lane ? 1u : 0u)
      : "memory");
}
// Arrive on `bar` when every matrix instruction that lane has issued is done.
__device__ __forceinline__ void commit(bool lane, uint32_t bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.u32 q, %1, 0;\n"
      "  @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
      "r"(lane ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The loads wait for their registers in the same statement, so that no use of
// them can be moved in front of the wait.  Whole warps call them converged.
//
// 16 lanes x 8 columns per group of 4 registers: thread t gets, of group j,
// lane t / 4 columns 8 j + 2 (t % 4) and + 1 in r[4 j], r[4 j + 1], and lane
// t / 4 + 8 in r[4 j + 2], r[4 j + 3].  G groups.
template <int G>
__device__ __forceinline__ void ld_16x256(uint32_t addr, uint32_t* r) {
  static_assert(G == 2 || G == 4, "groups built");
  if constexpr (G == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
  }
}

// 32 lanes x 16 columns: thread t gets lane t's 16 columns.
__device__ __forceinline__ void ld_32x16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void st_32x16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Four 8x8 matrices of 16-bit values stored transposed: thread t holds, of
// matrix i, row t / 4 columns 2 (t % 4) and + 1 in r_i; column c of matrix i goes
// to the 16 bytes whose address thread 8 i + c passes.
__device__ __forceinline__ void st_8x8_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                         uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// 16 bytes global -> shared, asynchronously; zeros when !valid (src is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16u : 0u)
               : "memory");
}
// The L2 policy of loads: first to be evicted, or as usual.
__device__ __forceinline__ uint64_t l2_policy(bool first) {
  uint64_t p;
  if (first) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// One box of a 3-dimensional tensor map to shared memory, completing on `bar`
// (parts outside the tensor are filled with zeros; x * element size a multiple of
// 16 bytes).
__device__ __forceinline__ void tma_load3(uint32_t dst, const void* map, int x, int y, int z,
                                          uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
// Arrive on `bar` when this thread's cp_async16 so far are done.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace tc
}  // namespace mla
