// Building blocks of the tcgen05 kernels (csa_cache_attend_wide.cu,
// csa_prompt_*.cu): mbarriers with bounded waits, matrix instructions, tensor
// memory, shared-memory operands, tiles copied by TMA. Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace csa {

constexpr int kPolls = 1 << 20;  // of a wait: a poll that fails takes about 2700 cycles, all of them 1.4 s

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded: after kPolls the CTA is marked dead and no further wait waits.
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, volatile int32_t* dead) {
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i) {
    if (mbar_try(bar, parity)) return;
    if (*dead) return;
  }
  *dead = 1;
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One matrix instruction, and the arrival on a barrier when all before it are
// done: called by a converged warp, executed by its elected lane.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// The same value in every lane, which the compiler then keeps in uniform
// registers, where the matrix instructions take their operands from.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
#define CSA_R10(b) "%" #b "0, %" #b "1, %" #b "2, %" #b "3, %" #b "4, %" #b "5, %" #b "6, %" #b "7, %" #b "8, %" #b "9"
__device__ __forceinline__ void tc_load32(uint32_t at, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, " CSA_R10(1) ", " CSA_R10(
          2) ", %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_store32(uint32_t at, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, " CSA_R10(1) ", " CSA_R10(
          2) ", %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(at)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
#undef CSA_R10
// Whether any of the `threads` threads of barrier `id` says so.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)mine), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void barrier_of(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Shared-memory operand in the 128-byte swizzle: groups of 8 rows of 128 bytes,
// 1024 bytes apart; `lead` bytes between 64-wide slabs of an M- or N-major one.
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t lead) {
  return (uint64_t)((at >> 4) & 0x3FFF) | ((uint64_t)((lead >> 4) & 0x3FFF) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same for a warp that elects its lane once (tc_leader) and keeps it: an election
// for each instruction made the issue, not the tensor core, the bound of the prompt
// kernels (a tile of the keys kernel 3060 cycles, its products 2048).
__device__ __forceinline__ uint32_t tc_leader() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tc_commit_by(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
// Four steps of 16 along the products' inner dimension, STEP (in units of 16 bytes) apart
// in the operands of shared memory; together, so that their predicates and operands are
// worked out once.
#define CSA_MMA4(A_DECL, A_REG, A_NEXT, A_ARG, STEP)                                                         \
  asm volatile(                                                                                               \
      "{\n\t.reg .pred p, q, t;\n\t" A_DECL                                                                  \
      ".reg .b64 b1, b2, b3;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"  \
      "add.s64 b1, %2, %6;\n\tadd.s64 b2, b1, %6;\n\tadd.s64 b3, b2, %6;\n\t" A_NEXT                         \
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], " A_REG("%1") ", %2, %3, p;\n\t"                          \
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], " A_REG("a1") ", b1, %3, t;\n\t"                          \
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], " A_REG("a2") ", b2, %3, t;\n\t"                          \
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], " A_REG("a3") ", b3, %3, t;\n\t}" ::"r"(d),               \
      A_ARG(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader), "n"(STEP)                                \
      : "memory")
#define CSA_SMEM_A(x) x
#define CSA_TMEM_A(x) "[" x "]"
template <int STEP>
__device__ __forceinline__ void tc_mma4(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  CSA_MMA4(".reg .b64 a1, a2, a3;\n\t", CSA_SMEM_A, "add.s64 a1, %1, %6;\n\tadd.s64 a2, a1, %6;\n\tadd.s64 a3, a2, %6;\n\t",
           "l", STEP);
}
// With a first operand in tensor memory: lanes are rows, a column holds two 16-bit
// values, a step has eight.
template <int STEP>
__device__ __forceinline__ void tc_mma4_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  CSA_MMA4(".reg .b32 a1, a2, a3;\n\t", CSA_TMEM_A, "add.s32 a1, %1, 8;\n\tadd.s32 a2, a1, 8;\n\tadd.s32 a3, a2, 8;\n\t", "r",
           STEP);
}
#undef CSA_MMA4
#undef CSA_SMEM_A
#undef CSA_TMEM_A
// 32 columns of a warp's 32 lanes, without waiting; tc_loaded(v) must follow
// tc_load_wait() before v is used (it ties the values to the wait).
#define CSA_R32(r)                                                                                               \
  "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, " \
  "%23, %24, %25, %26, %27, %28, %29, %30, %31}"
__device__ __forceinline__ void tc_load32_async(uint32_t at, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " CSA_R32(r) ", [%32];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                 "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
                 "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
                 "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
                 "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
               : "r"(at));
}
__device__ __forceinline__ void tc_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_loaded(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                 "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                 "+f"(v[29]));
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}
// 16 words a lane, without waiting (tc_store_wait).
__device__ __forceinline__ void tc_store16_async(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tc_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- tiles by TMA -----------------------------------------------------------

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of [tokens][heads][64 columns] to shared memory, in the 128-byte swizzle.
// col: a multiple of 64.
__device__ __forceinline__ void tma_load(uint32_t to, const CUtensorMap* map, int col, int head, int token,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(to),
      "l"(map), "r"(col), "r"(head), "r"(token), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace csa
