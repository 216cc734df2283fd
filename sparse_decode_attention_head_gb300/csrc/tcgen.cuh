// tcgen05 (fifth-generation tensor core) and tensor-memory primitives.
//
// Tensor memory (TMEM) is 128 lanes x 512 columns of 32 bits an SM; an address
// is lane << 16 | column, and warp w of a block reaches lanes 32 (w % 4) on.
// A matrix instruction is issued by one thread and runs asynchronously, in
// order with the others of that thread; its completion arrives on an mbarrier
// through a commit.
#pragma once

#include "sa_common.cuh"

namespace sa {

// One whole warp; the column count is a power of two from 32 on.
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_addr, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_addr)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives once on `bar` when every matrix instruction that this thread has
// issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, `lbo`
// (the stride between 64-value blocks of an operand whose rows run along the
// inner dimension of the product's output; unused for the other kind) and
// `sbo` (the stride between groups of 8 rows), in bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}

// Instruction descriptor: bf16 operands, fp32 accumulator, M x N tile; b_rows:
// B is stored with its rows along K (the output's N dimension is contiguous).
__host__ __device__ constexpr uint32_t bf16_idesc(int M, int N, bool b_rows) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// D (+)= A B, 16 values of K; A in shared memory (ss) or in TMEM (ts).
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// TMEM <-> registers, one lane a thread, 32 columns a call.  The load returns
// complete: nothing may use the registers ahead of the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
// 64 columns into v[O ..]: under way after the first call, there after the
// second (which names the registers, so that nothing reads them ahead of it).
template <int O, int N>
__device__ __forceinline__ void tmem_ld64_start(uint32_t addr, float (&v)[N]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, "
      "%44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
      "[%64 + 32];"
      : "=f"(v[O + 0]), "=f"(v[O + 1]), "=f"(v[O + 2]), "=f"(v[O + 3]), "=f"(v[O + 4]), "=f"(v[O + 5]), "=f"(v[O
        + 6]), "=f"(v[O + 7]), "=f"(v[O + 8]), "=f"(v[O + 9]), "=f"(v[O + 10]), "=f"(v[O + 11]), "=f"(v[O +
        12]), "=f"(v[O + 13]), "=f"(v[O + 14]), "=f"(v[O + 15]), "=f"(v[O + 16]), "=f"(v[O + 17]), "=f"(v[O +
        18]), "=f"(v[O + 19]), "=f"(v[O + 20]), "=f"(v[O + 21]), "=f"(v[O + 22]), "=f"(v[O + 23]), "=f"(v[O +
        24]), "=f"(v[O + 25]), "=f"(v[O + 26]), "=f"(v[O + 27]), "=f"(v[O + 28]), "=f"(v[O + 29]), "=f"(v[O +
        30]), "=f"(v[O + 31]), "=f"(v[O + 32]), "=f"(v[O + 33]), "=f"(v[O + 34]), "=f"(v[O + 35]), "=f"(v[O +
        36]), "=f"(v[O + 37]), "=f"(v[O + 38]), "=f"(v[O + 39]), "=f"(v[O + 40]), "=f"(v[O + 41]), "=f"(v[O +
        42]), "=f"(v[O + 43]), "=f"(v[O + 44]), "=f"(v[O + 45]), "=f"(v[O + 46]), "=f"(v[O + 47]), "=f"(v[O +
        48]), "=f"(v[O + 49]), "=f"(v[O + 50]), "=f"(v[O + 51]), "=f"(v[O + 52]), "=f"(v[O + 53]), "=f"(v[O +
        54]), "=f"(v[O + 55]), "=f"(v[O + 56]), "=f"(v[O + 57]), "=f"(v[O + 58]), "=f"(v[O + 59]), "=f"(v[O +
        60]), "=f"(v[O + 61]), "=f"(v[O + 62]), "=f"(v[O + 63])
      : "r"(addr)
      : "memory");
}
template <int O, int N>
__device__ __forceinline__ void tmem_ld64_finish(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[O + 0]), "+f"(v[O + 1]), "+f"(v[O + 2]), "+f"(v[O + 3]), "+f"(v[O + 4]), "+f"(v[O + 5]), "+f"(v[O
                 + 6]), "+f"(v[O + 7]), "+f"(v[O + 8]), "+f"(v[O + 9]), "+f"(v[O + 10]), "+f"(v[O + 11]), "+f"(v[O +
                 12]), "+f"(v[O + 13]), "+f"(v[O + 14]), "+f"(v[O + 15]), "+f"(v[O + 16]), "+f"(v[O + 17]), "+f"(v[O +
                 18]), "+f"(v[O + 19]), "+f"(v[O + 20]), "+f"(v[O + 21]), "+f"(v[O + 22]), "+f"(v[O + 23]), "+f"(v[O +
                 24]), "+f"(v[O + 25]), "+f"(v[O + 26]), "+f"(v[O + 27]), "+f"(v[O + 28]), "+f"(v[O + 29]), "+f"(v[O +
                 30]), "+f"(v[O + 31]), "+f"(v[O + 32]), "+f"(v[O + 33]), "+f"(v[O + 34]), "+f"(v[O + 35]), "+f"(v[O +
                 36]), "+f"(v[O + 37]), "+f"(v[O + 38]), "+f"(v[O + 39]), "+f"(v[O + 40]), "+f"(v[O + 41]), "+f"(v[O +
                 42]), "+f"(v[O + 43]), "+f"(v[O + 44]), "+f"(v[O + 45]), "+f"(v[O + 46]), "+f"(v[O + 47]), "+f"(v[O +
                 48]), "+f"(v[O + 49]), "+f"(v[O + 50]), "+f"(v[O + 51]), "+f"(v[O + 52]), "+f"(v[O + 53]), "+f"(v[O +
                 54]), "+f"(v[O + 55]), "+f"(v[O + 56]), "+f"(v[O + 57]), "+f"(v[O + 58]), "+f"(v[O + 59]), "+f"(v[O +
                 60]), "+f"(v[O + 61]), "+f"(v[O + 62]), "+f"(v[O + 63])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
        "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
        "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// One lane of a converged warp.  Matrix instructions and copies take uniform
// operands: a warp that computes them together and elects a lane to issue
// keeps them in uniform registers, a lane alone has to move each one there.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Two fp32 in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Registers of a whole warpgroup; the shares add up to what the block was
// launched with.
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace sa
