// umma_m64.cuh -- helpers of the kernels that use M = 64 tcgen05 products: their
// accumulators' rows lie in lanes 0..15 of each quarter of the tensor memory
// (row r in lane 32 (r / 16) + r % 16).
#pragma once

#include <stdint.h>

namespace csa2 {

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Barrier of N threads of the CTA.
template <int N>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
// The same, and whether all of them said so.
template <int N>
__device__ __forceinline__ bool bar_and(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "n"(N)
      : "memory");
  return r != 0;
}
// Each thread of a warp reads 2 x 2 of eight columns, of 16 lanes: columns 2
// (lane % 4) + {0, 1} of lane lane / 4, then of lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x1(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
// The same of 16 columns: r[4 n + 2 k + e] is column 8 n + 2 (lane % 4) + e
// of lane lane / 4 + 8 k.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

}  // namespace csa2
