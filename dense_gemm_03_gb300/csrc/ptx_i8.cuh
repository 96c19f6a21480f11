// ptx_i8.cuh -- inline PTX of the kernels of 8-bit integers, beside ptx.cuh.
#pragma once
#include "ptx_tmem_st.cuh"

namespace gb300 {

// The untiled copy: global to shared, addresses and size multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], halves, one thread issues.  A in tensor memory: lane = row, two K-neighbours to a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two 16 x 16 matrices of bytes, transposed: lanes 0-15 (16-31) give the addresses of the
// first's (second's) rows; thread 4 g + t receives of each bytes 4 t .. 4 t + 3 of the
// transpose's rows g and g + 8.
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared::cta.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

}  // namespace gb300
