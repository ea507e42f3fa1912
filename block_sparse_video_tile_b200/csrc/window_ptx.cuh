// window_ptx.cuh -- 4-D TMA copies of the strided head tensors and small
// helpers shared by the window-attention kernels.
#pragma once

#include "vsa_ptx.cuh"
#include "window_args.cuh"

namespace vsa {

// Head tensors are seen by TMA as (d, N, H, B); a box is 64 channels of some
// consecutive rows of one head (c0 in {0, 64}: 128-byte boundaries).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* desc, uint32_t bar, int c0, int n, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(bar), "r"(c0), "r"(n), "r"(h), "r"(b)
      : "memory");
}
// Rows past N are not written.
__device__ __forceinline__ void tma_store_4d(const void* desc, uint32_t src, int c0, int n, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group"
      " [%0, {%2, %3, %4, %5}], [%1];" ::"l"(reinterpret_cast<uint64_t>(desc)),
      "r"(src), "r"(c0), "r"(n), "r"(h), "r"(b)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A branch that is never taken (units are positive).  It ends a basic block, so
// the compiler keeps the work of the chunks around it apart; without it the
// chunks' exponentials are interleaved and every store of P comes late
// (window_wan5b 675 us instead of 575).
__device__ __forceinline__ void sched_fence(const WinArgs& a) {
  if (a.unit < 0) asm volatile("nanosleep.u32 0;");
}

// The lowest n bits (n may lie outside [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

}  // namespace vsa
