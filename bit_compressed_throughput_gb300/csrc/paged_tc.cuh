// What the tensor-core kernels over the paged 4-bit cache share (sm_103a): bounded waits, copies,
// shared and tensor memory access, and the extents of a call's sequences.
#pragma once
#include <stdint.h>

#include "attn_tc.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "paged.cuh"
#include "paged_work.cuh"

namespace fg {
namespace paged {

constexpr int BOX = 128 * 128;             // bytes of one 64-column x 128-row fp16 box
constexpr uint32_t TMEM_COLS = 512;
constexpr long long kWaitCycles = 1ll << 36;   // a row on its own may keep other warps waiting
constexpr long long kDrainCycles = 1ll << 32;  // for copies and products in flight
constexpr unsigned int kErrWait = 1u, kErrDrain = 2u;

__device__ __forceinline__ bool extent_of(const PagedAttn& a, int b, PagedSeq& e) {
  const int q0 = a.q_off[b], q1 = a.q_off[b + 1], n = a.lens[b];
  if (q0 < 0 || q0 > q1 || q1 > a.q_rows || q1 - q0 > a.max_q || n < 0 || n > a.cache.cap())
    return false;
  e = PagedSeq{q0, q1 - q0, n};
  return true;
}

// A wait that ran out, or another warp's.
static __device__ __noinline__ bool gave_up(long long t0, volatile int* abort_flag,
                                     unsigned int* word) {
  if (*abort_flag) return true;
  if (clock64() - t0 <= kWaitCycles) return false;
  *abort_flag = 1;
  atomicOr(word, kErrWait);
  return true;
}
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned int* word) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  for (unsigned n = 1;; ++n) {
    if (mbar_try(bar, parity)) return true;
    if ((n & 63u) == 0 && gave_up(t0, abort_flag, word)) return false;
  }
}
__device__ __forceinline__ void bounded_drain(uint32_t bar, uint32_t parity, unsigned int* word) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (clock64() - t0 > kDrainCycles) {
      atomicOr(word, kErrDrain);
      return;
    }
  }
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
// 16 TMEM columns, and the wait that ties them to it; 8 columns stored.
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld_dep(float (&v)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
        "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
        "+f"(v[14]), "+f"(v[15])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

}  // namespace paged
}  // namespace fg
