// Shared by the paged attention kernels: bounded waits that also give up when
// another thread of the block has, and the lengths of a sequence.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace lsa {
namespace paged {

template <bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag) {
  auto probe = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (probe()) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (probe()) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_timeout(status);
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void spin_ns(unsigned long long ns) {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) {
  }
}

// Cached tokens and new tokens of sequence b, clamped to what the table and the
// call can hold.
struct Lens {
  int len, n_new;
};
__device__ __forceinline__ Lens lens_of(const PagedArgs& a, int b) {
  Lens l;
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  const int s = __ldg(a.seq_len + b);
  l.len = s < 0 ? 0 : (s > cap ? static_cast<int>(cap) : s);
  if (s > cap && threadIdx.x == 0) record_bad_page(a.status);
  const int n = a.q_len ? __ldg(a.q_len + b) : a.T;
  l.n_new = n < 0 ? 0 : (n > a.T ? a.T : n);
  return l;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tiled load of a (columns, slot, page) map.
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t slot,
                                              int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(slot), "r"(page)
      : "memory");
}

}  // namespace paged
}  // namespace lsa
