// Shared by the paged attention kernels: bounded waits that also give up when
// another thread of the block has, the lengths of a sequence, and the division
// of the work.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace lsa {
namespace paged {

// Limits in SM cycles: reading the global timer takes longer than most waits.
constexpr long long kWaitLimitCycles = 2000000000ll;   // 1 s and a little

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
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

// The work is a list of key blocks: for every KV head g, sequence b and tile of
// query rows, the blocks that the tile's last row sees (one, all masked, where
// it sees none). The list is cut into equal contiguous parts, one per worker (a
// block, or a cluster of two): sequences of any lengths, and any number of
// tiles, load the GPU evenly, and only tiles that a cut goes through need a
// merge. A worker cuts at most two tiles; a piece that begins inside a tile is
// kept in the worker's slot 2 w, one that begins with the tile in 2 w + 1.
struct Work {
  long long left;      // key blocks to come, the current piece's included
  long long begin;     // of the current tile, in the list
  int g, bt;           // KV head; b * tiles + tile
  int blk0, n, all;    // the piece: blocks [blk0, blk0 + n) of the tile's `all`
};

template <int ROWS, int BN>
__device__ __forceinline__ int blocks_of(const PagedArgs& a, int bt) {
  const int b = bt / a.tiles, r0 = (bt - b * a.tiles) * ROWS;
  const Lens l = lens_of(a, b);
  const int rows = l.n_new * a.G;
  if (r0 >= rows) return 0;
  const int keys = min(l.len, l.len - l.n_new + (min(rows, r0 + ROWS) - 1) / a.G + 1);
  return keys <= 0 ? 1 : (keys + BN - 1) / BN;
}

// By one whole warp: worker w's part of the list. Worker 0 leaves the list's
// length and the number of workers in a.head for the merge.
template <int ROWS, int BN>
__device__ __forceinline__ Work plan_work(const PagedArgs& a, int w, int workers) {
  const int lane = threadIdx.x & 31;
  const int n_bt = a.B * a.tiles;
  long long sum = 0;
#pragma unroll 4
  for (int i = lane; i < n_bt; i += 32) sum += blocks_of<ROWS, BN>(a, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const long long total = sum * a.Hkv;
  const int used = static_cast<int>(total < workers ? total : workers);
  if (w == 0 && lane == 0) {
    a.head[0] = total;
    a.head[1] = used;
  }
  Work k{};
  if (w >= used) return k;
  long long s;
  if (total <= 0x00FFFFFFll) {              // 32-bit divisions: a third of the time (workers are at most 160)
    const uint32_t t = static_cast<uint32_t>(total), u = static_cast<uint32_t>(used);
    s = t * static_cast<uint32_t>(w) / u;
    k.left = t * static_cast<uint32_t>(w + 1) / u - s;
    k.g = static_cast<int>(static_cast<uint32_t>(s) / static_cast<uint32_t>(sum));
  } else {
    s = total * w / used;
    k.left = total * (w + 1) / used - s;
    k.g = static_cast<int>(s / sum);
  }
  long long at = k.g * sum;                 // the list position of tile i0
  for (int i0 = 0;; i0 += 32) {
    const int n = i0 + lane < n_bt ? blocks_of<ROWS, BN>(a, i0 + lane) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at + upto > s);
    if (past || i0 + 32 >= n_bt) {
      const int l = past ? __ffs(past) - 1 : 31;
      k.bt = i0 + l;
      k.all = __shfl_sync(0xffffffffu, n, l);
      k.begin = at + __shfl_sync(0xffffffffu, upto, l) - k.all;
      k.blk0 = static_cast<int>(s - k.begin);
      k.n = static_cast<int>(min(k.left, static_cast<long long>(k.all - k.blk0)));
      return k;
    }
    at += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// The worker's next piece; n = 0 when there is none.
template <int ROWS, int BN>
__device__ __forceinline__ void next_work(const PagedArgs& a, Work& k) {
  k.left -= k.n;
  k.n = 0;
  if (k.left <= 0) return;
  const int n_bt = a.B * a.tiles;
  k.begin += k.all;
  do {
    if (++k.bt == n_bt) {
      k.bt = 0;
      ++k.g;
    }
    k.all = blocks_of<ROWS, BN>(a, k.bt);
  } while (k.all == 0);
  k.blk0 = 0;
  k.n = static_cast<int>(min(k.left, static_cast<long long>(k.all)));
}

// The worker that has position x of a list of `total`.
__device__ __forceinline__ int worker_of(long long x, long long total, long long used) {
  if (total <= 0x00FFFFFFll)
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(used) - 1u) / static_cast<uint32_t>(total));
  return static_cast<int>(((x + 1) * used - 1) / total);
}

constexpr int kNoPage = -2147483647 - 1;   // past the sequence's end (other entries outside the pool are reported)

// One lane of the warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of fp32 operations in one instruction, and the largest of three.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// Same into this CTA's shared memory, counted on an mbarrier (cluster address)
// of either CTA of the pair.
__device__ __forceinline__ void tma_load_page_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t slot,
                                                   int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(slot), "r"(page)
      : "memory");
}

}  // namespace paged
}  // namespace lsa
