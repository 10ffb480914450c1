// Upkeep of a paged cache: reserving, forking, freeing, copying and compacting
// pages. Block tables and reference counts live on the device and so do these
// operations: nothing is read back, and a call can be captured into a graph.
//
// Which pages are taken is decided by one block (the lowest free pages, in a
// fixed order, so the result does not depend on scheduling): it ranks the free
// pages by prefix sums over the reference counts and stops at the last one it
// needs. The bytes are then moved by a grid of blocks, one 16 KB piece of a
// page each; that is what bounds a large call (HBM: every moved page is read
// and written once). Small calls are bound by launch latency.
#include <limits.h>

#include "internal.h"
#include "ptx.cuh"

namespace lsa {
namespace {

constexpr int kPlan = 1024;        // threads of a planning block
constexpr int kMove = 256;         // threads of a moving block
constexpr int kRowChunk = 2048;    // table entries of a row that one block handles

// Exclusive prefix sum of v over the block's kPlan threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                 // an earlier scan's sums have been read
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sum[lane] = w;            // inclusive
  }
  __syncthreads();
  *total = warp_sum[31];
  return x - v + (warp ? warp_sum[warp - 1] : 0);
}

// Calls take(rank, page) for the `need` lowest free pages (all of them if there
// are fewer) and returns how many there were. Every thread of the block enters.
template <class F>
__device__ __forceinline__ int take_free(const int* ref, int n_pages, int need, F take) {
  constexpr int kPer = 16;         // pages a thread looks at in one round (four loads in flight)
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < need; p0 += kPlan * kPer) {
    const int p = p0 + threadIdx.x * kPer;
    unsigned f = 0u;               // bit e: page p + e is free
    if (p + kPer <= n_pages) {
      int4 v[kPer / 4];
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) v[i] = reinterpret_cast<const int4*>(ref + p)[i];
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i)
        f |= ((v[i].x <= 0 ? 1u : 0u) | (v[i].y <= 0 ? 2u : 0u) | (v[i].z <= 0 ? 4u : 0u) | (v[i].w <= 0 ? 8u : 0u))
             << (4 * i);
    } else {
      for (int e = 0; e < n_pages - p; ++e) f |= (ref[p + e] <= 0 ? 1u : 0u) << e;
    }
    int total;
    int rank = found + block_scan(__popc(f), &total);
    for (; f && rank < need; f &= f - 1, ++rank) take(rank, p + __ffs(f) - 1);
    found += total;
  }
  return min(found, need);
}

// ------------------------------------------------------------------ reserve --
// shared memory: first[S] (first unmapped logical page), upto[S] (pages missing
// in sequences 0 .. s).
__global__ void __launch_bounds__(kPlan) reserve_kernel(const PageArgs a, const int* __restrict__ len) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sh[];
  int* first = sh;
  int* upto = sh + a.S;
  const int lane = threadIdx.x & 31;
  // The mapped entries are a prefix, so the last wanted entry tells at once
  // whether anything is missing; where it is, the warp walks back to the prefix.
  for (int s0 = 0; s0 < a.S; s0 += kPlan) {
    const int s = s0 + threadIdx.x;
    int want = 0, miss = 0;
    if (s < a.S) {
      const int l = len[s];
      want = l <= 0 ? 0 : (l - 1) / a.page_size + 1;
      if (want > a.max_pages) {
        record_bad_page(a.status);
        want = a.max_pages;
      }
      miss = want > 0 && a.table[static_cast<long long>(s) * a.max_pages + want - 1] < 0;
    }
    int mapped_to = want;                                // entries [mapped_to, want) of this lane's row are unmapped
    unsigned todo = __ballot_sync(0xffffffffu, miss);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int ss = s - lane + l;
      const int* row = a.table + static_cast<long long>(ss) * a.max_pages;
      int end = __shfl_sync(0xffffffffu, want, l);      // entries [end, want) are unmapped
      while (end > 0) {
        const int j = end - 32 + lane;
        const unsigned mapped = __ballot_sync(0xffffffffu, j >= 0 && row[j < 0 ? 0 : j] >= 0);
        if (mapped) {
          end = end - 32 + (32 - __clz(mapped));
          break;
        }
        end -= 32;
      }
      if (lane == l) mapped_to = end < 0 ? 0 : end;
    }
    if (s < a.S) {
      first[s] = mapped_to;
      upto[s] = want - mapped_to;
    }
  }
  __syncthreads();
  // Counts stop at one more than there can be pages, which no rank reaches: 8192 rows of 2^19 entries have more than
  // 32 bits hold.
  const int most = a.n_pages + 1;
  int need = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlan) {
    const int s = s0 + threadIdx.x;
    const int v = s < a.S ? min(upto[s], most) : 0;
    int total;
    const int before = block_scan(v, &total);
    if (s < a.S) upto[s] = min(need + before + v, most);
    need = min(need + total, most);
  }
  __syncthreads();
  if (need == 0) return;
  const int got = take_free(a.ref, a.n_pages, need, [&](int rank, int page) {
    int lo = 0, hi = a.S - 1;                            // the sequence with upto[s - 1] <= rank < upto[s]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (upto[mid] > rank) hi = mid; else lo = mid + 1;
    }
    const int j = first[lo] + rank - (lo ? upto[lo - 1] : 0);
    a.table[static_cast<long long>(lo) * a.max_pages + j] = page;
    a.ref[page] = 1;
  });
  if (got < need && threadIdx.x == 0) record_no_page(a.status);
}

// --------------------------------------------------------------------- free --
// grid (sequence, piece of its row). Each mapped entry is taken out by exactly
// one thread (exchange), so an id that repeats is freed once.
__global__ void __launch_bounds__(kMove) free_kernel(const PageArgs a, const int* __restrict__ seqs) {
  pdl_wait();
  pdl_trigger();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= a.S) {
    if (threadIdx.x == 0) record_bad_page(a.status);
    return;
  }
  int* row = a.table + static_cast<long long>(s) * a.max_pages;
  const int j0 = blockIdx.y * kRowChunk, j1 = min(a.max_pages, j0 + kRowChunk);
  for (int j = j0 + threadIdx.x; j < j1; j += kMove) {
    if (row[j] < 0) continue;
    const int p = atomicExch(row + j, -1);
    if (p < 0) continue;
    if (p >= a.n_pages) {
      record_bad_page(a.status);
    } else if (atomicSub(a.ref + p, 1) <= 0) {           // was not held: leave it free
      atomicAdd(a.ref + p, 1);
      record_bad_page(a.status);
    }
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) a.seq_len[s] = 0;
}

// --------------------------------------------------------------------- moves --
// 16-byte copy of `bytes` (a multiple of 16, at most kCopyChunk) by the block,
// every load of a thread in flight before its first store.
__device__ __forceinline__ void copy_piece(uint8_t* dst, const uint8_t* src, int bytes) {
  constexpr int kU = kCopyChunk / 16 / kMove;
  uint4 v[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int o = (i * kMove + threadIdx.x) * 16;
    if (o < bytes) v[i] = *reinterpret_cast<const uint4*>(src + o);
  }
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int o = (i * kMove + threadIdx.x) * 16;
    if (o < bytes) *reinterpret_cast<uint4*>(dst + o) = v[i];
  }
}

// Piece c (of pools.first[pools.n]) of page src -> page dst.
__device__ __forceinline__ void move_piece(const Pools& pools, int c, int src, int dst) {
  int i = 0;
  while (i + 1 < pools.n && c >= pools.first[i + 1]) ++i;
  const int o = (c - pools.first[i]) * kCopyChunk;
  copy_piece(pools.base[i] + dst * pools.stride[i] + o, pools.base[i] + src * pools.stride[i] + o,
             min(kCopyChunk, pools.bytes[i] - o));
}

// --------------------------------------------------------------------- fork --
// Tokens of a parent, at most what its row holds.
__device__ __forceinline__ int fork_len(const PageArgs& a, int p) {
  return min(max(0, a.seq_len[p]), a.max_pages * a.page_size);
}

// plan[i]: -2 = pair refused, -1 = no partly filled page, -3 = no free page for
// it, else the page that takes the copy. shared memory: owner[S], the lowest
// pair that names s as its child.
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const PageArgs a, const int* __restrict__ parent,
                                                          const int* __restrict__ child, int n, int* plan) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int owner[];
  for (int s = threadIdx.x; s < a.S; s += kPlan) owner[s] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int c = child[i];
    if (c >= 0 && c < a.S) atomicMin(owner + c, i);
  }
  __syncthreads();
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int tail = 0;
    if (i < n) {
      const int p = parent[i], c = child[i];
      const bool ok = p >= 0 && p < a.S && c >= 0 && c < a.S && owner[c] == i && owner[p] == INT_MAX;
      int code = -1;
      if (!ok) {
        record_bad_page(a.status);
        code = -2;
      } else {
        const int l = fork_len(a, p);
        if (l < a.seq_len[p]) record_bad_page(a.status);
        const int full = l / a.page_size;
        if (l - full * a.page_size > 0) {
          const int e = full < a.max_pages ? a.table[static_cast<long long>(p) * a.max_pages + full] : -1;
          if (e >= 0 && e < a.n_pages) {
            tail = 1;
          } else {
            record_bad_page(a.status);
            code = -3;
          }
        }
      }
      plan[i] = code;
    }
    int total;
    const int rank = need + block_scan(tail, &total);
    if (tail) plan[i] = -16 - rank;                      // the rank until its page is known
    need += total;
  }
  __syncthreads();
  if (need == 0) return;
  // page of rank r -> the free list kept behind the plan
  int* list = plan + n;
  const int got = take_free(a.ref, a.n_pages, need, [&](int rank, int page) {
    list[rank] = page;
    a.ref[page] = 1;
  });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int v = plan[i];
    if (v > -16) continue;
    const int rank = -16 - v;
    plan[i] = rank < got ? list[rank] : -3;
  }
  if (got < need && threadIdx.x == 0) record_no_page(a.status);
}

// grid (pair, pieces of its table row, then pieces of the partly filled page)
__global__ void __launch_bounds__(kMove) fork_kernel(const PageArgs a, const int* __restrict__ parent,
                                                     const int* __restrict__ child, const int* __restrict__ plan,
                                                     const __grid_constant__ Pools pools, int row_pieces) {
  pdl_wait();
  pdl_trigger();
  const int code = plan[blockIdx.x];
  if (code == -2) return;
  const int p = parent[blockIdx.x], c = child[blockIdx.x];
  const int l = fork_len(a, p);
  const int full = l / a.page_size;
  const int* from = a.table + static_cast<long long>(p) * a.max_pages;
  if (static_cast<int>(blockIdx.y) >= row_pieces) {
    if (code >= 0) move_piece(pools, blockIdx.y - row_pieces, from[full], code);
    return;
  }
  int* to = a.table + static_cast<long long>(c) * a.max_pages;
  const int j0 = blockIdx.y * kRowChunk, j1 = min(a.max_pages, j0 + kRowChunk);
  for (int j = j0 + threadIdx.x; j < j1; j += kMove) {
    int e = -1;
    if (j < full) {
      e = from[j];
      if (e >= a.n_pages) {
        record_bad_page(a.status);
        e = -1;
      }
      if (e >= 0) atomicAdd(a.ref + e, 1);
    } else if (j == full && code >= 0) {
      e = code;
    }
    to[j] = e;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) a.seq_len[c] = code == -3 ? full * a.page_size : l;
}

// --------------------------------------------------------------------- copy --
// ok[i] = 1 if pair i may run. Two bits a page in shared memory: it is some
// pair's dst; it is the dst of more than one pair. A third sweep refuses the
// dsts that are read.
__global__ void __launch_bounds__(kPlan) copy_plan_kernel(int n_pages, const int* __restrict__ src,
                                                          const int* __restrict__ dst, int n, int* ok, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t bits[];
  const int words = (n_pages + 31) / 32;
  uint32_t* is_dst = bits;
  uint32_t* refused = bits + words;
  for (int i = threadIdx.x; i < 2 * words; i += kPlan) bits[i] = 0u;
  __syncthreads();
  auto in_range = [&](int i) { return src[i] >= 0 && src[i] < n_pages && dst[i] >= 0 && dst[i] < n_pages; };
  for (int i = threadIdx.x; i < n; i += kPlan) {
    if (!in_range(i)) continue;
    const uint32_t m = 1u << (dst[i] & 31);
    if (atomicOr(is_dst + (dst[i] >> 5), m) & m) atomicOr(refused + (dst[i] >> 5), m);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    if (!in_range(i)) continue;
    const uint32_t m = 1u << (src[i] & 31);
    if (is_dst[src[i] >> 5] & m) atomicOr(refused + (src[i] >> 5), m);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const bool good = in_range(i) && !((refused[dst[i] >> 5] >> (dst[i] & 31)) & 1u);
    if (!good) record_bad_page(status);
    ok[i] = good;
  }
}

// ok null: every block looks through the list for its own pair (few pairs: less than a launch for a plan).
__global__ void __launch_bounds__(kMove) copy_kernel(const int* __restrict__ src, const int* __restrict__ dst,
                                                     const int* __restrict__ ok, int n, int n_pages, int* status,
                                                     const __grid_constant__ Pools pools) {
  pdl_wait();
  pdl_trigger();
  const int me = blockIdx.x, s = src[me], d = dst[me];
  if (ok) {
    if (!ok[me]) return;
  } else {
    auto inside = [&](int p) { return p >= 0 && p < n_pages; };
    bool refused = !inside(s) || !inside(d);
    for (int i = threadIdx.x; i < n && !refused; i += kMove) {
      const int si = src[i], di = dst[i];
      refused = inside(si) && inside(di) && ((di == d && i != me) || si == d);
    }
    if (__syncthreads_or(refused)) {
      if (threadIdx.x == 0) record_bad_page(status);
      return;
    }
  }
  move_piece(pools, blockIdx.y, s, d);
}

// ------------------------------------------------------------------ compact --
// The bits of the live pages, for the table entries: behind the pages to be moved, of which there are n_pages / 2 at
// most (as many as holes below n_live).
__device__ __forceinline__ uint32_t* live_words(int* ws, int n_pages) {
  return reinterpret_cast<uint32_t*>(ws + kCompactHeader + n_pages - (n_pages + 31) / 32);
}

// One bit a page in shared memory (live or not) and the live pages before each
// word. A hole below n_live and a live page at or above it of the same rank
// make a move.
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const int* ref, int n_pages, int* ref_out, int* n_live_out,
                                                             int* ws) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t live[];
  const int words = (n_pages + 31) / 32;
  int* before = reinterpret_cast<int*>(live + words);
  __shared__ int live_below;                             // live pages below n_live
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a warp takes 32 pages at a time, one per lane
  for (int w0 = warp; w0 < words; w0 += 4 * (kPlan / 32)) {
    int r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = (w0 + i * (kPlan / 32)) * 32 + lane;
      r[i] = p < n_pages ? ref[p] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = w0 + i * (kPlan / 32), p = w * 32 + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, r[i] > 0);
      if (lane == 0 && w < words) live[w] = m;
      if (p < n_pages && ref_out != ref) ref_out[p] = r[i];
    }
  }
  __syncthreads();
  const int per = (words + kPlan - 1) / kPlan;           // consecutive words of a thread
  const int w0 = min(words, static_cast<int>(threadIdx.x) * per), w1 = min(words, w0 + per);
  int c = 0;
  for (int w = w0; w < w1; ++w) c += __popc(live[w]);
  int n_live;
  int at = block_scan(c, &n_live);
  for (int w = w0; w < w1; ++w) {
    before[w] = at;
    at += __popc(live[w]);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int w = n_live >> 5;
    live_below = w < words ? before[w] + __popc(live[w] & ((1u << (n_live & 31)) - 1u)) : n_live;
    ws[0] = n_live;
    ws[1] = n_live - live_below;
    if (n_live_out) *n_live_out = n_live;
  }
  __syncthreads();
  int* src = ws + kCompactHeader;
  int* dst = src + n_pages;
  int* map = dst + n_pages;
  uint32_t* live_out = live_words(ws, n_pages);
  for (int w = warp; w < words; w += kPlan / 32) {
    const int p = w * 32 + lane;
    const uint32_t m = live[w];
    if (lane == 0) live_out[w] = m;
    const int rank = before[w] + __popc(m & ((1u << lane) - 1u));   // live pages below p
    const bool alive = (m >> lane) & 1u;
    if (p < n_live) {
      if (!alive) dst[p - rank] = p;                     // a hole
    } else if (p < n_pages) {
      if (alive) src[rank - live_below] = p;             // a page to be moved
      else map[p] = -1;
    }
  }
  __syncthreads();
  const int moves = n_live - live_below;
  for (int k = threadIdx.x; k < moves; k += kPlan) {
    const int s = src[k], d = dst[k];
    map[s] = d;
    ref_out[d] = ref[s];
    ref_out[s] = 0;
  }
}

// blocks [0, table_blocks): table entries; the rest: pieces of the moved pages
__global__ void __launch_bounds__(kMove) compact_kernel(const int* table, long long entries, int n_pages,
                                                        int* table_out, int* ws,
                                                        const __grid_constant__ Pools pools, int table_blocks,
                                                        int* status) {
  pdl_wait();
  pdl_trigger();
  const int n_live = ws[0], moves = ws[1];
  const int* src = ws + kCompactHeader;
  const int* dst = src + n_pages;
  const int* map = dst + n_pages;
  const uint32_t* live = live_words(ws, n_pages);
  if (static_cast<int>(blockIdx.x) < table_blocks) {
    for (long long i = static_cast<long long>(blockIdx.x) * kMove + threadIdx.x; i < entries;
         i += static_cast<long long>(table_blocks) * kMove) {
      int e = table[i];
      if (e >= n_pages) {
        record_bad_page(status);
      } else if (e >= 0) {
        // only a live page has a place; an entry of a free one would come to name another sequence's page
        const int to = !((live[e >> 5] >> (e & 31)) & 1u) ? -1 : e >= n_live ? map[e] : e;
        if (to < 0) record_bad_page(status);
        e = to;
      }
      table_out[i] = e;
    }
    return;
  }
  const int pieces = pools.first[pools.n];
  const long long items = static_cast<long long>(moves) * pieces;
  for (long long it = blockIdx.x - table_blocks; it < items; it += gridDim.x - table_blocks) {
    const int k = static_cast<int>(it / pieces);
    move_piece(pools, static_cast<int>(it - static_cast<long long>(k) * pieces), src[k], dst[k]);
  }
}

template <class... A>
cudaError_t plan_launch(const void* fn, size_t smem, cudaStream_t stream, A... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = set_max_smem(fn, smem);
    if (e != cudaSuccess) return e;
  }
  void* p[] = {static_cast<void*>(&args)...};
  return launch_pdl(fn, dim3(1), dim3(kPlan), smem, stream, p);
}

int row_pieces(int max_pages) { return (max_pages + kRowChunk - 1) / kRowChunk; }

}  // namespace

cudaError_t launch_reserve(const PageArgs& a, const int* len, cudaStream_t stream) {
  return plan_launch(reinterpret_cast<const void*>(&reserve_kernel), static_cast<size_t>(a.S) * 8, stream, a, len);
}

cudaError_t launch_free(const PageArgs& a, const int* seqs, int n, cudaStream_t stream) {
  void* args[] = {const_cast<PageArgs*>(&a), &seqs};
  return launch_pdl(reinterpret_cast<const void*>(&free_kernel), dim3(n, row_pieces(a.max_pages)), dim3(kMove), 0,
                    stream, args);
}

cudaError_t launch_fork_plan(const PageArgs& a, const int* parent, const int* child, int n, int* plan,
                             cudaStream_t stream) {
  return plan_launch(reinterpret_cast<const void*>(&fork_plan_kernel), static_cast<size_t>(a.S) * 4, stream, a, parent,
                     child, n, plan);
}

cudaError_t launch_fork(const PageArgs& a, const int* parent, const int* child, int n, const int* plan,
                        const Pools& pools, int rows, cudaStream_t stream) {
  int pieces = rows ? row_pieces(a.max_pages) : 0;
  const int total = pieces + pools.first[pools.n];
  if (total == 0) return cudaSuccess;
  void* args[] = {const_cast<PageArgs*>(&a), &parent, &child, &plan, const_cast<Pools*>(&pools), &pieces};
  return launch_pdl(reinterpret_cast<const void*>(&fork_kernel), dim3(n, total), dim3(kMove), 0, stream, args);
}

cudaError_t launch_copy_plan(int n_pages, const int* src, const int* dst, int n, int* ok, int* status,
                             cudaStream_t stream) {
  return plan_launch(reinterpret_cast<const void*>(&copy_plan_kernel),
                     static_cast<size_t>((n_pages + 31) / 32) * 8, stream, n_pages, src, dst, n, ok, status);
}

cudaError_t launch_copy(const Pools& pools, const int* src, const int* dst, const int* ok, int n, int n_pages, int* status,
                        cudaStream_t stream) {
  void* args[] = {&src, &dst, &ok, &n, &n_pages, &status, const_cast<Pools*>(&pools)};
  return launch_pdl(reinterpret_cast<const void*>(&copy_kernel), dim3(n, pools.first[pools.n]), dim3(kMove), 0, stream,
                    args);
}

cudaError_t launch_compact_plan(const int* ref, int n_pages, int* ref_out, int* n_live, int* ws, cudaStream_t stream) {
  return plan_launch(reinterpret_cast<const void*>(&compact_plan_kernel),
                     static_cast<size_t>((n_pages + 31) / 32) * 8, stream, ref, n_pages, ref_out, n_live, ws);
}

cudaError_t launch_compact(const int* table, int S, int max_pages, int n_pages, int* table_out, int* ws,
                           const Pools& pools, int rows, int* status, cudaStream_t stream) {
  long long entries = rows ? static_cast<long long>(S) * max_pages : 0;
  const int sms = device_sm_count();
  int table_blocks = static_cast<int>(entries > 0 ? (entries + kMove - 1) / kMove : 0);
  if (table_blocks > 2 * sms) table_blocks = 2 * sms;
  // 8 blocks an SM of 256 threads: 4 KB x 4 loads in flight each
  const int grid = table_blocks + (pools.first[pools.n] > 0 ? 8 * sms : 0);
  if (grid == 0) return cudaSuccess;
  void* args[] = {&table, &entries, &n_pages, &table_out, &ws, const_cast<Pools*>(&pools), &table_blocks, &status};
  return launch_pdl(reinterpret_cast<const void*>(&compact_kernel), dim3(grid), dim3(kMove), 0, stream, args);
}

}  // namespace lsa
