// Attention of new tokens over a paged latent cache (MLA: one 576-column row
// per token serves as K, its first 512 columns as V; bf16 or e4m3 with a scale
// per token).
//
//   o[r, :] = sum_{s <= pos(r)} softmax_s(scale * q[r] . c[s]) c[s][0:512],   row r = t * Hq + head
//
// 128 rows are one tile; the heads of a token and the tokens of a chunk fill it
// alike. The output alone (128 x 512 fp32) would fill an SM's tensor memory, so
// a cluster of two CTAs shares a tile:
//   - the score product is split over the columns: CTA 0 multiplies columns
//     [0, 320), CTA 1 [320, 576), with its part of q in tensor memory;
//   - each sends its partial scores of a 64-key block to the other as fp32
//     (st.async into the partner's shared memory, counted on its mbarrier) and
//     adds the partner's: both then hold the same bits (fp32 addition commutes)
//     and run the same softmax;
//   - each accumulates its 256 output columns, with P in tensor memory.
// Per block and CTA that is 128 x 64 x (288 + 256) multiply-adds on average and
// 32 KB exchanged; splitting the output alone would multiply the whole scores
// in both (1.5 times the products), and 1.8 times the cache bytes would cross
// from L2 to the SMs.
//
// Tensor memory (512 columns): O 256, S 64, P 32, q 160.
//
// Threads: warps 0-7 softmax (two threads per row, each 32 of a block's 64
// columns); warp 8 producer (TMA boxes of one page, or of the page's part of
// the block); warp 9 MMA issuer. e4m3: warps 8-11 stage rows (codes -> bf16,
// exact) in place of the producer and warp 12 issues. Masks, the zeroing of
// what lies past seq_len and the handling of unmapped pages are those of
// paged_attn.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace lsa {
namespace {

using namespace paged;

constexpr int BN = kPagedBNMla;
constexpr int kStages = 3;
constexpr int kChunks = 5;                       // 64-column chunks per CTA and block
constexpr int kChunkBytes = BN * 128;
constexpr int kStageBytes = kChunks * kChunkBytes;
constexpr int kSoft = 256;
constexpr int kXBytes = 128 * BN * 4;            // partial scores of a block: rows of 256 B, 16-byte units XOR-swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256, kColP = 320, kColQ = 352;
constexpr int kOffX = kStages * kStageBytes;     // [2] receive buffers
constexpr int kOffTag = kOffX + 2 * kXBytes;     // [2][2][128] u64 tagged maxima + [2][128] u64 tagged sums
constexpr int kOffMask = kOffTag + (4 * 128 + 2 * 128) * 8;
constexpr int kOffKScale = (kOffMask + kStages * 8 + 15) / 16 * 16;   // read 16 bytes at a time
constexpr int kOffBars = kOffKScale + kStages * BN * 4;
constexpr int kNumBars = 2 * kStages + 9;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr size_t kSmem = 1024 + kOffMisc + 16;
static_assert(kOffKScale % 16 == 0 && kOffBars % 8 == 0 && kSmem <= 227 * 1024, "shared memory layout");

__device__ __forceinline__ void put_tagged(volatile unsigned long long* slot, uint32_t tag, float v) {
  *slot = (static_cast<unsigned long long>(tag) << 32) | __float_as_uint(v);
}
__device__ __forceinline__ bool get_tagged(const volatile unsigned long long* slot, uint32_t tag, float* v,
                                           int* status, volatile int* abort_flag) {
  unsigned long long x = *slot;
  if (static_cast<uint32_t>(x >> 32) != tag) {
    const unsigned long long t0 = globaltimer_ns();
    while (static_cast<uint32_t>((x = *slot) >> 32) != tag) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_timeout(status);
        *abort_flag = 1;
        return false;
      }
    }
  }
  *v = __uint_as_float(static_cast<uint32_t>(x));
  return true;
}

// 16 bytes into the partner's shared memory, counted on its mbarrier.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(
                   addr),
               "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// e4m3 pair -> bf16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two_codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two_codes)));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return pack_bf16(f.x, f.y);
}

template <bool KV8>
constexpr int threads_of() { return KV8 ? 416 : 320; }

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of<KV8>(), 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap tm_k, const PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sStage = base;
  uint8_t* sX = base + kOffX;
  volatile unsigned long long* tag_max = reinterpret_cast<volatile unsigned long long*>(base + kOffTag);
  volatile unsigned long long* tag_sum = tag_max + 4 * 128;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(base + kOffMask);     // [kStages][2] rows that count
  float* kscale_s = reinterpret_cast<float*>(base + kOffKScale);       // [kStages][BN]
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kOffBars);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + kStages;
  uint64_t* s_full = bars + 2 * kStages;
  uint64_t* s_free = s_full + 1;
  uint64_t* p_full = s_free + 1;
  uint64_t* pv_done = p_full + 1;
  uint64_t* q_ready = pv_done + 1;
  uint64_t* x_full = q_ready + 1;      // [2] own expect_tx arrive + the partner's bytes
  uint64_t* x_free = x_full + 2;       // [2] the partner has read what this CTA sent into its buffer i
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr int kMmaWarp = KV8 ? 12 : 9;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const int tile = a.tiles - 1 - static_cast<int>(blockIdx.x >> 1);    // the longest rows first
  const int split = blockIdx.y, b = blockIdx.z;
  const int chunk0 = rank ? 4 : 0;        // global 64-column chunk of local chunk 0
  const int nq = rank ? 4 : 5;            // chunks multiplied
  const int qk_local0 = rank ? 1 : 0;     // local chunk of the first of them

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], KV8 ? 128 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kSoft);
    mbar_init(p_full, kSoft);
    mbar_init(pv_done, 1);
    mbar_init(q_ready, kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_free[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 6 * 128; i += threads_of<KV8>()) tag_max[i] = 0ull;   // 0 is never a live tag
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();   // the partner's barriers are initialised before any remote arrive
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem + kColO, tQ = tmem + kColQ, tS = tmem + kColS, tP = tmem + kColP;

  const Lens L = lens_of(a, b);
  const int rows = L.n_new * a.Hq;
  const int row0 = tile * 128;
  const int first_pos = L.len - L.n_new;
  int keys = 0;                           // keys the tile's last row sees
  if (row0 < rows) keys = max(0, min(L.len, first_pos + (min(rows, row0 + 128) - 1) / a.Hq + 1));
  const int all = (keys + BN - 1) / BN;
  const int per_split = (all + a.n_split - 1) / a.n_split;
  const int blk0 = split * per_split;
  const int nblk = max(0, min(all, blk0 + per_split) - blk0);

  if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer --
    if (lane == 0 && nblk > 0) {
      const uint32_t idesc_qk = make_idesc(1, 1, 128, BN, 0, 0);
      const uint32_t idesc_pv = make_idesc(1, 1, 128, 256, 0, 1);
      const uint32_t peer_xfree = mapa_shared(smem_u32(x_free), peer);
      auto issue_pv = [&](int pb) -> bool {
        if (!wait(p_full, pb & 1, a.status, abort_flag)) return false;
        tc_fence_after();
        const uint32_t vb = smem_u32(sStage + (pb % kStages) * kStageBytes);
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks)
          umma_f16_ts(tO, tP + ks * 8, make_sdesc(vb + ks * 2048, kChunkBytes, 1024, kLayoutSW128), idesc_pv,
                      (pb | ks) ? 1u : 0u);
        umma_commit(pv_done);
        umma_commit(&kv_empty[pb % kStages]);
        // P(pb) is stored, so every softmax thread has read block pb's partial
        // scores from buffer pb & 1: the partner may send block pb + 2 into it
        mbar_arrive_remote(peer_xfree + (pb & 1) * 8);
        return true;
      };
      bool ok = wait(q_ready, 0, a.status, abort_flag);
      for (int blk = 0; ok && blk < nblk; ++blk) {
        const int s = blk % kStages;
        ok = wait(&kv_full[s], (blk / kStages) & 1, a.status, abort_flag);
        if (ok && blk >= 1) ok = wait(s_free, (blk - 1) & 1, a.status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t kb = smem_u32(sStage + s * kStageBytes);
#pragma unroll 1
        for (int j = 0; j < nq; ++j) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ts(tS, tQ + j * 32 + ks * 8,
                        make_sdesc(kb + (qk_local0 + j) * kChunkBytes + ks * 32, 16, 1024, kLayoutSW128), idesc_qk,
                        (j | ks) ? 1u : 0u);
        }
        umma_commit(s_full);
        if (blk >= 1) ok = issue_pv(blk - 1);
      }
      if (ok) issue_pv(nblk - 1);
    }
    __syncwarp();
  } else if (warp >= 8) {
    if constexpr (!KV8) {
      // -------------------------------------------------------- producer --
      const int box = min(BN, 1 << a.page_shift);          // rows of a box
      const int per = BN / box;                            // boxes of a chunk
      const int n_ops = kChunks * per;                     // at most 20
      const int j = lane % per, c = lane / per;
      const int* row = a.table + static_cast<long long>(b) * a.max_pages;
      auto page_of = [&](int blk) -> int {
        const int tok = (blk0 + blk) * BN + j * box;
        if (blk >= nblk || tok >= L.len) return -1;
        const int p = __ldg(row + (tok >> a.page_shift));
        if (p < 0 || p >= a.n_pages) {
          if (c == 0 && rank == 0) record_bad_page(a.status);
          return -1;
        }
        return p;
      };
      int next = page_of(0);
      bool ok = true;
      for (int blk = 0; ok && blk < nblk; ++blk) {
        const int page = next;
        next = page_of(blk + 1);
        const int s = blk % kStages;
        if (blk >= kStages) {
          ok = __all_sync(0xffffffffu, wait(&kv_empty[s], ((blk / kStages) - 1) & 1, a.status, abort_flag));
          if (!ok) break;
        }
        // rows of the block that count: mapped, below seq_len
        const uint32_t mapped = __ballot_sync(0xffffffffu, page >= 0);
        if (lane < 2) {
          uint32_t m = 0u;
          const int left = L.len - (blk0 + blk) * BN - 32 * lane;       // rows of this word below seq_len
          for (int i = 0; i < 32; i += 16)
            if ((mapped >> ((32 * lane + i) / box)) & 1u) m |= 0xFFFFu << i;
          if (left < 32) m &= left > 0 ? (1u << left) - 1u : 0u;
          mask_s[2 * s + lane] = m;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], kStageBytes);
        __syncwarp();
        if (lane < n_ops) {
          const int tok = (blk0 + blk) * BN + j * box;
          tma_load_page(sStage + s * kStageBytes + c * kChunkBytes + j * box * 128, &tm_k, &kv_full[s], (chunk0 + c) * 64,
                        tok & ((1 << a.page_shift) - 1), page >= 0 ? page : a.n_pages);
        }
      }
    } else {
      // --------------------------------------------- e4m3: stage the rows --
      // Thread: half (160 codes) of a row's 320 columns. Its next block's codes
      // are loaded before this one's are converted.
      const int ct = tid - 256;
      const int row = ct & 63, part = ct >> 6;
      const int* trow = a.table + static_cast<long long>(b) * a.max_pages;
      constexpr int kU = kChunks * 4 / 2;                  // 16-code units of the thread
      uint4 v[kU];
      float sc;
      bool live;
      auto load = [&](int blk) {
        const int tok = (blk0 + blk) * BN + row;
        live = false;
        sc = 0.f;
        if (blk < nblk && tok < L.len) {
          const int p = __ldg(trow + (tok >> a.page_shift));
          if (p < 0 || p >= a.n_pages) {
            if (rank == 0 && part == 0) record_bad_page(a.status);
          } else {
            live = true;
            const int slot = tok & ((1 << a.page_shift) - 1);
            const uint4* src = reinterpret_cast<const uint4*>(a.kv8 + p * a.kv8_page + slot * a.kv8_row + chunk0 * 64) +
                               part * kU;
            sc = __ldg(a.k_scale + (static_cast<long long>(p) << a.page_shift) + slot);
#pragma unroll
            for (int i = 0; i < kU; ++i) v[i] = __ldg(src + i);
          }
        }
        if (!live) {
#pragma unroll
          for (int i = 0; i < kU; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      };
      load(0);
      for (int blk = 0; blk < nblk; ++blk) {
        const int s = blk % kStages;
        if (blk >= kStages &&
            !__all_sync(0xffffffffu, wait(&kv_empty[s], ((blk / kStages) - 1) & 1, a.status, abort_flag)))
          break;
        const uint32_t m = __ballot_sync(0xffffffffu, live);
        if (part == 0) {
          if (lane == 0) mask_s[2 * s + (row >> 5)] = m;
          kscale_s[s * BN + row] = sc;
        }
        uint8_t* dst = sStage + s * kStageBytes + row * 128;
        const int swz = row & 7;
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          const int u = part * kU + i, c = u >> 2, q = u & 3;
          const uint4 e = v[i];
          *reinterpret_cast<uint4*>(dst + c * kChunkBytes + (((2 * q) ^ swz) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(e.x), e4m3x2_to_bf16x2(e.x >> 16), e4m3x2_to_bf16x2(e.y),
                         e4m3x2_to_bf16x2(e.y >> 16));
          *reinterpret_cast<uint4*>(dst + c * kChunkBytes + (((2 * q + 1) ^ swz) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(e.z), e4m3x2_to_bf16x2(e.z >> 16), e4m3x2_to_bf16x2(e.w),
                         e4m3x2_to_bf16x2(e.w >> 16));
        }
        load(blk + 1);
        fence_proxy_async_smem();
        mbar_arrive(&kv_full[s]);
      }
    }
  } else {
    // ------------------------------------------------- softmax / epilogue --
    const int quarter = warp & 3, half = warp >> 2;        // columns [32 half, 32 half + 32) of a block
    const int h = quarter * 32 + lane;                     // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = row0 + h;
    const int t_row = r / a.Hq;
    const int bound = r < rows ? max(0, min(L.len, first_pos + t_row + 1)) : 0;
    const long long orow = static_cast<long long>(b) * a.T * a.Hq + r;
    bool ok = true;
    if (nblk > 0) {
      // q row -> TMEM columns (two bf16 per column, k ascending); the two
      // threads of a row take alternate chunks
      const uint4* qrow = reinterpret_cast<const uint4*>(a.q + orow * 576) + (chunk0 + qk_local0) * 8;
#pragma unroll
      for (int jj = 0; jj < 3; ++jj) {
        const int j = 2 * jj + half;
        if (j < nq) {
          uint32_t v[32];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const uint4 w = r < rows ? __ldg(qrow + j * 8 + t) : make_uint4(0u, 0u, 0u, 0u);
            v[4 * t] = w.x;
            v[4 * t + 1] = w.y;
            v[4 * t + 2] = w.z;
            v[4 * t + 3] = w.w;
          }
          tmem_st32(tQ + lane_base + j * 32, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(q_ready);
    }
    const int swz = h & 7;   // unit t of this thread's half-row sits at unit t ^ swz
    const uint32_t peer_x = mapa_shared(smem_u32(sX), peer) + h * (BN * 4) + half * 128;
    const uint32_t peer_xfull = mapa_shared(smem_u32(x_full), peer);
    const bool leader = tid == 0;
    // Partial scores of block bb: TMEM -> registers, S freed, sent to the partner.
    auto fetch_send = [&](int bb, uint32_t (&sv)[32]) -> bool {
      const int i = bb & 1;
      if (!__all_sync(0xffffffffu, wait(s_full, bb & 1, a.status, abort_flag))) return false;
      tc_fence_after();
      tmem_ld32(tS + lane_base + half * 32, sv);
      if (leader) mbar_arrive_expect_tx(&x_full[i], kXBytes);   // for what the partner sends of block bb
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(s_free);
      // the partner's buffer i holds block bb - 2 until its readers have signalled
      if (bb >= 2 && !__all_sync(0xffffffffu, wait<true>(&x_free[i], ((bb - 2) >> 1) & 1, a.status, abort_flag)))
        return false;
#pragma unroll
      for (int t = 0; t < 8; ++t)
        st_async_v4(peer_x + i * kXBytes + ((t ^ swz) << 4), peer_xfull + i * 8, sv[4 * t], sv[4 * t + 1], sv[4 * t + 2],
                    sv[4 * t + 3]);
      return true;
    };
    const float c = a.scale_log2;
    float m_run = -INFINITY, l_part = 0.f;   // log2 domain; l_part: this thread's columns
    uint32_t sv_cur[32], sv_nxt[32];
    if (nblk > 0) ok = fetch_send(0, sv_cur);
    for (int blk = 0; ok && blk < nblk; ++blk) {
      const int s = blk % kStages, i = blk & 1;
      const int key0 = (blk0 + blk) * BN;
      // Block blk + 1's partial leaves before block blk's softmax: the
      // partner's reply then has a whole iteration to arrive.
      if (blk + 1 < nblk) {
        ok = fetch_send(blk + 1, sv_nxt);
        if (!ok) break;
      }
      ok = __all_sync(0xffffffffu, wait<true>(&x_full[i], (blk >> 1) & 1, a.status, abort_flag));
      if (!ok) break;
      float x[32];
      {
        const float4* src = reinterpret_cast<const float4*>(sX + i * kXBytes + h * (BN * 4) + half * 128);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float4 w = src[t ^ swz];
          x[4 * t] = __uint_as_float(sv_cur[4 * t]) + w.x;
          x[4 * t + 1] = __uint_as_float(sv_cur[4 * t + 1]) + w.y;
          x[4 * t + 2] = __uint_as_float(sv_cur[4 * t + 2]) + w.z;
          x[4 * t + 3] = __uint_as_float(sv_cur[4 * t + 3]) + w.w;
        }
      }
      ok = __all_sync(0xffffffffu, wait(&kv_full[s], (blk / kStages) & 1, a.status, abort_flag));
      if (!ok) break;
      const float4* ks4 = reinterpret_cast<const float4*>(kscale_s + s * BN + 32 * half);   // KV8: token scales
      if constexpr (KV8) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float4 k4 = ks4[t];
          x[4 * t] *= k4.x;
          x[4 * t + 1] *= k4.y;
          x[4 * t + 2] *= k4.z;
          x[4 * t + 3] *= k4.w;
        }
      }
      const uint32_t counts = mask_s[2 * s + half];
      const int vis = bound - key0 - 32 * half;
      if (__any_sync(0xffffffffu, vis < 32) || counts != 0xFFFFFFFFu) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= vis || !((counts >> j) & 1u)) x[j] = -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
      const float mb_mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      put_tagged(tag_max + (i * 2 + half) * 128 + h, static_cast<uint32_t>(blk + 1), mb_mine);
      float mb_other;
      ok = __all_sync(0xffffffffu, get_tagged(tag_max + (i * 2 + (half ^ 1)) * 128 + h, static_cast<uint32_t>(blk + 1),
                                              &mb_other, a.status, abort_flag));
      if (!ok) break;
      const float mb = fmaxf(mb_mine, mb_other);
      const bool move = mb > m_run + 8.f || (m_run == -INFINITY && mb != -INFINITY);
      float corr = 1.f;
      if (move) {
        corr = m_run == -INFINITY ? 0.f : ex2(m_run - mb);
        l_part *= corr;
        m_run = mb;
      }
      const float mu = m_run == -INFINITY ? 0.f : m_run;
      float ps[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float p0 = ex2(fmaf(x[j], c, -mu)), p1 = ex2(fmaf(x[j + 1], c, -mu));
        ps[(j >> 1) & 3] += p0 + p1;
        if constexpr (KV8) {   // V row = code * scale: the scale rides on P
          const float2 k2 = reinterpret_cast<const float2*>(ks4)[j >> 1];
          p0 *= k2.x;
          p1 *= k2.y;
        }
        pk[j >> 1] = pack_bf16(p0, p1);
      }
      l_part += (ps[0] + ps[1]) + (ps[2] + ps[3]);
      // P and O are free once PV(blk - 1) has completed
      if (blk >= 1) {
        ok = __all_sync(0xffffffffu, wait(pv_done, (blk - 1) & 1, a.status, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, move)) {   // rescale this thread's 128 of the 256 columns
#pragma unroll 1
          for (int c0 = half * 128; c0 < half * 128 + 128; c0 += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + lane_base + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int t = 0; t < 32; ++t) ov[t] = __float_as_uint(__uint_as_float(ov[t]) * corr);
            tmem_st32(tO + lane_base + c0, ov);
          }
        }
      }
      tmem_st16(tP + lane_base + half * 16, pk);   // keys [32 half, 32 half + 32) of the row
      if (!KV8 && key0 + BN > L.len) {             // nothing past the sequence's end may reach the product
        const int z0 = max(0, L.len - key0);
        for (int z = tid; z < (BN - z0) * 32; z += kSoft) {
          const int zr = z0 + (z >> 5), u = z & 31;
          *reinterpret_cast<uint4*>(sStage + s * kStageBytes + (u >> 3) * kChunkBytes + zr * 128 + (u & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full);
#pragma unroll
      for (int t = 0; t < 32; ++t) sv_cur[t] = sv_nxt[t];
    }
    if (ok && nblk > 0) ok = __all_sync(0xffffffffu, wait(pv_done, (nblk - 1) & 1, a.status, abort_flag));
    // row sum over both halves (fixed order: both threads get the same value)
    float l_run = 0.f;
    if (ok) {
      put_tagged(tag_sum + half * 128 + h, 0xFFFFFFFFu, l_part);
      float l_other;
      ok = __all_sync(0xffffffffu,
                      get_tagged(tag_sum + (half ^ 1) * 128 + h, 0xFFFFFFFFu, &l_other, a.status, abort_flag));
      l_run = half == 0 ? l_part + l_other : l_other + l_part;
    }
    // ---- epilogue: this thread's 128 output columns, staged per warp for coalesced stores
    if (ok) {
      tc_fence_after();
      const bool have = nblk > 0;
      const bool direct = a.n_part == 1;
      const long long n_rows = static_cast<long long>(a.B) * a.T * a.Hq;
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      if (have || direct) {
        float* tile_s = reinterpret_cast<float*>(sX) + warp * 32 * 36;   // [32 rows][36]
#pragma unroll 1
        for (int c0 = half * 128; c0 < half * 128 + 128; c0 += 32) {
          uint32_t ov[32];
          if (have) {
            tmem_ld32(tO + lane_base + c0, ov);
            tmem_ld_wait();
          }
          float4* trow = reinterpret_cast<float4*>(tile_s + lane * 36);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);   // a row without keys is 0
            if (have && l_run > 0.f)
              w = make_float4(__uint_as_float(ov[4 * t]) * inv, __uint_as_float(ov[4 * t + 1]) * inv,
                              __uint_as_float(ov[4 * t + 2]) * inv, __uint_as_float(ov[4 * t + 3]) * inv);
            trow[t] = w;
          }
          __syncwarp();
          if (direct) {
            // 8 rows per instruction, 64 bytes (32 bf16) per row
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int rr = t * 8 + (lane >> 2), seg = lane & 3;
              const int gr = row0 + quarter * 32 + rr;
              const float4* sp = reinterpret_cast<const float4*>(tile_s + rr * 36 + seg * 8);
              const float4 v0 = sp[0], v1 = sp[1];
              if (gr < rows)
                *reinterpret_cast<uint4*>(a.out + (static_cast<long long>(b) * a.T * a.Hq + gr) * 512 + rank * 256 + c0 +
                                          seg * 8) =
                    make_uint4(pack_bf16(v0.x, v0.y), pack_bf16(v0.z, v0.w), pack_bf16(v1.x, v1.y), pack_bf16(v1.z, v1.w));
            }
          } else {
            // 4 rows per instruction, 128 bytes (32 fp32) per row
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const int rr = t * 4 + (lane >> 3), seg = lane & 7;
              const int gr = row0 + quarter * 32 + rr;
              const float4 v0 = *reinterpret_cast<const float4*>(tile_s + rr * 36 + seg * 4);
              if (gr < rows)
                *reinterpret_cast<float4*>(
                    a.part_o + (split * n_rows + static_cast<long long>(b) * a.T * a.Hq + gr) * 512 + rank * 256 + c0 +
                    seg * 4) = v0;
            }
          }
          __syncwarp();
        }
      }
      if (rank == 0 && half == 0 && r < rows) {
        if (direct) {
          if (a.lse) a.lse[orow] = l_run > 0.f ? (m_run + log2f(l_run)) * 0.69314718055994530942f : -INFINITY;
        } else {
          a.part_m[split * n_rows + orow] = m_run;
          a.part_l[split * n_rows + orow] = l_run;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) spin_ns(50000);   // let copies and MMAs in flight land before the exit
  cluster_sync_all();                // the partner has finished writing into this CTA's shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_paged_mla(const PagedMaps& m, const PagedArgs& a, cudaStream_t stream) {
  const bool kv8 = a.kv8 != nullptr;
  const void* fn = kv8 ? reinterpret_cast<const void*>(&paged_mla_kernel<true>)
                       : reinterpret_cast<const void*>(&paged_mla_kernel<false>);
  const cudaError_t e = set_max_smem(fn, kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<CUtensorMap*>(&m.k), const_cast<PagedArgs*>(&a)};
  return launch_pdl(fn, dim3(2 * a.tiles, a.n_split, a.B), dim3(kv8 ? threads_of<true>() : threads_of<false>()), kSmem,
                    stream, args);
}

}  // namespace lsa
