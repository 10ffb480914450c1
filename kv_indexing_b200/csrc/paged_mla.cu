// Attention of new tokens over a paged latent cache (MLA: one 576-column row
// per token serves as K, its first 512 columns as V; bf16 or e4m3 with a scale
// per token).
//
//   o[r, :] = sum_{s <= pos(r)} softmax_s(scale * q[r] . c[s]) c[s][0:512],   row r = t * Hq + head
//
// One pass over blocks of 128 keys with a running maximum and sum per row. 128
// rows are one tile; the heads of a token and the tokens of a chunk fill it
// alike.
//
// The output of 128 rows (128 x 512 fp32) would fill an SM's tensor memory, so
// two CTAs (a cluster) share a tile, 64 rows each, and run their products as
// one MMA of the pair (cta_group::2): every SM stages half of the keys (Q K^T)
// and half of the output columns (P V) and multiplies its own rows by both
// halves. Rows never cross CTAs: each keeps its own maximum, sum and P, and the
// pair exchanges nothing but barrier arrivals. (Splitting the products'
// contraction instead has the CTAs exchange 32 KB of partial scores per 64 keys;
// that measured 5.2 us a block, ten times the products themselves.)
//
// Per block and CTA: 128 x 128 x (576 + 512) / 2 multiply-adds, 2176 cycles at
// 4096 a cycle; loads of 136 KB do not slow them. A block takes 3.1 K cycles, 2.3
// K with the softmax left out: the issuing thread shares its scheduler with a
// softmax warp. Back to back, the power cap bounds long calls (1.25 PFLOP/s for a
// 500-token chunk over 32768 tokens; decode of 8 x 131072 tokens runs at 0.55 of
// the tensor and 0.6 of the HBM rate at once, at 1.43 GHz).
//
// Tensor memory (512 columns): O 256, S 64, q's columns [0, 384) as the A operand
// 192 (each row in lanes r and r + 64, as the pair's MMA reads it). Shared
// memory: q's columns [384, 576) 24 KB, P 2 x 16 KB, a ring of ten 16 KB slots
// (with all of q in shared memory there were seven, and loads came late: a block
// took 5100 cycles). A block takes nine of them: K as 64 keys x 128 columns
// (five, the last half empty), V as 64 keys x 128 columns (four). The scores of
// block j + 1 are issued before block j's P V, so the tensor cores work while a
// block's softmax runs; S is free once both CTAs hold its scores in registers.
//
// Threads: warps 0-3 softmax (two threads per row, 64 of the block's keys each:
// the layout of the pair's accumulator); warps 4-7 load every fourth slot each
// (TMA boxes of one page, or of the page's part of 64 keys; one warp alone issues
// boxes at 7 TB/s over the GPU, two at 13, four at 19); the last warp of CTA 0
// issues the MMAs.
//
// e4m3: warps 4-5 load raw codes and warps 6-13 convert them for the products.
// Scores take fp16: a code is an fp16 value, exactly, by one instruction per
// pair. q goes to fp16 times a power of two per row that brings its largest
// column to [2^14, 2^15): exact but for columns 2^28 below that, by 2^-39 of it.
// V and P take bf16, three instructions per pair more (376 us for 4 x 2 queries
// of 64 heads over 262144 ragged tokens, where V and P in fp16 took 361). A key's scale multiplies
// its score and its P; scales of a cache may lie any number of octaves apart
// (appending gives a row of zeros the scale 1, whatever the others have), and
// the keys that make a row's output need not have the large ones. P times the
// scale in fp16, even scaled by row, loses such weights: fp16 spans 2^30, bf16
// has fp32's range. P is rounded to 2^-8 as for a bf16 cache. A power of two that
// follows the largest scale so far keeps the accumulators in range and changes
// no bit of P above 2^-126; it and q's are taken back in fp32.
//
// The running maximum moves only when a block raises it by more than 2^8 (P in
// bf16 keeps its relative precision, sums are fp32), so O is rescaled rarely.
// Keys past a row's position are masked by select. Rows of V at and past
// seq_len, whatever the page still holds there, are cleared in shared memory
// before the product reads them (0 * NaN is NaN). Unmapped pages are read from
// past the pool's last page, which TMA fills with zeros, and masked.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace lsa {
namespace {

using namespace paged;

constexpr int BN = kPagedBN;
constexpr int kRows = 128;                       // rows of a tile, 64 per CTA
constexpr int kChunk = 64 * 128;                 // 64 keys (or rows) x 64 columns, bytes
constexpr int kSlot = 2 * kChunk;
constexpr int kPBytes = 2 * kChunk;              // 64 rows x 128 keys
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
constexpr int kTmemChunks = 6;                   // 64-column chunks of q in tensor memory, the rest in shared memory
constexpr int kOffP = (9 - kTmemChunks) * kChunk;
constexpr int kOffRing = kOffP + 2 * kPBytes;

// The ring, and for e4m3 a second one of raw codes (64 keys x 128 columns, 8 KB)
// before it, deep enough for the loads; the converted slots then need little.
template <bool KV8>
struct Lay {
  static constexpr int kSlots = KV8 ? 6 : 10, kRaw = KV8 ? 8 : 0;
  static constexpr int kOffRaw = kOffRing + kSlots * kSlot;
  static constexpr int kOffSwap = kOffRaw + kRaw * kChunk;       // [2][128] what a row's two threads tell each other
  static constexpr int kOffScale = kOffSwap + 2 * 128 * 4;       // e4m3: [4 warps][2][64] what multiplies scores and P
  static constexpr int kOffBars = kOffScale + (KV8 ? 2 : 0) * 4 * 64 * 4;
  // full, empty, raw_full, raw_empty, s_full, s_free, p_full[2], pv_done, o_full, q_full, tail[4], swap[2], q_tma, p_idle
  static constexpr int kNumBars = 2 * kSlots + 2 * kRaw + 15;
  static constexpr int kOffWork = kOffBars + kNumBars * 8;
  static constexpr int kOffMisc = kOffWork + static_cast<int>(sizeof(Work));
  static constexpr size_t kSmem = 1024 + kOffMisc + 16;
  static constexpr int kMmaWarp = KV8 ? 14 : 8;
  static constexpr int kThreads = (kMmaWarp + 1) * 32;
  static_assert(kOffRing % 1024 == 0 && kOffRaw % 1024 == 0 && kOffScale % 16 == 0 && kOffBars % 8 == 0 && kOffWork % 8 == 0 &&
                    kSmem <= 227 * 1024, "shared memory layout");
};

// Two of four e4m3 codes (the lower or the upper pair) -> an fp16 pair, exact.
template <int HIGH>
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t four) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(HIGH ? four >> 16 : four)));
  return h2;
}
// An fp16 pair that holds codes -> a bf16 pair, exact.
__device__ __forceinline__ uint32_t f16_to_bf16(uint32_t h2) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Lay<KV8>::kThreads, 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const PagedArgs a) {
  using Y = Lay<KV8>;
  constexpr int kSlots = Y::kSlots, kRaw = Y::kRaw, kMmaWarp = Y::kMmaWarp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sP = base + kOffP;
  uint8_t* sRing = base + kOffRing;
  float* swap_s = reinterpret_cast<float*>(base + Y::kOffSwap);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + Y::kOffBars);   // CTA 0: both halves of a slot are there
  uint64_t* empty = full + kSlots;
  uint64_t* raw_full = empty + kSlots;
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* s_full = raw_empty + kRaw;
  uint64_t* s_free = s_full + 1;       // CTA 0: both CTAs have read the scores
  uint64_t* p_full = s_free + 1;       // [2], CTA 0: P of both CTAs is stored
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_full = pv_done + 1;      // the piece's last product
  uint64_t* q_full = o_full + 1;       // CTA 0
  uint64_t* tail = q_full + 1;         // [4] a slot that is cleared in part before it counts, by loading warp
  uint64_t* swap = tail + 4;           // [2] warps w and w + 2 have stored theirs
  uint64_t* q_tma = swap + 2;          // q's columns in shared memory
  uint64_t* p_idle = q_tma + 1;        // the softmax warps are through with P's buffers
  Work* work_s = reinterpret_cast<Work*>(base + Y::kOffWork);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + Y::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = static_cast<int>(cluster_ctarank());
  const int worker = blockIdx.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], KV8 ? 4 : 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 2);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 8);
    for (int i = 0; i < 2; ++i) mbar_init(&p_full[i], 8);
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(q_full, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&tail[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&swap[i], 2);
    mbar_init(q_tma, 1);
    mbar_init(p_idle, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(tmem_slot, kTmemCols);
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    const Work k = plan_work<kRows, BN>(a, worker, a.workers);
    if (lane == 0) *work_s = k;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the partner's barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem + kColO, tS = tmem + kColS, tQ = tmem + kColQ;
  const uint32_t full0 = mapa_shared(smem_u32(full), 0);         // CTA 0's barriers
  bool ok = true;

  if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer --
    // One thread. A barrier is looked at while the products before it are
    // issued: waiting for each in turn, with the products in between, took
    // longer (3700 cycles a block) than the products themselves.
    if (rank == 0 && elect_one()) {
      constexpr uint32_t kType = KV8 ? 0 : 1;     // of q and K: fp16, bf16
      const uint32_t idesc_qk = make_idesc(kType, kType, 128, BN, 0, 0);
      const uint32_t idesc_pv = make_idesc(1, 1, 128, 256, 0, 1);
      const uint32_t hi = static_cast<uint32_t>(make_sdesc(0, 16, 1024, kLayoutSW128) >> 32);
      const uint32_t dQ = static_cast<uint32_t>(make_sdesc(smem_u32(sQ), 16, 1024, kLayoutSW128));
      const uint32_t dP = static_cast<uint32_t>(make_sdesc(smem_u32(sP), 16, 1024, kLayoutSW128));
      const uint32_t dK = static_cast<uint32_t>(make_sdesc(smem_u32(sRing), 16, 1024, kLayoutSW128));
      const uint32_t dV = static_cast<uint32_t>(make_sdesc(smem_u32(sRing), kChunk, 1024, kLayoutSW128));
      int st = 0, cur;                 // the ring's next slot and the parity of its phase; the slot at hand
      uint32_t ph = 0;
      bool seen = false;               // the next slot has been seen full
      // Waits for the next slot, makes it the current one and looks at the one after.
      auto take = [&]() -> bool {
        if (!seen && !wait(&full[st], ph, a.status, abort_flag)) return false;
        cur = st;
        if (++st == kSlots) {
          st = 0;
          ph ^= 1u;
        }
        seen = mbar_test_wait(&full[st], ph);
        tc_fence_after();
        return true;
      };
      uint32_t jb = 0, seg = 0;        // blocks and pieces so far
      bool seen_p = false, seen_s = false;
      auto qk = [&](uint32_t j) -> bool {
        if (j > 0 && !seen_s && !wait(s_free, (j - 1) & 1, a.status, abort_flag)) return false;
#pragma unroll
        for (int s = 0; s < 5; ++s) {        // columns [128 s, 128 s + 128)
          if (!take()) return false;
          const uint32_t k0 = dK + cur * (kSlot / 16);
          if (s == 4) seen_p = j > 0 && mbar_test_wait(&p_full[(j - 1) & 1], ((j - 1) >> 1) & 1);
#pragma unroll
          for (int c = 0; c < (s < 4 ? 2 : 1); ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t kd = k0 + c * (kChunk / 16) + 2 * i;
              if (2 * s + c < kTmemChunks)
                umma_f16_ts_pair(tS, tQ + (2 * s + c) * 32 + 8 * i, kd, hi, idesc_qk, (s | c | i) ? 1u : 0u);
              else
                umma_f16_pair(tS, dQ + (2 * s + c - kTmemChunks) * (kChunk / 16) + 2 * i, kd, hi, idesc_qk, 1u);
            }
          umma_commit_pair(&empty[cur]);
        }
        umma_commit_pair(s_full);
        return true;
      };
      auto pv = [&](uint32_t j, bool first, bool last) -> bool {
        if (!seen_p && !wait(&p_full[j & 1], (j >> 1) & 1, a.status, abort_flag)) return false;
        seen_p = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {        // (half of the keys, half of the columns)
          if (!take()) return false;
          const int h = i >> 1, n = i & 1;
          const uint32_t p0 = dP + ((j & 1) * kPBytes + h * kChunk) / 16, v0 = dV + cur * (kSlot / 16);
          if (i == 3) seen_s = !last && mbar_test_wait(s_free, (j + 1) & 1);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_pair(tO + n * 128, p0 + 2 * ks, v0 + 128 * ks, hi, idesc_pv, first && h == 0 && ks == 0 ? 0u : 1u);
          umma_commit_pair(&empty[cur]);
        }
        umma_commit_pair(pv_done);
        if (last) umma_commit_pair(o_full);
        return true;
      };
      for (Work k = *work_s; ok && k.n > 0; next_work<kRows, BN>(a, k), ++seg) {
        ok = wait(q_full, seg & 1, a.status, abort_flag) && qk(jb);
        seen_p = false;                      // (of the piece before)
        for (int j = 0; ok && j < k.n; ++j) {
          if (j + 1 < k.n) ok = qk(jb + j + 1);
          if (ok) ok = pv(jb + j, j == 0, j + 1 == k.n);
        }
        jb += k.n;
        seen_s = false;
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    if constexpr (!KV8) {
      // -------------------------------------------------------- producer --
      const int box = min(kPagedBox, 1 << a.page_shift);         // rows of a box
      const int per = 64 / box;                                  // boxes of 64 keys
      const int c = lane / per, i = lane - c * per;              // this lane's box: chunk c, rows i * box
      const uint32_t pw = warp - 4;
      uint64_t* my_tail = tail + pw;
      int st = 0;
      uint32_t ph = 1, seq = 0, n_tail = 0;                      // the ring starts empty
      for (Work k = *work_s; ok && k.n > 0; next_work<kRows, BN>(a, k)) {
        const int b = k.bt / a.tiles;
        const Lens L = lens_of(a, b);
        const int* row = a.table + static_cast<long long>(b) * a.max_pages;
        // lane g < 8: the table entry of the block's keys [16 g, 16 g + 16); looked at a block later
        auto entry_of = [&](int j) -> int {
          const int tok = (k.blk0 + j) * BN + lane * 16;
          return lane < 8 && j < k.n && tok < L.len ? __ldg(row + (tok >> a.page_shift)) : kNoPage;
        };
        auto page_of = [&](int p) -> int {
          if (p >= 0 && p < a.n_pages) return p;
          if (p != kNoPage && pw == 0) record_bad_page(a.status);
          return -1;
        };
        // a slot: 64 keys from `key` of block j, `nc` chunks of columns from `chunk`
        auto load = [&](int j, int pages, int key, int chunk, int nc, bool is_v) -> bool {
          const int at = st;
          const uint32_t parity = ph;
          if (++st == kSlots) {
            st = 0;
            ph ^= 1u;
          }
          if ((seq++ & 3u) != pw) return true;                   // another warp's
          if (!__all_sync(0xffffffffu, wait(&empty[at], parity, a.status, abort_flag))) return false;
          const int tok = (k.blk0 + j) * BN + key;
          const int page = __shfl_sync(0xffffffffu, pages, ((key + i * box) >> 4) & 31);
          const int rows = L.len - tok;                          // rows that hold a token
          const bool clear = is_v && rows > 0 && rows < 64;
          if (lane == 0) {
            if (clear) mbar_arrive_expect_tx(my_tail, nc * kChunk);
            else mbar_arrive_expect_tx_at(full0 + at * 8, nc * kChunk);
          }
          __syncwarp();
          uint8_t* dst = sRing + at * kSlot;
          if (lane < nc * per) {
            const int in_page = (tok + i * box) & ((1 << a.page_shift) - 1);
            if (clear)
              tma_load_page(dst + c * kChunk + i * box * 128, &tm_k, my_tail, (chunk + c) * 64, in_page, page >= 0 ? page : a.n_pages);
            else
              tma_load_page_pair(dst + c * kChunk + i * box * 128, &tm_k, full0 + at * 8, (chunk + c) * 64, in_page,
                                 page >= 0 ? page : a.n_pages);
          }
          if (clear) {
            if (!__all_sync(0xffffffffu, wait(my_tail, n_tail & 1, a.status, abort_flag))) return false;
            ++n_tail;
            for (int z = lane; z < (64 - rows) * 16; z += 32) {
              const int zr = rows + (z >> 4), u = z & 15;
              *reinterpret_cast<uint4*>(dst + (u >> 3) * kChunk + zr * 128 + (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(full0 + at * 8);
          }
          return true;
        };
        auto load_k = [&](int j, int pages) -> bool {
          for (int s = 0; s < 5; ++s)
            if (!load(j, pages, rank * 64, 2 * s, s < 4 ? 2 : 1, false)) return false;
          return true;
        };
        auto load_v = [&](int j, int pages) -> bool {
          for (int s = 0; s < 4; ++s)
            if (!load(j, pages, (s >> 1) * 64, (s & 1) * 4 + rank * 2, 2, true)) return false;
          return true;
        };
        int cur = page_of(entry_of(0)), entry = entry_of(1);
        ok = load_k(0, cur);
        for (int j = 0; ok && j < k.n; ++j) {
          const int nxt = page_of(entry);
          entry = entry_of(j + 2);
          if (j + 1 < k.n) ok = load_k(j + 1, nxt);
          if (ok) ok = load_v(j, cur);
          cur = nxt;
        }
      }
    } else {
      uint8_t* sRaw = base + Y::kOffRaw;
      if (warp < 6) {
        // ------------------------------- e4m3: raw codes, alternate slots --
        const uint32_t pw = warp - 4;
        const int box = min(kPagedBox, 1 << a.page_shift), per = 64 / box;
        uint32_t seq = 0;
        for (Work k = *work_s; ok && k.n > 0; next_work<kRows, BN>(a, k)) {
          const int b = k.bt / a.tiles;
          const Lens L = lens_of(a, b);
          const int* trow = a.table + static_cast<long long>(b) * a.max_pages;
          // lane g < 8: the table entry of the block's keys [16 g, 16 g + 16); looked at a block later
          auto entry_of = [&](int j) -> int {
            const int tok = (k.blk0 + j) * BN + lane * 16;
            return lane < 8 && j < k.n && tok < L.len ? __ldg(trow + (tok >> a.page_shift)) : kNoPage;
          };
          auto page_of = [&](int p) -> int {
            if (p >= 0 && p < a.n_pages) return p;
            if (p != kNoPage && pw == 0) record_bad_page(a.status);
            return -1;
          };
          // 64 keys from `key` of block j, 128 codes from `col`
          auto load = [&](int j, int pages, int key, int col) -> bool {
            const uint32_t at = seq++, rs = at % kRaw;
            if ((at & 1u) != pw) return true;                    // the other warp's
            if (!__all_sync(0xffffffffu, wait(&raw_empty[rs], ((at / kRaw) & 1) ^ 1, a.status, abort_flag))) return false;
            const int tok = (k.blk0 + j) * BN + key;
            const int page = __shfl_sync(0xffffffffu, pages, ((key + lane * box) >> 4) & 31);
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[rs], kChunk);
            __syncwarp();
            if (lane < per)
              tma_load_page(sRaw + rs * kChunk + lane * box * 128, &tm_k, &raw_full[rs], col,
                            (tok + lane * box) & ((1 << a.page_shift) - 1), page >= 0 ? page : a.n_pages);
            return true;
          };
          auto load_k = [&](int j, int pages) -> bool {
#pragma unroll 1
            for (int s = 0; s < 5; ++s)                          // the last one half past the row's end: zeros
              if (!load(j, pages, rank * 64, s * 128)) return false;
            return true;
          };
          auto load_v = [&](int j, int pages) -> bool {
#pragma unroll 1
            for (int s = 0; s < 4; ++s)
              if (!load(j, pages, (s >> 1) * 64, (s & 1) * 256 + rank * 128)) return false;
            return true;
          };
          int cur = page_of(entry_of(0)), entry = entry_of(1);
          ok = load_k(0, cur);
          for (int j = 0; ok && j < k.n; ++j) {
            const int nxt = page_of(entry);
            entry = entry_of(j + 2);
            if (j + 1 < k.n) ok = load_k(j + 1, nxt);
            if (ok) ok = load_v(j, cur);
            cur = nxt;
          }
        }
      } else {
        // ------------------- e4m3: codes -> fp16 (K), bf16 (V), into the ring --
        // Four groups of two warps take every fourth slot, any slot (two groups of four
        // took 5 % longer; groups for K and groups for V, with their codes in registers,
        // ran at a sixth of an instruction a cycle). No more groups than slots: a group that is at slot `at` has filled
        // at - 4, so at - 12 has been consumed and the parity of `empty` is not two
        // phases old. A lane converts 8 codes at a time; odd rows take a slot's
        // chunks the other way round, so that two rows' reads do not meet in a bank.
        constexpr uint32_t kGroups = 4;
        static_assert(kGroups <= kSlots && kRaw % kGroups == 0, "parities");
        const uint32_t group = (warp - 6) >> 1;
        const int t = (tid - 192) & 63;
        const int row = t >> 3, unit = t & 7;                    // rows row + 8 i
        uint32_t seq = 0;                                        // slots before the piece
        for (Work k = *work_s; ok && k.n > 0; next_work<kRows, BN>(a, k)) {
          const Lens L = lens_of(a, k.bt / a.tiles);
          const uint32_t n = 9 * k.n;
#pragma unroll 1
          for (uint32_t i = (group - seq) % kGroups; i < n; i += kGroups) {
            // the ring takes K(0), then K(j + 1) (while there is one) and V(j) in turn
            int rows = 64, chunks = 2;                           // rows that count (V), chunks of the slot
            bool is_v = false;
            if (i == 4) {
              chunks = 1;
            } else if (i > 4) {
              const int q = i - 5, j = q / 9, s = q - 9 * j;
              const bool last = j + 1 == k.n;
              if (!last && s < 5) {
                if (s == 4) chunks = 1;
              } else {
                const int half = (last ? s : s - 5) >> 1;
                is_v = true;
                rows = L.len - (k.blk0 + j) * BN - half * 64;
              }
            }
            const uint32_t at = seq + i, rs = at % kRaw, st = at % kSlots;
            ok = __all_sync(0xffffffffu, wait(&raw_full[rs], (at / kRaw) & 1, a.status, abort_flag) &&
                                             wait(&empty[st], ((at / kSlots) & 1) ^ 1, a.status, abort_flag));
            if (!ok) break;
            const uint8_t* src = sRaw + rs * kChunk;
            uint8_t* dst = sRing + st * kSlot;
            // (one test a slot: inside the loop K's codes would go through the longer way too)
            auto convert = [&](auto to) {
#pragma unroll
              for (int r4 = 0; r4 < 8; ++r4) {
                const int r = row + 8 * r4;
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                  const int c = cc ^ (row & 1);
                  if (c >= chunks) continue;
                  uint2 e = *reinterpret_cast<const uint2*>(src + r * 128 + c * 64 + unit * 8);
                  if (r >= rows) e = make_uint2(0u, 0u);         // past seq_len, whatever the page holds
                  *reinterpret_cast<uint4*>(dst + c * kChunk + r * 128 + ((unit ^ (r & 7)) << 4)) =
                      make_uint4(to(codes_to_f16<0>(e.x)), to(codes_to_f16<1>(e.x)), to(codes_to_f16<0>(e.y)),
                                 to(codes_to_f16<1>(e.y)));
                }
              }
            };
            if (is_v) convert([](uint32_t h2) { return f16_to_bf16(h2); });
            else convert([](uint32_t h2) { return h2; });
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&raw_empty[rs]);
              mbar_arrive_at(full0 + st * 8);
            }
          }
          seq += n;
        }
      }
    }
  } else {
    // ------------------------------------------------- softmax / epilogue --
    const int h = tid >> 6, r = tid & 63;          // half of the block's keys, row of the CTA
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t p_full0 = mapa_shared(smem_u32(p_full), 0), q_full0 = mapa_shared(smem_u32(q_full), 0);
    const uint32_t s_free0 = mapa_shared(smem_u32(s_free), 0);
    float* scale_s = reinterpret_cast<float*>(base + Y::kOffScale) + warp * 128;   // [2][64]
    uint32_t jb = 0, seg = 0, n_swap = 0;
    // Tells the row's other thread v and returns its value (through alternate buffers: a value is read before the
    // partner can get to the exchange after the next).
    auto exchange = [&](float v, float* other) -> bool {
      float* buf = swap_s + (n_swap & 1) * 128;
      buf[tid] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&swap[warp & 1]);
      const bool done = __all_sync(0xffffffffu, wait(&swap[warp & 1], n_swap & 1, a.status, abort_flag));
      ++n_swap;
      *other = buf[tid ^ 64];
      return done;
    };
    for (Work k = *work_s; ok && k.n > 0; next_work<kRows, BN>(a, k), ++seg) {
      const int b = k.bt / a.tiles, row0 = (k.bt - b * a.tiles) * kRows + rank * 64;
      const Lens L = lens_of(a, b);
      const int rows = L.n_new * a.Hq;
      const int* trow = a.table + static_cast<long long>(b) * a.max_pages;
      const long long q0 = static_cast<long long>(b) * a.T * a.Hq + row0;   // the CTA's first row of q and out
      float c;                                     // score -> log2 domain
      {
        c = a.scale_log2;
        // q's columns: [0, 256) by TMA into P's buffers and from there into tensor memory, [256, 384) into tensor memory
        // by loads, [384, 576) by TMA where the MMA reads them. (All by loads of each thread's row: 13000 cycles.) Rows
        // behind the sequence's last are whatever lies there; no row meets another.
        if (warp == 0) {
          if (seg > 0) ok = __all_sync(0xffffffffu, wait(p_idle, (seg - 1) & 1, a.status, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(q_tma, (9 - kTmemChunks + 4) * kChunk);
          __syncwarp();
          if (lane < 9 - kTmemChunks + 4) {
            const int ch = lane < 4 ? lane : kTmemChunks + lane - 4;
            tma_load_2d(lane < 4 ? sP + lane * kChunk : sQ + (lane - 4) * kChunk, &tm_q, q_tma, ch * 64, static_cast<int>(q0));
          }
        }
        const bool mine = row0 + r < rows;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (q0 + r) * 576);
        uint32_t v[2][32];
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)               // two bf16 per column, ascending; both threads of a row
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 w = mine ? __ldg(src + (4 + ch) * 8 + u) : make_uint4(0u, 0u, 0u, 0u);
            v[ch][4 * u] = w.x;
            v[ch][4 * u + 1] = w.y;
            v[ch][4 * u + 2] = w.z;
            v[ch][4 * u + 3] = w.w;
          }
        if constexpr (!KV8) {
          tmem_st32(tQ + lane_base + 4 * 32, v[0]);
          tmem_st32(tQ + lane_base + 5 * 32, v[1]);
        }
        ok = __all_sync(0xffffffffu, wait(q_tma, seg & 1, a.status, abort_flag));
        if (!ok) break;
        auto unit = [&](uint8_t* chunk, int u) -> uint4* {
          return reinterpret_cast<uint4*>(chunk + r * 128 + ((u ^ (r & 7)) << 4));
        };
        float up = 1.f;                              // e4m3: the row's power of two
        if constexpr (KV8) {
          float top = 0.f;
          auto see = [&](uint32_t w) {
            const float2 f = unpack_bf16(w);
            top = max3(top, fabsf(f.x), fabsf(f.y));
          };
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            see(v[0][i]);
            see(v[1][i]);
          }
#pragma unroll 4
          for (int i = h; i < (9 - kTmemChunks + 4) * 8; i += 2) {   // the row's threads share the rest
            const uint4 w = *unit((i < 32 ? sP : sQ - 4 * kChunk) + (i >> 3) * kChunk, i & 7);
            see(w.x);
            see(w.y);
            see(w.z);
            see(w.w);
          }
          float other;
          ok = exchange(top, &other);
          if (!ok) break;
          const int e = 14 + 127 - static_cast<int>(__float_as_uint(fmaxf(top, other)) >> 23);
          // c stays a normal number: masked scores are -inf times c
          const int pow = max(-100, min(min(100, e), static_cast<int>(__float_as_uint(a.scale_log2) >> 23) - 1));
          up = __uint_as_float(static_cast<uint32_t>(pow + 127) << 23);
          c = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - pow) << 23);
        }
        auto to_type = [&](uint32_t w) -> uint32_t {
          if constexpr (!KV8) return w;
          const float2 f = unpack_bf16(w);
          return pack_f16(f.x * up, f.y * up);
        };
        if constexpr (KV8) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[0][i] = to_type(v[0][i]);
            v[1][i] = to_type(v[1][i]);
          }
          tmem_st32(tQ + lane_base + 4 * 32, v[0]);
          tmem_st32(tQ + lane_base + 5 * 32, v[1]);
          for (int i = h; i < (9 - kTmemChunks) * 8; i += 2) {
            uint4* at = unit(sQ + (i >> 3) * kChunk, i & 7);
            const uint4 w = *at;
            *at = make_uint4(to_type(w.x), to_type(w.y), to_type(w.z), to_type(w.w));
          }
          fence_proxy_async_smem();
        }
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t x[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 w = *unit(sP + ch * kChunk, u);
            x[4 * u] = to_type(w.x);
            x[4 * u + 1] = to_type(w.y);
            x[4 * u + 2] = to_type(w.z);
            x[4 * u + 3] = to_type(w.w);
          }
          tmem_st32(tQ + lane_base + ch * 32, x);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(q_full0);
      }
      // keys this row sees; rows that do not exist see all, so that they make no block a masked one
      const int bound = row0 + r < rows ? max(0, min(L.len, L.len - L.n_new + (row0 + r) / a.Hq + 1)) : L.len;
      // lane g < 8: the table entry of the block's keys [16 g, 16 g + 16), to see whether they have a page
      auto entry_of = [&](int j) -> int {
        const int tok = (k.blk0 + j) * BN + lane * 16;
        return lane < 8 && j < k.n && tok < L.len ? __ldg(trow + (tok >> a.page_shift)) : kNoPage;
      };
      // e4m3: this lane's four of the block's scales, keys 64 h + lane + {0, 32} and those of the other half (0 where
      // there is none)
      auto key_at = [&](int j, int i) -> int { return (k.blk0 + j) * BN + (64 * h ^ (i & 2) * 32) + lane + (i & 1) * 32; };
      auto page_at = [&](int j, int i) -> int {
        const int tok = key_at(j, i);
        return j < k.n && tok < L.len ? __ldg(trow + (tok >> a.page_shift)) : kNoPage;
      };
      auto scale_at = [&](int j, int i, int page) -> float {
        if (page < 0 || page >= a.n_pages) return 0.f;
        return __ldg(a.k_scale + (static_cast<long long>(page) << a.page_shift) + (key_at(j, i) & ((1 << a.page_shift) - 1)));
      };
      int entry = entry_of(0);
      float sc[4];
      int pg[4];
      if constexpr (KV8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[i] = scale_at(0, i, page_at(0, i));
          pg[i] = page_at(1, i);
        }
      }
      // e4m3: the exponent field of the largest scale so far, and the power of two that P is multiplied by for it
      uint32_t top_exp = 7u;
      float p_up = __uint_as_float((260u - 7u) << 23);
      float m_run = -INFINITY, l_part = 0.f;       // log2 domain; l_part: this thread's keys
      for (int j = 0; j < k.n; ++j) {
        const uint32_t at = jb + j;
        const int key0 = (k.blk0 + j) * BN + 64 * h;
        const uint32_t pages = __ballot_sync(0xffffffffu, entry >= 0 && entry < a.n_pages) >> (4 * h) & 0xFu;
        entry = entry_of(j + 1);
        float o_down = 1.f;                        // e4m3: what O has to be multiplied by for a larger scale
        if constexpr (KV8) {
          uint32_t top = __float_as_uint(fmaxf(max3(fabsf(sc[0]), fabsf(sc[1]), fabsf(sc[2])), fabsf(sc[3])));
          top = min(__reduce_max_sync(0xffffffffu, top) >> 23, 250u);
          if (top > top_exp) {                     // (the same in every thread of the CTA)
            o_down = top - top_exp < 127u ? __uint_as_float((127u - (top - top_exp)) << 23) : 0.f;
            top_exp = top;
            p_up = __uint_as_float((260u - top) << 23);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            scale_s[lane + 32 * i] = sc[i];
            scale_s[64 + lane + 32 * i] = sc[i] * p_up;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[i] = scale_at(j + 1, i, pg[i]);
            pg[i] = page_at(j + 2, i);
          }
        }
        ok = __all_sync(0xffffffffu, wait(s_full, at & 1, a.status, abort_flag));
        if (!ok) break;
        tc_fence_after();
        float x[64];
        {
          uint32_t s0[32], s1[32];
          tmem_ld32(tS + lane_base, s0);
          tmem_ld32(tS + lane_base + 32, s1);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(s_free0);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(s0[i]);
            x[32 + i] = __uint_as_float(s1[i]);
          }
        }
        const float4* ks4 = reinterpret_cast<const float4*>(scale_s);
        if constexpr (KV8) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 k4 = ks4[i];
            x[4 * i] *= k4.x;
            x[4 * i + 1] *= k4.y;
            x[4 * i + 2] *= k4.z;
            x[4 * i + 3] *= k4.w;
          }
        }
        const int vis = bound - key0;              // visible keys of this half block
        if (__any_sync(0xffffffffu, vis < 64) || pages != 0xFu) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= vis || !((pages >> (i >> 4)) & 1u)) x[i] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[i + e], x[i + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[60 + e]);
        const float mine = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
        float other;
        ok = exchange(mine, &other);
        if (!ok) break;
        const float mb = fmaxf(mine, other);
        bool move = mb > m_run + 8.f || (m_run == -INFINITY && mb != -INFINITY);
        float corr = 1.f;
        if (move) {
          corr = m_run == -INFINITY ? 0.f : ex2(m_run - mb);
          l_part *= corr;
          m_run = mb;
        }
        if constexpr (KV8) {
          corr *= o_down;
          move = move || o_down != 1.f;
        }
        const float mu = m_run == -INFINITY ? 0.f : m_run;   // all masked so far: exp2(-inf) = 0
        // P of block at - 2 has been read: its product was issued before the scores of this block
        uint8_t* prow = sP + (at & 1) * kPBytes + h * kChunk + r * 128;
        float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 c2 = make_float2(c, c), mu2 = make_float2(-mu, -mu);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 8 * u + 2 * e;
            float2 p = fma2(make_float2(x[i], x[i + 1]), c2, mu2);
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            ps[e & 1] = add2(ps[e & 1], p);
            if constexpr (KV8) {                   // V row = code * scale: the scale rides on P
              const float2 k2 = reinterpret_cast<const float2*>(scale_s + 64)[i >> 1];
              p.x *= k2.x;
              p.y *= k2.y;
            }
            w[e] = pack_bf16(p.x, p.y);
          }
          *reinterpret_cast<uint4*>(prow + ((u ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        l_part += (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
        if (j > 0 && __any_sync(0xffffffffu, move)) {   // rescale this thread's part of O
          // (at most this block's product is unfinished besides: the scores at hand were issued after all before it)
          ok = __all_sync(0xffffffffu, wait(pv_done, (at - 1) & 1, a.status, abort_flag));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + lane_base + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * corr);
            tmem_st32(tO + lane_base + c0, ov);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(p_full0 + (at & 1) * 8);
      }
      jb += k.n;
      if (ok) ok = __all_sync(0xffffffffu, wait(o_full, seg & 1, a.status, abort_flag));
      if (!ok) break;
      // row sum over both halves (fixed order: both threads get the same value)
      float l_other;
      ok = exchange(l_part, &l_other);
      if (!ok) break;
      const float l_run = h == 0 ? l_part + l_other : l_other + l_part;
      // ---- epilogue: the accumulator holds columns [256 n + 128 h, + 128) of the row, n = 0, 1; staged per warp
      // (in P's buffers) for coalesced stores
      tc_fence_after();
      const bool whole = k.n == k.all;
      const int slot = 2 * worker + (k.blk0 == 0);
      float inv = l_run != 0.f ? 1.f / l_run : 0.f;
      if constexpr (KV8) inv *= __uint_as_float((top_exp - 6u) << 23);   // 1 / p_up
      const int wrow = (warp & 1) * 32;            // the warp's first row
      // [32 rows][64 floats], 16-byte units XOR-swizzled by the row
      float4* tile_s = reinterpret_cast<float4*>(sP + warp * 8192);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int col = (q >> 1) * 256 + h * 128 + (q & 1) * 64;
        uint32_t ov[2][32];
        tmem_ld32(tO + lane_base + q * 64, ov[0]);
        tmem_ld32(tO + lane_base + q * 64 + 32, ov[1]);
        tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const uint32_t* o = ov[u >> 3] + 4 * (u & 7);
          float4 w = make_float4(0.f, 0.f, 0.f, 0.f);      // a row without keys is 0
          if (l_run != 0.f)
            w = make_float4(__uint_as_float(o[0]) * inv, __uint_as_float(o[1]) * inv, __uint_as_float(o[2]) * inv,
                            __uint_as_float(o[3]) * inv);
          tile_s[lane * 16 + (u ^ (lane & 15))] = w;
        }
        __syncwarp();
        if (whole) {
          // 4 rows per instruction, 128 bytes (64 bf16) per row
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = i * 4 + (lane >> 3), u = 2 * (lane & 7);
            const float4 v0 = tile_s[rr * 16 + (u ^ (rr & 15))], v1 = tile_s[rr * 16 + ((u + 1) ^ (rr & 15))];
            if (row0 + wrow + rr < rows)
              *reinterpret_cast<uint4*>(a.out + (q0 + wrow + rr) * 512 + col + 4 * u) =
                  make_uint4(pack_bf16(v0.x, v0.y), pack_bf16(v0.z, v0.w), pack_bf16(v1.x, v1.y), pack_bf16(v1.z, v1.w));
          }
        } else {
          // 2 rows per instruction, 256 bytes (64 fp32) per row
          float* to = a.part_o + (static_cast<long long>(slot) * kRows + rank * 64 + wrow) * 512 + col;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int rr = i * 2 + (lane >> 4), u = lane & 15;
            const float4 v0 = tile_s[rr * 16 + (u ^ (rr & 15))];
            if (row0 + wrow + rr < rows) *reinterpret_cast<float4*>(to + rr * 512 + 4 * u) = v0;
          }
        }
        __syncwarp();
      }
      if (h == 0 && row0 + r < rows) {
        if (whole) {
          if (a.lse) a.lse[q0 + r] = l_run != 0.f ? (m_run + log2f(l_run)) * 0.69314718055994530942f : -INFINITY;
        } else {
          a.part_m[slot * kRows + rank * 64 + r] = m_run;
          a.part_l[slot * kRows + rank * 64 + r] = l_run;
        }
      }
      if (tid == 0 && rank == 0 && k.blk0 == 0) a.span[k.bt] = make_longlong2(k.begin, k.all);
      fence_proxy_async_smem();                    // the next piece's q comes into P's buffers by TMA
      __syncwarp();
      if (lane == 0) mbar_arrive(p_idle);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) spin_ns(50000);   // let copies and MMAs in flight land before the exit
  cluster_sync_all();                // no barrier of this CTA is used by the partner any more
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

template <bool KV8>
static cudaError_t launch_mla_t(const PagedMaps& m, const PagedArgs& a, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&paged_mla_kernel<KV8>);
  const cudaError_t e = set_max_smem(fn, Lay<KV8>::kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<CUtensorMap*>(&m.k), const_cast<CUtensorMap*>(&m.v), const_cast<PagedArgs*>(&a)};
  return launch_pdl(fn, dim3(2 * a.workers), dim3(Lay<KV8>::kThreads), Lay<KV8>::kSmem, stream, args);
}

cudaError_t launch_paged_mla(const PagedMaps& m, const PagedArgs& a, int e4m3, cudaStream_t stream) {
  return e4m3 ? launch_mla_t<true>(m, a, stream) : launch_mla_t<false>(m, a, stream);
}

}  // namespace lsa
