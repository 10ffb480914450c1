// Attention of new tokens over a paged cache, separate K and V, d = 64 or 128,
// grouped heads.
//
//   o[r, :] = sum_{s <= pos(r)} softmax_s(scale * q[r] . K[s]) V[s]
//
// One pass over the keys with a running maximum and sum per row. The rows of a
// KV head are its (token, head of the group) pairs, row = t * G + head, so any
// group size fills the 128 rows of the score MMA.
//
// A block works on two row tiles in turn, so that the tensor cores compute one
// tile's products while the other's softmax runs:
//   SHARED = 1 (more than 128 rows): two tiles of 128 rows over the same keys;
//   SHARED = 0 (a few rows): one tile of rows, the two halves taking a piece's
//     keys 64 by 64 in turn, each with its own maximum, sum and output; half 1
//     hands its output to half 0 through shared memory.
//
// A block works through the pieces of the work list (paged.cuh) that are its.
//
// Threads (384): warps 0-3 and 4-7 are the softmax of the two halves, one
// thread per row, with registers enough for a step's 128 scores (read twice from
// tensor memory instead, or split over two threads a row, a step's softmax took
// longer: 812 and 760 us where this takes 724, for chunks of 2 x 2000 tokens over
// 16384 in short runs; 800 to 825 back to back, under the power cap); warps 8 and
// 10 load K and V pages by TMA into a ring of tiles (boxes of one page, or of the
// page's part of the tile; one warp alone issues boxes more slowly than HBM
// delivers them); one thread of warp 9 issues the MMAs. Scores and O of both halves fill tensor memory. P (bf16) overwrites the
// scores it came from and is the A operand of the second MMA. MMAs issued by one
// thread run in order, so scores cannot overtake the product that reads their
// buffer's last P.
//
// A step is one K and one V tile.
//   SHARED = 1: 128 keys, one buffer of scores a half. One half's products run
//     while the other's softmax does; a half's second product starts on the
//     first 64 keys of P. (64 keys and two buffers, as below, let the products
//     run ahead, but a score product of 64 keys takes 1.5 times its share: its A
//     operand, q, is read from shared memory as often as for 128.)
//   SHARED = 0: 64 keys, two buffers a half, the scores of a half's next step
//     computed while its softmax runs. Bound by loads, not by products.
//
// The running maximum only moves when a block raises it by more than 2^8 (P keeps
// its relative precision), so O is rescaled rarely. Sums are fp32. P is rounded to
// bf16, the type of V, as one MMA's operands have one type: 2.3e-3 off in all (rms,
// relative, of normal inputs) where weights in fp32 and the output's own rounding
// give 1.7e-3.
//
// Keys past a row's position are masked by select. Rows of V at and past
// seq_len (whatever a page still holds there) are cleared in shared memory
// before the product reads them: 0 * NaN is NaN. Unmapped pages are loaded from
// past the pool's last page, which TMA fills with zeros, and masked.
//
// A row without keys has a sum of 0 and gets 0; a NaN of q makes the row's sum
// NaN (its maximum, which ignores NaN, does not show it) and its output NaN.
#include "paged.cuh"

namespace lsa {
namespace {

using namespace paged;

constexpr int kSoft = 256;             // softmax threads
constexpr int kThreads = 384;          // three warpgroups, for the register split
constexpr int BN = kPagedBN;           // keys of a block of the work list

template <int D, bool SHARED>
struct Cfg {
  static constexpr int kStep = SHARED ? 128 : 64;      // keys of a step
  static constexpr int kChunks = D / 64;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kQTiles = SHARED ? 2 : 1;
  static constexpr int kStage = kStep * D * 2;
  // SHARED = 0: at least six, since half 1's next scores are issued before half 0's product
  static constexpr int kStages = 160 * 1024 / kStage;
  static constexpr int kOffStage = kQTiles * kQTile;
  static constexpr int kOffMask = kOffStage + kStages * kStage;
  static constexpr int kOffBars = kOffMask + ((kStages * 4 + 7) / 8) * 8;
  static constexpr int kNumBars = 2 * kStages + 15;
  static_assert(kStages % 2 == 0 || SHARED, "K and V places");
  static constexpr int kOffWork = kOffBars + kNumBars * 8;
  static constexpr int kOffMerge = (kOffWork + 9 * static_cast<int>(sizeof(Work)) + 15) / 16 * 16;   // the block's, and the softmax warps'
  static constexpr int kMergeRow = 36;                 // floats: 32 columns, padded
  static constexpr int kOffMisc = kOffMerge + (SHARED ? 0 : 128 * kMergeRow * 4);
  static constexpr size_t kSmem = 1024 + kOffMisc + 16;
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // S of half i at 128 i (two buffers of 64 where a step is 64 keys), O at 256 + D i

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const PagedArgs a) {
  using C = Cfg<D, SHARED>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory budget");
  constexpr int kStep = C::kStep;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sStage = base + C::kOffStage;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(base + C::kOffMask);   // [kStages] of a V tile: which 16 keys have a page
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBars);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + C::kStages;
  uint64_t* s_full = bars + 2 * C::kStages;   // [2 halves][2 buffers]
  uint64_t* p_full = s_full + 4;              // [2][2 buffers, or 64-key parts of the one]
  uint64_t* pv_done = p_full + 4;             // [2]
  uint64_t* o_full = pv_done + 2;             // [2] the piece's last product
  uint64_t* q_full = o_full + 2;
  uint64_t* mg_full = q_full + 1;             // half 1's columns are in the merge buffer / have been read
  uint64_t* mg_empty = mg_full + 1;
  float* merge_s = reinterpret_cast<float*>(base + C::kOffMerge);
  Work* work_s = reinterpret_cast<Work*>(base + C::kOffWork);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  constexpr int kTile = SHARED ? 256 : 128;
  const int worker = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(q_full, kSoft);
    mbar_init(mg_full, 128);
    mbar_init(mg_empty, 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    const Work k = plan_work<kTile, BN>(a, worker, a.workers);
    if (lane == 0) *work_s = k;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  // A piece: its sequence, rows, and the steps of the halves (the same in every thread).
  struct Piece {
    int b, g, row0, rows, first_pos, len;
    int n0, n1;                                // steps of the halves
  };
  auto piece_of = [&](const Work& k) -> Piece {
    Piece p;
    p.b = k.bt / a.tiles;
    p.g = k.g;
    p.row0 = (k.bt - p.b * a.tiles) * kTile;
    const Lens L = lens_of(a, p.b);
    p.len = L.len;
    p.rows = L.n_new * a.G;
    p.first_pos = L.len - L.n_new;             // position of token t: first_pos + t
    // steps of the piece that the last of the rows [r0, r0 + n) sees
    auto steps = [&](int r0, int n) -> int {
      if (r0 >= p.rows) return 0;
      const int keys = max(0, min(L.len, p.first_pos + (min(p.rows, r0 + n) - 1) / a.G + 1));
      return max(0, min(k.n * (BN / kStep), (keys + kStep - 1) / kStep - k.blk0 * (BN / kStep)));
    };
    if (SHARED) {
      p.n0 = steps(p.row0, 128);
      p.n1 = steps(p.row0 + 128, 128);
    } else {
      const int n = steps(p.row0, 128);
      p.n0 = (n + 1) / 2;
      p.n1 = n / 2;
    }
    return p;
  };
  // tiles of K (and of V) that are loaded
  auto n_tiles_of = [&](const Piece& p) -> int { return SHARED ? max(p.n0, p.n1) : p.n0 + p.n1; };
  // tile of half i's step u; its K and V follow one another in the ring
  auto tile_of = [&](int i, int u) -> int { return SHARED ? u : 2 * u + i; };

  // Softmax threads hold 128 scores: 208 registers each, 80 for the others (256 x 208 + 128 x 80 of the block's 384 x 168)
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == 8 || warp == 10) {
    // ------------------------------------------------ producers (K and V) --
    const uint32_t kv = warp == 10;
    const int box = min(kPagedBox, 1 << a.page_shift), per = kStep / box;   // rows of a box, boxes of 64 columns
    const int n_ops = C::kChunks * per;
    const int j = lane % per, c = lane / per;
    const uint32_t groups = (1u << (box / 16)) - 1u;
    uint32_t seq = 0;
    for (Work k = *work_s; ok && k.n > 0; next_work<kTile, BN>(a, k)) {
      const Piece p = piece_of(k);
      const int n_tiles = n_tiles_of(p), first = k.blk0 * BN + j * box;
      const int* row = a.table + static_cast<long long>(p.b) * a.max_pages;
      auto page_of = [&](int tile) -> int {    // physical page of this lane's box of the tile
        const int tok = first + tile * kStep;
        return tile < n_tiles && tok < p.len ? __ldg(row + (tok >> a.page_shift)) : kNoPage;
      };
      int next = page_of(0);
      for (int tile = 0; ok && tile < n_tiles; ++tile) {
        int page = next;
        next = page_of(tile + 1);              // not looked at before the next tile: the load takes its time
        if (page < 0 || page >= a.n_pages) {
          if (page != kNoPage && c == 0 && kv == 0) record_bad_page(a.status);
          page = -1;
        }
        uint32_t mapped = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t at = seq + 2 * tile + kv, st = at % C::kStages;
        ok = __all_sync(0xffffffffu, wait(&kv_empty[st], ((at / C::kStages) & 1) ^ 1, a.status, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          if (kv) {
            uint32_t m = 0u;
            for (int i = 0; i < per; ++i, mapped >>= 1) m |= (mapped & 1u ? groups : 0u) << (i * (box / 16));
            mask_s[st] = m;
          }
          mbar_arrive_expect_tx(&kv_full[st], C::kStage);
        }
        __syncwarp();
        if (lane < n_ops)
          tma_load_page(sStage + st * C::kStage + c * (kStep * 128) + j * box * 128, kv ? &tm_v : &tm_k, &kv_full[st],
                        p.g * D + c * 64, (first + tile * kStep) & ((1 << a.page_shift) - 1), page >= 0 ? page : a.n_pages);
      }
      seq += 2 * n_tiles;
    }
  } else if (warp == 9) {
    // -------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      const uint32_t idesc_qk = make_idesc(1, 1, 128, kStep, 0, 0);
      const uint32_t idesc_pv = make_idesc(1, 1, 128, D, 0, 1);
      const uint32_t hi = static_cast<uint32_t>(make_sdesc(0, 16, 1024, kLayoutSW128) >> 32);
      const uint32_t dQ = static_cast<uint32_t>(make_sdesc(smem_u32(sQ), 16, 1024, kLayoutSW128));
      const uint32_t dK = static_cast<uint32_t>(make_sdesc(smem_u32(sStage), 16, 1024, kLayoutSW128));
      const uint32_t dV = static_cast<uint32_t>(make_sdesc(smem_u32(sStage), kStep * 128, 1024, kLayoutSW128));
      // Places of the next K and V tile in the ring (every other stage) and their phases. Barriers are looked at before
      // the products in front of them are issued; waiting for each when it is needed takes longer than the products.
      struct Place {
        int st;
        uint32_t ph;
        bool seen;
      } kp{0, 0u, false}, vp{1, 0u, false};
      auto look = [&](Place& p) { p.seen = mbar_test_wait(&kv_full[p.st], p.ph); };
      auto take = [&](Place& p) -> bool {
        if (!p.seen && !wait(&kv_full[p.st], p.ph, a.status, abort_flag)) return false;
        p.seen = true;
        tc_fence_after();
        return true;
      };
      auto release = [&](Place& p) {
        umma_commit(&kv_empty[p.st]);
        p.seen = false;
        if ((p.st += 2) >= C::kStages) {
          p.st -= C::kStages;
          p.ph ^= 1u;
        }
      };
      uint32_t seg = 0, at0 = 0, at1 = 0;                    // pieces, steps of the halves before this piece
      auto at = [&](int i, int u) -> uint32_t { return (i ? at1 : at0) + u; };
      auto qk = [&](int i, int u) {
        const uint32_t e = SHARED ? 0 : at(i, u) & 1, q0 = dQ + (SHARED ? i * (C::kQTile / 16) : 0);
        const uint32_t k0 = dK + kp.st * (C::kStage / 16), d = tmem + kColS + 128 * i + kStep * e;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_lo(d, q0 + c * 1024 + ks * 2, k0 + c * (kStep * 8) + ks * 2, hi, idesc_qk, (c | ks) ? 1u : 0u);
        umma_commit(&s_full[2 * i + e]);
      };
      // P of half i's step u; SHARED: 64 keys of it, part e
      auto look_p = [&](int i, int u, int e) -> bool {
        return SHARED ? mbar_test_wait(&p_full[2 * i + e], at(i, u) & 1)
                      : mbar_test_wait(&p_full[2 * i + (at(i, u) & 1)], (at(i, u) >> 1) & 1);
      };
      auto take_p = [&](int i, int u, int e, bool seen) -> bool {
        if (!seen && !wait(&p_full[2 * i + (SHARED ? e : at(i, u) & 1)], (SHARED ? at(i, u) : at(i, u) >> 1) & 1, a.status,
                           abort_flag))
          return false;
        tc_fence_after();
        return true;
      };
      // the product of 64 keys of P (part e of a tile of 128)
      auto pv = [&](int i, int u, int e) {
        const uint32_t v0 = dV + vp.st * (C::kStage / 16) + e * 512;
        const uint32_t p0 = tmem + kColS + 128 * i + (SHARED ? 32 * e : kStep * (at(i, u) & 1));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_f16_ts_lo(tmem + kColO + D * i, p0 + ks * 8, v0 + ks * 128, hi, idesc_pv, (u | e | ks) ? 1u : 0u);
      };
      for (Work k = *work_s; ok && k.n > 0; next_work<kTile, BN>(a, k), ++seg) {
        const Piece p = piece_of(k);
        const int n0 = p.n0, n1 = p.n1, n = max(n0, n1);
        ok = wait(q_full, seg & 1, a.status, abort_flag);
        if constexpr (SHARED) {
          if (ok && n > 0) {
            ok = take(kp);
            if (ok && n0 > 0) qk(0, 0);
            if (ok && n1 > 0) qk(1, 0);
            if (ok) release(kp);
          }
          for (int u = 0; ok && u < n; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int ni = i ? n1 : n0, other = i ? n0 : n1;
              if (!ok || u >= ni) continue;
              bool seen = look_p(i, u, 0);
              ok = take(vp);
              if (u + 1 < ni && !kp.seen) look(kp);
              ok = ok && take_p(i, u, 0, seen);
              if (!ok) break;
              seen = look_p(i, u, 1);
              pv(i, u, 0);
              ok = take_p(i, u, 1, seen);
              if (!ok) break;
              pv(i, u, 1);
              if (i == 1 || u >= other) release(vp);
              if (u + 1 == ni) {
                umma_commit(&o_full[i]);
              } else {
                ok = take(kp);
                if (!ok) break;
                qk(i, u + 1);
                if (i == 1 || u + 1 >= other) release(kp);
              }
            }
          }
        } else {
          // step u's scores of both halves
          auto scores = [&](int u) -> bool {
            if (u >= n) return true;
            if (!take(kp)) return false;                     // (n0 = n1 or n1 + 1)
            qk(0, u);
            release(kp);
            if (u < n1) {
              if (!take(kp)) return false;
              qk(1, u);
              release(kp);
            }
            return true;
          };
          auto product = [&](int i, int u, int ni, bool seen) -> bool {
            if (!take(vp) || !take_p(i, u, 0, seen)) return false;
            pv(i, u, 0);
            umma_commit(&pv_done[i]);
            release(vp);
            if (u + 1 == ni) umma_commit(&o_full[i]);
            return true;
          };
          ok = ok && scores(0);
          for (int u = 0; ok && u < n; ++u) {
            look(vp);
            ok = scores(u + 1);
            if (!ok) break;
            const bool p0 = look_p(0, u, 0);
            look(kp);
            ok = product(0, u, n0, p0);
            if (ok && u < n1) ok = product(1, u, n1, false);
          }
        }
        // a half without steps waits here too: it must not load the next piece's q before the other has loaded this one's
        if (ok && n0 == 0) umma_commit(&o_full[0]);
        if (ok && n1 == 0) umma_commit(&o_full[1]);
        at0 += n0;
        at1 += n1;
      }
    }
    __syncwarp();
  }
  } else {
    // ----------------------------------------------------------- softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = warp >> 2;
    const int rt = tid & 127;                   // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + kColS + 128 * half + lane_base, tO = tmem + kColO + D * half + lane_base;
    const float c = a.scale_log2;
    uint32_t seq0 = 0, done = 0, outs = 0;      // ring places, steps and pieces of this half so far
    uint32_t mg = 0;                            // merge buffer uses so far
    // the warp's place in the list is kept in shared memory between pieces
    Work* my_work = work_s + 1 + warp;
    if (lane == 0) *my_work = *work_s;
    __syncwarp();
    while (ok && my_work->n > 0) {
    int b, g, rows, len, rbase, n_steps, n_places, blk0, bound;
    {
      const Work k = *my_work;
      const Piece p = piece_of(k);
      b = p.b;
      g = p.g;
      rows = p.rows;
      len = p.len;
      rbase = p.row0 + (SHARED ? 128 * half : 0);
      n_steps = half ? p.n1 : p.n0;
      n_places = 2 * n_tiles_of(p);
      blk0 = k.blk0;
      // keys this row sees; rows that do not exist see all, so that they make no block a masked one
      bound = rbase + rt < rows ? max(0, min(len, p.first_pos + (rbase + rt) / a.G + 1)) : len;
    }
    const int r = rbase + rt;
    {
      // q rows into the swizzled tiles (16-byte units, 8 to a 128-byte row)
      const int qt = SHARED ? half : 0;
      constexpr int U = D / 8;
      uint8_t* dst = sQ + qt * C::kQTile;
      const int wq = warp & 3;
      if (SHARED || half == 0) {
#pragma unroll 4
        for (int i = lane; i < 32 * U; i += 32) {
          const int rr = wq * 32 + i / U, u = i % U;
          const int gr = rbase + rr;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (gr < rows) {
            const int t = gr / a.G, h = g * a.G + gr - t * a.G;
            v = __ldg(reinterpret_cast<const uint4*>(a.q + ((static_cast<long long>(b) * a.T + t) * a.Hq + h) * D) + u);
          }
          *reinterpret_cast<uint4*>(dst + (u >> 3) * 16384 + rr * 128 + (((u & 7) ^ (rr & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(q_full);
    }
    const bool idle = rbase + (warp & 3) * 32 >= rows;   // no row of this warp exists: its P and O are never used
    // nothing past the sequence's end may reach the product: the V rows there are cleared
    auto clear_tail = [&](uint32_t seq_v, int key0) {
      if (key0 + kStep <= len) return;
      uint8_t* vt = sStage + (seq_v % C::kStages) * C::kStage;
      const int z0 = max(0, len - key0);
#pragma unroll 1
      for (int i = rt; i < (kStep - z0) * C::kChunks * 8; i += 128) {
        const int row = z0 + i / (C::kChunks * 8), u = i % (C::kChunks * 8);
        *reinterpret_cast<uint4*>(vt + (u >> 3) * (kStep * 128) + row * 128 + (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
    };
    float m_run = -INFINITY, l_run = 0.f;       // log2 domain
#pragma unroll 1
    for (int u = 0; u < n_steps; ++u) {
      const uint32_t at = done + u, e = SHARED ? 0 : at & 1;
      const int tile = tile_of(half, u), key0 = blk0 * BN + tile * kStep;
      const uint32_t seq_v = seq0 + 2 * tile + 1;
      // the V tile's barrier also publishes the tile's mapped pages
      ok = __all_sync(0xffffffffu, wait(&s_full[2 * half + e], (SHARED ? at : at >> 1) & 1, a.status, abort_flag) &&
                                       wait(&kv_full[seq_v % C::kStages], (seq_v / C::kStages) & 1, a.status, abort_flag));
      if (!ok) break;
      clear_tail(seq_v, key0);
      if (idle) {
        mbar_arrive(&p_full[2 * half + e]);
        if (SHARED) mbar_arrive(&p_full[2 * half + 1]);
        continue;
      }
      tc_fence_after();
      const uint32_t tSe = tS + 64 * e;
      const uint32_t mapped = mask_s[seq_v % C::kStages];
      const int vis = bound - key0;               // visible keys of this step
      const bool masked = __any_sync(0xffffffffu, vis < kStep) || mapped != (1u << (kStep / 16)) - 1u;
      // scores [32 q, 32 q + 32) of the step
      auto mask = [&](uint32_t (&v)[32], int q) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * q + j >= vis || !((mapped >> (2 * q + (j >> 4))) & 1u)) v[j] = 0xFF800000u;
      };
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto largest = [&](const uint32_t (&v)[32]) {
#pragma unroll
        for (int j = 0; j < 32; j += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 4 + i]));
      };
      uint32_t v0[32], v1[32];                    // the step's first 64 scores
      tmem_ld32(tSe, v0);
      tmem_ld32(tSe + 32, v1);
      tmem_ld_wait();
      if (masked) {
        mask(v0, 0);
        mask(v1, 1);
      }
      uint32_t v2[32], v3[32];
      if constexpr (SHARED) {
        tmem_ld32(tSe + 64, v2);
        tmem_ld32(tSe + 96, v3);
      }
      largest(v0);
      largest(v1);
      if constexpr (SHARED) {
        tmem_ld_wait();
        if (masked) {
          mask(v2, 2);
          mask(v3, 3);
        }
        largest(v2);
        largest(v3);
      }
      const float mb = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
      const bool move = mb > m_run + 8.f || (m_run == -INFINITY && mb != -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        float corr = 1.f;
        if (move) {
          corr = m_run == -INFINITY ? 0.f : ex2(m_run - mb);
          l_run *= corr;
          m_run = mb;
        }
        if (u > 0) {
          // SHARED: the last product was issued before these scores, and has completed with them. Else only the last
          // step's can be unfinished.
          if (!SHARED) {
            ok = __all_sync(0xffffffffu, wait(&pv_done[half], (at - 1) & 1, a.status, abort_flag));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t ov[16];
            tmem_ld16(tO + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * corr);
            tmem_st16(tO + c0, ov);
          }
        }
      }
      const float mu = m_run == -INFINITY ? 0.f : m_run;     // all masked so far: exp2(-inf) = 0
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 c2 = make_float2(c, c), mu2 = make_float2(-mu, -mu);
      auto part = [&](const uint32_t (&v)[32], int q) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float2 p = fma2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), c2, mu2);
          p.x = ex2(p.x);
          p.y = ex2(p.y);
          ps[j & 1] = add2(ps[j & 1], p);
          pk[j] = pack_bf16(p.x, p.y);
        }
        tmem_st16(tSe + 16 * q, pk);
      };
      part(v0, 0);
      part(v1, 1);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[2 * half + e]);
      if constexpr (SHARED) {
        part(v2, 2);
        part(v3, 3);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[2 * half + 1]);
      }
      l_run += (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
    }
    // ---------------------------------------------------------- epilogue --
    seq0 += n_places;
    done += n_steps;
    if (!ok) break;
    ok = __all_sync(0xffffffffu, wait(&o_full[half], outs & 1, a.status, abort_flag));
    ++outs;
    if (!ok) break;
    tc_fence_after();
    const bool mine = r < rows;
    const Work k = *my_work;
    float w_own = 1.f, w_other = 0.f;           // weights of the halves' outputs (SHARED = 0)
    const float* other = merge_s + rt * C::kMergeRow;
    if constexpr (!SHARED) {
      // half 1's maximum and sum, then its output 32 columns at a time, go to half 0
      if (half) {
        if (!wait(mg_empty, (mg & 1) ^ 1, a.status, abort_flag)) ok = false;
        float* to = merge_s + rt * C::kMergeRow;
        to[0] = m_run;
        to[1] = l_run;
        mbar_arrive(mg_full);
        ++mg;
        for (int c0 = 0; c0 < D; c0 += 32, ++mg) {
          uint32_t ov[32];
          if (!idle) {
            tmem_ld32(tO + c0, ov);
            tmem_ld_wait();
          }
          ok = __all_sync(0xffffffffu, ok && wait(mg_empty, (mg & 1) ^ 1, a.status, abort_flag));
          if (!ok) break;
          if (mine) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(to)[i] = l_run != 0.f ? make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3])
                                                            : make_uint4(0u, 0u, 0u, 0u);
          }
          mbar_arrive(mg_full);
        }
        if (!ok) break;
        Work next = k;
        next_work<kTile, BN>(a, next);
        if (lane == 0) *my_work = next;
        __syncwarp();
        continue;
      }
      ok = __all_sync(0xffffffffu, wait(mg_full, mg & 1, a.status, abort_flag));
      if (!ok) break;
      const float m1 = other[0], l1 = other[1];
      mbar_arrive(mg_empty);
      ++mg;
      const float mt = fmaxf(m_run, m1);
      if (mt != -INFINITY) {
        w_own = ex2(m_run - mt);
        w_other = ex2(m1 - mt);
      }
      l_run = l_run * w_own + l1 * w_other;
      m_run = mt;
    }
    const int t_row = r / a.G;
    const long long orow = (static_cast<long long>(b) * a.T + t_row) * a.Hq + g * a.G + (r - t_row * a.G);
    const bool whole = k.n == k.all;
    const int slot = 2 * worker + (k.blk0 == 0);
    const int prow = slot * kTile + (SHARED ? 128 * half : 0) + rt;
    const float inv = l_run != 0.f ? 1.f / l_run : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t ov[32];
      if (!idle) {
        tmem_ld32(tO + c0, ov);
        tmem_ld_wait();
      }
      // a row without keys is 0, whatever its accumulator holds
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if constexpr (!SHARED) ov[i] = w_own > 0.f ? __float_as_uint(__uint_as_float(ov[i]) * w_own) : 0u;
        ov[i] = n_steps > 0 && l_run != 0.f ? __float_as_uint(__uint_as_float(ov[i]) * inv) : 0u;
      }
      if constexpr (!SHARED) {
        ok = __all_sync(0xffffffffu, wait(mg_full, mg & 1, a.status, abort_flag));
        if (!ok) break;
        if (mine && l_run != 0.f) {
          const float w = w_other * inv;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = reinterpret_cast<const float4*>(other)[i];
            ov[4 * i] = __float_as_uint(fmaf(o.x, w, __uint_as_float(ov[4 * i])));
            ov[4 * i + 1] = __float_as_uint(fmaf(o.y, w, __uint_as_float(ov[4 * i + 1])));
            ov[4 * i + 2] = __float_as_uint(fmaf(o.z, w, __uint_as_float(ov[4 * i + 2])));
            ov[4 * i + 3] = __float_as_uint(fmaf(o.w, w, __uint_as_float(ov[4 * i + 3])));
          }
        }
        mbar_arrive(mg_empty);
        ++mg;
      }
      if (!mine) continue;
      if (whole) {
        uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16(__uint_as_float(ov[8 * q + 2 * e]), __uint_as_float(ov[8 * q + 2 * e + 1]));
          dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        uint4* dst = reinterpret_cast<uint4*>(a.part_o + static_cast<long long>(prow) * D + c0);
#pragma unroll
        for (int q = 0; q < 8; ++q) dst[q] = make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
      }
    }
    if (!ok) break;
    if (mine) {
      if (whole) {
        if (a.lse) a.lse[orow] = l_run != 0.f ? (m_run + log2f(l_run)) * 0.69314718055994530942f : -INFINITY;
      } else {
        a.part_m[prow] = m_run;
        a.part_l[prow] = l_run;
      }
    }
    if (tid == 0 && k.blk0 == 0) a.span[static_cast<long long>(k.g) * a.B * a.tiles + k.bt] = make_longlong2(k.begin, k.all);
    Work next = k;
    next_work<kTile, BN>(a, next);
    if (lane == 0) *my_work = next;
    __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) spin_ns(50000);   // let copies and MMAs in flight land before the exit
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool SHARED>
cudaError_t launch_t(const PagedMaps& m, const PagedArgs& a, cudaStream_t stream) {
  using C = Cfg<D, SHARED>;
  const void* fn = reinterpret_cast<const void*>(&paged_attn_kernel<D, SHARED>);
  // at least half an SM's shared memory: one block per SM, as its tensor memory asks for
  const size_t smem = C::kSmem < 120 * 1024 ? 120 * 1024 : C::kSmem;
  const cudaError_t e = set_max_smem(fn, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<CUtensorMap*>(&m.k), const_cast<CUtensorMap*>(&m.v), const_cast<PagedArgs*>(&a)};
  return launch_pdl(fn, dim3(a.workers), dim3(kThreads), smem, stream, args);
}

// Merges the pieces of the rows of cut tiles: f_p = l_p 2^(m_p - m*), o = sum
// f_p o_p / sum f_p, lse = m* + log2 sum f_p. DV / 128 (at least 1) warps a row;
// empty pieces are not read.
template <int DV>
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = DV >= 128 ? DV / 128 : 1;      // warps of a row
  constexpr int kPer = DV >= 128 ? 4 : DV / 32;         // columns of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n_rows = static_cast<long long>(a.B) * a.T * a.Hq;
  const long long row = static_cast<long long>(blockIdx.x) * (4 / kWarps) + warp / kWarps;
  if (row >= n_rows) return;
  const int bt = static_cast<int>(row / a.Hq), b = bt / a.T, t = bt - b * a.T;
  if (t >= lens_of(a, b).n_new) return;                 // a padding row: left as it was
  const int head = static_cast<int>(row - static_cast<long long>(bt) * a.Hq), g = head / a.G;
  const int r = t * a.G + head - g * a.G;               // row of the KV head
  const int tile = r / a.tile_rows, in_tile = r - tile * a.tile_rows;
  const longlong2 span = a.span[(static_cast<long long>(g) * a.B + b) * a.tiles + tile];
  const long long total = a.head[0], used = a.head[1];
  // (a kernel that gave up waiting leaves spans unwritten: nothing is read by them)
  if (used < 1 || used > a.workers || span.x < 0 || span.y < 1 || span.y > total || span.x > total - span.y) return;
  const int w0 = worker_of(span.x, total, used), n_part = worker_of(span.x + span.y - 1, total, used) - w0 + 1;
  if (n_part == 1) return;                              // written by its worker
  // row of piece p among the slots
  auto at = [&](int p) -> long long { return static_cast<long long>(p == 0 ? 2 * w0 + 1 : 2 * (w0 + p)) * a.tile_rows + in_tile; };
  constexpr int kRegs = kMaxWorkers / 32;
  float f[kRegs], M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int p = i * 32 + lane;
    f[i] = 0.f;
    if (p < n_part) {
      f[i] = a.part_l[at(p)];
      if (f[i] != 0.f) M = fmaxf(M, a.part_m[at(p)]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float den = 0.f;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int p = i * 32 + lane;
    if (f[i] != 0.f) f[i] *= exp2f(a.part_m[at(p)] - M);
    den += f[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const int col = (warp % kWarps) * 128 + lane * kPer;
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  struct alignas(4 * kPer) Vec { float v[kPer]; };
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    if (i * 32 >= n_part) break;
    const int np = min(32, n_part - i * 32);
#pragma unroll 8
    for (int p = 0; p < np; ++p) {
      const float w = __shfl_sync(0xffffffffu, f[i], p);
      if (w != 0.f) {
        const Vec o = *reinterpret_cast<const Vec*>(a.part_o + at(i * 32 + p) * DV + col);
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(o.v[e], w, acc[e]);
      }
    }
  }
  uint16_t* dst = a.out + row * DV + col;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (a.lse && lane == 0 && warp % kWarps == 0)
    a.lse[row] = den != 0.f ? (M + log2f(den)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attn(const PagedMaps& m, const PagedArgs& a, int d, int shared_kv, cudaStream_t stream) {
  if (d == 128) return shared_kv ? launch_t<128, true>(m, a, stream) : launch_t<128, false>(m, a, stream);
  return shared_kv ? launch_t<64, true>(m, a, stream) : launch_t<64, false>(m, a, stream);
}

cudaError_t launch_paged_combine(const PagedArgs& a, int d_v, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.T * a.Hq;
  const int per = d_v == 512 ? 1 : 4;
  const void* fn = d_v == 512   ? reinterpret_cast<const void*>(&paged_combine_kernel<512>)
                   : d_v == 128 ? reinterpret_cast<const void*>(&paged_combine_kernel<128>)
                                : reinterpret_cast<const void*>(&paged_combine_kernel<64>);
  void* args[] = {const_cast<PagedArgs*>(&a)};
  return launch_pdl(fn, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(128), 0, stream, args);
}

}  // namespace lsa
