// C ABI of the paged cache (declarations and contracts in include/lsa.h):
// argument validation, launch plans and tensor maps of the rotary, append,
// paged-attention and page-upkeep calls. Host side only.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "internal.h"
#include "lsa.h"

namespace lsa {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

lsa_status_t cuda_check(cudaError_t e, const char* what) {
  return e == cudaSuccess ? LSA_OK : set_error(LSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

lsa_status_t check_pages(int n_pages, int page_size) {
  if (!page_size_ok(page_size))
    return set_error(LSA_ERR_UNSUPPORTED, "page size %d not in {16,32,64,128}", page_size);
  if (n_pages < 1) return set_error(LSA_ERR_INVALID_ARG, "n_pages must be >= 1");
  if (n_pages > LSA_MAX_PAGES) return set_error(LSA_ERR_UNSUPPORTED, "n_pages=%d above %d", n_pages, LSA_MAX_PAGES);
  return LSA_OK;
}

// A table of S rows of max_pages entries, addressed in tokens with 32 bits.
lsa_status_t check_table(int S, int max_pages, int page_size) {
  if (S < 1 || max_pages < 1) return set_error(LSA_ERR_INVALID_ARG, "the table needs at least one row and one entry");
  if (static_cast<long long>(max_pages) * page_size >= (1ll << 30))
    return set_error(LSA_ERR_UNSUPPORTED, "a table row of %d pages holds 2^30 tokens or more", max_pages);
  return LSA_OK;
}

lsa_status_t check_plan(const lsa_rope_plan_t* p, int d, int offset) {
  if (p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > 2 * LSA_ROPE_MAX_PAIRS)
    return set_error(LSA_ERR_INVALID_ARG, "rot_dim=%d: fill the plan with lsa_rope_plan", p->rot_dim);
  if (offset < 0 || offset > d - p->rot_dim)
    return set_error(LSA_ERR_INVALID_ARG, "columns [%d, %d + %d) do not lie in the %d of a head", offset, offset,
                     p->rot_dim, d);
  return LSA_OK;
}

void put_plan(RotateArgs* a, const lsa_rope_plan_t* p) {
  a->rot = p->rot_dim;
  a->interleaved = p->interleaved != 0;
  a->amplitude = static_cast<float>(p->amplitude);
  for (int i = 0; i < LSA_ROPE_MAX_PAIRS; ++i) a->freq[i] = p->freq[i] / 6.283185307179586477;   // turns per position
}

// ------------------------------------------------------------ tensor maps --
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Pages as (columns, slot, page). bf16: boxes of 64 columns x box_rows x 1, swizzled as the MMA reads them; e4m3 codes:
// boxes of 128 columns, plain.
lsa_status_t page_map(CUtensorMap* m, const void* base, bool e4m3, int cols, int page_size, int n_pages, int64_t row_stride,
                      int64_t page_stride, int box_rows) {
  auto fn = encoder();
  if (!fn) return set_error(LSA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int es = e4m3 ? 1 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(page_size),
                        static_cast<cuuint64_t>(n_pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride) * es, static_cast<cuuint64_t>(page_stride) * es};
  cuuint32_t box[3] = {e4m3 ? 128u : 64u, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                        dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(LSA_ERR_CUDA, "cuTensorMapEncodeTiled (pages) failed (%d)", static_cast<int>(r));
  return LSA_OK;
}

// q [rows, 576] bf16, boxes of 64 columns x 64 rows.
lsa_status_t query_map(CUtensorMap* m, const void* base, uint64_t rows) {
  auto fn = encoder();
  if (!fn) return set_error(LSA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {576, rows}, strides[1] = {576 * 2};
  cuuint32_t box[2] = {64, 64}, estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(LSA_ERR_CUDA, "cuTensorMapEncodeTiled (q) failed (%d)", static_cast<int>(r));
  return LSA_OK;
}

// --------------------------------------------------------- paged attention --
bool is_mla(const lsa_paged_attn_in_t* in) { return in->d_qk == 576; }

lsa_status_t check_paged(const lsa_paged_attn_in_t* in) {
  if (!in) return set_error(LSA_ERR_INVALID_ARG, "null paged attention descriptor");
  lsa_status_t s;
  if ((s = check_pages(in->n_pages, in->page_size)) != LSA_OK) return s;
  if (in->B < 1 || in->T < 1) return set_error(LSA_ERR_INVALID_ARG, "B and T must be >= 1");
  if ((s = check_table(in->B, in->max_pages, in->page_size)) != LSA_OK) return s;
  const bool mla = in->d_qk == 576 && in->d_v == 512;
  const bool gqa = (in->d_qk == 64 && in->d_v == 64) || (in->d_qk == 128 && in->d_v == 128);
  if (!mla && !gqa) return set_error(LSA_ERR_UNSUPPORTED, "(d_qk, d_v) = (%d, %d) unsupported", in->d_qk, in->d_v);
  if (in->Hq < 1 || in->Hkv < 1 || in->Hq % in->Hkv)
    return set_error(LSA_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d", in->Hq, in->Hkv);
  if (mla && (in->Hkv != 1 || in->Hq > 128))
    return set_error(LSA_ERR_UNSUPPORTED, "latent rows take Hkv = 1 and Hq <= 128 (got %d, %d)", in->Hkv, in->Hq);
  if (in->Hkv > 65535 || in->B > 65535) return set_error(LSA_ERR_UNSUPPORTED, "B or Hkv above 65535");
  if (static_cast<long long>(in->B) * in->T * in->Hq >= (1ll << 30))
    return set_error(LSA_ERR_UNSUPPORTED, "too many query rows");
  if (!in->seq_len || !in->table || !in->q || !in->k || !in->v)
    return set_error(LSA_ERR_INVALID_ARG, "null paged attention tensor");
  if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(in->table, 4))
    return set_error(LSA_ERR_INVALID_ARG, "paged attention tensors must be 16-byte aligned");
  if (mla && (in->v != in->k || in->v_page_stride != in->k_page_stride || in->v_row_stride != in->k_row_stride))
    return set_error(LSA_ERR_UNSUPPORTED, "d_qk=576 / d_v=512 takes v = k (latent rows)");
  if (in->kv_dtype != LSA_BF16 && in->kv_dtype != LSA_E4M3)
    return set_error(LSA_ERR_INVALID_ARG, "kv_dtype %d is neither LSA_BF16 nor LSA_E4M3", in->kv_dtype);
  const bool e4m3 = in->kv_dtype == LSA_E4M3;
  if (e4m3 && !mla) return set_error(LSA_ERR_UNSUPPORTED, "an e4m3 cache needs latent rows (d_qk=576, d_v=512)");
  if (e4m3 && (!in->k_scale || !aligned(in->k_scale, 4)))
    return set_error(LSA_ERR_INVALID_ARG, "an e4m3 cache needs k_scale (fp32)");
  if (!e4m3 && in->k_scale) return set_error(LSA_ERR_INVALID_ARG, "k_scale is for an e4m3 cache only");
  const int64_t unit = e4m3 ? 16 : 8;   // 16 bytes
  auto stride_ok = [&](int64_t row, int64_t page, int64_t width) {
    return row >= width && row % unit == 0 && page > 0 && page % unit == 0 && row < (1ll << 31) && page < (1ll << 38);
  };
  if (!stride_ok(in->k_row_stride, in->k_page_stride, static_cast<int64_t>(in->Hkv) * in->d_qk) ||
      !stride_ok(in->v_row_stride, in->v_page_stride, static_cast<int64_t>(in->Hkv) * in->d_v))
    return set_error(LSA_ERR_INVALID_ARG, "row strides must cover the row; strides are multiples of 16 bytes");
  if (!(in->scale > 0.f) || !std::isfinite(in->scale))
    return set_error(LSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  return LSA_OK;
}

struct PagedPlan {
  int shared_kv, tile_rows, tiles, workers;
};

// Latent rows: tiles of 128 rows, a worker is a pair of SMs. Else tiles of 256
// rows (two halves over the same keys) where a KV head has more than 128, and
// one tile (two halves over alternate keys) where it has fewer; a worker is an
// SM.
PagedPlan paged_plan(const lsa_paged_attn_in_t* in) {
  PagedPlan p{};
  const bool mla = is_mla(in);
  const long long rows = static_cast<long long>(in->T) * (in->Hq / in->Hkv);
  p.shared_kv = !mla && rows > 128;
  p.tile_rows = p.shared_kv ? 256 : 128;
  p.tiles = static_cast<int>((rows + p.tile_rows - 1) / p.tile_rows);
  const int sms = device_sm_count();
  const long long blocks = (static_cast<long long>(in->max_pages) * in->page_size + kPagedBN - 1) / kPagedBN;
  const long long most = static_cast<long long>(in->B) * in->Hkv * p.tiles * blocks;
  p.workers = static_cast<int>(std::min({static_cast<long long>(mla ? sms / 2 : sms), most, static_cast<long long>(kMaxWorkers)}));
  return p;
}

struct PagedLayout {
  size_t span, o, m, l, total;
};
PagedLayout paged_ws(const lsa_paged_attn_in_t* in, const PagedPlan& p) {
  PagedLayout w;
  const size_t rows = 2 * static_cast<size_t>(p.workers) * p.tile_rows;
  w.span = 256;
  w.o = w.span + up256(static_cast<size_t>(in->Hkv) * in->B * p.tiles * sizeof(longlong2));
  w.m = w.o + up256(rows * in->d_v * 4);
  w.l = w.m + up256(rows * 4);
  w.total = w.l + up256(rows * 4);
  return w;
}

lsa_status_t check_pools(const lsa_pool_t* pools, int n_pools) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return set_error(LSA_ERR_INVALID_ARG, "null pools");
  for (int i = 0; i < n_pools; ++i) {
    const lsa_pool_t& p = pools[i];
    if (!p.base || !aligned(p.base, 16)) return set_error(LSA_ERR_INVALID_ARG, "pool %d null or not 16-byte aligned", i);
    if (p.page_bytes < 16 || p.page_bytes % 16 || p.page_stride % 16 || p.page_stride < p.page_bytes)
      return set_error(LSA_ERR_INVALID_ARG, "pool %d: page bytes and stride must be multiples of 16, stride >= bytes", i);
    if (p.page_bytes > (64ll << 20)) return set_error(LSA_ERR_UNSUPPORTED, "pool %d: a page above 64 MB", i);
  }
  return LSA_OK;
}

// Pools [first, first + kMaxLaunchPools) as a launch takes them, at most
// kMaxPieces pieces of a page in all (a grid dimension).
constexpr int kMaxPieces = 60000;
Pools take_pools(const lsa_pool_t* pools, int n_pools, int* first) {
  Pools out{};
  while (*first < n_pools && out.n < kMaxLaunchPools) {
    const lsa_pool_t& p = pools[*first];
    const int pieces = static_cast<int>((p.page_bytes + kCopyChunk - 1) / kCopyChunk);
    if (out.n > 0 && out.first[out.n] + pieces > kMaxPieces) break;
    out.base[out.n] = static_cast<uint8_t*>(p.base);
    out.stride[out.n] = p.page_stride;
    out.bytes[out.n] = static_cast<int>(p.page_bytes);
    out.first[out.n + 1] = out.first[out.n] + pieces;
    ++out.n;
    ++*first;
  }
  return out;
}

lsa_status_t check_cache(const void* table, const void* ref, int S, int max_pages, int n_pages) {
  if (!table || !ref) return set_error(LSA_ERR_INVALID_ARG, "null table or ref");
  if (!aligned(table, 4) || !aligned(ref, 16))
    return set_error(LSA_ERR_INVALID_ARG, "ref must be 16-byte aligned");
  if (S > LSA_MAX_SEQS) return set_error(LSA_ERR_UNSUPPORTED, "S=%d above %d sequences", S, LSA_MAX_SEQS);
  const lsa_status_t s = check_table(S, max_pages, 1);
  if (s != LSA_OK) return s;
  if (max_pages > LSA_MAX_PAGES)
    return set_error(LSA_ERR_UNSUPPORTED, "max_pages=%d above %d", max_pages, LSA_MAX_PAGES);
  return check_pages(n_pages, 16);
}

lsa_status_t check_space(void* ws, size_t have, size_t need) {
  if (have < need) return set_error(LSA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", have, need);
  if (need > 0 && (!ws || !aligned(ws, 256)))
    return set_error(LSA_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  return LSA_OK;
}

size_t fork_ws(int n) { return up256(static_cast<size_t>(n) * 8); }
size_t copy_ws(int n) { return n > kCopyNoPlan ? up256(static_cast<size_t>(n) * 4) : 0; }
size_t compact_ws(int n_pages) { return up256((kCompactHeader + 3 * static_cast<size_t>(n_pages)) * 4); }

}  // namespace

lsa_status_t paged_attn_workspace(const lsa_paged_attn_in_t* in, size_t* bytes) {
  const lsa_status_t s = check_paged(in);
  if (s != LSA_OK) return s;
  *bytes = paged_ws(in, paged_plan(in)).total;
  return LSA_OK;
}

lsa_status_t pages_workspace(lsa_op_t op, int n, int n_pages, size_t* bytes) {
  if (op == LSA_OP_PAGES_COMPACT) {
    const lsa_status_t s = check_pages(n_pages, 16);
    if (s != LSA_OK) return s;
    *bytes = compact_ws(n_pages);
    return LSA_OK;
  }
  if (n < 0) return set_error(LSA_ERR_INVALID_ARG, "n must be >= 0");
  *bytes = op == LSA_OP_PAGES_FORK ? fork_ws(n) : copy_ws(n);
  return LSA_OK;
}

}  // namespace lsa

using namespace lsa;

extern "C" {

lsa_status_t lsa_rope_plan(int32_t rot_dim, int32_t interleaved, double theta, lsa_rope_scaling_t scaling,
                           double factor, int32_t orig_len, double beta_fast, double beta_slow, double amplitude,
                           lsa_rope_plan_t* plan) {
  if (!plan) return set_error(LSA_ERR_INVALID_ARG, "null plan");
  if (rot_dim < 2 || rot_dim % 2) return set_error(LSA_ERR_INVALID_ARG, "rot_dim=%d must be even and >= 2", rot_dim);
  if (rot_dim > 2 * LSA_ROPE_MAX_PAIRS)
    return set_error(LSA_ERR_UNSUPPORTED, "rot_dim=%d above %d", rot_dim, 2 * LSA_ROPE_MAX_PAIRS);
  if (!(theta > 1.0) || !std::isfinite(theta)) return set_error(LSA_ERR_INVALID_ARG, "theta must be finite and > 1");
  if (scaling != LSA_ROPE_PLAIN && scaling != LSA_ROPE_LINEAR && scaling != LSA_ROPE_YARN)
    return set_error(LSA_ERR_INVALID_ARG, "unknown scaling %d", static_cast<int>(scaling));
  if (scaling != LSA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return set_error(LSA_ERR_INVALID_ARG, "factor must be finite and > 0");
  if (!(amplitude >= 0.0) || !std::isfinite(amplitude))
    return set_error(LSA_ERR_INVALID_ARG, "amplitude must be finite and >= 0");
  double low = 0.0, high = 0.0;
  if (scaling == LSA_ROPE_YARN) {
    if (orig_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
      return set_error(LSA_ERR_INVALID_ARG, "yarn needs orig_len >= 1 and beta_fast > beta_slow > 0");
    // the (fractional) pair that turns `turns` times in orig_len positions
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(orig_len / (turns * 6.283185307179586477)) / (2.0 * std::log(theta));
    };
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
  }
  plan->rot_dim = rot_dim;
  plan->interleaved = interleaved != 0;
  plan->amplitude = amplitude > 0.0 ? amplitude
                    : scaling == LSA_ROPE_YARN && factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
  for (int i = 0; i < LSA_ROPE_MAX_PAIRS; ++i) {
    double f = 0.0;
    if (i < rot_dim / 2) {
      f = std::pow(theta, -2.0 * i / rot_dim);
      if (scaling == LSA_ROPE_LINEAR) f /= factor;
      if (scaling == LSA_ROPE_YARN) {
        const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
        f = f * (1.0 - ramp) + f / factor * ramp;
      }
    }
    plan->freq[i] = f;
  }
  return LSA_OK;
}

lsa_status_t lsa_rope(const lsa_rope_in_t* in, const lsa_rope_plan_t* plan, void* out, lsa_stream_t stream) {
  if (!in || !plan) return set_error(LSA_ERR_INVALID_ARG, "null rope descriptor or plan");
  if (in->B < 1 || in->T < 1 || in->H < 1 || in->d < 1) return set_error(LSA_ERR_INVALID_ARG, "B, T, H and d must be >= 1");
  if (in->dtype != LSA_BF16 && in->dtype != LSA_FP32)
    return set_error(LSA_ERR_INVALID_ARG, "dtype %d is neither LSA_BF16 nor LSA_FP32", in->dtype);
  if (!in->x || !in->seq_len || !out) return set_error(LSA_ERR_INVALID_ARG, "null rope tensor");
  lsa_status_t s = check_plan(plan, in->d, in->offset);
  if (s != LSA_OK) return s;
  if (in->d > 65536) return set_error(LSA_ERR_UNSUPPORTED, "d=%d above 65536", in->d);
  if (static_cast<long long>(in->B) * in->T >= (1ll << 30) || in->H > (1 << 20))
    return set_error(LSA_ERR_UNSUPPORTED, "too many rows");
  const int es = in->dtype == LSA_BF16 ? 2 : 4;
  if (!aligned(in->x, es) || !aligned(out, es)) return set_error(LSA_ERR_INVALID_ARG, "rope tensors must be element-aligned");
  RotateArgs a{};
  a.B = in->B; a.T = in->T; a.H = in->H; a.d = in->d; a.offset = in->offset;
  put_plan(&a, plan);
  a.sign = in->inverse ? -1.f : 1.f;
  a.seq_len = in->seq_len; a.q_len = in->q_len;
  a.x = in->x; a.out = out;
  a.xb = in->x_stride_b; a.xt = in->x_stride_t; a.xh = in->x_stride_h;
  a.ob = in->out_stride_b; a.ot = in->out_stride_t; a.oh = in->out_stride_h;
  a.in_place = in->x == out;
  if ((in->B > 1 && a.ob == 0) || (in->T > 1 && a.ot == 0) || (in->H > 1 && a.oh == 0))
    return set_error(LSA_ERR_INVALID_ARG, "out must have a row of its own for every (b, t, h)");
  if (a.in_place && (a.xb != a.ob || a.xt != a.ot || a.xh != a.oh))
    return set_error(LSA_ERR_INVALID_ARG, "an in-place rotation needs the same strides on both sides");
  // 16-byte accesses where every row, the rotated part and (half layout) its
  // halves start on 16 bytes; else element by element
  const int v = 16 / es;
  const int part = a.interleaved ? a.rot : a.rot / 2;
  auto whole = [&](long long x) { return x % v == 0; };
  const bool wide = aligned(in->x, 16) && aligned(out, 16) && whole(in->d) && whole(in->offset) && whole(part) &&
                    whole(a.rot) && whole(a.xb) && whole(a.xt) && whole(a.xh) && whole(a.ob) && whole(a.ot) && whole(a.oh);
  a.vec = wide ? v : 1;
  a.status = device_status_ptr();
  return cuda_check(launch_rope(a, in->dtype == LSA_FP32, reinterpret_cast<cudaStream_t>(stream)), "rope launch");
}

lsa_status_t lsa_pages_append(const lsa_append_in_t* in, const lsa_rope_plan_t* plan, lsa_stream_t stream) {
  if (!in) return set_error(LSA_ERR_INVALID_ARG, "null append descriptor");
  lsa_status_t s;
  if ((s = check_pages(in->n_pages, in->page_size)) != LSA_OK) return s;
  if (in->B < 1 || in->T < 1 || in->H < 1 || in->d < 1) return set_error(LSA_ERR_INVALID_ARG, "B, T, H and d must be >= 1");
  if ((s = check_table(in->B, in->max_pages, in->page_size)) != LSA_OK) return s;
  if (in->dtype != LSA_BF16 && in->dtype != LSA_E4M3)
    return set_error(LSA_ERR_INVALID_ARG, "dtype %d is neither LSA_BF16 nor LSA_E4M3", in->dtype);
  if (!in->x || !in->seq_len || !in->table || !in->pool) return set_error(LSA_ERR_INVALID_ARG, "null append tensor");
  if (!aligned(in->x, 16) || !aligned(in->pool, 16))
    return set_error(LSA_ERR_INVALID_ARG, "rows and pool must be 16-byte aligned");
  if (in->d % 8 || in->d > 65536) return set_error(LSA_ERR_UNSUPPORTED, "d=%d must be a multiple of 8, at most 65536", in->d);
  const long long width = static_cast<long long>(in->H) * in->d;
  if (static_cast<long long>(in->B) * in->T >= (1ll << 30) || width >= (1ll << 20))
    return set_error(LSA_ERR_UNSUPPORTED, "too many rows, or rows of 2^20 columns or more");
  const bool e4m3 = in->dtype == LSA_E4M3;
  if (e4m3) {
    if (width > 1024 || width % 16) return set_error(LSA_ERR_UNSUPPORTED, "an e4m3 row of %lld columns: a multiple of 16, at most 1024", width);
    if (!in->scales || !aligned(in->scales, 4)) return set_error(LSA_ERR_INVALID_ARG, "an e4m3 pool needs scales (fp32)");
  } else if (in->scales) {
    return set_error(LSA_ERR_INVALID_ARG, "scales are for an e4m3 pool only");
  }
  const int64_t unit = e4m3 ? 16 : 8;
  if (in->row_stride < width || in->row_stride % unit || in->page_stride < 1 || in->page_stride % unit)
    return set_error(LSA_ERR_INVALID_ARG, "the row stride must cover the row; strides are multiples of 16 bytes");
  RotateArgs a{};
  if (plan) {
    if ((s = check_plan(plan, in->d, in->offset)) != LSA_OK) return s;
    if (plan->rot_dim % 16 || in->offset % 8)
      return set_error(LSA_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 and offset=%d of 8", plan->rot_dim, in->offset);
    put_plan(&a, plan);
    a.offset = in->offset;
  }
  a.B = in->B; a.T = in->T; a.H = in->H; a.d = in->d;
  a.sign = 1.f;
  a.seq_len = in->seq_len; a.q_len = in->q_len;
  a.x = in->x; a.out = in->pool;
  a.xh = in->d; a.xt = width; a.xb = width * in->T;
  a.ob = in->page_stride; a.ot = in->row_stride; a.oh = in->d;
  a.table = in->table; a.n_pages = in->n_pages; a.page_size = in->page_size; a.max_pages = in->max_pages;
  a.scales = in->scales;
  a.vec = 8;
  a.status = device_status_ptr();
  return cuda_check(launch_append(a, e4m3, reinterpret_cast<cudaStream_t>(stream)), "append launch");
}

lsa_status_t lsa_paged_attn(const lsa_paged_attn_in_t* in, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_paged(in)) != LSA_OK) return s;
  if (!out) return set_error(LSA_ERR_INVALID_ARG, "null out");
  if (!aligned(out, 16) || (lse && !aligned(lse, 4)))
    return set_error(LSA_ERR_INVALID_ARG, "out must be 16-byte aligned");
  const PagedPlan p = paged_plan(in);
  const PagedLayout lay = paged_ws(in, p);
  if ((s = check_space(workspace, workspace_bytes, lay.total)) != LSA_OK) return s;
  PagedArgs a{};
  a.B = in->B; a.T = in->T; a.Hq = in->Hq; a.Hkv = in->Hkv; a.G = in->Hq / in->Hkv;
  a.n_pages = in->n_pages; a.max_pages = in->max_pages;
  while ((1 << a.page_shift) < in->page_size) ++a.page_shift;
  a.tiles = p.tiles; a.tile_rows = p.tile_rows; a.workers = p.workers;
  a.scale_log2 = in->scale * 1.4426950408889634f;
  a.seq_len = in->seq_len; a.q_len = in->q_len; a.table = in->table;
  a.q = static_cast<const uint16_t*>(in->q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = device_status_ptr();
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.head = reinterpret_cast<long long*>(w);
  a.span = reinterpret_cast<longlong2*>(w + lay.span);
  a.part_o = reinterpret_cast<float*>(w + lay.o);
  a.part_m = reinterpret_cast<float*>(w + lay.m);
  a.part_l = reinterpret_cast<float*>(w + lay.l);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PagedMaps m{};
  if (is_mla(in)) {
    const bool e4m3 = in->kv_dtype == LSA_E4M3;
    if (e4m3) a.k_scale = in->k_scale;
    if ((s = page_map(&m.k, in->k, e4m3, 576, in->page_size, in->n_pages, in->k_row_stride, in->k_page_stride,
                      std::min(in->page_size, kPagedBox))) != LSA_OK)
      return s;
    if ((s = query_map(&m.v, in->q, static_cast<uint64_t>(in->B) * in->T * in->Hq)) != LSA_OK) return s;
    s = cuda_check(launch_paged_mla(m, a, e4m3, st), "paged latent attention launch");
  } else {
    const int box = std::min(in->page_size, kPagedBox);
    if ((s = page_map(&m.k, in->k, false, in->Hkv * in->d_qk, in->page_size, in->n_pages, in->k_row_stride, in->k_page_stride,
                      box)) != LSA_OK)
      return s;
    if ((s = page_map(&m.v, in->v, false, in->Hkv * in->d_v, in->page_size, in->n_pages, in->v_row_stride, in->v_page_stride,
                      box)) != LSA_OK)
      return s;
    s = cuda_check(launch_paged_attn(m, a, in->d_qk, p.shared_kv, st), "paged attention launch");
  }
  if (s != LSA_OK) return s;
  return cuda_check(launch_paged_combine(a, in->d_v, st), "paged combine launch");
}

lsa_status_t lsa_pages_reserve(int32_t* table, int32_t* ref, const int32_t* len, int32_t S, int32_t max_pages,
                               int32_t n_pages, int32_t page_size, lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_cache(table, ref, S, max_pages, n_pages)) != LSA_OK) return s;
  if ((s = check_pages(n_pages, page_size)) != LSA_OK) return s;
  if (!len) return set_error(LSA_ERR_INVALID_ARG, "null len");
  const PageArgs a{table, ref, nullptr, S, max_pages, n_pages, page_size, device_status_ptr()};
  return cuda_check(launch_reserve(a, len, reinterpret_cast<cudaStream_t>(stream)), "reserve launch");
}

lsa_status_t lsa_pages_free(int32_t* table, int32_t* ref, int32_t* seq_len, int32_t S, int32_t max_pages,
                            int32_t n_pages, const int32_t* seqs, int32_t n, lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_cache(table, ref, S, max_pages, n_pages)) != LSA_OK) return s;
  if (!seq_len || n < 0 || (n > 0 && !seqs)) return set_error(LSA_ERR_INVALID_ARG, "null seq_len or seqs, or n < 0");
  if (n == 0) return LSA_OK;
  const PageArgs a{table, ref, seq_len, S, max_pages, n_pages, 1, device_status_ptr()};
  return cuda_check(launch_free(a, seqs, n, reinterpret_cast<cudaStream_t>(stream)), "free launch");
}

lsa_status_t lsa_pages_fork(int32_t* table, int32_t* ref, int32_t* seq_len, int32_t S, int32_t max_pages,
                            int32_t n_pages, int32_t page_size, const int32_t* parent, const int32_t* child, int32_t n,
                            const lsa_pool_t* pools, int32_t n_pools, void* workspace, size_t workspace_bytes,
                            lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_cache(table, ref, S, max_pages, n_pages)) != LSA_OK) return s;
  if ((s = check_pages(n_pages, page_size)) != LSA_OK) return s;
  if ((s = check_pools(pools, n_pools)) != LSA_OK) return s;
  if (!seq_len || n < 0 || (n > 0 && (!parent || !child)))
    return set_error(LSA_ERR_INVALID_ARG, "null seq_len, parent or child, or n < 0");
  if (n == 0) return LSA_OK;
  if ((s = check_space(workspace, workspace_bytes, fork_ws(n))) != LSA_OK) return s;
  const PageArgs a{table, ref, seq_len, S, max_pages, n_pages, page_size, device_status_ptr()};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* plan = static_cast<int*>(workspace);
  if ((s = cuda_check(launch_fork_plan(a, parent, child, n, plan, st), "fork plan launch")) != LSA_OK) return s;
  // the rows go last: the partly filled pages are found through the parents' lengths and rows either way
  int first = 0;
  do {
    const Pools p = take_pools(pools, n_pools, &first);
    if ((s = cuda_check(launch_fork(a, parent, child, n, plan, p, first >= n_pools, st), "fork launch")) != LSA_OK) return s;
  } while (first < n_pools);
  return LSA_OK;
}

lsa_status_t lsa_pages_copy(const lsa_pool_t* pools, int32_t n_pools, int32_t n_pages, const int32_t* src,
                            const int32_t* dst, int32_t n, void* workspace, size_t workspace_bytes,
                            lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_pages(n_pages, 16)) != LSA_OK) return s;
  if ((s = check_pools(pools, n_pools)) != LSA_OK) return s;
  if (n < 0 || (n > 0 && (!src || !dst))) return set_error(LSA_ERR_INVALID_ARG, "null src or dst, or n < 0");
  if (n == 0) return LSA_OK;
  if ((s = check_space(workspace, workspace_bytes, copy_ws(n))) != LSA_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // A block of the copy reads the whole list where there is no plan: 8 KB for 1024 pairs. With a plan 1025 pairs take
  // 2 us more than 1024 without, at 1, 5 and 15 pieces a page alike (12.3 and 10.2, 34.8 and 32.8, 79.9 and 77.8 us).
  int* ok = n > kCopyNoPlan ? static_cast<int*>(workspace) : nullptr;
  if (ok && (s = cuda_check(launch_copy_plan(n_pages, src, dst, n, ok, device_status_ptr(), st), "copy plan launch")) != LSA_OK)
    return s;
  for (int first = 0; first < n_pools;) {
    const Pools p = take_pools(pools, n_pools, &first);
    if ((s = cuda_check(launch_copy(p, src, dst, ok, n, n_pages, device_status_ptr(), st), "copy launch")) != LSA_OK) return s;
  }
  return LSA_OK;
}

lsa_status_t lsa_pages_compact(const int32_t* table, const int32_t* ref, int32_t S, int32_t max_pages, int32_t n_pages,
                               const lsa_pool_t* pools, int32_t n_pools, int32_t* table_out, int32_t* ref_out,
                               int32_t* n_live, void* workspace, size_t workspace_bytes, lsa_stream_t stream) {
  lsa_status_t s;
  if ((s = check_cache(table, ref, S, max_pages, n_pages)) != LSA_OK) return s;
  if ((s = check_pools(pools, n_pools)) != LSA_OK) return s;
  if (!table_out || !ref_out || !aligned(ref_out, 16))
    return set_error(LSA_ERR_INVALID_ARG, "table_out or ref_out null, or ref_out not 16-byte aligned");
  if ((s = check_space(workspace, workspace_bytes, compact_ws(n_pages))) != LSA_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* ws = static_cast<int*>(workspace);
  if ((s = cuda_check(launch_compact_plan(ref, n_pages, ref_out, n_live, ws, st), "compact plan launch")) != LSA_OK) return s;
  int first = 0;
  bool rows = true;
  do {
    const Pools p = take_pools(pools, n_pools, &first);
    if ((s = cuda_check(launch_compact(table, S, max_pages, n_pages, table_out, ws, p, rows, device_status_ptr(), st),
                        "compact launch")) != LSA_OK)
      return s;
    rows = false;
  } while (first < n_pools);
  return LSA_OK;
}

}  // extern "C"
