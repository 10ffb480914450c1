// Rotary positions, and the writing of new rows into a paged cache.
//
//   a = pos * f_i,  y0 = m (x0 cos a - s x1 sin a),  y1 = m (x1 cos a + s x0 sin a)
//
// for pair i of a row at position pos (s = -1: the transposed rotation, which
// is the gradient). The angle, in turns, is a 64-bit product whose whole turns
// are dropped in 64 bits: at position 10^6 a 32-bit product alone is off by 0.06
// rad. Sine and cosine are those of the angle's fp32 head, with its tail added to
// first order; they and the rotation are fp32. A result is rounded once.
//
// Bound by bytes: every row is read and written once. A block takes a few
// tokens, computes their angles once into shared memory (they are the same for
// every head) and then streams rows; a thread keeps one column unit and steps
// over rows, four rows in flight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace lsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 32;        // tokens of a block
constexpr int kInFlight = 4;       // rows a thread loads before it stores

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements moved by one access.
template <class T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// Position of token t of sequence b, or -1 for padding.
__device__ __forceinline__ int token_pos(const RotateArgs& a, int b, int t) {
  int n = a.q_len ? __ldg(a.q_len + b) : a.T;
  n = n < 0 ? 0 : (n > a.T ? a.T : n);
  if (t >= n) return -1;
  const long long pos = static_cast<long long>(__ldg(a.seq_len + b)) - n + t;
  return pos < 0 ? -1 : static_cast<int>(pos);
}

// m cos a, s m sin a of pair i at position pos. a.freq is in turns: the turns of
// pos are reduced to [-1/2, 1/2] by a subtraction that is exact.
__device__ __forceinline__ float2 turn_of(const RotateArgs& a, int pos, int i) {
  const double w = static_cast<double>(pos) * a.freq[i];
  const double r = 2.0 * (w - rint(w));                          // half turns
  const float hi = static_cast<float>(r), lo = static_cast<float>(r - hi) * 3.14159265358979f;
  float s, c;
  sincospif(hi, &s, &c);
  return make_float2(a.amplitude * fmaf(-lo, s, c), a.sign * a.amplitude * fmaf(lo, c, s));   // to first order in lo
}

// Slot of position pos of sequence b in the pool (page, row in page); page -1 if unmapped.
__device__ __forceinline__ int2 slot_of(const RotateArgs& a, int b, int pos) {
  const int j = pos / a.page_size;
  int page = -1;
  if (j < a.max_pages) page = __ldg(a.table + static_cast<long long>(b) * a.max_pages + j);
  if (page < 0 || page >= a.n_pages) {
    record_bad_page(a.status);
    page = -1;
  }
  return make_int2(page, pos - j * a.page_size);
}

// x rows -> rotated rows. VEC elements per access (16 bytes, or 1 where the
// layout does not allow more). Units of a row: first the rotated ones (one pack
// of an interleaved layout holds VEC / 2 pairs; a half layout takes two packs,
// VEC pairs), then the packs that are only copied.
template <class T, int VEC, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a, int tok_per_block,
                                                          int heads_per_block) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float2 cs[];                 // [tok][rot / 2]
  __shared__ long long s_out[kMaxTok];           // element offset of the token's row in out, -1: skip
  const int n0 = blockIdx.x * tok_per_block;
  const int n_tok = min(tok_per_block, a.B * a.T - n0);
  const int h0 = blockIdx.y * heads_per_block;
  const int nh = min(heads_per_block, a.H - h0);
  const int pairs = a.rot / 2;
  constexpr int kUnitPairs = INTER ? (VEC > 1 ? VEC / 2 : 1) : VEC;
  constexpr int kPacks = (INTER && VEC > 1) ? 1 : 2;             // packs of a rotated unit
  const int n_rot = pairs / kUnitPairs;
  const int n_copy = a.in_place ? 0 : (a.d - a.rot) / VEC;
  const int units = n_rot + n_copy;
  const int rows = n_tok * nh;
  using P = Pack<T, VEC>;
  const T* x = static_cast<const T*>(a.x);
  T* out = static_cast<T*>(a.out);
  P v0[kInFlight], v1[kInFlight];
  // The unit's columns, and the rows that this thread has of it: r0, r0 + r_step, ...
  bool rotated;
  int u, r0, r_step, c0, c1;
  auto unit_of = [&](int u0) {
    const int nu = min(kThreads, units - u0);
    r_step = kThreads / nu;
    u = u0 + threadIdx.x % nu;
    r0 = threadIdx.x / nu;
    if (r0 >= r_step) r0 = rows;                  // threads left over
    rotated = u < n_rot;
    if (rotated) {
      c0 = a.offset + (INTER ? u * 2 * kUnitPairs : u * VEC);
      c1 = c0 + (INTER ? 1 : pairs);              // INTER with VEC = 1: the odd column
    } else {
      c0 = (u - n_rot) * VEC;
      if (c0 >= a.offset) c0 += a.rot;
      c1 = c0;
    }
  };
  auto load = [&](int r) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int rr = r + k * r_step;
      if (rr < rows) {
        const int tok = rr / nh, h = h0 + rr - tok * nh;
        const int b = (n0 + tok) / a.T, t = (n0 + tok) - b * a.T;
        const T* src = x + b * a.xb + t * a.xt + h * a.xh;
        v0[k] = *reinterpret_cast<const P*>(src + c0);
        if (kPacks == 2 && rotated) v1[k] = *reinterpret_cast<const P*>(src + c1);
      }
    }
  };
  // the first rows are on their way while the angles are computed
  unit_of(0);
  load(r0);
  for (int i = threadIdx.x; i < n_tok; i += kThreads) {
    const int b = (n0 + i) / a.T, t = (n0 + i) - b * a.T;
    const int pos = token_pos(a, b, t);
    long long o = -1;
    if (pos >= 0) {
      if (PAGED) {
        const int2 sl = slot_of(a, b, pos);
        if (sl.x >= 0) o = sl.x * a.ob + sl.y * a.ot;
      } else {
        o = b * a.ob + t * a.ot;
      }
    }
    s_out[i] = o;
  }
  for (int i = threadIdx.x; i < n_tok * pairs; i += kThreads) {
    const int tok = i / pairs, p = i - tok * pairs;
    const int b = (n0 + tok) / a.T, t = (n0 + tok) - b * a.T;
    const int pos = token_pos(a, b, t);
    cs[i] = pos >= 0 ? turn_of(a, pos, p) : make_float2(1.f, 0.f);
  }
  __syncthreads();
  // units per pass of the block: all of them, or kThreads at a time
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    if (u0) unit_of(u0);
    for (int r = r0; r < rows; r += r_step * kInFlight) {
      if (u0 || r != r0) load(r);
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int rr = r + k * r_step;
        if (rr >= rows) continue;
        const int tok = rr / nh, h = h0 + rr - tok * nh;
        const long long to = s_out[tok];
        if (to < 0) continue;
        T* dst = out + to + h * a.oh;
        if (rotated) {
          const float2* t = cs + tok * pairs + u * kUnitPairs;
          if (kPacks == 1) {
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
              const float2 w = t[e];
              const float x0 = to_f(v0[k].v[2 * e]), x1 = to_f(v0[k].v[2 * e + 1]);
              v0[k].v[2 * e] = from_f<T>(x0 * w.x - x1 * w.y);
              v0[k].v[2 * e + 1] = from_f<T>(x1 * w.x + x0 * w.y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float2 w = t[e];
              const float x0 = to_f(v0[k].v[e]), x1 = to_f(v1[k].v[e]);
              v0[k].v[e] = from_f<T>(x0 * w.x - x1 * w.y);
              v1[k].v[e] = from_f<T>(x1 * w.x + x0 * w.y);
            }
            *reinterpret_cast<P*>(dst + c1) = v1[k];
          }
        }
        *reinterpret_cast<P*>(dst + c0) = v0[k];
      }
    }
  }
}

// New rows -> e4m3 codes with a per-token scale. Half a warp per token: the row
// (<= 1024 columns, 8 per lane and pass) stays in registers between its maximum
// and its codes. Quotients are rounded as divisions are: the codes are those of
// the formula, not of a product with a reciprocal.
constexpr int kRowLanes = 16, kRowPasses = 8;
constexpr int kRowsPerBlock = kThreads / kRowLanes;
template <bool INTER>
__global__ void __launch_bounds__(kThreads) append_e4m3_kernel(const __grid_constant__ RotateArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float2 cs_all[];             // [rows of the block][rot / 2]
  const int lane = threadIdx.x % kRowLanes, in_block = threadIdx.x / kRowLanes;
  const int n = blockIdx.x * kRowsPerBlock + in_block;
  const bool exists = n < a.B * a.T;
  const int b = exists ? n / a.T : 0, t = exists ? n - b * a.T : 0;
  const int pairs = a.rot / 2;
  float2* cs = cs_all + in_block * pairs;
  const int vecs = exists ? a.H * a.d / 8 : 0;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.x) + static_cast<long long>(n) * a.H * a.d;
  using P = Pack<__nv_bfloat16, 8>;
  P raw[kRowPasses];
#pragma unroll
  for (int q = 0; q < kRowPasses; ++q) {         // on their way while position, page and angles are worked out
    const int u = q * kRowLanes + lane;
    if (u < vecs) raw[q] = *reinterpret_cast<const P*>(src + u * 8);
  }
  const int pos = exists ? token_pos(a, b, t) : -1;
  int2 sl = make_int2(-1, 0);
  if (pos >= 0) {
    sl = slot_of(a, b, pos);
    for (int i = lane; i < pairs; i += kRowLanes) cs[i] = turn_of(a, pos, i);
  }
  __syncwarp();
  float v[kRowPasses][8];
  float amax = 0.f;
#pragma unroll
  for (int q = 0; q < kRowPasses; ++q) {
    const int u = q * kRowLanes + lane;
    if (u >= vecs) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[q][e] = __bfloat162float(raw[q].v[e]);
    const int h = a.H > 1 ? u * 8 / a.d : 0;
    const int c = u * 8 - h * a.d - a.offset;    // column within the rotated part
    if (pos >= 0 && c >= 0 && c < a.rot) {
      if (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 w = cs[c / 2 + e];
          const float x0 = v[q][2 * e], x1 = v[q][2 * e + 1];
          v[q][2 * e] = x0 * w.x - x1 * w.y;
          v[q][2 * e + 1] = x1 * w.x + x0 * w.y;
        }
      } else {   // the other half of the pair comes from its own columns
        const bool low = c < pairs;
        const P other = *reinterpret_cast<const P*>(src + u * 8 + (low ? pairs : -pairs));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = cs[(low ? c : c - pairs) + e];
          const float y = __bfloat162float(other.v[e]);
          v[q][e] = low ? v[q][e] * w.x - y * w.y : v[q][e] * w.x + y * w.y;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[q][e]));
  }
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (sl.x < 0) return;
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  // x / scale by one division for the row: with 1 / scale rounded correctly, a product and one residual step round
  // the quotient correctly (Markstein 1990), away from the ends of the exponent range. A division for every column
  // bounds the kernel by instructions.
  const bool divide = !(scale > 1e-30f && scale < 1e30f);
  const float inv = __frcp_rn(scale);
  uint8_t* dst = static_cast<uint8_t*>(a.out) + sl.x * a.ob + sl.y * a.ot;
#pragma unroll
  for (int q = 0; q < kRowPasses; ++q) {
    const int u = q * kRowLanes + lane;
    if (u >= vecs) continue;
    if (divide) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[q][e] = __fdiv_rn(v[q][e], scale);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[q][e] * inv;
        v[q][e] = fmaf(fmaf(-x, scale, v[q][e]), inv, x);
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = __nv_cvt_float2_to_fp8x2(make_float2(v[q][2 * e], v[q][2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(dst + u * 8) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
  if (lane == 0) a.scales[static_cast<long long>(sl.x) * a.page_size + sl.y] = scale;
}

template <class T, int VEC, bool PAGED>
cudaError_t launch_t(const RotateArgs& a, cudaStream_t stream) {
  const void* fn = a.interleaved ? reinterpret_cast<const void*>(&rotate_kernel<T, VEC, true, PAGED>)
                                 : reinterpret_cast<const void*>(&rotate_kernel<T, VEC, false, PAGED>);
  // A block's share: about kInFlight packs per thread (32 KB for 16-byte packs), fewer where that leaves SMs without
  // a block; in whole tokens, or part of the heads of one token when its rows alone are more.
  const long long n = static_cast<long long>(a.B) * a.T;
  const int units = a.in_place ? a.rot / VEC : a.d / VEC;
  const long long per_row = units > 0 ? units : 1, per_tok = per_row * a.H;
  const long long even = (n * per_tok + device_sm_count() - 1) / device_sm_count();
  const long long target = std::max(std::min(even, static_cast<long long>(kThreads) * kInFlight), static_cast<long long>(kThreads));
  const long long tok = std::max(1ll, std::min(target / per_tok, static_cast<long long>(kMaxTok)));
  int heads = a.H;
  if (per_tok > target) {
    heads = static_cast<int>((target + per_row - 1) / per_row);
    if ((a.H + heads - 1) / heads > 65535) heads = (a.H + 65534) / 65535;
  }
  const dim3 grid(static_cast<unsigned>((n + tok - 1) / tok), (a.H + heads - 1) / heads);
  int tok_i = static_cast<int>(tok);
  const size_t smem = static_cast<size_t>(tok_i) * (a.rot / 2) * sizeof(float2);
  void* args[] = {const_cast<RotateArgs*>(&a), &tok_i, &heads};
  return launch_pdl(fn, grid, dim3(kThreads), smem, stream, args);
}

}  // namespace

cudaError_t launch_rope(const RotateArgs& a, int fp32, cudaStream_t stream) {
  if (fp32) return a.vec > 1 ? launch_t<float, 4, false>(a, stream) : launch_t<float, 1, false>(a, stream);
  return a.vec > 1 ? launch_t<__nv_bfloat16, 8, false>(a, stream) : launch_t<__nv_bfloat16, 1, false>(a, stream);
}

cudaError_t launch_append(const RotateArgs& a, int e4m3, cudaStream_t stream) {
  if (!e4m3) return launch_t<__nv_bfloat16, 8, true>(a, stream);
  const long long n = static_cast<long long>(a.B) * a.T;
  const int per = kRowsPerBlock;
  const void* fn = a.interleaved ? reinterpret_cast<const void*>(&append_e4m3_kernel<true>)
                                 : reinterpret_cast<const void*>(&append_e4m3_kernel<false>);
  void* args[] = {const_cast<RotateArgs*>(&a)};
  return launch_pdl(fn, dim3(static_cast<unsigned>((n + per - 1) / per)), dim3(kThreads),
                    static_cast<size_t>(per) * (a.rot / 2) * sizeof(float2), stream, args);
}

}  // namespace lsa
