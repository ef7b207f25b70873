// attn_common.cuh -- shared by the paged-attention kernels: the call's arguments,
// which keys each packed query row may attend, how the work is cut into equal
// runs of key tiles, the joining of split results, and non-finite values in
// places that some rows attend and others do not.
//
// Row r = t G + g of request b and kv head h is token t (of n_b) under query
// head h G + g (G = Hq / Hkv query heads share a kv head), so all rows of
// (b, h) read the same keys.  Token t stands at position p = kv_len_b - n_b + t
// and attends positions max(0, p - window + 1) .. p (from 0 when window is 0):
//   out_r = sum_j softmax_j(scale q_r . k_j) v_j
// and a row with no position (p < 0) is zero, its log-sum-exp -inf.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sv_device.cuh"

namespace sv {
namespace attn {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMaxCtas = 512;           // of one launch
constexpr size_t kCounterBytes = 4096;  // the start of the workspace

// The item that begins in a CTA's run and ends in a later one's: its rows
// [r0, r0 + count) under kv head h of the request whose packed rows begin at
// q0, shared by n CTAs; n = 0 for none.
struct SplitItem {
  int n, q0, h, r0, count, unused[3];
};

struct Args {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, out_stride;  // elements from a row to the next
  __nv_bfloat16 *out;
  float *lse;  // [rows][Hq] or null
  const int32_t *table, *q_start, *kv_len;
  int B, rows, Hq, Hkv, G;
  int num_pages, max_pages, page_shift, window;
  float scale, scale_log2;  // scale, scale * log2(e)
  unsigned *counters;  // attn_tc_kernel's arrivals, zero between calls
  SplitItem *splits;   // attn_rows_kernel's split items [CTAs]
  float *partials;
};

struct Request {
  int q0, n, len;  // first packed row, new tokens, positions in the cache
};
__device__ __forceinline__ Request load_request(const Args &a, int b) {
  Request r;
  r.q0 = min(max(__ldg(a.q_start + b), 0), a.rows);
  r.n = min(max(__ldg(a.q_start + b + 1), r.q0), a.rows) - r.q0;
  const long long most = (long long)a.max_pages << a.page_shift;
  r.len = (int)min((long long)max(__ldg(a.kv_len + b), 0), most);
  return r;
}
// Rows [r0, r0 + count) of a request: positions [lo, hi) hold every key that
// one of them attends; [all_lo, all_hi) the keys that all of them attend.
struct Span {
  int lo, hi, all_lo, all_hi;
};
__device__ __forceinline__ Span rows_span(const Args &a, const Request &q, int r0, int count) {
  const int t0 = r0 / a.G, t1 = (r0 + count - 1) / a.G;
  const int p0 = q.len - q.n + t0, p1 = q.len - q.n + t1;
  Span s;
  s.hi = max(p1 + 1, 0);
  s.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), s.hi) : 0;
  s.all_lo = a.window > 0 ? max(p1 - a.window + 1, 0) : 0;
  s.all_hi = max(p0 + 1, 0);
  return s;
}

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap *map, int x, int y,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Nonzero when one of the two bf16 values is infinite or NaN: adding a unit to
// a full exponent carries into the sign's place.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t u) {
  return ((u & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Bounded waits that gave up, a word for each translation unit.
static __device__ unsigned int g_give_up;
__device__ __forceinline__ void report_give_up(unsigned bit) { atomicOr(&g_give_up, bit); }

// log-sum-exp of a row from its sum l and the maximum m of its raw scores
__device__ __forceinline__ float row_lse(const Args &a, float m, float l) {
  return l > 0.f || l != l ? fmaf(m, a.scale, logf(l)) : kNegInf;
}

// The first tensor-map row of page `idx` of request b under head h, or the row
// past the last (read as zeros) when the page holds no key in [lo, hi) or its
// id is out of range.
__device__ __forceinline__ int page_row(const Args &a, int b, int h, int idx, int lo, int hi) {
  int page = a.num_pages;
  const long long first = (long long)idx << a.page_shift;
  if (first < hi && first + (1 << a.page_shift) > lo && idx < a.max_pages) {
    page = __ldg(a.table + (size_t)b * a.max_pages + idx);
    if ((unsigned)page >= (unsigned)a.num_pages) page = a.num_pages;
  }
  return (page * a.Hkv + (page < a.num_pages ? h : 0)) << a.page_shift;
}

// A value that some rows of a tile attend and others do not would meet weights of
// zero; where it is not finite the kernels put zero in its place, in shared
// memory (clear_nonfinite), and afterwards add it to the rows that attend it.  A
// weight of a finite score is positive, so the sum gets the value itself; a
// score of -inf has weight zero, and the product is NaN.  Such positions lie
// outside [all_lo, all_hi): at most a tile's tokens on either side (and what a
// shorter window leaves between), however long the context is.
__device__ __forceinline__ uint32_t nonfinite_bits(const uint4 &v) {
  return nonfinite_bits(v.x) | nonfinite_bits(v.y) | nonfinite_bits(v.z) | nonfinite_bits(v.w);
}
__device__ __forceinline__ void clear_nonfinite(uint4 &v) {
  v.x &= ~((nonfinite_bits(v.x) >> 15) * 0xFFFFu);
  v.y &= ~((nonfinite_bits(v.y) >> 15) * 0xFFFFu);
  v.z &= ~((nonfinite_bits(v.z) >> 15) * 0xFFFFu);
  v.w &= ~((nonfinite_bits(v.w) >> 15) * 0xFFFFu);
}
__device__ __forceinline__ float2 two_floats(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ float add_if_nonfinite(float sum, float v, bool weightless) {
  if (fabsf(v) < -kNegInf) return sum;
  return weightless ? __int_as_float(0x7fffffff) : sum + v;
}
// The first element of position j's key and value under head h, or -1 where the
// page's id is out of range.
__device__ __forceinline__ long long position_at(const Args &a, int b, int h, int j, int D) {
  const int page = __ldg(a.table + (size_t)b * a.max_pages + (j >> a.page_shift));
  if ((unsigned)page >= (unsigned)a.num_pages) return -1;
  return ((((long long)page * a.Hkv + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
}

// ---- equal runs of work ------------------------------------------------------
// The items (request, row tile, kv head) each own a run of key tiles; laid end
// to end they make `units` tiles, cut into `ctas` runs that differ by at most
// one tile, so ragged lengths balance by themselves and a single long request
// spreads over the device.  A CTA's run holds at most two items that it does
// not own whole: the one it begins inside and the one it ends inside.
struct Runs {
  long long units;
  int ctas;
  __device__ long long begin(int c) const { return units * c / ctas; }
  // the CTA whose run holds unit u
  __device__ int owner(long long u) const { return (int)(((u + 1) * ctas - 1) / units); }
};

// A split item's partial result: unnormalised sums, then maxima and sums [rows]
// each.  CTA c has two: 2 c + 1 for the item that begins in its run and ends in
// a later one, 2 c for the one that began in an earlier run.
__device__ __forceinline__ float *partial_at(const Args &a, int slot, int tile_rows, int D) {
  return a.partials + (size_t)slot * tile_rows * (D + 2);
}

// Elements d .. d + 3 of row r, normalised and rounded, and with element 0 the
// row's log-sum-exp.  A row that attends nothing is zero.
template <int D>
__device__ __forceinline__ void store_out4(const Args &a, int q0, int h, int r, int d,
                                           float4 o, float m, float l) {
  const int t = r / a.G, g = r - t * a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2 *>(a.out + (long long)(q0 + t) * a.out_stride +
                             (long long)(h * a.G + g) * D + d) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (d == 0 && a.lse) a.lse[(long long)(q0 + t) * a.Hq + h * a.G + g] = row_lse(a, m, l);
}

// Weight of a partial with maximum m and sum l against the joint maximum; one
// without keys has none (its maximum is -inf, and so may be every other).
__device__ __forceinline__ float join_weight(const Args &a, float m, float l, float joint) {
  return m == kNegInf && l == 0.f ? 0.f : exp2_approx((m - joint) * a.scale_log2);
}

}  // namespace attn
}  // namespace sv
