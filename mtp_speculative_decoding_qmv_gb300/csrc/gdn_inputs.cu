// gdn_inputs.cu -- what the gated delta rule of a GatedDeltaNet layer reads, from
// the layer's projections, in one pass over packed rows, sm_103a.
//
//   y[c]  = silu(sum_j weight[j][c] x[t - (W - 1) + j][c])   (before row 0: the window)
//   q     = scale y_q / sqrt(sum y_q^2 + eps) per head, k likewise without scale, v = y_v
//   alpha = exp(-exp(a_log) softplus(a + dt_bias)),  beta = 1 / (1 + exp(-b))
//
// Bound by memory: every input is read once and every output written once (the
// rows before a tile are read twice).  A warp takes one head (up to 128
// channels, four a lane) of a tile of rows of one sequence and slides the
// window along in registers, so the W taps cost no loads; four to eight rows' loads
// are in flight a warp, 24 warps an SM (16 for the widest windows, whose registers they
// are).  The heads of a row are neighbouring warps, so
// a CTA reads and writes runs of 1 KB.  The tiles begin at the sequences' first rows: a
// sequence's first tile alone reads its window, and the same warp writes it, so
// one launch needs no order among its CTAs.
// Measured, 10240 channels and 48 heads, bf16, W = 4: three prompts of 7519 rows in all
// 81 us (313 MB, 3.9 TB/s; ncu: issue 51 %, DRAM 43 %: a batch's loads, then its
// arithmetic; with fewer warps and no batch ahead 236 us), 256 single tokens with
// their windows 23 us (74 MB); four rows of one sequence 5 us, a launch and its
// dependent loads.  W = 2 .. 8, 7500 rows: 72, 77, 79, 85, 89, 95, 98 us; 256 tokens: 14,
// 16, 18, 20, 22, 26, 30 (in a graph).  Each width has its kernel: one for all of them, W
// known at run time, took 310 .. 323 and 58 .. 84.
#include <cuda_runtime.h>

#include "gdn_rows.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxW = 8;
constexpr int kBatch = 4;  // rows whose loads go together, a batch ahead

struct InputsArgs {
  const void *x, *a, *b;
  long long x_stride, a_stride, b_stride;
  const float *weight;  // [W][C]
  float *window;        // [slots][W - 1][C]
  const float *a_log, *dt_bias;
  const int32_t *q_start, *window_index;
  void *q, *k, *v;
  float *alpha, *beta;
  float q_scale, eps;
  int B, rows, slots, Hk, H, dk, dv, C, shift, update, heads, tasks;
};

// Four consecutive values.
__device__ __forceinline__ float4 load4(const float *p) {
  return __ldg(reinterpret_cast<const float4 *>(p));
}
__device__ __forceinline__ uint2 load4(const __nv_bfloat16 *p) {
  return __ldg(reinterpret_cast<const uint2 *>(p));
}
__device__ __forceinline__ float4 widen4(float4 v) { return v; }
__device__ __forceinline__ float4 widen4(uint2 v) {
  const float2 a = floats_of(v.x), b = floats_of(v.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}
// y / (1 + 2^(-y log2 e)) by the approximate power and reciprocal: each off by about
// 2^-22 of the value, and the exponent by its rounding, in the range that silu does not
// send to zero; below y = -87 it is zero.
__device__ __forceinline__ float silu(float y) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return y * r;
}

// CTAs an SM by what spills: at 6, 7500 bf16 rows take 79 us (W = 4; 83 at 5 or 4), 111 and
// 153 (W = 7, 8; 95 and 98 at 4); at 5, fp32 rows of W = 6 take 116 (144 at 6, 120 at 4).
template <class X, class Y, int kW>
__global__ void __launch_bounds__(kWarps * 32, kW <= 4 ? 6 : kW <= 6 ? 5 : 4) gdn_inputs_kernel(const InputsArgs a) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= a.tasks) return;
  // head `unit` of the row: q heads, then k heads, then v heads
  const int kind = unit < a.Hk ? 0 : unit < 2 * a.Hk ? 1 : 2;
  const int head = kind == 2 ? unit - 2 * a.Hk : kind == 1 ? unit - a.Hk : unit;
  const int d = kind == 2 ? a.dv : a.dk;
  const int c0 = (kind == 2 ? 2 * a.Hk * a.dk + head * a.dv : unit * a.dk) + 4 * lane;
  const bool mine = 4 * lane < d && unit < a.heads;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 w[kW], h[kW];  // h[i]: the input kW - 1 - i places back; h[kW - 1] the newest
#pragma unroll
  for (int i = 0; i < kW; ++i) {  // on their way while the tile is looked for
    w[i] = h[i] = zero;
    if (mine) w[i] = load4(a.weight + (long long)i * a.C + c0);
  }
  int j;
  const int b = tile_owner(a.q_start, a.B, a.rows, a.shift, blockIdx.y, j);
  Rows s;
  int slot = -1;
  if (b < a.B) {
    s = rows_of(a.q_start, b, a.rows);
    slot = slot_of(a.window_index, b, a.slots);
  } else {
    s.start = min(max(__ldg(a.q_start + a.B), 0), a.rows);
    s.n = a.rows - s.start;
  }
  const int t0 = j << a.shift;
  if (j < 0 || t0 >= s.n) return;
  const int n = min(1 << a.shift, s.n - t0);  // rows of this tile
  const bool real = slot >= 0;

  if (unit >= a.heads) {  // the gates of 32 heads
    const int h = (unit - a.heads) * 32 + lane;
    if (h >= a.H) return;
    const float rate = expf(a.a_log[h]), bias = a.dt_bias[h];
    for (int t = 0; t < n; ++t) {
      const long long r = s.start + t0 + t;
      float al = 0.f, be = 0.f;
      if (real) {
        const float z = as_float(static_cast<const X *>(a.a)[r * a.a_stride + h]) + bias;
        const float y = as_float(static_cast<const X *>(a.b)[r * a.b_stride + h]);
        // softplus(z) = max(z, 0) + log(1 + exp(-|z|))
        al = expf(-rate * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)))));
        be = 1.f / (1.f + expf(-y));
      }
      a.alpha[r * a.H + h] = al;
      a.beta[r * a.H + h] = be;
    }
    return;
  }

  Y *to = static_cast<Y *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
  const long long to_row = (long long)(kind == 2 ? a.H : a.Hk) * d;
  to += head * d + 4 * lane + (s.start + t0) * to_row;
  if (!real) {
    for (int t = 0; t < n; ++t)
      if (mine) store4(to + t * to_row, zero);
    return;
  }
  const X *x = static_cast<const X *>(a.x) + (s.start + t0) * a.x_stride + c0;
  float *window = a.window + (long long)slot * (kW - 1) * a.C + c0;
#pragma unroll
  for (int i = 0; i < kW - 1; ++i)
    if (mine)
      h[i + 1] = t0 == 0 ? *reinterpret_cast<const float4 *>(window + (long long)i * a.C)
                         : widen4(load4(x + (long long)(i - (kW - 1)) * a.x_stride));
  if (t0 == 0 && a.update && mine) {
    // entry i of the next window: the input of row n - (kW - 1) + i, or the old
    // window's where that is before the first row
    float4 next[kW - 1];
#pragma unroll
    for (int i = 0; i < kW - 1; ++i) {
      const int last = s.n - (kW - 1) + i;
      next[i] = last >= 0 ? widen4(load4(x + (long long)last * a.x_stride))
                          : *reinterpret_cast<const float4 *>(window + (long long)(last + kW - 1) * a.C);
    }
#pragma unroll
    for (int i = 0; i < kW - 1; ++i) *reinterpret_cast<float4 *>(window + (long long)i * a.C) = next[i];
  }
  decltype(load4(x)) next[kBatch];
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t + i < n && mine) next[i] = load4(x + (long long)i * a.x_stride);
    x += (long long)kBatch * a.x_stride;
  };
  load(0);
  const float scale = kind == 0 ? a.q_scale : 1.f;
  for (int t = 0; t < n; t += kBatch) {
    decltype(load4(x)) raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) raw[i] = next[i];
    load(t + kBatch);
    float4 y[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
#pragma unroll
      for (int o = 0; o < kW - 1; ++o) h[o] = h[o + 1];
      h[kW - 1] = t + i < n && mine ? widen4(raw[i]) : zero;
      float4 sum = zero;
#pragma unroll
      for (int o = 0; o < kW; ++o) {
        sum.x = fmaf(w[o].x, h[o].x, sum.x);
        sum.y = fmaf(w[o].y, h[o].y, sum.y);
        sum.z = fmaf(w[o].z, h[o].z, sum.z);
        sum.w = fmaf(w[o].w, h[o].w, sum.w);
      }
      y[i] = make_float4(silu(sum.x), silu(sum.y), silu(sum.z), silu(sum.w));
    }
    if (kind < 2) {
      float ss[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        ss[i] = fmaf(y[i].x, y[i].x, fmaf(y[i].y, y[i].y, fmaf(y[i].z, y[i].z, y[i].w * y[i].w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float f = rsqrtf(ss[i] + a.eps) * scale;
        y[i] = make_float4(y[i].x * f, y[i].y * f, y[i].z * f, y[i].w * f);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t + i < n && mine) store4(to + i * to_row, y[i]);
    to += kBatch * to_row;
  }
}

using Kernel = void (*)(InputsArgs);
template <class X, class Y>
Kernel pick(int W) {
  constexpr Kernel of[kMaxW - 1] = {gdn_inputs_kernel<X, Y, 2>, gdn_inputs_kernel<X, Y, 3>,
                                    gdn_inputs_kernel<X, Y, 4>, gdn_inputs_kernel<X, Y, 5>,
                                    gdn_inputs_kernel<X, Y, 6>, gdn_inputs_kernel<X, Y, 7>,
                                    gdn_inputs_kernel<X, Y, 8>};
  return of[W - 2];
}

}  // namespace
}  // namespace gdn
}  // namespace sv

using namespace sv;
using namespace sv::gdn;

extern "C" sv_status gdn_inputs(const void *x, const void *a, const void *b, sv_dtype x_dtype,
                                long long x_row_stride, long long a_row_stride,
                                long long b_row_stride, const float *weight, float *window,
                                const float *a_log, const float *dt_bias, const int32_t *q_start,
                                const int32_t *window_index, int B, int rows, int max_new,
                                int slots, int W, int Hk, int Hv, int dk, int dv,
                                int update_window, float q_scale, float eps, sv_dtype out_dtype,
                                void *q, void *k, void *v, float *alpha, float *beta,
                                sv_stream_t stream) {
  clear_error();
  const char *who = "gdn_inputs";
  if (B < 0 || rows < 0 || max_new < 0 || slots < 0)
    return fail(SV_ERR_INVALID_ARG, "%s: B, rows, max_new and slots must not be negative", who);
  if (Hk < 1 || Hv < 1 || Hv % Hk)
    return fail(SV_ERR_INVALID_ARG, "%s: Hv=%d must be a positive multiple of Hk=%d", who, Hv, Hk);
  if (dk < 8 || dv < 8 || dk % 8 || dv % 8 || dk > 128 || dv > 128)
    return fail(SV_ERR_UNSUPPORTED, "%s: dk, dv must be multiples of 8 in [8, 128] (dk=%d dv=%d)",
                who, dk, dv);
  if (W < 2 || W > kMaxW) return fail(SV_ERR_UNSUPPORTED, "%s: W=%d outside [2, 8]", who, W);
  if (Hk > 16384 || Hv > 16384) return fail(SV_ERR_UNSUPPORTED, "%s: too many heads", who);
  if ((x_dtype != SV_F32 && x_dtype != SV_BF16) || (out_dtype != SV_F32 && out_dtype != SV_BF16))
    return fail(SV_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (!(eps >= 0.f) || !(q_scale == q_scale))
    return fail(SV_ERR_INVALID_ARG, "%s: eps must not be negative, q_scale a number", who);
  if (!window_index && slots < B)
    return fail(SV_ERR_INVALID_ARG, "%s: %d slots for %d sequences", who, slots, B);
  if (rows == 0) return SV_OK;
  if (!x || !a || !b || !weight || (!window && slots) || !a_log || !dt_bias || !q_start || !q || !k || !v ||
      !alpha || !beta)
    return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  const int C = 2 * Hk * dk + Hv * dv;
  const size_t size = x_dtype == SV_F32 ? 4 : 2, to = out_dtype == SV_F32 ? 4 : 2;
  if (rows > 1 && (x_row_stride < C || a_row_stride < Hv || b_row_stride < Hv))
    return fail(SV_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", who);
  if (rows > 1 && x_row_stride % 4)
    return fail(SV_ERR_INVALID_ARG, "%s: x's row stride must be a multiple of 4 elements", who);
  for (const void *p : {(const void *)x, (const void *)weight, (const void *)window,
                        (const void *)q, (const void *)k, (const void *)v})
    if (!aligned(p, 16))
      return fail(SV_ERR_INVALID_ARG, "%s: x, weight, window, q, k, v must be 16-byte aligned", who);
  if (!aligned(a, size) || !aligned(b, size))
    return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  for (const void *p : {(const void *)a_log, (const void *)dt_bias, (const void *)q_start,
                        (const void *)window_index, (const void *)alpha, (const void *)beta})
    if (p && !aligned(p, 4)) return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  struct Buf {
    const void *p;
    size_t n;
  };
  const size_t R = rows;
  const Buf in[] = {{x, ((R - 1) * (rows > 1 ? x_row_stride : 0) + C) * size},
                    {a, ((R - 1) * (rows > 1 ? a_row_stride : 0) + Hv) * size},
                    {b, ((R - 1) * (rows > 1 ? b_row_stride : 0) + Hv) * size},
                    {weight, (size_t)W * C * 4},
                    {a_log, (size_t)Hv * 4},
                    {dt_bias, (size_t)Hv * 4},
                    {q_start, ((size_t)B + 1) * 4},
                    {window_index, window_index ? (size_t)B * 4 : 0}};
  const Buf out[] = {{window, (size_t)slots * (W - 1) * C * 4},
                     {q, R * Hk * dk * to},
                     {k, R * Hk * dk * to},
                     {v, R * Hv * dv * to},
                     {alpha, R * Hv * 4},
                     {beta, R * Hv * 4}};
  for (int i = 0; i < 6; ++i) {
    for (const Buf &o : in)
      if (overlaps(out[i].p, out[i].n, o.p, o.n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
    for (int o = 0; o < i; ++o)
      if (overlaps(out[i].p, out[i].n, out[o].p, out[o].n))
        return fail(SV_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  }
  InputsArgs p = {};
  p.x = x;
  p.a = a;
  p.b = b;
  p.x_stride = x_row_stride;
  p.a_stride = a_row_stride;
  p.b_stride = b_row_stride;
  p.weight = weight;
  p.window = window;
  p.a_log = a_log;
  p.dt_bias = dt_bias;
  p.q_start = q_start;
  p.window_index = window_index;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.q_scale = q_scale;
  p.eps = eps;
  p.B = B;
  p.rows = rows;
  p.slots = slots;
  p.Hk = Hk;
  p.H = Hv;
  p.dk = dk;
  p.dv = dv;
  p.C = C;
  p.update = update_window != 0;
  p.heads = 2 * Hk + Hv;
  p.tasks = p.heads + (Hv + 31) / 32;
  // at least kMaxW rows a tile: a later tile's taps are then all rows of x
  p.shift = max_new <= 16 ? 4 : 5;
  auto tiles = [&] { return ((long long)rows >> p.shift) + B + 1; };
  while (tiles() > 65535 && p.shift < 20) ++p.shift;  // grid.y
  if (tiles() > 65535) return fail(SV_ERR_UNSUPPORTED, "%s: too many sequences", who);
  const dim3 grid((unsigned)((p.tasks + kWarps - 1) / kWarps),
                  (unsigned)tiles());
  const Kernel kernel =
      x_dtype == SV_F32
          ? (out_dtype == SV_F32 ? pick<float, float>(W) : pick<float, __nv_bfloat16>(W))
          : (out_dtype == SV_F32 ? pick<__nv_bfloat16, float>(W)
                                 : pick<__nv_bfloat16, __nv_bfloat16>(W));
  kernel<<<grid, kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return check_launch(who);
}
