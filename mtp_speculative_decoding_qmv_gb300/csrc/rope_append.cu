// rope_append.cu -- a step's queries, keys and values on their way to paged
// attention, sm_103a: the norm of each query and key head, rotary positions
// with one or more axes, and the keys and values into their slots of the paged
// cache, in one pass over the projections' outputs.
//
// Per head x of D values (norm where a weight is given, queries and keys only):
//   y_e = x_e w_e / sqrt(sum_i x_i^2 / D + eps)                        (fp32)
// and for rotary pair f < R / 2 with elements (a, b) = (f, f + R / 2), or
// (2f, 2f + 1) when interleaved, and t = position[axis_f] * freq_f:
//   y_a' = y_a cos t - y_b sin t,   y_b' = y_b cos t + y_a sin t
// Elements past R pass through; values only change their type.  Everything is
// computed in fp32 and rounded once, to bf16, at the store.
//
// The angle of a far position needs more bits than fp32 has (position 10^6
// times a frequency near 1 leaves an error of 0.06 rad), so frequencies come
// as turns per position in 64-bit fixed point (2^-64 turns): the product with
// the integer position wraps modulo one turn by itself and is exact to
// position x 2^-65 turns.  Its top 32 bits, a signed fraction of a turn, go to
// sincospi as a float (2^-26 turns at most off): an absolute error near 2e-7 rad
// at any position, with no double precision arithmetic.
//
// Memory traffic is the bound: each input read once, each output written once.
// A lane holds eight consecutive elements of a head (one or two 16-byte loads),
// so D / 8 lanes hold a head and a warp 1, 2 or 4 heads of D 256, 128 or 64 at
// a time; it takes kIter such sets of one row's queries, keys and values, all
// loads in flight together.  The row's angles are computed once by the warp,
// spread over its lanes, and shared by shuffles; they serve all its heads.  The
// partner element of a pair is in the same lane (interleaved) or R / 16 lanes
// away (one shuffle).
//
// Measured (GB300): 8191 rows of 20 + 4 + 4 bf16 heads of 256, normed, a quarter
// turned: 52.4 us (235 MB, 4.5 TB/s), with 60 % of the issue slots used, most by
// the norm's and the turn's fp32 work.  From fp32, without the norm, it streams
// at 6.0 TB/s.  4 rows: 2.1 us, 128 rows: 3.1 us, the launch and one round trip
// to memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kMaxAxes = 4;

struct RopeArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements from a row to the next
  const int32_t *positions, *slots;
  const uint64_t *freqs;
  const uint8_t *axis;
  const float *q_weight, *k_weight;
  float eps;
  int rows, axes, Hq, Hkv, R, page_shift;
  int num_slots;
  __nv_bfloat16 *q_out, *k_cache, *v_cache;
};

// N values as they lie in memory, 32 bits at a time, and widened.
template <int W>
__device__ __forceinline__ void load_words(const void *p, uint32_t (&x)[W]) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const uint4 v = __ldg(static_cast<const uint4 *>(p) + i);
    x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
  }
}
template <typename T, int W, int N>
__device__ __forceinline__ void widen(const uint32_t (&x)[W], float (&y)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __uint_as_float(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      y[2 * i] = __uint_as_float(x[i] << 16);
      y[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
  }
}

// Two fp32 operations in one instruction, each rounded as the scalar one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
template <int N>
__device__ __forceinline__ void store_bf16(__nv_bfloat16 *p, const float (&x)[N]) {
  static_assert(N == 8, "16 bytes");
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                             pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <typename T, int D, bool kPairs, int kIter>
__global__ void __launch_bounds__(kRopeWarps * 32, sizeof(T) == 4 ? 5 : 6)
    rope_append_kernel(const RopeArgs a) {
  constexpr int E = 8;                        // elements a lane holds
  constexpr int W = E * (int)sizeof(T) / 4;
  constexpr int kLanes = D / E, kSet = 32 / kLanes;  // lanes a head, heads a set
  const int lane = threadIdx.x & 31;
  const int rotated = a.Hq + a.Hkv, total = rotated + a.Hkv;
  const unsigned groups = (unsigned)(total + kIter * kSet - 1) / (kIter * kSet);
  const unsigned task = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  if (task >= (unsigned)a.rows * groups) return;
  const int row = (int)(task / groups);
  const int h_warp = (int)(task - (unsigned)row * groups) * (kIter * kSet);
  const int h0 = h_warp + lane / kLanes, e0 = lane % kLanes * E;

  // every head's load is issued before anything waits for one
  uint32_t raw[kIter][W];
  {
    const T *q = static_cast<const T *>(a.q) + (long long)row * a.q_stride + e0;
    const T *k = static_cast<const T *>(a.k) + (long long)row * a.k_stride + e0;
    const T *v = static_cast<const T *>(a.v) + (long long)row * a.v_stride + e0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int h = h0 + i * kSet;
      const T *src = h < a.Hq ? q + h * D : h < rotated ? k + (h - a.Hq) * D : v + (h - rotated) * D;
#pragma unroll
      for (int j = 0; j < W; ++j) raw[i][j] = 0;
      if (h < total) load_words<W>(src, raw[i]);
    }
  }
  const int slot = __ldg(a.slots + row);
  const bool keep = (unsigned)slot < (unsigned)a.num_slots;

  const int half = a.R / 2;
  const bool turned = e0 < a.R;  // R is a multiple of 2 E: a lane is wholly in or out
  const bool first = e0 < half;
  float cs[E], sn[E];
#pragma unroll
  for (int e = 0; e < E; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (h_warp < rotated && half > 0) {
    auto angle = [&](int f, float &c, float &s) {
      const int ax = a.axis ? min((int)__ldg(a.axis + f), a.axes - 1) : 0;
      const int pos = __ldg(a.positions + (long long)row * a.axes + ax);
      const uint64_t turns = (uint64_t)(int64_t)pos * __ldg(a.freqs + f);
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    };
    // the lane's elements turn by angles f0 .. (every second element a new one
    // when interleaved); the warp computes each angle once, kOwn a lane, or one
    // where 32 lanes are enough
    constexpr int kOwn = D / 64;
    constexpr int kStep = kPairs ? 2 : 1;
    const int f0 = kPairs ? e0 / 2 : first ? e0 : e0 - half;
    if (half <= 32) {
      float c, s;
      angle(min(lane, half - 1), c, s);
#pragma unroll
      for (int e = 0; e < E; e += kStep) {
        cs[e] = __shfl_sync(0xffffffffu, c, f0 + e / kStep);
        sn[e] = __shfl_sync(0xffffffffu, s, f0 + e / kStep);
      }
    } else {
      float c[kOwn], s[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) angle(min(lane * kOwn + i, half - 1), c[i], s[i]);
#pragma unroll
      for (int e = 0; e < E; e += kStep) {
        const int f = e / kStep;  // f0 is a multiple of 4, so of kOwn
        cs[e] = __shfl_sync(0xffffffffu, c[f % kOwn], (f0 + f) / kOwn);
        sn[e] = __shfl_sync(0xffffffffu, s[f % kOwn], (f0 + f) / kOwn);
      }
    }
#pragma unroll
    for (int e = 0; e < E; e += kStep) {
      if (!turned) cs[e] = 1.f, sn[e] = 0.f;
      if constexpr (kPairs) {
        cs[e + 1] = cs[e];
        sn[e + 1] = sn[e];
        sn[e] = -sn[e];
      } else if (first) {
        sn[e] = -sn[e];
      }
    }
  }
  const int partner = !turned ? lane : first ? lane + half / E : lane - half / E;
  float w[E];  // the weights of the lane's elements, the queries' or the keys'
  const float *held = nullptr;
  const long long page = keep ? slot >> a.page_shift : 0;
  const int off = slot & ((1 << a.page_shift) - 1);
  __nv_bfloat16 *q_out = a.q_out + (long long)row * a.Hq * D + e0;
  const long long cache = (((page * a.Hkv) << a.page_shift) + off) * D + e0;
  const int per_head = D << a.page_shift;

#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (h_warp + i * kSet >= total) break;  // the same for the warp
    const int h = h0 + i * kSet;
    float x[E];
    widen<T>(raw[i], x);
    if (h_warp + i * kSet < rotated) {  // some head of the set is a query or a key
      const bool value = h >= rotated;
      const float *weights = value ? nullptr : h < a.Hq ? a.q_weight : a.k_weight;
      if (weights != held && weights) {
        uint32_t y[E];
        load_words<E>(weights + e0, y);
        widen<float>(y, w);
      }
      held = weights;
      if (a.q_weight || a.k_weight) {  // the same for the warp
        float2 two = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = make_float2(x[e], x[e + 1]);
          two = fma2(v, v, two);
        }
        float ss = two.x + two.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        if (weights) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 v = mul2(mul2(make_float2(x[e], x[e + 1]), make_float2(r, r)),
                                  make_float2(w[e], w[e + 1]));
            x[e] = v.x;
            x[e + 1] = v.y;
          }
        }
      }
      float y[E];
      if constexpr (kPairs) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = x[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
      }
      if (turned && !value) {  // else as it is, infinities included
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = fma2(make_float2(y[e], y[e + 1]), make_float2(sn[e], sn[e + 1]),
                                mul2(make_float2(x[e], x[e + 1]), make_float2(cs[e], cs[e + 1])));
          x[e] = v.x;
          x[e + 1] = v.y;
        }
      }
    }
    if (h < a.Hq)
      store_bf16<E>(q_out + h * D, x);
    else if (keep && h < total)
      store_bf16<E>(h < rotated ? a.k_cache + cache + (long long)(h - a.Hq) * per_head
                                : a.v_cache + cache + (long long)(h - rotated) * per_head,
                    x);
  }
}

typedef void (*RopeKernel)(const RopeArgs);

template <typename T, int D>
RopeKernel pick(bool pairs, bool many) {
  return pairs ? (many ? rope_append_kernel<T, D, true, 4> : rope_append_kernel<T, D, true, 1>)
               : (many ? rope_append_kernel<T, D, false, 4> : rope_append_kernel<T, D, false, 1>);
}
template <typename T>
RopeKernel pick(int D, bool pairs, bool many) {
  return D == 64 ? pick<T, 64>(pairs, many)
                 : D == 128 ? pick<T, 128>(pairs, many) : pick<T, 256>(pairs, many);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status rope_kv_append(const void *q, const void *k, const void *v, sv_dtype x_dtype,
                                    long long q_row_stride, long long k_row_stride,
                                    long long v_row_stride, const int32_t *positions, int axes,
                                    const int32_t *slots, const uint64_t *freqs,
                                    const uint8_t *axis, const float *q_weight,
                                    const float *k_weight, float eps, int rows, int Hq, int Hkv,
                                    int D, int rotary_dim, int interleaved, int page_size,
                                    int num_pages, uint16_t *q_out, uint16_t *k_cache,
                                    uint16_t *v_cache, sv_stream_t stream) {
  clear_error();
  const char *who = "rope_kv_append";
  if (rows < 0 || Hq < 1 || Hkv < 1 || num_pages < 1)
    return fail(SV_ERR_INVALID_ARG,
                "%s: need rows >= 0, Hq >= 1, Hkv >= 1, num_pages >= 1 (rows=%d Hq=%d Hkv=%d "
                "num_pages=%d)",
                who, rows, Hq, Hkv, num_pages);
  if (x_dtype != SV_F32 && x_dtype != SV_BF16)
    return fail(SV_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)x_dtype);
  if (D != 64 && D != 128 && D != 256)
    return fail(SV_ERR_UNSUPPORTED, "%s: D=%d is not 64, 128 or 256", who, D);
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16)
    return fail(SV_ERR_INVALID_ARG, "%s: rotary_dim=%d is not a multiple of 16 in [0, D=%d]", who,
                rotary_dim, D);
  if (axes < 1 || axes > kMaxAxes)
    return fail(SV_ERR_UNSUPPORTED, "%s: axes=%d outside [1, %d]", who, axes, kMaxAxes);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(SV_ERR_UNSUPPORTED, "%s: page_size=%d is not 16, 32, 64, 128 or 256", who,
                page_size);
  if ((long long)num_pages * page_size >= (1ll << 31))
    return fail(SV_ERR_UNSUPPORTED, "%s: slots pass 31 bits", who);
  if (Hq > 4096 || Hkv > 4096) return fail(SV_ERR_UNSUPPORTED, "%s: more than 4096 heads", who);
  if (!(eps >= 0.f)) return fail(SV_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  if (rows == 0) return SV_OK;
  if (!q || !k || !v || !positions || !slots || (rotary_dim > 0 && !freqs) || !q_out || !k_cache ||
      !v_cache || (axes > 1 && rotary_dim > 0 && !axis))
    return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  const int size = x_dtype == SV_F32 ? 4 : 2;
  if (q_row_stride < (long long)Hq * D || k_row_stride < (long long)Hkv * D ||
      v_row_stride < (long long)Hkv * D)
    return fail(SV_ERR_INVALID_ARG, "%s: a row stride is smaller than its row", who);
  if (q_row_stride * size % 16 || k_row_stride * size % 16 || v_row_stride * size % 16)
    return fail(SV_ERR_INVALID_ARG, "%s: row strides must be multiples of 16 bytes", who);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(SV_ERR_INVALID_ARG, "%s: q, k, v, q_out and the caches must be 16-byte aligned",
                who);
  if (!aligned(positions, 4) || !aligned(slots, 4) || (freqs && !aligned(freqs, 8)) ||
      (q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
    return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  const size_t cache = (size_t)num_pages * Hkv * page_size * D * 2;
  const size_t qo = (size_t)rows * Hq * D * 2;
  struct Buf {
    const void *p;
    size_t n;
  };
  const Buf in[] = {
      {q, ((size_t)(rows - 1) * q_row_stride + (size_t)Hq * D) * size},
      {k, ((size_t)(rows - 1) * k_row_stride + (size_t)Hkv * D) * size},
      {v, ((size_t)(rows - 1) * v_row_stride + (size_t)Hkv * D) * size},
      {positions, (size_t)rows * axes * 4}, {slots, (size_t)rows * 4},
      {freqs, (size_t)rotary_dim * 4}, {axis, axis ? (size_t)rotary_dim / 2 : 0},
      {q_weight, (size_t)D * 4}, {k_weight, (size_t)D * 4}};
  const Buf out[] = {{q_out, qo}, {k_cache, cache}, {v_cache, cache}};
  for (int i = 0; i < 3; ++i) {
    for (const Buf &b : in)
      if (overlaps(out[i].p, out[i].n, b.p, b.n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(SV_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  }
  RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.positions = positions;
  a.slots = slots;
  a.freqs = freqs;
  a.axis = axes > 1 ? axis : nullptr;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.rows = rows;
  a.axes = axes;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.R = rotary_dim;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.num_slots = num_pages * page_size;
  a.q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
  a.k_cache = reinterpret_cast<__nv_bfloat16 *>(k_cache);
  a.v_cache = reinterpret_cast<__nv_bfloat16 *>(v_cache);

  // One set of heads a warp while that leaves the SMs fewer than 32 warps each,
  // so a small step spreads over the device; four beyond, where a row's angles
  // serve more heads and more loads are in flight.
  const int total = Hq + 2 * Hkv, set = 256 / D;
  const bool many = (long long)rows * total / set > (long long)device_sm_count() * 32;
  const int per = set * (many ? 4 : 1);
  const long long tasks = (long long)rows * ((total + per - 1) / per);
  const long long ctas = (tasks + kRopeWarps - 1) / kRopeWarps;
  if (ctas * kRopeWarps >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "%s: too many rows", who);
  const RopeKernel kernel = x_dtype == SV_F32 ? pick<float>(D, interleaved != 0, many)
                                              : pick<__nv_bfloat16>(D, interleaved != 0, many);
  kernel<<<(unsigned)ctas, kRopeWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return check_launch(who);
}
