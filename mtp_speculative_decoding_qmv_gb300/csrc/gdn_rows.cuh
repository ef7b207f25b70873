// gdn_rows.cuh -- shared by the GatedDeltaNet kernels over packed rows: a
// sequence's rows and slot, loads of eight values, packed fp32 arithmetic.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace gdn {

// Sequence b's rows [start, start + n).  q_start is clamped to [0, rows], so
// that whatever it holds no row outside the tensors is touched.
struct Rows {
  int start, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t *q_start, int b, int rows) {
  const int s = min(max(__ldg(q_start + b), 0), rows);
  const int e = min(max(__ldg(q_start + b + 1), 0), rows);
  return {s, max(e - s, 0)};
}
// Sequence b's slot of `slots`, -1 where the index names none.
__device__ __forceinline__ int slot_of(const int32_t *index, int b, int slots) {
  const int i = index ? __ldg(index + b) : b;
  return i >= 0 && i < slots ? i : -1;
}

// Tiles of 1 << shift rows that begin at the sequences' first rows, numbered so that
// sequence b's first is (q_start[b] >> shift) + b: room for the tiles of every sequence
// before it, those that are not full included.  The owner of tile number i, in [0, B]
// (B: the rows past the last sequence), and its place j among the owner's tiles (past
// its last: no such tile).  By a whole warp.
__device__ __forceinline__ int tile_owner(const int32_t *q_start, int B, int rows, int shift, int i,
                                          int &j) {
  const int lane = threadIdx.x & 31;
  auto first = [&](int b) { return (min(max(__ldg(q_start + b), 0), rows) >> shift) + b; };
  int lo = 0, n = B + 1;  // the owner is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool upto = at < lo + n && first(at) <= i;
    const int found = max(__popc(__ballot_sync(0xffffffffu, upto)) - 1, 0);
    n = min(step, n - found * step);
    lo += found * step;
  }
  j = i - first(lo);
  return lo;
}

// Eight consecutive values, 32 bytes of fp32 or 16 of bf16, still as loaded.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
__device__ __forceinline__ Raw8<float> load8(const float *p) {
  Raw8<float> r;
  r.a = __ldg(reinterpret_cast<const float4 *>(p));
  r.b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  return r;
}
__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16 *p) {
  return {__ldg(reinterpret_cast<const uint4 *>(p))};
}
__device__ __forceinline__ float2 floats_of(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
__device__ __forceinline__ void widen8(const Raw8<float> &r, float2 (&v)[4]) {
  v[0] = make_float2(r.a.x, r.a.y);
  v[1] = make_float2(r.a.z, r.a.w);
  v[2] = make_float2(r.b.x, r.b.y);
  v[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16> &r, float2 (&v)[4]) {
  v[0] = floats_of(r.a.x);
  v[1] = floats_of(r.a.y);
  v[2] = floats_of(r.a.z);
  v[3] = floats_of(r.a.w);
}
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

struct AdvanceArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride, out_stride;  // elements from row to row
  const float *alpha, *beta;                           // [rows][H]
  const int32_t *q_start, *state_index;
  float *state;  // [slots][H][dv][dk]
  void *out;     // [rows][H][dv]
  int B, rows, slots, Hk, H, dk, dv;
};

// gdn_chunk.cu: bf16 rows in chunks on the tensor cores.
size_t chunk_workspace_bytes(int rows, int B, int H);
sv_status chunk_run(const AdvanceArgs &a, void *workspace, cudaStream_t stream);

}  // namespace gdn
}  // namespace sv
