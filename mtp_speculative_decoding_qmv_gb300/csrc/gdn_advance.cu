// gdn_advance.cu -- the gated delta rule over packed rows, token by token, and
// the entry point that picks between this and the chunks (gdn_chunk.cu), sm_103a.
//
//   S' = alpha_t S;  e_t = beta_t (v_t - S' k_t);  S = S' + e_t k_t^T;  o_t = S q_t
//
// A single token reads and writes its sequence's whole state (64 KB a head at
// 128 x 128) for 6 dk dv operations: bound by memory.  Rows of S never interact:
// eight lanes share a row, eight columns each of every 64, so the state moves in
// 32-byte pieces a lane and a row's dot products end with three shuffles.  Keys
// and queries are read straight into the registers that multiply them (the four
// rows of a warp read the same addresses; no shared memory, no barrier), the next
// token's while this one is computed.
// Measured, 48 heads of 128 x 128, bf16, in a graph: 64 sequences' single tokens 70 us
// (406 MB, 5.8 TB/s); one sequence's token 4.5 us (the launch, and two trips to memory
// one after the other), each of its next tokens 0.5 us: a token waits for the one before
// it, and few warps have nothing else to do.  Two to six tokens loaded ahead (more
// registers, no faster a token), o as S' q + e (k . q) with its sums beside that of e,
// and scalar in place of paired products were measured: level or slower.
#include <cuda_runtime.h>

#include "gdn_rows.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int kLanesPerRow = 8;
constexpr int kRowsPerCta = 16;
constexpr int kThreads = kRowsPerCta * kLanesPerRow;
constexpr int kMaxDim = 128;
// The bound on a sequence's rows from which all of a call's go in chunks (bf16).  In
// graphs, 48 heads of 128 x 128, us of the row after row kernel and of the chunks at 24,
// 32 and 48 rows: one sequence 14 and 16, 18 and 16, 26 and 16; 4 sequences 35 and 31, 46
// and 30, 66 and 32; 16 sequences 86 and 89, 113 and 91, 164 and 94.  A call that mixes
// lengths pays for it: 64 single tokens beside a prompt of 512 rows take 360, as two
// calls 113 (67 and 43).
constexpr int kChunkFrom = 32;

__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

// One token's share of a lane: its columns of k and q, its rows' values, the gates.
template <class T, int kR>
struct Token {
  Raw8<T> k[2], q[2];
  float v[kR], alpha, beta;
};

// kFull: dk == 128, every lane's columns are real.  kR: state rows a thread.
template <class T, bool kFull, int kR>
__global__ void __launch_bounds__(kThreads) gdn_recur_kernel(const AdvanceArgs a) {
  const int tid = threadIdx.x, rg = tid / kLanesPerRow, j = tid % kLanesPerRow;
  const int h = blockIdx.y, b = blockIdx.z, r0 = blockIdx.x * kRowsPerCta * kR + rg;
  Rows s;
  int slot = -1;
  if (b < a.B) {
    s = rows_of(a.q_start, b, a.rows);
    slot = slot_of(a.state_index, b, a.slots);
  } else {  // the rows past the last sequence's
    s.start = min(max(__ldg(a.q_start + a.B), 0), a.rows);
    s.n = a.rows - s.start;
  }
  if (s.n == 0) return;
  T *out = static_cast<T *>(a.out) + s.start * a.out_stride + (long long)h * a.dv;
  if (slot < 0) {
    for (int t = 0; t < s.n; ++t)
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (j == 0 && r0 + kRowsPerCta * r < a.dv)
          out[t * a.out_stride + r0 + kRowsPerCta * r] = rounded<T>(0.f);
    return;
  }
  const int hk = h / (a.H / a.Hk);
  const T *q = static_cast<const T *>(a.q) + s.start * a.q_stride + (long long)hk * a.dk + 8 * j;
  const T *k = static_cast<const T *>(a.k) + s.start * a.k_stride + (long long)hk * a.dk + 8 * j;
  const T *v = static_cast<const T *>(a.v) + s.start * a.v_stride + (long long)h * a.dv + r0;
  const long long gate = (long long)s.start * a.H + h;
  const bool col[2] = {kFull || 8 * j < a.dk, kFull || 64 + 8 * j < a.dk};
  float *state = a.state + ((long long)slot * a.H + h) * a.dv * a.dk + (long long)r0 * a.dk + 8 * j;
  float2 S[kR][8];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r0 + kRowsPerCta * r < a.dv && col[c]) {
        const float4 *p = reinterpret_cast<const float4 *>(state + (long long)kRowsPerCta * r * a.dk + 64 * c);
        x = __ldcg(p);
        y = __ldcg(p + 1);
      }
      S[r][4 * c] = make_float2(x.x, x.y);
      S[r][4 * c + 1] = make_float2(x.z, x.w);
      S[r][4 * c + 2] = make_float2(y.x, y.y);
      S[r][4 * c + 3] = make_float2(y.z, y.w);
    }
  auto load = [&](int t, Token<T, kR> &x) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (col[c]) {
        x.k[c] = load8(k + t * a.k_stride + 64 * c);
        x.q[c] = load8(q + t * a.q_stride + 64 * c);
      }
#pragma unroll
    for (int r = 0; r < kR; ++r)
      x.v[r] = r0 + kRowsPerCta * r < a.dv ? as_float(v[t * a.v_stride + kRowsPerCta * r]) : 0.f;
    x.alpha = __ldg(a.alpha + gate + (long long)t * a.H);
    x.beta = __ldg(a.beta + gate + (long long)t * a.H);
  };
  Token<T, kR> next = {};  // columns past dk stay zero
  load(0, next);
  for (int t = 0; t < s.n; ++t) {
    const Token<T, kR> x = next;
    if (t + 1 < s.n) load(t + 1, next);
    float2 kk[8], qq[8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      widen8(x.k[c], reinterpret_cast<float2(&)[4]>(kk[4 * c]));
      widen8(x.q[c], reinterpret_cast<float2(&)[4]>(qq[4 * c]));
    }
    const float2 al = make_float2(x.alpha, x.alpha);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 u0 = make_float2(0.f, 0.f), u1 = u0;
#pragma unroll
      for (int m = 0; m < 8; m += 2) {
        S[r][m] = __fmul2_rn(al, S[r][m]);
        S[r][m + 1] = __fmul2_rn(al, S[r][m + 1]);
        u0 = __ffma2_rn(S[r][m], kk[m], u0);
        u1 = __ffma2_rn(S[r][m + 1], kk[m + 1], u1);
      }
      const float2 u = __fadd2_rn(u0, u1);
      const float e = x.beta * (x.v[r] - row_sum(u.x + u.y));
      const float2 e2 = make_float2(e, e);
      float2 o0 = make_float2(0.f, 0.f), o1 = o0;
#pragma unroll
      for (int m = 0; m < 8; m += 2) {
        S[r][m] = __ffma2_rn(e2, kk[m], S[r][m]);
        S[r][m + 1] = __ffma2_rn(e2, kk[m + 1], S[r][m + 1]);
        o0 = __ffma2_rn(S[r][m], qq[m], o0);
        o1 = __ffma2_rn(S[r][m + 1], qq[m + 1], o1);
      }
      const float2 o = __fadd2_rn(o0, o1);
      const float sum = row_sum(o.x + o.y);
      if (j == r && r0 + kRowsPerCta * r < a.dv)
        out[t * a.out_stride + r0 + kRowsPerCta * r] = rounded<T>(sum);
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (r0 + kRowsPerCta * r < a.dv && col[c]) {
        float4 *p = reinterpret_cast<float4 *>(state + (long long)kRowsPerCta * r * a.dk + 64 * c);
        p[0] = make_float4(S[r][4 * c].x, S[r][4 * c].y, S[r][4 * c + 1].x, S[r][4 * c + 1].y);
        p[1] = make_float4(S[r][4 * c + 2].x, S[r][4 * c + 2].y, S[r][4 * c + 3].x, S[r][4 * c + 3].y);
      }
}

template <class T>
sv_status recur_run(const AdvanceArgs &a, cudaStream_t stream) {
  // two rows a thread once the CTAs fill the device several times over: they share the
  // loads and the widening of k and q.  (48 heads of 128 x 128, us with one and with two:
  // single tokens of 1, 4, 7, 16 and 64 sequences 3.2 and 3.6, 5.9 and 6.0, 8.7 and 8.6,
  // 16.2 and 15.4, 79 and 67; 8 rows each of 4, 16 and 64: 14.9 and 12.9, 46 and 36, 229
  // and 171.  The rule changes at 7 sequences.)
  const long long one = (long long)((a.dv + kRowsPerCta - 1) / kRowsPerCta) * a.H * a.B;
  const int R = one > 16ll * device_sm_count() ? 2 : 1;
  const dim3 grid((unsigned)((a.dv + kRowsPerCta * R - 1) / (kRowsPerCta * R)), (unsigned)a.H,
                  (unsigned)a.B + 1);
  void (*kernel)(AdvanceArgs) =
      a.dk == kMaxDim ? (R == 2 ? gdn_recur_kernel<T, true, 2> : gdn_recur_kernel<T, true, 1>)
                      : (R == 2 ? gdn_recur_kernel<T, false, 2> : gdn_recur_kernel<T, false, 1>);
  kernel<<<grid, kThreads, 0, stream>>>(a);
  return check_launch("gdn_advance");
}

}  // namespace
}  // namespace gdn
}  // namespace sv

using namespace sv;
using namespace sv::gdn;

extern "C" size_t gdn_advance_workspace_bytes(sv_dtype dtype, int B, int rows, int max_new, int Hv) {
  if (B < 0 || rows < 0 || Hv < 1 || dtype != SV_BF16 || max_new < kChunkFrom) return 0;
  return chunk_workspace_bytes(rows, B, Hv);
}

extern "C" sv_status gdn_advance(const void *q, const void *k, const void *v, sv_dtype dtype,
                                 long long q_row_stride, long long k_row_stride,
                                 long long v_row_stride, const float *alpha, const float *beta,
                                 float *state, const int32_t *q_start, const int32_t *state_index,
                                 int B, int rows, int max_new, int slots, int Hk, int Hv, int dk,
                                 int dv, void *out, long long out_row_stride, void *workspace,
                                 size_t workspace_bytes, sv_stream_t stream) {
  clear_error();
  const char *who = "gdn_advance";
  if (B < 0 || rows < 0 || max_new < 0 || slots < 0)
    return fail(SV_ERR_INVALID_ARG, "%s: B, rows, max_new and slots must not be negative", who);
  if (Hk < 1 || Hv < 1 || Hv % Hk)
    return fail(SV_ERR_INVALID_ARG, "%s: Hv=%d must be a positive multiple of Hk=%d", who, Hv, Hk);
  if (dk < 8 || dv < 8 || dk % 8 || dv % 8 || dk > kMaxDim || dv > kMaxDim)
    return fail(SV_ERR_UNSUPPORTED, "%s: dk, dv must be multiples of 8 in [8, 128] (dk=%d dv=%d)",
                who, dk, dv);
  if (Hv > 65535 || B > 65534) return fail(SV_ERR_UNSUPPORTED, "%s: too many heads or sequences", who);
  if (dtype != SV_F32 && dtype != SV_BF16)
    return fail(SV_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
  if (!state_index && slots < B)
    return fail(SV_ERR_INVALID_ARG, "%s: %d slots for %d sequences", who, slots, B);
  if (rows == 0) return SV_OK;
  if (!q || !k || !v || !alpha || !beta || (!state && slots) || !q_start || !out)
    return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  const size_t size = dtype == SV_F32 ? 4 : 2, R = rows;
  if (rows > 1) {
    if (q_row_stride < (long long)Hk * dk || k_row_stride < (long long)Hk * dk ||
        v_row_stride < (long long)Hv * dv || out_row_stride < (long long)Hv * dv)
      return fail(SV_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", who);
    if (q_row_stride % 8 || k_row_stride % 8 || v_row_stride % 8 || out_row_stride % 8)
      return fail(SV_ERR_INVALID_ARG, "%s: row strides must be multiples of 8 elements", who);
  }
  for (const void *p : {q, k, v, (const void *)state, (const void *)out})
    if (!aligned(p, 16))
      return fail(SV_ERR_INVALID_ARG, "%s: q, k, v, state and out must be 16-byte aligned", who);
  for (const void *p : {(const void *)alpha, (const void *)beta, (const void *)q_start,
                        (const void *)state_index})
    if (p && !aligned(p, 4)) return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  auto span = [&](long long stride, long long row) {
    return ((R - 1) * (size_t)(rows > 1 ? stride : 0) + (size_t)row) * size;
  };
  struct Buf {
    const void *p;
    size_t n;
  };
  const Buf in[] = {{q, span(q_row_stride, (long long)Hk * dk)},
                    {k, span(k_row_stride, (long long)Hk * dk)},
                    {v, span(v_row_stride, (long long)Hv * dv)},
                    {alpha, R * Hv * 4},
                    {beta, R * Hv * 4},
                    {q_start, ((size_t)B + 1) * 4},
                    {state_index, state_index ? (size_t)B * 4 : 0}};
  const Buf to[] = {{state, (size_t)slots * Hv * dv * dk * 4},
                    {out, span(out_row_stride, (long long)Hv * dv)}};
  for (const Buf &o : to)
    for (const Buf &i : in)
      if (overlaps(o.p, o.n, i.p, i.n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
  if (overlaps(to[0].p, to[0].n, to[1].p, to[1].n))
    return fail(SV_ERR_INVALID_ARG, "%s: out overlaps the state", who);
  const size_t need = gdn_advance_workspace_bytes(dtype, B, rows, max_new, Hv);
  if (need) {
    if (!workspace || !aligned(workspace, 256))
      return fail(SV_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", who);
    if (workspace_bytes < need)
      return fail(SV_ERR_INVALID_ARG, "%s: the workspace has %zu bytes, %zu are needed", who,
                  workspace_bytes, need);
    for (const Buf &i : in)
      if (overlaps(workspace, need, i.p, i.n))
        return fail(SV_ERR_INVALID_ARG, "%s: the workspace overlaps an input", who);
    for (const Buf &o : to)
      if (overlaps(workspace, need, o.p, o.n))
        return fail(SV_ERR_INVALID_ARG, "%s: the workspace overlaps an output", who);
  }
  AdvanceArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.out_stride = out_row_stride;
  a.alpha = alpha;
  a.beta = beta;
  a.q_start = q_start;
  a.state_index = state_index;
  a.state = state;
  a.out = out;
  a.B = B;
  a.rows = rows;
  a.slots = slots;
  a.Hk = Hk;
  a.H = Hv;
  a.dk = dk;
  a.dv = dv;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16 && max_new >= kChunkFrom) return chunk_run(a, workspace, s);
  return dtype == SV_F32 ? recur_run<float>(a, s) : recur_run<__nv_bfloat16>(a, s);
}
