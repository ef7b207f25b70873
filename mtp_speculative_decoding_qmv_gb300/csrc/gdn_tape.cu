// gdn_tape.cu -- GatedDeltaNet innovation tape: capture over the verify tokens
// and replay over the accepted prefix, sm_103a.
//
// Sources: "MTPLX 2.24x faster TPS", section "Layer 0: MLX Runtime"
// (innovation-tape GDN capture records KB-scale (token, gate, state-delta)
// tuples; a rejection replays the tape instead of restoring a snapshot, bit
// exact) and "Layer 2: Speculative cycle" (the tape commits accepted deltas,
// rolls back rejected ones); "MTP와 DFlash" (mlxcel manual), section
// "Qwen3.8-Flash-Next (qwen4_exp) MTP" (rollback replays the GatedDeltaNet
// recurrence over the accepted tokens).
//
// Gated delta rule per (sequence b, head h), S in R^{dv x dk} (fp32):
//   S' = alpha_t S;  u = S' k_t;  e_t = beta_t (v_t - u);  S_t = S' + e_t k_t^T;
//   o_t = S_t q_t.
// Rows of S never interact: row i needs only v_t[i] and the shared k_t, q_t,
// alpha_t, beta_t.  Eight lanes share a row, each holding 16 of its fp32
// elements in registers at columns 32c + 4j + [0, 4) (lane j of the row), so
// every load and store of the state is a run of 128 contiguous bytes per row;
// the row's dot products are finished with three shuffles.  The capture CTA
// owns 16 rows of one head, or 32 (two rows per thread, one read of each
// token's keys and queries serving both) once a batch would fill more than
// two waves of CTAs; small batches keep (dv / 16) x H CTAs (384 at H = 48,
// dv = 128) for latency.  The capture's arithmetic is packed fp32
// (fma.rn.f32x2 / mul.rn.f32x2: two independent IEEE operations each), and
// the state element update is the same explicit roundings in both kernels --
// a round-to-nearest multiply by the gate, then one fused multiply-add of the
// rank-1 term -- so replaying the tape reproduces the capture's states bit
// for bit.
#include <cuda_runtime.h>

#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kLanesPerRow = 8;
constexpr int kChunks = 4;                   // float4 chunks per lane
constexpr int kMaxDim = kLanesPerRow * kChunks * 4;  // 128
constexpr int kRowsPerCta = 16;
constexpr int kThreads = kRowsPerCta * kLanesPerRow;  // 128
constexpr int kMaxT = 16;
// float4 loads per thread to stage kMaxT tokens of one kMaxDim-wide vector
constexpr int kStage4 = kMaxT * kMaxDim / 4 / kThreads;  // 4


// Tape: one block per sequence b of tape_block_floats(T,H,dk,dv) floats, each
// block holding e [T][H][dv], then k [T][H][dk], then alpha [T][H] (padded to
// 4 floats).  Stacking the tapes of several batches gives the tape of the
// concatenated batch.
__host__ __device__ inline size_t tape_block_floats(int T, int H, int dk, int dv) {
  return (size_t)T * H * (dv + dk) + (((size_t)T * H + 3) / 4) * 4;
}
struct TapeView {
  float *base;
  size_t blk;
  int T, H, dk, dv;
  __device__ float *e(int b, int t, int h) const {
    return base + b * blk + ((size_t)t * H + h) * dv;
  }
  __device__ float *k(int b, int t, int h) const {
    return base + b * blk + (size_t)T * H * dv + ((size_t)t * H + h) * dk;
  }
  __device__ float *alpha(int b, int t, int h) const {
    return base + b * blk + (size_t)T * H * (dv + dk) + (size_t)t * H + h;
  }
};

struct GdnArgs {
  const float *state0;  // capture: snapshot (read only)
  float *state;         // replay: in/out
  const float *q, *k, *v, *alpha, *beta;
  float *out;
  float *state_out;  // capture: S_T (may be null)
  TapeView tape;
  const int32_t *n_replay;
  int n_replay_count;
  int n_replay_bias;
  int32_t *err_flags;
  int B, T, H, dk, dv;
};

// Column of element 4 * c of lane j's chunks.
__device__ __forceinline__ int chunk_col(int j, int c) { return 32 * c + 4 * j; }

// Row-local dot product finished across the row's eight lanes.
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

// kFull: dk == kMaxDim, so every lane's chunks are real columns (no checks).
// kR: state rows per thread; the CTA covers 16 kR rows of one head, row
// group g = tid / 8 holding rows r0 + g + 16 r.  One read of a token's keys
// and queries from shared memory serves all kR rows.  Lane j keeps its row
// elements as float2 pairs (columns 32c + 4j + {0,1} and + {2,3}) for the
// packed fp32 instructions: per element the same IEEE roundings as scalar
// code (the decay a round-to-nearest multiply, the rank-1 term one fused
// multiply-add), so replay still reproduces the capture bit for bit.
// kT > 0: the token count is known at compile time (the token loop unrolls).
// Register budgets: two rows per thread (large batches) at 80 registers, six
// CTAs per SM (16 sequences x 48 heads take 3.4 waves of CTAs instead of
// 4.04); one row at 64, eight CTAs per SM (the verify cycle's batch 1: 0.5 %
// more cycles/s than at 72).
template <bool kFull, int kR, int kT>
__global__ void __launch_bounds__(kThreads, kR == 2 ? 6 : 8) gdn_capture_kernel(const GdnArgs a) {
  constexpr int kRows = kRowsPerCta * kR;
  const int T = kT > 0 ? kT : a.T;
  static_assert(kMaxT * (kRows / 4) <= kThreads, "one float4 of values per thread");
  __shared__ __align__(16) float ks[kMaxT][kMaxDim];
  __shared__ __align__(16) float qs[kMaxT][kMaxDim];
  __shared__ __align__(16) float vs[kMaxT][kRows];
  __shared__ float als[kMaxT], bes[kMaxT];
  const int tid = threadIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  const int r0 = blockIdx.x * kRows;
  const int rg = tid / kLanesPerRow;
  const int j = tid % kLanesPerRow;
  pdl_launch_dependents();
  // the committed state does not depend on the preceding kernel: its load
  // overlaps that kernel's tail under programmatic dependent launch
  float2 S[kR][2 * kChunks];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int i = r0 + rg + kRowsPerCta * r;
    const bool ok = i < a.dv;
    const float *src = a.state0 + (((size_t)b * a.H + h) * a.dv + (ok ? i : 0)) * a.dk;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ok && (kFull || chunk_col(j, c) < a.dk))
        f = __ldcg(reinterpret_cast<const float4 *>(src + chunk_col(j, c)));
      S[r][2 * c] = make_float2(f.x, f.y);
      S[r][2 * c + 1] = make_float2(f.z, f.w);
    }
  }
  pdl_wait();  // the verify tokens' q, k, v and gates are the preceding kernels' outputs
  // The tokens' keys, queries, gates and this CTA's values, once.  Every load
  // names the global space and all of them are issued before the first
  // shared-memory store: a generic load might alias those stores and would
  // wait behind each one, one round trip per load.
  {
    const int dk4 = a.dk / 4, nk4 = T * dk4;
    float4 kr[kStage4], qr[kStage4];
    // float4 e = tid + u kThreads of the staged tokens is (t, c4) = (e / dk4,
    // e % dk4); at full width (dk4 = 32, kThreads = 128) that is
    // (tid / 32 + 4 u, tid % 32), one fixed stride per u
    static_assert(kThreads == 4 * 32, "full-width staging: four tokens per pass");
    const size_t tok_stride = (size_t)a.H * a.dk;  // floats from token t to t + 1
    const size_t off0 = ((size_t)b * T * a.H + h) * a.dk;
#pragma unroll
    for (int u = 0; u < kStage4; ++u) {
      if constexpr (kFull) {
        const int t = (tid >> 5) + 4 * u;
        if (t < T) {
          const size_t off = off0 + t * tok_stride + 4 * (tid & 31);
          kr[u] = __ldcg(reinterpret_cast<const float4 *>(a.k + off));
          qr[u] = __ldcg(reinterpret_cast<const float4 *>(a.q + off));
        }
      } else {
        const int e = tid + u * kThreads;
        if (e < nk4) {
          const int t = e / dk4, c4 = e - t * dk4;
          const size_t off = off0 + t * tok_stride + 4 * c4;
          kr[u] = __ldcg(reinterpret_cast<const float4 *>(a.k + off));
          qr[u] = __ldcg(reinterpret_cast<const float4 *>(a.q + off));
        }
      }
    }
    // this CTA's value rows per token as float4 (dv % 4 == 0, so a float4 is
    // either wholly inside the rows or wholly past them)
    const int t_v = tid / (kRows / 4), r_v = 4 * (tid % (kRows / 4));
    const bool has_v = tid < T * (kRows / 4);
    float4 vr = make_float4(0.f, 0.f, 0.f, 0.f);
    if (has_v && r0 + r_v < a.dv)
      vr = __ldcg(reinterpret_cast<const float4 *>(
          a.v + (((size_t)b * T + t_v) * a.H + h) * a.dv + r0 + r_v));
    float al_r = 0.f, be_r = 0.f;
    if (tid < T) {
      const size_t bth = ((size_t)b * T + tid) * a.H + h;
      al_r = __ldcg(a.alpha + bth);
      be_r = __ldcg(a.beta + bth);
    }
#pragma unroll
    for (int u = 0; u < kStage4; ++u) {
      if constexpr (kFull) {
        const int t = (tid >> 5) + 4 * u;
        if (t < T) {
          *reinterpret_cast<float4 *>(&ks[t][4 * (tid & 31)]) = kr[u];
          *reinterpret_cast<float4 *>(&qs[t][4 * (tid & 31)]) = qr[u];
        }
      } else {
        const int e = tid + u * kThreads;
        if (e < nk4) {
          const int t = e / dk4, c4 = e - t * dk4;
          *reinterpret_cast<float4 *>(&ks[t][4 * c4]) = kr[u];
          *reinterpret_cast<float4 *>(&qs[t][4 * c4]) = qr[u];
        }
      }
    }
    if (has_v) *reinterpret_cast<float4 *>(&vs[t_v][r_v]) = vr;
    if (tid < T) {
      als[tid] = al_r;
      bes[tid] = be_r;
    }
  }

  __syncthreads();

  // the token's records and outputs advance by fixed strides
  float *e_out = a.tape.e(b, 0, h) + r0 + rg;
  float *o_out = a.out ? a.out + ((size_t)b * T * a.H + h) * a.dv + r0 + rg : nullptr;
  float *k_out = a.tape.k(b, 0, h);
  float *al_out = a.tape.alpha(b, 0, h);
  const size_t e_step = (size_t)a.H * a.dv, k_step = (size_t)a.H * a.dk;
#pragma unroll
  for (int t = 0; t < (kT > 0 ? kT : kMaxT); ++t) {
    if (kT == 0 && t >= T) break;
    const float al = als[t], be = bes[t];
    const float2 al2 = make_float2(al, al);
    // this lane's key columns (zeros past dk, where the state is zero too)
    float2 kk[2 * kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const float4 f = (kFull || chunk_col(j, c) < a.dk)
                           ? *reinterpret_cast<const float4 *>(&ks[t][chunk_col(j, c)])
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      kk[2 * c] = make_float2(f.x, f.y);
      kk[2 * c + 1] = make_float2(f.z, f.w);
    }
    // S' = alpha S ; u = S' k   (two pair accumulators per row)
    float u[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < 2 * kChunks; m += 2) {
        S[r][m] = __fmul2_rn(al2, S[r][m]);
        S[r][m + 1] = __fmul2_rn(al2, S[r][m + 1]);
        acc0 = __ffma2_rn(S[r][m], kk[m], acc0);
        acc1 = __ffma2_rn(S[r][m + 1], kk[m + 1], acc1);
      }
      const float2 a2 = __fadd2_rn(acc0, acc1);
      u[r] = row_sum(a2.x + a2.y);
    }
    // S_t = S' + e k^T (the keys' last use, so the queries take their
    // registers), then o = S_t q
    float ev[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int rr = rg + kRowsPerCta * r;
      ev[r] = be * (vs[t][rr] - u[r]);
      const float2 e2 = make_float2(ev[r], ev[r]);
#pragma unroll
      for (int m = 0; m < 2 * kChunks; ++m) S[r][m] = __ffma2_rn(e2, kk[m], S[r][m]);
    }
    float2 qq[2 * kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const float4 f = (kFull || chunk_col(j, c) < a.dk)
                           ? *reinterpret_cast<const float4 *>(&qs[t][chunk_col(j, c)])
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      qq[2 * c] = make_float2(f.x, f.y);
      qq[2 * c + 1] = make_float2(f.z, f.w);
    }
    float op[kR];  // the lane's partial of each row's output
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < 2 * kChunks; m += 2) {
        acc0 = __ffma2_rn(S[r][m], qq[m], acc0);
        acc1 = __ffma2_rn(S[r][m + 1], qq[m + 1], acc1);
      }
      const float2 a2 = __fadd2_rn(acc0, acc1);
      op[r] = a2.x + a2.y;
    }
    // The outputs leave the critical chain, so two rows share one butterfly:
    // the row group's lanes first swap halves (even lanes keep row 0, odd
    // lanes row 1), then every step adds the same row's partials -- the same
    // additions in the same order as one row at a time.  Then one store per
    // lane: the outputs from lanes 0 (row 0) and 1 (row 1), the records e
    // from lanes 2 and 3 (one row: lane 0 the record, lane 1 the output).
    if constexpr (kR == 2) {
      const int rsel = j & 1;
      float o = rsel ? op[1] : op[0];
      o += __shfl_xor_sync(0xffffffffu, rsel ? op[0] : op[1], 1);
      o += __shfl_xor_sync(0xffffffffu, o, 2);
      o += __shfl_xor_sync(0xffffffffu, o, 4);
      float *dst = j < 2 ? o_out : e_out;
      const float val = j < 2 ? o : (rsel ? ev[1] : ev[0]);
      if (j < 4 && dst && r0 + rg + kRowsPerCta * rsel < a.dv) dst[kRowsPerCta * rsel] = val;
    } else {
      const float o = row_sum(op[0]);
      float *dst = j == 0 ? e_out : o_out;
      if (j < 2 && dst && r0 + rg < a.dv) dst[0] = j == 0 ? ev[0] : o;
    }
    if (blockIdx.x == 0) {
      for (int c = tid; c < a.dk; c += kThreads) k_out[c] = ks[t][c];
      if (tid == 0) *al_out = al;
    }
    e_out += e_step;
    if (o_out) o_out += e_step;
    k_out += k_step;
    al_out += a.H;
  }
  if (a.state_out) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int i = r0 + rg + kRowsPerCta * r;
      if (i >= a.dv) continue;
      float *dst = a.state_out + (((size_t)b * a.H + h) * a.dv + i) * a.dk;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (chunk_col(j, c) < a.dk)
          *reinterpret_cast<float4 *>(dst + chunk_col(j, c)) =
              make_float4(S[r][2 * c].x, S[r][2 * c].y, S[r][2 * c + 1].x, S[r][2 * c + 1].y);
    }
  }
}

__global__ void __launch_bounds__(kThreads) gdn_replay_kernel(const GdnArgs a) {
  __shared__ __align__(16) float ks[kMaxT][kMaxDim];
  __shared__ __align__(16) float es[kMaxT][kRowsPerCta];
  __shared__ float als[kMaxT];
  const int tid = threadIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  pdl_launch_dependents();
  pdl_wait();  // the accepted counts are the preceding kernel's output
  int L = a.n_replay[b % a.n_replay_count] + a.n_replay_bias;
  const bool clamped = L < 0 || L > a.T;
  L = min(max(L, 0), a.T);
  if (clamped && a.err_flags && blockIdx.x == 0 && h == 0 && tid == 0)
    atomicOr(&a.err_flags[b], SV_FLAG_REPLAY_RANGE);
  if (L == 0) return;  // nothing accepted: the state is untouched
  const int r0 = blockIdx.x * kRowsPerCta;
  const int i = r0 + tid / kLanesPerRow;
  const int j = tid % kLanesPerRow;
  const bool row_ok = i < a.dv;
  // The accepted records and this row's state: every load names the global
  // space and all are issued before the first shared-memory store (a
  // generic load might alias those stores and would wait behind each one).
  float S[kChunks * 4];
  float *dst = a.state + (((size_t)b * a.H + h) * a.dv + (row_ok ? i : 0)) * a.dk;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row_ok && chunk_col(j, c) < a.dk)
      f = __ldcg(reinterpret_cast<const float4 *>(dst + chunk_col(j, c)));
    S[4 * c] = f.x;
    S[4 * c + 1] = f.y;
    S[4 * c + 2] = f.z;
    S[4 * c + 3] = f.w;
  }
  {
    const int dk4 = a.dk / 4, nk4 = L * dk4;
    float4 kr[kStage4];
#pragma unroll
    for (int u = 0; u < kStage4; ++u) {
      const int e = tid + u * kThreads;
      if (e < nk4) {
        const int t = e / dk4, c4 = e - t * dk4;
        kr[u] = __ldcg(reinterpret_cast<const float4 *>(a.tape.k(b, t, h) + 4 * c4));
      }
    }
    const int t_e = tid / (kRowsPerCta / 4), r_e = 4 * (tid % (kRowsPerCta / 4));
    const bool has_e = tid < L * (kRowsPerCta / 4);
    float4 er = make_float4(0.f, 0.f, 0.f, 0.f);
    if (has_e && r0 + r_e < a.dv)
      er = __ldcg(reinterpret_cast<const float4 *>(a.tape.e(b, t_e, h) + r0 + r_e));
    const float al_r = tid < L ? __ldcg(a.tape.alpha(b, tid, h)) : 0.f;
#pragma unroll
    for (int u = 0; u < kStage4; ++u) {
      const int e = tid + u * kThreads;
      if (e < nk4) {
        const int t = e / dk4, c4 = e - t * dk4;
        *reinterpret_cast<float4 *>(&ks[t][4 * c4]) = kr[u];
      }
    }
    if (has_e) *reinterpret_cast<float4 *>(&es[t_e][r_e]) = er;
    if (tid < L) als[tid] = al_r;
  }
  __syncthreads();
  if (!row_ok) return;
  for (int t = 0; t < L; ++t) {
    const float al = als[t], et = es[t][tid / kLanesPerRow];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (chunk_col(j, c) < a.dk) {
        const float4 kk = *reinterpret_cast<const float4 *>(&ks[t][chunk_col(j, c)]);
        S[4 * c] = __fmaf_rn(et, kk.x, __fmul_rn(al, S[4 * c]));
        S[4 * c + 1] = __fmaf_rn(et, kk.y, __fmul_rn(al, S[4 * c + 1]));
        S[4 * c + 2] = __fmaf_rn(et, kk.z, __fmul_rn(al, S[4 * c + 2]));
        S[4 * c + 3] = __fmaf_rn(et, kk.w, __fmul_rn(al, S[4 * c + 3]));
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    if (chunk_col(j, c) < a.dk)
      *reinterpret_cast<float4 *>(dst + chunk_col(j, c)) =
          make_float4(S[4 * c], S[4 * c + 1], S[4 * c + 2], S[4 * c + 3]);
}

sv_status validate(const char *who, int B, int T, int H, int dk, int dv) {
  if (B < 0 || T < 1 || H < 1 || dk < 1 || dv < 1)
    return fail(SV_ERR_INVALID_ARG, "%s: need B >= 0, T, H, dk, dv >= 1", who);
  if (T > kMaxT) return fail(SV_ERR_UNSUPPORTED, "%s: T=%d > %d", who, T, kMaxT);
  if (dk > kMaxDim || dv > kMaxDim || dk % 4 || dv % 4)
    return fail(SV_ERR_UNSUPPORTED, "%s: dk, dv must be multiples of 4 and <= 128 (dk=%d dv=%d)",
                who, dk, dv);
  if ((long long)H > 65535 || (long long)B > 65535)
    return fail(SV_ERR_UNSUPPORTED, "%s: B and H must be <= 65535", who);
  return SV_OK;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" size_t gdn_tape_bytes(int B, int T, int H, int dk, int dv) {
  if (B < 0 || T < 1 || H < 1 || dk < 1 || dv < 1) return 0;
  return (size_t)B * tape_block_floats(T, H, dk, dv) * sizeof(float);
}

extern "C" sv_status gdn_tape_capture(const float *state0, const float *q, const float *k,
                                      const float *v, const float *alpha, const float *beta,
                                      int B, int T, int H, int dk, int dv, float *out, float *tape,
                                      float *state_out, sv_stream_t stream) {
  clear_error();
  sv_status st = validate("gdn_tape_capture", B, T, H, dk, dv);
  if (st != SV_OK) return st;
  if (B == 0) return SV_OK;
  if (!state0 || !q || !k || !v || !alpha || !beta || !tape)
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_capture: null pointer");
  const void *ptrs[9] = {state0, q, k, v, alpha, beta, out, tape, state_out};
  for (const void *p : ptrs)
    if (p && !aligned(p, 16))
      return fail(SV_ERR_INVALID_ARG, "gdn_tape_capture: pointers must be 16-byte aligned");
  const size_t n_bth = (size_t)B * T * H;
  const size_t sb = (size_t)B * H * dv * dk * 4, qkb = n_bth * dk * 4, vb = n_bth * dv * 4,
               ab = n_bth * 4, tb = gdn_tape_bytes(B, T, H, dk, dv);
  const void *ins[6] = {state0, q, k, v, alpha, beta};
  const size_t insb[6] = {sb, qkb, qkb, vb, ab, ab};
  for (int j = 0; j < 6; ++j)
    if (overlaps(tape, tb, ins[j], insb[j]) || overlaps(out, vb, ins[j], insb[j]) ||
        overlaps(state_out, sb, ins[j], insb[j]))
      return fail(SV_ERR_INVALID_ARG, "gdn_tape_capture: an output overlaps an input");
  if (overlaps(out, vb, tape, tb) || overlaps(state_out, sb, tape, tb) ||
      overlaps(state_out, sb, out, vb))
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_capture: outputs overlap");
  GdnArgs args = {};
  args.state0 = state0;
  args.q = q;
  args.k = k;
  args.v = v;
  args.alpha = alpha;
  args.beta = beta;
  args.out = out;
  args.state_out = state_out;
  args.tape = TapeView{tape, tape_block_floats(T, H, dk, dv), T, H, dk, dv};
  args.B = B;
  args.T = T;
  args.H = H;
  args.dk = dk;
  args.dv = dv;
  // two rows per thread once one row per thread would take more than two
  // waves of resident CTAs (a small batch keeps the wider grid for latency)
  const int ctas1 = ((dv + kRowsPerCta - 1) / kRowsPerCta) * H * B;
  const int R = ctas1 > 2 * 7 * device_sm_count() ? 2 : 1;
  dim3 grid((unsigned)((dv + kRowsPerCta * R - 1) / (kRowsPerCta * R)), (unsigned)H, (unsigned)B);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  // launched in stream order (starting early measured slower); the kernel
  // triggers its dependents at entry so the following kernel may start early
  // full-width heads at the verify widths M = K + 1 = 3..6 take kernels with
  // the token count built in
  void (*kern)(const GdnArgs) = nullptr;
  if (dk == kMaxDim) {
    switch (T * 4 + R) {
      case 3 * 4 + 1: kern = gdn_capture_kernel<true, 1, 3>; break;
      case 4 * 4 + 1: kern = gdn_capture_kernel<true, 1, 4>; break;
      case 5 * 4 + 1: kern = gdn_capture_kernel<true, 1, 5>; break;
      case 6 * 4 + 1: kern = gdn_capture_kernel<true, 1, 6>; break;
      case 3 * 4 + 2: kern = gdn_capture_kernel<true, 2, 3>; break;
      case 4 * 4 + 2: kern = gdn_capture_kernel<true, 2, 4>; break;
      case 5 * 4 + 2: kern = gdn_capture_kernel<true, 2, 5>; break;
      case 6 * 4 + 2: kern = gdn_capture_kernel<true, 2, 6>; break;
      default: kern = R == 2 ? gdn_capture_kernel<true, 2, 0> : gdn_capture_kernel<true, 1, 0>;
    }
  } else {
    kern = R == 2 ? gdn_capture_kernel<false, 2, 0> : gdn_capture_kernel<false, 1, 0>;
  }
  if (cudaLaunchKernelEx(&cfg, kern, args) != cudaSuccess)
    return fail(SV_ERR_CUDA, "gdn_capture: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return check_launch("gdn_tape_capture");
}

extern "C" sv_status gdn_tape_replay(float *state, const float *tape, const int32_t *n_replay,
                                     int n_replay_count, int n_replay_bias, int B, int T, int H,
                                     int dk, int dv, int32_t *err_flags, sv_stream_t stream) {
  clear_error();
  sv_status st = validate("gdn_tape_replay", B, T, H, dk, dv);
  if (st != SV_OK) return st;
  if (B == 0) return SV_OK;
  if (!state || !tape || !n_replay)
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_replay: null pointer");
  if (n_replay_count < 1 || n_replay_count > B)
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_replay: n_replay_count=%d outside [1, B=%d]",
                n_replay_count, B);
  if (!aligned(state, 16) || !aligned(tape, 16) || !aligned(n_replay, 4) ||
      (err_flags && !aligned(err_flags, 4)))
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_replay: misaligned pointer");
  const size_t sb = (size_t)B * H * dv * dk * 4, tb = gdn_tape_bytes(B, T, H, dk, dv);
  if (overlaps(state, sb, tape, tb) || overlaps(state, sb, n_replay, (size_t)n_replay_count * 4) ||
      overlaps(err_flags, (size_t)B * 4, state, sb) || overlaps(err_flags, (size_t)B * 4, tape, tb))
    return fail(SV_ERR_INVALID_ARG, "gdn_tape_replay: state/flags overlap the tape or counts");
  GdnArgs args = {};
  args.state = state;
  args.tape = TapeView{const_cast<float *>(tape), tape_block_floats(T, H, dk, dv), T, H, dk, dv};
  args.n_replay = n_replay;
  args.n_replay_count = n_replay_count;
  args.n_replay_bias = n_replay_bias;
  args.err_flags = err_flags;
  args.B = B;
  args.T = T;
  args.H = H;
  args.dk = dk;
  args.dv = dv;
  dim3 grid((unsigned)((dv + kRowsPerCta - 1) / kRowsPerCta), (unsigned)H, (unsigned)B);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  // launched in stream order (starting early measured slower); the kernel
  // triggers its dependents at entry so the following kernel may start early
  if (cudaLaunchKernelEx(&cfg, gdn_replay_kernel, args) != cudaSuccess)
    return fail(SV_ERR_CUDA, "gdn_replay: launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return check_launch("gdn_tape_replay");
}
