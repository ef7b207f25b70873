// kv_pages.cu -- the paged cache's bookkeeping of one step, on the device,
// sm_103a: commit of the previous step's tokens, pages for the new ones from a
// ring of free pages, pages of ended requests back into it, and for every new
// token its row, position and slot.
//
// With ps tokens a page, request b of B in order, L = its committed length:
//   L_b   = length_b + commit_b            (0 when n_new_b < 0: the request ended)
//   q_b   = sum_{i < b} n_i                (n = max(n_new, 0): first packed row)
//   need_b = max(0, ceil((L_b + n_b) / ps) - held_b)
//   a_b   = sum_{i < b} need_i             (place of its first page in the ring)
//   table[b][held_b + i] = ring[(head + a_b + i) mod P]
//   row q_b + t: position L_b + t, slot table[b][(L_b + t) / ps] * ps + (L_b + t) mod ps
// Three prefix sums over the requests and then gathers; the bytes are a few
// per request and row, so the launch and a handful of dependent memory round
// trips (lengths, cursor, table or ring) are the whole cost.  One cluster does
// it in one launch: every CTA scans all requests itself (at most 4096, held in
// shared memory) and, after a cluster barrier that orders every read of the
// state before the first write of it (outputs may be the inputs' own buffers),
// fills its share of the pages and rows, finding their requests by search in
// the prefix sums, so one long prompt among many single tokens is spread over
// all threads.
//
// Measured (GB300, device time in a graph): 3.3 us for one verify block, 4.0
// for 32, 11.5 for 1000 requests with 103,502 new rows (1 MB: 0.15 us at the
// memory's rate).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kMaxRequests = 4096;
constexpr int kMaxThreads = 1024;
constexpr int kCluster = 16;

struct PagesArgs {
  const int32_t *len_in, *held_in, *cursor_in, *n_new, *n_commit;
  int n_commit_count, n_commit_bias;
  int B, page_shift, max_pages, num_pages, rows;
  int32_t *table, *ring;
  int32_t *len_out, *held_out, *cursor_out;
  int32_t *q_start, *kv_len, *slots, *positions, *err;
};

// Inclusive sums of kN values over the CTA's threads, in thread order, in place;
// the totals are the same for all.
template <int kN>
__device__ void block_scan(long long (&v)[kN], long long (*warp_sums)[kMaxThreads / 32],
                           long long (&total)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const long long w = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += w;
    }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31)
    for (int k = 0; k < kN; ++k) warp_sums[k][warp] = v[k];
  __syncthreads();
  long long s[kN], p[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) p[k] = s[k] = lane < nw ? warp_sums[k][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const long long w = __shfl_up_sync(0xffffffffu, p[k], o);
      if (lane >= o) p[k] += w;
    }
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    total[k] = __shfl_sync(0xffffffffu, p[k], 31);
    v[k] += __shfl_sync(0xffffffffu, p[k] - s[k], warp);
  }
}

// Largest power of two below or at n, 0 for 0.
__device__ __forceinline__ int floor_pow2(int n) { return n > 0 ? 1 << (31 - __clz(n)) : 0; }

// For the warp's kBatch x 32 ascending values x[u] (lane after lane within u),
// the last index i in [0, n) with a[i] <= x, for a[0] <= x and a ascending.
// The whole array is searched for the first and the last value only; between
// them there are few requests, most often one.
template <int kBatch>
__device__ __forceinline__ void last_at_most(const int *a, int n, const int (&x)[kBatch],
                                             int (&at)[kBatch]) {
  const int lane = threadIdx.x & 31;
  const int end = __shfl_sync(0xffffffffu, lane == 0 ? x[0] : x[kBatch - 1], lane & 1 ? 31 : 0);
  int lo = 0;  // of the first value in even lanes, of the last in odd ones
  for (int step = floor_pow2(n - 1); step > 0; step >>= 1)
    if (lo + step < n && a[lo + step] <= end) lo += step;
  const int first = __shfl_sync(0xffffffffu, lo, 0), last = __shfl_sync(0xffffffffu, lo, 1);
#pragma unroll
  for (int u = 0; u < kBatch; ++u) at[u] = first;
  for (int step = floor_pow2(last - first); step > 0; step >>= 1) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = at[u] + step;
      if (i <= last && a[i] <= x[u]) at[u] = i;
    }
  }
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

template <int kBatch>
__global__ void __launch_bounds__(kMaxThreads, 1) kv_pages_kernel(const PagesArgs a) {
  extern __shared__ int sm[];
  int *s_q = sm, *s_need = s_q + a.B, *s_rel = s_need + a.B, *s_len = s_rel + a.B,
      *s_held = s_len + a.B, *s_ok = s_held + a.B;
  __shared__ long long warp_sums[2][kMaxThreads / 32];
  __shared__ int s_used;  // pages given out
  const int tid = threadIdx.x, nt = blockDim.x;
  const bool writer = blockIdx.x == 0;  // per-request outputs: one CTA
  const int P = a.num_pages;
  int head = __ldg(a.cursor_in), n_free = __ldg(a.cursor_in + 1);
  bool bad_cursor = head < 0 || head >= P || n_free < 0 || n_free > P;
  head = min(max(head, 0), P - 1);
  n_free = min(max(n_free, 0), P);

  if (tid == 0) s_used = 0;  // next touched past the first scan's barriers
  long long q_base = 0, need_base = 0, rel_base = 0;
  for (int b0 = 0; b0 < a.B; b0 += nt) {
    const int b = b0 + tid;
    const bool real = b < a.B;
    int n = 0, held = 0, L = 0, flags = bad_cursor && real ? SV_FLAG_PAGE_STATE : 0;
    bool ended = false;
    if (real) {
      const int wanted = __ldg(a.n_new + b), h = __ldg(a.held_in + b);
      long long grown = __ldg(a.len_in + b);
      if (a.n_commit) grown += (long long)__ldg(a.n_commit + b % a.n_commit_count) + a.n_commit_bias;
      ended = wanted < 0;
      n = max(wanted, 0);
      held = min(max(h, 0), a.max_pages);
      if (held != h) flags |= SV_FLAG_PAGE_STATE;
      const long long cap = (long long)held << a.page_shift;
      const long long Lc = min(max(grown, 0ll), cap);
      if (Lc != grown && !ended) flags |= SV_FLAG_REPLAY_RANGE;
      L = ended ? 0 : (int)Lc;
    }
    const int rel = ended ? held : 0;
    long long sums[2] = {n, rel}, totals[2];
    block_scan(sums, warp_sums, totals);
    const long long q_end = q_base + sums[0], q0 = q_end - n, rel_end = rel_base + sums[1];
    q_base += totals[0];
    rel_base += totals[1];
    const bool unfit = n > 0 && q_end > a.rows;
    const long long want = ((long long)L + n + (1 << a.page_shift) - 1) >> a.page_shift;
    const bool too_long = want > a.max_pages;
    const int need = (unfit || too_long || ended) ? 0 : (int)max(0ll, want - held);
    long long needs[1] = {need}, all[1];
    block_scan(needs, warp_sums, all);
    const long long need_end = need_base + needs[0];
    need_base += all[0];
    const bool no_pages = need > 0 && need_end > n_free;
    if (too_long || no_pages) flags |= SV_FLAG_NO_PAGES;
    if (unfit) flags |= SV_FLAG_ROWS;
    // served requests come before all that want pages in vain
    if (need > 0 && !no_pages) atomicMax(&s_used, (int)need_end);
    if (real) {
      s_q[b] = (int)min(q0, (long long)a.rows);
      s_need[b] = (int)min(need_end - need, (long long)P);  // past the served ones: not read
      s_rel[b] = (int)min(rel_end - rel, (long long)P);
      s_len[b] = L;
      s_held[b] = held;
      // bits 0..15 the flags; 16 refused; 17 ended
      s_ok[b] = flags | ((unfit || too_long || no_pages) ? 1 << 16 : 0) | (ended ? 1 << 17 : 0);
    }
  }
  const int rows_used = (int)min(q_base, (long long)a.rows);
  const int pages_back = (int)min(rel_base, (long long)(P - n_free));  // the ring's room
  // Every CTA has read the state; from here on it may be overwritten.
  if constexpr (kBatch == 1)
    __syncthreads();  // launched as one CTA
  else
    cluster_sync_all();
  const int pages_used = s_used;  // <= n_free <= P

  const int gt = blockIdx.x * nt + tid, gn = gridDim.x * nt;
  if (writer) {
    for (int b = tid; b < a.B; b += nt) {
      const int ok = s_ok[b], L = s_len[b], q0 = s_q[b];
      const int q1 = b + 1 < a.B ? s_q[b + 1] : rows_used;
      const bool refused = ok >> 16 & 1, ended = ok >> 17 & 1;
      const int got = refused || ended
                          ? 0
                          : max(0, ((L + (q1 - q0) + (1 << a.page_shift) - 1) >> a.page_shift) -
                                       s_held[b]);
      a.len_out[b] = L;
      a.held_out[b] = ended ? 0 : s_held[b] + got;
      a.q_start[b] = q0;
      a.kv_len[b] = refused ? 0 : L + (q1 - q0);
      if (a.err)
        a.err[b] = (ok & 0xFFFF) | (rel_base > pages_back && ended ? SV_FLAG_PAGE_STATE : 0);
    }
    if (tid == 0) {
      a.q_start[a.B] = rows_used;
      const long long h = (long long)head + pages_used;
      a.cursor_out[0] = (int)(h >= P ? h - P : h);
      a.cursor_out[1] = n_free - pages_used + pages_back;
    }
  }
  auto ring_at = [&](long long i) {  // entry i after head, 0 <= i <= P
    long long x = head + i;
    return (int)(x >= P ? x - P : x);
  };
  // a page a thread at a time: they are fewer
  const int lane = tid & 31;
  for (int i0 = gt; i0 - lane < pages_used; i0 += gn) {
    const int i[1] = {min(i0, pages_used - 1)};
    int b[1];
    last_at_most<1>(s_need, a.B, i, b);
    a.table[(size_t)b[0] * a.max_pages + s_held[b[0]] + (i[0] - s_need[b[0]])] =
        a.ring[ring_at(i[0])];
  }
  for (int i0 = gt; i0 - lane < pages_back; i0 += gn) {
    const int i[1] = {min(i0, pages_back - 1)};
    int b[1];
    last_at_most<1>(s_rel, a.B, i, b);
    a.ring[ring_at((long long)n_free + i[0])] =
        a.table[(size_t)b[0] * a.max_pages + (i[0] - s_rel[b[0]])];
  }
  // a warp takes 32 x kBatch consecutive rows at a time, their loads in flight
  // together; those past the end repeat the last
  const int w0 = (gt >> 5) * 32 * kBatch + lane, wn = (gn >> 5) * 32 * kBatch;
  for (int r0 = w0; r0 - lane < a.rows; r0 += wn) {
    int r[kBatch], b[kBatch], pos[kBatch], page[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) r[u] = min(r0 + u * 32, a.rows - 1);
    last_at_most<kBatch>(s_q, a.B, r, b);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int x = b[u];
      pos[u] = 0;
      page[u] = -1;
      if (r[u] < rows_used) {
        pos[u] = s_len[x] + (r[u] - s_q[x]);
        if (!(s_ok[x] >> 16 & 1)) {
          const int idx = pos[u] >> a.page_shift, held = s_held[x];
          page[u] = idx < held ? a.table[(size_t)x * a.max_pages + idx]
                               : a.ring[ring_at((long long)s_need[x] + (idx - held))];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      a.slots[r[u]] = (unsigned)page[u] < (unsigned)P
                          ? (page[u] << a.page_shift) + (pos[u] & ((1 << a.page_shift) - 1))
                          : -1;
      a.positions[r[u]] = pos[u];
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status kv_pages_step(const int32_t *length, const int32_t *held,
                                   const int32_t *cursor, const int32_t *n_new,
                                   const int32_t *n_commit, int n_commit_count, int n_commit_bias,
                                   int B, int page_size, int max_pages, int num_pages, int rows,
                                   int32_t *block_table, int32_t *ring, int32_t *length_out,
                                   int32_t *held_out, int32_t *cursor_out, int32_t *q_start,
                                   int32_t *kv_len, int32_t *slots, int32_t *positions,
                                   int32_t *err_flags, sv_stream_t stream) {
  clear_error();
  const char *who = "kv_pages_step";
  if (B < 0 || rows < 0 || max_pages < 1 || num_pages < 1)
    return fail(SV_ERR_INVALID_ARG,
                "%s: need B >= 0, rows >= 0, max_pages >= 1, num_pages >= 1 (B=%d rows=%d "
                "max_pages=%d num_pages=%d)",
                who, B, rows, max_pages, num_pages);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(SV_ERR_UNSUPPORTED, "%s: page_size=%d is not 16, 32, 64, 128 or 256", who,
                page_size);
  if (B > kMaxRequests) return fail(SV_ERR_UNSUPPORTED, "%s: B=%d > %d", who, B, kMaxRequests);
  if ((long long)max_pages * page_size + rows >= (1ll << 31) ||
      (long long)num_pages * page_size >= (1ll << 31))
    return fail(SV_ERR_UNSUPPORTED, "%s: positions or slots pass 31 bits", who);
  if (B == 0) return SV_OK;
  if (n_commit && (n_commit_count < 1 || n_commit_count > B))
    return fail(SV_ERR_INVALID_ARG, "%s: n_commit_count=%d outside [1, B=%d]", who,
                n_commit_count, B);
  if (!length || !held || !cursor || !n_new || !block_table || !ring || !length_out ||
      !held_out || !cursor_out || !q_start || !kv_len || (rows > 0 && (!slots || !positions)))
    return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  const size_t b4 = (size_t)B * 4, r4 = (size_t)rows * 4;
  struct Buf {
    const void *p;
    size_t n;
  };
  const Buf in[] = {{length, b4}, {held, b4}, {cursor, 8}, {n_new, b4},
                    {n_commit, (size_t)n_commit_count * 4}};
  const Buf out[] = {{length_out, b4}, {held_out, b4}, {cursor_out, 8},
                     {block_table, (size_t)B * max_pages * 4}, {ring, (size_t)num_pages * 4},
                     {q_start, b4 + 4}, {kv_len, b4}, {slots, r4}, {positions, r4},
                     {err_flags, b4}};
  for (const Buf &x : in)
    if (x.p && !aligned(x.p, 4)) return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  for (size_t i = 0; i < sizeof out / sizeof *out; ++i) {
    if (out[i].p && !aligned(out[i].p, 4))
      return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    for (size_t j = 0; j < sizeof in / sizeof *in; ++j) {
      if (i == j && i < 3 && out[i].p == in[j].p) continue;  // updated in place
      if (in[j].p && overlaps(out[i].p, out[i].n, in[j].p, in[j].n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
    }
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(SV_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  }
  PagesArgs a = {};
  a.len_in = length;
  a.held_in = held;
  a.cursor_in = cursor;
  a.n_new = n_new;
  a.n_commit = n_commit;
  a.n_commit_count = n_commit_count;
  a.n_commit_bias = n_commit_bias;
  a.B = B;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.rows = rows;
  a.table = block_table;
  a.ring = ring;
  a.len_out = length_out;
  a.held_out = held_out;
  a.cursor_out = cursor_out;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.slots = slots;
  a.positions = positions;
  a.err = err_flags;

  static PerDeviceOnce once;
  const cudaError_t ce = once.run([] {
    cudaError_t e = cudaFuncSetAttribute(
        kv_pages_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, 6 * kMaxRequests * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_pages_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               6 * kMaxRequests * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_pages_kernel<4>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                               1);
    return e;
  });
  if (ce != cudaSuccess)
    return fail(SV_ERR_CUDA, "%s: cudaFuncSetAttribute failed: %s", who, cudaGetErrorString(ce));
  // One CTA, a row a thread at a time, while its threads cover the rows and
  // requests twice over; beyond that a cluster of 16 (1000 requests with
  // 103502 rows: half as long again with eight).
  const int span = std::max(B, rows);
  const int threads = std::min(kMaxThreads, std::max(64, (span + 31) / 32 * 32));
  const bool wide = span > 2 * kMaxThreads;
  const int cluster = wide ? kCluster : 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)6 * B * 4;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = wide ? 1 : 0;  // a cluster attribute costs 0.4 us even for one CTA
  if (cudaLaunchKernelEx(&cfg, wide ? kv_pages_kernel<4> : kv_pages_kernel<1>, a) != cudaSuccess)
    return fail(SV_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(cudaGetLastError()));
  return check_launch(who);
}
