// paged_attn.cu -- attention of a step's new tokens over a paged cache,
// sm_103a: the entry point, and the kernel for few rows (single tokens and
// verify blocks); the mathematics and the split of work are in attn_common.cuh.
//
// Few rows read each key and value once and do little with it: D products and
// sums per row against 4 D bytes, so streaming the cache bounds it.  A CTA
// takes a run of 64-key tiles (attn_common.cuh): one producer warp copies them
// with TMA, page by page, 128-byte swizzled, into a ring of key and value
// slots; four consumer warps hold 16 rows each in registers and multiply with
// mma.sync (16 x 8 x 16): kRowGroups warps side by side in rows, the others
// splitting a tile's keys, each with its own running maximum and sum (no
// barrier per tile), joined through shared memory at the end of an item.  The
// rows of the G query heads of a kv head are packed together, so a key read
// once serves them all.  Scores, maxima, sums and outputs are fp32; weights
// are rounded to bf16 for the second product (at most half a step, 2^-8 of
// each weight, the type of the values they multiply), their sum is not.
//
// CTAs that share an item leave partial results, which a second launch joins
// (attn_join_kernel below), in an order that does not depend on the run.
//
// Measured (GB300, head dim 128 unless said): 4 rows over 100,005 positions of
// 40 kv heads 297 us (6.9 TB/s, a plain copy's rate), 32 requests' 4 rows over
// ragged contexts 153 us (6.2 TB/s), 16 single tokens at head dim 256 76 us
// (5.3 TB/s); one token over 999 positions 10.4 to 11.5 us: two launches and the
// dependent trips to memory of each, not the 4 MB of keys and values.
#include <algorithm>

#include "attn_common.cuh"
#include "attn_host.h"
#include "qmv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace attn {

namespace {

constexpr int kBK = 64;  // keys per tile
constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kConsumers = kWarps * 32;
// An item's cost beside its tiles (queries, joining the warps, the output: about
// 6 us, of which the ring's two tiles hide some), in key tiles, when the work is
// cut into runs.  With 2, 4 and 5: 32 verify blocks over 200 to 30,000 positions
// 163, 153 and 150 us, 300 tokens over 20 to 3000 at head dim 256 156, 138 and
// 134, 48 blocks of 40 kv heads 257, 242 and 245, one request of one kv head over
// 100,000 28.7, 28.9 and 30.9, one token over 999 10.7, 11.5 and 11.5.
constexpr int kItemUnits = 4;

template <int D>
struct RowsShape {
  static constexpr uint32_t kSlotBytes = kBK * D * 2;    // a tile's keys, or its values
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kOutStride = D + 8;               // floats: rows 8 banks apart
  static constexpr uint32_t kOutBytes = kWarps * 16 * kOutStride * 4;
  static constexpr uint32_t kSmem = kSlots * kSlotBytes + kOutBytes + 1024;
  static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

// Key tiles of every item of a request: enough for its longest row tile, so
// that items can be found by division; an item's own tiles come first, the
// rest of them is empty.
__device__ __forceinline__ int tiles_per_item(const Args &a, const Request &q, int tile_rows) {
  long long tiles = (q.len + kBK - 1) / kBK;
  if (a.window > 0)
    tiles = min(tiles, ((long long)a.window + tile_rows / a.G + 2 + kBK - 1) / kBK + 1);
  return (int)max(tiles, 1ll);
}
__device__ __forceinline__ long long request_units(const Args &a, const Request &q,
                                                   int tile_rows) {
  const long long nt = ((long long)q.n * a.G + tile_rows - 1) / tile_rows;
  return nt * a.Hkv * (tiles_per_item(a, q, tile_rows) + kItemUnits);
}

struct Segment {
  Request rq;
  int b, h, r0, count;  // rows [r0, r0 + count) of kv head h of request b
  Span span;
  int tile0, tiles;     // key tiles [tile0, tile0 + tiles) (may be none)
  long long item;       // first unit of the item
  int first, width;     // the segment's first tile of the item, the item's tiles
  bool whole;
};

// Walks a run's segments in order.  An item is its tiles and then kItemUnits
// more; a run that ends among those takes the item to its end, and one that
// begins there leaves it alone, so only tiles are ever split.
struct Walk {
  long long u, end, base;  // next unit, end of the run, first unit of request b
  int b;
  __device__ bool next(const Args &a, int tile_rows, Segment &s) {
    for (;;) {
      if (u >= end) return false;
      for (;;) {
        s.rq = load_request(a, b);
        const long long size = request_units(a, s.rq, tile_rows);
        if (u - base < size) break;
        base += size;
        ++b;
      }
      s.width = tiles_per_item(a, s.rq, tile_rows);
      const long long item = (u - base) / (s.width + kItemUnits);
      s.item = base + item * (s.width + kItemUnits);
      s.h = (int)(item % a.Hkv);
      s.r0 = (int)(item / a.Hkv) * tile_rows;
      s.first = (int)(u - s.item);
      if (s.first < s.width) break;
      u = s.item + s.width + kItemUnits;
    }
    const int n = (int)min((long long)(s.width - s.first), end - u);
    s.b = b;
    s.count = min(tile_rows, s.rq.n * a.G - s.r0);
    s.span = rows_span(a, s.rq, s.r0, s.count);
    s.whole = n == s.width;
    s.tile0 = s.span.lo / kBK + s.first;
    s.tiles = max(0, min((s.span.hi + kBK - 1) / kBK - s.tile0, n));
    u = s.first + n == s.width ? s.item + s.width + kItemUnits : u + n;
    return true;
  }
};

// Adds to the rows' sums in shared memory the non-finite values that the tiles
// left out (see clear_nonfinite), a row a warp at a time, into the sums of the
// warps whose maximum is the row's.
template <int D, int kRowGroups>
__device__ __noinline__ void add_nonfinite(const Args &a, const Segment &s, float *s_out,
                                           const float (*s_m)[16]) {
  constexpr int kKeyGroups = kWarps / kRowGroups, E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int rr = warp; rr < s.count; rr += kWarps) {
    const int t = (s.r0 + rr) / a.G, g = s.r0 + rr - t * a.G;
    const int last = s.rq.len - s.rq.n + t;
    const int lo = max(max(s.span.lo, s.tile0 * kBK), a.window > 0 ? last - a.window + 1 : 0);
    const int hi = min(min(s.span.hi, (s.tile0 + s.tiles) * kBK), last + 1);
    const __nv_bfloat16 *q = a.q + (long long)(s.rq.q0 + t) * a.q_stride +
                             (long long)(s.h * a.G + g) * D + lane * E;
    int w = (rr >> 4) * kKeyGroups;
    for (int i = w + 1; i < (rr >> 4) * kKeyGroups + kKeyGroups; ++i)
      if (s_m[i][rr & 15] > s_m[w][rr & 15]) w = i;
    float *sums = s_out + (w * 16 + (rr & 15)) * RowsShape<D>::kOutStride + lane * E;
    for (int j = lo; j < hi; ++j) {
      if (j >= s.span.all_lo && j < s.span.all_hi) {
        j = s.span.all_hi - 1;
        continue;
      }
      const long long at = position_at(a, s.b, s.h, j, D);
      if (at < 0) continue;  // zeros
      const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v + at + lane * E);
      uint32_t odd = 0;
#pragma unroll
      for (int e = 0; e < E; e += 2) odd |= nonfinite_bits(v[e / 2]);
      if (!__any_sync(0xffffffffu, odd)) continue;
      float score = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        score = fmaf(__bfloat162float(q[e]), __bfloat162float(a.k[at + lane * E + e]), score);
      score = warp_sum(score);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 y = two_floats(v[e / 2]);
        sums[e] = add_if_nonfinite(sums[e], y.x, score == kNegInf);
        sums[e + 1] = add_if_nonfinite(sums[e + 1], y.y, score == kNegInf);
      }
    }
  }
}

template <int D, int kRowGroups>
__global__ void __launch_bounds__(kThreads, RowsShape<D>::kCtasPerSm)
    attn_rows_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  using S = RowsShape<D>;
  constexpr int kKeyGroups = kWarps / kRowGroups;
  constexpr int kWarpKeys = kBK / kKeyGroups;  // 16, 32 or 64
  constexpr int kTileRows = 16 * kRowGroups;
  constexpr int kSteps = D / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[S::kSlots], empty[S::kSlots];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  __shared__ long long s_scan[kThreads / 32], s_base;
  __shared__ int s_b, s_nonfinite, s_more;
  __shared__ Runs s_runs;
  __shared__ Walk s_walk;  // the consumers': their registers hold the tiles
  __shared__ Segment s;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = raw + ((1024u - (raw & 1023u)) & 1023u);
  float *s_out = reinterpret_cast<float *>(smem_raw + (ring - raw) + S::kSlots * S::kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    s_nonfinite = 0;
    fence_mbar_init();
  }
  // ---- this CTA's run of units, and the request that it begins in ----
  Runs runs;
  auto block_sum = [&](long long v, long long &upto) {  // inclusive scan and total
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    long long all = 0;
    upto = v;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) upto += s_scan[i];
      all += s_scan[i];
    }
    return all;
  };
  auto units_of = [&](int b) {
    return b < a.B ? request_units(a, load_request(a, b), kTileRows) : 0;
  };
  long long size = units_of(tid), upto;  // the first block of requests, kept for the search
  long long all = block_sum(size, upto);
  runs.units = all;
  for (int b0 = kThreads; b0 < a.B; b0 += kThreads) {
    long long past;
    runs.units += block_sum(units_of(b0 + tid), past);
  }
  runs.ctas = (int)min((long long)gridDim.x, runs.units);
  // rows past the last request's: zero
  const int used = min(max(__ldg(a.q_start + a.B), 0), a.rows);
  for (int r = used + blockIdx.x; r < a.rows; r += gridDim.x) {
    for (int i = tid; i < a.Hq * (D / 8); i += kThreads)
      reinterpret_cast<uint4 *>(a.out + (long long)r * a.out_stride)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(long long)r * a.Hq + i] = kNegInf;
  }
  pdl_launch_dependents();
  if (tid == 0) a.splits[blockIdx.x].n = 0;
  if ((int)blockIdx.x >= runs.ctas) return;  // uniform
  Walk walk;
  walk.u = runs.begin(blockIdx.x);
  walk.end = runs.begin(blockIdx.x + 1);
  long long before = 0;  // units of the blocks of requests already searched
  for (int b0 = 0;;) {
    if (before + upto > walk.u && before + upto - size <= walk.u) {
      s_b = b0 + tid;
      s_base = before + upto - size;
    }
    b0 += kThreads;
    if (b0 >= a.B) break;
    before += all;
    size = units_of(b0 + tid);
    all = block_sum(size, upto);
  }
  __syncthreads();
  walk.b = s_b;
  walk.base = s_base;

  uint32_t slot = 0, phase = 0;  // of the next ring slot
  auto advance = [&] {
    if (++slot == (uint32_t)S::kSlots) {
      slot = 0;
      phase ^= 1u;
    }
  };
  bool dead = false;  // a wait gave up: the rest runs without waiting, results are invalid

  if (warp == kWarps) {
    // ------------------------------ producer ------------------------------
    const int per_page = min(kBK, 1 << a.page_shift);  // rows of one copy
    const int pages = kBK / per_page;
    const int boxes = pages * (D / 64);
    const int blk = lane / pages, pg = lane - blk * pages;
    long long issued = 0;
    Segment x;
    while (walk.next(a, kTileRows, x)) {
      for (int t = 0; t < x.tiles; ++t) {
        const int j = (x.tile0 + t) * kBK + pg * per_page;
        int y = 0;
        if (lane < boxes)
          y = page_row(a, x.b, x.h, j >> a.page_shift, x.span.lo, x.span.hi) +
              (j & ((1 << a.page_shift) - 1));
        for (int kv = 0; kv < 2; ++kv) {
          if (issued >= S::kSlots && !dead && !mbar_wait(&empty[slot], phase ^ 1u)) dead = true;
          dead = __any_sync(0xffffffffu, dead);
          if (dead) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], S::kSlotBytes);
          __syncwarp();
          if (lane < boxes)
            tma_load_rows(ring + slot * S::kSlotBytes + (uint32_t)blk * (kBK * 128) +
                              (uint32_t)pg * per_page * 128,
                          kv ? &vmap : &kmap, blk * 64, y, smem_addr(&full[slot]));
          ++issued;
          advance();
        }
        if (dead) break;
      }
      if (dead) break;
    }
    if (dead && lane == 0) report_give_up(1u);
    // every copy has landed before the CTA may exit
    for (long long k = max(0ll, issued - S::kSlots); k < issued; ++k)
      (void)mbar_wait(&full[k % S::kSlots], (uint32_t)((k / S::kSlots) & 1));
    return;
  }

  // ------------------------------- consumers ------------------------------
  const int wr = warp / kKeyGroups, wk = warp % kKeyGroups;
  const int gq = lane >> 2, gc = lane & 3;  // row and column pair of an accumulator
  // ldmatrix rows of this lane: keys for the first product, keys for the second
  const int k_key = wk * kWarpKeys + ((lane >> 4) << 3) + (lane & 7), k_half = (lane >> 3) & 1;
  const int v_key = wk * kWarpKeys + (lane & 15), v_half = lane >> 4;
  auto wait_full = [&] {
    if (!dead && !mbar_wait(&full[slot], phase)) {
      dead = true;
      report_give_up(2u);
    }
  };

  if (tid == 0) {
    s_walk = walk;
    s_runs = runs;
  }
  for (;;) {
    if (tid == 0) s_more = s_walk.next(a, kTileRows, s);
    consumer_sync();
    if (!s_more) break;
    // queries as A fragments; rows past the tile are zero
    uint32_t qf[kSteps][4];
    int last[2], first[2];  // positions that rows gq and gq + 8 attend: first .. last
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = wr * 16 + gq + 8 * i;
      const int r = s.r0 + rr;
      const int t = r / a.G, g = r - t * a.G;
      const bool ok = rr < s.count;
      last[i] = ok ? s.rq.len - s.rq.n + t : -1;
      first[i] = a.window > 0 ? last[i] - a.window + 1 : 0;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(
          a.q + (long long)(s.rq.q0 + (ok ? t : 0)) * a.q_stride +
          (long long)(s.h * a.G + (ok ? g : 0)) * D);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        qf[k][i] = ok ? __ldg(src + k * 8 + gc) : 0u;
        qf[k][2 + i] = ok ? __ldg(src + k * 8 + 4 + gc) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};

    for (int t = 0; t < s.tiles; ++t) {
      const int j0 = (s.tile0 + t) * kBK;
      const bool masked = j0 < s.span.all_lo || j0 + kBK > s.span.all_hi;
      // ---- scores of this warp's keys ----
      float x[kWarpKeys / 8][4];
#pragma unroll
      for (int n = 0; n < kWarpKeys / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
      wait_full();
      uint32_t base = ring + slot * S::kSlotBytes;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int c = 2 * k + k_half;  // 16-byte column of the key row
#pragma unroll
        for (int n = 0; n < kWarpKeys / 16; ++n) {
          const int key = k_key + 16 * n;
          uint32_t f[4];
          qmv::ldmatrix_x4(f, base + (uint32_t)(c >> 3) * (kBK * 128) + (uint32_t)key * 128 +
                                  (uint32_t)(((c & 7) ^ (key & 7)) << 4));
          mma_bf16_m16n8k16(x[2 * n], qf[k][0], qf[k][1], qf[k][2], qf[k][3], f[0], f[1]);
          mma_bf16_m16n8k16(x[2 * n + 1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], f[2], f[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      advance();
      if (masked) {
#pragma unroll
        for (int n = 0; n < kWarpKeys / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + wk * kWarpKeys + n * 8 + gc * 2 + (e & 1);
            if (j < first[e >> 1] || j > last[e >> 1]) x[n][e] = kNegInf;
          }
      }
      // ---- running maximum and sum, weights ----
      float keep[2];
      uint32_t p[kWarpKeys / 8][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = kNegInf;
#pragma unroll
        for (int n = 0; n < kWarpKeys / 8; ++n) mx = fmaxf(mx, fmaxf(x[n][2 * i], x[n][2 * i + 1]));
        const float mn = fmaxf(m[i], quad_max(mx));
        const float ms = mn == kNegInf ? 0.f : mn;
        keep[i] = exp2_approx((m[i] - ms) * a.scale_log2);
        m[i] = mn;
        const float off = ms * a.scale_log2;
        float sum_p = 0.f;
#pragma unroll
        for (int n = 0; n < kWarpKeys / 8; ++n) {
          const float p0 = exp2_approx(fmaf(x[n][2 * i], a.scale_log2, -off));
          const float p1 = exp2_approx(fmaf(x[n][2 * i + 1], a.scale_log2, -off));
          sum_p += p0 + p1;
          p[n][i] = pack_bf16(p0, p1);
        }
        l[i] = l[i] * keep[i] + sum_p;
      }
      if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][0] *= keep[0];
          o[d][1] *= keep[0];
          o[d][2] *= keep[1];
          o[d][3] *= keep[1];
        }
      }
      // ---- weights times values ----
      wait_full();
      base = ring + slot * S::kSlotBytes;
      if (masked) {
        // places no row attends may hold anything: zero, so that a weight of
        // zero meets no NaN, and so is what is not finite where some rows attend
        // and others do not (added to their sums at the end)
        consumer_sync();
        const int key = tid >> 1, pos = j0 + key;
        const bool none = pos < s.span.lo || pos >= s.span.hi;
        if (none || pos < s.span.all_lo || pos >= s.span.all_hi) {
          bool odd = false;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint4 *at = reinterpret_cast<uint4 *>(
                smem_raw + (base - raw) + (size_t)((tid & 1) * (D / 16) + c) / 8 * (kBK * 128) +
                key * 128 + ((((tid & 1) * (D / 16) + c) & 7) << 4));
            if (none) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              uint4 v = *at;
              if (nonfinite_bits(v)) {
                clear_nonfinite(v);
                *at = v;
                odd = true;
              }
            }
          }
          if (odd) s_nonfinite = 1;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        consumer_sync();
      }
#pragma unroll
      for (int n = 0; n < kWarpKeys / 16; ++n) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const int key = v_key + 16 * n, c = 2 * d + v_half;
          uint32_t f[4];
          ldmatrix_x4_trans(f, base + (uint32_t)(c >> 3) * (kBK * 128) + (uint32_t)key * 128 +
                                   (uint32_t)(((c & 7) ^ (key & 7)) << 4));
          mma_bf16_m16n8k16(o[2 * d], p[2 * n][0], p[2 * n][1], p[2 * n + 1][0], p[2 * n + 1][1],
                            f[0], f[1]);
          mma_bf16_m16n8k16(o[2 * d + 1], p[2 * n][0], p[2 * n][1], p[2 * n + 1][0],
                            p[2 * n + 1][1], f[2], f[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      advance();
    }

    // ---- the warps' sums to shared memory ----
    consumer_sync();  // s_out of the segment before has been read, s_nonfinite is written
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] = quad_sum(l[i]);
      if (gc == 0) {
        s_m[warp][gq + 8 * i] = m[i];
        s_l[warp][gq + 8 * i] = l[i];
      }
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2 *>(
            &s_out[(warp * 16 + gq + 8 * i) * S::kOutStride + d * 8 + gc * 2]) =
            make_float2(o[d][2 * i], o[d][2 * i + 1]);
    }
    const bool odd = s_nonfinite != 0;
    consumer_sync();
    if (odd) {
      add_nonfinite<D, kRowGroups>(a, s, s_out, s_m);
      if (tid == 0) s_nonfinite = 0;  // next written after the next segment's barrier
      consumer_sync();
    }

    float *part = partial_at(a, 2 * (int)blockIdx.x + (s.first == 0 ? 1 : 0), kTileRows, D);
    for (int i = tid; i < s.count * (D / 4); i += kConsumers) {
      const int rr = i / (D / 4), d = 4 * (i - rr * (D / 4));
      const int w0 = (rr >> 4) * kKeyGroups;
      float mm = kNegInf, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kKeyGroups; ++w) mm = fmaxf(mm, s_m[w0 + w][rr & 15]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kKeyGroups; ++w) {
        const float mw = s_m[w0 + w][rr & 15];
        if (mw == kNegInf && s_l[w0 + w][rr & 15] == 0.f) continue;  // no keys
        const float f = exp2_approx((mw - mm) * a.scale_log2);
        const float4 v = *reinterpret_cast<const float4 *>(
            &s_out[((w0 + w) * 16 + (rr & 15)) * S::kOutStride + d]);
        ll = fmaf(s_l[w0 + w][rr & 15], f, ll);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (s.whole) {
        store_out4<D>(a, s.rq.q0, s.h, s.r0 + rr, d, acc, mm, ll);
      } else {
        __stcg(reinterpret_cast<float4 *>(part + rr * D + d), acc);
        if (d == 0) {
          __stcg(part + kTileRows * D + rr, mm);
          __stcg(part + kTileRows * (D + 1) + rr, ll);
        }
      }
    }
    if (tid == 0 && s.first == 0 && !s.whole)
      a.splits[blockIdx.x] = SplitItem{s_runs.owner(s.item + s.width - 1) - (int)blockIdx.x + 1,
                                       s.rq.q0, s.h, s.r0, s.count, {0, 0, 0}};
    consumer_sync();  // the segment has been read
  }
}

// ---- joining split items ------------------------------------------------------
// With M the largest of an item's partials' maxima, each row's
//   out = sum_k 2^(c (m_k - M)) O_k / sum_k 2^(c (m_k - M)) l_k.
// The partials are a few megabytes in L2 and each is read once: latency is the
// cost.  A piece of work is a few rows of an item, the fewer the more partials
// it has; a block's threads split the partials of a row among them, keep eight
// loads in flight each and have the first on their way before the weights are
// known; every block finds its pieces by itself from the items' list.
// (Joining in the CTA that finishes last instead took 5 us for 16 partials of
// five rows and 60 us for 304: a fence, an atomic and one SM's latency.)
constexpr int kJoinThreads = 512;
constexpr int kJoinDepth = 8;                // loads in flight a thread
constexpr int kJoinWeights = 4 * kMaxCtas;   // rows of a piece x partials, at most

// Rows of a piece of an item with n partials: a power of two of thread groups
// that take kJoinDepth partials each, but four rows at least.
__device__ __forceinline__ int piece_rows(int n, int D) {
  int rows = kJoinThreads / (D / 4);
  while (rows > 4 && rows * (D / 4) * n > kJoinThreads * kJoinDepth) rows >>= 1;
  return rows;
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2)
    attn_join_kernel(const __grid_constant__ Args a, int ctas, int tile_rows) {
  __shared__ float s_f[kJoinWeights], s_l[kJoinWeights];
  __shared__ float4 s_sum[kJoinThreads];
  __shared__ int s_end[kMaxCtas], s_warp[kJoinThreads / 32];
  static_assert(kMaxCtas <= kJoinThreads, "an item a thread");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // pieces up to and with each CTA's item
  int pieces = 0;
  if (tid < ctas && a.splits[tid].n > 0) {
    const int rows = piece_rows(a.splits[tid].n, D);
    pieces = (a.splits[tid].count + rows - 1) / rows;
  }
  if (!__syncthreads_or(pieces)) return;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xffffffffu, pieces, o);
    if (lane >= o) pieces += w;
  }
  if (lane == 31) s_warp[warp] = pieces;
  __syncthreads();
  int total = 0;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < warp) pieces += s_warp[i];
    total += s_warp[i];
  }
  if (tid < ctas) s_end[tid] = pieces;
  __syncthreads();

  for (int piece = blockIdx.x; piece < total; piece += gridDim.x) {
    int c0 = 0, hi = ctas - 1;  // the first item whose pieces end after this one
    while (c0 < hi) {
      const int mid = (c0 + hi) >> 1;
      if (s_end[mid] > piece)
        hi = mid;
      else
        c0 = mid + 1;
    }
    const SplitItem it = a.splits[c0];
    const int most = piece_rows(it.n, D);
    const int row0 = (piece - (c0 > 0 ? s_end[c0 - 1] : 0)) * most;
    const int rows = min(most, it.count - row0);
    const int items = rows * (D / 4);         // at most kJoinThreads
    const int groups = kJoinThreads / items;  // of partials
    const int i = tid % items, group = tid / items;
    const int rr = i / (D / 4), d = 4 * (i % (D / 4));
    // partial k: the first CTA's second place, the others' first
    auto part = [&](int k) { return partial_at(a, 2 * (c0 + k) + (k == 0 ? 1 : 0), tile_rows, D); };
    float4 v[kJoinDepth];
    auto load = [&](int k0) {
#pragma unroll
      for (int u = 0; u < kJoinDepth; ++u)
        if (group < groups && k0 + u * groups < it.n)
          v[u] = __ldcg(reinterpret_cast<const float4 *>(part(k0 + u * groups) +
                                                         (row0 + rr) * D + d));
    };
    load(group);
    for (int j = tid; j < it.n * rows; j += kJoinThreads) {
      const int k = j / rows;
      const float *ml = part(k) + tile_rows * D + row0 + (j - k * rows);
      s_f[j] = __ldcg(ml);
      s_l[j] = __ldcg(ml + tile_rows);
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kJoinThreads / 32) {
      float m = kNegInf, l = 0.f;
      for (int k = lane; k < it.n; k += 32) m = fmaxf(m, s_f[k * rows + r]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      for (int k = lane; k < it.n; k += 32) {
        const float lk = s_l[k * rows + r], f = join_weight(a, s_f[k * rows + r], lk, m);
        l = fmaf(lk, f, l);
        s_f[k * rows + r] = f;
      }
      l = warp_sum(l);
      __syncwarp();
      if (lane == 0) {  // at least two partials
        s_l[r] = m;
        s_l[rows + r] = l;
      }
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = group; group < groups;) {
#pragma unroll
      for (int u = 0; u < kJoinDepth; ++u)
        if (k0 + u * groups < it.n) {
          const float f = s_f[(k0 + u * groups) * rows + rr];
          acc.x = fmaf(v[u].x, f, acc.x);
          acc.y = fmaf(v[u].y, f, acc.y);
          acc.z = fmaf(v[u].z, f, acc.z);
          acc.w = fmaf(v[u].w, f, acc.w);
        }
      k0 += kJoinDepth * groups;
      if (k0 >= it.n) break;
      load(k0);
    }
    s_sum[tid] = acc;
    __syncthreads();
    if (group == 0) {
      for (int g = 1; g < groups; ++g) {
        const float4 x = s_sum[g * items + i];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      store_out4<D>(a, it.q0, it.h, it.r0 + row0 + rr, d, acc, s_l[rr], s_l[rows + rr]);
    }
    __syncthreads();
  }
}

template <int D>
sv_status join(const Args &a, int ctas, int tile_rows, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * device_sm_count()));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, a, ctas, tile_rows) != cudaSuccess)
    return fail(SV_ERR_CUDA, "paged_attention: join launch failed: %s",
                cudaGetErrorString(cudaGetLastError()));
  return check_launch("paged_attention (join)");
}

template <int D, int kRowGroups>
sv_status launch_rows(const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a, int ctas,
                      cudaStream_t stream) {
  using S = RowsShape<D>;
  static PerDeviceOnce once;
  const cudaError_t ce = once.run([] {
    return cudaFuncSetAttribute(attn_rows_kernel<D, kRowGroups>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  });
  if (ce != cudaSuccess)
    return fail(SV_ERR_CUDA, "paged_attention: cudaFuncSetAttribute failed: %s",
                cudaGetErrorString(ce));
  attn_rows_kernel<D, kRowGroups><<<(unsigned)ctas, kThreads, S::kSmem, stream>>>(kmap, vmap, a);
  const sv_status st = check_launch("paged_attention");
  return st == SV_OK ? join<D>(a, ctas, 16 * kRowGroups, stream) : st;
}

template <int D>
sv_status launch_rows(int groups, const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a,
                      int ctas, cudaStream_t stream) {
  if (groups == 1) return launch_rows<D, 1>(kmap, vmap, a, ctas, stream);
  if (groups == 2) return launch_rows<D, 2>(kmap, vmap, a, ctas, stream);
  return launch_rows<D, 4>(kmap, vmap, a, ctas, stream);
}

size_t split_bytes() { return (size_t)kMaxCtas * sizeof(SplitItem); }
int rows_ctas(int D) { return std::min(kMaxCtas, device_sm_count() * (D == 256 ? 1 : 2)); }

size_t workspace_bytes(int D) {
  size_t part = (size_t)rows_ctas(D) * 2 * 64 * (D + 2) * 4;
  part = std::max(part, D == 256 ? tc256_partial_bytes() : tc_partial_bytes(D));
  return kCounterBytes + split_bytes() + part;
}

}  // namespace
}  // namespace attn

unsigned take_device_error_attn() {
  unsigned v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, attn::g_give_up, sizeof v);
  cudaMemcpyToSymbol(attn::g_give_up, &zero, sizeof zero);
  return v | attn::tc_take_give_up() | attn::tc256_take_give_up();
}

}  // namespace sv

using namespace sv;

extern "C" size_t paged_attention_workspace_bytes(int D) {
  clear_error();
  if (D != 64 && D != 128 && D != 256) {
    fail(SV_ERR_UNSUPPORTED, "paged_attention_workspace_bytes: D=%d is not 64, 128 or 256", D);
    return 0;
  }
  return attn::workspace_bytes(D);
}

extern "C" sv_status paged_attention(const uint16_t *q, long long q_row_stride,
                                     const uint16_t *k_cache, const uint16_t *v_cache,
                                     const int32_t *block_table, const int32_t *q_start,
                                     const int32_t *kv_len, int B, int rows, int max_new, int Hq,
                                     int Hkv, int D, int page_size, int num_pages, int max_pages,
                                     float scale, int window, uint16_t *out,
                                     long long out_row_stride, float *lse, void *workspace,
                                     size_t workspace_bytes, sv_stream_t stream) {
  clear_error();
  const char *who = "paged_attention";
  if (B < 0 || rows < 0 || max_new < 0 || Hq < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1)
    return fail(SV_ERR_INVALID_ARG,
                "%s: need B, rows, max_new >= 0 and Hq, Hkv, num_pages, max_pages >= 1 (B=%d "
                "rows=%d max_new=%d Hq=%d Hkv=%d num_pages=%d max_pages=%d)",
                who, B, rows, max_new, Hq, Hkv, num_pages, max_pages);
  if (Hq % Hkv) return fail(SV_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of Hkv=%d", who, Hq, Hkv);
  if (D != 64 && D != 128 && D != 256)
    return fail(SV_ERR_UNSUPPORTED, "%s: D=%d is not 64, 128 or 256", who, D);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(SV_ERR_UNSUPPORTED, "%s: page_size=%d is not 16, 32, 64, 128 or 256", who,
                page_size);
  if (!(scale > 0.f) || scale > 2.0e38f)  // times log2(e) finite as well
    return fail(SV_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
  if (window < 0) return fail(SV_ERR_INVALID_ARG, "%s: window must be >= 0", who);
  if (((long long)num_pages + 1) * Hkv * page_size >= (1ll << 31) ||
      (long long)max_pages * page_size + rows + 256 >= (1ll << 31))
    return fail(SV_ERR_UNSUPPORTED, "%s: cache rows or positions pass 31 bits", who);
  if ((long long)rows * (Hq / Hkv) + 256 >= (1ll << 31) || Hq > 65536)
    return fail(SV_ERR_UNSUPPORTED, "%s: too many rows or heads", who);
  if (B == 0 || rows == 0) return SV_OK;
  if (!q || !k_cache || !v_cache || !block_table || !q_start || !kv_len || !out || !workspace)
    return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (q_row_stride < (long long)Hq * D || out_row_stride < (long long)Hq * D)
    return fail(SV_ERR_INVALID_ARG, "%s: a row stride is smaller than its row", who);
  if (q_row_stride % 8 || out_row_stride % 8)
    return fail(SV_ERR_INVALID_ARG, "%s: row strides must be multiples of 16 bytes", who);
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return fail(SV_ERR_INVALID_ARG, "%s: q, the caches and out must be 16-byte aligned", who);
  if (!aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      (lse && !aligned(lse, 4)))
    return fail(SV_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  if (!aligned(workspace, 256))
    return fail(SV_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  const size_t need = attn::workspace_bytes(D);
  if (workspace_bytes < need)
    return fail(SV_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, workspace_bytes,
                need);
  const size_t cache = (size_t)num_pages * Hkv * page_size * D * 2;
  struct Buf {
    const void *p;
    size_t n;
  };
  const Buf in[] = {{q, ((size_t)(rows - 1) * q_row_stride + (size_t)Hq * D) * 2},
                    {k_cache, cache}, {v_cache, cache},
                    {block_table, (size_t)B * max_pages * 4}, {q_start, ((size_t)B + 1) * 4},
                    {kv_len, (size_t)B * 4}};
  const Buf outs[] = {{out, ((size_t)(rows - 1) * out_row_stride + (size_t)Hq * D) * 2},
                      {lse, (size_t)rows * Hq * 4}, {workspace, need}};
  for (int i = 0; i < 3; ++i) {
    for (const Buf &b : in)
      if (overlaps(outs[i].p, outs[i].n, b.p, b.n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return fail(SV_ERR_INVALID_ARG, "%s: two of out, lse and workspace overlap", who);
  }
  attn::Args a = {};
  a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  a.k = reinterpret_cast<const __nv_bfloat16 *>(k_cache);
  a.v = reinterpret_cast<const __nv_bfloat16 *>(v_cache);
  a.q_stride = q_row_stride;
  a.out_stride = out_row_stride;
  a.out = reinterpret_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.table = block_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.B = B;
  a.rows = rows;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  // a window of every position is none (and positions minus it stay in 32 bits)
  a.window = window >= max_pages * page_size ? 0 : window;
  a.scale = scale;
  a.scale_log2 = scale * 1.44269504088896340736f;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.counters = reinterpret_cast<unsigned *>(ws);
  a.splits = reinterpret_cast<attn::SplitItem *>(ws + attn::kCounterBytes);
  a.partials = reinterpret_cast<float *>(ws + attn::kCounterBytes + attn::split_bytes());

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // More rows a kv head than a 64-row tile of the streaming kernel holds go to
  // the tensor-core kernels (their tiles are 128 rows).
  const long long most = (long long)std::min(max_new, rows) * a.G;
  if (most > 64) return D == 256 ? attn::tc256_run(a, s) : attn::tc_run(D, a, s);
  CUtensorMap kmap, vmap;
  sv_status st = attn::encode_cache(&kmap, a.k, D, a, attn::kBK);
  if (st == SV_OK) st = attn::encode_cache(&vmap, a.v, D, a, attn::kBK);
  if (st != SV_OK) return st;
  // Row tiles of 16, 32 or 64 rows, the least that holds a request's rows.
  const int groups = most <= 16 ? 1 : most <= 32 ? 2 : 4;
  const int ctas = attn::rows_ctas(D);
  if (D == 64) return attn::launch_rows<64>(groups, kmap, vmap, a, ctas, s);
  if (D == 128) return attn::launch_rows<128>(groups, kmap, vmap, a, ctas, s);
  return attn::launch_rows<256>(groups, kmap, vmap, a, ctas, s);
}
