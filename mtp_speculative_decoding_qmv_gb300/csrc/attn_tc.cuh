// attn_tc.cuh -- shared by the tensor-core attention kernels: the cut of the
// work into items of kRows packed rows of a kv head, packed fp32 arithmetic,
// and the joining of split items.
#pragma once
#include <cstdint>

#include "attn_common.cuh"
#include "tc05.cuh"

namespace sv {
namespace attn {
namespace {

constexpr int kBK = 128;         // keys per tile
constexpr int kTile = 128;       // rows per tensor-core tile
constexpr int kMmaWarp = 8, kTmaWarp = 9, kQueryWarp = 10;
// The softmax groups take registers from the third warpgroup (launched at 168 a
// thread: 256 x 216 + 128 x 72 = 384 x 168).
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr uint32_t kTmemCols = 512;
// An item's cost beside its tiles (queries, the first scores, the last
// products, the output), in key tiles, when the work is cut into runs: 6.6 us
// or 4.6 tiles of two row tiles (5000 tokens from their start: 200 us with 3,
// 191 with 4, 190 with 5; 16 chunks of 256 after 2000: 191, 167, 173), less of
// the longer tiles at head dim 256 (217.6 us with 3, 218.6 with 4).
template <int kRows>
constexpr int kItemUnits = kRows == 256 ? 4 : 3;
// Items of at most so many key tiles are not split: writing and joining partials
// costs about six tiles' time, half an item is the most it could even out.
constexpr int kWholeTiles = 8;
// Such an item goes to the run that holds the middle of its units; at head dim
// 256 of its tiles, which is better for one short prompt (20 heads, 1000 tokens:
// 27.9 against 31.1 us, 600: 20.1 against 20.5) and worse for several (4 of 900:
// 64.1 against 62.2).
template <int kRows>
__device__ __forceinline__ int whole_units(int width) {
  return kRows == 256 ? width : width - kItemUnits<kRows>;
}
constexpr float kRescale = 8.f;  // base-2 exponent by which a maximum may lag

constexpr uint32_t idesc(int n, bool b_mn_major) {
  return (1u << 4)                              // D: f32
         | (1u << 7) | (1u << 10)               // A, B: bf16
         | (b_mn_major ? 1u << 16 : 0u)         // B with its N index contiguous
         | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void advance(uint32_t slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

struct Segment {
  Request rq;
  int b, h, r0, count;
  Span span;
  int tile0, tiles;           // key tiles [tile0, tile0 + tiles), maybe none
  long long item;             // first unit of the item
  int first, n_units, width;  // the segment's units of the item, the item's
};

template <int kRows>
__device__ __forceinline__ int row_tiles(const Args &a, const Request &q) {
  return (int)(((long long)q.n * a.G + kRows - 1) / kRows);
}
template <int kRows>
__device__ __forceinline__ int item_width(const Args &a, const Request &q, int i) {
  const Span s = rows_span(a, q, i * kRows, min(kRows, q.n * a.G - i * kRows));
  return (s.hi + kBK - 1) / kBK - s.lo / kBK + kItemUnits<kRows>;
}
__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Units of one kv head of a request, by a whole warp.
template <int kRows>
__device__ __forceinline__ long long head_units(const Args &a, const Request &q) {
  const int nt = row_tiles<kRows>(a, q), lane = threadIdx.x & 31;
  long long sum = 0;
  for (int i0 = 0; i0 < nt; i0 += 32)
    sum += warp_sum_int(i0 + lane < nt ? item_width<kRows>(a, q, i0 + lane) : 0);
  return sum;
}

// Walks a run's segments.  An item is its key tiles and then kItemUnits more; a
// run that ends among those takes the item to its end, and one that begins
// there leaves it alone, so only tiles are ever split; an item of few tiles goes
// as a whole to the run on the side of its larger part.  Items are ordered by
// request, kv head, row tile, so neighbouring CTAs read the same keys at about
// the same time.  All calls by a whole warp.
template <int kRows>
struct Walk {
  long long u, end, base, per_head, item;
  int b, h, i, nt, width;
  Request rq;
  __device__ void request(const Args &a) {
    rq = load_request(a, b);
    nt = row_tiles<kRows>(a, rq);
    per_head = head_units<kRows>(a, rq);
  }
  __device__ void start(const Args &a) {  // u, end, base and b are set
    request(a);
    const int lane = threadIdx.x & 31;
    h = (int)((u - base) / per_head);
    long long rem = u - base - h * per_head;
    item = base + h * per_head;
    for (int i0 = 0;; i0 += 32) {
      const int w = i0 + lane < nt ? item_width<kRows>(a, rq, i0 + lane) : 0;
      int upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto > rem);
      if (past) {
        const int src = __ffs(past) - 1;
        i = i0 + src;
        width = __shfl_sync(0xffffffffu, w, src);
        item += __shfl_sync(0xffffffffu, upto, src) - width;
        break;
      }
      const int all = __shfl_sync(0xffffffffu, upto, 31);
      rem -= all;
      item += all;
    }
    const int tiles = max(width - kItemUnits<kRows>, 1);
    const long long at = u - item;
    if (tiles <= kWholeTiles ? 2 * at > whole_units<kRows>(width) : at >= tiles)
      u = item + width;
    else if (tiles <= kWholeTiles)
      u = item;
  }
  __device__ bool next(const Args &a, Segment &s) {
    if (u >= end) return false;
    if (u == item + width) {  // on to the next item
      item = u;
      if (++i == nt) {
        i = 0;
        if (++h == a.Hkv) {
          h = 0;
          base = u;
          do {
            ++b;
            request(a);
          } while (nt == 0);
        }
      }
      width = item_width<kRows>(a, rq, i);
    }
    s.rq = rq;
    s.b = b;
    s.h = h;
    s.item = item;
    s.width = width;
    s.first = (int)(u - item);
    s.n_units = width - s.first;
    const int tiles = max(width - kItemUnits<kRows>, 1);
    if (tiles > kWholeTiles) {
      if (end - u < tiles - s.first) s.n_units = (int)(end - u);  // the run ends among its tiles
    } else if (2 * (end - item) <= whole_units<kRows>(width)) {
      u = end;
      return false;
    }
    s.r0 = i * kRows;
    s.count = min(kRows, rq.n * a.G - s.r0);
    s.span = rows_span(a, rq, s.r0, s.count);
    const int t0 = s.span.lo / kBK, t1 = (s.span.hi + kBK - 1) / kBK;
    s.tile0 = t0 + s.first;
    s.tiles = max(0, min(t1 - s.tile0, s.n_units));
    u += s.n_units;
    return true;
  }
};

// One non-blocking test of a phase.  The roles' waits begin with it: the
// blocking one costs more even when the phase is complete (1000 tokens over
// 30000: 428 us without the test, 404 with it, more than one test no better).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Uses of registers that a tcgen05.ld fills stay behind its wait.
__device__ __forceinline__ void pin(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]),
                      "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7]));
}
// Adds to the kCols output columns from col0 on that a thread's row has in tensor
// memory (at o_at) the non-finite values of positions [lo, hi) that the row
// attends (first .. last) and that not all rows do.  q is the row's query, null
// for none.  By whole warps.
template <int D, int kCols>
__device__ __noinline__ void add_nonfinite(const Args &a, int b, int h, int lo, int hi, int all_lo,
                                           int all_hi, const __nv_bfloat16 *q, int first, int last,
                                           uint32_t o_at, int col0) {
  const int lane = threadIdx.x & 31;
  for (int j = lo; j < hi; ++j) {
    if (j >= all_lo && j < all_hi) {
      j = all_hi - 1;
      continue;
    }
    const long long at = position_at(a, b, h, j, D);
    if (at < 0) continue;  // zeros
    const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v + at + col0);
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < kCols / 64; ++i) odd |= nonfinite_bits(v[i * 32 + lane]);
    const bool mine = q && j >= first && j <= last;
    if (!__any_sync(0xffffffffu, odd) || !__any_sync(0xffffffffu, mine)) continue;
    float s = 0.f;
    if (mine)
      for (int d = 0; d < D; d += 2) {
        const float2 x = two_floats(*reinterpret_cast<const uint32_t *>(q + d));
        const float2 k = two_floats(*reinterpret_cast<const uint32_t *>(a.k + at + d));
        s = fmaf(x.y, k.y, fmaf(x.x, k.x, s));
      }
#pragma unroll 1
    for (int d = 0; d < kCols; d += 32) {
      uint32_t o[32];
      __syncwarp();
      tc_ld_x32(o_at + d, o);
      tc_wait_ld();
      pin(o);
      if (mine) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 y = two_floats(v[(d + i) / 2]);
          o[i] = __float_as_uint(add_if_nonfinite(__uint_as_float(o[i]), y.x, s == kNegInf));
          o[i + 1] = __float_as_uint(add_if_nonfinite(__uint_as_float(o[i + 1]), y.y, s == kNegInf));
        }
      }
      __syncwarp();
      tc_st_x32(o_at + d, o);
    }
    tc_wait_st();
  }
}
__device__ __forceinline__ void group_sync(int wg) {  // the warps of a softmax group
  asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
}

// This CTA's run of units, and through s_b and s_base (for all threads after a
// barrier) the request that it begins in and its first unit; false, for the
// whole CTA, when it has none.  Zeroes the rows past the last request's.
template <int kRows, int D>
__device__ __forceinline__ bool begin_run(const Args &a, long long *s_scan, int *s_b,
                                          long long *s_base, Runs &runs, Walk<kRows> &walk) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  // request tid + b0's units: few row tiles by its thread, more by the warp
  auto units_of = [&](int b) {
    const bool real = b < a.B;
    Request rq = {0, 0, 0};
    if (real) rq = load_request(a, b);
    const int nt = real ? row_tiles<kRows>(a, rq) : 0;
    long long w = 0;
    if (nt <= 4)
      for (int i = 0; i < nt; ++i) w += item_width<kRows>(a, rq, i);
    unsigned big = __ballot_sync(0xffffffffu, nt > 4);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      Request x;
      x.q0 = 0;
      x.n = __shfl_sync(0xffffffffu, rq.n, src);
      x.len = __shfl_sync(0xffffffffu, rq.len, src);
      const long long sum = head_units<kRows>(a, x);
      if (lane == src) w = sum;
    }
    return w * a.Hkv;
  };
  long long size = units_of(tid), upto;  // the first block of requests, kept for the search
  long long all = block_sum(size, upto);
  runs.units = all;
  for (int b0 = kThreads; b0 < a.B; b0 += kThreads) {
    long long past;
    runs.units += block_sum(units_of(b0 + tid), past);
  }
  runs.ctas = (int)min((long long)gridDim.x, runs.units);
  const int used = min(max(__ldg(a.q_start + a.B), 0), a.rows);
  for (int r = used + blockIdx.x; r < a.rows; r += gridDim.x) {  // past the last request: zero
    for (int i = tid; i < a.Hq * (D / 8); i += kThreads)
      reinterpret_cast<uint4 *>(a.out + (long long)r * a.out_stride)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(long long)r * a.Hq + i] = kNegInf;
  }
  if ((int)blockIdx.x >= runs.ctas) return false;  // uniform
  walk.u = runs.begin(blockIdx.x);
  walk.end = runs.begin(blockIdx.x + 1);
  long long before = 0;  // units of the blocks of requests already searched
  for (int b0 = 0;;) {
    if (before + upto > walk.u && before + upto - size <= walk.u) {
      *s_b = b0 + tid;
      *s_base = before + upto - size;
    }
    b0 += kThreads;
    if (b0 >= a.B) break;
    before += all;
    size = units_of(b0 + tid);
    all = block_sum(size, upto);
  }
  return true;
}

// ---- joining split items ------------------------------------------------------
// The CTAs c0 .. c1 that share an item each leave a partial.  Most often there
// are two or three, of every row, and the last CTA to arrive joins them while
// others still work (a launch of its own for it made a 5000-token prompt 290
// instead of 210 us).  More than kJoin are joined in two rounds, groups of
// kJoin (the result takes the first member's place) and then the groups, so
// that no CTA reads more than about kJoin of them.  Partials are always added
// in CTA order, whichever CTA does it.
//
// A partial is written and read back only where it has to wait: a CTA that
// finds the others' (of at most kDirect) all there adds them to the sums in its
// tensor memory (8 us from its last product, where writing its own, arriving
// and joining took 14).
constexpr int kMaxTcCtas = 170;
constexpr int kJoin = 16;
constexpr int kDirect = 4;
static_assert(2 * 3 * kMaxTcCtas * 4 <= kCounterBytes, "counters");
static_assert(kMaxTcCtas <= kJoin * kJoin , "two rounds");
__device__ __forceinline__ unsigned load_relaxed(const unsigned *p) {
  unsigned v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
struct Group {
  int first, stride, n;  // CTAs first, first + stride, ..
  int counter;           // its arrivals, of 3 ctas
  bool final;            // its result is the item's
};
// The group in which CTA c of the item arrives first, or with `again` the
// groups' own.  `ctas` bounds the CTA numbers.
__device__ __forceinline__ Group join_group(int c0, int c1, int c, bool again, int ctas) {
  const int n = c1 - c0 + 1;
  Group g;
  if (again) {
    g.first = c0;
    g.stride = kJoin;
    g.n = (n + kJoin - 1) / kJoin;
    g.counter = 2 * ctas + c0;
    g.final = true;
  } else {
    const int k = (c - c0) / kJoin * kJoin;
    g.first = c0 + k;
    g.stride = 1;
    g.n = min(kJoin, n - k);
    // a CTA can be first of a group in the item that it ends and in the one
    // that it begins
    g.counter = 2 * g.first + (k == 0 ? 1 : 0);
    g.final = n <= kJoin;
  }
  return g;
}
// Partial k of the group (see partial_at): an item's first CTA has it in its
// second place.
__device__ __forceinline__ int join_slot(const Group &g, int c0, int k) {
  const int c = g.first + k * g.stride;
  return 2 * c + (c == c0 ? 1 : 0);
}

}  // namespace
}  // namespace attn
}  // namespace sv
