// paged_attn_tc.cu -- attention of prompt chunks (many rows a request) over a
// paged cache on the 5th-generation tensor cores, sm_103a; the mathematics and
// the split of work are in attn_common.cuh.
//
// Per key, R packed rows of a kv head take 4 R D flops against 4 D bytes, so
// from about 300 rows on (this card's tensor rate over its bandwidth) the
// tensor cores bound it, not the cache.  A CTA takes 256 rows of one kv head,
// as two tiles of 128, against a run of 128-key tiles:
//   warp 9      copies keys and values page by page with TMA, 128-byte
//               swizzled, through one ring of 128-key slots;
//   warp 8      issues tcgen05.mma: S = Q K^T (both from shared memory), then
//               O += P V with the weights P from tensor memory;
//   warps 0-3   softmax of the first tile, a row a thread: scores from tensor
//   warps 4-7   memory, running maximum and sum in fp32 registers, weights
//               back in bf16 over the scores' own columns; same for the second.
// Tensor memory holds S and O of both tiles (2 x 128 + 2 x D columns).  The
// tensor cores work for one tile while the other's weights are made: per key
// tile the issue order is P0 V, Q0 K', P1 V, Q1 K' (K' the next keys), so each
// softmax has the other tile's two products to hide behind.
//
// O is rescaled only when a row's maximum grew by more than 2^8 in weight
// (the first tile sets it): until then weights up to 2^8 are relative to the
// older maximum, which loses nothing in bf16 or fp32, and a rescale, a read
// and write of the row's O, stays rare.  Scores, sums and O are fp32; weights
// are rounded to bf16 (at most half a step, 2^-8 of each), their sum is not.
//
// Measured (GB300, 40 heads of 128 over 8 kv heads): 1000 rows after 30,000
// positions 404 to 465 us on different days (1.3 to 1.5 PFLOP/s), 3 chunks of
// 3500 after 9000 1490 us (1.5); a prompt of 5000 from its start 191 us (1.34),
// where about 4 us pass before the first product, 6 around each item and 8 at
// the last join.  A key tile takes 1.5 us for both row tiles, 1.3 at a large
// library product's rate: the tensor cores bound it then.  Leaving the
// exponentials out did not shorten it.
#include <algorithm>

#include "attn_common.cuh"
#include "attn_host.h"
#include "attn_tc.cuh"
#include "qmv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace attn {
namespace {

constexpr int kRows = 2 * kTile;  // rows per item

template <int D>
struct TcShape {
  static constexpr uint32_t kBlock = kBK * 128;              // 64 values of 128 rows
  static constexpr uint32_t kTileBytes = kBlock * (D / 64);  // queries, keys or values
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr uint32_t kStage = kTile * 128;  // 64 output values of a tile's rows
  static constexpr uint32_t kSmem = (2 + kSlots) * kTileBytes + 2 * kStage + 1024;
  static constexpr uint32_t kOCol = 2 * kBK;  // tensor-memory column of O of tile 0
  static_assert(kJoin * kTile * 4 <= kStage, "a join's weights");
};

// A split item's partial: sums as [D / 4][rows][4] (a thread owns a row, so
// accesses of a warp are contiguous), then maxima and sums [rows] each.
template <int D>
__device__ __forceinline__ float *part_row(const Args &a, int slot, int rr) {
  return partial_at(a, slot, kRows, D) + rr * 4;
}

// The result of packed row r (row rr of the item, kept if `ok`) of which this
// CTA's tensor memory holds its own sums (if `any`) and the others of c0 .. c1
// have left theirs: added in CTA order, as in the join of partials alone.
template <int D>
__device__ __noinline__ void add_and_write(const Args &a, int q0, int h, int r, int rr, bool ok,
                                           bool any, uint32_t o_at, float m, float l, int c0,
                                           int c1) {
  const int me = (int)blockIdx.x, t = r / a.G, g = r - t * a.G;
  auto slot = [&](int k) { return 2 * (c0 + k) + (k == 0 ? 1 : 0); };
  float weight[kDirect], lk[kDirect], mm = kNegInf, ll = 0.f;
#pragma unroll
  for (int k = 0; k < kDirect; ++k) {
    const float *ml = partial_at(a, slot(k), kRows, D) + kRows * D + rr;
    const bool other = ok && c0 + k <= c1 && c0 + k != me;
    weight[k] = other ? __ldcg(ml) : c0 + k == me ? m : kNegInf;
    lk[k] = other ? __ldcg(ml + kRows) : c0 + k == me ? l : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kDirect; ++k) mm = fmaxf(mm, weight[k]);
#pragma unroll
  for (int k = 0; k < kDirect; ++k) {
    weight[k] = join_weight(a, weight[k], lk[k], mm);
    ll = fmaf(lk[k], weight[k], ll);
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  __nv_bfloat16 *dst = a.out + (long long)(q0 + t) * a.out_stride + (long long)(h * a.G + g) * D;
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    uint32_t o[32];
    __syncwarp();
    if (any) {
      tc_ld_x32(o_at + d, o);
      tc_wait_ld();
      pin(o);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    }
    if (!ok) continue;  // the loads are the warp's, the rest the row's
    float acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kDirect; ++k) {
      if (c0 + k > c1) break;
      float4 y[8];
      const float *part = part_row<D>(a, slot(k), rr) + (size_t)(d >> 2) * kRows * 4;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = c0 + k == me
                   ? make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                 __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]))
                   : __ldcg(reinterpret_cast<const float4 *>(part + (size_t)i * kRows * 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[4 * i] = fmaf(y[i].x, weight[k], acc[4 * i]);
        acc[4 * i + 1] = fmaf(y[i].y, weight[k], acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(y[i].z, weight[k], acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(y[i].w, weight[k], acc[4 * i + 3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      *reinterpret_cast<uint4 *>(dst + d + i) = make_uint4(
          pack_bf16(acc[i] * inv, acc[i + 1] * inv), pack_bf16(acc[i + 2] * inv, acc[i + 3] * inv),
          pack_bf16(acc[i + 4] * inv, acc[i + 5] * inv),
          pack_bf16(acc[i + 6] * inv, acc[i + 7] * inv));
  }
  if (ok && a.lse) a.lse[(long long)(q0 + t) * a.Hq + h * a.G + g] = row_lse(a, mm, ll);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  using S = TcShape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[S::kSlots], kv_empty[S::kSlots];
  __shared__ __align__(8) uint64_t q_full[2], q_free[2], s_full[2], p_full[2][2], o_done[2];
  __shared__ __align__(8) uint64_t mma_done;
  __shared__ long long s_scan[kThreads / 32], s_base;
  __shared__ uint32_t s_row[2][kTile];
  __shared__ uint32_t s_tmem;
  __shared__ int s_b, s_last[2];
  __shared__ uint32_t s_odd[2][2];  // items with non-finite values left out (see the softmax)
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t q_smem = raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t ring0 = q_smem + 2 * S::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 4);
      mbar_init(&p_full[i][1], 4);
      mbar_init(&o_done[i], 1);
      s_odd[i][0] = s_odd[i][1] = 0;
    }
    mbar_init(&mma_done, 1);
    fence_mbar_init();
  }
  Runs runs;
  Walk<kRows> walk;
  if (!begin_run<kRows, D>(a, s_scan, &s_b, &s_base, runs, walk)) return;  // uniform
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  walk.b = s_b;
  walk.base = s_base;
  walk.start(a);
  const uint32_t tmem = *const_cast<const volatile uint32_t *>(&s_tmem);
  bool dead = false;  // a wait gave up: the rest runs without waiting, results are invalid
  Segment s;

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      // ------------------------------ producer ------------------------------
      const int per_page = min(kBK, 1 << a.page_shift);
      const int pages = kBK / per_page;
      const int boxes = pages * (D / 64);
      const int blk = lane / pages, pg = lane - blk * pages;
      Ring ring;
      long long issued = 0;
      while (!dead && walk.next(a, s)) {
        for (int t = 0; !dead && t < s.tiles; ++t) {
          const int j = (s.tile0 + t) * kBK + pg * per_page;
          int y = 0;
          if (lane < boxes)
            y = page_row(a, s.b, s.h, j >> a.page_shift, s.span.lo, s.span.hi) +
                (j & ((1 << a.page_shift) - 1));
          for (int kv = 0; kv < 2; ++kv) {
            if (issued >= S::kSlots && !mbar_wait(&kv_empty[ring.slot], ring.phase ^ 1u))
              dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[ring.slot], S::kTileBytes);
            __syncwarp();
            if (lane < boxes)
              tma_load_rows(ring0 + ring.slot * S::kTileBytes + (uint32_t)blk * S::kBlock +
                                (uint32_t)pg * per_page * 128,
                            kv ? &vmap : &kmap, blk * 64, y, smem_addr(&kv_full[ring.slot]));
            ++issued;
            ring.advance(S::kSlots);
          }
        }
      }
      if (dead && lane == 0) report_give_up(4u);
      // every copy has landed before the CTA may exit
      for (long long k = max(0ll, issued - S::kSlots); k < issued; ++k)
        (void)mbar_wait(&kv_full[k % S::kSlots], (uint32_t)((k / S::kSlots) & 1));
    } else if (warp == kMmaWarp) {
      // -------------------------- matrix products ---------------------------
      // The whole warp walks and waits, so that descriptors stay in uniform
      // registers; one lane issues.
      constexpr uint32_t kQk = idesc(kBK, false), kPv = idesc(D, true);
      const bool leader = elect_one();
      Ring ring;
      uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};  // phases of q_full and p_full
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        if (!__all_sync(0xffffffffu, mbar_test(bar, phase)) && !dead)
          dead = !__all_sync(0xffffffffu, mbar_wait(bar, phase));
        tc_fence_after();
      };
      const uint64_t q_desc = smem_desc_sw128(q_smem), k_desc = smem_desc_sw128(ring0),
                     v_desc = smem_desc_sw128_mn(ring0, S::kBlock);
      // a descriptor's address field counts 16-byte units: offsets add to it
      auto qk = [&](int w, uint32_t slot, bool last) {
        const uint64_t qd = q_desc + (uint32_t)w * (S::kTileBytes >> 4);
        const uint64_t kd = k_desc + slot * (S::kTileBytes >> 4);
        if (leader) {
          if (!dead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = ((uint32_t)(k >> 2) * S::kBlock + (uint32_t)(k & 3) * 32) >> 4;
              tc_mma_ss(tmem + (uint32_t)w * kBK, qd + at, kd + at, kQk, k > 0);
            }
          }
          tc_commit(smem_addr(&s_full[w]));
          if (last) tc_commit(smem_addr(&q_free[w]));  // the segment's queries are done with
        }
        __syncwarp();
      };
      auto pv = [&](int w, uint32_t slot, bool first) {
        const uint64_t vd = v_desc + slot * (S::kTileBytes >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(&p_full[w][half], pn[w]);
          if (leader && !dead) {
#pragma unroll
            for (int k = half * (kBK / 32); k < (half + 1) * (kBK / 32); ++k)
              tc_mma_ts(tmem + S::kOCol + (uint32_t)w * D, tmem + (uint32_t)w * kBK + k * 8,
                        vd + k * (2048 >> 4), kPv, !first || k > 0);
          }
          __syncwarp();
        }
        pn[w] ^= 1u;
        if (leader) tc_commit(smem_addr(&o_done[w]));
        __syncwarp();
      };
      auto release = [&](uint32_t slot) {
        if (leader) tc_commit(smem_addr(&kv_empty[slot]));
        __syncwarp();
      };
      while (walk.next(a, s)) {
        if (s.tiles == 0) continue;
        const bool two = s.count > kTile;
        wait(&q_full[0], qn[0]);
        qn[0] ^= 1u;
        wait(&kv_full[ring.slot], ring.phase);
        qk(0, ring.slot, s.tiles == 1);
        if (two) {
          wait(&q_full[1], qn[1]);
          qn[1] ^= 1u;
          qk(1, ring.slot, s.tiles == 1);
        }
        release(ring.slot);
        ring.advance(S::kSlots);
        for (int t = 0; t < s.tiles; ++t) {
          const uint32_t v_slot = ring.slot;
          const bool more = t + 1 < s.tiles;
          wait(&kv_full[v_slot], ring.phase);
          ring.advance(S::kSlots);
          pv(0, v_slot, t == 0);
          // The products run in issue order, so Q K' may overwrite the columns
          // that hold the weights of the product issued before it.
          if (more) {
            wait(&kv_full[ring.slot], ring.phase);
            qk(0, ring.slot, t + 2 == s.tiles);
          }
          if (two) pv(1, v_slot, t == 0);
          release(v_slot);
          if (more) {
            if (two) qk(1, ring.slot, t + 2 == s.tiles);
            release(ring.slot);
            ring.advance(S::kSlots);
          }
        }
      }
      if (dead && lane == 0) report_give_up(8u);
      if (leader) {  // no product is in flight when the tensor memory is freed
        tc_commit(smem_addr(&mma_done));
        (void)mbar_wait(&mma_done, 0);
      }
      __syncwarp();
    } else {
      // ------------------------------- queries ------------------------------
      // the next segment's are fetched while the last products of this one run
      const int w = warp - kQueryWarp;
      uint32_t free = 0;
      bool loaded = false;
      while (walk.next(a, s)) {
        const int n = min(kTile, s.count - w * kTile);
        if (s.tiles == 0 || n <= 0) continue;
        if (loaded) {
          if (!dead && !mbar_wait(&q_free[w], free)) {
            dead = true;
            report_give_up(32u);
          }
          free ^= 1u;
        }
        loaded = true;
        __syncwarp();
        constexpr int kChunks = D / 8;         // 16-byte pieces of a row
        constexpr int kStep = 32 / kChunks;    // rows at a time
        const int ch = lane % kChunks, first = lane / kChunks;
        // a row's address moves with its token and head, without a division a row
        const int t = (s.r0 + w * kTile + first) / a.G;
        int g = s.r0 + w * kTile + first - t * a.G;
        const int dt = kStep / a.G, dg = kStep - dt * a.G;
        const long long step = dt * a.q_stride + dg * D, carry = a.q_stride - (long long)a.G * D;
        const __nv_bfloat16 *base =
            a.q + (long long)s.rq.q0 * a.q_stride + (long long)s.h * a.G * D + ch * 8;
        const __nv_bfloat16 *src = base + (long long)t * a.q_stride + (long long)g * D;
        const uint32_t dst = q_smem + (uint32_t)w * S::kTileBytes + (uint32_t)(ch >> 3) * S::kBlock;
#pragma unroll 4
        for (int rr = first; rr < kTile; rr += kStep) {
          const bool real = rr < n;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           dst + (uint32_t)rr * 128 + (uint32_t)(((ch & 7) ^ (rr & 7)) << 4)),
                       "l"(real ? src : base), "r"(real ? 16 : 0)
                       : "memory");
          src += step;
          g += dg;
          if (g >= a.G) {
            g -= a.G;
            src += carry;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[w]);
      }
    }
  } else {
    // ------------------------------- softmax ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 tensor-memory lanes a warp
    const uint32_t s_at = tmem + lanes + (uint32_t)wg * kBK;
    const uint32_t o_at = tmem + lanes + S::kOCol + (uint32_t)wg * D;
    const float c = a.scale_log2;
    Ring ring;  // of the segment's first key slot
    uint32_t sn = 0;  // key tiles done by this group
    // The first group clears the values of masked places for both, and where one
    // that some rows attend was not finite it leaves the item's number among those
    // of two row tiles (or of one) in s_odd, for the rows to add it at the end.
    // Numbers alternate between two words: an item's products wait for the
    // weights of all warps concerned, so a word is written again only when all
    // have read it.
    uint32_t items[2] = {0, 0};
    auto wait = [&](uint64_t *bar, uint32_t phase) {
      if (!mbar_test(bar, phase) && !dead && !mbar_wait(bar, phase)) {
        dead = true;
        report_give_up(16u);
      }
      __syncwarp();  // the tensor-memory accesses that follow want the whole warp
    };
    while (walk.next(a, s)) {
      const int count = min(kTile, s.count - wg * kTile);  // rows of this tile, maybe none
      const bool ok = row < count;
      const int r = s.r0 + wg * kTile + row;
      const int t_row = ok ? r / a.G : 0;
      const int last = ok ? s.rq.len - s.rq.n + t_row : -1;
      const int first = a.window > 0 ? last - a.window + 1 : 0;
      float m = kNegInf, l = 0.f;
      const bool two = s.count > kTile;
      uint32_t item_no = 0;
      if (s.tiles > 0) item_no = two ? ++items[1] : ++items[0];
      volatile uint32_t *odd_word = &s_odd[two ? 1 : 0][item_no & 1u];
      if (count > 0) {
        for (int t = 0; t < s.tiles; ++t, ++sn) {
          const int j0 = (s.tile0 + t) * kBK;
          const bool masked = j0 < s.span.all_lo || j0 + kBK > s.span.all_hi;
          ring.advance(S::kSlots);  // to the tile's values
          wait(&s_full[wg], sn & 1u);
          tc_fence_after();
          uint32_t x[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tc_ld_x32(s_at + 32 * q, x[q]);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) pin(x[q]);
          if (masked) {
            const int lo = first - j0, hi = last - j0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * q + i > hi) x[q][i] = __float_as_uint(kNegInf);
            if (a.window > 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (32 * q + i < lo) x[q][i] = __float_as_uint(kNegInf);
            }
          }
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(x[q][i]), __uint_as_float(x[q][i + 1])));
          const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          if (t == 0) {
            m = mn;
          } else {
            const bool grew = (mn - m) * c > kRescale;
            if (__any_sync(0xffffffffu, grew)) {
              float f = 1.f;
              if (grew) {
                f = exp2_approx((m - mn) * c);
                m = mn;
                l *= f;
              }
              // (these scores were issued after the product before the last, so
              // the barrier is at most one phase behind)
              wait(&o_done[wg], (sn - 1u) & 1u);
              tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                tc_ld_x32(o_at + d, o);
                tc_wait_ld();
                pin(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tc_st_x32(o_at + d, o);
              }
            }
          }
          if (wg == 0 && masked) {
            // places no row of the item attends may hold anything: their values
            // are zeroed, so that a weight of zero meets no NaN, and so is what is
            // not finite where some rows attend and others do not
            wait(&kv_full[ring.slot], ring.phase);
            uint8_t *v = smem_raw + (ring0 - raw) + ring.slot * S::kTileBytes + row * 16;
            bool odd = false;
#pragma unroll 1
            for (int i = 0; i < kBK / 16; ++i) {  // eight threads a key: a warp reads 512 bytes
              const int p0 = j0 + i * 16, pos = p0 + (row >> 3);
              if (p0 >= s.span.all_lo && p0 + 16 <= s.span.all_hi) continue;
              const bool none = pos < s.span.lo || pos >= s.span.hi;
              const bool part = !none && (pos < s.span.all_lo || pos >= s.span.all_hi);
              uint4 *at = reinterpret_cast<uint4 *>(v + i * 2048), y[D / 64];
              if (part) {
                uint32_t bits = 0;
#pragma unroll
                for (int blk = 0; blk < D / 64; ++blk) {
                  y[blk] = at[blk * (S::kBlock / 16)];
                  bits |= nonfinite_bits(y[blk]);
                }
                if (bits) {
                  odd = true;
#pragma unroll
                  for (int blk = 0; blk < D / 64; ++blk) {
                    clear_nonfinite(y[blk]);
                    at[blk * (S::kBlock / 16)] = y[blk];
                  }
                }
              }
              if (none)
#pragma unroll
                for (int blk = 0; blk < D / 64; ++blk)
                  at[blk * (S::kBlock / 16)] = make_uint4(0, 0, 0, 0);
            }
            if (odd) *odd_word = item_no;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          const float off = m == kNegInf ? 0.f : m * c;
          const uint64_t c2 = pack2(c, c), off2 = pack2(-off, -off);
          uint64_t acc[4] = {0, 0, 0, 0};  // pairs of zeros
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(x[q][2 * i]), __uint_as_float(x[q][2 * i + 1])),
                           c2, off2),
                      e0, e1);
              e0 = exp2_approx(e0);
              e1 = exp2_approx(e1);
              acc[i & 3] = add2(acc[i & 3], pack2(e0, e1));
              p[i] = pack_bf16(e0, e1);
            }
            tc_st_x16(s_at + 16 * q, p);
            if (q & 1) {  // half of the weights: their product may begin
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[wg][q >> 1]);
            }
          }
          {
            float e0, e1;
            unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), e0, e1);
            l += e0 + e1;
          }
          ring.advance(S::kSlots);
        }
      } else {
        for (int t = 0; t < 2 * s.tiles; ++t) ring.advance(S::kSlots);
      }

      if (count > 0) {
        const bool whole = s.first == 0 && s.n_units == s.width;
        const int slot = 2 * (int)blockIdx.x + (s.first == 0 ? 1 : 0);
        const int rr = wg * kTile + row;
        // A split item's CTAs c0 .. c1.  When all others have left their partials,
        // this one adds them to what it holds and writes the result.
        const int c0 = whole ? 0 : runs.owner(s.item);
        const int c1 = whole ? 0 : runs.owner(s.item + s.width - kItemUnits<kRows> - 1);
        bool direct = !whole && c1 - c0 < kDirect;
        unsigned *arrivals = nullptr, arrived = 0;
        if (direct && row == 0) {
          arrivals = a.counters + wg * 3 * gridDim.x +
                     join_group(c0, c1, (int)blockIdx.x, false, (int)gridDim.x).counter;
          arrived = load_relaxed(arrivals);
        }
        if (s.tiles > 0) {
          wait(&o_done[wg], (sn - 1u) & 1u);
          tc_fence_after();
          if (*odd_word == item_no)
            add_nonfinite<D, D>(a, s.b, s.h, max(s.span.lo, s.tile0 * kBK),
                                min(s.span.hi, (s.tile0 + s.tiles) * kBK), s.span.all_lo,
                                s.span.all_hi,
                                ok ? a.q + (long long)(s.rq.q0 + t_row) * a.q_stride +
                                         (long long)(s.h * a.G + (r - t_row * a.G)) * D
                                   : nullptr,
                                first, last, o_at, 0);
        }
        if (direct) {
          if (row == 0) {
            __threadfence();
            s_last[wg] = arrived == (unsigned)(c1 - c0);
            if (s_last[wg]) *arrivals = 0;  // ready for the next call
          }
          group_sync(wg);
          direct = s_last[wg] != 0;
        }
        if (direct) {
          add_and_write<D>(a, s.rq.q0, s.h, r, rr, ok, s.tiles > 0, o_at, m, l, c0, c1);
        } else {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int g = r - t_row * a.G, t0 = (s.r0 + wg * kTile) / a.G;
          float *part = part_row<D>(a, slot, rr);
          // whole rows go through shared memory, so that eight threads write
          // 128 contiguous bytes of a row
          s_row[wg][row] = (uint32_t)(t_row - t0) << 16 | (uint32_t)g;
          uint8_t *stage = smem_raw + (q_smem - raw) + (2 + S::kSlots) * S::kTileBytes +
                           (uint32_t)wg * S::kStage;
          __nv_bfloat16 *dst = a.out + (long long)(s.rq.q0 + t0) * a.out_stride +
                               (long long)s.h * a.G * D;
#pragma unroll 1
          for (int d = 0; d < D; d += 64) {
#pragma unroll
            for (int e = 0; e < 64; e += 32) {
              uint32_t o[32];
              if (s.tiles > 0) {
                tc_ld_x32(o_at + d + e, o);
                tc_wait_ld();
                pin(o);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0;
              }
              if (whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                  auto two = [&](int k) {
                    return pack_bf16(__uint_as_float(o[i + k]) * inv,
                                     __uint_as_float(o[i + k + 1]) * inv);
                  };
                  *reinterpret_cast<uint4 *>(stage + row * 128 +
                                             ((((e + i) >> 3) ^ (row & 7)) << 4)) =
                      make_uint4(two(0), two(2), two(4), two(6));
                }
              } else if (ok) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  __stcg(reinterpret_cast<uint4 *>(part + (size_t)((d + e + i) >> 2) * kRows * 4),
                         make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
              }
              __syncwarp();
            }
            if (whole) {
              group_sync(wg);
#pragma unroll 4
              for (int i = row >> 3; i < count; i += 16) {
                const uint32_t at = s_row[wg][i];
                const uint4 y = *reinterpret_cast<const uint4 *>(
                    stage + i * 128 + (((row & 7) ^ (i & 7)) << 4));
                *reinterpret_cast<uint4 *>(dst + (at >> 16) * a.out_stride + (at & 0xFFFFu) * D + d +
                                           (row & 7) * 8) = y;
              }
              group_sync(wg);
            }
          }
          if (ok && whole && a.lse)
            a.lse[(long long)(s.rq.q0 + t_row) * a.Hq + s.h * a.G + g] = row_lse(a, m, l);
          if (ok && !whole) {
            float *ml = partial_at(a, slot, kRows, D) + kRows * D + rr;
            __stcg(ml, m);
            __stcg(ml + kRows, l);
          }
        }
        tc_fence_before();  // O has been read before the next segment's products write it
        if (!whole && !direct) {
          // ---- the last CTA to arrive joins this tile's partials ----
          float *weights = reinterpret_cast<float *>(  // [partial][row]
              smem_raw + (q_smem - raw) + (2 + S::kSlots) * S::kTileBytes +
              (uint32_t)wg * S::kStage);
          for (int again = 0; again < 2; ++again) {
            const Group gr = join_group(c0, c1, (int)blockIdx.x, again != 0, (int)gridDim.x);
            __threadfence();
            group_sync(wg);
            if (row == 0) {
              unsigned *counter = a.counters + wg * 3 * gridDim.x + gr.counter;
              s_last[wg] = atomicAdd(counter, 1u) == (unsigned)(gr.n - 1);
              if (s_last[wg]) *counter = 0;  // all have arrived: ready for the next call
            }
            group_sync(wg);
            if (!s_last[wg]) break;
            __threadfence();
            if (ok) {
              float mm = kNegInf, ll = 0.f;
#pragma unroll 4
              for (int k = 0; k < gr.n; ++k)
                mm = fmaxf(mm, __ldcg(partial_at(a, join_slot(gr, c0, k), kRows, D) + kRows * D + rr));
#pragma unroll 4
              for (int k = 0; k < gr.n; ++k) {
                const float *ml = partial_at(a, join_slot(gr, c0, k), kRows, D) + kRows * D + rr;
                const float lk = __ldcg(ml + kRows), f = join_weight(a, __ldcg(ml), lk, mm);
                ll = fmaf(lk, f, ll);
                weights[k * kTile + row] = f;  // read by this thread alone
              }
              const float inv = ll == 0.f ? 0.f : 1.f / ll;
              const int g = r - t_row * a.G;
              __nv_bfloat16 *dst = a.out + (long long)(s.rq.q0 + t_row) * a.out_stride +
                                   (long long)(s.h * a.G + g) * D;
              const int to = join_slot(gr, c0, 0);
#pragma unroll 1
              for (int d = 0; d < D; d += 64) {
                float o[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) o[i] = 0.f;
#pragma unroll 2
                for (int k = 0; k < gr.n; ++k) {
                  const float f = weights[k * kTile + row];
                  const float *part = part_row<D>(a, join_slot(gr, c0, k), rr) +
                                      (size_t)(d >> 2) * kRows * 4;
                  float4 y[16];
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    y[i] = __ldcg(reinterpret_cast<const float4 *>(part + (size_t)i * kRows * 4));
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    o[4 * i] = fmaf(y[i].x, f, o[4 * i]);
                    o[4 * i + 1] = fmaf(y[i].y, f, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(y[i].z, f, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(y[i].w, f, o[4 * i + 3]);
                  }
                }
                if (gr.final) {
#pragma unroll
                  for (int i = 0; i < 64; i += 8)
                    *reinterpret_cast<uint4 *>(dst + d + i) = make_uint4(
                        pack_bf16(o[i] * inv, o[i + 1] * inv),
                        pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                        pack_bf16(o[i + 4] * inv, o[i + 5] * inv),
                        pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
                } else {
                  float *part = part_row<D>(a, to, rr) + (size_t)(d >> 2) * kRows * 4;
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    __stcg(reinterpret_cast<float4 *>(part + (size_t)i * kRows * 4),
                           make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
                }
              }
              if (!gr.final) {
                float *ml = partial_at(a, to, kRows, D) + kRows * D + rr;
                __stcg(ml, mm);
                __stcg(ml + kRows, ll);
              } else if (a.lse) {
                a.lse[(long long)(s.rq.q0 + t_row) * a.Hq + s.h * a.G + g] = row_lse(a, mm, ll);
              }
            }
            if (gr.final) break;
          }
          // the weights have been read: the next item's rows may be staged over
          // them (one without key tiles waits for nothing before it does)
          group_sync(wg);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
sv_status launch(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, int ctas,
                 cudaStream_t stream) {
  using S = TcShape<D>;
  static PerDeviceOnce once;
  const cudaError_t ce = once.run([] {
    return cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)S::kSmem);
  });
  if (ce != cudaSuccess)
    return fail(SV_ERR_CUDA, "paged_attention: cudaFuncSetAttribute failed: %s",
                cudaGetErrorString(ce));
  attn_tc_kernel<D><<<(unsigned)ctas, kThreads, S::kSmem, stream>>>(kmap, vmap, a);
  return check_launch("paged_attention");
}

int tc_ctas() { return std::min(kMaxTcCtas, device_sm_count()); }

}  // namespace

size_t tc_partial_bytes(int D) { return (size_t)tc_ctas() * 2 * kRows * (D + 2) * 4; }

unsigned tc_take_give_up() {
  unsigned v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_give_up, sizeof v);
  cudaMemcpyToSymbol(g_give_up, &zero, sizeof zero);
  return v;
}

sv_status tc_run(int D, const Args &a, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  sv_status st = encode_cache(&kmap, a.k, D, a, kBK);
  if (st == SV_OK) st = encode_cache(&vmap, a.v, D, a, kBK);
  if (st != SV_OK) return st;
  return D == 64 ? launch<64>(a, kmap, vmap, tc_ctas(), stream)
                 : launch<128>(a, kmap, vmap, tc_ctas(), stream);
}

}  // namespace attn
}  // namespace sv
