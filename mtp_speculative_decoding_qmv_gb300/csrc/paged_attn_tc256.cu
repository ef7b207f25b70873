// paged_attn_tc256.cu -- attention of prompt chunks over a paged cache for head
// dim 256 on the 5th-generation tensor cores, sm_103a; the mathematics and the
// split of work are in attn_common.cuh, the smaller head dims' kernel in
// paged_attn_tc.cu.
//
// An output row takes 256 of tensor memory's 512 columns, so a CTA holds one
// tile of 128 rows, and the scores of two key tiles beside it: the tensor
// cores multiply Q K' for the next 128 keys while the softmax works on these.
// Both softmax groups work on the same rows, 64 keys each: a row's maximum goes
// through shared memory (one barrier of 256 threads a tile), which halves the
// time from scores to weights, the part that the tensor cores wait for.
//   issue order per tile t: Q K(t + 1), then P(t) V(t)
// A tile's keys and values are 64 KB each, so the ring has slots of 16 KB, 128
// keys by 64 values, released one by one: Q K accumulates over four of them,
// P V is four products of 64 output columns.  Every row re-reads the cache
// twice as often as with two tiles of rows: at 128 rows a key tile of 128 KB
// carries 17 MFLOP, so L2 has to deliver 10 TB/s at 1.3 PFLOP/s.
// Masks, rescaling, rounding, splitting and joining are as in paged_attn_tc.cu.
//
// Measured (GB300, 20 heads over 4 kv heads unless said): a prompt of 5000 from
// its start 217 us, 1000 rows after 30,000 positions 526 us (1.2 PFLOP/s both).
#include <algorithm>

#include "attn_common.cuh"
#include "attn_host.h"
#include "attn_tc.cuh"
#include "qmv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace attn {
namespace {

constexpr int D = 256;
constexpr int kRows = kTile;
constexpr int kBlocks = D / 64;                          // ring slots of a tile's keys or values
constexpr uint32_t kBlock = kBK * 128;                   // 16 KB: 128 rows of 64 values
constexpr int kSlots = 2 * kBlocks;                      // two groups of blocks
constexpr uint32_t kQBytes = kBlocks * kBlock;
constexpr uint32_t kStage = kTile * 64;                  // 32 output values of the rows
constexpr uint32_t kSmem = kQBytes + kSlots * kBlock + 2 * kStage + 1024;
constexpr uint32_t kOCol = 2 * kBK;
static_assert(kOCol + D <= kTmemCols, "tensor memory");
static_assert(kJoin * kTile * 4 <= kStage, "a join's weights");
// floats of a partial: sums [D / 4][rows][4], then for each softmax group its
// own copy of the maxima and sums [rows] (each joins half of the columns)
constexpr size_t kPartial = (size_t)kRows * (D + 4);

__device__ __forceinline__ float *part_base(const Args &a, int slot) {
  return a.partials + slot * kPartial;
}
__device__ __forceinline__ float *part_ml(const Args &a, int slot, int wg) {
  return part_base(a, slot) + kRows * (D + 2 * wg);
}
__device__ __forceinline__ void pair_sync() {  // both softmax groups
  asm volatile("bar.sync 3, 256;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_tc256_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[kSlots], kv_empty[kSlots];
  __shared__ __align__(8) uint64_t q_full, q_free, s_full[2], p_full[2][2], o_done[2];
  __shared__ __align__(8) uint64_t mma_done;
  __shared__ long long s_scan[kThreads / 32], s_base;
  __shared__ uint32_t s_row[kTile];
  __shared__ float s_x[2][2][kTile];  // [tile parity][group][row]: maxima; at the end sums
  __shared__ uint32_t s_tmem;
  __shared__ int s_b, s_odd, s_last[2];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t q_smem = raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t ring0 = q_smem + kQBytes;
  const uint32_t stage0 = ring0 + kSlots * kBlock;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&q_full, 2);
    mbar_init(&q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&p_full[i][0], 4);
      mbar_init(&p_full[i][1], 4);
    }
    mbar_init(&mma_done, 1);
    s_odd = 0;
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

  // Blocks travel in groups of kBlocks, a tile's keys or its values, in the
  // order of their use: K(0), K(1), V(0), K(2), V(1), .. V(last).  Group g of
  // the CTA fills half g & 1 of the ring, for the (g >> 1)-th time.
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      // ----------------------------- producer -----------------------------
      const int per_page = min(kBK, 1 << a.page_shift);
      const int pages = kBK / per_page;  // at most 8: a copy a lane
      const int blk = lane / pages, pg = lane - blk * pages;
      const bool mine = blk < kBlocks;
      uint32_t g = 0;
      auto load = [&](const Segment &s, int t, const CUtensorMap *map) {
        const uint32_t slot = (g & 1u) * kBlocks + (uint32_t)(mine ? blk : 0);
        const int j = (s.tile0 + t) * kBK + pg * per_page;
        int y = 0;
        if (mine)
          y = page_row(a, s.b, s.h, j >> a.page_shift, s.span.lo, s.span.hi) +
              (j & ((1 << a.page_shift) - 1));
        if (g >= 2 && !dead && !mbar_wait(&kv_empty[slot], ((g >> 1) & 1u) ^ 1u)) dead = true;
        dead = __any_sync(0xffffffffu, dead);
        if (dead) return;
        if (mine && pg == 0) mbar_arrive_expect_tx(&kv_full[slot], kBlock);
        __syncwarp();
        if (mine)
          tma_load_rows(ring0 + slot * kBlock + (uint32_t)pg * per_page * 128, map, blk * 64, y,
                        smem_addr(&kv_full[slot]));
        ++g;
      };
      while (!dead && walk.next(a, s)) {
        for (int t = 0; !dead && t <= s.tiles && s.tiles > 0; ++t) {
          if (t < s.tiles) load(s, t, &kmap);
          if (t > 0 && !dead) load(s, t - 1, &vmap);
        }
      }
      if (dead && lane == 0) report_give_up(4u);
      // every copy has landed before the CTA may exit
      if (lane < kBlocks)
        for (uint32_t k = g > 2 ? g - 2 : 0; k < g; ++k)
          (void)mbar_wait(&kv_full[(k & 1u) * kBlocks + lane], (k >> 1) & 1u);
    } else if (warp == kMmaWarp) {
      // ------------------------- matrix products --------------------------
      constexpr uint32_t kQk = idesc(kBK, false), kPv = idesc(64, true);
      const bool leader = elect_one();
      uint32_t g = 0, sn = 0, qn = 0;  // block groups and key tiles so far, phase of q_full
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        if (!__all_sync(0xffffffffu, mbar_test(bar, phase)) && !dead)
          dead = !__all_sync(0xffffffffu, mbar_wait(bar, phase));
        tc_fence_after();
      };
      const uint64_t q_desc = smem_desc_sw128(q_smem), k_desc = smem_desc_sw128(ring0),
                     v_desc = smem_desc_sw128_mn(ring0, kBlock);
      auto qk = [&](uint32_t tile, bool last) {  // scores of the CTA's tile-th key tile
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk) {
          const uint32_t slot = (g & 1u) * kBlocks + blk;
          wait(&kv_full[slot], (g >> 1) & 1u);
          if (leader) {
            if (!dead) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma_ss(tmem + (tile & 1u) * kBK, q_desc + (blk * kBlock + k * 32 >> 4),
                          k_desc + (slot * kBlock >> 4) + (k * 32 >> 4), kQk, blk + k > 0);
            }
            tc_commit(smem_addr(&kv_empty[slot]));
          }
          __syncwarp();
        }
        if (leader) {
          tc_commit(smem_addr(&s_full[tile & 1u]));
          if (last) tc_commit(smem_addr(&q_free));  // the segment's queries are done with
        }
        __syncwarp();
        ++g;
      };
      auto pv = [&](uint32_t tile, bool first) {
        wait(&p_full[tile & 1u][0], (tile >> 1) & 1u);
        wait(&p_full[tile & 1u][1], (tile >> 1) & 1u);
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk) {
          const uint32_t slot = (g & 1u) * kBlocks + blk;
          wait(&kv_full[slot], (g >> 1) & 1u);
          if (leader) {
            if (!dead) {
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                tc_mma_ts(tmem + kOCol + blk * 64, tmem + (tile & 1u) * kBK + k * 8,
                          v_desc + (slot * kBlock >> 4) + k * (2048 >> 4), kPv, !first || k > 0);
            }
            tc_commit(smem_addr(&kv_empty[slot]));
          }
          __syncwarp();
        }
        if (leader) tc_commit(smem_addr(&o_done[tile & 1u]));
        __syncwarp();
        ++g;
      };
      while (walk.next(a, s)) {
        if (s.tiles == 0) continue;
        wait(&q_full, qn);
        qn ^= 1u;
        qk(sn, s.tiles == 1);
        for (int t = 0; t < s.tiles; ++t, ++sn) {
          // The products run in issue order: these scores take the place of the
          // weights that the product before last has read.
          if (t + 1 < s.tiles) qk(sn + 1, t + 2 == s.tiles);
          pv(sn, t == 0);
        }
      }
      if (dead && lane == 0) report_give_up(8u);
      if (leader) {  // no product is in flight when the tensor memory is freed
        tc_commit(smem_addr(&mma_done));
        (void)mbar_wait(&mma_done, 0);
      }
      __syncwarp();
    } else {
      // ----------------------------- queries ------------------------------
      // 64 rows a warp; the next segment's while the last products of this run
      const int w = warp - kQueryWarp;
      uint32_t free = 0;
      bool loaded = false;
      while (walk.next(a, s)) {
        if (s.tiles == 0) continue;
        if (loaded) {
          if (!dead && !mbar_wait(&q_free, free)) {
            dead = true;
            report_give_up(32u);
          }
          free ^= 1u;
        }
        loaded = true;
        __syncwarp();
        // lane: one of a row's 32 16-byte pieces
        const int t = (s.r0 + w * 64) / a.G;
        int gq = s.r0 + w * 64 - t * a.G;
        const int dt = 1 / a.G, dg = 1 - dt * a.G;
        const long long step = dt * a.q_stride + dg * D, carry = a.q_stride - (long long)a.G * D;
        const __nv_bfloat16 *base =
            a.q + (long long)s.rq.q0 * a.q_stride + (long long)s.h * a.G * D + lane * 8;
        const __nv_bfloat16 *src = base + (long long)t * a.q_stride + (long long)gq * D;
        const uint32_t dst = q_smem + (uint32_t)(lane >> 3) * kBlock;
#pragma unroll 4
        for (int rr = w * 64; rr < w * 64 + 64; ++rr) {
          const bool real = rr < s.count;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           dst + (uint32_t)rr * 128 + (uint32_t)(((lane & 7) ^ (rr & 7)) << 4)),
                       "l"(real ? src : base), "r"(real ? 16 : 0)
                       : "memory");
          src += step;
          gq += dg;
          if (gq >= a.G) {
            gq -= a.G;
            src += carry;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
    }
  } else {
    // ------------------------------- softmax ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 tensor-memory lanes a warp
    const uint32_t o_at = tmem + lanes + kOCol + (uint32_t)wg * (D / 2);  // this group's columns
    const float c = a.scale_log2;
    uint32_t g0 = 0, sn = 0;  // block groups of the segments before, key tiles so far
    auto wait = [&](uint64_t *bar, uint32_t phase) {
      if (!mbar_test(bar, phase) && !dead && !mbar_wait(bar, phase)) {
        dead = true;
        report_give_up(16u);
      }
      __syncwarp();  // the tensor-memory accesses that follow want the whole warp
    };
    // The product of a tile is done.  Tiles alternate between two barriers: the
    // scores that a group holds may be a product ahead, so the last two products
    // can both be open, and one barrier's parity would not tell them apart.
    auto wait_product = [&](uint32_t tile) { wait(&o_done[tile & 1u], (tile >> 1) & 1u); };
    while (walk.next(a, s)) {
      const bool ok = row < s.count;
      const int r = s.r0 + row;
      const int t_row = ok ? r / a.G : 0;
      const int last = ok ? s.rq.len - s.rq.n + t_row : -1;
      const int first = a.window > 0 ? last - a.window + 1 : 0;
      float m = kNegInf, l = 0.f;
      bool any_masked = false;
      for (int t = 0; t < s.tiles; ++t, ++sn) {
        const int j0 = (s.tile0 + t) * kBK;
        const bool masked = j0 < s.span.all_lo || j0 + kBK > s.span.all_hi;
        const uint32_t s_at = tmem + lanes + (sn & 1u) * kBK;
        wait(&s_full[sn & 1u], (sn >> 1) & 1u);
        tc_fence_after();
        uint32_t x[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tc_ld_x32(s_at + wg * 64 + 32 * q, x[q]);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 2; ++q) pin(x[q]);
        if (masked) {
          any_masked = true;
          const int lo = first - j0 - wg * 64, hi = last - j0 - wg * 64;
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * q + i > hi || 32 * q + i < lo) x[q][i] = __float_as_uint(kNegInf);
        }
        float mx[2] = {kNegInf, kNegInf};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(x[q][i]), __uint_as_float(x[q][i + 1])));
        const float mine = fmaxf(mx[0], mx[1]);
        s_x[sn & 1u][wg][row] = mine;
        tc_fence_before();
        pair_sync();  // both groups have read the scores: the weights may take their place
        tc_fence_after();
        const float mn = fmaxf(m, fmaxf(mine, s_x[sn & 1u][wg ^ 1][row]));
        if (t == 0) {
          m = mn;
        } else {
          const bool grew = (mn - m) * c > kRescale;  // the same in both groups
          if (__any_sync(0xffffffffu, grew)) {
            float f = 1.f;
            if (grew) {
              f = exp2_approx((m - mn) * c);
              m = mn;
              l *= f;
            }
            wait_product(sn - 1u);
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < D / 2; d += 32) {
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
        if (masked) {
          // as in paged_attn_tc.cu, two blocks of the tile's values a group
          const uint32_t vg = g0 + (t + 1 < s.tiles ? 2 + 2 * t : 2 * s.tiles - 1);
          bool odd = false;
          // the values before these in the slot have landed when their product
          // is done (at a first tile it held what is long multiplied)
          if (t > 0) wait_product(sn - 1u);
#pragma unroll 1
          for (int blk = 2 * wg; blk < 2 * wg + 2; ++blk) {
            const uint32_t slot_v = (vg & 1u) * kBlocks + blk;
            wait(&kv_full[slot_v], (vg >> 1) & 1u);
            uint8_t *v = smem_raw + (ring0 - raw) + slot_v * kBlock + row * 16;
#pragma unroll 1
            for (int i = 0; i < kBK / 16; ++i) {  // eight threads a key
              const int p0 = j0 + i * 16, pos = p0 + (row >> 3);
              if (p0 >= s.span.all_lo && p0 + 16 <= s.span.all_hi) continue;
              const bool none = pos < s.span.lo || pos >= s.span.hi;
              uint4 *at = reinterpret_cast<uint4 *>(v + i * 2048);
              if (none) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (pos < s.span.all_lo || pos >= s.span.all_hi) {
                uint4 y = *at;
                if (nonfinite_bits(y)) {
                  clear_nonfinite(y);
                  *at = y;
                  odd = true;
                }
              }
            }
          }
          if (odd) s_odd = 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const float off = m == kNegInf ? 0.f : m * c;
        const uint64_t c2 = pack2(c, c), off2 = pack2(-off, -off);
        uint64_t acc[4] = {0, 0, 0, 0};  // pairs of zeros
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            unpack2(fma2(pack2(__uint_as_float(x[q][2 * i]), __uint_as_float(x[q][2 * i + 1])), c2,
                         off2),
                    e0, e1);
            e0 = exp2_approx(e0);
            e1 = exp2_approx(e1);
            acc[i & 3] = add2(acc[i & 3], pack2(e0, e1));
            p[i] = pack_bf16(e0, e1);
          }
          tc_st_x16(s_at + 32 * wg + 16 * q, p);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sn & 1u][wg]);
        {
          float e0, e1;
          unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), e0, e1);
          l += e0 + e1;
        }
      }
      g0 += 2 * s.tiles;

      // ---- the segment's rows: half of the columns a group ----
      const bool whole = s.first == 0 && s.n_units == s.width;
      const int slot = 2 * (int)blockIdx.x + (s.first == 0 ? 1 : 0);
      pair_sync();  // s_x of the last tile has been read, s_odd is written
      s_x[0][wg][row] = l;
      const bool odd = any_masked && s_odd != 0;
      pair_sync();
      l = s_x[0][0][row] + s_x[0][1][row];
      if (tid == 0) s_odd = 0;  // next written after the next segment's first barrier
      if (s.tiles > 0) {
        wait_product(sn - 1u);
        tc_fence_after();
        if (odd)
          add_nonfinite<D, D / 2>(a, s.b, s.h, max(s.span.lo, s.tile0 * kBK),
                                  min(s.span.hi, (s.tile0 + s.tiles) * kBK), s.span.all_lo,
                                  s.span.all_hi,
                                  ok ? a.q + (long long)(s.rq.q0 + t_row) * a.q_stride +
                                           (long long)(s.h * a.G + (r - t_row * a.G)) * D
                                     : nullptr,
                                  first, last, o_at, wg * (D / 2));
      }
      uint8_t *stage = smem_raw + (stage0 - raw) + (uint32_t)wg * kStage;
      const int g = r - t_row * a.G, t0 = s.r0 / a.G;
      if (wg == 0) s_row[row] = (uint32_t)(t_row - t0) << 16 | (uint32_t)g;
      pair_sync();  // s_x has been read, s_row is written
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float *part = part_base(a, slot) + row * 4;
      __nv_bfloat16 *dst = a.out + (long long)(s.rq.q0 + t0) * a.out_stride +
                           (long long)s.h * a.G * D + wg * (D / 2);
#pragma unroll 1
      for (int d = 0; d < D / 2; d += 32) {
        uint32_t o[32];
        if (s.tiles > 0) {
          tc_ld_x32(o_at + d, o);
          tc_wait_ld();
          pin(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (whole) {
          // through shared memory: four threads write 64 bytes of a row
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            auto two = [&](int k) {
              return pack_bf16(__uint_as_float(o[i + k]) * inv,
                               __uint_as_float(o[i + k + 1]) * inv);
            };
            *reinterpret_cast<uint4 *>(stage + row * 64 +
                                       (((i >> 3) ^ ((row >> 1) & 3)) << 4)) =
                make_uint4(two(0), two(2), two(4), two(6));
          }
          group_sync(wg);
#pragma unroll 4
          for (int i = row >> 2; i < s.count; i += 32) {
            const uint32_t at = s_row[i];
            const uint4 y = *reinterpret_cast<const uint4 *>(
                stage + i * 64 + (((row & 3) ^ ((i >> 1) & 3)) << 4));
            *reinterpret_cast<uint4 *>(dst + (at >> 16) * a.out_stride + (at & 0xFFFFu) * D + d +
                                       (row & 3) * 8) = y;
          }
          group_sync(wg);
        } else if (ok) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            __stcg(reinterpret_cast<uint4 *>(
                       part + (size_t)((wg * (D / 2) + d + i) >> 2) * kRows * 4),
                   make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
        }
        __syncwarp();
      }
      if (ok && whole && a.lse && wg == 0)
        a.lse[(long long)(s.rq.q0 + t_row) * a.Hq + s.h * a.G + g] = row_lse(a, m, l);
      if (ok && !whole) {
        __stcg(part_ml(a, slot, wg) + row, m);
        __stcg(part_ml(a, slot, wg) + kRows + row, l);
      }
      tc_fence_before();  // O has been read before the next segment's products write it
      if (!whole) {
        // ---- the last CTA to arrive joins this group's columns ----
        const int c0 = runs.owner(s.item), c1 = runs.owner(s.item + s.width - kItemUnits<kRows> - 1);
        float *weights = reinterpret_cast<float *>(stage);  // [partial][row]
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
              mm = fmaxf(mm, __ldcg(part_ml(a, join_slot(gr, c0, k), wg) + row));
#pragma unroll 4
            for (int k = 0; k < gr.n; ++k) {
              const float *ml = part_ml(a, join_slot(gr, c0, k), wg) + row;
              const float lk = __ldcg(ml + kRows), f = join_weight(a, __ldcg(ml), lk, mm);
              ll = fmaf(lk, f, ll);
              weights[k * kTile + row] = f;  // read by this thread alone
            }
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            __nv_bfloat16 *dst = a.out + (long long)(s.rq.q0 + t_row) * a.out_stride +
                                 (long long)(s.h * a.G + g) * D;
            const int to = join_slot(gr, c0, 0);
#pragma unroll 1
            for (int d = wg * (D / 2); d < (wg + 1) * (D / 2); d += 64) {
              float o[64];
#pragma unroll
              for (int i = 0; i < 64; ++i) o[i] = 0.f;
#pragma unroll 2
              for (int k = 0; k < gr.n; ++k) {
                const float f = weights[k * kTile + row];
                const float *part = part_base(a, join_slot(gr, c0, k)) + row * 4 +
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
                float *part = part_base(a, to) + row * 4 + (size_t)(d >> 2) * kRows * 4;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  __stcg(reinterpret_cast<float4 *>(part + (size_t)i * kRows * 4),
                         make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
              }
            }
            if (!gr.final) {
              __stcg(part_ml(a, to, wg) + row, mm);
              __stcg(part_ml(a, to, wg) + kRows + row, ll);
            } else if (a.lse && wg == 0) {
              a.lse[(long long)(s.rq.q0 + t_row) * a.Hq + s.h * a.G + g] = row_lse(a, mm, ll);
            }
          }
          if (gr.final) break;
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

int tc256_ctas() { return std::min(kMaxTcCtas, device_sm_count()); }

}  // namespace

size_t tc256_partial_bytes() { return (size_t)tc256_ctas() * 2 * kPartial * 4; }

unsigned tc256_take_give_up() {
  unsigned v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_give_up, sizeof v);
  cudaMemcpyToSymbol(g_give_up, &zero, sizeof zero);
  return v;
}

sv_status tc256_run(const Args &a, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  sv_status st = encode_cache(&kmap, a.k, D, a, kBK);
  if (st == SV_OK) st = encode_cache(&vmap, a.v, D, a, kBK);
  if (st != SV_OK) return st;
  static PerDeviceOnce once;
  const cudaError_t ce = once.run([] {
    return cudaFuncSetAttribute(attn_tc256_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kSmem);
  });
  if (ce != cudaSuccess)
    return fail(SV_ERR_CUDA, "paged_attention: cudaFuncSetAttribute failed: %s",
                cudaGetErrorString(ce));
  attn_tc256_kernel<<<(unsigned)tc256_ctas(), kThreads, kSmem, stream>>>(kmap, vmap, a);
  return check_launch("paged_attention");
}

}  // namespace attn
}  // namespace sv
