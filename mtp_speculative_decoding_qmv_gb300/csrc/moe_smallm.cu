// moe_smallm.cu -- a mixture-of-experts layer for few rows (1..128): router, the
// chosen experts' 4-bit products, their weighted sum, sm_103a.
//
//   z_e = x . r_e;  the top_k largest z (ties: the lower expert) with weights
//   w = softmax over them (or over all experts);
//   y = sum_j w_j down_ej(silu(gate_ej x) * up_ej x)
//
// A few rows meet most of their experts once, so the layer streams the chosen
// experts' weights (0.5625 bytes each) and is bound by memory.  Four launches,
// the later ones starting as the one before drains:
//  * route: 8 experts a CTA, K over its warps, bf16 MMAs (exact products, fp32 sums),
//    and the rows of x in the products' form; the last CTA of 16 rows chooses their
//    experts, the last of all sorts the (row, expert) pairs by expert and cuts each
//    expert's rows into slots of up to 8, the columns of one MMA;
//  * gate and up, then down: the stages of all slots' tiles laid out flat and cut
//    evenly over the resident CTAs, so every SM streams the same number of bytes
//    whichever experts were chosen.  A stage is 128 weight rows x 256 inputs: 64
//    rows of gate and the same 64 of up (their product leaves in one place), or
//    128 of down, with the rows' activations.  Eight warps take 32 rows by half of
//    the inputs each.  A producer warp keeps the ring of stages full across tiles, and
//    a warp of its own takes the sums of a finished tile, so that neither the copies
//    nor the products wait for it.  A tile cut between CTAs leaves partial sums, which
//    whichever CTA comes last adds in CTA order; nobody waits for another CTA, so the
//    launches need not be resident together;
//  * the sum of a row's experts, in the order of choice.
// Measured (us, in a graph): one row of 2048 inputs, 8 of 256 experts of 512, 27 (15
// MB, 4 launches of 3 .. 9 us that wait for one another); 4 rows of 5120, 6 of 64
// experts of 1024, 67 .. 72 (2.6 TB/s: the later launches' first loads, the merge of the
// split tiles and the launch itself are 8 .. 10 us each); 128 rows of
// 2048, 6 of 96 experts of 1024, 153 .. 158 (2.2 TB/s: products and the masking of nibbles).
//
// The nibbles are fp16 numbers as they stand: of a word, the even ones of each half
// masked are the subnormals q 2^-24, the odd ones 16 q 2^-24 against activations divided by
// 16, which the MMAs multiply exactly.  Five integer operations a word of eight, and
// nothing is added to a nibble that would have to be taken off a sum again.  (As 1024 + q,
// the form of a normal number, 1 to 2 % of the outputs were not the bf16 nearest to the
// exact value, now 0.1 to 0.3 %; 128 rows took 166 us, now 153 to 158.)
// The activations become fp16 once, before they are multiplied: per row and group of
// 64 scaled by a power of two that brings the largest to 2^14 .. 2^15, which loses
// nothing of a bf16 value down to 2^-28 of it.  Beside them lie the scale and the
// group's sum, for the bias.  The activations between the products are two such parts
// (2^-22).  As operands of down the parts of up to four rows share one MMA's eight
// columns; five to eight rows take two MMAs.
#include <cuda_fp16.h>

#include <algorithm>

#include "qmv_common.cuh"

namespace sv {
namespace {
using namespace qmv;

constexpr int kMaxRows = 128, kMaxTop = 16, kMaxExperts = 512;
constexpr int kSlotRows = 8;       // pairs of a slot
constexpr int kTileRows = 128;     // weight rows of a tile
constexpr int kStageK = 256;       // inputs of a stage
constexpr int kGroupsOf = kStageK / 64;
constexpr int kWarps = 8;          // that multiply; then the producer, then the finisher
constexpr int kMoeThreads = (kWarps + 2) * 32;
// A row's activations of a stage: four groups of 64 fp16, then a Group each.
struct alignas(16) Group {
  float f, sum;  // 1 / scale; the inputs' sum
};
constexpr uint32_t kRecord = kGroupsOf * (128 + (uint32_t)sizeof(Group));  // 576
constexpr uint32_t kXOff = 2 * kRows * 128;
// Scales, then biases, of a block of four stages: [128 rows][16 groups] bf16.
constexpr int kBlock = 4;
constexpr uint32_t kSbRow = kBlock * kGroupsOf * 2, kSbBytes = kTileRows * kSbRow;
template <bool kDown>
struct Ring {  // down: the two parts of eight rows
  static constexpr int kStages = kDown ? 2 : 3, kRecords = kDown ? 16 : 8;
  static constexpr uint32_t kStage = (kXOff + kRecords * kRecord + 1023) / 1024 * 1024;
  static constexpr uint32_t kSbOff = kStages * kStage;  // two blocks
  static constexpr uint32_t kRedOff = kSbOff + 2 * 2 * kSbBytes;
};
constexpr int kRedPitch = kTileRows + 4;  // floats: conflict-free both ways
constexpr uint32_t kRedPlane = kSlotRows * kRedPitch;      // floats: a half of the inputs
constexpr uint32_t kRedSize = 2 * kRedPlane * 4;           // two of them
template <bool kDown>
struct Smem {
  static constexpr uint32_t kLastOff = Ring<kDown>::kRedOff + 2 * kRedSize;
  static constexpr uint32_t kBarOff = kLastOff + 16;
  static constexpr uint32_t kTotal = kBarOff + (2 * Ring<kDown>::kStages + 9) * 8 + 1024;
};
constexpr int kPartFloats = kTileRows * kSlotRows;

__device__ unsigned int g_moe_device_error;

struct alignas(16) Slot {
  int expert, first, n, pad;
};
// What the caller's workspace holds.  The counters come first: zero before a call
// and left zero by it.
struct Space {
  uint32_t *routed;   // [row tiles] CTAs of the router that are done, then row tiles that are
  uint32_t *tiles;    // [slots][tiles] segments of a split tile
  float *logits;      // [rows][experts]
  int32_t *ids;       // [rows][top]
  float *weights;     // [rows][top]
  int32_t *order;     // the pairs row * top + j by expert
  int32_t *n_slots;
  Slot *slots;
  uint8_t *x;         // [rows][stages of gate and up] records
  uint8_t *h;         // [2][pairs][stages of down] records: the first parts, the second
  float *d;           // [pairs][hidden]
  float *parts;       // [CTAs][2][kPartFloats]
  size_t counters, total;  // bytes
};
inline int slots_most(int rows, int experts, int top) {
  const int pairs = rows * top;
  return std::min(experts, pairs) + pairs / kSlotRows;
}
Space space_of(void *base, int rows, int hidden, int inter, int experts, int top, int ctas) {
  Space s = {};
  size_t at = 0;
  uint8_t *b = static_cast<uint8_t *>(base);
  auto take = [&](auto *&p, size_t n) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(b + at);
    at += (n * sizeof(*p) + 255) / 256 * 256;
  };
  const size_t pairs = (size_t)rows * top, slots = (size_t)slots_most(rows, experts, top);
  const size_t up = inter / 64, down = hidden / kTileRows;
  // the counters' place is that of the most rows, so that a workspace serves any fewer
  take(s.routed, kMaxRows / 16 + 1);
  take(s.tiles, (size_t)slots_most(kMaxRows, experts, top) * std::max(up, down));
  s.counters = at;
  take(s.logits, (size_t)rows * experts);
  take(s.ids, pairs);
  take(s.weights, pairs);
  take(s.order, pairs);
  take(s.n_slots, 1);
  take(s.slots, slots);
  take(s.x, (size_t)rows * ((hidden + kStageK - 1) / kStageK) * kRecord);
  take(s.h, 2 * pairs * ((inter + kStageK - 1) / kStageK) * kRecord);
  take(s.d, pairs * hidden);
  take(s.parts, (size_t)ctas * 2 * kPartFloats);
  s.total = at;
  return s;
}

struct MoeArgs {
  const __nv_bfloat16 *x, *router;
  const uint16_t *gate_s, *gate_b, *up_s, *up_b, *down_s, *down_b;
  __nv_bfloat16 *y;
  int32_t *ids_out;     // may be null
  float *weights_out;   // may be null
  Space ws;
  int rows, hidden, inter, experts, top, renormalize;
};

// ---- activations in the products' form ----------------------------------------------
// A group's 64 inputs, two a lane (2 lane and 2 lane + 1), to its place in a record:
// scaled, the odd ones of each word of eight divided by 16, a word's in the order 0 4 1
// 5 2 6 3 7 of the masked nibbles.  kParts 2: what the fp16 values leave goes to the
// record `low` bytes further, the same way.  By a whole warp.
template <int kParts>
__device__ __forceinline__ void put_group(uint8_t *record, size_t low, int group, float2 v) {
  const int lane = threadIdx.x & 31;
  auto finite = [](float x) {
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
  };
  const uint32_t most = __reduce_max_sync(0xffffffffu, max(finite(v.x), finite(v.y)));
  const int e = min(14 - ((int)(most >> 23) - 127), 126);
  const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  float2 rest = make_float2(v.x * scale, v.y * scale);
  // inputs 2 i and 2 i + 1 of a word: places i < 2: 4 i and 4 i + 2, else 4 i - 7 and 4 i - 5
  const int i = lane & 3, place = i < 2 ? 4 * i : 4 * i - 7;
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    uint8_t *to = record + part * low;
    const __half a = __float2half_rn(rest.x), b = __float2half_rn(rest.y * 0.0625f);
    const float fa = __half2float(a), fb = __half2float(b);
    __half *h = reinterpret_cast<__half *>(to + (group & 3) * 128) + (lane >> 2) * 8 + place;
    h[0] = a;
    h[2] = b;
    const float sum = warp_sum(fa + 16.f * fb);
    if (lane == 0)
      *reinterpret_cast<float2 *>(to + kGroupsOf * 128 + (group & 3) * sizeof(Group)) =
          make_float2(f, f * sum);
    rest.x -= fa;
    rest.y -= 16.f * fb;
  }
}

// ---- router ---------------------------------------------------------------------
constexpr int kRouteTile = 16;     // rows of x
constexpr int kRouteExperts = 8;

// Larger floats have larger keys; NaN has the smallest.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if (f != f) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The experts of row t, by a warp: top times the largest key, of equal ones the
// lowest expert.  Lane l holds experts l + 32 i, and the best of them that is left;
// only the lane whose best is taken looks for its next.
template <int kPer>
__device__ void choose(const MoeArgs &a, int t, int32_t *ids) {
  const int lane = threadIdx.x & 31;
  const float *z = a.ws.logits + (size_t)t * a.experts;
  float v[kPer];
  uint32_t key[kPer];  // 0: none (a NaN is 1)
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = lane + 32 * i < a.experts ? __ldcg(z + lane + 32 * i) : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < a.experts ? order_key(v[i]) + 1u : 0u;
  uint32_t best;
  int at;
  float value;
  auto look = [&] {
    best = key[0];
    at = lane;
    value = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
        value = v[i];
      }
  };
  look();
  float mine = 0.f, most = 0.f;  // lane j: the logit of choice j
  int id = 0;
  for (int j = 0; j < a.top; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int chosen = __reduce_min_sync(0xffffffffu, best == top ? at : kMaxExperts);
    const float x = __shfl_sync(0xffffffffu, value, chosen & 31);
    if (j == 0) most = x;
    if (lane == j) {
      mine = x;
      id = chosen;
    }
    if (lane == (chosen & 31)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i == chosen) key[i] = 0u;
      look();
    }
    __syncwarp();
  }
  float w = lane < a.top ? expf(mine - most) : 0.f, sum = w;
  if (!a.renormalize) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < a.experts) sum += expf(v[i] - most);
  }
  w /= warp_sum(sum);
  if (lane < a.top) {
    const int p = t * a.top + lane;
    a.ws.ids[p] = id;
    a.ws.weights[p] = w;
    ids[lane] = id;
    if (a.ids_out) a.ids_out[p] = id;
    if (a.weights_out) a.weights_out[p] = w;
  }
}

// The pairs by expert (rows ascending), and the slots.  A bit a row and expert
// makes the order the same whoever sets the bits first.
constexpr int kRouteThreads = 512;
__device__ void make_slots(const MoeArgs &a, const int32_t (*chosen)[kMaxTop], uint32_t (*bits)[4],
                           int *first, int *scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = a.rows * a.top;
  // one CTA has chosen for up to 16 rows
  auto expert = [&](int p, int t) {
    return a.rows <= kRouteTile ? chosen[t][p - t * a.top] : __ldcg(a.ws.ids + p);
  };
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int t = p / a.top, e = expert(p, t);
    atomicOr(&bits[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // an expert a thread: its pairs and slots in one scan (pairs << 16 | slots)
  static_assert(kRouteThreads == kMaxExperts, "an expert a thread");
  const int n = __popc(bits[tid][0]) + __popc(bits[tid][1]) + __popc(bits[tid][2]) + __popc(bits[tid][3]);
  int upto = (n << 16) | ((n + kSlotRows - 1) / kSlotRows);
  const int own = upto;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  int before = upto - own;
  for (int i = 0; i < warp; ++i) before += scan[i];
  const int at = before >> 16;
  int slot = before & 0xffff;
  first[tid] = at;
  for (int i = 0; i < n; i += kSlotRows)
    a.ws.slots[slot++] = Slot{tid, at + i, min(kSlotRows, n - i), 0};
  if (tid == kRouteThreads - 1) *a.ws.n_slots = slot;
  __syncthreads();
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int t = p / a.top, e = expert(p, t);
    int rank = __popc(bits[e][t >> 5] & ((1u << (t & 31)) - 1u));
    for (int i = 0; i < t >> 5; ++i) rank += __popc(bits[e][i]);
    a.ws.order[first[e] + rank] = p;
  }
}

__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const MoeArgs a) {
  constexpr int kRouteWarps = kRouteThreads / 32;
  __shared__ float red[kRouteWarps][kRouteTile][kRouteExperts];
  __shared__ uint32_t bits[kMaxExperts][4];
  __shared__ int first[kMaxExperts], scan[kRouteWarps];
  __shared__ int32_t chosen[kRouteTile][kMaxTop];
  __shared__ uint32_t s_old;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  const int routers = (a.experts + kRouteExperts - 1) / kRouteExperts;
  const int e0 = blockIdx.x * kRouteExperts, t0 = blockIdx.y * kRouteTile;
  pdl_launch_dependents();
  *reinterpret_cast<uint4 *>(bits[tid]) = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();
  if ((int)blockIdx.x >= routers) {
    // a row a warp: one record of the rows' form for the products
    const int t = t0 + warp, record = blockIdx.x - routers, records = gridDim.x - routers;
    if (t >= a.rows) return;
    uint32_t u[kGroupsOf];
#pragma unroll
    for (int i = 0; i < kGroupsOf; ++i) {
      const int g = record * kGroupsOf + i;
      u[i] = 64 * g < a.hidden
                 ? __ldg(reinterpret_cast<const uint32_t *>(a.x + (size_t)t * a.hidden + 64 * g) + lane)
                 : 0u;
    }
#pragma unroll
    for (int i = 0; i < kGroupsOf; ++i)
      put_group<1>(a.ws.x + ((size_t)t * records + record) * kRecord, 0, i,
                   make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)));
    return;
  }
  // A: 16 rows of x, B: 8 experts.  A lane's 16 bytes are 8 inputs of a block of
  // 32, in the same places of both, so their order within the block does not matter.
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 *ra = reinterpret_cast<const uint4 *>(a.x + (size_t)(t0 + g8) * a.hidden) + t4;
  const uint4 *rb = reinterpret_cast<const uint4 *>(a.x + (size_t)(t0 + g8 + 8) * a.hidden) + t4;
  const uint4 *we = reinterpret_cast<const uint4 *>(a.router + (size_t)(e0 + g8) * a.hidden) + t4;
  const bool has_a = t0 + g8 < a.rows, has_b = t0 + g8 + 8 < a.rows, has_e = e0 + g8 < a.experts;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int blocks = a.hidden / 32;
  constexpr int kFly = 5;
  for (int b0 = warp; b0 < blocks; b0 += kRouteWarps * kFly) {
    uint4 xa[kFly], xb[kFly], w[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int b = b0 + kRouteWarps * i;
      const bool in = b < blocks;
      xa[i] = in && has_a ? __ldg(ra + 4 * b) : zero;
      xb[i] = in && has_b ? __ldg(rb + 4 * b) : zero;
      w[i] = in && has_e ? __ldg(we + 4 * b) : zero;
    }
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      mma_bf16_m16n8k16(acc, xa[i].x, xb[i].x, xa[i].y, xb[i].y, w[i].x, w[i].y);
      mma_bf16_m16n8k16(acc, xa[i].z, xb[i].z, xa[i].w, xb[i].w, w[i].z, w[i].w);
    }
  }
  red[warp][g8][2 * t4] = acc[0];
  red[warp][g8][2 * t4 + 1] = acc[1];
  red[warp][g8 + 8][2 * t4] = acc[2];
  red[warp][g8 + 8][2 * t4 + 1] = acc[3];
  __syncthreads();
  if (tid < kRouteTile * kRouteExperts) {
    const int t = tid / kRouteExperts, e = tid % kRouteExperts;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) sum += red[w][t][e];
    if (t0 + t < a.rows && e0 + e < a.experts)
      __stcg(a.ws.logits + (size_t)(t0 + t) * a.experts + e0 + e, sum);
    __threadfence();
  }
  // the last CTA of these rows chooses their experts
  auto last = [&](uint32_t *counter, uint32_t of) {
    __syncthreads();
    if (tid == 0) {
      s_old = atomicAdd(counter, 1u);
      __threadfence();
    }
    __syncthreads();
    const bool is = s_old == of - 1u;
    if (is && tid == 0) *counter = 0u;
    return is;
  };
  if (!last(a.ws.routed + blockIdx.y, routers)) return;
  static_assert(kRouteWarps == kRouteTile, "a row a warp");
  if (t0 + warp < a.rows) {
    if (a.experts <= 64)
      choose<2>(a, t0 + warp, chosen[warp]);
    else if (a.experts <= 256)
      choose<8>(a, t0 + warp, chosen[warp]);
    else
      choose<kMaxExperts / 32>(a, t0 + warp, chosen[warp]);
  }
  __threadfence();
  if (gridDim.y == 1)
    __syncthreads();
  else if (!last(a.ws.routed + kMaxRows / 16, gridDim.y))
    return;
  make_slots(a, chosen, bits, first, scan);
}

// ---- the experts' products ---------------------------------------------------------
template <int kBytes>
__device__ __forceinline__ void copy_small(uint32_t dst, const uint8_t *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
// (no eviction hint: an expert with more than 8 rows has its weights read again)
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_record(uint32_t dst, const uint8_t *src, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(kRecord), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 lds64(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// A group's products of two tiles of 16 weight rows (w: ldmatrix of words t and 4 + t of
// rows g8 and g8 + 8) with the rows of x in fragments x[2], added to d; kParts 2: with
// low as well.  The tiles' chains alternate, so that no MMA waits for the one just issued.
template <int kParts>
__device__ __forceinline__ void group_f16(float (&d)[2][4], const uint32_t (&w)[2][4], const uint4 (&x)[2],
                                          const uint4 (&low)[2]) {
  constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      const uint32_t b0 = step ? x[i].z : x[i].x, b1 = step ? x[i].w : x[i].y;
      uint32_t q[2][4];
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        const uint32_t a = w[tile][2 * i] >> (8 * step), b = w[tile][2 * i + 1] >> (8 * step);
        q[tile][0] = a & kEven;
        q[tile][1] = b & kEven;
        q[tile][2] = a & kOdd;
        q[tile][3] = b & kOdd;
        mma_f16(d[tile], q[tile][0], q[tile][1], q[tile][2], q[tile][3], b0, b1);
      }
      if constexpr (kParts == 2) {
        const uint32_t c0 = step ? low[i].z : low[i].x, c1 = step ? low[i].w : low[i].y;
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
          mma_f16(d[tile], q[tile][0], q[tile][1], q[tile][2], q[tile][3], c0, c1);
      }
    }
}

// A warp's part of stages [s0, s1) of a tile: rows 32 (w % 4) .. of the stage and half
// w / 4 of its inputs.  Lane (g8, t4): weight rows g8 + 8 i; of the activations column
// (row) g8; of the sums columns 2 t4 and 2 t4 + 1.  kBoth: a column a row, its two parts
// one after the other; else down's second parts are columns of their own.
template <bool kDown, bool kBoth>
__device__ __forceinline__ bool multiply(float2 (&acc)[2][2], uint32_t base, uint32_t full0,
                                         uint32_t empty0, uint32_t sb_full0, uint32_t sb_empty0,
                                         int &st, int &ph, int &blocks, int s0, int s1, int groups,
                                         int n) {
  using R = Ring<kDown>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3, rows0 = 32 * (warp & 3), half = warp >> 2;
  constexpr int apart = kDown && !kBoth ? 4 : kSlotRows;
  const bool valid = g8 % apart < n, real0 = 2 * t4 % apart < n, real1 = (2 * t4 + 1) % apart < n;
  const uint32_t w_at = (uint32_t)(rows0 + (lane & 15)) * 128;  // the second box follows the first
  const uint32_t x_at = kXOff + g8 * kRecord + half * 256 + t4 * 16;
  const uint32_t group_at =
      kXOff + 2 * t4 * kRecord + kGroupsOf * 128 + half * 2 * (uint32_t)sizeof(Group);
  constexpr uint32_t kLow = kSlotRows * kRecord;  // to a row's second part
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const float2 none = make_float2(0.f, 0.f), unit = make_float2(0x1p24f, 0x1p24f);
  for (int c = s0; c < s1; ++c) {
    if ((c == s0 || c % kBlock == 0) && !warp_wait_stage(sb_full0 + 8u * (blocks & 1), (blocks >> 1) & 1))
      return false;
    if (!warp_wait_stage(full0 + 8u * st, ph)) return false;
    const uint32_t at = base + st * R::kStage;
    const uint32_t sb_at = base + R::kSbOff + (blocks & 1) * 2 * kSbBytes + (rows0 + g8) * kSbRow +
                           (c % kBlock) * 8 + half * 4;
    if (c * kGroupsOf + 2 * half < groups) {
      uint4 x[2][2], low[2][2];
      float2 r[2][2];
      uint32_t w[2][2][4], sw[4], bw[4];
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
          ldmatrix_x4(w[gi][tile], at + w_at + tile * 16 * 128 +
                                       (((4 * half + 2 * gi + (lane >> 4)) ^ (lane & 7)) << 4));
        x[gi][0] = valid ? lds128(at + x_at + gi * 128) : zero;
        x[gi][1] = valid ? lds128(at + x_at + gi * 128 + 64) : zero;
        r[gi][0] = real0 ? lds64(at + group_at + gi * 16) : none;
        r[gi][1] = real1 ? lds64(at + group_at + kRecord + gi * 16) : none;
        if constexpr (kBoth) {
          low[gi][0] = valid ? lds128(at + x_at + kLow + gi * 128) : zero;
          low[gi][1] = valid ? lds128(at + x_at + kLow + gi * 128 + 64) : zero;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sw[i] = lds32(sb_at + i * 8 * kSbRow);
        bw[i] = lds32(sb_at + kSbBytes + i * 8 * kSbRow);
      }
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
        const float2 f = make_float2(r[gi][0].x, r[gi][1].x);
        float2 sum = make_float2(r[gi][0].y, r[gi][1].y);
        if constexpr (kBoth) {
          const float2 q0 = real0 ? lds64(at + group_at + kLow + gi * 16) : none;
          const float2 q1 = real1 ? lds64(at + group_at + kLow + kRecord + gi * 16) : none;
          sum.x += q0.y;
          sum.y += q1.y;
        }
        float d[2][4] = {};
        group_f16<kBoth ? 2 : 1>(d, w[gi], x[gi], kBoth ? low[gi] : x[gi]);
        auto of = [&](uint32_t word) { return __uint_as_float(gi ? word & 0xFFFF0000u : word << 16); };
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // rows g8 and g8 + 8; columns 2 t4 and 2 t4 + 1
            const float s = of(sw[2 * tile + i]), b = of(bw[2 * tile + i]);
            // (the unit apart from 1 / scale, which alone may be 2^113)
            const float2 v = __fmul2_rn(f, __fmul2_rn(unit, make_float2(d[tile][2 * i], d[tile][2 * i + 1])));
            float2 &to = acc[tile][i];
            to = __ffma2_rn(make_float2(s, s), v, __ffma2_rn(make_float2(b, b), sum, to));
          }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(empty0 + 8u * st);
    if (c + 1 == s1 || c % kBlock == kBlock - 1) {
      if (lane == 0) mbar_arrive_u32(sb_empty0 + 8u * (blocks & 1));
      ++blocks;
    }
    if (++st == R::kStages) {
      st = 0;
      ph ^= 1;
    }
  }
  return true;
}

// The weights of a stage's two blocks of 64 rows.
struct Maps {
  CUtensorMap w[2];
};

// kDown false: h = silu(gate x) * (up x) of every slot; true: d = weight * (down h).
template <bool kDown>
__global__ void __launch_bounds__(kMoeThreads, 2)
    moe_experts_kernel(const __grid_constant__ Maps maps, const MoeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  using R = Ring<kDown>;
  using S = Smem<kDown>;
  constexpr int kStages = R::kStages;
  const uint32_t full0 = base + S::kBarOff, empty0 = full0 + 8 * kStages;
  const uint32_t red_full0 = empty0 + 8 * kStages, red_empty0 = red_full0 + 16;
  const uint32_t sb_full0 = red_empty0 + 16, sb_empty0 = sb_full0 + 16, done = sb_empty0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init_u32(full0 + 8u * i, 1);
      mbar_init_u32(empty0 + 8u * i, kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_u32(red_full0 + 8u * i, kWarps);
      mbar_init_u32(red_empty0 + 8u * i, 1);
      mbar_init_u32(sb_full0 + 8u * i, 32);
      mbar_init_u32(sb_empty0 + 8u * i, kWarps);
    }
    mbar_init_u32(done, 1);
    fence_mbar_init();
  }
  __syncthreads();
  // The slots are the router's, finished before any CTA of the gate and up launch
  // is past its wait; the down launch begins after that, and may read them and its
  // weights while the launch before it still runs.
  if (!kDown) pdl_wait();
  pdl_launch_dependents();
  const int K = kDown ? a.inter : a.hidden, N = kDown ? a.hidden : a.inter;
  constexpr int kStep = kDown ? kTileRows : kTileRows / 2;  // outputs of a tile
  const int tiles = N / kStep, stages = (K + kStageK - 1) / kStageK, groups = K / 64;
  const int n_slots = __ldcg(a.ws.n_slots), pairs = a.rows * a.top;
  const long long W = (long long)n_slots * tiles * stages;
  // Units a CTA: as few as the CTAs allow, or up to a quarter more where a tile is then
  // cut evenly, or not at all (W is below 2^28): a CTA with ends of two tiles joins both
  // of them.  (Us, without and with: one row, 8 of 256 experts, 2048 x 512, 30.5 and
  // 27.1; 4 rows, 6 of 64, 5120 x 1024, 72.7 and 67.9; 19 rows, 4 of 60, 2560 x 896, 73.7
  // and 69.8.  Up to half more: 27.7, 69.8, 70.1, and 128 rows 172 as against 167.)
  const int least = (int)((W + gridDim.x - 1) / gridDim.x);
  int p = least;
  while (4 * p <= 5 * least && (p < stages ? stages % p : p % stages) != 0) ++p;
  if (4 * p > 5 * least) p = least;
  const long long u_begin = (long long)p * blockIdx.x, u_end = min(W, u_begin + p);
  if (u_begin >= W) return;

  struct Segment {
    int tile, slot, n0, s0, s1;
  };
  auto segment = [&](long long u) {
    Segment g;
    g.tile = (int)(u / stages);
    g.slot = g.tile / tiles;
    g.n0 = (g.tile - g.slot * tiles) * kStep;
    g.s0 = (int)(u - (long long)g.tile * stages);
    g.s1 = (int)min((long long)stages, g.s0 + (u_end - u));
    return g;
  };

  // lane c: pair and weight of column c of a slot
  auto columns_of = [&](const Segment &g, int &n, int &pair, float &weight) {
    const int4 facts = __ldcg(reinterpret_cast<const int4 *>(a.ws.slots + g.slot));
    n = facts.z;
    pair = lane < n ? __ldcg(a.ws.order + facts.y + lane) : 0;
    weight = kDown && lane < n ? __ldcg(a.ws.weights + pair) : 0.f;
  };
  // a column's sums, rows 2 lane and 2 lane + 1 of both blocks of a tile
  auto emit = [&](const Segment &g, int p, float weight, float2 v0, float2 v1) {
    if constexpr (!kDown) {
      // a tile's 64 rows are one of down's groups
      const float2 h = make_float2(v0.x / (1.f + expf(-v0.x)) * v1.x, v0.y / (1.f + expf(-v0.y)) * v1.y);
      const int group = g.n0 / 64, records = (N + kStageK - 1) / kStageK;
      put_group<2>(a.ws.h + ((size_t)p * records + group / kGroupsOf) * kRecord,
                   (size_t)pairs * records * kRecord, group, h);
    } else {
      float *d = a.ws.d + (size_t)p * N + g.n0 + 2 * lane;
      __stcg(reinterpret_cast<float2 *>(d), make_float2(weight * v0.x, weight * v0.y));
      __stcg(reinterpret_cast<float2 *>(d + kRows), make_float2(weight * v1.x, weight * v1.y));
    }
  };

  if (warp == kWarps) {
    // ---- producer: weights by tensor copies, records by bulk copies, scales and
    // biases by small copies of a lane 8 (or 4) bytes, a block of four stages at a time: a
    // row's 32 bytes.  (Gate and up of 4 rows, 5120 x 1024, take 32 us with these copies
    // and 25 without; as tensor boxes of 16-byte rows 39.  Two stages a block and rings
    // of 4 and 3 stages: 128 rows in 177 us, as against 173.)  ---------------------------
    const bool wide = groups % 4 == 0;
    int st = 0, ph = 0, issued = 0, blocks = 0;
    bool ok = true;
    // down's first stages begin with their weights: the records are the launch
    // before's, and follow once it has ended
    bool waited = !kDown;
    const uint8_t *pending[kStages];
    auto bring_pending = [&] {
      pdl_wait();
      waited = true;
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        if (i < issued && pending[i])
          load_record(base + i * R::kStage + kXOff + lane * kRecord, pending[i], full0 + 8u * i);
    };
    // a slot's facts, read again where the slot changes: two trips to memory
    int slot = -1, n = 0;
    long long expert0 = 0;
    bool brings = false;
    const uint8_t *from = nullptr;
    for (long long u = u_begin; ok && u < u_end;) {
      const Segment g = segment(u);
      u += g.s1 - g.s0;
      if (g.slot != slot) {
        slot = g.slot;
        const int4 facts = __ldcg(reinterpret_cast<const int4 *>(a.ws.slots + slot));
        expert0 = (long long)facts.x * N;
        n = facts.z;
        // lane r brings record r: of row r, or of down's two parts r < n and the rest,
        // from place 4 on (up to four rows) or 8
        const int apart = n <= 4 ? 4 : 8, col = kDown ? lane % apart : lane;
        brings = col < n && lane < (kDown ? 2 * apart : kSlotRows);
        const int pair = brings ? __ldcg(a.ws.order + facts.y + col) : 0;
        from = kDown ? a.ws.h + ((size_t)pair + (lane >= apart ? pairs : 0)) * stages * kRecord
                     : a.ws.x + (size_t)(pair / a.top) * stages * kRecord;
      }
      const long long row0 = expert0 + g.n0;
      auto bring_block = [&](int block) {
        const uint32_t at = base + R::kSbOff + (blocks & 1) * 2 * kSbBytes;
        const uint16_t *from[4] = {kDown ? a.down_s : a.gate_s, kDown ? a.down_s : a.up_s,
                                   kDown ? a.down_b : a.gate_b, kDown ? a.down_b : a.up_b};
        constexpr int kLanes = kBlock * kGroupsOf / 4;  // a row's 8-byte pieces
        const int pieces = wide ? kLanes : 2 * kLanes, piece = lane % pieces, r = lane / pieces;
        const int group = block * kBlock * kGroupsOf + piece * (wide ? 4 : 2);
        if (group < groups) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {  // scales of the two blocks of rows, biases
            const uint8_t *p = reinterpret_cast<const uint8_t *>(
                from[m] + (row0 + (kDown ? kRows * (m & 1) : 0) + r) * groups + group);
            uint32_t to = at + m * (kRows * kSbRow) + r * kSbRow + piece * (wide ? 8 : 4);
            if (wide) {
#pragma unroll
              for (int i = 0; i < kRows; i += 32 / kLanes, p += 64 / kLanes * groups, to += 32 / kLanes * kSbRow)
                copy_small<8>(to, p);
            } else {
#pragma unroll 4
              for (int i = 0; i < kRows; i += 16 / kLanes, p += 32 / kLanes * groups, to += 16 / kLanes * kSbRow)
                copy_small<4>(to, p);
            }
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(sb_full0 + 8u * (blocks & 1))
                     : "memory");
        ++blocks;
      };
      const uint32_t bytes = 2 * kRows * 128 + (kDown ? 2 : 1) * n * kRecord;
      for (int c = g.s0; c < g.s1; ++c) {
        // (nothing is given free before the records are there)
        const bool new_block = c == g.s0 || c % kBlock == 0;
        if (!waited && (issued == kStages || (new_block && blocks == 2))) bring_pending();
        if (new_block) {
          if (blocks >= 2)
            ok = __all_sync(0xffffffffu,
                            mbar_wait_u32(sb_empty0 + 8u * (blocks & 1), ((blocks >> 1) & 1) ^ 1));
          if (!ok) break;
          bring_block(c / kBlock);
        }
        if (issued >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait_u32(empty0 + 8u * st, ph ^ 1));
        if (!ok) break;
        const uint32_t at = base + st * R::kStage, full = full0 + 8u * st;
        if (lane == 0) {
          mbar_arrive_expect_tx_u32(full, bytes);
          const int x = c * (kStageK / 8);
          load_box(at, &maps.w[0], x, (int)row0, full);
          load_box(at + kRows * 128, &maps.w[1], x, (int)row0 + (kDown ? kRows : 0), full);
        }
        __syncwarp();
        const uint8_t *record = brings ? from + (size_t)c * kRecord : nullptr;
        if (waited) {
          if (record) load_record(at + kXOff + lane * kRecord, record, full);
        } else {
#pragma unroll
          for (int i = 0; i < kStages; ++i)
            if (i == issued) pending[i] = record;
        }
        ++issued;
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!waited) bring_pending();
    if (!ok) {
      if (lane == 0) atomicOr(&g_moe_device_error, 1u);
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int i = max(0, issued - kStages); i < issued; ++i)  // the copies in flight
        (void)mbar_wait_u32(full0 + 8u * (i % kStages), (i / kStages) & 1);
    }
    return;
  }

  if (warp == kWarps + 1) {
    // ---- finisher: a tile's sums to where they go -----------------------------------
    if (kDown) pdl_wait();  // the partials' places are the launch before's
    int k = 0, slot = -1, n = 0, pair = 0;
    float weight = 0.f;
    bool ok = true;
    for (long long u = u_begin; ok && u < u_end; ++k) {
      const Segment g = segment(u);
      u += g.s1 - g.s0;
      if (g.slot != slot) columns_of(g, n, pair, weight);
      slot = g.slot;
      const bool whole = g.s0 == 0 && g.s1 == stages;
      // down's slots of up to four rows have the second parts' sums in columns 4..7
      const bool doubled = kDown && n <= 4;
      float *part = a.ws.parts + (size_t)(2 * blockIdx.x + (g.s0 == 0 ? 1 : 0)) * kPartFloats + 2 * lane;
      ok = __all_sync(0xffffffffu, mbar_wait_u32(red_full0 + 8u * (k & 1), (k >> 1) & 1));
      if (!ok) break;
      const float *red = reinterpret_cast<const float *>(smem + R::kRedOff + (k & 1) * kRedSize) + 2 * lane;
      for (int col = 0; col < n; ++col) {
        float2 v[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          v[x] = make_float2(0.f, 0.f);
          for (int y = col; y < (doubled ? kSlotRows : col + 1); y += 4)
#pragma unroll
            for (int plane = 0; plane < 2; ++plane) {
              const float2 f = *reinterpret_cast<const float2 *>(red + plane * kRedPlane + y * kRedPitch + x * kRows);
              v[x].x += f.x;
              v[x].y += f.y;
            }
        }
        if (whole) {
          emit(g, __shfl_sync(0xffffffffu, pair, col), __shfl_sync(0xffffffffu, weight, col), v[0], v[1]);
        } else {
          __stcg(reinterpret_cast<float2 *>(part + col * kTileRows), v[0]);
          __stcg(reinterpret_cast<float2 *>(part + col * kTileRows + kRows), v[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_u32(red_empty0 + 8u * (k & 1));
    }
    __threadfence();
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(done);
    if (!ok && lane == 0) atomicOr(&g_moe_device_error, 4u);
    return;
  }

  // ---- the products ----------------------------------------------------------------
  const int rows0 = 32 * (warp & 3), half = warp >> 2;
  int st = 0, ph = 0, blocks = 0, k = 0, slot = -1, n = 0;
  bool ok = true;
  for (long long u = u_begin; ok && u < u_end; ++k) {
    const Segment g = segment(u);
    u += g.s1 - g.s0;
    if (g.slot != slot) n = __ldcg(&a.ws.slots[g.slot].n);
    slot = g.slot;
    float2 acc[2][2] = {};
    if (kDown && n > 4)
      ok = multiply<kDown, kDown>(acc, base, full0, empty0, sb_full0, sb_empty0, st, ph, blocks, g.s0, g.s1,
                                   groups, n);
    else
      ok = multiply<kDown, false>(acc, base, full0, empty0, sb_full0, sb_empty0, st, ph, blocks, g.s0, g.s1,
                                   groups, n);
    // the sums to the finisher, red[half][column][row]
    if (ok && k >= 2)
      ok = __all_sync(0xffffffffu, mbar_wait_u32(red_empty0 + 8u * (k & 1), ((k >> 1) & 1) ^ 1));
    if (!ok) break;
    float *red = reinterpret_cast<float *>(smem + R::kRedOff + (k & 1) * kRedSize) + half * kRedPlane +
                 2 * (lane & 3) * kRedPitch + rows0 + (lane >> 2);
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      red[16 * tile] = acc[tile][0].x;
      red[16 * tile + kRedPitch] = acc[tile][0].y;
      red[16 * tile + 8] = acc[tile][1].x;
      red[16 * tile + 8 + kRedPitch] = acc[tile][1].y;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(red_full0 + 8u * (k & 1));
  }
  // ---- the end: what others count on, and what counts on others.  Once, when this
  // CTA's segments are all done: a fence and an atomic a segment took longer than a short
  // segment's products.
  if (ok) ok = __all_sync(0xffffffffu, mbar_wait_u32(done, 0));
  if (kDown) pdl_wait();  // (over by now)
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
  // a split tile at the beginning, one at the end: whoever comes last adds all of
  // their parts, in CTA order
  const int tile0 = (int)(u_begin / stages), tile1 = (int)((u_end - 1) / stages);
  const bool split0 = u_begin % stages != 0 || (tile0 == tile1 && u_end % stages != 0);
  const bool split1 = tile1 != tile0 && u_end % stages != 0;
  volatile int *last = reinterpret_cast<volatile int *>(smem + S::kLastOff);
  if (threadIdx.x < 2) {
    const int tile = threadIdx.x ? tile1 : tile0;
    bool is = false;
    if (ok && (threadIdx.x ? split1 : split0)) {
      const long long t0 = (long long)tile * stages;
      const uint32_t others = (uint32_t)(((int)t0 + stages - 1) / p - (int)t0 / p);
      __threadfence();  // the finisher's partial sums before the count
      is = atomicAdd(a.ws.tiles + tile, 1u) == others;
      if (is) a.ws.tiles[tile] = 0u;
      __threadfence();
    }
    last[threadIdx.x] = is;
  }
  sync();
  const bool last0 = last[0], last1 = last[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!(i ? last1 : last0)) continue;
    const long long t0 = (long long)(i ? tile1 : tile0) * stages;
    const Segment g = segment(t0);
    const int c0 = (int)t0 / p, c1 = ((int)t0 + stages - 1) / p;
    int n, pair;
    float weight;
    columns_of(g, n, pair, weight);
    if (warp < n) {  // a column a warp
      float2 v[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int c = c0; c <= c1; c += 4) {  // four CTAs' in flight
        float2 f[4][2];
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float *from = a.ws.parts + (size_t)(2 * (c + y) + (c + y == c0 ? 1 : 0)) * kPartFloats +
                                warp * kTileRows + x * kRows + 2 * lane;
            f[y][x] = c + y <= c1 ? __ldcg(reinterpret_cast<const float2 *>(from)) : make_float2(0.f, 0.f);
          }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            v[x].x += f[y][x].x;
            v[x].y += f[y][x].y;
          }
      }
      emit(g, __shfl_sync(0xffffffffu, pair, warp), __shfl_sync(0xffffffffu, weight, warp), v[0], v[1]);
    }
  }
  if (!ok && lane == 0) atomicOr(&g_moe_device_error, 2u);
}

// y: a row's sums over its experts, in the order of choice; four columns a thread.
// (By whichever CTA of the launch before came last at a tile of y, without this launch:
// most tiles' last slots end together, and one CTA was left with nearly all of them.)
constexpr int kSumThreads = 128;
__global__ void __launch_bounds__(kSumThreads) moe_sum_kernel(const MoeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int n = 4 * (blockIdx.x * kSumThreads + threadIdx.x);
  if (n >= a.hidden) return;
  const float *d = a.ws.d + (size_t)blockIdx.y * a.top * a.hidden + n;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < a.top; j0 += 8) {
    float4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = j0 + j < a.top ? __ldcg(reinterpret_cast<const float4 *>(d + (size_t)(j0 + j) * a.hidden))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum.x += x[j].x;
      sum.y += x[j].y;
      sum.z += x[j].z;
      sum.w += x[j].w;
    }
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
  *reinterpret_cast<uint2 *>(a.y + (size_t)blockIdx.y * a.hidden + n) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

int moe_ctas() { return 2 * device_sm_count(); }

sv_status check_sizes(const char *who, int rows, int hidden, int inter, int experts, int top) {
  if (rows < 0 || hidden < 1 || inter < 1 || experts < 1 || top < 1 || top > experts)
    return fail(SV_ERR_INVALID_ARG, "%s: need rows >= 0, hidden, inter, experts >= 1, 1 <= top_k <= experts",
                who);
  if (rows > kMaxRows) return fail(SV_ERR_UNSUPPORTED, "%s: %d rows > %d", who, rows, kMaxRows);
  if (experts > kMaxExperts)
    return fail(SV_ERR_UNSUPPORTED, "%s: %d experts > %d", who, experts, kMaxExperts);
  if (top > kMaxTop) return fail(SV_ERR_UNSUPPORTED, "%s: top_k=%d > %d", who, top, kMaxTop);
  if (hidden % 128 || inter % 128)
    return fail(SV_ERR_UNSUPPORTED, "%s: hidden and inter must be multiples of 128 (%d, %d)", who,
                hidden, inter);
  if (hidden > 65536 || inter > 65536 || (long long)experts * std::max(hidden, inter) > (1ll << 30))
    return fail(SV_ERR_UNSUPPORTED, "%s: sizes too large", who);
  return SV_OK;
}

}  // namespace

unsigned take_device_error_moe() {
  unsigned v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_moe_device_error, sizeof v);
  cudaMemcpyToSymbol(g_moe_device_error, &zero, sizeof zero);
  return v;
}

}  // namespace sv

using namespace sv;

extern "C" size_t moe_smallm_workspace_bytes(int rows, int hidden, int inter, int experts, int top_k,
                                             size_t *zero_bytes) {
  clear_error();
  if (check_sizes("moe_smallm_workspace_bytes", rows, hidden, inter, experts, top_k) != SV_OK) return 0;
  const Space s = space_of(nullptr, std::max(rows, 1), hidden, inter, experts, top_k, moe_ctas());
  if (zero_bytes) *zero_bytes = s.counters;
  return s.total;
}

extern "C" sv_status moe_smallm(const uint16_t *x, const uint16_t *router, const uint32_t *gate_w,
                                const uint16_t *gate_s, const uint16_t *gate_b,
                                const uint32_t *up_w, const uint16_t *up_s, const uint16_t *up_b,
                                const uint32_t *down_w, const uint16_t *down_s,
                                const uint16_t *down_b, int rows, int hidden, int inter,
                                int experts, int top_k, int renormalize, uint16_t *y, int32_t *ids,
                                float *weights, void *workspace, size_t workspace_bytes,
                                sv_stream_t stream) {
  clear_error();
  const char *who = "moe_smallm";
  sv_status st = check_sizes(who, rows, hidden, inter, experts, top_k);
  if (st != SV_OK) return st;
  if (rows == 0) return SV_OK;
  struct Buf {
    const void *p;
    size_t n;
    size_t align;
  };
  const size_t gate_n = (size_t)experts * inter * hidden;
  const Buf in[] = {{x, (size_t)rows * hidden * 2, 16},
                    {router, (size_t)experts * hidden * 2, 16},
                    {gate_w, gate_n / 2, 16},
                    {gate_s, gate_n / 32, 16},
                    {gate_b, gate_n / 32, 16},
                    {up_w, gate_n / 2, 16},
                    {up_s, gate_n / 32, 16},
                    {up_b, gate_n / 32, 16},
                    {down_w, gate_n / 2, 16},
                    {down_s, gate_n / 32, 16},
                    {down_b, gate_n / 32, 16}};
  for (const Buf &b : in)
    if (!b.p) return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!y || !workspace) return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const Buf &b : in)
    if (!aligned(b.p, b.align))
      return fail(SV_ERR_INVALID_ARG,
                  "%s: x, router, w_packed, scales and biases must be 16-byte aligned", who);
  if (!aligned(y, 8) || (ids && !aligned(ids, 4)) || (weights && !aligned(weights, 4)) ||
      !aligned(workspace, 256))
    return fail(SV_ERR_INVALID_ARG, "%s: y must be 8-byte, the workspace 256-byte aligned", who);
  const int ctas = moe_ctas();
  const Space ws = space_of(workspace, rows, hidden, inter, experts, top_k, ctas);
  if (workspace_bytes < ws.total)
    return fail(SV_ERR_INVALID_ARG, "%s: the workspace has %zu bytes, %zu are needed", who,
                workspace_bytes, ws.total);
  const Buf out[] = {{y, (size_t)rows * hidden * 2, 8},
                     {ids, ids ? (size_t)rows * top_k * 4 : 0, 4},
                     {weights, weights ? (size_t)rows * top_k * 4 : 0, 4},
                     {workspace, ws.total, 256}};
  for (int i = 0; i < 4; ++i) {
    for (const Buf &b : in)
      if (overlaps(out[i].p, out[i].n, b.p, b.n))
        return fail(SV_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(SV_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap", who);
  }
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    const cudaError_t x = cudaFuncSetAttribute(
        moe_experts_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<false>::kTotal);
    return x != cudaSuccess ? x
                            : cudaFuncSetAttribute(moe_experts_kernel<true>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Smem<true>::kTotal);
  });
  if (e != cudaSuccess)
    return fail(SV_ERR_CUDA, "%s: cudaFuncSetAttribute failed: %s", who, cudaGetErrorString(e));
  Maps up_maps, down_maps;
  auto encode = [&](CUtensorMap *map, const uint32_t *w, int n, int k) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, w, (uint64_t)k / 8, (uint64_t)experts * n,
                     (uint64_t)k / 2, kBoxWords, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  st = encode(&up_maps.w[0], gate_w, inter, hidden);
  if (st == SV_OK) st = encode(&up_maps.w[1], up_w, inter, hidden);
  if (st == SV_OK) st = encode(&down_maps.w[0], down_w, hidden, inter);
  if (st != SV_OK) return st;
  down_maps.w[1] = down_maps.w[0];
  MoeArgs a = {};
  a.x = reinterpret_cast<const __nv_bfloat16 *>(x);
  a.router = reinterpret_cast<const __nv_bfloat16 *>(router);
  a.gate_s = gate_s;
  a.gate_b = gate_b;
  a.up_s = up_s;
  a.up_b = up_b;
  a.down_s = down_s;
  a.down_b = down_b;
  a.y = reinterpret_cast<__nv_bfloat16 *>(y);
  a.ids_out = ids;
  a.weights_out = weights;
  a.ws = ws;
  a.rows = rows;
  a.hidden = hidden;
  a.inter = inter;
  a.experts = experts;
  a.top = top_k;
  a.renormalize = renormalize;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = &early;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cfg.gridDim = dim3((experts + kRouteExperts - 1) / kRouteExperts + (hidden + kStageK - 1) / kStageK,
                     (rows + kRouteTile - 1) / kRouteTile);
  cfg.blockDim = dim3(kRouteThreads);
  cudaError_t le = cudaLaunchKernelEx(&cfg, moe_route_kernel, a);
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = Smem<false>::kTotal;
  if (le == cudaSuccess) le = cudaLaunchKernelEx(&cfg, moe_experts_kernel<false>, up_maps, a);
  cfg.dynamicSmemBytes = Smem<true>::kTotal;
  if (le == cudaSuccess) le = cudaLaunchKernelEx(&cfg, moe_experts_kernel<true>, down_maps, a);
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3((hidden + 4 * kSumThreads - 1) / (4 * kSumThreads), rows);
  cfg.blockDim = dim3(kSumThreads);
  if (le == cudaSuccess) le = cudaLaunchKernelEx(&cfg, moe_sum_kernel, a);
  if (le != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(SV_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(le));
  }
  return check_launch(who);
}
