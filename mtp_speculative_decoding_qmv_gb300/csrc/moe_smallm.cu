// moe_smallm.cu -- a mixture-of-experts layer for few rows (1..128): router, the
// chosen experts' 4-bit products, their weighted sum, sm_103a.
//
//   z_e = x . r_e;  the top_k largest z (ties: the lower expert) with weights
//   w = softmax over them (or over all experts);
//   y = sum_j w_j down_ej(silu(gate_ej x) * up_ej x)
//
// A few rows meet most of their experts once, so the layer streams the chosen
// experts' weights (0.5625 bytes each) and is bound by memory.  Three launches,
// the later two starting as the one before drains:
//  * route: 8 experts a CTA, K over its warps, bf16 MMAs (exact products, fp32
//    sums), and the rows of x in the products' form; the last CTA of 16 rows chooses their experts, the last of all sorts
//    the (row, expert) pairs by expert and cuts each expert's rows into slots of
//    up to 8, the columns of one MMA;
//  * gate and up, then down: the stages of all slots' tiles laid out flat and cut
//    evenly over the resident CTAs, so every SM streams the same number of bytes
//    whichever experts were chosen.  A stage is 128 weight rows x 256 inputs: 64
//    rows of gate and the same 64 of up (their product leaves in one place), or
//    128 of down, with the rows' activations.  Eight warps take 32 rows by half of
//    the inputs each.  A producer warp keeps the ring of stages full across tiles, and a warp of its
//    own takes the sums of a finished tile, so that neither the copies nor the
//    products wait for the fences below.  A tile cut between CTAs leaves partial
//    sums, which whichever CTA comes last adds in CTA order; nobody waits for
//    another CTA, so the launches need not be resident together.
//
// The nibbles are widened to fp16: of a word, the even ones of each half as 1024 + q,
// the odd ones, left where they are, as 1024 + 16 q against activations divided by
// 16: five integer operations a word of eight, where bf16 (128 + q, every nibble
// shifted down) takes seven, and these operations are what the products are bound by.
// The activations become fp16 once, before they are multiplied: per row and group of
// 64 scaled by a power of two that brings the largest to 2^14 .. 2^15, which loses
// nothing of a bf16 value down to 2^-28 of it.  Beside them lie the scale, what the
// 1024s contribute (the sums start from its negative) and the group's sum, for the
// bias.  The activations between the products are two such parts (2^-22).  As
// operands of down the parts of up to four rows share one MMA's eight columns; five
// to eight rows take two MMAs.
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
struct Group {
  float f, start, sum, pad;  // 1 / scale; minus the 1024s' part; the inputs' sum
};
constexpr uint32_t kRecord = kGroupsOf * (128 + (uint32_t)sizeof(Group));  // 576
constexpr uint32_t kSb = 2 * kRows * 128;                // [128 rows][4 scales, 4 biases]
constexpr uint32_t kXOff = kSb + kTileRows * kGroupsOf * 4;
template <bool kDown>
struct Ring {  // down: the two parts of eight rows
  static constexpr int kStages = kDown ? 3 : 4, kRecords = kDown ? 16 : 8;
  static constexpr uint32_t kStage = (kXOff + kRecords * kRecord + 1023) / 1024 * 1024;
  static constexpr uint32_t kRedOff = kStages * kStage;
};
constexpr int kRedPitch = kTileRows + 4;  // floats: conflict-free both ways
constexpr uint32_t kRedPlane = kSlotRows * kRedPitch;      // floats: a half of the inputs
constexpr uint32_t kRedSize = 2 * kRedPlane * 4;           // two of them
constexpr int kMostColumns = 128;  // tiles of y that a CTA may come last at
template <bool kDown>
struct Smem {
  static constexpr uint32_t kColumnsOff = Ring<kDown>::kRedOff + 2 * kRedSize;  // number, then they
  static constexpr uint32_t kBarOff = kColumnsOff + (kMostColumns + 2) * 4;
  static constexpr uint32_t kTotal = kBarOff + (2 * Ring<kDown>::kStages + 5) * 8 + 1024;
};
constexpr int kPartFloats = kTileRows * kSlotRows;

__device__ unsigned int g_moe_device_error;

struct Slot {
  int expert, first, n, pad;
};
// What the caller's workspace holds.  The counters come first: zero before a call
// and left zero by it.
struct Space {
  uint32_t *routed;   // [row tiles] CTAs of the router that are done, then row tiles that are
  uint32_t *tiles;    // [slots][tiles] segments of a split tile
  uint32_t *columns;  // [tiles of down] slots that are done
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
  take(s.routed, kMaxRows / 16 + 1);
  take(s.tiles, slots * std::max(up, down));
  take(s.columns, down);
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
// 5 2 6 3 7 of the widened nibbles.  kParts 2: what the fp16 values leave goes to the
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
    const float sum = warp_sum(fa + 16.f * fb), start = warp_sum(fa + fb);
    if (lane == 0)
      *reinterpret_cast<float4 *>(to + kGroupsOf * 128 + (group & 3) * sizeof(Group)) =
          make_float4(f, -1024.f * start, f * sum, 0.f);
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
// lowest expert.
__device__ void choose(const MoeArgs &a, int t) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kMaxExperts / 32;
  const float *z = a.ws.logits + (size_t)t * a.experts;
  float v[kPer];
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < a.experts ? __ldcg(z + e) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)  // 0: none (a NaN is 1)
    key[i] = lane + 32 * i < a.experts ? order_key(v[i]) + 1u : 0u;
  float mine = 0.f, most = 0.f;  // lane j: the logit of choice j
  int id = 0;
  for (int j = 0; j < a.top; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (key[i] == top) e = lane + 32 * i;
    const int chosen = (int)__reduce_min_sync(0xffffffffu, e);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == chosen) {
        x = v[i];
        key[i] = 0u;
      }
    x = __shfl_sync(0xffffffffu, x, chosen & 31);
    if (j == 0) most = x;
    if (lane == j) {
      mine = x;
      id = chosen;
    }
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
    if (a.ids_out) a.ids_out[p] = id;
    if (a.weights_out) a.weights_out[p] = w;
  }
}

// The pairs by expert (rows ascending), and the slots.  A bit a row and expert
// makes the order the same whoever sets the bits first.
constexpr int kRouteThreads = 512;
__device__ void make_slots(const MoeArgs &a, uint32_t (*bits)[4], int *first, int *scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = a.rows * a.top;
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int t = p / a.top, e = __ldcg(a.ws.ids + p);
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
    const int t = p / a.top, e = __ldcg(a.ws.ids + p);
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
  __shared__ uint32_t s_old;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  const int e0 = blockIdx.x * kRouteExperts, t0 = blockIdx.y * kRouteTile;
  pdl_launch_dependents();
  *reinterpret_cast<uint4 *>(bits[tid]) = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();
  // this CTA's share of the rows' groups
  if (t0 + warp < a.rows) {
    const int t = t0 + warp, records = (a.hidden + kStageK - 1) / kStageK;
    for (int g = blockIdx.x; g < a.hidden / 64; g += gridDim.x) {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(a.x + (size_t)t * a.hidden + 64 * g) + lane);
      put_group<1>(a.ws.x + ((size_t)t * records + g / kGroupsOf) * kRecord, 0, g,
                   make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)));
    }
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
  if (!last(a.ws.routed + blockIdx.y, gridDim.x)) return;
  static_assert(kRouteWarps == kRouteTile, "a row a warp");
  if (t0 + warp < a.rows) choose(a, t0 + warp);
  __threadfence();
  if (gridDim.y == 1)
    __syncthreads();
  else if (!last(a.ws.routed + kMaxRows / 16, gridDim.y))
    return;
  make_slots(a, bits, first, scan);
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
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// A group's products of 16 weight rows (w: ldmatrix of words t and 4 + t of rows g8 and
// g8 + 8) with the rows of x in fragments x[2], added to d; kParts 2: with low as well.
template <int kParts>
__device__ __forceinline__ void group_f16(float (&d)[4], const uint32_t (&w)[4], const uint4 (&x)[2],
                                          const uint4 (&low)[2]) {
  constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u, k1024 = 0x64006400u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = w[2 * i], b = w[2 * i + 1], a8 = a >> 8, b8 = b >> 8;
    const uint32_t a0 = and_or(a, kEven, k1024), a1 = and_or(b, kEven, k1024),
                   a2 = and_or(a, kOdd, k1024), a3 = and_or(b, kOdd, k1024);
    mma_f16(d, a0, a1, a2, a3, x[i].x, x[i].y);
    if constexpr (kParts == 2) mma_f16(d, a0, a1, a2, a3, low[i].x, low[i].y);
    const uint32_t c0 = and_or(a8, kEven, k1024), c1 = and_or(b8, kEven, k1024),
                   c2 = and_or(a8, kOdd, k1024), c3 = and_or(b8, kOdd, k1024);
    mma_f16(d, c0, c1, c2, c3, x[i].z, x[i].w);
    if constexpr (kParts == 2) mma_f16(d, c0, c1, c2, c3, low[i].z, low[i].w);
  }
}

// kDown false: h = silu(gate x) * (up x) of every slot; true: d = weight * (down h),
// and y once a tile's slots are all there.
template <bool kDown>
__global__ void __launch_bounds__(kMoeThreads, 2)
    moe_experts_kernel(const __grid_constant__ CUtensorMap map0,
                       const __grid_constant__ CUtensorMap map1, const MoeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  using R = Ring<kDown>;
  using S = Smem<kDown>;
  constexpr int kStages = R::kStages;
  const uint32_t full0 = base + S::kBarOff, empty0 = full0 + 8 * kStages;
  const uint32_t red_full0 = empty0 + 8 * kStages, red_empty0 = red_full0 + 16;
  const uint32_t done = red_empty0 + 16;
  volatile int *columns = reinterpret_cast<volatile int *>(smem + S::kColumnsOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init_u32(full0 + 8u * i, 1 + 32);
      mbar_init_u32(empty0 + 8u * i, kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_u32(red_full0 + 8u * i, kWarps);
      mbar_init_u32(red_empty0 + 8u * i, 1);
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
  const int ctas = (int)min((long long)gridDim.x, W);
  if ((int)blockIdx.x >= ctas) return;
  const long long u_begin = W * blockIdx.x / ctas, u_end = W * (blockIdx.x + 1) / ctas;

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

  if (warp == kWarps) {
    // ---- producer: weights by tensor copies, records by bulk copies, scales and
    // biases, a row's few bytes at a time, by small ones ------------------------------
    const bool wide = groups % 4 == 0;
    int st = 0, ph = 0, issued = 0;
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
    for (long long u = u_begin; ok && u < u_end;) {
      const Segment g = segment(u);
      u += g.s1 - g.s0;
      const long long row0 = (long long)__ldcg(&a.ws.slots[g.slot].expert) * N + g.n0;
      // lane r brings record r: of row r, or of down's two parts r < n and the rest,
      // from place 4 on (up to four rows) or 8
      const int n = __ldcg(&a.ws.slots[g.slot].n), apart = n <= 4 ? 4 : 8;
      const int col = kDown ? lane % apart : lane;
      const bool brings = col < n && lane < (kDown ? 2 * apart : kSlotRows);
      const int pair = brings ? __ldcg(a.ws.order + __ldcg(&a.ws.slots[g.slot].first) + col) : 0;
      const uint8_t *from =
          kDown ? a.ws.h + ((size_t)pair + (lane >= apart ? pairs : 0)) * stages * kRecord
                : a.ws.x + (size_t)(pair / a.top) * stages * kRecord;
      const uint8_t *sp[4], *bp[4];  // of rows lane + 32 i of the stage
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long off = ((row0 + (kDown ? 32 * i : 32 * (i & 1)) + lane) * groups + g.s0 * kGroupsOf) * 2;
        sp[i] = reinterpret_cast<const uint8_t *>(kDown ? a.down_s : i < 2 ? a.gate_s : a.up_s) + off;
        bp[i] = reinterpret_cast<const uint8_t *>(kDown ? a.down_b : i < 2 ? a.gate_b : a.up_b) + off;
      }
      const uint32_t bytes = 2 * kRows * 128 + (kDown ? 2 : 1) * n * kRecord;
      for (int c = g.s0; c < g.s1; ++c) {
        if (!waited && issued == kStages) bring_pending();
        if (issued >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait_u32(empty0 + 8u * st, ph ^ 1));
        if (!ok) break;
        const uint32_t at = base + st * R::kStage, full = full0 + 8u * st;
        if (lane == 0) {
          mbar_arrive_expect_tx_u32(full, bytes);
          const int x = c * (kStageK / 8);
          load_box(at, &map0, x, (int)row0, full);
          load_box(at + kRows * 128, &map1, x, (int)row0 + (kDown ? kRows : 0), full);
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
        const uint32_t sb = at + kSb + lane * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (wide) {
            copy_small<8>(sb + i * 512, sp[i]);
            copy_small<8>(sb + i * 512 + 8, bp[i]);
          } else {  // an even number of groups, the last stage's two
            copy_small<4>(sb + i * 512, sp[i]);
            copy_small<4>(sb + i * 512 + 8, bp[i]);
            if (c * kGroupsOf + 2 < groups) {
              copy_small<4>(sb + i * 512 + 4, sp[i] + 4);
              copy_small<4>(sb + i * 512 + 12, bp[i] + 4);
            }
          }
          sp[i] += 8;
          bp[i] += 8;
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(full) : "memory");
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
    // ---- finisher: rows 2 lane and 2 lane + 1 of both blocks of a tile -------------
    if (kDown) pdl_wait();  // the tiles' counters and partials are the launch before's
    int at_end = 0, k = 0;
    bool ok = true;
    for (long long u = u_begin; ok && u < u_end; ++k) {
      const Segment g = segment(u);
      u += g.s1 - g.s0;
      const int first = __ldcg(&a.ws.slots[g.slot].first), n = __ldcg(&a.ws.slots[g.slot].n);
      const bool whole = g.s0 == 0 && g.s1 == stages;
      // down's slots of up to four rows have the second parts' sums in columns 4..7
      const bool doubled = kDown && n <= 4;
      float *part = a.ws.parts + (size_t)(2 * blockIdx.x + (g.s0 == 0 ? 1 : 0)) * kPartFloats + 2 * lane;
      auto emit = [&](int col, float2 v0, float2 v1) {
        const int p = __ldcg(a.ws.order + first + col);
        if constexpr (!kDown) {
          // a tile's 64 rows are one of down's groups
          const float2 h = make_float2(v0.x / (1.f + expf(-v0.x)) * v1.x, v0.y / (1.f + expf(-v0.y)) * v1.y);
          const int group = g.n0 / 64, records = (N + kStageK - 1) / kStageK;
          put_group<2>(a.ws.h + ((size_t)p * records + group / kGroupsOf) * kRecord,
                       (size_t)pairs * records * kRecord, group, h);
        } else {
          const float w = __ldcg(a.ws.weights + p);
          float *d = a.ws.d + (size_t)p * N + g.n0 + 2 * lane;
          __stcg(reinterpret_cast<float2 *>(d), make_float2(w * v0.x, w * v0.y));
          __stcg(reinterpret_cast<float2 *>(d + kRows), make_float2(w * v1.x, w * v1.y));
        }
      };
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
          emit(col, v[0], v[1]);
        } else {
          __stcg(reinterpret_cast<float2 *>(part + col * kTileRows), v[0]);
          __stcg(reinterpret_cast<float2 *>(part + col * kTileRows + kRows), v[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_u32(red_empty0 + 8u * (k & 1));
      // the warp's stores, then one of its lanes counts; the count's last adds up
      auto count = [&](uint32_t *counter, uint32_t of) {
        __threadfence();
        __syncwarp();
        uint32_t old = 0;
        if (lane == 0) {
          old = atomicAdd(counter, 1u);
          if (old == of - 1u) *counter = 0u;
        }
        old = __shfl_sync(0xffffffffu, old, 0);
        __threadfence();
        return old == of - 1u;
      };
      if (!whole) {
        // a part of the tile: whoever comes last adds them all, in CTA order
        const long long t0 = (long long)g.tile * stages;
        const int c0 = (int)(((t0 + 1) * ctas - 1) / W), c1 = (int)(((t0 + stages) * ctas - 1) / W);
        if (!count(a.ws.tiles + g.tile, (uint32_t)(c1 - c0 + 1))) continue;
        for (int col = 0; col < n; ++col) {
          float2 v[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          for (int c = c0; c <= c1; ++c) {
            const float *from = a.ws.parts + (size_t)(2 * c + (c == c0 ? 1 : 0)) * kPartFloats +
                                col * kTileRows + 2 * lane;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 f = __ldcg(reinterpret_cast<const float2 *>(from + x * kRows));
              v[x].x += f.x;
              v[x].y += f.y;
            }
          }
          emit(col, v[0], v[1]);
        }
      }
      if (kDown) {
        const int column = g.n0 / kStep;
        if (count(a.ws.columns + column, (uint32_t)n_slots)) {
          if (lane == 0) columns[1 + at_end] = column;
          ++at_end;
        }
      }
    }
    if (kDown) {
      __syncwarp();
      if (lane == 0) {
        columns[0] = at_end;
        mbar_arrive_u32(done);
      }
    }
    if (!ok && lane == 0) atomicOr(&g_moe_device_error, 4u);
    return;
  }

  // ---- the products ----------------------------------------------------------------
  // Warp w: rows 32 (w % 4) .. of the stage and half w / 4 of its inputs.  Lane (g8, t4):
  // weight rows g8 + 8 i; of the activations column (row) g8; of the sums columns 2 t4
  // and 2 t4 + 1.
  const int g8 = lane >> 2, t4 = lane & 3, rows0 = 32 * (warp & 3), half = warp >> 2;
  const uint32_t w_at = (uint32_t)(rows0 + (lane & 15)) * 128;  // the second box follows the first
  if (kDown) pdl_wait();  // the partials' places are the launch before's
  int st = 0, ph = 0, k = 0;
  bool ok = true;
  for (long long u = u_begin; ok && u < u_end; ++k) {
    const Segment g = segment(u);
    u += g.s1 - g.s0;
    const int n = __ldcg(&a.ws.slots[g.slot].n);
    const bool both = kDown && n > 4;  // a column a row, its two parts one after the other
    const int apart = kDown && !both ? 4 : kSlotRows;
    const bool valid = g8 % apart < n, real[2] = {2 * t4 % apart < n, (2 * t4 + 1) % apart < n};
    float acc[2][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c = g.s0; c < g.s1; ++c) {
      ok = warp_wait_stage(full0 + 8u * st, ph);
      if (!ok) break;
      const uint32_t at = base + st * R::kStage;
      const uint32_t sb_at = at + kSb + (uint32_t)(rows0 + g8) * 16 + half * 4;
      const uint32_t x_at = at + kXOff + g8 * kRecord + half * 256 + t4 * 16;
      const uint32_t group_at =
          at + kXOff + 2 * t4 * kRecord + kGroupsOf * 128 + half * 2 * (uint32_t)sizeof(Group);
      if (c * kGroupsOf + 2 * half < groups) {
        uint32_t sw[4], bw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sw[i] = lds32(sb_at + i * 8 * 16);
          bw[i] = lds32(sb_at + i * 8 * 16 + 8);
        }
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
          uint32_t w[2][4];
#pragma unroll
          for (int tile = 0; tile < 2; ++tile)
            ldmatrix_x4(w[tile], at + w_at + tile * 16 * 128 +
                                     (((4 * half + 2 * gi + (lane >> 4)) ^ (lane & 7)) << 4));
          uint4 x[2], low[2];
          x[0] = valid ? lds128(x_at + gi * 128) : zero;
          x[1] = valid ? lds128(x_at + gi * 128 + 64) : zero;
          const uint4 r0 = real[0] ? lds128(group_at + gi * 16) : zero;
          const uint4 r1 = real[1] ? lds128(group_at + kRecord + gi * 16) : zero;
          float start0 = __uint_as_float(r0.y), start1 = __uint_as_float(r1.y);
          float sum0 = __uint_as_float(r0.z), sum1 = __uint_as_float(r1.z);
          if (both) {
            low[0] = valid ? lds128(x_at + kSlotRows * kRecord + gi * 128) : zero;
            low[1] = valid ? lds128(x_at + kSlotRows * kRecord + gi * 128 + 64) : zero;
            const uint4 q0 = real[0] ? lds128(group_at + kSlotRows * kRecord + gi * 16) : zero;
            const uint4 q1 = real[1] ? lds128(group_at + (kSlotRows + 1) * kRecord + gi * 16) : zero;
            start0 += __uint_as_float(q0.y);
            start1 += __uint_as_float(q1.y);
            sum0 += __uint_as_float(q0.z);
            sum1 += __uint_as_float(q1.z);
          }
          const float f0 = __uint_as_float(r0.x), f1 = __uint_as_float(r1.x);
          auto of = [&](uint32_t word) {
            return __uint_as_float(gi ? word & 0xFFFF0000u : word << 16);
          };
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
            float d[4] = {start0, start1, start0, start1};
            if (both)
              group_f16<2>(d, w[tile], x, low);
            else
              group_f16<1>(d, w[tile], x, x);
            const float s0 = of(sw[2 * tile]), s8 = of(sw[2 * tile + 1]);
            const float b0 = of(bw[2 * tile]), b8 = of(bw[2 * tile + 1]);
            acc[tile][0] = fmaf(s0, f0 * d[0], fmaf(b0, sum0, acc[tile][0]));
            acc[tile][1] = fmaf(s0, f1 * d[1], fmaf(b0, sum1, acc[tile][1]));
            acc[tile][2] = fmaf(s8, f0 * d[2], fmaf(b8, sum0, acc[tile][2]));
            acc[tile][3] = fmaf(s8, f1 * d[3], fmaf(b8, sum1, acc[tile][3]));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_u32(empty0 + 8u * st);
      if (++st == kStages) {
        st = 0;
        ph ^= 1;
      }
    }
    // the sums to the finisher, red[half][column][row]
    if (ok && k >= 2)
      ok = __all_sync(0xffffffffu, mbar_wait_u32(red_empty0 + 8u * (k & 1), ((k >> 1) & 1) ^ 1));
    if (!ok) break;
    float *red = reinterpret_cast<float *>(smem + R::kRedOff + (k & 1) * kRedSize) + half * kRedPlane +
                 2 * t4 * kRedPitch + rows0 + g8;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      red[16 * tile] = acc[tile][0];
      red[16 * tile + kRedPitch] = acc[tile][1];
      red[16 * tile + 8] = acc[tile][2];
      red[16 * tile + 8 + kRedPitch] = acc[tile][3];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(red_full0 + 8u * (k & 1));
  }
  if constexpr (kDown) {
    // the tiles of y at which this CTA came last: the rows' sums over their experts, in
    // the order of choice, four columns a lane
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_u32(done, 0));
    const int count = ok ? columns[0] : 0;
    for (int i = 0; i < count; ++i) {
      const int n = columns[1 + i] * kTileRows + 4 * lane;
      for (int t = warp; t < a.rows; t += 2 * kWarps) {
        float4 sum[2] = {};
        for (int j0 = 0; j0 < a.top; j0 += 4) {
          float4 x[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[y][j] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (j0 + j < a.top && t + y * kWarps < a.rows)
                x[y][j] = __ldcg(reinterpret_cast<const float4 *>(
                    a.ws.d + (size_t)((t + y * kWarps) * a.top + j0 + j) * N + n));
            }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              sum[y].x += x[y][j].x;
              sum[y].y += x[y][j].y;
              sum[y].z += x[y][j].z;
              sum[y].w += x[y][j].w;
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (t + y * kWarps < a.rows) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(sum[y].x, sum[y].y);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(sum[y].z, sum[y].w);
            *reinterpret_cast<uint2 *>(a.y + (size_t)(t + y * kWarps) * N + n) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                           *reinterpret_cast<const uint32_t *>(&hi));
          }
      }
    }
  }
  if (!ok && lane == 0) atomicOr(&g_moe_device_error, 2u);
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
  if (hidden > kMostColumns * kTileRows || inter > 65536 || (long long)experts * std::max(hidden, inter) > (1ll << 30))
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
                    {gate_s, gate_n / 32, 8},
                    {gate_b, gate_n / 32, 8},
                    {up_w, gate_n / 2, 16},
                    {up_s, gate_n / 32, 8},
                    {up_b, gate_n / 32, 8},
                    {down_w, gate_n / 2, 16},
                    {down_s, gate_n / 32, 8},
                    {down_b, gate_n / 32, 8}};
  for (const Buf &b : in)
    if (!b.p) return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!y || !workspace) return fail(SV_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const Buf &b : in)
    if (!aligned(b.p, b.align))
      return fail(SV_ERR_INVALID_ARG,
                  "%s: x, router and w_packed must be 16-byte, scales and biases 8-byte aligned", who);
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
  CUtensorMap gate_map, up_map, down_map;
  auto encode = [&](CUtensorMap *map, const uint32_t *w, int n, int k) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, w, (uint64_t)k / 8, (uint64_t)experts * n,
                     (uint64_t)k / 2, kBoxWords, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  st = encode(&gate_map, gate_w, inter, hidden);
  if (st == SV_OK) st = encode(&up_map, up_w, inter, hidden);
  if (st == SV_OK) st = encode(&down_map, down_w, hidden, inter);
  if (st != SV_OK) return st;
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
  cfg.gridDim = dim3((experts + kRouteExperts - 1) / kRouteExperts, (rows + kRouteTile - 1) / kRouteTile);
  cfg.blockDim = dim3(kRouteThreads);
  cudaError_t le = cudaLaunchKernelEx(&cfg, moe_route_kernel, a);
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = Smem<false>::kTotal;
  if (le == cudaSuccess) le = cudaLaunchKernelEx(&cfg, moe_experts_kernel<false>, gate_map, up_map, a);
  cfg.dynamicSmemBytes = Smem<true>::kTotal;
  if (le == cudaSuccess) le = cudaLaunchKernelEx(&cfg, moe_experts_kernel<true>, down_map, down_map, a);
  if (le != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(SV_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(le));
  }
  return check_launch(who);
}
