// gdn_chunk.cu -- the gated delta rule over packed bf16 rows in chunks of 64, on
// the tcgen05 tensor cores, sm_103a.
//
// Within a chunk, with S0 the state before it, G[i] the product of the gates from
// the chunk's first row to i, D[i][j] that from j + 1 to i (D[i][i] = 1):
//   e_i  = beta_i (v_i - G[i] S0 k_i - sum_{j<i} D[i][j] (k_i . k_j) e_j)
//   o_i  = G[i] S0 q_i + sum_{j<=i} D[i][j] (q_i . k_j) e_j
//   S    = G[63] S0 + sum_j D[63][j] e_j k_j^T
// With L = tril(beta D K K^T, -1), T = (1 + L)^-1 beta and P = tril(D Q K^T), as
// columns over the chunk's rows:
//   E = V T^T + R T^T, R = -G S0 K^T;  O = G S0 Q^T + E P^T;  S = G[63] S0 + E' K
// Two launches.  The first makes T and P of every chunk of every head, all chunks
// side by side (mma.sync for K K^T and Q K^T, whose results are wanted in
// registers; T by substitution).  The second follows the state from chunk
// to chunk, a CTA a (sequence, head): six products a chunk, each with 128 rows
// (dv) in tensor memory's lanes; S0, R and E are A operands in tensor memory, V in
// shared memory, K, Q, T and P (bf16, shared memory) are B.  K serves both as rows of
// dk (S0 K^T) and with dk contiguous (E' K), from one copy.
//
// Precision: the state stays in fp32 registers, and outputs are sums to fp32 rounded
// once.  An fp32 operand is cut into three bf16 parts that add up to it exactly (8 bits
// of it each): S0 K^T, S0 Q^T, E' K and V T^T take all three (K, Q and V are bf16 as
// given), R T^T and E P^T the six products of parts above 2^-24.  T's diagonal blocks
// of 16 are made in fp32, those below by products of two tf32 parts (2^-21 of the
// terms).  Sums in tensor memory are cut off at each step, which leaves a prompt's
// states off by 7e-7.  (S0, P and E in two parts for the outputs: 317 us where three
// take 328, but 1 % of the outputs of a chunk were not the bf16 nearest to the exact
// value, as against 0.03 %.)
//
// What bounds the second is the chain from chunk to chunk: tensor-core time of S0
// K^T, R T^T and E' K (about 2000 cycles a chunk), and between them the warps that
// read a product, cut it and write the next operand.  The chunk's rows, and the
// state's columns, go through in two halves, so that one half's products run while
// the other half is cut.  S0 Q^T, V T^T and E P^T run in the gaps, and the outputs
// leave by four warps of their own.
//
// Measured, 48 heads of 128 x 128: a prompt of 5000 rows 328 us (matrices
// 60, states 268: 3.4 us a chunk; 72 TFLOP/s of the recurrence's own operations), five
// prompts of 77 to 2000 rows 198 us, 64 rows 15 us.  The second launch begins as the
// first drains (4 to 5 us less).  Both in one launch, chains waiting for each chunk's
// matrices: 338 us, as the matrices' code costs the chains registers.
#include <cuda.h>
#include <cuda_runtime.h>

#include "gdn_rows.cuh"
#include "qmv_common.cuh"
#include "tc05.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int kC = 64;    // rows a chunk (1 << 6)
constexpr int kD = 128;   // dk and dv, narrower ones padded with zeros

// What the first launch leaves of a chunk of a head, as the second wants it in
// shared memory: T and P in three parts ([64 rows][64 columns] bf16 each, in the
// 128-byte swizzle; P's third where its first two are not read), G and D[63].
constexpr uint32_t kTile = kC * kD * 2;             // K, Q or V of a chunk
constexpr uint32_t kPanel = kC * 128;               // 64 columns of it, 128-byte swizzle
constexpr uint32_t kPart = kC * kC * 2;
constexpr int kTParts = 3, kPTiles = 2;
constexpr uint32_t kOffP = kTParts * kPart, kOffG = kOffP + kPTiles * kPart;  // G, D[63], -G
constexpr uint32_t kBlob = kOffG + 1024;

__device__ unsigned int g_give_up;

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Cuts 2 kN values into kParts bf16 parts, packed in pairs: each part is the upper
// half of what the parts before it leave, an exact difference.
template <int kN, int kParts>
__device__ __forceinline__ void cut(const float *x, uint32_t (&part)[kParts][kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      part[p][i] = prmt(ua, ub, 0x7632);
      if (p + 1 < kParts) {
        a -= __uint_as_float(ua & 0xFFFF0000u);
        b -= __uint_as_float(ub & 0xFFFF0000u);
      }
    }
  }
}
// Address of the 16-byte piece `piece` (of 8) of a row of a 128-byte swizzled panel.
__device__ __forceinline__ uint32_t swizzled(int row, int piece) {
  return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

// P's third part.  P is lower triangular: of the 16 columns of step j the rows from 16 j
// on are read, so the rows above are free in the tiles of the first two parts.  Rows
// [16 j, 64) of step j lie there as rows [0, 64 - 16 j) of another step (step 0's last 16
// rows apart, as no step has 64 rows free).  The moves are by 16 rows, so the swizzle's
// order within eight rows is kept.
struct Place {
  int tile, step;
};
__host__ __device__ constexpr Place third_of_p(int j, bool last_rows) {
  return j == 0 ? Place{0, last_rows ? 1 : 3}
                : j == 1 ? Place{1, 3} : j == 2 ? Place{0, 2} : Place{1, 1};
}

// ---- T and P of a chunk: four warps ----------------------------------------------
// Bound by latency (a chain of small steps; issue 47 %, DRAM 43 %), so as many chunks
// as fit share an SM: the scratch matrix lies where K was, P where Q was.
constexpr int kPrepThreads = 128;
constexpr int kPitch = kC + 4;  // floats a row of the scratch matrix
constexpr uint32_t kPrepQ = (kC * kPitch * 4 + 1023) / 1024 * 1024;
constexpr uint32_t kPrepAlpha = kPrepQ + kTile, kPrepBeta = kPrepAlpha + kC * 4;
constexpr uint32_t kPrepSmem = kPrepBeta + kC * 4 + 1024;
static_assert(kTile <= kPrepQ && kPTiles * kPart == kTile, "K under the scratch, Q under P");

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
  // 16 bytes to shared memory, zeros where there is no source
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// d (+)= 16 x kK floats at `left` times kK x 8 at `right`, both of the scratch matrix, by
// a warp.  Each factor is cut into two tf32 parts (rounded to 11 bits, and 11 of what
// that leaves), three products of them: below 2^-21 of the terms.  Sums of fp32 products
// took 70 us for the 3792 chunk heads of a 5000-token prompt (bound by their loads from
// shared memory), these 59.
template <int kK>
__device__ __forceinline__ void times(float (&d)[4], const float *left, const float *right) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int k = 0; k < kK; k += 8) {
    uint32_t a[2][4], b[2][2];
    auto cut_tf32 = [](float x, uint32_t &high, uint32_t &low) {
      high = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
      low = __float_as_uint(x - __uint_as_float(high)) & 0xFFFFE000u;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cut_tf32(left[(g8 + 8 * (i & 1)) * kPitch + k + t4 + 4 * (i >> 1)], a[0][i], a[1][i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) cut_tf32(right[(k + t4 + 4 * i) * kPitch + g8], b[0][i], b[1][i]);
    mma_tf32(d, a[0], b[1]);
    mma_tf32(d, a[1], b[0]);
    mma_tf32(d, a[0], b[0]);
  }
}
// A product's 16 x 8 values to the scratch matrix, times `sign`.
__device__ __forceinline__ void put_product(float *to, const float (&d)[4], float sign) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  *reinterpret_cast<float2 *>(to + g8 * kPitch + 2 * t4) = make_float2(sign * d[0], sign * d[1]);
  *reinterpret_cast<float2 *>(to + (g8 + 8) * kPitch + 2 * t4) = make_float2(sign * d[2], sign * d[3]);
}

__global__ void __launch_bounds__(kPrepThreads, 5) gdn_chunk_matrices(const AdvanceArgs a,
                                                                      uint8_t *blobs) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % a.H, place = blockIdx.x / a.H, hk = h / (a.H / a.Hk);
  int c;
  const int b = tile_owner(a.q_start, a.B, a.rows, 6, place, c);
  if (b >= a.B) return;
  const Rows s = rows_of(a.q_start, b, a.rows);
  if (c < 0 || c * kC >= s.n || slot_of(a.state_index, b, a.slots) < 0) return;
  const int left = min(kC, s.n - c * kC);
  const long long row0 = s.start + c * kC;
  float *scratch = reinterpret_cast<float *>(smem);
  float *alpha = reinterpret_cast<float *>(smem + kPrepAlpha);
  float *beta = reinterpret_cast<float *>(smem + kPrepBeta);
  uint8_t *blob = blobs + (long long)blockIdx.x * kBlob;
  float *G = reinterpret_cast<float *>(blob + kOffG), *last = G + kC;
  {
    using B16 = __nv_bfloat16;
    const B16 *k = static_cast<const B16 *>(a.k) + row0 * a.k_stride + (long long)hk * a.dk;
    const B16 *q = static_cast<const B16 *>(a.q) + row0 * a.q_stride + (long long)hk * a.dk;
    const int piece = tid & 15;
    const uint32_t to = (piece >> 3) * kPanel;
#pragma unroll
    for (int row = tid >> 4; row < kC; row += kPrepThreads / 16) {
      const bool in = row < left && 8 * piece < a.dk;
      const uint32_t at = base + to + swizzled(row, piece & 7);
      copy16(at, in ? k + row * a.k_stride + 8 * piece : k, in);
      copy16(at + kPrepQ, in ? q + row * a.q_stride + 8 * piece : q, in);
    }
    if (tid < kC) {
      const long long g = (row0 + tid) * a.H + h;
      alpha[tid] = tid < left ? __ldg(a.alpha + g) : 1.f;
      beta[tid] = tid < left ? __ldg(a.beta + g) : 0.f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncthreads();
  // K K^T and Q K^T of the warp's 16 rows and the columns up to them
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) kk[i][m] = qk[i][m] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < kD / 16; ++ks) {
    const uint32_t panel = base + (ks >> 2) * kPanel;
    const int piece = (ks & 3) * 2;
    uint32_t ak[4], aq[4];
    const uint32_t a_at = panel + swizzled(16 * warp + (lane & 15), piece + (lane >> 4));
    qmv::ldmatrix_x4(ak, a_at);
    qmv::ldmatrix_x4(aq, a_at + kPrepQ);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np <= warp) {
        uint32_t x[4];
        const int row = 16 * np + ((lane >> 4) << 3) + (lane & 7);
        qmv::ldmatrix_x4(x, panel + swizzled(row, piece + ((lane >> 3) & 1)));
        mma_bf16_m16n8k16(kk[2 * np], ak[0], ak[1], ak[2], ak[3], x[0], x[1]);
        mma_bf16_m16n8k16(kk[2 * np + 1], ak[0], ak[1], ak[2], ak[3], x[2], x[3]);
        mma_bf16_m16n8k16(qk[2 * np], aq[0], aq[1], aq[2], aq[3], x[0], x[1]);
        mma_bf16_m16n8k16(qk[2 * np + 1], aq[0], aq[1], aq[2], aq[3], x[2], x[3]);
      }
    }
  }
  __syncthreads();  // K and Q have been read
  // D from the diagonal down, by products (a gate of 0 or gates whose product
  // underflows need no care): warp 0 rows 0..31 of columns 0..31, warps 2 and 3
  // rows 32..63, a column a thread; warp 1 G, by a scan
  if (warp == 1) {
    const float2 x = *reinterpret_cast<const float2 *>(alpha + 2 * lane);
    float upto = x.x * x.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto *= y;
    }
    float before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) before = 1.f;
    const float2 g = make_float2(before * x.x, before * x.x * x.y);
    *reinterpret_cast<float2 *>(G + 2 * lane) = g;
    *reinterpret_cast<float2 *>(G + 2 * kC + 2 * lane) = make_float2(-g.x, -g.y);
  } else {
    const int j = warp == 3 ? 32 + lane : lane, low = warp ? 32 : 0;
    float d = 1.f;
    if (warp == 2) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(alpha + i);
        if (i > j) d *= x.x;
        if (i + 1 > j) d *= x.y;
        if (i + 2 > j) d *= x.z;
        if (i + 3 > j) d *= x.w;
      }
    }
    float *to = scratch + low * kPitch + j;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {  // 1 above the diagonal, where it is not used
      const float4 x = *reinterpret_cast<const float4 *>(alpha + low + i);
      if (low + i > j) d *= x.x;
      to[i * kPitch] = d;
      if (low + i + 1 > j) d *= x.y;
      to[(i + 1) * kPitch] = d;
      if (low + i + 2 > j) d *= x.z;
      to[(i + 2) * kPitch] = d;
      if (low + i + 3 > j) d *= x.w;
      to[(i + 3) * kPitch] = d;
    }
    if (warp) last[j] = d;
  }
  __syncthreads();  // D is there
  const int g8 = lane >> 2, t4 = lane & 3;
  const float be2[2] = {beta[16 * warp + g8], beta[16 * warp + g8 + 8]};
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    if (nt >= 2 * (warp + 1)) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 16 * warp + g8 + 8 * half, j = 8 * nt + 2 * t4;
      float2 *d = reinterpret_cast<float2 *>(scratch + i * kPitch + j);
      const float2 w = *d;
      // the diagonal is P's alone
      const float p[2] = {j <= i ? qk[nt][2 * half] * w.x : 0.f,
                          j < i ? qk[nt][2 * half + 1] * w.y : 0.f};
      *d = make_float2(j < i ? be2[half] * (kk[nt][2 * half] * w.x) : 0.f,
                       j + 1 < i ? be2[half] * (kk[nt][2 * half + 1] * w.y) : 0.f);
      uint32_t part[3][1];
      cut<1, 3>(p, part);
#pragma unroll
      for (int x = 0; x < kPTiles; ++x)
        *reinterpret_cast<uint32_t *>(smem + kPrepQ + x * kPart + swizzled(i, nt) + t4 * 4) =
            part[x][0];
      const int step = nt >> 1;
      const bool last_rows = step == 0 && warp == 3;
      const Place to = third_of_p(step, last_rows);
      *reinterpret_cast<uint32_t *>(smem + kPrepQ + to.tile * kPart + t4 * 4 +
                                    swizzled(i - (last_rows ? 48 : 16 * step), 2 * to.step + (nt & 1))) =
          part[2][0];
    }
  }
  fence_async();
  __syncthreads();  // L and P are there
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(blob + kOffP),
                 "r"(base + kPrepQ), "r"(kPTiles * kPart)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  // (1 + L)^-1: the four diagonal blocks of 16, one a warp, a column a lane, by
  // substitution
  {
    const int col = lane & 15;
    float *block = scratch + 16 * warp * (kPitch + 1);
    float t[16];
    t[0] = col == 0 ? 1.f : 0.f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(block + i * kPitch + m);
        const float lm[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (m + x < i) sum[x & 1] = fmaf(lm[x], t[m + x], sum[x & 1]);
      }
      t[i] = (col == i ? 1.f : 0.f) - (sum[0] + sum[1]);
    }
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) block[i * kPitch + col] = t[i];
    } else if (!(warp & 1)) {  // zeros beside the upper block of a pair
#pragma unroll
      for (int i = 0; i < 16; ++i) block[i * kPitch + lane] = 0.f;
    }
  }
  __syncthreads();
  // the 16 x 16 blocks below them, -T11 (L10 T00) of each pair, eight columns a warp
  {
    float *pair = scratch + 32 * (warp >> 1) * (kPitch + 1), *below = pair + 16 * kPitch;
    const int col = 8 * (warp & 1);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    times<16>(d, below, pair + col);
    __syncthreads();  // L10 has been read
    put_product(below + col, d, 1.f);
    __syncthreads();
    float e[4] = {0.f, 0.f, 0.f, 0.f};
    times<16>(e, below + 16, below + col);
    __syncthreads();
    put_product(below + col, e, -1.f);
  }
  __syncthreads();
  // the 32 x 32 block below, the same way: 16 rows by 16 columns a warp
  {
    float *rows = scratch + (32 + 16 * (warp >> 1)) * kPitch;
    const int col = 16 * (warp & 1);
    float d[2][4] = {};
    times<32>(d[0], rows, scratch + col);
    times<32>(d[1], rows, scratch + col + 8);
    __syncthreads();
    put_product(rows + col, d[0], 1.f);
    put_product(rows + col + 8, d[1], 1.f);
    __syncthreads();
    float e[2][4] = {};
    times<32>(e[0], rows + 32, scratch + 32 * kPitch + col);
    times<32>(e[1], rows + 32, scratch + 32 * kPitch + col + 8);
    __syncthreads();
    put_product(rows + col, e[0], -1.f);
    put_product(rows + col + 8, e[1], -1.f);
  }
  __syncthreads();
  // T, its columns times their beta, in parts: eight columns of three rows a thread
#pragma unroll
  for (int y = 0; y < 3; ++y) {
    const int i = tid + y * kPrepThreads;  // rows 0..31: four pieces, 32..63: eight
    const int row = i < 128 ? i >> 2 : 32 + ((i - 128) >> 3), piece = i < 128 ? i & 3 : i & 7;
    float v[8];
#pragma unroll
    for (int x = 0; x < 8; x += 4) {
      const float4 t = *reinterpret_cast<const float4 *>(scratch + row * kPitch + 8 * piece + x);
      const float4 be = *reinterpret_cast<const float4 *>(beta + 8 * piece + x);
      v[x] = t.x * be.x;
      v[x + 1] = t.y * be.y;
      v[x + 2] = t.z * be.z;
      v[x + 3] = t.w * be.w;
    }
    uint32_t part[kTParts][4];
    cut<4, kTParts>(v, part);
#pragma unroll
    for (int p = 0; p < kTParts; ++p)
      *reinterpret_cast<uint4 *>(blob + p * kPart + swizzled(row, piece)) =
          make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- the state from chunk to chunk ---------------------------------------------------
constexpr int kChainWarps = 16, kOutWarps = 4, kMmaWarp = 20, kLoadWarp = 21;
constexpr int kThreads = 768;
// 512 x 96 + 128 x 64 + 128 x 32 = 768 x 80 registers
constexpr int kChainRegs = 96, kOutRegs = 64, kOtherRegs = 32;
constexpr uint32_t kStage = 3 * kTile + kBlob;  // K, Q, V, blob
constexpr uint32_t kOffOut = 2 * kStage;  // a chunk's outputs, [64 rows][128] bf16
constexpr uint32_t kOffBars = kOffOut + kTile;
enum Bar {
  kFull = 0,     // [2 stages] loaded
  kEmpty = 2,    // [2] read
  kTail = 4,     // the last chunk's loads, whose rows past the end are then zeroed
  kState = 5,    // [2 halves of dk] the state's parts are written
  kR = 7,        // [2 halves of the rows] R's are
  kE = 9,        // [2] E's are
  kOutRead = 11, // S0 Q^T and E P^T have been read
  kKs = 12,      // [2 halves of the rows] S0 K^T is there
  kTr = 14,      // [2] R T^T is
  kQs = 16,      // S0 Q^T is
  kSu = 17,      // [2 halves of dk] E' K is
  kOut = 19,     // E P^T is
  kBars = 20
};
constexpr uint32_t kOffTmem = kOffBars + 8 * kBars;
constexpr uint32_t kSmem = kOffTmem + 16 + 1024;

// Tensor memory (columns).  The state's parts: of each half of dk 12 pieces of 8
// columns (16 of dk, one part); E' K of that half first lands in the first 64 of these
// 96 columns, and the warp that reads 32 of them writes its own pieces over them.
constexpr uint32_t kColState = 0, kColHalf = 96;
constexpr uint32_t kColK = 192;   // S0 K^T, then E
constexpr uint32_t kColQ = 256;   // S0 Q^T
constexpr uint32_t kColE = 320;   // R T^T, then E P^T
constexpr uint32_t kColR = 384;   // R's parts, then those of E'
constexpr uint32_t kColLow = 480; // E's third part
constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t state_col(int half, int part, int step) {
  return kColState + kColHalf * half +
         (part < 2 ? 32 * (step >> 1) + 16 * part : 64 + 16 * (step >> 1)) + 8 * (step & 1);
}

// E's first two parts lie over S0 K^T, each half's over the columns that the warps of that
// half have read; the third behind all else.
__host__ __device__ constexpr uint32_t e_col(int part, int step) {
  return part < 2 ? kColK + 32 * (step >> 1) + 16 * part + 8 * (step & 1) : kColLow + 8 * step;
}

constexpr uint32_t idesc(int n, bool mn_major, bool a_mn_major = false) {
  return (1u << 4) | (1u << 7) | (1u << 10)  // D fp32; A, B bf16
         | (a_mn_major ? 1u << 15 : 0u) | (mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kD >> 4) << 24);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
        "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
// Uses of registers that a tcgen05.ld fills stay behind its wait.
template <int kN>
__device__ __forceinline__ void pin(uint32_t (&v)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]),
                      "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7]));
}

// A warp's wait for a phase.  It begins with a non-blocking test: the blocking one
// takes longer even when the phase is complete.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok != 0)) return true;
  return __all_sync(0xffffffffu, mbar_wait_u32(bar, parity));
}

struct Item {
  int start, n, slot, h, hk, chunks;
  long long blob;  // of its first chunk; the next H further
};

// R T^T, D[dv][64 rows] += A parts x B parts, both lower triangular: the 16 columns of
// step j reach the rows from 16 j on.  Steps [kJ0, kJ1).  Parts whose weights add up past
// 2 are left out.  Here and below the least parts come first: a sum in tensor memory is
// cut off, not rounded, at each step, and a small sum loses less by it (the states of a
// prompt: 7e-7, as against 11e-7, relative to their norm).
template <int kJ0, int kJ1>
__device__ __forceinline__ void mma_lower(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int weight = 2; weight >= 0; --weight)
#pragma unroll
    for (int pa = 0; pa <= weight; ++pa)
#pragma unroll
      for (int j = kJ0; j < kJ1; ++j)
        tc_mma_ts(d + 16 * j, a + 32 * pa + 8 * j,
                  smem_desc_sw128(b + (weight - pa) * kPart + j * 2048 + j * 32),
                  idesc(kC - 16 * j, false), true);
}
// E P^T, the same: E's third part first, whose product sets the sum.
__device__ __forceinline__ void mma_out(uint32_t d, uint32_t tmem, uint32_t p) {
#pragma unroll
  for (int weight = 2; weight >= 0; --weight)
#pragma unroll
    for (int pa = weight; pa >= 0; --pa)
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) {
        const uint32_t e = tmem + e_col(pa, j);
        if (weight - pa < kPTiles) {
          tc_mma_ts(d + 16 * j, e, smem_desc_sw128(p + (weight - pa) * kPart + j * 2048 + j * 32),
                    idesc(kC - 16 * j, false), weight < 2 || pa < 2 || j > 0);
        } else {
          const Place at = third_of_p(j, false);
          tc_mma_ts(d + 16 * j, e, smem_desc_sw128(p + at.tile * kPart + at.step * 32),
                    idesc(j == 0 ? 48 : kC - 16 * j, false), true);
          const Place rest = third_of_p(0, true);
          if (j == 0)
            tc_mma_ts(d + 48, e, smem_desc_sw128(p + rest.tile * kPart + rest.step * 32),
                      idesc(16, false), true);
        }
      }
}
// V T^T, the same with V from shared memory, dv contiguous.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t v, uint32_t t) {
#pragma unroll
  for (int p = kTParts - 1; p >= 0; --p)
#pragma unroll
    for (int j = 0; j < kC / 16; ++j)
      tc_mma_ss(d + 16 * j, smem_desc_sw128_mn(v + j * 2048, kPanel),
                smem_desc_sw128(t + p * kPart + j * 2048 + j * 32),
                idesc(kC - 16 * j, false, true), p < kTParts - 1 || j > 0);
}
// S0 times kRows rows of K or Q, from half `half` of dk.
template <int kParts, int kRowsOf>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t tmem, uint32_t b, int half) {
#pragma unroll
  for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc_mma_ts(d, tmem + state_col(half, p, ks),
                smem_desc_sw128(b + half * kPanel + ks * 32), idesc(kRowsOf, false),
                p < kParts - 1 || half + ks > 0);
}
// E' K: steps [j0, j0 + 2) of the chunk's rows, half `half` of dk.
__device__ __forceinline__ void mma_update(uint32_t tmem, uint32_t k_at, int half, int j0) {
#pragma unroll
  for (int p = 2; p >= 0; --p)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      tc_mma_ts(tmem + kColState + half * kColHalf, tmem + kColR + 32 * p + 8 * (j0 + j),
                smem_desc_sw128_mn(k_at + half * kPanel + (j0 + j) * 2048, kPanel), idesc(64, true),
                p < 2 || j0 + j > 0);
}

__device__ void issue_chunks(uint32_t base, uint32_t tmem, const Item &it) {
  auto bar = [&](int i) { return base + kOffBars + 8u * i; };
  const bool one = elect_one();
  tmem = __reduce_max_sync(0xffffffffu, tmem);  // known to be the warp's: no move before every product
  bool ok = true;
  auto wait = [&](int i, uint32_t parity) {
    ok = wait_phase(bar(i), parity);
    tc_fence_after();
    return ok;
  };
  for (int c = 0; c < it.chunks; ++c) {
    const uint32_t s = c & 1, odd = c & 1, pair = (c >> 1) & 1;
    const uint32_t k_at = base + s * kStage, q_at = k_at + kTile, v_at = q_at + kTile;
    const uint32_t t_at = v_at + kTile, p_at = t_at + kOffP;
    if (c > 0 && !wait(kOut, odd ^ 1)) break;  // E P^T has read what S0 K^T overwrites
    if (!wait(kFull + s, pair) || !wait(kState, odd)) break;
    if (one) mma_state<3, 64>(tmem + kColK, tmem, k_at, 0);
    __syncwarp();
    if (!wait(kState + 1, odd)) break;
    if (one) {
      mma_state<3, 32>(tmem + kColK, tmem, k_at, 1);
      tc_commit(bar(kKs));
      mma_state<3, 32>(tmem + kColK + 32, tmem, k_at + 32 * 128, 1);
      tc_commit(bar(kKs + 1));
    }
    if (c > 0 && !wait(kOutRead, odd ^ 1)) break;
    if (one) mma_values(tmem + kColE, v_at, t_at);
    __syncwarp();
    if (!wait(kR, odd)) break;
    if (one) {
      mma_lower<0, 2>(tmem + kColE, tmem + kColR, t_at);
      tc_commit(bar(kTr));
    }
    __syncwarp();
    if (!wait(kR + 1, odd)) break;
    if (one) {
      mma_lower<2, 4>(tmem + kColE, tmem + kColR, t_at);
      tc_commit(bar(kTr + 1));
      mma_state<3, 64>(tmem + kColQ, tmem, q_at, 0);
      mma_state<3, 64>(tmem + kColQ, tmem, q_at, 1);
      tc_commit(bar(kQs));
    }
    __syncwarp();
    if (!wait(kQs, odd) || !wait(kE, odd)) break;  // S0 Q^T has read what E' K overwrites
    if (one) {
      mma_update(tmem, k_at, 0, 0);
      mma_update(tmem, k_at, 1, 0);
    }
    __syncwarp();
    if (!wait(kE + 1, odd)) break;
    if (one) {
      mma_update(tmem, k_at, 0, 2);
      tc_commit(bar(kSu));
      mma_update(tmem, k_at, 1, 2);
      tc_commit(bar(kSu + 1));
      mma_out(tmem + kColE, tmem, p_at);
      tc_commit(bar(kOut));
      tc_commit(bar(kEmpty + s));
    }
    __syncwarp();
  }
  if (!ok && one) atomicOr(&g_give_up, 1u);
}

// The chain's warps: lane = row of the state (dv); warps 4 g .. 4 g + 3 take rows
// 16 g .. of the chunk and columns 32 g .. of the state.
__device__ void run_chain(const AdvanceArgs &a, const Item &it, uint8_t *smem, uint32_t base,
                          uint32_t tmem_base) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = 32 * (warp & 3) + lane, g = warp >> 2, half = g >> 1;
  const uint32_t tmem = tmem_base + ((uint32_t)(warp & 3) << 21);
  auto bar = [&](int b) { return base + kOffBars + 8u * b; };
  auto arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(bar(b));
  };
  bool ok = true;
  auto wait = [&](int b, uint32_t parity) {
    ok = wait_phase(bar(b), parity);
    tc_fence_after();
    return ok;
  };
  float S[32];
  float *state = a.state + (((long long)it.slot * a.H + it.h) * a.dv + (i < a.dv ? i : 0)) * a.dk + 32 * g;
#pragma unroll
  for (int m = 0; m < 32; m += 4) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < a.dv && 32 * g + m < a.dk) x = __ldcg(reinterpret_cast<const float4 *>(state + m));
    S[m] = x.x;
    S[m + 1] = x.y;
    S[m + 2] = x.z;
    S[m + 3] = x.w;
  }
  auto put_state = [&] {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t part[3][8];
      cut<8, 3>(S + 16 * x, part);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        tc_st_x8(tmem + kColHalf * half + (p < 2 ? 32 * (g & 1) + 16 * p : 64 + 16 * (g & 1)) + 8 * x,
                 part[p]);
    }
    tc_wait_st();
    arrive(kState + half);
  };
  put_state();
  for (int c = 0; c < it.chunks; ++c) {
    const uint32_t s = c & 1, odd = c & 1, pair = (c >> 1) & 1;
    const float *G = reinterpret_cast<const float *>(smem + s * kStage + 3 * kTile + kOffG);
    // R = -G S0 k
    if (!wait(kFull + s, pair) || !wait(kKs + half, odd)) break;
    {
      uint32_t x[16];
      tc_ld_x16(tmem + kColK + 16 * g, x);
      float r[16];
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4 *>(r + j) =
            *reinterpret_cast<const float4 *>(G + 2 * kC + 16 * g + j);
      tc_wait_ld();
      pin(x);
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] *= __uint_as_float(x[j]);
      const int left = it.n - c * kC - 16 * g;
      if (left < 16) {  // no row: a state that is not finite must not count
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j >= left) r[j] = 0.f;
      }
      uint32_t part[3][8];
      cut<8, 3>(r, part);
#pragma unroll
      for (int p = 0; p < 3; ++p) tc_st_x8(tmem + kColR + 32 * p + 8 * g, part[p]);
      tc_wait_st();
      arrive(kR + half);
    }
    // E and E' = D[63] E
    if (!wait(kTr + half, odd)) break;
    {
      uint32_t x[16];
      tc_ld_x16(tmem + kColE + 16 * g, x);
      float e[16];
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4 *>(e + j) = *reinterpret_cast<const float4 *>(G + kC + 16 * g + j);
      tc_wait_ld();
      pin(x);
#pragma unroll
      for (int j = 0; j < 16; ++j) e[j] *= __uint_as_float(x[j]);
      uint32_t part[3][8];
      cut<8, 3>(e, part);
#pragma unroll
      for (int p = 0; p < 3; ++p) tc_st_x8(tmem + kColR + 32 * p + 8 * g, part[p]);
      cut<8, 3>(reinterpret_cast<const float *>(x), part);
#pragma unroll
      for (int p = 0; p < 3; ++p) tc_st_x8(tmem + e_col(p, g), part[p]);
      tc_wait_st();
      arrive(kE + half);
    }
    // S = G[63] S0 + E' K
    if (!wait(kSu + half, odd)) break;
    {
      const float2 all = make_float2(G[kC - 1], G[kC - 1]);
      uint32_t x[2][16];
      tc_ld_x16(tmem + kColHalf * half + 32 * (g & 1), x[0]);
      tc_ld_x16(tmem + kColHalf * half + 32 * (g & 1) + 16, x[1]);
      tc_wait_ld();
      pin(x[0]);
      pin(x[1]);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 n = __ffma2_rn(all, make_float2(S[j], S[j + 1]),
                                    make_float2(__uint_as_float(x[j >> 4][j & 15]),
                                                __uint_as_float(x[j >> 4][(j & 15) + 1])));
        S[j] = n.x;
        S[j + 1] = n.y;
      }
      if (lane == 0) mbar_arrive_u32(bar(kEmpty + s));
      if (c + 1 < it.chunks) put_state();
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(&g_give_up, 2u);
    return;
  }
  if (i < a.dv) {
#pragma unroll
    for (int m = 0; m < 32; m += 4)
      if (32 * g + m < a.dk)
        *reinterpret_cast<float4 *>(state + m) = make_float4(S[m], S[m + 1], S[m + 2], S[m + 3]);
  }
}

// The outputs' warps: o = G S0 q + E P, lane = dv.
__device__ void write_out(const AdvanceArgs &a, const CUtensorMap *omap, const Item &it,
                          uint8_t *smem, uint32_t base, uint32_t tmem_base) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = 32 * (warp & 3) + lane;
  const uint32_t tmem = tmem_base + ((uint32_t)(warp & 3) << 21);
  auto bar = [&](int b) { return base + kOffBars + 8u * b; };
  for (int c = 0; c < it.chunks; ++c) {
    const uint32_t s = c & 1, odd = c & 1, pair = (c >> 1) & 1;
    const float *G = reinterpret_cast<const float *>(smem + s * kStage + 3 * kTile + kOffG);
    const bool ok = wait_phase(bar(kFull + s), pair) && wait_phase(bar(kOut), odd);
    tc_fence_after();
    // the copy of the chunk before has left shared memory; all four warps go on or none
    if (threadIdx.x == kChainWarps * 32)
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((int)ok)
        : "memory");
    if (!all) {
      if (lane == 0) atomicOr(&g_give_up, 8u);
      break;
    }
    // all of it is read before any is stored: the next chunk waits for the place
    uint32_t o[kC / 2];
#pragma unroll
    for (int x = 0; x < kC; x += 16) {
      uint32_t q[16], e[16];
      tc_ld_x16(tmem + kColQ + x, q);
      tc_ld_x16(tmem + kColE + x, e);
      tc_wait_ld();
      pin(q);
      pin(e);
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 f = *reinterpret_cast<const float2 *>(G + x + j);
        const __nv_bfloat162 y =
            __floats2bfloat162_rn(fmaf(f.x, __uint_as_float(q[j]), __uint_as_float(e[j])),
                                  fmaf(f.y, __uint_as_float(q[j + 1]), __uint_as_float(e[j + 1])));
        o[(x + j) / 2] = *reinterpret_cast<const uint32_t *>(&y);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive_u32(bar(kOutRead));
      mbar_arrive_u32(bar(kEmpty + s));
    }
    const int left = it.n - c * kC;
    if (left >= kC) {
      uint16_t *to = reinterpret_cast<uint16_t *>(smem + kOffOut) + i;
#pragma unroll
      for (int j = 0; j < kC; ++j) to[j * kD] = (uint16_t)(j & 1 ? o[j / 2] >> 16 : o[j / 2]);
      fence_async();
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
      if (threadIdx.x == kChainWarps * 32) {
        asm volatile(
            "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                omap),
            "r"(0), "r"(it.h), "r"(it.start + c * kC), "r"(base + kOffOut)
            : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else if (i < a.dv) {  // the rows behind the sequence are another's
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) +
                           (long long)(it.start + c * kC) * a.out_stride + (long long)it.h * a.dv + i;
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if (j < left)
          reinterpret_cast<uint16_t *>(out)[j * a.out_stride] =
              (uint16_t)(j & 1 ? o[j / 2] >> 16 : o[j / 2]);
    }
  }
  if (threadIdx.x == kChainWarps * 32)
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ void load_chunks(const CUtensorMap *kmap, const CUtensorMap *qmap, const CUtensorMap *vmap,
                            const uint8_t *blobs, int H, const Item &it, uint8_t *smem, uint32_t base) {
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + kOffBars + 8u * i; };
  bool ok = true;
  int c = 0;
  pdl_wait();  // T and P are the launch before's; what all others read is older
  for (; c < it.chunks; ++c) {
    const uint32_t s = c & 1, at = base + s * kStage;
    if (c >= 2) ok = __all_sync(0xffffffffu, mbar_wait_u32(bar(kEmpty + s), ((c >> 1) & 1) ^ 1));
    if (!ok) break;
    const int left = it.n - c * kC;
    const uint32_t full = bar(left < kC ? (int)kTail : (int)(kFull + s));
    if (lane == 0) {
      const int row = it.start + c * kC;
      mbar_arrive_expect_tx_u32(full, kStage);
      for (int x = 0; x < 2; ++x) {
        tma_load_3d(at + x * kPanel, kmap, 64 * x, it.hk, row, full);
        tma_load_3d(at + kTile + x * kPanel, qmap, 64 * x, it.hk, row, full);
        tma_load_3d(at + 2 * kTile + x * kPanel, vmap, 64 * x, it.h, row, full);
      }
      asm volatile(
          "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              at + 3 * kTile),
          "l"(blobs + (it.blob + (long long)c * H) * kBlob), "r"(kBlob), "r"(full)
          : "memory");
    }
    __syncwarp();
    if (left < kC) {
      // the rows behind the sequence are another's: they must not meet the zeros of E' and T
      ok = __all_sync(0xffffffffu, mbar_wait_u32(full, 0));
      uint8_t *k = smem + s * kStage;
      for (int x = lane; x < (kC - left) * 16; x += 32) {
        uint8_t *to = k + (x & 1) * kPanel + (left + (x >> 4)) * 128 + ((x >> 1) & 7) * 16;
        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<uint4 *>(to + 2 * kTile) =
            make_uint4(0, 0, 0, 0);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive_u32(bar(kFull + s));
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(&g_give_up, 4u);
    for (int x = max(0, c - 2); x < c; ++x)  // the copies in flight
      if (it.n - x * kC >= kC) (void)mbar_wait_u32(bar(kFull + (x & 1)), (x >> 1) & 1);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    gdn_chunk_states(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap omap, const AdvanceArgs a,
                     const uint8_t *blobs) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  Item it;
  it.h = blockIdx.x;
  it.hk = it.h / (a.H / a.Hk);
  const int b = blockIdx.y;
  if (b == a.B) {  // the rows past the last sequence's
    it.start = min(max(__ldg(a.q_start + a.B), 0), a.rows);
    it.n = a.rows - it.start;
    it.slot = -1;
  } else {
    const Rows s = rows_of(a.q_start, b, a.rows);
    it.start = s.start;
    it.n = s.n;
    it.slot = slot_of(a.state_index, b, a.slots);
  }
  if (it.n == 0) return pdl_wait();
  if (it.slot < 0) {  // zeros
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (long long)it.start * a.out_stride +
                         (long long)it.h * a.dv;
    for (long long i = threadIdx.x; i < (long long)it.n * a.dv; i += kThreads)
      out[i / a.dv * a.out_stride + i % a.dv] = __float2bfloat16_rn(0.f);
    return pdl_wait();
  }
  it.chunks = (it.n + kC - 1) / kC;
  it.blob = (long long)(it.start / kC + b) * a.H + it.h;
  auto bar = [&](int i) { return base + kOffBars + 8u * i; };
  if (warp == kMmaWarp) tmem_alloc(base + kOffTmem, kTmemCols);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init_u32(bar(kFull + s), 1);
      mbar_init_u32(bar(kEmpty + s), 1 + kChainWarps + kOutWarps);
      mbar_init_u32(bar(kState + s), kChainWarps / 2);
      mbar_init_u32(bar(kR + s), kChainWarps / 2);
      mbar_init_u32(bar(kE + s), kChainWarps / 2);
      for (int i : {kKs, kTr, kSu}) mbar_init_u32(bar(i + s), 1);
    }
    mbar_init_u32(bar(kOutRead), kOutWarps);
    for (int i : {kTail, kQs, kOut}) mbar_init_u32(bar(i), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffTmem);
  if (warp < kChainWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChainRegs));
    run_chain(a, it, smem, base, tmem);
  } else if (warp < kChainWarps + kOutWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    write_out(a, &omap, it, smem, base, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp)
      issue_chunks(base, tmem, it);
    else if (warp == kLoadWarp)
      load_chunks(&kmap, &qmap, &vmap, blobs, a.H, it, smem, base);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows [rows][heads][dim] in boxes of kC rows of a head's columns: `box` of them.
sv_status encode_rows(CUtensorMap *map, const void *p, long long row_stride, int rows, int heads,
                      int dim, uint32_t box, CUtensorMapSwizzle swizzle) {
  qmv::EncodeTiledFn enc = qmv::encode_tiled();
  if (!enc) return fail(SV_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  if (rows == 1) row_stride = (long long)heads * dim;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)row_stride * 2};
  const cuuint32_t boxes[3] = {box, 1, kC}, ones[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides,
                         boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SV_ERR_CUDA, "tensor map encode failed (%d)", (int)r);
  return SV_OK;
}

}  // namespace

size_t chunk_workspace_bytes(int rows, int B, int H) {
  return (size_t)((long long)rows / kC + B) * H * kBlob;
}

sv_status chunk_run(const AdvanceArgs &a, void *workspace, cudaStream_t stream) {
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    const cudaError_t x = cudaFuncSetAttribute(
        gdn_chunk_matrices, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPrepSmem);
    return x != cudaSuccess ? x
                            : cudaFuncSetAttribute(gdn_chunk_states,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kSmem);
  });
  if (e != cudaSuccess)
    return fail(SV_ERR_CUDA, "gdn_advance: cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
  CUtensorMap kmap, qmap, vmap, omap;
  sv_status st = encode_rows(&kmap, a.k, a.k_stride, a.rows, a.Hk, a.dk, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == SV_OK)
    st = encode_rows(&qmap, a.q, a.q_stride, a.rows, a.Hk, a.dk, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == SV_OK)
    st = encode_rows(&vmap, a.v, a.v_stride, a.rows, a.H, a.dv, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == SV_OK)
    st = encode_rows(&omap, a.out, a.out_stride, a.rows, a.H, a.dv, kD, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != SV_OK) return st;
  uint8_t *blobs = static_cast<uint8_t *>(workspace);
  const long long items = ((long long)a.rows / kC + a.B) * a.H;
  if (items >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "gdn_advance: too many rows");
  if (items > 0) {
    gdn_chunk_matrices<<<(unsigned)items, kPrepThreads, kPrepSmem, stream>>>(a, blobs);
    st = check_launch("gdn_advance");
    if (st != SV_OK) return st;
  }
  // The states' launch begins as the matrices' drains.
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.H, (unsigned)a.B + 1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = items > 0 ? 1 : 0;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, gdn_chunk_states, kmap, qmap, vmap, omap, a,
                                            static_cast<const uint8_t *>(blobs));
  if (le != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(SV_ERR_CUDA, "gdn_advance: launch failed: %s", cudaGetErrorString(le));
  }
  return check_launch("gdn_advance");
}

}  // namespace gdn

// The GatedDeltaNet kernels' bounded waits are all in this unit.
unsigned take_device_error_gdn() {
  unsigned v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, gdn::g_give_up, sizeof v);
  cudaMemcpyToSymbol(gdn::g_give_up, &zero, sizeof zero);
  return v;
}

}  // namespace sv
