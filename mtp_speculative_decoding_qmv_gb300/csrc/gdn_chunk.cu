// gdn_chunk.cu -- the gated delta rule over packed bf16 rows in chunks of 64, on
// the tcgen05 tensor cores, sm_103a.
//
// Within a chunk, with S0 the state before it, G[i] the product of the gates from
// the chunk's first row to i, D[i][j] that from j + 1 to i (D[i][i] = 1):
//   e_i  = beta_i (v_i - G[i] S0 k_i - sum_{j<i} D[i][j] (k_i . k_j) e_j)
//   o_i  = G[i] S0 q_i + sum_{j<=i} D[i][j] (q_i . k_j) e_j
//   S    = G[63] S0 + sum_j D[63][j] e_j k_j^T
// With L = tril(beta D K K^T, -1), T = (1 + L)^-1 and P = tril(D Q K^T), as columns
// over the chunk's rows:
//   R = beta (V - G S0 K^T);  E = R T^T;  O = G S0 Q^T + E P^T;  S = G[63] S0 + E' K
// so the state enters five products a chunk, each with 128 rows (dv) in tensor
// memory's lanes: S0, R and E are A operands in tensor memory, K, Q, T and P (bf16,
// shared memory) are B.  K serves both as rows of dk (S0 K^T) and with dk
// contiguous (E' K), from one copy.
//
// Precision: the state stays in fp32 registers.  An fp32 operand is cut into three
// bf16 parts that add up to it exactly (8 bits of it each), so what reaches the
// state is fp32-exact products of K (bf16 as given): S0 K^T and E' K with three
// parts, R T^T with the six products of parts above 2^-24.  The output, bf16 in
// the end, takes two parts of S0, E and P: 2^-16, far below its own rounding.
//
// What bounds it is the chain from chunk to chunk, one CTA a (sequence, head): per
// chunk about 2000 cycles of tensor-core time on the chain (S0 K^T 768, R T^T 480,
// E' K 768), and between them the hand-overs to the warps that cut the parts.
// Everything off the chain runs beside it: S0 Q^T and E P^T in the gaps, T and P of
// the next chunk on four warps of their own (mma.sync for K K^T and Q K^T: small,
// and their results are wanted in registers), loads two chunks ahead.
#include <cuda_runtime.h>

#include "gdn_rows.cuh"
#include "tc05.cuh"

namespace sv {
namespace gdn {
namespace {

constexpr int kC = 64;    // rows a chunk
constexpr int kD = 128;   // dk and dv, narrower ones padded with zeros
constexpr int kChainWarps = 8, kPrepWarps = 4, kMmaWarp = 12, kLoadWarp = 13, kLoadWarps = 3;
constexpr int kThreads = 512;
// 256 x 160 + 256 x 96 = 512 x 128 registers
constexpr int kChainRegs = 160, kOtherRegs = 96;

// ---- shared memory ----------------------------------------------------------
constexpr uint32_t kTile = kC * kD * 2;             // K, Q or V of a chunk
constexpr uint32_t kPanel = kC * 128;               // 64 columns of it, 128-byte swizzle
constexpr uint32_t kStage = 3 * kTile;
constexpr uint32_t kPart = kC * kC * 2;             // a bf16 part of T or P
constexpr uint32_t kTParts = 3, kPParts = 2;
constexpr uint32_t kMats = (kTParts + kPParts) * kPart;
constexpr int kPitch = kC + 4;                      // floats a row of the scratch matrix
constexpr uint32_t kOffMats = 2 * kStage;
constexpr uint32_t kOffScratch = kOffMats + 2 * kMats;
constexpr uint32_t kOffGates = kOffScratch + kC * kPitch * 4;  // [2][alpha 64 | beta 64]
constexpr uint32_t kOffDecay = kOffGates + 2 * 2 * kC * 4;     // [2][G 64 | D[63] 64]
constexpr uint32_t kOffBars = kOffDecay + 2 * 2 * kC * 4;
enum Bar { kKvFull = 0, kKvEmpty = 2, kMatFull = 4, kMatEmpty = 6, kState = 8, kKs, kR, kTr, kQs, kE, kSu, kOut, kBars };
constexpr uint32_t kOffTmem = kOffBars + 8 * kBars;
constexpr uint32_t kSmem = kOffTmem + 16 + 1024;

// ---- tensor memory (columns) ------------------------------------------------
// The state's parts: of each half of dk (64 columns of it), three parts of 32
// columns; E' K of that half first lands in the same place.
constexpr uint32_t kColState = 0, kColHalf = 96;
constexpr uint32_t kColK = 192;   // S0 K^T, then E's two parts
constexpr uint32_t kColQ = 256;   // S0 Q^T
constexpr uint32_t kColE = 320;   // R T^T, then E P^T
constexpr uint32_t kColR = 384;   // R's parts, then E''s
constexpr uint32_t kTmemCols = 512;

__device__ unsigned int g_give_up;

constexpr uint32_t idesc(int n, bool mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10)  // D fp32; A, B bf16
         | (mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kD >> 4) << 24);
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  return mbar_wait_u32(bar, parity);
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Uses of registers that a tcgen05.ld fills stay behind its wait.
__device__ __forceinline__ void pin(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]),
                      "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7]));
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
        const float2 rest =
            __fadd2_rn(make_float2(a, b), make_float2(-__uint_as_float(ua & 0xFFFF0000u),
                                                      -__uint_as_float(ub & 0xFFFF0000u)));
        a = rest.x;
        b = rest.y;
      }
    }
  }
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes to shared memory, zeros where there is no source.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Address of the 16-byte piece `piece` (of 8) of a row of a 128-byte swizzled panel.
__device__ __forceinline__ uint32_t swizzled(int row, int piece) {
  return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

struct Item {
  int start, n, slot, h, hk, chunks;
};

// ---- the loads: K, Q, V and the gates of chunk c into stage c % 2 --------------
__device__ void load_chunk(const AdvanceArgs &a, const Item &it, uint8_t *smem, uint32_t base, int c,
                           int tid) {
  const int s = c & 1, t0 = c * kC, left = min(kC, it.n - t0);
  using B = __nv_bfloat16;
  const long long row0 = it.start + t0;
  const B *k = static_cast<const B *>(a.k) + row0 * a.k_stride + (long long)it.hk * a.dk;
  const B *q = static_cast<const B *>(a.q) + row0 * a.q_stride + (long long)it.hk * a.dk;
  const B *v = static_cast<const B *>(a.v) + row0 * a.v_stride + (long long)it.h * a.dv;
  const uint32_t at = base + s * kStage;
  for (int i = tid; i < kC * 16; i += kLoadWarps * 32) {
    const int row = i >> 4, piece = i & 15;
    const bool in = row < left;
    const bool col = in && 8 * piece < a.dk;
    const uint32_t to = (piece >> 3) * kPanel + swizzled(row, piece & 7);
    copy16(at + to, col ? k + row * a.k_stride + 8 * piece : k, col);
    copy16(at + kTile + to, col ? q + row * a.q_stride + 8 * piece : q, col);
    const bool value = in && 8 * piece < a.dv;
    copy16(at + 2 * kTile + row * (kD * 2) + piece * 16, value ? v + row * a.v_stride + 8 * piece : v,
           value);
  }
  float *gates = reinterpret_cast<float *>(smem + kOffGates) + s * 2 * kC;
  for (int i = tid; i < kC; i += kLoadWarps * 32) {
    const long long g = (row0 + i) * a.H + it.h;
    gates[i] = i < left ? __ldg(a.alpha + g) : 1.f;
    gates[kC + i] = i < left ? __ldg(a.beta + g) : 0.f;
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// ---- T and P of chunk c, by four warps ------------------------------------------
__device__ __forceinline__ void store_parts(uint8_t *mats, int i, int j, float x) {
  float a = x;
#pragma unroll
  for (int p = 0; p < (int)kTParts; ++p) {
    const uint32_t u = __float_as_uint(a);
    *reinterpret_cast<uint16_t *>(mats + p * kPart + swizzled(i, j >> 3) + (j & 7) * 2) =
        (uint16_t)(u >> 16);
    a -= __uint_as_float(u & 0xFFFF0000u);
  }
}

__device__ void prepare(uint8_t *smem, uint32_t base, int c) {
  const int s = c & 1, tid = threadIdx.x - kChainWarps * 32, warp = tid >> 5, lane = tid & 31;
  float *scratch = reinterpret_cast<float *>(smem + kOffScratch);
  const float *alpha = reinterpret_cast<const float *>(smem + kOffGates) + s * 2 * kC;
  const float *beta = alpha + kC;
  float *decay = reinterpret_cast<float *>(smem + kOffDecay) + s * 2 * kC;
  uint8_t *mats = smem + kOffMats + s * kMats;
  // D below the diagonal, a column a thread, by products (a gate of 0 or gates
  // whose product underflows need no care); the column before the first is G
  if (tid <= kC) {
    float d = 1.f;
    const int j = tid - 1;
#pragma unroll 8
    for (int i = 0; i < kC; ++i) {
      if (i > j) d *= alpha[i];
      if (j < 0)
        decay[i] = d;
      else
        scratch[i * kPitch + j] = i >= j ? d : 0.f;
    }
    if (j >= 0) decay[kC + j] = d;
  }
  // K K^T and Q K^T of the warp's 16 rows and the columns up to them
  const uint32_t k_at = base + s * kStage, q_at = k_at + kTile;
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) kk[i][m] = qk[i][m] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < kD / 16; ++ks) {
    const uint32_t panel = (ks >> 2) * kPanel;
    const int piece = (ks & 3) * 2;
    uint32_t ak[4], aq[4];
    const uint32_t a_off = panel + swizzled(16 * warp + (lane & 15), piece + (lane >> 4));
    ldmatrix_x4(ak, k_at + a_off);
    ldmatrix_x4(aq, q_at + a_off);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np <= warp) {
        uint32_t b[4];
        const int row = 16 * np + ((lane >> 4) << 3) + (lane & 7);
        ldmatrix_x4(b, k_at + panel + swizzled(row, piece + ((lane >> 3) & 1)));
        mma_bf16_m16n8k16(kk[2 * np], ak[0], ak[1], ak[2], ak[3], b[0], b[1]);
        mma_bf16_m16n8k16(kk[2 * np + 1], ak[0], ak[1], ak[2], ak[3], b[2], b[3]);
        mma_bf16_m16n8k16(qk[2 * np], aq[0], aq[1], aq[2], aq[3], b[0], b[1]);
        mma_bf16_m16n8k16(qk[2 * np + 1], aq[0], aq[1], aq[2], aq[3], b[2], b[3]);
      }
    }
  }
  prep_sync();  // D is there
  const int g8 = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    if (nt >= 2 * (warp + 1)) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 16 * warp + g8 + 8 * half, j = 8 * nt + 2 * t4;
      float2 *d = reinterpret_cast<float2 *>(scratch + i * kPitch + j);
      const float2 w = *d;
      const float be = beta[i];
      // above the diagonal D is 0; the diagonal is P's alone
      float p[2] = {j <= i ? qk[nt][2 * half] * w.x : 0.f, j < i ? qk[nt][2 * half + 1] * w.y : 0.f};
      *d = make_float2(j < i ? be * (kk[nt][2 * half] * w.x) : 0.f,
                       j + 1 < i ? be * (kk[nt][2 * half + 1] * w.y) : 0.f);
      uint32_t part[kPParts][1];
      cut<1, kPParts>(p, part);
#pragma unroll
      for (int x = 0; x < (int)kPParts; ++x)
        *reinterpret_cast<uint32_t *>(mats + (kTParts + x) * kPart + swizzled(i, nt) + t4 * 4) =
            part[x][0];
    }
  }
  prep_sync();  // L is there
  // T: the two diagonal blocks of 32, a column a lane, by substitution
  if (warp < 2) {
    const float *block = scratch + (32 * kPitch + 32) * warp;
    float t[32];
    t[0] = lane == 0 ? 1.f : 0.f;
#pragma unroll
    for (int i = 1; i < 32; ++i) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(block + i * kPitch + m);
        const float lm[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (m + x < i) sum[x] = fmaf(lm[x], t[m + x], sum[x]);
      }
      t[i] = (lane == i ? 1.f : 0.f) - ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
    __syncwarp();
    float *to = scratch + (32 * kPitch + 32) * warp + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      to[i * kPitch] = t[i];
      store_parts(mats, 32 * warp + i, 32 * warp + lane, t[i]);
    }
  }
  prep_sync();
  // the block below: -T11 (L10 T00), two rows by four columns a thread
  const int r = 2 * (tid >> 3), c4 = 4 * (tid & 7);
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    // pass 0: X = L10 T00 in L10's place; pass 1: T11 X
    const float *left = scratch + (32 + r) * kPitch + (pass ? 32 : 0);
    const float *right = scratch + (pass ? 32 * kPitch : 0) + c4;
    float2 x[2][2] = {};
#pragma unroll
    for (int m = 0; m < 32; m += 4) {
      const float4 l0 = *reinterpret_cast<const float4 *>(left + m);
      const float4 l1 = *reinterpret_cast<const float4 *>(left + kPitch + m);
      const float w0[4] = {l0.x, l0.y, l0.z, l0.w}, w1[4] = {l1.x, l1.y, l1.z, l1.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4 t = *reinterpret_cast<const float4 *>(right + (m + y) * kPitch);
        const float2 lo = make_float2(t.x, t.y), hi = make_float2(t.z, t.w);
        x[0][0] = __ffma2_rn(make_float2(w0[y], w0[y]), lo, x[0][0]);
        x[0][1] = __ffma2_rn(make_float2(w0[y], w0[y]), hi, x[0][1]);
        x[1][0] = __ffma2_rn(make_float2(w1[y], w1[y]), lo, x[1][0]);
        x[1][1] = __ffma2_rn(make_float2(w1[y], w1[y]), hi, x[1][1]);
      }
    }
    if (pass == 0) {
      __syncwarp();  // the rows of L10 that this warp reads are this warp's alone
#pragma unroll
      for (int y = 0; y < 2; ++y)
        *reinterpret_cast<float4 *>(scratch + (32 + r + y) * kPitch + c4) =
            make_float4(x[y][0].x, x[y][0].y, x[y][1].x, x[y][1].y);
      prep_sync();
    } else {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float v[4] = {-x[y][0].x, -x[y][0].y, -x[y][1].x, -x[y][1].y};
        uint32_t part[kTParts][2];
        cut<2, kTParts>(v, part);
#pragma unroll
        for (int p = 0; p < (int)kTParts; ++p)
          *reinterpret_cast<uint2 *>(mats + p * kPart + swizzled(32 + r + y, c4 >> 3) + (c4 & 7) * 2) =
              make_uint2(part[p][0], part[p][1]);
      }
    }
  }
}

// E or the outputs: D[dv][64 rows] (+)= A parts x B parts, lower triangular: the
// 16 columns of k step j reach the rows from 16 j on.
template <int kNa, int kNb>
__device__ __forceinline__ void mma_lower(uint32_t d, uint32_t a, uint32_t b, int least) {
  uint32_t acc = 0;
#pragma unroll
  for (int pa = 0; pa < kNa; ++pa)
#pragma unroll
    for (int pb = 0; pb < kNb; ++pb) {
      if (pa + pb > least) continue;  // below the last part's weight
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) {
        tc_mma_ts(d + 16 * j, a + 32 * pa + 8 * j,
                  smem_desc_sw128(b + pb * kPart + j * 2048 + j * 32), idesc(kC - 16 * j, false), acc);
        acc = 1;
      }
    }
}
// S0 times K^T or Q^T.
template <int kNp>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t tmem, uint32_t b) {
#pragma unroll
  for (int p = 0; p < kNp; ++p)
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks)
      tc_mma_ts(d, tmem + kColState + (ks >> 2) * kColHalf + 32 * p + 8 * (ks & 3),
                smem_desc_sw128(b + (ks >> 2) * kPanel + (ks & 3) * 32), idesc(kC, false),
                p + ks > 0);
}

__device__ void issue_chunks(uint32_t base, uint32_t tmem, const Item &it) {
  auto bar = [&](int i) { return base + kOffBars + 8u * i; };
  const bool one = elect_one();
  bool ok = true;
  auto wait = [&](int i, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar(i), parity));
    tc_fence_after();
    return ok;
  };
  for (int c = 0; c < it.chunks && ok; ++c) {
    const uint32_t s = c & 1, odd = c & 1, pair = (c >> 1) & 1;
    const uint32_t k_at = base + s * kStage, q_at = k_at + kTile;
    const uint32_t t_at = base + kOffMats + s * kMats, p_at = t_at + kTParts * kPart;
    if (c > 0 && !wait(kOut, odd ^ 1)) break;  // E P^T read what S0 K^T overwrites
    if (!wait(kKvFull + s, pair) || !wait(kState, odd)) break;
    if (one) {
      mma_state<3>(tmem + kColK, tmem, k_at);
      tc_commit(bar(kKs));
    }
    __syncwarp();
    if (!wait(kMatFull + s, pair) || !wait(kR, odd)) break;
    if (one) {
      mma_lower<3, 3>(tmem + kColE, tmem + kColR, t_at, 2);
      tc_commit(bar(kTr));
      mma_state<2>(tmem + kColQ, tmem, q_at);
      tc_commit(bar(kQs));
    }
    __syncwarp();
    if (!wait(kQs, odd) || !wait(kE, odd)) break;
    if (one) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int j = 0; j < kC / 16; ++j)
            tc_mma_ts(tmem + kColState + half * kColHalf, tmem + kColR + 32 * p + 8 * j,
                      smem_desc_sw128_mn(k_at + half * kPanel + j * 2048, kPanel), idesc(64, true),
                      p + j > 0);
      tc_commit(bar(kSu));
      mma_lower<2, 2>(tmem + kColE, tmem + kColK, p_at, 1);
      tc_commit(bar(kOut));
      tc_commit(bar(kKvEmpty + s));
      tc_commit(bar(kMatEmpty + s));
    }
    __syncwarp();
  }
  if (!ok && one) atomicOr(&g_give_up, 1u);
}

// ---- the chain: lane = row of the state (dv), warps 0..3 the first half of the
// chunk's rows and of dk, 4..7 the second ------------------------------------------
__device__ void run_chain(const AdvanceArgs &a, const Item &it, uint8_t *smem, uint32_t base,
                          uint32_t tmem_base) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = 32 * (warp & 3) + lane, half = warp >> 2;
  const uint32_t tmem = tmem_base + ((uint32_t)(warp & 3) << 21);
  auto bar = [&](int b) { return base + kOffBars + 8u * b; };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive_u32(bar(b));
  };
  bool ok = true;
  auto wait = [&](int b, uint32_t parity) {
    ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity));
    tc_fence_after();
    return ok;
  };
  float S[64];
  float *state = a.state + (((long long)it.slot * a.H + it.h) * a.dv + (i < a.dv ? i : 0)) * a.dk + 64 * half;
#pragma unroll
  for (int m = 0; m < 64; m += 4) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < a.dv && 64 * half + m < a.dk) x = __ldcg(reinterpret_cast<const float4 *>(state + m));
    S[m] = x.x;
    S[m + 1] = x.y;
    S[m + 2] = x.z;
    S[m + 3] = x.w;
  }
  const uint32_t s_at = tmem + kColState + half * kColHalf;
  auto put_state = [&] {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t part[3][16];
      cut<16, 3>(S + 32 * g, part);
#pragma unroll
      for (int p = 0; p < 3; ++p) tc_st_x16(s_at + 32 * p + 16 * g, part[p]);
    }
    tc_wait_st();
    tc_fence_before();
    arrive(kState);
  };
  put_state();
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (long long)it.start * a.out_stride +
                       (long long)it.h * a.dv + i;
  for (int c = 0; c < it.chunks; ++c) {
    const uint32_t s = c & 1, odd = c & 1, pair = (c >> 1) & 1;
    const float *beta = reinterpret_cast<const float *>(smem + kOffGates) + s * 2 * kC + kC + 32 * half;
    const float *G = reinterpret_cast<const float *>(smem + kOffDecay) + s * 2 * kC + 32 * half;
    const float *last = G + kC;
    const uint16_t *v = reinterpret_cast<const uint16_t *>(smem + s * kStage + 2 * kTile) +
                        32 * half * kD + i;
    const int left = it.n - c * kC - 32 * half;  // rows of this half
    // R = beta (v - G S0 k)
    if (!wait(kKvFull + s, pair) || !wait(kMatFull + s, pair) || !wait(kKs, odd)) break;
    {
      uint32_t x[32];
      tc_ld_x32(tmem + kColK + 32 * half, x);
      float val[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) val[j] = __uint_as_float((uint32_t)v[j * kD] << 16);
      tc_wait_ld();
      pin(x);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 be = *reinterpret_cast<const float4 *>(beta + j);
        const float4 g = *reinterpret_cast<const float4 *>(G + j);
        val[j] = be.x * fmaf(-g.x, __uint_as_float(x[j]), val[j]);
        val[j + 1] = be.y * fmaf(-g.y, __uint_as_float(x[j + 1]), val[j + 1]);
        val[j + 2] = be.z * fmaf(-g.z, __uint_as_float(x[j + 2]), val[j + 2]);
        val[j + 3] = be.w * fmaf(-g.w, __uint_as_float(x[j + 3]), val[j + 3]);
      }
      if (left < 32) {  // no row: a state that is not finite must not reach it
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= left) val[j] = 0.f;
      }
      uint32_t part[3][16];
      cut<16, 3>(val, part);
#pragma unroll
      for (int p = 0; p < 3; ++p) tc_st_x16(tmem + kColR + 32 * p + 16 * half, part[p]);
      tc_wait_st();
      tc_fence_before();
      arrive(kR);
      arrive(kKvEmpty + s);
    }
    // E and E' = D[63] E
    if (!wait(kTr, odd)) break;
    {
      uint32_t x[32];
      tc_ld_x32(tmem + kColE + 32 * half, x);
      tc_wait_ld();
      pin(x);
      float e[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 d = *reinterpret_cast<const float4 *>(last + j);
        e[j] = d.x * __uint_as_float(x[j]);
        e[j + 1] = d.y * __uint_as_float(x[j + 1]);
        e[j + 2] = d.z * __uint_as_float(x[j + 2]);
        e[j + 3] = d.w * __uint_as_float(x[j + 3]);
      }
      {
        uint32_t part[3][16];
        cut<16, 3>(e, part);
#pragma unroll
        for (int p = 0; p < 3; ++p) tc_st_x16(tmem + kColR + 32 * p + 16 * half, part[p]);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) e[j] = __uint_as_float(x[j]);
      {
        uint32_t part[2][16];
        cut<16, 2>(e, part);
#pragma unroll
        for (int p = 0; p < 2; ++p) tc_st_x16(tmem + kColK + 32 * p + 16 * half, part[p]);
      }
      tc_wait_st();
      tc_fence_before();
      arrive(kE);
    }
    // S = G[63] S0 + E' K
    if (!wait(kSu, odd)) break;
    {
      const float g = reinterpret_cast<const float *>(smem + kOffDecay)[s * 2 * kC + kC - 1];
      const float2 g2 = make_float2(g, g);
#pragma unroll
      for (int m = 0; m < 64; m += 32) {
        uint32_t x[32];
        tc_ld_x32(s_at + m, x);
        tc_wait_ld();
        pin(x);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 n = __ffma2_rn(g2, make_float2(S[m + j], S[m + j + 1]),
                                      make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
          S[m + j] = n.x;
          S[m + j + 1] = n.y;
        }
      }
      if (c + 1 < it.chunks) put_state();
    }
    // o = G S0 q + E P
    if (!wait(kOut, odd)) break;
    {
      uint32_t x[32], y[32];
      tc_ld_x32(tmem + kColQ + 32 * half, x);
      tc_ld_x32(tmem + kColE + 32 * half, y);
      tc_wait_ld();
      pin(x);
      pin(y);
      __nv_bfloat16 *to = out + (long long)(c * kC + 32 * half) * a.out_stride;
      if (i < a.dv) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < left)
            to[j * a.out_stride] =
                __float2bfloat16_rn(fmaf(G[j], __uint_as_float(x[j]), __uint_as_float(y[j])));
      }
      tc_fence_before();
      arrive(kMatEmpty + s);
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(&g_give_up, 2u);
    return;
  }
  if (i < a.dv) {
#pragma unroll
    for (int m = 0; m < 64; m += 4)
      if (64 * half + m < a.dk)
        *reinterpret_cast<float4 *>(state + m) = make_float4(S[m], S[m + 1], S[m + 2], S[m + 3]);
  }
}

__global__ void __launch_bounds__(kThreads, 1) gdn_chunk_kernel(const AdvanceArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  if (it.n == 0) return;
  if (it.slot < 0) {  // zeros
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (long long)it.start * a.out_stride +
                         (long long)it.h * a.dv;
    for (long long i = threadIdx.x; i < (long long)it.n * a.dv; i += kThreads)
      out[i / a.dv * a.out_stride + i % a.dv] = __float2bfloat16_rn(0.f);
    return;
  }
  it.chunks = (it.n + kC - 1) / kC;
  auto bar = [&](int i) { return base + kOffBars + 8u * i; };
  if (warp == kMmaWarp) tmem_alloc(base + kOffTmem, kTmemCols);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init_u32(bar(kKvFull + s), kLoadWarps * 32);
      mbar_init_u32(bar(kKvEmpty + s), 1 + kChainWarps + kPrepWarps);
      mbar_init_u32(bar(kMatFull + s), kPrepWarps);
      mbar_init_u32(bar(kMatEmpty + s), 1 + kChainWarps);
    }
    mbar_init_u32(bar(kState), kChainWarps);
    mbar_init_u32(bar(kR), kChainWarps);
    mbar_init_u32(bar(kE), kChainWarps);
    for (int i : {kKs, kTr, kQs, kSu, kOut}) mbar_init_u32(bar(i), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffTmem);

  if (warp < kChainWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChainRegs));
    run_chain(a, it, smem, base, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kMmaWarp) {
      bool ok = true;
      for (int c = 0; c < it.chunks; ++c) {
        const uint32_t s = c & 1, pair = (c >> 1) & 1;
        ok = wait_bar(bar(kKvFull + s), pair);
        if (ok && c >= 2) ok = wait_bar(bar(kMatEmpty + s), pair ^ 1);
        // all four warps go on or none does
        int all;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
            "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
            : "=r"(all)
            : "r"((int)ok)
            : "memory");
        ok = all != 0;
        if (!ok) break;
        prepare(smem, base, c);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_u32(bar(kMatFull + s));
          mbar_arrive_u32(bar(kKvEmpty + s));
        }
      }
      if (!ok && lane == 0) atomicOr(&g_give_up, 4u);
    } else if (warp == kMmaWarp) {
      issue_chunks(base, tmem, it);
    } else {
      const int tid = threadIdx.x - kLoadWarp * 32;
      bool ok = true;
      load_chunk(a, it, smem, base, 0, tid);
      for (int c = 0; c < it.chunks; ++c) {
        if (c + 1 < it.chunks) {
          const uint32_t s = (c + 1) & 1;
          if (c + 1 >= 2) ok = wait_bar(bar(kKvEmpty + s), (((c + 1) >> 1) & 1) ^ 1);
          if (!ok) break;
          load_chunk(a, it, smem, base, c + 1, tid);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        fence_async();
        mbar_arrive_u32(bar(kKvFull + (c & 1)));
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok && lane == 0) atomicOr(&g_give_up, 8u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

sv_status chunk_run(const AdvanceArgs &a, cudaStream_t stream) {
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(gdn_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kSmem);
  });
  if (e != cudaSuccess)
    return fail(SV_ERR_CUDA, "gdn_advance: cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
  const dim3 grid((unsigned)a.H, (unsigned)a.B + 1);
  gdn_chunk_kernel<<<grid, kThreads, kSmem, stream>>>(a);
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
