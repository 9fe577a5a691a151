// Split-KV paged GQA decode attention over a 4-bit pool (e2m1 codes, a power of two as
// the scale of each 32 values of a token's head) with a per-tile log-sum-exp, for
// sm_103a.
//
// A token of a kv head has D + D / 16 bytes, 17/64 of the bf16 pool's, so at the memory's rate
// an SM has ~750 cycles for a page of 64 tokens at 256 dims.  What bounds the kernel is work on
// the codes: 128 conversions of two codes, 48 products and 64 multiplications by V's scales a
// warp and page, ~940 cycles with four warps per scheduler and all in shared memory (products
// share their issue with fp32 and fp16 arithmetic), ~1,150 in place, where no pipe is full and a
// scheduler's warps wait for each other's results and barriers.  4 x 31,744 tokens of 4 kv heads
// of 256 dims: 39.5 us (20 at the memory's rate), 262,144 tokens 80.4 (42).
//
// Scales differ along the dims of a head, so they cannot go with the rows of a product as the
// 8-bit pool's do: codes become fp16 in registers and both products run as mma.sync m16n8k16
// with fp32 sums.  (The fifth-generation tensor cores take K with its scales as it lies, but
// V's scales are per token, its sum's index.  With their scores, four softmax warps and eight for
// the products: 4 x 31,744 tokens 38 us, but 64 requests of up to 3,000 tokens of 128 dims 40
// instead of 35; with V's fp16 values in tensor memory 52 and 44.)
//
//  * Work split and partials: as the other decode kernels (split_units.cuh, unit_plan.h);
//    a request's tiles are merged by a kernel of its own (tile_merge.cuh).
//  * One thread streams pages with TMA into a ring of stages: the codes of a page's K and V of
//    a head (one box, swizzled), and their scales (another).
//  * A page is a team's: four warps at 256 dims, two at 128, 16 warps in all.  A warp has the
//    scores of its share of the tokens, then the products of all 64 with its 64 dims: 16
//    registers of sums, so that four warps fit a scheduler.  (With all dims of 32 tokens in a
//    warp, two to a scheduler, its straight code outran the instruction cache: 91 us for the
//    262,144 tokens.)  The team meets once per page, at a barrier that also tells whether any
//    warp's scores or scales are beyond the references.
//  * S = K Q^T: 16 tokens as the rows of A, the G <= 8 heads as the columns of B, so no row
//    is idle.  A 16-byte run of a row is one scale's group; ldmatrix gives a lane 8 of its
//    values in one word, two products sum the group, and an fp32 FMA with the token's scale
//    adds it to the score.  q is scaled by a power of two per head and held in fp16: all its
//    8 bits down to 2^-31 of the head's largest.
//  * Softmax: e = 2^(x - m) for the sum, with m a multiple of 8 near the largest score; the
//    product's weight is w = e 2^(v - m') in fp16 as a high and a low part (22 bits), with 2^v
//    the token's largest V scale and m' such that w is at most 2^15 whatever the scales: a
//    weight is within 2^-23 of itself, or 2^-37 of the row's largest.  m and m' move rarely
//    (m' leaves three bits of room), then by an exact power of two.
//  * O^T = V^T P^T: 16 dims as rows (a lane's words hold the dims of one group, two tokens'
//    codes are interleaved by nibble so that one conversion gives a register of A), tokens
//    as k, heads as columns; P comes from the scores' layout by movmatrix, through shared
//    memory.  V's codes are multiplied by their scale relative to the token's largest (exact).
//    Every 32 tokens' product starts from zero and is added to fp32 registers.
//  * The teams' parts of a segment meet in shared memory; two output warps add and store them
//    (and merge split units) while the teams are at the next segment.
//  * A launch starts under programmatic dependent launch; only what reads or writes global
//    memory waits for the kernels before it.  All waits on loads have a time limit; a warp that
//    gives up goes on meeting its team, at barriers without one, until all have.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>
#include <vector>

#include "common.h"
#include "f32x2.cuh"
#include "fp4.cuh"
#include "ptx.cuh"
#include "split_units.cuh"
#include "tile_merge.cuh"
#include "unit_plan.h"
#include "unit_walk.cuh"

namespace pa {
namespace decode_q4 {

using namespace split;

constexpr int kGroup = PA_Q4_GROUP;
constexpr int kConsumers = 16, kOutWarps = 2, kOut = 32 * kOutWarps;
constexpr int kTmaWarp = kConsumers + kOutWarps, kHelperWarp = kTmaWarp + 1;
constexpr int kThreads = 32 * (kHelperWarp + 1);
constexpr int kTop = 15;                     // log2 of the largest weight
constexpr int kUp = 13;                      // V's codes go in times 2^13: 6 * 2^13 is in range
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNoRef = -1e30f;             // m before the first score
constexpr int kNoRho = -1000;
constexpr float kMostExp = 0x1p64f;          // e may lie above 1, up to this
constexpr int kSlack = 3;                    // what m' leaves above the largest weight so far (log2)
constexpr float kMostWeight = 65000.f;       // in fp16, which ends at 65504
constexpr int kSpread = 16;                  // see attend()
constexpr int kAlways = 4096;                // see Part::most
constexpr float kLargeFactor = 0x1p60f;      // (a product is below 2^23: 2^-127 of it 2^-44 here)

// Shared memory of a CTA; offsets from a 1024-byte boundary.
template <int D>
struct Smem {
  static constexpr int kTeam = D / 64;                     // warps to a page
  static constexpr int kTeams = kConsumers / kTeam;        // pages at once
  static constexpr int kOwn = kPage / kTeam;               // tokens that a warp has the scores of
  static constexpr int kRow = D / 2;                       // a token's codes
  static constexpr int kHalf = kPage * kRow;               // K (or V) of a page
  static constexpr int kScaleRow = D / kGroup;
  static constexpr int kScaleHalf = kPage * kScaleRow;
  static constexpr int kStages = D == 256 ? 9 : 16;
  static constexpr int kScales = kStages * 2 * kHalf;      // [stage][K | V]
  static constexpr int kQ = kScales + kStages * 2 * kScaleHalf;   // [2][group][lane] 16 bytes
  static constexpr int kQBytes = D / kGroup * 32 * 16;
  // [team][2]: a page's weights as registers of B, [16 tokens][lane] 16 bytes; of a page whose
  // scales lie far apart the probabilities [token][head]
  static constexpr int kP = kQ + 2 * kQBytes;
  static constexpr int kPBytes = kPage * kMaxG * 4;
  // [team][2][group][place_of(token)]: what V's codes are multiplied by, in fp16 (a group's row
  // is padded by four banks)
  static constexpr int kF = kP + kTeams * 2 * kPBytes;
  static constexpr int kFRow = kPage * 2 + 16, kFBytes = D / kGroup * kFRow;
  // [team][8 dims][dim][head]; the rows of 8 dims are padded so that the eight that a warp
  // writes lie 8 banks apart
  static constexpr int kX = kF + kTeams * 2 * kFBytes;
  static constexpr int kXRow = 8 * kMaxG + 8;
  static constexpr int kXPart = D / 8 * kXRow * 4;
  static constexpr int kStats = kX + kTeams * kXPart;      // [team][m | rho][head]
  static constexpr int kSums = kStats + kTeams * 2 * kMaxG * 4;   // [warp][head]
  static constexpr int kMeet = kSums + kConsumers * kMaxG * 4;    // [team] Meet
  static constexpr int kMeetBytes = (2 * kMaxG + 2) * kTeam * 4;
  static constexpr int kQFactor = kMeet + kTeams * kMeetBytes;    // [2][head]
  static constexpr int kFactors = kQFactor + 2 * kMaxG * 4;   // of each output warp
  static constexpr int kBars = kFactors + kOutWarps * (kTeams + 2) * kMaxG * 4;
  static constexpr int kFull = 0, kEmpty = kFull + kStages, kQFull = kEmpty + kStages,
                       kQEmpty = kQFull + 2, kXFull = kQEmpty + 2, kXEmpty = kXFull + 1,
                       kNumBars = kXEmpty + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;       // ints, see View
  static constexpr int kUsed = kMisc + (kStages + 4 + 2 * kTeams) * 4;
  static constexpr int kAlloc = kUsed + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
};
// What the warps of a team tell each other when references move.
template <int D>
struct Meet {
  float top[Smem<D>::kTeam][kMaxG], up[Smem<D>::kTeam][kMaxG];
  int most[Smem<D>::kTeam], least[Smem<D>::kTeam];
};

template <int kMaxUnits>
struct Params {
  const __nv_bfloat16* q;
  const int32_t* page_table;
  float* out;
  float* lse;
  int32_t* status;
  unsigned long long* arrivals;
  float* part_o;
  float* part_ml;
  long long pool_pages;
  int max_pages;
  int T;
  int Hq;
  int Hkv;
  int G;
  int n_units;
  int n_full;   // units with pages; the others follow them
  int grid;
  float scale_log2;
  unsigned long long wait_limit_ns;
  int stall_iteration;
  unsigned long long slice_wait_ns;
  // One tile per request: its output may be the merged one too, written with it.
  static constexpr bool kAllSlices = true, kMerge = false, kSecondOut = true;
  float* out2;
  float* lse2;
  int32_t starts[kMaxGrid + 1];      // CTA k takes flattened pages [k], [k + 1)
  int16_t first_unit[kMaxGrid + 1];  // and its first unit
  DevUnit units[kMaxUnits];
};
static_assert(sizeof(Params<kMaxUnitsLarge>) <= 32764, "kernel parameters too large");

struct View {
  uint8_t* base;
  uint32_t addr;          // shared-space address of base
  uint32_t bars;
  volatile int* poison;   // [stages] the page is not there
  volatile int* abort_flag;
  volatile int* merge_info;
  volatile int* given_up;  // [team] a wait of one of its warps has run out
  volatile int* idle;      // [team] no page of the segment was its
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
};

__device__ __forceinline__ void load_codes(uint32_t dst, const CUtensorMap* tmap, int head, int page,
                                           uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %3, %2, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void load_scales(uint32_t dst, const CUtensorMap* tmap, int head,
                                            int page, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %2, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(pol)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ float ex2(float x) {   // 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A B + C for a 16x8x16 fp16 tile with fp32 sums.
struct Acc {
  float2 lo, hi;   // rows lane / 4 and + 8, columns 2 (lane % 4) and + 1
};
__device__ __forceinline__ Acc mma(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                   uint32_t b1, const Acc& c) {
  Acc d;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d.lo.x), "=f"(d.lo.y), "=f"(d.hi.x), "=f"(d.hi.y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c.lo.x), "f"(c.lo.y),
        "f"(c.hi.x), "f"(c.hi.y));
  return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {   // fp16 pairs
  return as_u32(__hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y)));
}
// Token that row r (0 .. 15) of a product's tile stands for, relative to the tile's first:
// at 128 dims the two low bits change places, so that the rows that four neighbouring lanes
// read of V lie in different banks.
template <int D>
__device__ __forceinline__ int place(int r) {
  return D == 256 ? r : (r & 12) | (r & 1) << 1 | (r >> 1 & 1);
}
// Where 16-byte run c of token row r lies in a page's codes (the copies' swizzle).
template <int D>
__device__ __forceinline__ int run_at(int r, int c) {
  return r * Smem<D>::kRow + ((c ^ (D == 256 ? r & 7 : r >> 1 & 3)) << 4);
}

// Tokens of 32 are ordered so that 16 bytes hold the eight that lane t of four has in two
// tiles of 16: t's 2t, 2t + 1, 2t + 8, 2t + 9 of both.  n: 16 tile + row.
__device__ __forceinline__ int place_of(int n) {
  return (n & ~31) | (n >> 1 & 3) << 3 | (n >> 4 & 1) << 2 | (n >> 3 & 1) << 1 | (n & 1);
}

// ---------------------------------------------------------------------------
// Warps 0-15: teams of D / 64 warps.
// ---------------------------------------------------------------------------

// What a lane keeps of its team's part of a segment: for heads 2 (lane % 4) and + 1 the
// reference m and the difference rho of m' to it (the team's), its share of the sum; and the
// products of those heads with dims 8 (lane / 4) ... of its warp's 64.
struct Part {
  float2 o[4][2];           // [byte of codes][dim of the byte]
  float m[2], l[2];
  int rho[2];
  int most;                 // largest byte of V's scales so far, less kAlways: every page moves
};

// Scale bytes of V: word i holds those of group kWords t + i of rows g (low half) and g + 8 of a
// tile.
template <int D>
struct Bytes {
  static constexpr int kWords = D / 128;
  uint32_t b[kWords];
  __device__ __forceinline__ void load(uint32_t row, int t) {
    constexpr int kNext = 8 * Smem<D>::kScaleRow;
    if constexpr (D == 256) {
      const uint32_t x = lds16(row + 2 * t), y = lds16(row + kNext + 2 * t);
      b[0] = __byte_perm(x, y, 0x2420);
      b[kWords - 1] = __byte_perm(x, y, 0x2521);
    } else {
      b[0] = lds8(row + t) | lds8(row + kNext + t) << 16;
    }
  }
  // the rows' largest, over all lanes t
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t e = __vmaxu2(b[0], b[kWords - 1]);
    e = __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 1));
    return __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 2));
  }
};

// The products of a page whose V scales lie far apart: in fp32, token by token, from the weights
// and largest scales of its tokens.
template <int D>
__device__ __forceinline__ void attend_wide(Part& part, uint32_t codes, uint32_t vscales,
                                            const float* weights, uint32_t largest, int own,
                                            int lo, int hi, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll (D == 128 ? 2 : 1)
  for (int i = 0; i < kPage; ++i) {
    const int row = (i & ~7) + place<D>(i & 7);
    if (row < lo || row >= hi) continue;
    const int b = lds8(vscales + row * S::kScaleRow + own);
    float2 w = f32x2::mul(
        *reinterpret_cast<const float2*>(weights + i * kMaxG + 2 * t),
        f32x2::both(__int_as_float(max(b - (int)lds8(largest + i) + kUp + 127, 0) << 23)));
    if (b == fp4::kNanScale) w = f32x2::both(__int_as_float(0x7fc00000));
    float y[8];
    fp4::unpack8(lds32(codes + run_at<D>(row, own) + 4 * (g & 3)), y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2& o = part.o[k / 2][k % 2];
      o = f32x2::fma(w, f32x2::both(y[k]), o);
    }
  }
}

// The scores of 16 kTiles tokens from token item0 of a page, but for q's factors.
template <int D, int kTiles>
__device__ __forceinline__ void scores(float2 (&x)[kTiles][2], uint32_t codes, uint32_t scales,
                                       uint32_t q, int item0, int lane) {
  using S = Smem<D>;
  constexpr int kChunks = D / kGroup;
  const int g = lane >> 2;
  // the scales of four groups from group c, and of the four after them
  uint32_t ks[kTiles][2][kChunks / 4];
#pragma unroll
  for (int i = 0; i < 2 * kTiles; ++i) {
    const uint32_t a = scales + (item0 + 16 * (i >> 1) + 8 * (i & 1) + place<D>(g)) * S::kScaleRow;
    x[i >> 1][i & 1] = make_float2(0.f, 0.f);
    if constexpr (D == 256) {
      const uint2 w = lds64(a);
      ks[i >> 1][i & 1][0] = w.x;
      ks[i >> 1][i & 1][kChunks / 4 - 1] = w.y;
    } else {
      ks[i >> 1][i & 1][0] = lds32(a);
    }
  }
  const int r = place<D>(lane & 7) + (lane & 8);
  const uint32_t k0 = codes + run_at<D>(item0 + r, lane >> 4);
#pragma unroll
  for (int c = 0; c < kChunks; c += 2) {
    const uint4 qa = lds128(q + (c * 32 + lane) * 16), qb = lds128(q + (c * 32 + 32 + lane) * 16);
#pragma unroll
    for (int tile = 0; tile < kTiles; ++tile) {
      uint32_t w[4];
      ptx::ldmatrix_x4((k0 ^ (c << 4)) + tile * 16 * S::kRow, w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[4], b[4];
        fp4::unpack8(w[2 * j], a);
        fp4::unpack8(w[2 * j + 1], b);
        const uint4 qj = j ? qb : qa;
        Acc s = mma(a[0], b[0], a[1], b[1], qj.x, qj.y, Acc{});
        s = mma(a[2], b[2], a[3], b[3], qj.z, qj.w, s);
        auto scale = [&](uint32_t bytes) {
          return __uint_as_float(bytes << (23 - 8 * j) & 0x7f800000u);
        };
        x[tile][0] = f32x2::fma(s.lo, f32x2::both(scale(ks[tile][0][0])), x[tile][0]);
        x[tile][1] = f32x2::fma(s.hi, f32x2::both(scale(ks[tile][1][0])), x[tile][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      uint32_t(&w)[kChunks / 4] = ks[i >> 1][i & 1];
      if constexpr (kChunks == 8) {
        w[0] = __funnelshift_r(w[0], w[kChunks / 4 - 1], 16);
        w[kChunks / 4 - 1] >>= 16;
      } else {
        w[0] >>= 16;
      }
    }
  }
}

// A lane's scores that are not finite, or of a head with a factor so large that a scale of 2^-127
// counts, once more: K's scales come ahead of q's factors, and products may pass fp32's range
// where scores do not, so here a group's product meets the smaller of the two first.  What is not
// finite then is NaN.  x: [token][head] of the page.  (Rare, so it is short: with the matrix
// products a second time, or a call, first pages paid for its code or its registers, 252 requests
// of 103 tokens 25.0 us for 23.)
template <int D, int kTiles>
__device__ __forceinline__ void scores_far(float* x, uint32_t codes, uint32_t scales, uint32_t q,
                                           float2 qf, int item0, int lo, int hi, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int i = 0; i < 2 * kTiles; ++i) {
    const int row = item0 + 8 * i + place<D>(g);
    if (row < lo || row >= hi) continue;
    float2 y = f32x2::both(0.f);
#pragma unroll 1
    for (int c = 0; c < D / kGroup; ++c) {
      float2 s = f32x2::both(0.f);
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {          // 8 dims
        float k[8];
        fp4::unpack8(lds32(codes + run_at<D>(row, c) + 4 * u), k);
        const uint32_t at = q + (c * 32 + 8 * t + u) * 16;
        const uint4 a = lds128(at), b = lds128(at + 64);
        const uint32_t qa[4] = {a.x, a.y, a.z, a.w}, qb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&qa[j]));
          const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&qb[j]));
          s.x = fmaf(k[2 * j + 1], fa.y, fmaf(k[2 * j], fa.x, s.x));
          s.y = fmaf(k[2 * j + 1], fb.y, fmaf(k[2 * j], fb.x, s.y));
        }
      }
      const float k = fp4::scale_of(lds8(scales + row * Smem<D>::kScaleRow + c));
      y.x += fabsf(qf.x) < k ? s.x * qf.x * k : s.x * k * qf.x;   // (NaN of a NaN)
      y.y += fabsf(qf.y) < k ? s.y * qf.y * k : s.y * k * qf.y;
    }
    float2& z = *reinterpret_cast<float2*>(x + (item0 + 8 * i + g) * kMaxG + 2 * t);
    if (!(fabsf(z.x) <= FLT_MAX) || fabsf(qf.x) > kLargeFactor) z.x = y.x;
    if (!(fabsf(z.y) <= FLT_MAX) || fabsf(qf.y) > kLargeFactor) z.y = y.y;
    z = f32x2::fma(z, f32x2::both(0.f), z);
  }
}

// A page, by warp w of a team.  lo, hi: its live rows; buf: of the team's two buffers; first: in
// the segment; ok: false once a wait of this warp has run out, and of all the team's from the next
// page on (they meet at barriers without a time limit, so a warp that has given up goes on
// meeting).
template <int D>
__device__ __forceinline__ void attend(Part& part, const View& v, int stage, uint32_t q, float2 qf,
                                       int team, int w, int buf, bool first, int lo, int hi,
                                       int lane, bool& ok) {
  using S = Smem<D>;
  constexpr int kTiles = S::kOwn / 16;
  const int g = lane >> 2, t = lane & 3, item0 = w * S::kOwn;
  const uint32_t codes = v.addr + stage * 2 * S::kHalf;
  const uint32_t scales_at = v.addr + S::kScales + stage * 2 * S::kScaleHalf;
  const uint32_t vscales = scales_at + S::kScaleHalf;
  uint8_t* to = v.base + S::kP + (2 * team + buf) * S::kPBytes;
  uint8_t* factors = v.base + S::kF + (2 * team + buf) * S::kFBytes;

  float2 x[kTiles][2];      // [tile][row g | g + 8]
  Bytes<D> bytes[kTiles] = {};
  uint32_t e[kTiles];       // largest scales of those rows
  float2 p[kTiles][2], wt[kTiles][2];
  auto weigh = [&]() {
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      const float2 y = x[i >> 1][i & 1];
      float2& pi = p[i >> 1][i & 1];
      pi = make_float2(ex2(y.x - part.m[0]), ex2(y.y - part.m[1]));
      // 2^(v + kTop - rho): v is the scale's byte less 127
      const int b = i & 1 ? e[i >> 1] >> 16 : e[i >> 1] & 0xffff;
      wt[i >> 1][i & 1] = make_float2(
          pi.x * __int_as_float(__viaddmin_s32_relu(b, kTop - part.rho[0], 254) << 23),
          pi.y * __int_as_float(__viaddmin_s32_relu(b, kTop - part.rho[1], 254) << 23));
    }
  };
  auto largest = [](const float2 (&a)[kTiles][2]) {
    float y = fmaxf(a[0][0].x, a[0][0].y);
#pragma unroll
    for (int i = 1; i < 2 * kTiles; ++i)
      y = fmaxf(y, fmaxf(a[i >> 1][i & 1].x, a[i >> 1][i & 1].y));
    return y;
  };
  auto publish = [&]() {
#pragma unroll
    for (int tile = 0; tile < kTiles; ++tile) {
      uint32_t b[2][2];     // [high | low part][tokens 2t, 2t + 1 | 2t + 8, 2t + 9]
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 y = wt[tile][i];
        const __half2 h = __floats2half2_rn(y.x, y.y);
        const float2 back = __half22float2(h);
        b[0][i] = transpose8x8(as_u32(h));
        b[1][i] = transpose8x8(as_u32(__floats2half2_rn(y.x - back.x, y.y - back.y)));
      }
      const int n = w * kTiles + tile;
      *reinterpret_cast<uint4*>(to + (n * 32 + lane) * 16) =
          make_uint4(b[0][0], b[0][1], b[1][0], b[1][1]);
    }
  };
  // fp16 2^(scale - largest + kUp), 0 below 2^-14: the exponent's bits are the difference + 28
  auto factor = [&](int tile, int i) {
    return __viaddmax_s16x2(bytes[tile].b[i] + (0x00010001u * (256 + 15 + kUp) - e[tile]),
                            0xff00ff00u, 0u) << 10;
  };
  auto publish_factor = [&](int tile, int i, uint32_t f) {
    uint16_t* row = reinterpret_cast<uint16_t*>(
        factors + (Bytes<D>::kWords * t + i) * S::kFRow) + place_of(item0 + 16 * tile + g);
    row[0] = (uint16_t)f;
    row[2] = (uint16_t)(f >> 16);
  };

  scores<D, kTiles>(x, codes, scales_at, q, item0, lane);
  // Weights are fp16 pairs, and a group of dims is held to its own size as long as its
  // scales lie within 2^kSpread of the largest scale that the team has met (a weight that
  // counts for it is then at least 2^-3 and has 22 bits).  The test takes bounds that are a
  // little closer, and bytes of rows that are not live with the others.  A group that lies
  // further down does not count if it is all zeros (heads padded to 128 or 256 dims have
  // such ones in every token).
  uint32_t in = 0x80008000u, near = in;
  const int floor = max(part.most - (kSpread - 4), 0);
#pragma unroll
  for (int tile = 0; tile < kTiles; ++tile) {
    bytes[tile].load(vscales + (item0 + 16 * tile + place<D>(g)) * S::kScaleRow, t);
    e[tile] = bytes[tile].largest();
#pragma unroll
    for (int i = 0; i < Bytes<D>::kWords; ++i) {
      near &= bytes[tile].b[i] + 0x00010001u * (0x8000 - floor);
      if (!first) publish_factor(tile, i, factor(tile, i));
    }
    in &= ~(e[tile] + 0x00010001u * (0x7fff - min(part.most + 4, 254)));
  }
  auto holds_codes = [&](int tile, int k) {  // of V, group kWords t + k / 2 of row g + 8 (k % 2)
    const int row = item0 + 16 * tile + 8 * (k & 1) + place<D>(g);
    const uint4 c = lds128(codes + S::kHalf + run_at<D>(row, Bytes<D>::kWords * t + (k >> 1)));
    return ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0;
  };
  if (near != 0x80008000u) {
#pragma unroll
    for (int i = 0; i < 2 * Bytes<D>::kWords * kTiles; ++i) {
      const int tile = i / (2 * Bytes<D>::kWords), k = i % (2 * Bytes<D>::kWords);
      const uint32_t word = bytes[tile].b[k >> 1];
      if ((int)(k & 1 ? word >> 16 : word & 0xffffu) < floor && holds_codes(tile, k)) in = 0;
    }
  }
  auto live = [&](int i) {                   // tile i / 2, row g or g + 8
    const int row = item0 + 16 * (i >> 1) + 8 * (i & 1) + place<D>(g);
    return row >= lo && row < hi;
  };
  float2 sum = f32x2::both(0.f);
#pragma unroll
  for (int i = 0; i < 2 * kTiles; ++i) {
    float2& y = x[i >> 1][i & 1];
    y = f32x2::mul(y, qf);
    sum = f32x2::add(sum, y);
  }
  if (lo > item0 || hi < item0 + S::kOwn) {
    sum = f32x2::both(0.f);
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      float2& y = x[i >> 1][i & 1];
      if (live(i)) sum = f32x2::add(sum, y);
      else y = f32x2::both(-INFINITY);
    }
  }
  // K's scales came ahead of q's factors, so products may pass fp32's range where scores do
  // not; and a scale of 2^-127 was zero, which shows beside the largest factors.
  auto passes = [](float s, float f) { return !(fabsf(s) <= FLT_MAX) && f == f; };
  auto large = [](float f) { return fabsf(f) > kLargeFactor; };
  const bool again = passes(sum.x, qf.x) || passes(sum.y, qf.y);
  if (!ok && lane == 0) v.given_up[team] = 1;
  bool move = first;
  if (!first) {
    weigh();
    publish();
    move = any_in_group(2 + team, 32 * S::kTeam,
                        !ok || again || in != 0x80008000u || largest(wt) > kMostWeight ||
                            largest(p) > kMostExp);
  }
  bool wide = false;
  if (move) {
    // The references move, and scores and scales are looked at again: of live rows, scales of
    // groups that are not all zeros, without NaN.
    Meet<D>& all = reinterpret_cast<Meet<D>*>(v.base + S::kMeet)[team];
    int most = 0, least = 255;
#pragma unroll
    for (int tile = 0; tile < kTiles; ++tile) {
      uint32_t nan = 0;
#pragma unroll
      for (int k = 0; k < 2 * Bytes<D>::kWords; ++k) {
        uint32_t& word = bytes[tile].b[k >> 1];
        const uint32_t half = k & 1 ? 0xffff0000u : 0xffffu;
        const int row = item0 + 16 * tile + 8 * (k & 1) + place<D>(g);
        const int b = k & 1 ? word >> 16 : word & 0xffffu;
        if (b == fp4::kNanScale) {
          nan |= 1u << k;
          word &= ~half;
        } else if (row >= lo && row < hi) {
          if (holds_codes(tile, k)) least = min(least, b);
        }
      }
      e[tile] = bytes[tile].largest();
      bool is_live[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = item0 + 16 * tile + 8 * k + place<D>(g);
        is_live[k] = row >= lo && row < hi;
        if (is_live[k]) most = max(most, (int)(k ? e[tile] >> 16 : e[tile] & 0xffffu));
      }
#pragma unroll
      for (int i = 0; i < Bytes<D>::kWords; ++i) {
        uint32_t f = factor(tile, i);
        if (nan >> 2 * i & 1) f = (f & 0xffff0000u) | (is_live[0] ? 0x7e00u : 0u);
        if (nan >> 2 * i & 2) f = (f & 0xffffu) | (is_live[1] ? 0x7e000000u : 0u);
        publish_factor(tile, i, f);
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      all.most[w] = most;
      all.least[w] = least;
    }
    if (__builtin_expect(again || large(qf.x) || large(qf.y), 0)) {
      float2* far = reinterpret_cast<float2*>(to) + (item0 + g) * (kMaxG / 2) + t;
#pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) far[8 * i * (kMaxG / 2)] = x[i >> 1][i & 1];
      scores_far<D, kTiles>(reinterpret_cast<float*>(to), codes, scales_at, q, qf, item0, lo, hi,
                            lane);
#pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) x[i >> 1][i & 1] = far[8 * i * (kMaxG / 2)];
    }
    __syncwarp();
    // this warp's largest scores, and largest weights relative to them (NaN ignored)
    auto heads_max = [](float2 y) {
#pragma unroll
      for (int off = 4; off < 32; off *= 2) {
        y.x = fmaxf(y.x, __shfl_xor_sync(0xffffffffu, y.x, off));
        y.y = fmaxf(y.y, __shfl_xor_sync(0xffffffffu, y.y, off));
      }
      return y;
    };
    float2 top = f32x2::both(-INFINITY), up = top;
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      top.x = fmaxf(top.x, x[i >> 1][i & 1].x);
      top.y = fmaxf(top.y, x[i >> 1][i & 1].y);
    }
    top = heads_max(top);
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      const float b = (float)((int)(i & 1 ? e[i >> 1] >> 16 : e[i >> 1] & 0xffff) -
                              fp4::kScaleBias);
      up.x = fmaxf(up.x, x[i >> 1][i & 1].x - top.x + b);
      up.y = fmaxf(up.y, x[i >> 1][i & 1].y - top.y + b);
    }
    up = heads_max(up);
    if (g == 0) {
      *reinterpret_cast<float2*>(all.top[w] + 2 * t) = top;
      *reinterpret_cast<float2*>(all.up[w] + 2 * t) = up;
    }
    ptx::named_barrier(2 + team, 32 * S::kTeam);
    if (v.given_up[team]) {
      ok = false;
      return;
    }
    most = part.most < -2000 ? part.most + kAlways : part.most;
#pragma unroll
    for (int n = 0; n < S::kTeam; ++n) {
      most = max(most, all.most[n]);
      least = min(least, all.least[n]);
    }
    float m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float high = -INFINITY;
#pragma unroll
      for (int n = 0; n < S::kTeam; ++n) high = fmaxf(high, all.top[n][2 * t + h]);
      m[h] = fmaxf(part.m[h], ref_ceil(high));
      float over = -INFINITY;
#pragma unroll
      for (int n = 0; n < S::kTeam; ++n)
        over = fmaxf(over, all.top[n][2 * t + h] - m[h] + all.up[n][2 * t + h]);
      (h ? up.y : up.x) = over;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool fresh = part.m[h] == kNoRef;
      const int down = max((int)(part.m[h] - m[h]), -(1 << 20));
      const int had = fresh ? -(1 << 20) : part.rho[h] + down;
      const int need = (int)ceilf(h ? up.y : up.x);
      const int rho = max(need > had ? need + kSlack : had, kNoRho);
      const float by = ptx::pow2i(had - rho);
      part.l[h] *= fresh ? 0.f : ptx::pow2i(down);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2& o = part.o[j / 2][j % 2];
        if (h) o.y *= by;
        else o.x *= by;
      }
      part.m[h] = m[h];
      part.rho[h] = rho;
    }
    // m' bounds e 2^v, not 2^v, which may pass the range of weigh()'s factors; until the next move
    // scales are at most 2^4 above the largest.  (A head of NaN has no rho.)
    auto over = [&](int rho) { return rho != kNoRho && most + 4 + kTop - rho > 254; };
    const bool beyond = __any_sync(0xffffffffu, over(part.rho[0]) || over(part.rho[1]));
    wide = least < most - kSpread;
    const bool always = __any_sync(0xffffffffu, beyond || large(qf.x) || large(qf.y));
    part.most = always ? most - kAlways : most;
    weigh();
    if (beyond) {
      // what the factors of weigh() were cut by
#pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) {
        const int b = i & 1 ? e[i >> 1] >> 16 : e[i >> 1] & 0xffff;
        float2& y = wt[i >> 1][i & 1];
        y.x *= ptx::pow2i(min(max(b + kTop - part.rho[0] - 254, 0), 127));
        y.y *= ptx::pow2i(min(max(b + kTop - part.rho[1] - 254, 0), 127));
      }
    }
    if (wide) {
#pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) {
        const int item = item0 + 8 * i + g;
        *reinterpret_cast<float2*>(to + (item * kMaxG + 2 * t) * 4) = wt[i >> 1][i & 1];
        if (t == 0) factors[item] = (uint8_t)(i & 1 ? e[i >> 1] >> 16 : e[i >> 1]);
      }
    } else {
      publish();
    }
    ptx::named_barrier(2 + team, 32 * S::kTeam);
  }
#pragma unroll
  for (int i = 0; i < 2 * kTiles; ++i) {
    part.l[0] += p[i >> 1][i & 1].x;
    part.l[1] += p[i >> 1][i & 1].y;
  }
  // ---- products ----
  const int own = 2 * w + (g >> 2);          // this lane's group
  if (wide) {
    attend_wide<D>(part, codes + S::kHalf, vscales, reinterpret_cast<const float*>(to),
                   ptx::smem_addr(factors), own, lo, hi, lane);
    return;
  }
  const uint32_t b_at = ptx::smem_addr(to) + lane * 16,
                 f_at = ptx::smem_addr(factors) + own * S::kFRow + 16 * t;
  const uint32_t v_even = codes + S::kHalf + run_at<D>(place<D>(2 * t), own) + 4 * (g & 3),
                 v_odd = codes + S::kHalf + run_at<D>(place<D>(2 * t + 1), own) + 4 * (g & 3);
#pragma unroll
  for (int pair = 0; pair < 2; ++pair) {     // 32 tokens
    const uint4 f4 = lds128(f_at + pair * 64);
    const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
    uint32_t y[4], z[4];                     // codes of eight tokens each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = lds32(v_even + (32 * pair + 8 * i) * S::kRow);
      z[i] = lds32(v_odd + (32 * pair + 8 * i) * S::kRow);
    }
    Acc s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = Acc{};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint4 b = lds128(b_at + (2 * pair + n) * 512);
      uint32_t a[4][4];   // [byte: dims 2 byte and + 1][tokens 2t, 2t + 1 | 2t + 8, 2t + 9][dim]
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t ye = y[2 * n + i], zo = z[2 * n + i];
        uint32_t even[4], odd[4];
        fp4::unpack8((ye & 0x0f0f0f0fu) | (zo << 4 & 0xf0f0f0f0u), even);
        fp4::unpack8((ye >> 4 & 0x0f0f0f0fu) | (zo & 0xf0f0f0f0u), odd);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k][2 * i] = times(even[k], f[2 * n + i]);
          a[k][2 * i + 1] = times(odd[k], f[2 * n + i]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[k] = mma(a[k][0], a[k][1], a[k][2], a[k][3], b.z, b.w, s[k]);
        s[k] = mma(a[k][0], a[k][1], a[k][2], a[k][3], b.x, b.y, s[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      part.o[k][0] = f32x2::add(part.o[k][0], s[k].lo);
      part.o[k][1] = f32x2::add(part.o[k][1], s[k].hi);
    }
  }
}

template <int D, class P>
__device__ __forceinline__ void consumer_warp(const P& p, const View& v, int warp, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, t = lane & 3;
  const int team = warp / S::kTeam, w = warp % S::kTeam;
  int at = 0;                      // page number n of the CTA: this team's are n % kTeams == team
  int stage = team, buf = 0;
  uint32_t phase = 0, x_phase = 0;
  Ring<2> qr;
  bool ok = true;                  // no wait has run out
  for_segments(p, [&](const Segment& s, int) {
    Part part;
#pragma unroll
    for (int i = 0; i < 8; ++i) part.o[i / 2][i % 2] = make_float2(0.f, 0.f);
    part.m[0] = part.m[1] = kNoRef;
    part.l[0] = part.l[1] = 0.f;
    part.rho[0] = part.rho[1] = 0;
    part.most = -1000;
    ok = warp_wait(p, v, S::kQFull + qr.i, qr.phase, ok);
    const uint32_t q = v.addr + S::kQ + qr.i * S::kQBytes;
    const float2 qf =
        reinterpret_cast<const float2*>(v.base + S::kQFactor)[qr.i * (kMaxG / 2) + t];
    const int pages = s.hi - s.lo;
    const int first = team < at ? team - at + S::kTeams : team - at;
    int poisoned = 0;
    for (int i = first; i < pages; i += S::kTeams) {
      // Where stages are not a multiple of the teams (9 and 4), the stage's last page was another
      // team's: a wait for this load has a meaning once that page is done with (parities tell
      // two loads apart, not three).  The one before it is: the load of this team's last page
      // came after it.  Otherwise (16 and 8) this team was done with the stage's last page itself.
      if constexpr (S::kStages % S::kTeams != 0)
        ok = warp_wait(p, v, S::kEmpty + stage, phase ^ 1, ok);
      ok = warp_wait(p, v, S::kFull + stage, phase, ok);
      poisoned |= v.poison[stage];
      // the page's live tokens, from its first
      const int tok = s.first_tok + (s.lo + i) * kPage;
      attend<D>(part, v, stage, q, qf, team, w, buf, i == first, max(s.U.tok_start - tok, 0),
                min(s.U.tok_end - tok, kPage), lane, ok);
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(v.bar(S::kEmpty + stage));
      buf ^= 1;
      stage += S::kTeams;
      if (stage >= S::kStages) {
        stage -= S::kStages;
        phase ^= 1;
      }
    }
    at = (at + pages) % S::kTeams;
    if (ok && lane == 0) ptx::mbar_arrive(v.bar(S::kQEmpty + qr.i));
    qr.next();
    // ---- to the output warps ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 4; off < 32; off *= 2)
        part.l[h] += __shfl_xor_sync(0xffffffffu, part.l[h], off);
      if (poisoned) part.l[h] = __int_as_float(0x7fc00000);
    }
    ok = warp_wait(p, v, S::kXEmpty, x_phase ^ 1, ok);
    x_phase ^= 1;
    if (!ok) return true;
    if (first < pages) {
      if (g == 0) {
        float* stats = reinterpret_cast<float*>(v.base + S::kStats) + team * 2 * kMaxG + 2 * t;
        float* sums = reinterpret_cast<float*>(v.base + S::kSums) + warp * kMaxG + 2 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (w == 0) {
            stats[h] = part.m[h];
            stats[kMaxG + h] = (float)part.rho[h];
          }
          sums[h] = part.l[h];
        }
      }
      float* x = reinterpret_cast<float*>(v.base + S::kX + team * S::kXPart) +
                 (8 * w + g) * S::kXRow + 2 * t;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(x + kMaxG * i) = part.o[i / 2][i % 2];
    }
    if (lane == 0 && w == 0) v.idle[team] = first >= pages;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kXFull));
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 16 and 17: the teams' parts of a segment, added and stored.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void output_warps(const P& p, const View& v, int warp, int lane) {
  using S = Smem<D>;
  constexpr int kRounds = 2 * D / kOut;
  const int ct = warp * 32 + lane;
  uint32_t phase = 0;
  ptx::grid_dependency_wait();   // earlier kernels may still read the outputs
  // of each team the weight of its products, and two factors of the output: [teams + 2][head]
  float* factors = reinterpret_cast<float*>(v.base + S::kFactors) +
                   warp * (S::kTeams + 2) * kMaxG;
  for_segments(p, [&](const Segment& s, int) {
    const bool fail = !wait(p, v, S::kXFull, phase);
    phase ^= 1;
    if (any_in_group(1, kOut, fail)) return false;
    const size_t orow = (size_t)s.bt * p.Hq + s.g * p.G;
    uint32_t parts = 0;          // the teams that had pages
#pragma unroll
    for (int i = 0; i < S::kTeams; ++i) parts |= v.idle[i] ? 0u : 1u << i;
    float m = kNoRef, l = 0.f;   // of head `lane`
    if (lane < kMaxG) {
      const float* stats = reinterpret_cast<const float*>(v.base + S::kStats) + lane;
      const float* sums = reinterpret_cast<const float*>(v.base + S::kSums) + lane;
#pragma unroll
      for (int i = 0; i < S::kTeams; ++i)
        if (parts >> i & 1) m = fmaxf(m, stats[i * 2 * kMaxG]);
      float up = -1e6f;
#pragma unroll
      for (int i = 0; i < S::kTeams; ++i) {
        if (!(parts >> i & 1)) continue;
        const float mi = stats[i * 2 * kMaxG];
        float li = 0.f;
#pragma unroll
        for (int k = 0; k < S::kTeam; ++k) li += sums[(i * S::kTeam + k) * kMaxG];
        l = fmaf(ref_weight(mi, m), li, l);
        if (mi != kNoRef) up = fmaxf(up, mi - m + stats[(i * 2 + 1) * kMaxG]);
      }
#pragma unroll
      for (int i = 0; i < S::kTeams; ++i) {
        const float mi = stats[i * 2 * kMaxG];
        factors[i * kMaxG + lane] =
            !(parts >> i & 1) || mi == kNoRef
                ? 0.f : ref_weight(mi - m + stats[(i * 2 + 1) * kMaxG], up);
      }
      // The weighted sum of products is relative to m + up; the output, or the partial, to the
      // sum's own magnitude 2^(m + k), with l 2^-k in (2^-8, 1].  (Two factors, as the first
      // may be as large as the largest V scale.)
      const int k = l > 0.f ? ((__float_as_int(l) >> 23) - 127 + 8) >> 3 << 3 : 0;
      const int by = max(-240, min(240, (int)up - kTop - kUp - k));
      l *= ptx::pow2i(max(-126, -k));
      m += (float)k;
      const float f = ptx::pow2i(by - (by >> 1));
      factors[S::kTeams * kMaxG + lane] = ptx::pow2i(by >> 1);
      factors[(S::kTeams + 1) * kMaxG + lane] = s.whole() ? f / l : f;
      if (warp == 0 && lane < p.G && !s.whole())
        reinterpret_cast<float2*>(p.part_ml)[s.slot() * kMaxG + lane] =
            make_float2(l != l ? l : m, l);
    }
    __syncwarp();
    const int half = ct & 1, d0 = ct >> 1;   // four heads of dims d0 + 32 k
    const float4* weights = reinterpret_cast<const float4*>(factors) + half;
    float4 y[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < S::kTeams; ++i) {
      if (!(parts >> i & 1)) continue;
      const float4 a = weights[i * (kMaxG / 4)];
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int d = d0 + kOut / 2 * k;
        const float4 x = *reinterpret_cast<const float4*>(
            v.base + S::kX + i * S::kXPart + (d / 8 * S::kXRow + d % 8 * kMaxG + 4 * half) * 4);
        y[k].x = fmaf(a.x, x.x, y[k].x);
        y[k].y = fmaf(a.y, x.y, y[k].y);
        y[k].z = fmaf(a.z, x.z, y[k].z);
        y[k].w = fmaf(a.w, x.w, y[k].w);
      }
    }
    const float4 f1 = weights[S::kTeams * (kMaxG / 4)],
                 f2 = weights[(S::kTeams + 1) * (kMaxG / 4)];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kXEmpty));
    float* dst = s.whole() ? p.out + orow * D : p.part_o + s.slot() * kMaxG * D;
    float* dst2 = s.whole() && p.out2 ? p.out2 + orow * D : nullptr;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const float z[4] = {y[k].x * f1.x * f2.x, y[k].y * f1.y * f2.y, y[k].z * f1.z * f2.z,
                          y[k].w * f1.w * f2.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (4 * half + h >= p.G) break;
        dst[(4 * half + h) * D + d0 + kOut / 2 * k] = z[h];
        if (dst2) dst2[(4 * half + h) * D + d0 + kOut / 2 * k] = z[h];
      }
    }
    if (s.whole()) {
      if (warp == 0 && lane < p.G) {
        const float x = lse_of(m, l);
        p.lse[orow + lane] = x;
        if (p.lse2) p.lse2[orow + lane] = x;
      }
    } else {
      Unit U{};
      U.n_parts = s.U.n_parts;
      U.part_base = s.U.part_base;
      finish_split_unit<D, kOut>(p, v, U, s.u, 0, s.bt, s.g, s.U.first_cta, ct, warp, lane);
      ptx::named_barrier(1, kOut);   // merge_info is read before it is written again
    }
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warp 18: pages into the ring.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void tma_thread(const P& p, const View& v, const CUtensorMap* codes,
                                           const CUtensorMap* scales) {
  using S = Smem<D>;
  Ring<S::kStages> ring;
  int loads = 0;
  uint32_t marked = 0;     // stages marked as bad
  const uint64_t pol = ptx::policy_evict_first();   // every page is read once
  const int stall = blockIdx.x == 0 ? p.stall_iteration : -1;
  ptx::grid_dependency_wait();
  for_segments(p, [&](const Segment& s, int) {
    const int32_t* prow =
        p.page_table + (size_t)request_of(p, s.bt) * p.max_pages + s.U.tok_start / kPage;
    int next = __ldg(prow + s.lo);
    for (int i = s.lo; i < s.hi; ++i, ++loads) {
      int page = next;
      if (i + 1 < s.hi) next = __ldg(prow + i + 1);
      if (!wait(p, v, S::kEmpty + ring.i, ring.phase ^ 1)) return false;
      const bool bad = (uint32_t)page >= (uint64_t)p.pool_pages;
      if (bad || (marked >> ring.i & 1)) {
        // a page that is not there: page 0 in its place, its stage marked (before the arrival
        // that publishes it)
        if (bad) {
          page = 0;
          atomicOr(p.status, PA_STATUS_BAD_PAGE);
        }
        v.poison[ring.i] = bad;
        marked ^= (uint32_t)(bad != (marked >> ring.i & 1)) << ring.i;
      }
      if (loads != stall) {
        const uint32_t full = v.bar(S::kFull + ring.i);
        ptx::mbar_arrive_expect_tx(full, 2 * (S::kHalf + S::kScaleHalf));
        load_codes(v.addr + ring.i * 2 * S::kHalf, codes, s.g, page, full, pol);
        load_scales(v.addr + S::kScales + ring.i * 2 * S::kScaleHalf, scales, s.g, page, full,
                    pol);
      }
      ring.next();
    }
    return true;
  });
  // Every page of this CTA is requested: the next kernel in the stream may
  // start its prologue.
  ptx::launch_dependents();
  // The copies issued land before the CTA can exit, whatever became of the
  // other warps.
  for (int k = max(0, loads - S::kStages); k < loads; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kFull + k % S::kStages), (k / S::kStages) & 1,
                           p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Warp 19: units without pages, and q of each segment as registers of B: lane (g, t) has
// dims 8 t .. 8 t + 7 of every group of head g, as its codes of a row of K.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void helper_warp(const P& p, const View& v, int lane) {
  using S = Smem<D>;
  constexpr int kChunks = D / kGroup;
  Ring<2> ring;
  ptx::grid_dependency_wait();
  const int h = lane >> 2, t = lane & 3;
  for_segments(p, [&](const Segment& s, int) {
    uint4 raw[kChunks];
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + ((size_t)request_of(p, s.bt) * p.Hq + s.g * p.G + (h < p.G ? h : 0)) * D) + t;
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      raw[c] = h < p.G ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
    }
    most = max(most & 0xffffu, most >> 16);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    // Largest value to [2^14, 2^15), unless that takes the factor below fp32's range.  A head
    // with a NaN or an infinity becomes NaN (its scores would be).
    const int of_scale = (__float_as_int(fabsf(p.scale_log2)) >> 23) - 127;
    const int e = most ? min(14 - ((int)(most >> 7) - 127), 120 + min(of_scale, 0)) : 0;
    const float up = ptx::pow2i(e);
    const float back = most < 0x7f80u ? p.scale_log2 * ptx::pow2i(-e) : __int_as_float(0x7fc00000);
    if (!warp_wait(p, v, S::kQEmpty + ring.i, ring.phase ^ 1)) return false;
    if (t == 0) reinterpret_cast<float*>(v.base + S::kQFactor)[ring.i * kMaxG + h] = back;
    uint4* dst = reinterpret_cast<uint4*>(v.base + S::kQ + ring.i * S::kQBytes) + lane;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = as_u32(__floats2half2_rn(ptx::bf16_lo_to_f32(w[i]) * up,
                                        ptx::bf16_hi_to_f32(w[i]) * up));
      dst[32 * c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQFull + ring.i));
    ring.next();
    return true;
  });
  // Empty units: output 0, LSE -inf.
  for (int u = p.n_full + blockIdx.x; u < p.n_units; u += p.grid) {
    const DevUnit& U = p.units[u];
    const size_t row = (size_t)U.bt * p.Hq + U.g * p.G;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = lane; i < p.G * D / 4; i += 32) {
      reinterpret_cast<float4*>(p.out + row * D)[i] = zero;
      if (p.out2) reinterpret_cast<float4*>(p.out2 + row * D)[i] = zero;
    }
    if (lane < p.G) {
      p.lse[row + lane] = -INFINITY;
      if (p.lse2) p.lse2[row + lane] = -INFINITY;
    }
  }
}

template <int D, int kMaxUnits>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q4_kernel(const __grid_constant__ CUtensorMap codes,
                     const __grid_constant__ CUtensorMap scales,
                     const __grid_constant__ Params<kMaxUnits> p) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  View v;
  v.base = smem_raw + (-ptx::smem_addr(smem_raw) & 1023);   // (known to be shared memory so)
  v.addr = ptx::smem_addr(v.base);
  v.bars = v.addr + S::kBars;
  int* misc = reinterpret_cast<int*>(v.base + S::kMisc);
  v.poison = misc;
  v.abort_flag = misc + S::kStages;
  v.merge_info = misc + S::kStages + 1;
  v.given_up = misc + S::kStages + 4;
  v.idle = v.given_up + S::kTeams;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) {
      int n = 1;
      if (i >= S::kEmpty && i < S::kQFull) n = S::kTeam;
      if (i >= S::kQEmpty && i <= S::kXFull) n = kConsumers;
      if (i == S::kXEmpty) n = kOutWarps;
      ptx::mbar_init(v.bar(i), n);
    }
    *v.abort_flag = 0;
    for (int i = 0; i < S::kTeams; ++i) v.given_up[i] = 0;
    for (int i = 0; i < S::kStages; ++i) v.poison[i] = 0;
    ptx::mbar_init_fence();
  }
  if (warp == kTmaWarp && lane == 0) {
    ptx::prefetch_tensormap(&codes);
    ptx::prefetch_tensormap(&scales);
  }
  __syncthreads();
  if (warp < kConsumers) consumer_warp<D>(p, v, warp, lane);
  else if (warp < kTmaWarp) output_warps<D>(p, v, warp - kConsumers, lane);
  else if (warp == kHelperWarp) helper_warp<D>(p, v, lane);
  else if (lane == 0) tma_thread<D>(p, v, &codes, &scales);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
using Common = Params<kMaxUnitsSmall>;

// As the 8-bit kernel's where not noted.  A page costs less, and sums per CTA are fewer, so
// units are split further: at least 2 pages to a CTA (4: 900 tokens 13.3 us instead of 10.1;
// 1: 12.6), whole up to 4 (16: 15.6).  The SMs' time bounds long launches, so they are cut for
// all SMs (85%: 64 requests of up to 3,000 tokens 40.4 us, 34.9 on all); but units of one length
// still go to the next grid that divides them (144 CTAs for 16 units, 128 for 32).  The two rules
// in bytes are the 8-bit kernel's and have not been measured here.
Rules rules_of(int D) {
  const int page_bytes = 2 * (kPage * D / 2 + kPage * D / kGroup);
  Rules r;
  r.segment_charge = 2;
  r.whole_pages = 4;
  r.min_pages = 2;
  r.long_pages = 64;
  r.long_grid_pct = 100;
  r.two_parts_pages = (400 << 10) / page_bytes;
  r.whole_extra_pages = (1600 << 10) / page_bytes;
  r.unit_charge = 1;
  r.snap_pages = 2;
  return r;
}

template <int D, int N>
int launch_units(const CUtensorMap (&tmaps)[2], const Plan& plan, const Launch& L,
                 const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  using Prm = Params<N>;
  static_assert(N >= kMaxUnitsSmall && offsetof(Prm, starts) == offsetof(Common, starts), "");
  Prm prm;
  std::memcpy(static_cast<void*>(&prm), &common, offsetof(Common, starts));
  fill_units(plan, L, order, &prm);
  static PerContext smem_limit;   // the attribute lives in the context
  cudaError_t e = smem_limit.apply([] {
    return cudaFuncSetAttribute(decode_q4_kernel<D, N>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc);
  });
  if (e == cudaSuccess)
    e = launch_dependent(decode_q4_kernel<D, N>, dim3(L.grid), dim3(kThreads), Smem<D>::kAlloc,
                         stream, tmaps[0], tmaps[1], prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "4-bit paged decode launch failed: %s", cudaGetErrorString(e));
  return PA_OK;
}

int launch(int D, const CUtensorMap (&tmaps)[2], const Plan& plan, const Launch& L,
           const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  const bool small = L.n <= (size_t)kMaxUnitsSmall;
  if (D == 128)
    return small ? launch_units<128, kMaxUnitsSmall>(tmaps, plan, L, order, common, stream)
                 : launch_units<128, kMaxUnitsLarge>(tmaps, plan, L, order, common, stream);
  return small ? launch_units<256, kMaxUnitsSmall>(tmaps, plan, L, order, common, stream)
               : launch_units<256, kMaxUnitsLarge>(tmaps, plan, L, order, common, stream);
}

int run(const void* q, const void* pool, const uint8_t* scales, int64_t pool_pages,
        const int32_t* page_table, int max_pages, const int32_t* tiles, int B, int T, int Hq,
        int Hkv, int D, float scale, float* out, float* lse, float* merged_out, float* merged_lse,
        void* workspace, size_t ws_bytes, cudaStream_t stream) {
  PA_REQUIRE(B >= 0 && T >= 0, "B and T must be >= 0 (got %d, %d)", B, T);
  if ((long long)B * T == 0) return PA_OK;
  int rc = check_decode(q, pool, scales, pool_pages, (1ll << 31) / std::max(1, 2 * Hkv),
                        page_table, max_pages, tiles, B, T, Hq, Hkv, D, out, lse, merged_out,
                        merged_lse, workspace, ws_bytes);
  if (rc != PA_OK) return rc;
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  CUtensorMap tmaps[2];   // a page's K and V of a head: codes, scales
  {
    const cuuint32_t row = D / 2, heads = Hkv;
    const cuuint64_t dims[5] = {row, kPage, heads, 2, (cuuint64_t)pool_pages};
    const cuuint64_t strides[4] = {row, (cuuint64_t)row * kPage, (cuuint64_t)row * kPage * heads,
                                   (cuuint64_t)row * kPage * heads * 2};
    const cuuint32_t box[5] = {row, kPage, 1, 2, 1}, estr[5] = {1, 1, 1, 1, 1};
    CUresult r = enc(&tmaps[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(pool), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     D == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) {
      const cuuint32_t words = kPage * D / kGroup / 4;
      const cuuint64_t sdims[4] = {words, heads, 2, (cuuint64_t)pool_pages};
      const cuuint64_t sstrides[3] = {4ull * words, 4ull * words * heads, 8ull * words * heads};
      const cuuint32_t sbox[4] = {words, 1, 2, 1};
      r = enc(&tmaps[1], CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, const_cast<uint8_t*>(scales), sdims,
              sstrides, sbox, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  int sms = sm_count();
  if (sms <= 0) return fail(PA_ERR_CUDA, "cannot query the device's SM count");
  sms = std::min(sms, kMaxGrid);
  Plan plan;
  const Rules rules = rules_of(D);
  rc = plan_units(
      tiles, B, T, Hkv, rules.segment_charge, false,
      [&](const Unit* units, const int32_t* pages, size_t n, long long total,
          std::vector<int32_t>* starts) { cut(units, pages, n, total, sms, Hkv, rules, starts); },
      &plan);
  if (rc != PA_OK) return rc;

  Common common{};
  common.q = static_cast<const __nv_bfloat16*>(q);
  common.page_table = page_table;
  common.out = out;
  common.lse = lse;
  const Workspace ws(workspace, B, T, Hkv, D);
  common.status = ws.status;
  common.arrivals = ws.arrivals;
  common.part_o = ws.part_o;
  common.part_ml = ws.part_ml;
  common.pool_pages = pool_pages;
  common.max_pages = max_pages;
  common.T = T;
  common.Hq = Hq;
  common.Hkv = Hkv;
  common.G = Hq / Hkv;
  common.scale_log2 = scale * kLog2e;
  if (T == 1) {
    common.out2 = merged_out;
    common.lse2 = merged_lse;
  }
  const TestHooks hooks = take_test_hooks();
  common.wait_limit_ns = hooks.wait_limit_ns;
  common.stall_iteration = hooks.stall_iteration;
  common.slice_wait_ns = hooks.slice_wait_ns;
  for (Launch& L : plan.launches) {
    const std::vector<int> order = pack(&plan, &L, sms, rules);
    rc = launch(D, tmaps, plan, L, order, common, stream);
    if (rc != PA_OK) return rc;
  }
  if (T > 1 && merged_out != nullptr) {
    auto merge = D == 128 ? tilemerge::launch_merge<128> : tilemerge::launch_merge<256>;
    PA_CHECK_CUDA(merge(out, lse, T, Hq, B * Hq, merged_out, merged_lse, stream));
    PA_CHECK_CUDA(cudaGetLastError());
  }
  return PA_OK;
}

}  // namespace decode_q4
}  // namespace pa

extern "C" size_t paged_decode_attn_q4_workspace_bytes(int B, int T, int n_q_heads, int n_kv_heads,
                                                       int head_dim) {
  if (B < 0 || T < 0 || (head_dim != 128 && head_dim != 256) || n_kv_heads < 1 ||
      n_q_heads < n_kv_heads || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > pa::split::kMaxG)
    return 0;
  return pa::split::workspace_bytes(B, T, n_kv_heads, head_dim);
}

extern "C" int paged_decode_attn_q4_lse(const void* q, const void* pool, const uint8_t* scales,
                                        int64_t pool_pages, const int32_t* page_table,
                                        int max_pages, const int32_t* tiles, int B, int T,
                                        int n_q_heads, int n_kv_heads, int head_dim, float scale,
                                        float* out, float* lse, float* merged_out,
                                        float* merged_lse, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  pa::clear_error();
  try {
    return pa::decode_q4::run(q, pool, scales, pool_pages, page_table, max_pages, tiles, B, T,
                              n_q_heads, n_kv_heads, head_dim, scale, out, lse, merged_out,
                              merged_lse, workspace, workspace_bytes, stream);
  } catch (const std::exception& e) {
    return pa::fail(PA_ERR_INVALID, "host memory for the plan: %s", e.what());
  }
}
