// Split-KV paged GQA decode attention over a 4-bit pool (e2m1 codes, a power of two as
// the scale of each 32 values of a token's head) with a per-tile log-sum-exp, for
// sm_103a.
//
// The bytes of codes and scales bound it: (D + D / 16) bytes per token and kv head, 17/64
// of the bf16 pool's, so an SM has a quarter of the bf16 kernel's time per token.  Scales
// differ along the dims of a head, so they cannot go with the rows of a product as the
// 8-bit pool's do; codes are turned into fp16 in registers (one instruction per two) and
// both products run as mma.sync m16n8k16 with fp32 sums.
//
//  * Work split and partials: as the other decode kernels (split_units.cuh, unit_plan.h);
//    a request's tiles are merged by a kernel of its own (tile_merge.cuh).
//  * One warp streams pages with TMA: the codes of a page's K head and V head (a box each,
//    swizzled) and their scales (a bulk copy each) into a ring of stages.
//  * Eight consumer warps take half a page (32 tokens) each and never meet: two warps to
//    a page, four pages at once, each warp with a softmax of its own.
//  * S = K Q^T: 16 tokens as the rows of A, the G <= 8 heads as the columns of B, so no row
//    is idle.  A 16-byte run of a row is one scale's group; ldmatrix gives a lane 8 of its
//    values in one word, two products sum the group, and an fp32 FMA with the token's scale
//    adds it to the score.  q is scaled by a power of two per head and held in fp16: all its
//    8 bits down to 2^-32 of the head's largest.
//  * Softmax: e = 2^(x - m) for the sum, with m a multiple of 8 near the largest score; the
//    product's weight is w = e 2^(v - m') in fp16 as a high and a low part (22 bits), with 2^v
//    the token's largest V scale and m' such that w is at most 2^15 whatever the scales: a
//    weight is within 2^-23 of itself, or 2^-40 of the row's largest.  m and m' move rarely,
//    then by an exact power of two.
//  * O^T = V^T P^T: 16 dims as rows (a lane's words hold the dims of one group, two tokens'
//    codes are interleaved by nibble so that one conversion gives a register of A), tokens
//    as k, heads as columns; P comes from the scores' layout by movmatrix.  V's codes are
//    multiplied by their scale relative to the token's largest (exact).  Every 32 tokens'
//    product starts from zero and is added to fp32 registers.
//  * A segment's eight parts meet in shared memory; four output warps add and store them
//    (and merge split units) while the consumers are at the next segment.
//  * A launch starts under programmatic dependent launch; only what reads or writes global
//    memory waits for the kernels before it.  All waits have a time limit.
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
constexpr int kItem = kPage / 2;             // tokens that a warp takes at once
constexpr int kConsumers = 8, kOutWarps = 4, kOut = 32 * kOutWarps;
constexpr int kPageSlots = kConsumers / 2;   // pages at once
constexpr int kTmaWarp = kConsumers + kOutWarps, kHelperWarp = kTmaWarp + 1;
constexpr int kThreads = 32 * 16;            // (four warpgroups; the last two warps idle)
// Registers: 128 a thread at launch, moved to the consumers (256 * 160 + 256 * 96 = 65536).
constexpr int kConsumerRegs = 160, kOtherRegs = 96;
constexpr int kTop = 15;                     // log2 of the largest weight
constexpr int kUp = 13;                      // V's codes go in times 2^13: 6 * 2^13 is in range
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNoRef = -1e30f;             // m before the first score
constexpr int kNoRho = -1000;
constexpr float kMaxOver = 64.f;             // how far a score may lie above m
constexpr float kMostWeight = 65000.f;       // in fp16, which ends at 65504
constexpr int kSpread = 16;                  // see attend()

// Shared memory of a CTA; offsets from a 1024-byte boundary.
template <int D>
struct Smem {
  static constexpr int kRow = D / 2;                       // a token's codes
  static constexpr int kHalf = kPage * kRow;               // K (or V) of a page
  static constexpr int kScaleRow = D / kGroup;
  static constexpr int kScaleHalf = kPage * kScaleRow;
  static constexpr int kStages = D == 256 ? 8 : 20;
  static constexpr int kScales = kStages * 2 * kHalf;      // [stage][K | V]
  static constexpr int kQ = kScales + kStages * 2 * kScaleHalf;   // [2][group][lane] 16 bytes
  static constexpr int kQBytes = D / kGroup * 32 * 16;
  // [warp][g][dim of g][head]: a lane's g = lane / 4 has D / 8 dims; the rows are padded so
  // that the eight lay 8 banks apart
  static constexpr int kX = kQ + 2 * kQBytes;
  static constexpr int kXRow = D + 8;
  static constexpr int kXWarp = 8 * kXRow * 4;
  static constexpr int kStats = kX + kConsumers * kXWarp;  // [warp][m | rho | l][head]
  static constexpr int kQFactor = kStats + kConsumers * 3 * kMaxG * 4;    // [2][head]
  static constexpr int kFactors = kQFactor + 2 * kMaxG * 4;   // of each output warp
  static constexpr int kBars = kFactors + kOutWarps * (kConsumers + 2) * kMaxG * 4;
  static constexpr int kFull = 0, kEmpty = kFull + kStages, kQFull = kEmpty + kStages,
                       kQEmpty = kQFull + 2, kXFull = kQEmpty + 2, kXEmpty = kXFull + 1,
                       kNumBars = kXEmpty + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;       // ints, see View
  static constexpr int kUsed = kMisc + (kStages + 4) * 4;
  static constexpr int kAlloc = kUsed + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
};

template <int kMaxUnits>
struct Params {
  const __nv_bfloat16* q;
  const uint8_t* scales;
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
  static constexpr bool kInlineWaits = true;
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
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* tmap, int z,
                                         uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(z), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* src, int bytes, uint32_t bar,
                                           uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(pol)
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
// Byte i of four code words, as fp16 pairs.
template <int kByte>
__device__ __forceinline__ uint32_t unpack2(uint32_t codes) {
  uint32_t h[4];   // (the others are not made)
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h[0]) : "r"(codes));
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h[1]) : "r"(codes));
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h[2]) : "r"(codes));
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(h[3]) : "r"(codes));
  return h[kByte];
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

// ---------------------------------------------------------------------------
// Warps 0-7.
// ---------------------------------------------------------------------------
// What a lane keeps of its warp's part of a segment: for heads 2 (lane % 4) and + 1 the
// reference m, the difference rho of m' to it, its share of the sum; and the products of
// those heads with dims D / 8 * (lane / 4) ...
template <int D>
struct Part {
  static constexpr int kWords = D / 64;
  float2 o[kWords][4][2];   // [word][byte][dim of the byte]
  float m[2], l[2];
  int rho[2];
  int most;                 // largest byte of V's scales so far
};

// Scale bytes of V: the largest of rows lane / 4 (low half) and + 8 of a tile.  kSkip:
// without NaN.
template <int D, bool kSkip>
__device__ __forceinline__ uint32_t largest_scale(uint32_t row, int t) {
  using S = Smem<D>;
  uint32_t e;
  auto use = [](uint32_t b) { return kSkip && b == fp4::kNanScale ? 0u : b; };
  if constexpr (D == 256) {
    const uint32_t a = lds16(row + 2 * t), b = lds16(row + 8 * S::kScaleRow + 2 * t);
    if constexpr (kSkip)
      e = max(use(a & 255), use(a >> 8)) | max(use(b & 255), use(b >> 8)) << 16;
    else
      e = __vmaxu2(__byte_perm(a, b, 0x2420), __byte_perm(a, b, 0x2521));
  } else {
    e = use(lds8(row + t)) | use(lds8(row + 8 * S::kScaleRow + t)) << 16;
  }
  e = __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 1));
  return __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 2));
}

// The products of 32 tokens whose V scales lie far apart: in fp32, token by token, from the
// probabilities p [tile][row] of their scores.
template <int D>
__device__ __forceinline__ void attend_wide(Part<D>& part, uint32_t codes, uint32_t vscales,
                                            const float2 (&p)[2][2], int item0, int lo, int hi,
                                            int lane) {
  using S = Smem<D>;
  constexpr int kWords = Part<D>::kWords;
  const int g = lane >> 2, t = lane & 3, own = D == 256 ? g : g >> 1;
#pragma unroll 1
  for (int i = 0; i < kItem; ++i) {
    const int row = item0 + (i & ~7) + place<D>(i & 7);
    const float2 a = i & 16 ? (i & 8 ? p[1][1] : p[1][0]) : (i & 8 ? p[0][1] : p[0][0]);
    const float2 e = make_float2(__shfl_sync(0xffffffffu, a.x, 4 * (i & 7) + t),
                                 __shfl_sync(0xffffffffu, a.y, 4 * (i & 7) + t));
    if (row < lo || row >= hi) continue;
    const int b = lds8(vscales + (row - item0) * S::kScaleRow + own);
    float2 w = make_float2(
        e.x * __int_as_float(__viaddmin_s32_relu(b, kTop + kUp - part.rho[0], 254) << 23),
        e.y * __int_as_float(__viaddmin_s32_relu(b, kTop + kUp - part.rho[1], 254) << 23));
    if (b == fp4::kNanScale) w = f32x2::both(__int_as_float(0x7fc00000));
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      float y[8];
      fp4::unpack8(lds32(codes + S::kHalf + run_at<D>(row, own) + (D == 256 ? 0 : (g & 1) * 8) +
                         4 * j), y);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float2& o = part.o[j][k / 2][k % 2];
        o = f32x2::fma(w, f32x2::both(y[k]), o);
      }
    }
  }
}

// 32 tokens of a page.  lo, hi: the live ones among them.
template <int D>
__device__ __forceinline__ void attend(Part<D>& part, uint32_t codes, uint32_t scales, uint32_t q,
                                       float2 qf, int item0, int lo, int hi, int lane) {
  using S = Smem<D>;
  constexpr int kChunks = D / kGroup, kWords = Part<D>::kWords;
  const int g = lane >> 2, t = lane & 3;
  // ---- scores ----
  float2 x[2][2];   // [tile][row g | g + 8]
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i >> 1][i & 1] = make_float2(0.f, 0.f);
  {
    uint32_t ks[2][2][kChunks / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = scales + (item0 + 16 * (i >> 1) + 8 * (i & 1) + place<D>(g)) * S::kScaleRow;
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
      for (int tile = 0; tile < 2; ++tile) {
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
          const int byte = (c + j) & 3;
          auto scale = [&](uint32_t bytes) {
            return __uint_as_float((byte == 3 ? bytes >> 1 : bytes << (23 - 8 * byte)) & 0x7f800000u);
          };
          x[tile][0] = f32x2::fma(s.lo, f32x2::both(scale(ks[tile][0][(c + j) / 4])), x[tile][0]);
          x[tile][1] = f32x2::fma(s.hi, f32x2::both(scale(ks[tile][1][(c + j) / 4])), x[tile][1]);
        }
      }
    }
  }
  // ---- V's scales ----
  const uint32_t vscales = scales + S::kScaleHalf + item0 * S::kScaleRow;
  uint32_t e[2];
#pragma unroll
  for (int tile = 0; tile < 2; ++tile)
    e[tile] = largest_scale<D, false>(vscales + (16 * tile + place<D>(g)) * S::kScaleRow, t);
  const int own = D == 256 ? g : g >> 1;   // this lane's group
  uint32_t vs[2][2];                       // scales of tokens 2t, 2t + 1 | 2t + 8, 2t + 9 of it
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = vscales + (16 * (i >> 1) + 8 * (i & 1)) * S::kScaleRow + own;
    vs[i >> 1][i & 1] = lds8(a + place<D>(2 * t) * S::kScaleRow) |
                        lds8(a + place<D>(2 * t + 1) * S::kScaleRow) << 16;
  }
  // Weights are fp16 pairs, and a group of dims is held to its own size as long as its
  // scales lie within 2^kSpread of the largest scale that the warp has met (a weight that
  // counts for it is then at least 2^-3 and has 22 bits).  The test takes bounds that are a
  // little closer, and bytes of rows that are not live with the others.
  const uint32_t over = __vmaxu2(e[0], e[1]) + 0x00010001u * (0x7fff - min(part.most + 4, 254));
  const uint32_t above = __vminu2(__vminu2(vs[0][0], vs[0][1]), __vminu2(vs[1][0], vs[1][1])) +
                         0x00010001u * (0x8000 - max(part.most - (kSpread - 4), 0));
  const bool odd = __any_sync(0xffffffffu, (over | ~above) & 0x80008000u);
  bool wide = false;
  if (odd) {
    // Look again, at live rows and groups that are not all zeros, without NaN.
    int most = 0, least = 255;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tile = i >> 1, tok = item0 + 16 * tile + 8 * (i & 1);
      if (!(i & 1))
        e[tile] = largest_scale<D, true>(vscales + (16 * tile + place<D>(g)) * S::kScaleRow, t);
      if (tok + place<D>(g) >= lo && tok + place<D>(g) < hi)
        most = max(most, (int)(i & 1 ? e[tile] >> 16 : e[tile] & 0xffff));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = tok + place<D>(2 * t + k), b = vs[tile][i & 1] >> 16 * k & 255;
        const uint32_t a = codes + S::kHalf + run_at<D>(row, own) + (D == 256 ? 0 : (g & 1) * 8);
        uint2 w = lds64(a);
        if constexpr (D == 256) {
          const uint2 w2 = lds64(a + 8);
          w.x |= w2.x | w2.y;
        }
        const bool counts = row >= lo && row < hi && ((w.x | w.y) & 0x77777777u) != 0;
        if (counts && b != fp4::kNanScale) least = min(least, b);
      }
    }
    part.most = max(part.most, __reduce_max_sync(0xffffffffu, most));
    wide = __reduce_min_sync(0xffffffffu, least) < part.most - kSpread;
  }
#pragma unroll
  for (int tile = 0; tile < 2; ++tile) {
    // 28 + 256 - e of tokens 2t and 2t + 8, 2t + 1 and 2t + 9
    const uint32_t under = 0x011c011cu - e[tile];
    const uint32_t n0 = __shfl_sync(0xffffffffu, under, 8 * t);
    const uint32_t n1 = __shfl_sync(0xffffffffu, under, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t sum = vs[tile][i] + __byte_perm(n0, n1, i ? 0x7632 : 0x5410);
      // fp16 2^(scale - e + kUp), 0 below 2^-14
      uint32_t f = __viaddmax_s16x2(sum, 0xff00ff00u, 0u) << 10;
      if (odd) {   // NaN, where the row is live
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if ((vs[tile][i] >> 16 * k & 255) != fp4::kNanScale) continue;
          const int tok = item0 + 16 * tile + 8 * i + place<D>(2 * t + k);
          f = (f & (k ? 0xffffu : 0xffff0000u)) | (tok >= lo && tok < hi ? 0x7e00u << 16 * k : 0u);
        }
      }
      vs[tile][i] = f;
    }
  }
  // ---- softmax ----
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2& y = x[i >> 1][i & 1];
    y = f32x2::mul(y, qf);
    y = f32x2::fma(y, f32x2::both(0.f), y);   // an infinite score is NaN
  }
  if (lo > item0 || hi < item0 + kItem) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = item0 + 16 * (i >> 1) + 8 * (i & 1) + place<D>(g);
      if (tok < lo || tok >= hi) x[i >> 1][i & 1] = f32x2::both(-INFINITY);
    }
  }
  float2 p[2][2], w[2][2];
  auto weigh = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = x[i >> 1][i & 1];
      float2& pi = p[i >> 1][i & 1];
      pi = make_float2(ptx::ex2(y.x - part.m[0]), ptx::ex2(y.y - part.m[1]));
      // 2^(v + kTop - rho): v is the scale's byte less 127
      const int v = i & 1 ? e[i >> 1] >> 16 : e[i >> 1] & 0xffff;
      w[i >> 1][i & 1] = make_float2(
          pi.x * __int_as_float(__viaddmin_s32_relu(v, kTop - part.rho[0], 254) << 23),
          pi.y * __int_as_float(__viaddmin_s32_relu(v, kTop - part.rho[1], 254) << 23));
    }
  };
  weigh();
  {
    auto most = [](const float2 (&a)[2][2]) {
      return fmaxf(fmaxf(fmaxf(a[0][0].x, a[0][0].y), fmaxf(a[0][1].x, a[0][1].y)),
                   fmaxf(fmaxf(a[1][0].x, a[1][0].y), fmaxf(a[1][1].x, a[1][1].y)));
    };
    const bool above = most(w) > kMostWeight || most(p) > ptx::pow2i((int)kMaxOver);
    if (__any_sync(0xffffffffu, above)) {
      // The references move.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY, up = -INFINITY;   // (NaN ignored)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, h ? x[i >> 1][i & 1].y : x[i >> 1][i & 1].x);
#pragma unroll
        for (int off = 4; off < 32; off *= 2)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float m = fmaxf(part.m[h], ref_ceil(top));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = (int)(i & 1 ? e[i >> 1] >> 16 : e[i >> 1] & 0xffff) - fp4::kScaleBias;
          up = fmaxf(up, (h ? x[i >> 1][i & 1].y : x[i >> 1][i & 1].x) - m + (float)v);
        }
#pragma unroll
        for (int off = 4; off < 32; off *= 2)
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, off));
        const bool fresh = part.m[h] == kNoRef;
        const int had = fresh ? -(1 << 20)
                              : part.rho[h] + max((int)(part.m[h] - m), -(1 << 20));
        const int rho = max(max(had, (int)ceilf(up)), kNoRho);
        const float by = ptx::pow2i(had - rho);
        part.l[h] *= fresh ? 0.f : ptx::pow2i(max((int)(part.m[h] - m), -(1 << 20)));
#pragma unroll
        for (int j = 0; j < kWords * 8; ++j) {
          float2& o = part.o[j / 8][j / 2 % 4][j % 2];
          if (h) o.y *= by;
          else o.x *= by;
        }
        part.m[h] = m;
        part.rho[h] = rho;
      }
      weigh();
    }
  }
  part.l[0] += (p[0][0].x + p[0][1].x) + (p[1][0].x + p[1][1].x);
  part.l[1] += (p[0][0].y + p[0][1].y) + (p[1][0].y + p[1][1].y);
  if (wide) {
    attend_wide<D>(part, codes, vscales, p, item0, lo, hi, lane);
    return;
  }
  uint32_t ph[2][2], pl[2][2];   // B's registers: [tile][tokens 2t, 2t + 1 | 2t + 8, 2t + 9]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = w[i >> 1][i & 1];
    const __half2 h = __floats2half2_rn(y.x, y.y);
    const float2 back = __half22float2(h);
    ph[i >> 1][i & 1] = transpose8x8(as_u32(h));
    pl[i >> 1][i & 1] = transpose8x8(as_u32(__floats2half2_rn(y.x - back.x, y.y - back.y)));
  }
  // ---- products ----
#pragma unroll
  for (int tile = 0; tile < 2; ++tile) {
    uint32_t v[4][kWords];   // of tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = codes + S::kHalf + run_at<D>(item0 + place<D>(2 * t + (i & 1)), own) +
                         (16 * tile + 8 * (i >> 1)) * S::kRow + (D == 256 ? 0 : (g & 1) * 8);
      if constexpr (D == 256) {
        const uint4 y = lds128(a);
        v[i][0] = y.x;
        v[i][1] = y.y;
        v[i][kWords - 2] = y.z;
        v[i][kWords - 1] = y.w;
      } else {
        const uint2 y = lds64(a);
        v[i][0] = y.x;
        v[i][1] = y.y;
      }
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      uint32_t c[4];   // even | odd dims of tokens 2t and 2t + 1, of 2t + 8 and 2t + 9
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a = v[2 * i][j], b = v[2 * i + 1][j];
        c[2 * i] = (a & 0x0f0f0f0fu) | (b << 4 & 0xf0f0f0f0u);
        c[2 * i + 1] = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
      }
      auto byte = [&](auto unpack, float2 (&o)[2]) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = times(unpack(c[i]), vs[tile][i >> 1]);
        Acc s = mma(a[0], a[1], a[2], a[3], pl[tile][0], pl[tile][1], Acc{});
        s = mma(a[0], a[1], a[2], a[3], ph[tile][0], ph[tile][1], s);
        o[0] = f32x2::add(o[0], s.lo);
        o[1] = f32x2::add(o[1], s.hi);
      };
      byte([](uint32_t y) { return unpack2<0>(y); }, part.o[j][0]);
      byte([](uint32_t y) { return unpack2<1>(y); }, part.o[j][1]);
      byte([](uint32_t y) { return unpack2<2>(y); }, part.o[j][2]);
      byte([](uint32_t y) { return unpack2<3>(y); }, part.o[j][3]);
    }
  }
}

template <int D, class P>
__device__ __forceinline__ void consumer_warp(const P& p, const View& v, int warp, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, t = lane & 3;
  const int slot = warp >> 1, item0 = (warp & 1) * kItem;
  int at = 0;                      // page number n of the CTA: this warp's are n % 4 == slot
  int stage = slot;
  uint32_t phase = 0, x_phase = 0;
  Ring<2> qr;
  for_segments(p, [&](const Segment& s, int) {
    Part<D> part;
#pragma unroll
    for (int i = 0; i < Part<D>::kWords * 8; ++i)
      part.o[i / 8][i / 2 % 4][i % 2] = make_float2(0.f, 0.f);
    part.m[0] = part.m[1] = kNoRef;
    part.l[0] = part.l[1] = 0.f;
    part.rho[0] = part.rho[1] = 0;
    part.most = -1000;
    if (!warp_wait(p, v, S::kQFull + qr.i, qr.phase)) return false;
    const uint32_t q = v.addr + S::kQ + qr.i * S::kQBytes;
    const float2 qf =
        reinterpret_cast<const float2*>(v.base + S::kQFactor)[qr.i * (kMaxG / 2) + t];
    const int pages = s.hi - s.lo;
    int poisoned = 0;
    for (int i = (slot - at) & (kPageSlots - 1); i < pages; i += kPageSlots) {
      if (!warp_wait(p, v, S::kFull + stage, phase)) return false;
      poisoned |= v.poison[stage];
      // the page's live tokens, from its first
      const int tok = s.first_tok + (s.lo + i) * kPage;
      const int lo = max(s.U.tok_start - tok, 0), hi = min(s.U.tok_end - tok, kPage);
      if (lo < item0 + kItem && hi > item0)
        attend<D>(part, v.addr + stage * 2 * S::kHalf,
                  v.addr + S::kScales + stage * 2 * S::kScaleHalf, q, qf, item0, lo, hi, lane);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(v.bar(S::kEmpty + stage));
      stage += kPageSlots;
      if (stage >= S::kStages) {
        stage -= S::kStages;
        phase ^= 1;
      }
    }
    at = (at + pages) & (kPageSlots - 1);
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQEmpty + qr.i));
    qr.next();
    // ---- to the output warps ----
    if (!warp_wait(p, v, S::kXEmpty, x_phase ^ 1)) return false;
    x_phase ^= 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 4; off < 32; off *= 2)
        part.l[h] += __shfl_xor_sync(0xffffffffu, part.l[h], off);
      if (poisoned) part.l[h] = __int_as_float(0x7fc00000);
      float* stats = reinterpret_cast<float*>(v.base + S::kStats) + warp * 3 * kMaxG + 2 * t + h;
      if (g == 0) {
        stats[0] = part.m[h];
        stats[kMaxG] = (float)part.rho[h];
        stats[2 * kMaxG] = part.l[h];
      }
    }
    float* x = reinterpret_cast<float*>(v.base + S::kX + warp * S::kXWarp) + g * S::kXRow + 2 * t;
#pragma unroll
    for (int i = 0; i < Part<D>::kWords * 8; ++i)
      *reinterpret_cast<float2*>(x + 8 * i) = part.o[i / 8][i / 2 % 4][i % 2];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kXFull));
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 8-11: a segment's eight parts, added and stored.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void output_warps(const P& p, const View& v, int warp, int lane) {
  using S = Smem<D>;
  constexpr int kRounds = D / 64;
  const int ct = warp * 32 + lane;
  uint32_t phase = 0;
  ptx::grid_dependency_wait();   // earlier kernels may still read the outputs
  // of each consumer warp the weight of its products, and two factors of the output: [8 + 2][head]
  float* factors = reinterpret_cast<float*>(v.base + S::kFactors) +
                   warp * (kConsumers + 2) * kMaxG;
  for_segments(p, [&](const Segment& s, int) {
    const bool fail = !wait(p, v, S::kXFull, phase);
    phase ^= 1;
    if (any_in_group(1, kOut, fail)) return false;
    const size_t orow = (size_t)s.bt * p.Hq + s.g * p.G;
    float m = kNoRef, l = 0.f;   // of head `lane`
    if (lane < kMaxG) {
      const float* stats = reinterpret_cast<const float*>(v.base + S::kStats) + lane;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) m = fmaxf(m, stats[i * 3 * kMaxG]);
      float up = -1e6f;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) {
        const float mi = stats[i * 3 * kMaxG];
        l = fmaf(ref_weight(mi, m), stats[(i * 3 + 2) * kMaxG], l);
        if (mi != kNoRef) up = fmaxf(up, mi - m + stats[(i * 3 + 1) * kMaxG]);
      }
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) {
        const float mi = stats[i * 3 * kMaxG];
        factors[i * kMaxG + lane] =
            mi == kNoRef ? 0.f : ref_weight(mi - m + stats[(i * 3 + 1) * kMaxG], up);
      }
      // The weighted sum of products is relative to m + up; the output, or the partial, to the
      // sum's own magnitude 2^(m + k), with l 2^-k in (2^-8, 1].  (Two factors, as the first
      // may be as large as the largest V scale.)
      const int k = l > 0.f ? ((__float_as_int(l) >> 23) - 127 + 8) >> 3 << 3 : 0;
      const int by = max(-240, min(240, (int)up - kTop - kUp - k));
      l *= ptx::pow2i(max(-126, -k));
      m += (float)k;
      const float f = ptx::pow2i(by - (by >> 1));
      factors[kConsumers * kMaxG + lane] = ptx::pow2i(by >> 1);
      factors[(kConsumers + 1) * kMaxG + lane] = s.whole() ? f / l : f;
      if (warp == 0 && lane < p.G && !s.whole())
        reinterpret_cast<float2*>(p.part_ml)[s.slot() * kMaxG + lane] =
            make_float2(l != l ? l : m, l);
    }
    __syncwarp();
    const int half = ct & 1, d0 = ct >> 1;   // four heads of dims d0 + 64 k
    const float4* weights = reinterpret_cast<const float4*>(factors) + half;
    float4 y[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kConsumers; ++i) {
      const float4 a = weights[i * (kMaxG / 4)];
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int d = d0 + 64 * k;
        const float4 x = *reinterpret_cast<const float4*>(
            v.base + S::kX + i * S::kXWarp +
            (d / (D / 8) * S::kXRow + d % (D / 8) * kMaxG + 4 * half) * 4);
        y[k].x = fmaf(a.x, x.x, y[k].x);
        y[k].y = fmaf(a.y, x.y, y[k].y);
        y[k].z = fmaf(a.z, x.z, y[k].z);
        y[k].w = fmaf(a.w, x.w, y[k].w);
      }
    }
    const float4 f1 = weights[kConsumers * (kMaxG / 4)], f2 = weights[(kConsumers + 1) * (kMaxG / 4)];
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
        dst[(4 * half + h) * D + d0 + 64 * k] = z[h];
        if (dst2) dst2[(4 * half + h) * D + d0 + 64 * k] = z[h];
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
// Warp 12: pages into the ring.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void tma_warp(const P& p, const View& v, const CUtensorMap* tmap,
                                         int lane) {
  using S = Smem<D>;
  Ring<S::kStages> ring;
  int loads = 0;
  const uint64_t pol = ptx::policy_evict_first();   // every page is read once
  const int stall = blockIdx.x == 0 && p.stall_iteration >= 0
                        ? p.stall_iteration & ~(int)PA_STALL_VALUES : -1;
  const int heads = 2 * p.Hkv;
  ptx::grid_dependency_wait();
  for_segments(p, [&](const Segment& s, int) {
    const int32_t* prow =
        p.page_table + (size_t)request_of(p, s.bt) * p.max_pages + s.U.tok_start / kPage;
    int next_pid = s.lo + lane < s.hi ? __ldg(prow + s.lo + lane) : 0;
    for (int base = s.lo; base < s.hi; base += 32) {
      const int cnt = min(32, s.hi - base);
      // a page that is not there: page 0 in its place, its stage marked
      const bool bad = lane < cnt && (uint32_t)next_pid >= (uint64_t)p.pool_pages;
      const uint32_t bad_pages = __ballot_sync(0xffffffffu, bad);
      const int my_pid = bad ? 0 : next_pid;
      if (bad) atomicOr(p.status, PA_STATUS_BAD_PAGE);
      if (base + 32 + lane < s.hi) next_pid = __ldg(prow + base + 32 + lane);
      for (int j = 0; j < cnt; ++j, ++loads) {
        const int z = __shfl_sync(0xffffffffu, my_pid, j) * heads + s.g;
        if (!warp_wait(p, v, S::kEmpty + ring.i, ring.phase ^ 1)) return false;
        if (loads != stall && elect()) {
          const uint32_t full = v.bar(S::kFull + ring.i);
          v.poison[ring.i] = bad_pages >> j & 1;   // set before the arrival that publishes it
          ptx::mbar_arrive_expect_tx(full, 2 * (S::kHalf + S::kScaleHalf));
          const uint32_t codes = v.addr + ring.i * 2 * S::kHalf;
          const uint32_t scales = v.addr + S::kScales + ring.i * 2 * S::kScaleHalf;
          load_box(codes, tmap, z, full, pol);
          load_bytes(scales, p.scales + (size_t)z * S::kScaleHalf, S::kScaleHalf, full, pol);
          load_box(codes + S::kHalf, tmap, z + p.Hkv, full, pol);
          load_bytes(scales + S::kScaleHalf, p.scales + (size_t)(z + p.Hkv) * S::kScaleHalf,
                     S::kScaleHalf, full, pol);
        }
        __syncwarp();
        ring.next();
      }
    }
    return true;
  });
  // Every page of this CTA is requested: the next kernel in the stream may
  // start its prologue.
  if (lane == 0) ptx::launch_dependents();
  // The copies issued land before the CTA can exit, whatever became of the
  // other warps.
  for (int k = max(0, loads - S::kStages); k < loads; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kFull + k % S::kStages), (k / S::kStages) & 1,
                           p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Warp 13: units without pages, and q of each segment as registers of B: lane (g, t) has
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
    // Largest value to [2^14, 2^15).  A head with a NaN or an infinity becomes NaN (its
    // scores would be).
    const int e = most ? min(14 - ((int)(most >> 7) - 127), 120) : 0;
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
    decode_q4_kernel(const __grid_constant__ CUtensorMap tmap,
                     const __grid_constant__ Params<kMaxUnits> p) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  View v;
  v.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  v.addr = ptx::smem_addr(v.base);
  v.bars = v.addr + S::kBars;
  int* misc = reinterpret_cast<int*>(v.base + S::kMisc);
  v.poison = misc;
  v.abort_flag = misc + S::kStages;
  v.merge_info = misc + S::kStages + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) {
      int n = 1;
      if (i >= S::kEmpty && i < S::kQFull) n = 2;             // a page's two warps
      if (i >= S::kQEmpty && i <= S::kXFull) n = kConsumers;
      if (i == S::kXEmpty) n = kOutWarps;
      ptx::mbar_init(v.bar(i), n);
    }
    *v.abort_flag = 0;
    ptx::mbar_init_fence();
  }
  if (warp == kTmaWarp && lane == 0) ptx::prefetch_tensormap(&tmap);
  __syncthreads();
  if (warp < kConsumers) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    consumer_warp<D>(p, v, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kTmaWarp) output_warps<D>(p, v, warp - kConsumers, lane);
    else if (warp == kTmaWarp) tma_warp<D>(p, v, &tmap, lane);
    else if (warp == kHelperWarp) helper_warp<D>(p, v, lane);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
using Common = Params<kMaxUnitsSmall>;

Rules rules_of(int D) {
  const int page_bytes = 2 * (kPage * D / 2 + kPage * D / kGroup);
  return {6, 16, 4, 64, 85, (400 << 10) / page_bytes, (1600 << 10) / page_bytes, 3, 4};
}

template <int D, int N>
int launch_units(const CUtensorMap& tmap, const Plan& plan, const Launch& L,
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
                         stream, tmap, prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "4-bit paged decode launch failed: %s", cudaGetErrorString(e));
  return PA_OK;
}

int launch(int D, const CUtensorMap& tmap, const Plan& plan, const Launch& L,
           const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  const bool small = L.n <= (size_t)kMaxUnitsSmall;
  if (D == 128)
    return small ? launch_units<128, kMaxUnitsSmall>(tmap, plan, L, order, common, stream)
                 : launch_units<128, kMaxUnitsLarge>(tmap, plan, L, order, common, stream);
  return small ? launch_units<256, kMaxUnitsSmall>(tmap, plan, L, order, common, stream)
               : launch_units<256, kMaxUnitsLarge>(tmap, plan, L, order, common, stream);
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
  CUtensorMap tmap;
  {
    const cuuint32_t row = D / 2;
    const cuuint64_t dims[3] = {row, kPage, (cuuint64_t)pool_pages * 2 * Hkv};
    const cuuint64_t strides[2] = {row, (cuuint64_t)row * kPage};
    const cuuint32_t box[3] = {row, kPage, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(&tmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           D == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
  common.scales = scales;
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
    rc = launch(D, tmap, plan, L, order, common, stream);
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
