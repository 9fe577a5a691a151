// Split-KV paged GQA decode attention over a 4-bit pool (e2m1 codes, a power of two as
// the scale of each 32 values of a token's head) with a per-tile log-sum-exp, for
// sm_103a.
//
// The bytes of codes and scales bound it: (D + D / 16) bytes per token and kv head, 17/64
// of the bf16 pool's, so an SM has a quarter of the bf16 kernel's time per token, and the
// instructions per value decide.  No thread converts a code of K, and one of V takes two
// thirds of an instruction of one lane:
//
//  * Work split and partials: as the other decode kernels (split_units.cuh, unit_plan.h);
//    a request's tiles are merged by a kernel of its own (tile_merge.cuh).  A CTA streams its
//    pages two at a time: a step is 128 tokens of one kv head.
//  * S = K Q^T on the fifth-generation tensor cores with block scales: M = 128 tokens, N = 32,
//    K = D.  TMA unpacks the codes to the bytes that the product takes, a token's scales go to
//    tensor memory beside them (one byte per 32 dims, the pool's own groups), and q is held
//    as four e4m3 parts (q_parts.cuh) with scales of one.
//  * Softmax: a thread per token, four warps.  e = 2^(x - m) for the sum, with m a multiple of
//    8 near a head's largest score; the product's weight is w = e 2^(v - m'), 2^v the token's
//    largest V scale, in fp16 as a high and a low part (22 bits), with m' such that w is below
//    2^15 whatever the scales: a weight is within 2^-23 of itself, or 2^-40 of the row's
//    largest.  m and m' move rarely, then by an exact power of two.
//  * O^T = V^T P^T as mma.sync m16n8k16 in fp16 (V's scales differ along its rows, which no
//    product on the fifth-generation tensor cores takes): a warp has one group of 32 dims, so
//    its scales (relative to the token's largest) are factors of P, two heads of four dims per
//    lane are all that it keeps, and no sums meet at a segment's end.  ldmatrix transposes
//    four codes at a time; two tokens' codes are interleaved by nibble so that one conversion
//    gives a register of A.  Every 32 tokens' product starts from zero and is added to fp32
//    registers.
//  * Warps: 0-7 products, 8-11 softmax, one each for TMA, scores, K's scales and what is done
//    once per segment.  All waits are on mbarriers with a time limit; S, its scales and P have
//    two buffers each, K and V rings of their own.
//  * A launch starts under programmatic dependent launch; only what reads or writes global
//    memory waits for the kernels before it.
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
#include "q_parts.cuh"
#include "split_units.cuh"
#include "tc.cuh"
#include "tile_merge.cuh"
#include "unit_plan.h"
#include "unit_walk.cuh"

namespace pa {
namespace decode_q4 {

using namespace split;

constexpr int kGroup = PA_Q4_GROUP;
constexpr int kStep = 2 * kPage;             // tokens per step
constexpr int kValueWarps = 8, kValues = 32 * kValueWarps;
constexpr int kScoreWarps = 4, kScores = 32 * kScoreWarps;
constexpr int kScoreWarp = kValueWarps, kTmaWarp = kScoreWarp + kScoreWarps,
              kMmaWarp = kTmaWarp + 1, kScaleWarp = kMmaWarp + 1, kHelperWarp = kScaleWarp + 1;
constexpr int kThreads = 32 * (kHelperWarp + 1);
constexpr int kTop = 14;                     // log2 of the largest weight
constexpr int kUp = 1;                       // it goes in times 2 and its scale's factor
constexpr float kMostWeight = 32500.f;       // twice that is in fp16, which ends at 65504
// How far V scales may lie below the largest that the CTA has met in the segment (log2):
// factors are normal fp16 numbers then.
constexpr int kSpread = 15;
constexpr int kTiny = fp4::kScaleBias + fp4::kMinScaleExp;   // the smallest scale written
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNoRef = -1e30f;             // m before the first score
constexpr int kNoRho = -1000;
constexpr float kMostExp = 0x1p64f;          // e may lie above 1, up to this
constexpr int kTmemCols = 128, kSfCols = 2 * kQCols, kOnesCols = kSfCols + 2 * 8;

static_assert(kStep == kScores && kScoreWarp % 4 == 0, "a thread per token");

// A step's weights, from the softmax warps to the product warps.
template <int D>
struct alignas(16) Weights {
  // fp16 high and low parts, [part][token][head]; where V's scales lie far apart (kWide) the
  // probabilities in fp32, [token][head]
  union {
    __half parts[2][kStep][kMaxG];
    float p[kStep][kMaxG];
  };
  // [group][place_of(token)]: what a group's scale gives P, in fp16; with kWide its byte
  uint16_t factor[D / kGroup][kStep];
  float by[kMaxG];         // what the products so far are multiplied by, with kMoved
  int top[kMaxG];          // kTop - rho, see State
  int flags;
};
constexpr int kMoved = 1, kWide = 2;
// Tokens of 32 are ordered so that 16 bytes hold the eight that lane t of four has in two
// products: t's 2t, 2t + 1, 2t + 8, 2t + 9 of both.
__device__ __forceinline__ int place_of(int tok) {
  return (tok & ~31) | (tok >> 1 & 3) << 3 | (tok >> 4 & 1) << 2 | (tok >> 3 & 1) << 1 | (tok & 1);
}

// The softmax warps' references, per head: m; kTop - rho with rho = m' - m; what a sum so
// far, and products so far, are multiplied by at a move.
struct State {
  float m[kMaxG];
  int top[kMaxG];
  float down[kMaxG], by[kMaxG];
  // of each warp, for a move: largest score, largest v over m, largest scale
  float warp_top[kScoreWarps][kMaxG], warp_up[kScoreWarps][kMaxG];
  int warp_most[kScoreWarps];
  float sums[kScoreWarps][kMaxG];   // of a segment
};

// Shared memory of a CTA; offsets from a 1024-byte boundary.
template <int D>
struct Smem {
  static constexpr int kChunks = D / kChunk;
  static constexpr int kPageBytes = kPage * kChunk;        // one page and chunk of K, a byte a code
  static constexpr int kChunkBytes = 2 * kPageBytes;
  static constexpr int kKBytes = kChunks * kChunkBytes;    // of a step
  static constexpr int kRow = D / 2;                       // a token's codes of V, as they are
  static constexpr int kVPage = kPage * kRow;
  static constexpr int kVBytes = 2 * kVPage;
  static constexpr int kScaleRow = D / kGroup;
  static constexpr int kScalePage = kPage * kScaleRow;
  static constexpr int kScaleBytes = 4 * kScalePage;       // of a step: [page][K | V]
  static constexpr int kKStages = D == 256 ? 3 : 6;
  static constexpr int kVStages = D == 256 ? 5 : 10;
  static constexpr int kV = kKStages * kKBytes;
  static constexpr int kQ = kV + kVStages * kVBytes;       // [2]
  static constexpr int kQChunkBytes = kQCols * kChunk;
  static constexpr int kQBytes = kChunks * kQChunkBytes;
  static constexpr int kScales = kQ + 2 * kQBytes;         // [K stage]
  static constexpr int kSf = kScales + kKStages * kScaleBytes;   // [2][chunk][512]
  static constexpr int kOnes = kSf + 2 * kChunks * 512;
  static constexpr int kP = kOnes + 512;                   // Weights [2]
  static constexpr int kQRaw = kP + 2 * sizeof(Weights<D>);   // [head][dim] of a later segment
  static constexpr int kX = kQRaw + kMaxG * D * 2;         // D = 128: [warp][lane][8]
  static constexpr int kState = kX + (D == 128 ? kValues / 2 * 32 : 0);
  static constexpr int kQScale = kState + sizeof(State);   // [2][head]
  static constexpr int kQs = kQScale + 2 * kMaxG * 4;      // a softmax warp's copy: [warp][head]
  static constexpr int kFactor = kQs + kScoreWarps * kMaxG * 4;   // [2][two factors][head]
  static constexpr int kBars = (kFactor + 2 * 2 * kMaxG * 4 + 7) / 8 * 8;
  static constexpr int kKFull = 0, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages,
                       kVEmpty = kVFull + kVStages, kSfFull = kVEmpty + kVStages,
                       kSfEmpty = kSfFull + 2, kSFull = kSfEmpty + 2, kSEmpty = kSFull + 2,
                       kPFull = kSEmpty + 2, kPEmpty = kPFull + 2, kQFull = kPEmpty + 2,
                       kQEmpty = kQFull + 2, kLFull = kQEmpty + 2, kLEmpty = kLFull + 2,
                       kDrain = kLEmpty + 2, kNumBars = kDrain + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;       // ints, see View
  static constexpr int kUsed = kMisc + (kKStages + 4) * 4;
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
  static constexpr bool kInlineWaits = false;
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
  volatile int* poison;   // [K stages] the step holds a page that is not there
  volatile int* abort_flag;
  volatile int* merge_info;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* tmap, int x, int z,
                                         uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(0), "r"(z), "r"(bar), "l"(pol)
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
               : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float warp_max(float x) {   // (NaN ignored)
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
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

__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {   // fp16 pairs
  return as_u32(__hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y)));
}

// Where group c of row r lies in a page's codes of V (the copies' swizzle).
template <int D>
__device__ __forceinline__ int run_at(int r, int c) {
  return r * Smem<D>::kRow + ((c ^ (D == 256 ? r & 7 : r >> 1 & 3)) << 4);
}

// ---------------------------------------------------------------------------
// Warp 12: the pages' K (with both scales) and V into their rings.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void tma_warp(const P& p, const View& v, const CUtensorMap* keys,
                                         const CUtensorMap* values, int lane) {
  using S = Smem<D>;
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  int keys_loaded = 0, values_loaded = 0;   // steps
  const uint64_t pol = ptx::policy_evict_first();   // every page is read once
  const int stall = blockIdx.x == 0 ? p.stall_iteration : -1;
  const int stall_values = stall - (int)PA_STALL_VALUES;   // (negative without the flag)
  const int heads = 2 * p.Hkv;
  ptx::grid_dependency_wait();
  for_segments(p, [&](const Segment& s, int) {
    const int32_t* prow =
        p.page_table + (size_t)request_of(p, s.bt) * p.max_pages + s.U.tok_start / kPage;
    int next_pid = s.lo + lane < s.hi ? __ldg(prow + s.lo + lane) : 0;
    for (int base = s.lo; base < s.hi; base += 32) {
      const int cnt = min(32, s.hi - base);
      // a page that is not there: page 0 in its place, its step marked
      const bool bad = lane < cnt && (uint32_t)next_pid >= (uint64_t)p.pool_pages;
      const uint32_t bad_pages = __ballot_sync(0xffffffffu, bad);
      const int my_pid = bad ? 0 : next_pid;
      if (bad) atomicOr(p.status, PA_STATUS_BAD_PAGE);
      if (base + 32 + lane < s.hi) next_pid = __ldg(prow + base + 32 + lane);
      for (int j = 0; j < cnt; j += 2) {
        const int z0 = __shfl_sync(0xffffffffu, my_pid, j) * heads + s.g;
        const int z1 = __shfl_sync(0xffffffffu, my_pid, (j + 1) & 31) * heads + s.g;
        const int n = min(2, cnt - j);
        if (!warp_wait(p, v, S::kKEmpty + kr.i, kr.phase ^ 1)) return false;
        if (keys_loaded != stall && elect()) {
          const uint32_t full = v.bar(S::kKFull + kr.i);
          v.poison[kr.i] = (bad_pages >> j) & 3;   // set before the arrival that publishes it
          // (bytes count as they lie in the pool)
          ptx::mbar_arrive_expect_tx(full, n * (S::kVPage + 2 * S::kScalePage));
          for (int i = 0; i < n; ++i) {
            const int z = i ? z1 : z0;
            const uint32_t dst = v.addr + kr.i * S::kKBytes + i * S::kPageBytes;
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c)
              load_box(dst + c * S::kChunkBytes, keys, c * kChunk, z, full, pol);
            const uint32_t scales = v.addr + S::kScales + kr.i * S::kScaleBytes +
                                    i * 2 * S::kScalePage;
            load_bytes(scales, p.scales + (size_t)z * S::kScalePage, S::kScalePage, full, pol);
            load_bytes(scales + S::kScalePage, p.scales + (size_t)(z + p.Hkv) * S::kScalePage,
                       S::kScalePage, full, pol);
          }
        }
        __syncwarp();
        kr.next();
        ++keys_loaded;
        if (!warp_wait(p, v, S::kVEmpty + vr.i, vr.phase ^ 1)) return false;
        if (values_loaded != stall_values && elect()) {
          const uint32_t full = v.bar(S::kVFull + vr.i);
          ptx::mbar_arrive_expect_tx(full, n * S::kVPage);
          for (int i = 0; i < n; ++i)
            load_box(v.addr + S::kV + vr.i * S::kVBytes + i * S::kVPage, values, 0,
                     (i ? z1 : z0) + p.Hkv, full, pol);
        }
        __syncwarp();
        vr.next();
        ++values_loaded;
      }
    }
    return true;
  });
  // Every page of this CTA is requested: the next kernel in the stream may
  // start its prologue.
  if (lane == 0) ptx::launch_dependents();
  // The copies issued land before the CTA can exit, whatever became of the
  // other warps.
  for (int k = max(0, keys_loaded - S::kKStages); k < keys_loaded; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kKFull + k % S::kKStages), (k / S::kKStages) & 1,
                           p.wait_limit_ns);
  for (int k = max(0, values_loaded - S::kVStages); k < values_loaded; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kVFull + k % S::kVStages), (k / S::kVStages) & 1,
                           p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Warp 14: K's scales, from token rows to the rows that the product's copy takes: token i
// of a step is row i % 32, word i / 32 of its chunk.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void scale_warp(const P& p, const View& v, int lane) {
  using S = Smem<D>;
  Ring<S::kKStages> kr;
  Ring<2> sr;
  for_segments(p, [&](const Segment& s, int) {
    for (int left = s.steps(); left > 0; --left) {
      if (!warp_wait(p, v, S::kKFull + kr.i, kr.phase) ||
          !warp_wait(p, v, S::kSfEmpty + sr.i, sr.phase ^ 1))
        return false;
      const uint32_t src = v.addr + S::kScales + kr.i * S::kScaleBytes + lane * S::kScaleRow;
      uint32_t w[S::kChunks][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = src + (i >> 1) * 2 * S::kScalePage + (i & 1) * 32 * S::kScaleRow;
        if constexpr (S::kChunks == 2) {
          const uint2 y = lds64(a);
          w[0][i] = y.x;
          w[S::kChunks - 1][i] = y.y;
        } else {
          w[0][i] = lds32(a);
        }
      }
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
        *reinterpret_cast<uint4*>(v.base + S::kSf + (sr.i * S::kChunks + c) * 512 + lane * 16) =
            make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(v.bar(S::kSfFull + sr.i));
        ptx::mbar_arrive(v.bar(S::kKEmpty + kr.i));
      }
      kr.next();
      sr.next();
    }
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warp 13: scores.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void mma_warp(const P& p, const View& v, uint32_t tmem) {
  using S = Smem<D>;
  Ring<S::kKStages> kr;
  Ring<2> sr, qr;
  if (elect()) tc::copy_scales(tmem + kOnesCols, tc::desc_plain(v.addr + S::kOnes));
  __syncwarp();
  for_segments(p, [&](const Segment& s, int) {
    if (!warp_wait(p, v, S::kQFull + qr.i, qr.phase)) return false;
    const uint64_t b = tc::desc_sw128(v.addr + S::kQ + qr.i * S::kQBytes);
    for (int left = s.steps(); left > 0; --left) {
      if (!warp_wait(p, v, S::kSEmpty + sr.i, sr.phase ^ 1) ||
          !warp_wait(p, v, S::kKFull + kr.i, kr.phase) ||
          !warp_wait(p, v, S::kSfFull + sr.i, sr.phase))
        return false;
      tc::fence_after();
      const uint64_t a = tc::desc_sw128(v.addr + kr.i * S::kKBytes);
      const uint32_t sf = tmem + kSfCols + sr.i * 8;
      if (elect()) {
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c)
          tc::copy_scales(sf + 4 * c,
                          tc::desc_plain(v.addr + S::kSf + (sr.i * S::kChunks + c) * 512));
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_scaled(tmem + sr.i * kQCols, a + (c * S::kChunkBytes >> 4) + 2 * k,
                           b + (c * S::kQChunkBytes >> 4) + 2 * k,
                           tc::idesc_e2m1_e4m3(kStep, kQCols, k), sf + 4 * c, tmem + kOnesCols,
                           c + k > 0);
        }
        tc::commit(v.bar(S::kSFull + sr.i));
        tc::commit(v.bar(S::kKEmpty + kr.i));
        tc::commit(v.bar(S::kSfEmpty + sr.i));
        // and an arrival of its own: the scales and the mark that came with K
        ptx::mbar_arrive(v.bar(S::kSFull + sr.i));
        if (left == 1) tc::commit(v.bar(S::kQEmpty + qr.i));
      }
      __syncwarp();
      kr.next();
      sr.next();
    }
    qr.next();
    return true;
  });
  // Every product this warp issued, and every arrival that follows from one, ends before
  // the CTA can.
  if (elect()) tc::commit(v.bar(S::kDrain));
  __syncwarp();
  ptx::mbar_wait_bounded(v.bar(S::kDrain), 0, p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Warp 15: units without pages, and q of every segment but a CTA's first.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void helper_warp(const P& p, const View& v, int lane) {
  using S = Smem<D>;
  ptx::grid_dependency_wait();
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
  Ring<2> qr;
  int heads = kMaxG;
  QVec<D>* staged = reinterpret_cast<QVec<D>*>(v.base + S::kQRaw) + lane;   // [head][lane]
  for_segments(p, [&](const Segment& s, int index) {
    if (index > 0) {
      // (a lane's dims by that lane, so no lane waits for another)
#pragma unroll 1
      for (int h = 0; h < p.G; ++h)
        copy_own(ptx::smem_addr(staged + 32 * h), q_of<D>(p, s, h, lane));
      const bool free = warp_wait(p, v, S::kQEmpty + qr.i, qr.phase ^ 1);
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!free) return false;
#pragma unroll 1
      for (int h = 0; h < heads; ++h)
        convert_head<S, D>(p, v, h < p.G ? staged[32 * h] : QVec<D>{}, qr.i, h, lane);
      heads = p.G;   // the first conversion clears the columns without a head
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane < kValueWarps) ptx::mbar_arrive(v.bar(S::kQFull + qr.i));
    }
    qr.next();
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 8-11: a thread per token.
// ---------------------------------------------------------------------------
// Scale bytes of a token's groups, two to a word.
template <int D>
struct Bytes {
  static constexpr int kN = D / 64;
  uint32_t b[kN];
  // word i holds groups group(i) (low half) and group(i) + 2
  __device__ __forceinline__ static int group(int i) { return i / 2 * 4 + i % 2; }
};

template <int D, class P>
__device__ __forceinline__ void score_warps(const P& p, const View& v, uint32_t tmem, int warp,
                                            int lane) {
  using S = Smem<D>;
  constexpr int kBarrier = 2;
  const int tok = warp * 32 + lane, page = tok / kPage, row = tok % kPage;
  State& st = *reinterpret_cast<State*>(v.base + S::kState);
  Weights<D>* buffers = reinterpret_cast<Weights<D>*>(v.base + S::kP);
  float* qs = reinterpret_cast<float*>(v.base + S::kQs) + warp * kMaxG;
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  int it = 0;
  bool fail = false;   // of this lane; the waits of a step ask all of the warp
  ptx::grid_dependency_wait();   // earlier kernels may still read the log-sum-exps
  for_segments(p, [&](const Segment& s, int seg) {
    float2 l[kMaxG / 2];
#pragma unroll
    for (int h = 0; h < kMaxG / 2; ++h) l[h] = f32x2::both(0.f);
    fail |= !wait(p, v, S::kQFull + (seg & 1), (seg >> 1) & 1);
    if (lane < kMaxG) {
      const float x = reinterpret_cast<const float*>(v.base + S::kQScale)[(seg & 1) * kMaxG + lane];
      qs[lane] = fminf(fmaxf(x, -FLT_MAX), FLT_MAX);   // (infinite for |q| above 2^113)
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQEmpty + (seg & 1)));
    int poisoned = 0, most = 0;
    bool first = true;
    const int steps = s.steps();
    for (int i = 0; i < steps; ++i, ++it) {
      const int buf = it & 1;
      const uint32_t phase = (it >> 1) & 1;
      const int tok0 = s.first_tok + (s.lo + 2 * i) * kPage;
      const int pages = min(2, s.hi - (s.lo + 2 * i));
      const bool live = page < pages && tok0 + tok >= s.U.tok_start && tok0 + tok < s.U.tok_end;
      float2 x[kMaxG / 2];
      Bytes<D> e;
      fail = !warp_wait(p, v, S::kSFull + buf, phase, !fail);
      if (!fail) {
        const uint32_t scales = v.addr + S::kScales + kr.i * S::kScaleBytes +
                                (2 * page + 1) * S::kScalePage + row * S::kScaleRow;
        uint32_t w[S::kChunks];
        if constexpr (D == 256) {
          const uint2 y = lds64(scales);
          w[0] = y.x;
          w[S::kChunks - 1] = y.y;
        } else {
          w[0] = lds32(scales);
        }
#pragma unroll
        for (int k = 0; k < S::kChunks; ++k) {
          if (!live) w[k] = 0;   // whatever its row holds
          e.b[2 * k] = w[k] & 0x00ff00ffu;
          e.b[2 * k + 1] = w[k] >> 8 & 0x00ff00ffu;
        }
        poisoned |= v.poison[kr.i];
        tc::fence_after();
        uint32_t r[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          tc::ld16(tmem + buf * kQCols + 16 * k + ((uint32_t)(warp * 32) << 16), r[k]);
#pragma unroll
        for (int k = 0; k < 2; ++k) tc::wait_ld(r[k]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(v.bar(S::kSEmpty + buf));
          ptx::mbar_arrive(v.bar(S::kKEmpty + kr.i));
        }
#pragma unroll
        for (int h = 0; h < kMaxG / 2; ++h) {
          auto part = [&](int n) {
            const int col = n * kMaxG + 2 * h;
            return make_float2(__uint_as_float(r[col / 16][col % 16]),
                               __uint_as_float(r[col / 16][col % 16 + 1]));
          };
          float2 d = f32x2::fma(part(3), f32x2::both(1.f / kQScale3), part(2));
          d = f32x2::fma(d, f32x2::both(1.f / kQScale2), part(1));
          d = f32x2::fma(d, f32x2::both(1.f / kQScale1), part(0));
          d = f32x2::mul(d, reinterpret_cast<const float2*>(qs)[h]);
          x[h] = f32x2::fma(d, f32x2::both(0.f), d);   // an infinite score is NaN
          if (!live) x[h] = f32x2::both(-INFINITY);
        }
      }
      // The token's largest scale; a scale that is NaN is left out, and so is its group.
      auto largest = [&]() {
        uint32_t m = e.b[0];
#pragma unroll
        for (int k = 1; k < Bytes<D>::kN; ++k) m = __vmaxu2(m, e.b[k]);
        return (int)max(m & 0xffffu, m >> 16);
      };
      int top = largest();
      uint32_t nan = 0;   // bit 2 i (+ 1): word i's low (high) half
      if (top == fp4::kNanScale) {
#pragma unroll
        for (int k = 0; k < Bytes<D>::kN; ++k) {
          if ((e.b[k] & 0xffffu) == fp4::kNanScale) nan |= 1u << 2 * k, e.b[k] &= 0xffff0000u;
          if (e.b[k] >> 16 == fp4::kNanScale) nan |= 2u << 2 * k, e.b[k] &= 0xffffu;
        }
        top = largest();
      }
      float2 ex[kMaxG / 2], w[kMaxG / 2];
      auto weigh = [&]() {
#pragma unroll
        for (int h = 0; h < kMaxG / 2; ++h) {
          const float2 m = reinterpret_cast<const float2*>(st.m)[h];
          const int2 t = reinterpret_cast<const int2*>(st.top)[h];
          ex[h] = make_float2(ptx::ex2(x[h].x - m.x), ptx::ex2(x[h].y - m.y));
          // 2^(v + kTop - rho): v is the scale's byte less 127
          w[h] = make_float2(
              ex[h].x * __int_as_float(__viaddmin_s32_relu(top, t.x, 254) << 23),
              ex[h].y * __int_as_float(__viaddmin_s32_relu(top, t.y, 254) << 23));
        }
      };
      // Groups of dims are held to their own sizes as long as V's scales lie within 2^kSpread
      // of the largest met (a weight that counts for a group is then at least 2^-1 with its
      // factor, and has 22 bits); the test takes bounds that are a little closer.  Scales as
      // small as the smallest that appends write do not count beside much larger ones: their
      // groups are zeros, or what such a pool cannot tell from them.
      auto below = [&](int limit) {
        const uint32_t from = 0x00010001u * (0x8000 - max(limit, 0));
        const uint32_t counts = 0x00010001u * (0x8000 - (limit > kTiny ? kTiny + 1 : 0));
        uint32_t y = 0;
#pragma unroll
        for (int k = 0; k < Bytes<D>::kN; ++k) y |= ~(e.b[k] + from) & (e.b[k] + counts);
        return y & 0x80008000u;
      };
      bool move = first;
      if (!move) {
        weigh();
        auto most_of = [](const float2 (&a)[kMaxG / 2]) {
          return fmaxf(fmaxf(fmaxf(a[0].x, a[0].y), fmaxf(a[1].x, a[1].y)),
                       fmaxf(fmaxf(a[2].x, a[2].y), fmaxf(a[3].x, a[3].y)));
        };
        const bool beyond = most_of(w) > kMostWeight || most_of(ex) > kMostExp ||
                            (live && (top > most + 4 || below(most - (kSpread - 4))));
        move = any_in_group(kBarrier, kScores, fail || beyond);
      }
      Weights<D>& to = buffers[buf];
      int flags = 0;
      if (move) {
        // The references move, or scales are looked at more closely.
#pragma unroll
        for (int h = 0; h < kMaxG / 2; ++h) {
          const float a = warp_max(x[h].x), b = warp_max(x[h].y);
          if (lane == 0) reinterpret_cast<float2*>(st.warp_top[warp])[h] = make_float2(a, b);
        }
        const int warp_most = __reduce_max_sync(0xffffffffu, live ? top : 0);
        if (lane == 0) st.warp_most[warp] = warp_most;
        if (any_in_group(kBarrier, kScores, fail)) return false;
        most = first ? 0 : most;
#pragma unroll
        for (int k = 0; k < kScoreWarps; ++k) most = max(most, st.warp_most[k]);
#pragma unroll
        for (int h = 0; h < kMaxG / 2; ++h) {
          float2 m = first ? f32x2::both(kNoRef) : reinterpret_cast<const float2*>(st.m)[h];
          float2 t = f32x2::both(-INFINITY);
#pragma unroll
          for (int k = 0; k < kScoreWarps; ++k) {
            const float2 y = reinterpret_cast<const float2*>(st.warp_top[k])[h];
            t = make_float2(fmaxf(t.x, y.x), fmaxf(t.y, y.y));
          }
          m = make_float2(fmaxf(m.x, ref_ceil(t.x)), fmaxf(m.y, ref_ceil(t.y)));
          const float up = (float)(top - fp4::kScaleBias);
          const float a = warp_max((x[h].x - m.x) + up), b = warp_max((x[h].y - m.y) + up);
          if (lane == 0) reinterpret_cast<float2*>(st.warp_up[warp])[h] = make_float2(a, b);
        }
        bool far = live && below(most - kSpread);
        if (far) {   // does it hold anything?
          far = false;
          fail = !wait(p, v, S::kVFull + vr.i, vr.phase);
#pragma unroll
          for (int k = 0; k < 2 * Bytes<D>::kN; ++k) {
            const int b = k & 1 ? e.b[k / 2] >> 16 : e.b[k / 2] & 0xffff;
            if (fail || b >= most - kSpread || (b <= kTiny && most - kSpread > kTiny) ||
                (nan >> k & 1))
              continue;
            const int g = Bytes<D>::group(k / 2) + 2 * (k & 1);
            const uint4 c = lds128(v.addr + S::kV + vr.i * S::kVBytes + page * S::kVPage +
                                   run_at<D>(row, g));
            far |= ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0;
          }
        }
        if (any_in_group(kBarrier, kScores, far || fail)) flags |= kWide;
        if (tok < kMaxG) {
          float t = -INFINITY, up = -INFINITY;
#pragma unroll
          for (int k = 0; k < kScoreWarps; ++k) {
            t = fmaxf(t, st.warp_top[k][tok]);
            up = fmaxf(up, st.warp_up[k][tok]);
          }
          const float old = first ? kNoRef : st.m[tok], m = fmaxf(old, ref_ceil(t));
          const bool fresh = old == kNoRef;
          const int down = max((int)(old - m), -(1 << 20));
          const int had = fresh ? -(1 << 20) : kTop - st.top[tok] + down;
          const int rho = max(max(had, (int)ceilf(up)), kNoRho);
          st.m[tok] = m;
          st.top[tok] = kTop - rho;
          st.down[tok] = fresh ? 0.f : ptx::pow2i(down);
          st.by[tok] = ptx::pow2i(had - rho);
        }
        ptx::named_barrier(kBarrier, kScores);
        flags |= kMoved;
#pragma unroll
        for (int h = 0; h < kMaxG / 2; ++h)
          l[h] = f32x2::mul(l[h], reinterpret_cast<const float2*>(st.down)[h]);
        weigh();
      }
#pragma unroll
      for (int h = 0; h < kMaxG / 2; ++h) l[h] = f32x2::add(l[h], ex[h]);
      fail = !warp_wait(p, v, S::kPEmpty + buf, phase ^ 1, !fail);
      if (!fail) {
        if (tok < kMaxG) {
          to.top[tok] = st.top[tok];
          to.by[tok] = st.by[tok];
        }
        if (tok == 0) to.flags = flags;
        const int at = place_of(tok);
#pragma unroll
        for (int k = 0; k < Bytes<D>::kN; ++k) {
          // fp16 2^(scale - top + kUp), 0 below 2^-14: the exponent's bits are scale - top + 16
          uint32_t f = e.b[k];
          if (!(flags & kWide))
            f = __viaddmax_s16x2(f + 0x00010001u * (256 + 15 + kUp - top), 0xff00ff00u, 0u) << 10;
          if (nan) {
            const uint32_t as = flags & kWide ? fp4::kNanScale : 0x7e00u;
            if (nan >> 2 * k & 1) f = (f & 0xffff0000u) | as;
            if (nan >> 2 * k & 2) f = (f & 0xffffu) | as << 16;
          }
          to.factor[Bytes<D>::group(k)][at] = (uint16_t)f;
          to.factor[Bytes<D>::group(k) + 2][at] = (uint16_t)(f >> 16);
        }
        if (flags & kWide) {
          reinterpret_cast<float4*>(to.p[tok])[0] = make_float4(ex[0].x, ex[0].y, ex[1].x, ex[1].y);
          reinterpret_cast<float4*>(to.p[tok])[1] = make_float4(ex[2].x, ex[2].y, ex[3].x, ex[3].y);
        } else {
          uint32_t hi[kMaxG / 2], lo[kMaxG / 2];
#pragma unroll
          for (int h = 0; h < kMaxG / 2; ++h) {
            const __half2 y = __floats2half2_rn(w[h].x, w[h].y);
            const float2 back = __half22float2(y);
            hi[h] = as_u32(y);
            lo[h] = as_u32(__floats2half2_rn(w[h].x - back.x, w[h].y - back.y));
          }
          *reinterpret_cast<uint4*>(to.parts[0][tok]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to.parts[1][tok]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(v.bar(S::kPFull + buf));
      }
      first = false;
      kr.next();
      vr.next();
    }
    // ---- the segment's sums ----
#pragma unroll
    for (int h = 0; h < kMaxG / 2; ++h) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        l[h].x += __shfl_xor_sync(0xffffffffu, l[h].x, off);
        l[h].y += __shfl_xor_sync(0xffffffffu, l[h].y, off);
      }
      if (lane == 0) reinterpret_cast<float2*>(st.sums[warp])[h] = l[h];
    }
    fail |= !wait(p, v, S::kLEmpty + (seg & 1), ((seg >> 1) & 1) ^ 1);
    if (any_in_group(kBarrier, kScores, fail)) return false;
    const bool bad = any_in_group(kBarrier, kScores, poisoned);
    if (warp == 0) {
      if (lane < kMaxG) {
        float* factor = reinterpret_cast<float*>(v.base + S::kFactor) + (seg & 1) * 2 * kMaxG;
        float sum = (st.sums[0][lane] + st.sums[1][lane]) + (st.sums[2][lane] + st.sums[3][lane]);
        if (bad) sum = __int_as_float(0x7fc00000);
        // Products are relative to m + rho; the output, or the partial, to the sum's own
        // magnitude 2^(m + k), with sum 2^-k in (2^-8, 1].  (Two factors, as the first may be
        // as large as the largest V scale.)
        const int k = sum > 0.f ? ((__float_as_int(sum) >> 23) - 127 + 8) >> 3 << 3 : 0;
        const int by = max(-240, min(240, -st.top[lane] - kUp - k));
        const float m = st.m[lane] + (float)k;
        sum *= ptx::pow2i(max(-126, -k));
        const float f = ptx::pow2i(by - (by >> 1));
        factor[lane] = ptx::pow2i(by >> 1);
        factor[kMaxG + lane] = s.whole() ? f / sum : sum != sum ? sum : f;
        if (lane < p.G) {
          if (s.whole()) {
            const size_t at = (size_t)s.bt * p.Hq + s.g * p.G + lane;
            const float y = lse_of(m, sum);
            p.lse[at] = y;
            if (p.lse2) p.lse2[at] = y;
          } else {
            reinterpret_cast<float2*>(p.part_ml)[s.slot() * kMaxG + lane] =
                make_float2(sum != sum ? sum : m, sum);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(v.bar(S::kLFull + (seg & 1)));
    }
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 0-7: products with V.  At 256 dims a warp has a group of dims, at 128 dims a group
// and a page of the step.
// ---------------------------------------------------------------------------
// A lane's sums: dims 4 (lane / 4) .. + 3 of the group, heads 2 (lane % 4) and + 1.
struct Out {
  float2 o[4];
};

// The 32 tokens from token tok of the step.  codes: of their first one's page.
template <int D>
__device__ __forceinline__ void add_products(Out& out, const Weights<D>& from, uint32_t codes,
                                             int group, int tok, int lane) {
  uint32_t c[4], b[2][4];   // c: four codes of tokens 2t, 2t + 1 of eight each
  ptx::ldmatrix_x4_trans(codes + run_at<D>((tok + lane) % kPage, group), c[0], c[1], c[2], c[3]);
#pragma unroll
  for (int k = 0; k < 2; ++k)   // [part, tokens 2t and 2t + 1 | 2t + 8 and 2t + 9]
    ptx::ldmatrix_x4_trans(ptx::smem_addr(&from.parts[lane >> 4][tok + 16 * k + (lane & 15)][0]),
                           b[k][0], b[k][1], b[k][2], b[k][3]);
  const uint4 f4 = *reinterpret_cast<const uint4*>(&from.factor[group][tok + 8 * (lane & 3)]);
  const uint32_t f[2][2] = {{f4.x, f4.y}, {f4.z, f4.w}};
  uint32_t a[2][2][4];   // [k][dims 0 and 1 | 2 and 3]
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t y = __byte_perm(c[2 * k], c[2 * k + 1], 0x5410);   // tokens 2t and 2t + 8
    const uint32_t z = __byte_perm(c[2 * k], c[2 * k + 1], 0x7632);   // 2t + 1 and 2t + 9
    uint32_t even[4], odd[4];   // dims 0, 2 of tokens 2t and 2t + 1, of 2t + 8 and 2t + 9
    fp4::unpack8((y & 0x0f0f0f0fu) | (z << 4 & 0xf0f0f0f0u), even);
    fp4::unpack8((y >> 4 & 0x0f0f0f0fu) | (z & 0xf0f0f0f0u), odd);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[k][j][0] = even[j];
      a[k][j][1] = odd[j];
      a[k][j][2] = even[2 + j];
      a[k][j][3] = odd[2 + j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) b[k][i] = times(b[k][i], f[k][i & 1]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    Acc s = {};
#pragma unroll
    for (int part = 1; part >= 0; --part) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        s = mma(a[k][j][0], a[k][j][1], a[k][j][2], a[k][j][3], b[k][2 * part], b[k][2 * part + 1],
                s);
    }
    out.o[2 * j] = f32x2::add(out.o[2 * j], s.lo);
    out.o[2 * j + 1] = f32x2::add(out.o[2 * j + 1], s.hi);
  }
}

// 32 tokens of a step whose V scales lie far apart: in fp32, token by token.
template <int D>
__device__ __forceinline__ void add_wide(Out& out, const Weights<D>& from, uint32_t codes,
                                         int group, int tok, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int up0 = from.top[2 * t] + kUp, up1 = from.top[2 * t + 1] + kUp;
#pragma unroll 1
  for (int i = tok; i < tok + 32; ++i) {
    const int b = from.factor[group][place_of(i)];
    float2 w = *reinterpret_cast<const float2*>(&from.p[i][2 * t]);
    w.x *= __int_as_float(__viaddmin_s32_relu(b, up0, 254) << 23);
    w.y *= __int_as_float(__viaddmin_s32_relu(b, up1, 254) << 23);
    if (b == fp4::kNanScale) w = f32x2::both(__int_as_float(0x7fc00000));
    float y[8];
    fp4::unpack8(lds16(codes + run_at<D>(i % kPage, group) + 2 * g), y);
#pragma unroll
    for (int k = 0; k < 4; ++k) out.o[k] = f32x2::fma(w, f32x2::both(y[k]), out.o[k]);
  }
}

template <int D, class P>
__device__ __forceinline__ void value_warps(const P& p, const View& v, int warp, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, t = lane & 3;
  const int group = D == 256 ? warp : warp & 3, half = D == 256 ? 0 : warp >> 2;
  ptx::grid_dependency_wait();   // earlier kernels write q and may still read the outputs
  for_segments(p, [&](const Segment& s, int) {
    const QVec<D> raw = warp < p.G ? __ldg(q_of<D>(p, s, warp, lane)) : QVec<D>{};
    convert_head<S, D>(p, v, raw, 0, warp, lane);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQFull));
    return false;   // the first segment's
  });
  const Weights<D>* buffers = reinterpret_cast<const Weights<D>*>(v.base + S::kP);
  Ring<S::kVStages> vr;
  int it = 0;
  for_segments(p, [&](const Segment& s, int seg) {
    Out out;
#pragma unroll
    for (int k = 0; k < 4; ++k) out.o[k] = f32x2::both(0.f);
    bool fail = false;
    for (int left = s.hi - s.lo; left > 0; left -= 2, ++it) {
      const int buf = it & 1;
      fail = !warp_wait(p, v, S::kPFull + buf, (it >> 1) & 1) ||
             !warp_wait(p, v, S::kVFull + vr.i, vr.phase);
      if (fail) break;
      const Weights<D>& w = buffers[buf];
      const int flags = w.flags;
      if (flags & kMoved) {
        const float2 by = *reinterpret_cast<const float2*>(&w.by[2 * t]);
#pragma unroll
        for (int k = 0; k < 4; ++k) out.o[k] = f32x2::mul(out.o[k], by);
      }
      const uint32_t codes = v.addr + S::kV + vr.i * S::kVBytes;
      const int first = D == 256 ? 0 : half, last = D == 256 ? min(left, 2) : min(left, half + 1);
      if (flags & kWide) {
        for (int page = first; page < last; ++page)
          for (int i = 0; i < kPage; i += 32)
            add_wide<D>(out, w, codes + page * S::kVPage, group, page * kPage + i, lane);
      } else {
#pragma unroll 2
        for (int page = first; page < last; ++page) {
          add_products<D>(out, w, codes + page * S::kVPage, group, page * kPage, lane);
          add_products<D>(out, w, codes + page * S::kVPage, group, page * kPage + 32, lane);
        }
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(v.bar(S::kPEmpty + buf));
        ptx::mbar_arrive(v.bar(S::kVEmpty + vr.i));
      }
      vr.next();
    }
    fail = fail || !wait(p, v, S::kLFull + (seg & 1), (seg >> 1) & 1);
    if (any_in_group(1, kValues, fail)) return false;
    // ---- the segment's output or partial ----
    const float* factor = reinterpret_cast<const float*>(v.base + S::kFactor) +
                          (seg & 1) * 2 * kMaxG + 2 * t;
    const float2 f1 = *reinterpret_cast<const float2*>(factor);
    const float2 f2 = *reinterpret_cast<const float2*>(factor + kMaxG);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kLEmpty + (seg & 1)));
    if constexpr (D == 128) {   // the second page's sums to the first's
      float4* x = reinterpret_cast<float4*>(v.base + S::kX) + (warp & 3) * 64 + lane;
      if (half) {
        x[0] = make_float4(out.o[0].x, out.o[0].y, out.o[1].x, out.o[1].y);
        x[32] = make_float4(out.o[2].x, out.o[2].y, out.o[3].x, out.o[3].y);
      }
      ptx::named_barrier(1, kValues);
      if (!half) {
        const float4 a = x[0], b = x[32];
        out.o[0] = f32x2::add(out.o[0], make_float2(a.x, a.y));
        out.o[1] = f32x2::add(out.o[1], make_float2(a.z, a.w));
        out.o[2] = f32x2::add(out.o[2], make_float2(b.x, b.y));
        out.o[3] = f32x2::add(out.o[3], make_float2(b.z, b.w));
      }
      ptx::named_barrier(1, kValues);   // read before the next segment's are written
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) out.o[k] = f32x2::mul(f32x2::mul(out.o[k], f1), f2);
    const size_t orow = (size_t)s.bt * p.Hq + s.g * p.G;
    const int d = group * kGroup + 4 * g;
    float* dst = (s.whole() ? p.out + orow * D : p.part_o + s.slot() * kMaxG * D) + d;
    float* dst2 = s.whole() && p.out2 ? p.out2 + orow * D + d : nullptr;
    if (!half) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * t + h >= p.G) break;
        const float4 y = h ? make_float4(out.o[0].y, out.o[1].y, out.o[2].y, out.o[3].y)
                           : make_float4(out.o[0].x, out.o[1].x, out.o[2].x, out.o[3].x);
        *reinterpret_cast<float4*>(dst + (2 * t + h) * D) = y;
        if (dst2) *reinterpret_cast<float4*>(dst2 + (2 * t + h) * D) = y;
      }
    }
    if (!s.whole()) {
      Unit U{};
      U.n_parts = s.U.n_parts;
      U.part_base = s.U.part_base;
      finish_split_unit<D, kValues>(p, v, U, s.u, 0, s.bt, s.g, s.U.first_cta, warp * 32 + lane,
                                    warp, lane);
      ptx::named_barrier(1, kValues);   // merge_info is read before it is written again
    }
    return true;
  });
}

template <int D, int kMaxUnits>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q4_kernel(const __grid_constant__ CUtensorMap keys,
                     const __grid_constant__ CUtensorMap values,
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
  v.abort_flag = misc + S::kKStages;
  v.merge_info = misc + S::kKStages + 1;
  int* tmem_slot = misc + S::kKStages + 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) {
      int n = 1;
      if (i >= S::kKEmpty && i < S::kVFull) n = 2 + kScoreWarps;   // products, scales, softmax
      if (i >= S::kVEmpty && i < S::kSfFull) n = kValueWarps;
      if (i >= S::kSFull && i < S::kSEmpty) n = 2;                 // products and scales
      if (i >= S::kSEmpty && i < S::kPEmpty) n = kScoreWarps;      // S empty, P full
      if (i >= S::kPEmpty && i < S::kQEmpty) n = kValueWarps;      // P empty, q full
      if (i >= S::kQEmpty && i < S::kLFull) n = kScoreWarps + 1;   // and the last product
      if (i >= S::kLEmpty && i < S::kDrain) n = kValueWarps;
      ptx::mbar_init(v.bar(i), n);
    }
    *v.abort_flag = 0;
    ptx::mbar_init_fence();
  }
  if (warp == kTmaWarp && lane == 0) {
    ptx::prefetch_tensormap(&keys);
    ptx::prefetch_tensormap(&values);
  }
  if (warp == kScaleWarp) {
    for (int i = 0; i < 4; ++i)   // scales of one
      reinterpret_cast<uint32_t*>(v.base + S::kOnes)[32 * i + lane] = 0x7f7f7f7fu;
    ptx::fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) tc::alloc(ptx::smem_addr(tmem_slot), kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile int*>(tmem_slot);
  if (warp < kScoreWarp) value_warps<D>(p, v, warp, lane);
  else if (warp < kTmaWarp) score_warps<D>(p, v, tmem, warp - kScoreWarp, lane);
  else if (warp == kTmaWarp) tma_warp<D>(p, v, &keys, &values, lane);
  else if (warp == kMmaWarp) mma_warp<D>(p, v, tmem);
  else if (warp == kScaleWarp) scale_warp<D>(p, v, lane);
  else helper_warp<D>(p, v, lane);
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, kTmemCols);
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
int launch_units(const CUtensorMap* maps, const Plan& plan, const Launch& L,
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
                         stream, maps[0], maps[1], prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "4-bit paged decode launch failed: %s", cudaGetErrorString(e));
  return PA_OK;
}

int launch(int D, const CUtensorMap* maps, const Plan& plan, const Launch& L,
           const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  const bool small = L.n <= (size_t)kMaxUnitsSmall;
  if (D == 128)
    return small ? launch_units<128, kMaxUnitsSmall>(maps, plan, L, order, common, stream)
                 : launch_units<128, kMaxUnitsLarge>(maps, plan, L, order, common, stream);
  return small ? launch_units<256, kMaxUnitsSmall>(maps, plan, L, order, common, stream)
               : launch_units<256, kMaxUnitsLarge>(maps, plan, L, order, common, stream);
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
  PA_REQUIRE(reinterpret_cast<uintptr_t>(pool) % 32 == 0, "pool must be 32-byte aligned");
  // K's codes go to shared memory in bytes, 128 to a row, V's as they are.
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    const cuuint32_t row = i ? D / 2 : D;   // elements
    const cuuint64_t dims[3] = {row, kPage, (cuuint64_t)pool_pages * 2 * Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)D / 2, (cuuint64_t)D / 2 * kPage};
    const cuuint32_t box[3] = {i ? row : (cuuint32_t)kChunk, kPage, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(&maps[i],
                           i ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B,
                           3, const_cast<void*>(pool), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           i && D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
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
    rc = launch(D, maps, plan, L, order, common, stream);
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
