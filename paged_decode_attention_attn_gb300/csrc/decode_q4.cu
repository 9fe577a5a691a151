// Split-KV paged GQA decode attention over a 4-bit pool (e2m1 codes, a power of two as
// the scale of each 32 values of a token's head) with a per-tile log-sum-exp, for
// sm_103a.
//
// The bytes of codes and scales bound it: (D + D / 16) bytes per token and kv head, 17/64
// of the bf16 pool's, so an SM has a quarter of the bf16 kernel's time per token, and the
// instructions per value decide.  No thread converts a code of K, and one of V takes half an
// instruction of one lane:
//
//  * Work split and partials: as the other decode kernels (split_units.cuh, unit_plan.h);
//    a request's tiles are merged by a kernel of its own (tile_merge.cuh).  A CTA streams its
//    pages two at a time: a step is 128 tokens of one kv head.
//  * S = K Q^T on the fifth-generation tensor cores with block scales: M = 128 tokens, N = 32,
//    K = D.  TMA unpacks the codes to the bytes that the product takes, a token's scales go to
//    tensor memory beside them (one byte per 32 dims, the pool's own groups), and q is held
//    as four e4m3 parts (q_parts.cuh) with scales of one.
//  * Softmax: a thread per token, two groups of four warps on alternating steps; a warp has
//    references of its own.  e = 2^(x - m) for the sum, with m a multiple of 8 near a head's
//    largest score; the product's weight is w = e 2^(v - m'), 2^v the token's largest V scale,
//    in fp16 as a high and a low part (22 bits), with m' such that w is below 2^15 whatever the
//    scales: a weight is within 2^-23 of itself, or 2^-39 of the row's largest.  m and m' move
//    rarely, then by an exact power of two.
//  * O^T = V^T P^T on the same tensor cores in fp16: V's scales differ along its rows, which no
//    block scale does, so its codes are turned to fp16 in registers, times their scales relative
//    to the token's largest, and go to tensor memory as the operand of M = 128 dims.  A warp has
//    one group of 32 dims: ldmatrix transposes four codes at a time, two tokens' codes are
//    interleaved by nibble so that one conversion gives a word of two tokens, and the registers
//    are the fragment that a store of 16 lanes takes.  N = 16 (the parts of all heads), K = 32
//    tokens: each softmax warp's product starts from zero and is added to fp32 registers (a
//    thread per dim), weighed by that warp's reference.
//    (mma.sync instead: a step of 256 dims 0.54 us, and twice that beside the scores' products,
//    since the two kinds of tensor instructions hold each other up.)
//  * Warps: 0-7 V and outputs, 8-15 softmax, one each for TMA, scores, products with V and what
//    is done once per segment.  All waits are on mbarriers with a time limit; S, its scales, P
//    and V's operand have two buffers each, K and V rings of their own.
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
constexpr int kGroups = 2, kGroupWarps = 4, kScoreWarps = kGroups * kGroupWarps;
constexpr int kScoreWarp = kValueWarps, kTmaWarp = kScoreWarp + kScoreWarps,
              kMmaWarp = kTmaWarp + 1, kProductWarp = kMmaWarp + 1, kHelperWarp = kProductWarp + 1;
constexpr int kThreads = 32 * (kHelperWarp + 1);
constexpr int kTop = 15;                     // log2 of the largest weight
constexpr float kMostWeight = 65000.f;       // in fp16, which ends at 65504
constexpr int kUp = 13;                      // V's codes go in times 2^13: 6 * 2^13 is in range
// How far V scales may lie below the largest that a softmax warp has met in the segment
// (log2).
constexpr int kSpread = 16;
constexpr int kTiny = fp4::kScaleBias + fp4::kMinScaleExp;   // the smallest scale written
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNoRef = -1e30f;             // m before the first score
constexpr int kNoRho = -1000;
constexpr float kMostExp = 0x1p64f;          // e may lie above 1, up to this
// Tensor memory: S [2], its scales [2], scales of one, products [chunk][32 tokens][kPCols], V
// [2][chunk][two tokens].
constexpr int kPCols = 2 * kMaxG;
constexpr int kTmemCols = 512, kSfCols = 2 * kQCols, kOnesCols = kSfCols + 2 * 8, kDCols = 128,
              kACols = 256, kAStep = kStep / 2;

static_assert(kStep == 32 * kGroupWarps && kScoreWarp % 4 == 0, "a thread per token");

// A step's weights, from the softmax warps to the product warps; kH: heads (4 or 8).
template <int D, int kH>
struct alignas(256) Weights {
  // A token's row: fp16 high and low parts of all heads, as the product's operand (N-major, rows
  // of 32 bytes whose halves change places every four tokens); where V's scales lie far apart
  // (kWide, of 32 tokens each) its probabilities in fp32.
  float p[kStep][8];
  // [group][place_of(token)]: what V's codes are multiplied by, in fp16; with kWide its byte
  uint16_t factor[D / kGroup][kStep];
  // of each 32 tokens: the references, m and kTop - (m' - m), written with kMoved or kWide
  float m[kGroupWarps][kH];
  int top[kGroupWarps][kH];
  int flags[kGroupWarps];
};
// Where the high (0) or low parts of 8 heads lie in a token's row, in floats; 4 heads have both
// in the place of the high.
__device__ __forceinline__ int part_at(int tok, int part) {
  return 4 * (part ^ (tok >> 2 & 1));
}
constexpr int kMoved = 1, kWide = 2;
// Tokens of 32 are ordered so that 16 bytes hold the eight that lane t of four has in two
// products: t's 2t, 2t + 1, 2t + 8, 2t + 9 of both.
__device__ __forceinline__ int place_of(int tok) {
  return (tok & ~31) | (tok >> 1 & 3) << 3 | (tok >> 4 & 1) << 2 | (tok >> 3 & 1) << 1 | (tok & 1);
}

// Shared memory of a CTA; offsets from a 1024-byte boundary.
template <int D, int kH>
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
  static constexpr int kP = (kOnes + 512 + 255) / 256 * 256;   // Weights [2]
  static constexpr int kQRaw = kP + 2 * sizeof(Weights<D, kH>);   // [head][dim] of a later segment
  // D = 128: sums of the second page, [warp][lane][head], and their references [warp][head]
  static constexpr int kX = kQRaw + kMaxG * D * 2;
  // [2][softmax warp][m | sum][head] of a segment
  static constexpr int kStats = kX + (D == 128 ? kValueWarps / 2 * (32 * kMaxG + 2 * kMaxG) * 4 : 0);
  static constexpr int kQScale = kStats + 2 * kScoreWarps * 2 * kMaxG * 4;   // [2][head]
  static constexpr int kQs = kQScale + 2 * kMaxG * 4;      // a softmax warp's copy: [warp][head]
  // [product warp][softmax warp][head]: what products are weighed by
  static constexpr int kBy = kQs + kScoreWarps * kMaxG * 4;
  static constexpr int kBars = kBy + kValueWarps * kScoreWarps * kMaxG * 4;
  static constexpr int kKFull = 0, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages,
                       kVEmpty = kVFull + kVStages, kSfEmpty = kVEmpty + kVStages,
                       kSFull = kSfEmpty + 2, kSEmpty = kSFull + 2, kPFull = kSEmpty + 2,
                       kPEmpty = kPFull + 2, kAFull = kPEmpty + 2, kAEmpty = kAFull + 2,
                       kDFull = kAEmpty + 2, kDEmpty = kDFull + 1, kQFull = kDEmpty + 1,
                       kQEmpty = kQFull + 2, kLFull = kQEmpty + 2, kLEmpty = kLFull + 2,
                       kDrain = kLEmpty + 2, kNumBars = kDrain + 2;
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
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float warp_max(float x) {   // (NaN ignored)
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {   // fp16 pairs
  return as_u32(__hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y)));
}

// Where group c of row r lies in a page's codes of V (the copies' swizzle).
template <int D>
__device__ __forceinline__ int run_at(int r, int c) {
  return r * (D / 2) + ((c ^ (D == 256 ? r & 7 : r >> 1 & 3)) << 4);
}

// ---------------------------------------------------------------------------
// Warp 16: the pages' K (with both scales) and V into their rings.
// ---------------------------------------------------------------------------
template <int D, int kH, class P>
__device__ __forceinline__ void tma_warp(const P& p, const View& v, const CUtensorMap* keys,
                                         const CUtensorMap* values, int lane) {
  using S = Smem<D, kH>;
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
// Warp 17: scores.  K's scales go from token rows to the rows that the copy to tensor memory
// takes: token i of a step is row i % 32, word i / 32 of its chunk.  Warp 18: products with V.
// ---------------------------------------------------------------------------
// Every product this warp issued, and every arrival that follows from one, ends before the
// CTA can.
template <class P>
__device__ __forceinline__ void drain(const P& p, const View& v, int bar) {
  if (elect()) tc::commit(v.bar(bar));
  __syncwarp();
  ptx::mbar_wait_bounded(v.bar(bar), 0, p.wait_limit_ns);
}

template <int D, int kH, class P>
__device__ __forceinline__ void mma_warp(const P& p, const View& v, uint32_t tmem, int lane) {
  using S = Smem<D, kH>;
  Ring<S::kKStages> kr;
  Ring<2> sr, qr;
  if (elect()) tc::copy_scales(tmem + kOnesCols, tc::desc_plain(v.addr + S::kOnes));
  __syncwarp();
  for_segments(p, [&](const Segment& s, int) {
    if (!warp_wait(p, v, S::kQFull + qr.i, qr.phase)) return false;
    const uint64_t b = tc::desc_sw128(v.addr + S::kQ + qr.i * S::kQBytes);
    for (int left = s.steps(); left > 0; --left) {
      if (!warp_wait(p, v, S::kKFull + kr.i, kr.phase) ||
          !warp_wait(p, v, S::kSfEmpty + sr.i, sr.phase ^ 1))
        return false;
      const uint32_t src = v.addr + S::kScales + kr.i * S::kScaleBytes + lane * S::kScaleRow;
      uint32_t w[S::kChunks][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t from = src + (i >> 1) * 2 * S::kScalePage + (i & 1) * 32 * S::kScaleRow;
        if constexpr (S::kChunks == 2) {
          const uint2 y = lds64(from);
          w[0][i] = y.x;
          w[S::kChunks - 1][i] = y.y;
        } else {
          w[0][i] = lds32(from);
        }
      }
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
        *reinterpret_cast<uint4*>(v.base + S::kSf + (sr.i * S::kChunks + c) * 512 + lane * 16) =
            make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (!warp_wait(p, v, S::kSEmpty + sr.i, sr.phase ^ 1)) return false;
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
        // and an arrival of its own: V's scales and the mark that came with K
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
  drain(p, v, S::kDrain);
}

template <int D, int kH, class P>
__device__ __forceinline__ void product_warp(const P& p, const View& v, uint32_t tmem) {
  using S = Smem<D, kH>;
  constexpr uint32_t kIdesc = tc::idesc_f16(kChunk, kPCols, false, true);
  Ring<2> pr;
  Ring<1> dr;
  for_segments(p, [&](const Segment& s, int) {
    for (int left = s.hi - s.lo; left > 0; left -= 2) {
      if (!warp_wait(p, v, S::kPFull + pr.i, pr.phase) ||
          !warp_wait(p, v, S::kAFull + pr.i, pr.phase) ||
          !warp_wait(p, v, S::kDEmpty, dr.phase ^ 1))
        return false;
      tc::fence_after();
      const uint64_t b = tc::desc_sw32(v.addr + S::kP + pr.i * sizeof(Weights<D, kH>));
      const uint32_t a = tmem + kACols + pr.i * S::kChunks * kAStep;
      if (elect()) {
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c) {
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k) {   // 16 tokens
            if (k >= kPage / 16 && left < 2) break;
            tc::mma_f16(tmem + kDCols + (c * 4 + k / 2) * kPCols, a + c * kAStep + 8 * k,
                        b + (16 * 32 * k >> 4), kIdesc, k & 1);
          }
        }
        tc::commit(v.bar(S::kDFull));
        tc::commit(v.bar(S::kAEmpty + pr.i));
        tc::commit(v.bar(S::kPEmpty + pr.i));
      }
      __syncwarp();
      pr.next();
      dr.next();
    }
    return true;
  });
  drain(p, v, S::kDrain + 1);
}

// ---------------------------------------------------------------------------
// Warp 19: units without pages, and q of every segment but a CTA's first.
// ---------------------------------------------------------------------------
template <int D, int kH, class P>
__device__ __forceinline__ void helper_warp(const P& p, const View& v, int lane) {
  using S = Smem<D, kH>;
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
// Warps 8-11 and 12-15: a thread per token of every other step.
// ---------------------------------------------------------------------------
// Scale bytes of a token's groups, two to a word: word i holds groups group(i) (low half)
// and group(i) + 2.
template <int D>
struct Bytes {
  static constexpr int kN = D / 64;
  uint32_t b[kN];
  __device__ __forceinline__ static int group(int i) { return i / 2 * 4 + i % 2; }
};

// Lane 0's values of all heads to shared memory.
template <int kH>
__device__ __forceinline__ void store_heads(float* to, const float2 (&x)[kH / 2]) {
#pragma unroll
  for (int h = 0; h < kH / 2; h += 2)
    *reinterpret_cast<float4*>(to + 2 * h) = make_float4(x[h].x, x[h].y, x[h + 1].x, x[h + 1].y);
}

template <int D, int kH, class P>
__device__ __forceinline__ void score_warps(const P& p, const View& v, uint32_t tmem, int sw,
                                            int lane) {
  using S = Smem<D, kH>;
  constexpr int kN = kH / 2;           // heads go in pairs
  const int group = sw / kGroupWarps, warp = sw % kGroupWarps;
  const int tok = warp * 32 + lane, page = tok / kPage, row = tok % kPage;
  Weights<D, kH>& to = reinterpret_cast<Weights<D, kH>*>(v.base + S::kP)[group];
  float* qs = reinterpret_cast<float*>(v.base + S::kQs) + sw * kMaxG;
  Ring<S::kKStages> kr;
  Ring<S::kVStages> vr;
  int it = 0;
  ptx::grid_dependency_wait();
  for_segments(p, [&](const Segment& s, int seg) {
    // references (see the top of the file): m, and kTop - (m' - m)
    float2 l[kN], m[kN];
    int2 top[kN];
#pragma unroll
    for (int h = 0; h < kN; ++h) {
      l[h] = f32x2::both(0.f);
      m[h] = f32x2::both(kNoRef);
      top[h] = make_int2(0, 0);
    }
    if (!warp_wait(p, v, S::kQFull + (seg & 1), (seg >> 1) & 1)) return false;
    if (lane < kMaxG) {
      const float x = reinterpret_cast<const float*>(v.base + S::kQScale)[(seg & 1) * kMaxG + lane];
      qs[lane] = fminf(fmaxf(x, -FLT_MAX), FLT_MAX);   // (infinite for |q| above 2^113)
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQEmpty + (seg & 1)));
    int poisoned = 0, most = -1000;    // most: the largest V scale met in the segment, its byte
    const int steps = s.steps();
    for (int i = 0; i < steps; ++i, ++it, kr.next(), vr.next()) {
      if ((it & 1) != group) continue;
      const uint32_t phase = (it >> 1) & 1;
      const int tok0 = s.first_tok + (s.lo + 2 * i) * kPage;
      const int pages = min(2, s.hi - (s.lo + 2 * i));
      const bool live = page < pages && tok0 + tok >= s.U.tok_start && tok0 + tok < s.U.tok_end;
      if (!warp_wait(p, v, S::kSFull + group, phase)) return false;
      Bytes<D> e;
      {
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
      }
      tc::fence_after();
      uint32_t r[2][16];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        tc::ld16(tmem + group * kQCols + 16 * k + ((uint32_t)(warp * 32) << 16), r[k]);
#pragma unroll
      for (int k = 0; k < 2; ++k) tc::wait_ld(r[k]);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(v.bar(S::kSEmpty + group));
        ptx::mbar_arrive(v.bar(S::kKEmpty + kr.i));
      }
      float2 x[kN];
#pragma unroll
      for (int h = 0; h < kN; ++h) {
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
      // The token's largest scale; a scale that is NaN is left out, and so is its group.
      auto largest = [&]() {
        uint32_t y = e.b[0];
#pragma unroll
        for (int k = 1; k < Bytes<D>::kN; ++k) y = __vmaxu2(y, e.b[k]);
        return (int)max(y & 0xffffu, y >> 16);
      };
      int scale = largest();
      uint32_t nan = 0;   // bit 2 i (+ 1): word i's low (high) half
      if (scale == fp4::kNanScale) {
#pragma unroll
        for (int k = 0; k < Bytes<D>::kN; ++k) {
          if ((e.b[k] & 0xffffu) == fp4::kNanScale) nan |= 1u << 2 * k, e.b[k] &= 0xffff0000u;
          if (e.b[k] >> 16 == fp4::kNanScale) nan |= 2u << 2 * k, e.b[k] &= 0xffffu;
        }
        scale = largest();
      }
      float2 ex[kN], w[kN];
      auto weigh = [&]() {
#pragma unroll
        for (int h = 0; h < kN; ++h) {
          ex[h] = make_float2(ptx::ex2(x[h].x - m[h].x), ptx::ex2(x[h].y - m[h].y));
          // 2^(v + top): v is the scale's byte less 127
          w[h] = make_float2(
              ex[h].x * __int_as_float(__viaddmin_s32_relu(scale, top[h].x, 254) << 23),
              ex[h].y * __int_as_float(__viaddmin_s32_relu(scale, top[h].y, 254) << 23));
        }
      };
      // Groups of dims are held to their own sizes as long as V's scales lie within 2^kSpread
      // of the largest met (a weight that counts for a group is then at least 2^-2, and has 22
      // bits); the test takes bounds that are a little closer.  Scales as
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
      weigh();
      float largest_w = fmaxf(w[0].x, w[0].y), largest_e = fmaxf(ex[0].x, ex[0].y);
#pragma unroll
      for (int h = 1; h < kN; ++h) {
        largest_w = fmaxf(largest_w, fmaxf(w[h].x, w[h].y));
        largest_e = fmaxf(largest_e, fmaxf(ex[h].x, ex[h].y));
      }
      const bool beyond = largest_w > kMostWeight || largest_e > kMostExp ||
                          (live && (scale > most + 4 || below(most - (kSpread - 4))));
      int flags = 0;
      if (__any_sync(0xffffffffu, beyond)) {
        // The references move, or scales are looked at more closely.
        flags = kMoved;
        most = max(most, (int)__reduce_max_sync(0xffffffffu, live ? scale : 0));
        const float up = (float)(scale - fp4::kScaleBias);
        auto move = [&](float y, float& mh, int& th, float& lh) {
          const float to_m = fmaxf(mh, ref_ceil(warp_max(y)));
          const float over = warp_max((y - to_m) + up);
          const bool fresh = mh == kNoRef;
          const int down = max((int)(mh - to_m), -(1 << 20));
          const int had = fresh ? -(1 << 20) : kTop - th + down;
          lh *= fresh ? 0.f : ptx::pow2i(down);
          mh = to_m;
          th = kTop - max(max(had, (int)ceilf(over)), kNoRho);
        };
#pragma unroll
        for (int h = 0; h < kN; ++h) {
          move(x[h].x, m[h].x, top[h].x, l[h].x);
          move(x[h].y, m[h].y, top[h].y, l[h].y);
        }
        bool far = live && below(most - kSpread), ok = true;
        if (far) {   // does it hold anything?
          far = false;
          ok = wait(p, v, S::kVFull + vr.i, vr.phase);
#pragma unroll
          for (int k = 0; k < 2 * Bytes<D>::kN; ++k) {
            const int b = k & 1 ? e.b[k / 2] >> 16 : e.b[k / 2] & 0xffff;
            if (!ok || b >= most - kSpread || (b <= kTiny && most - kSpread > kTiny) ||
                (nan >> k & 1))
              continue;
            const int g = Bytes<D>::group(k / 2) + 2 * (k & 1);
            const uint4 c = lds128(v.addr + S::kV + vr.i * S::kVBytes + page * S::kVPage +
                                   run_at<D>(row, g));
            far |= ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0;
          }
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (__any_sync(0xffffffffu, far)) flags |= kWide;
        weigh();
      }
#pragma unroll
      for (int h = 0; h < kN; ++h) l[h] = f32x2::add(l[h], ex[h]);
      // fp16 2^(scale - largest + kUp), 0 below 2^-14: the exponent's bits are the difference
      // + 28
      uint32_t f[Bytes<D>::kN];
#pragma unroll
      for (int k = 0; k < Bytes<D>::kN; ++k) {
        f[k] = e.b[k];
        if (!(flags & kWide))
          f[k] = __viaddmax_s16x2(f[k] + 0x00010001u * (256 + 15 + kUp - scale), 0xff00ff00u, 0u)
                 << 10;
        if (nan) {
          const uint32_t as = flags & kWide ? fp4::kNanScale : 0x7e00u;
          if (nan >> 2 * k & 1) f[k] = (f[k] & 0xffff0000u) | as;
          if (nan >> 2 * k & 2) f[k] = (f[k] & 0xffffu) | as << 16;
        }
      }
      uint32_t hi[kN], lo[kN];
#pragma unroll
      for (int h = 0; h < kN; ++h) {
        const __half2 y = __floats2half2_rn(w[h].x, w[h].y);
        const float2 back = __half22float2(y);
        hi[h] = as_u32(y);
        lo[h] = as_u32(__floats2half2_rn(w[h].x - back.x, w[h].y - back.y));
      }
      if (!warp_wait(p, v, S::kPEmpty + group, phase ^ 1)) return false;
      const int at = place_of(tok);
#pragma unroll
      for (int k = 0; k < Bytes<D>::kN; ++k) {
        to.factor[Bytes<D>::group(k)][at] = (uint16_t)f[k];
        to.factor[Bytes<D>::group(k) + 2][at] = (uint16_t)(f[k] >> 16);
      }
      if (flags & kWide) {
        store_heads<kH>(to.p[tok], ex);
      } else if constexpr (kH == 8) {
        *reinterpret_cast<uint4*>(to.p[tok] + part_at(tok, 0)) =
            make_uint4(hi[0], hi[1], hi[2], hi[kN - 1]);
        *reinterpret_cast<uint4*>(to.p[tok] + part_at(tok, 1)) =
            make_uint4(lo[0], lo[1], lo[2], lo[kN - 1]);
      } else {
        *reinterpret_cast<uint4*>(to.p[tok] + part_at(tok, 0)) =
            make_uint4(hi[0], hi[1], lo[0], lo[1]);
      }
      if (lane == 0) {
        to.flags[warp] = flags;
        if (flags) {
          store_heads<kH>(to.m[warp], m);
#pragma unroll
          for (int h = 0; h < kN; ++h) *reinterpret_cast<int2*>(&to.top[warp][2 * h]) = top[h];
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(v.bar(S::kPFull + group));
    }
    // ---- the segment's sums ----
#pragma unroll
    for (int h = 0; h < kN; ++h) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        l[h].x += __shfl_xor_sync(0xffffffffu, l[h].x, off);
        l[h].y += __shfl_xor_sync(0xffffffffu, l[h].y, off);
      }
      if (poisoned) l[h] = f32x2::both(__int_as_float(0x7fc00000));
    }
    if (!warp_wait(p, v, S::kLEmpty + (seg & 1), ((seg >> 1) & 1) ^ 1)) return false;
    if (lane == 0) {
      float* stats = reinterpret_cast<float*>(v.base + S::kStats) +
                     ((seg & 1) * kScoreWarps + sw) * 2 * kMaxG;
      store_heads<kH>(stats, m);
      store_heads<kH>(stats + kMaxG, l);
      ptx::mbar_arrive(v.bar(S::kLFull + (seg & 1)));
    }
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 0-7: V and outputs.  At 256 dims a warp has a group of dims, at 128 dims a group and a
// page of the step; its lanes of tensor memory are those of its group in its chunk.
// ---------------------------------------------------------------------------
// Dim of the group that a lane of tensor memory stands for: rows lane / 4 and + 8 of two
// fragments hold the four dims that a 16-bit unit of codes has.
__device__ __forceinline__ int dim_of(int lane) {
  return 4 * (lane & 7) + 2 * (lane >> 4) + (lane >> 3 & 1);
}

// V of the 32 tokens from token tok of the step to tensor memory.  codes: of their page.
template <int D, int kH>
__device__ __forceinline__ void store_values(const Weights<D, kH>& from, uint32_t codes, int group,
                                             int tok, uint32_t tmem, int lane) {
  uint32_t c[4];   // four codes of tokens 2t and 2t + 1 of eight each
  ptx::ldmatrix_x4_trans(codes + run_at<D>((tok + lane) % kPage, group), c[0], c[1], c[2], c[3]);
  const uint4 f4 = *reinterpret_cast<const uint4*>(&from.factor[group][tok + 8 * (lane & 3)]);
  const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};   // of c's tokens
  uint32_t a[2][8];   // [dims 0 and 1 | 2 and 3][8 tokens][dim]
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t y = __byte_perm(c[2 * k], c[2 * k + 1], 0x5410);   // tokens 2t and 2t + 8
    const uint32_t z = __byte_perm(c[2 * k], c[2 * k + 1], 0x7632);   // 2t + 1 and 2t + 9
    uint32_t even[4], odd[4];   // dims 0, 2 of tokens 2t and 2t + 1, of 2t + 8 and 2t + 9
    fp4::unpack8((y & 0x0f0f0f0fu) | (z << 4 & 0xf0f0f0f0u), even);
    fp4::unpack8((y >> 4 & 0x0f0f0f0fu) | (z & 0xf0f0f0f0u), odd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // [8 tokens][dims 0 and 1 | 2 and 3]
      a[i & 1][4 * k + 2 * (i >> 1)] = times(even[i], f[2 * k + (i >> 1)]);
      a[i & 1][4 * k + 2 * (i >> 1) + 1] = times(odd[i], f[2 * k + (i >> 1)]);
    }
  }
  tc::st_16x128b_x4(tmem, a[0]);
  tc::st_16x128b_x4(tmem + (16u << 16), a[1]);
}

// A dim's sums, for all heads.  They are relative to 2^(m - top), as a softmax warp's products
// to that of its references; lane h has head h's m and top.
template <int kH>
struct Out {
  float2 o[kH / 2];
  float m;
  int top;
  __device__ __forceinline__ void scale(float f) {   // f: of lane h for head h
#pragma unroll
    for (int h = 0; h < kH / 2; ++h)
      o[h] = f32x2::mul(o[h], make_float2(__shfl_sync(0xffffffffu, f, 2 * h),
                                          __shfl_sync(0xffffffffu, f, 2 * h + 1)));
  }
};

// The references of a softmax warp (whose weight is by_now[h]) have moved to m and top.  The
// sums keep the largest reference met; what is relative to a smaller one is weighed.
template <int kH>
__device__ __forceinline__ void follow(Out<kH>& out, const float* m, const int* top, float* by,
                                       float* by_now, int lane) {
  float f = 1.f;
  if (lane < kH) {
    const float mw = m[lane];
    const int tw = top[lane];
    float weight = 1.f;   // (without a reference products are NaN, or there are none)
    if (mw != kNoRef) {
      int d = 1 << 20;
      if (out.m != kNoRef)
        d = max(min((int)(mw - out.m), 1 << 20), -(1 << 20)) + (out.top - tw);
      if (d > 0) {
        f = ptx::pow2i(-d);
        for (int n = 0; n < kScoreWarps; ++n) by[n * kMaxG + lane] *= f;
        out.m = mw;
        out.top = tw;
      }
      weight = ptx::pow2i(min(d, 0));
    }
    by_now[lane] = weight;
  }
  __syncwarp();
  if (__any_sync(0xffffffffu, f != 1.f)) out.scale(f);
}

// 32 tokens of a step whose V scales lie far apart: in fp32, token by token.
template <int D, int kH>
__device__ __forceinline__ void add_wide(Out<kH>& out, const Weights<D, kH>& from, uint32_t codes,
                                         int group, int tok, const float* by, int lane) {
  const int d = dim_of(lane);
  const int* top = from.top[tok / 32];
#pragma unroll 1
  for (int i = tok; i < tok + 32; ++i) {
    const int b = from.factor[group][place_of(i)];
    float y[8];
    fp4::unpack8(lds8(codes + run_at<D>(i % kPage, group) + d / 2) >> 4 * (d & 1), y);
    if (b == fp4::kNanScale) y[0] = __int_as_float(0x7fc00000);
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      float w = from.p[i][h] * __int_as_float(__viaddmin_s32_relu(b, top[h] + kUp, 254) << 23);
      float& o = h % 2 ? out.o[h / 2].y : out.o[h / 2].x;
      o = fmaf(w * by[h], y[0], o);
    }
  }
}

template <int D, int kH, class P>
__device__ __forceinline__ void value_warps(const P& p, const View& v, uint32_t tmem, int warp,
                                            int lane) {
  using S = Smem<D, kH>;
  const int group = D == 256 ? warp : warp & 3, half = D == 256 ? 0 : warp >> 2;
  const int chunk = D == 256 ? warp >> 2 : 0;
  tmem += (uint32_t)(warp % 4 * 32) << 16;
  const uint32_t tmem_a = tmem + kACols + chunk * kAStep, tmem_d = tmem + kDCols + chunk * 4 * kPCols;
  float* by = reinterpret_cast<float*>(v.base + S::kBy) + warp * kScoreWarps * kMaxG;
  ptx::grid_dependency_wait();   // earlier kernels write q and may still read the outputs
  for_segments(p, [&](const Segment& s, int) {
    const QVec<D> raw = warp < p.G ? __ldg(q_of<D>(p, s, warp, lane)) : QVec<D>{};
    convert_head<S, D>(p, v, raw, 0, warp, lane);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQFull));
    return false;   // the first segment's
  });
  const Weights<D, kH>* buffers = reinterpret_cast<const Weights<D, kH>*>(v.base + S::kP);
  Ring<S::kVStages> vr;
  int it = 0;
  for_segments(p, [&](const Segment& s, int seg) {
    Out<kH> out;
#pragma unroll
    for (int h = 0; h < kH / 2; ++h) out.o[h] = f32x2::both(0.f);
    out.m = kNoRef;
    out.top = 0;
    for (int i = lane; i < kScoreWarps * kMaxG; i += 32) by[i] = 0.f;
    __syncwarp();
    bool fail = false;
    // A step's V goes to tensor memory ahead of the sums of the step before it, whose product
    // runs meanwhile.
    const int steps = s.steps(), it0 = it;
    int wide = 0;   // blocks of the step before
    for (int i = 0; i <= steps; ++i) {
      const int first = 2 * half;
      int wide_now = 0;
      if (i < steps) {
        const int pages = min(2, s.hi - s.lo - 2 * i), buf = it & 1;
        const int last = D == 256 ? 2 * pages : min(2 * pages, first + 2);
        fail = !warp_wait(p, v, S::kPFull + buf, (it >> 1) & 1) ||
               !warp_wait(p, v, S::kVFull + vr.i, vr.phase) ||
               !warp_wait(p, v, S::kAEmpty + buf, ((it >> 1) & 1) ^ 1);
        if (fail) break;
        tc::fence_after();
        const Weights<D, kH>& w = buffers[buf];
        const uint32_t codes = v.addr + S::kV + vr.i * S::kVBytes;
#pragma unroll 2
        for (int block = first; block < last; ++block)
          store_values<D, kH>(w, codes + (block >> 1) * S::kVPage, group, 32 * block,
                              tmem_a + buf * S::kChunks * kAStep + 16 * block, lane);
        const int4 f = *reinterpret_cast<const int4*>(w.flags);
        if (f.x | f.y | f.z | f.w) {
          float* by_now = by + buf * kGroupWarps * kMaxG;
#pragma unroll 1
          for (int block = first; block < last; ++block) {
            const int flags = w.flags[block];
            if (flags & kMoved)
              follow<kH>(out, w.m[block], w.top[block], by, by_now + block * kMaxG, lane);
            if (flags & kWide) {
              add_wide<D, kH>(out, w, codes + (block >> 1) * S::kVPage, group, 32 * block,
                              by_now + block * kMaxG, lane);
              wide_now |= 1 << block;
            }
          }
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(v.bar(S::kAFull + buf));
          ptx::mbar_arrive(v.bar(S::kPEmpty + buf));
          ptx::mbar_arrive(v.bar(S::kVEmpty + vr.i));
        }
        vr.next();
        ++it;
      }
      if (i > 0) {
        const int pages = min(2, s.hi - s.lo - 2 * (i - 1)), before = it0 + i - 1;
        const int last = D == 256 ? 2 * pages : min(2 * pages, first + 2);
        fail = !warp_wait(p, v, S::kDFull, before & 1);
        if (fail) break;
        tc::fence_after();
        const float* by_then = by + (before & 1) * kGroupWarps * kMaxG;
#pragma unroll
        for (int k = 0; k < (D == 256 ? 2 : 1); ++k) {   // two blocks at once
          const int block = first + 2 * k;
          if (block >= last) break;
          uint32_t r[2][2 * kH];
#pragma unroll
          for (int j = 0; j < 2; ++j) tc::ld_cols(tmem_d + (block + j) * kPCols, r[j]);
#pragma unroll
          for (int j = 0; j < 2; ++j) tc::wait_ld_cols(r[j]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (wide >> (block + j) & 1) continue;
#pragma unroll
            for (int h = 0; h < kH / 2; ++h) {
              const float2 f = *reinterpret_cast<const float2*>(by_then + (block + j) * kMaxG + 2 * h);
              const float2 hi = make_float2(__uint_as_float(r[j][2 * h]),
                                            __uint_as_float(r[j][2 * h + 1]));
              const float2 lo = make_float2(__uint_as_float(r[j][kH + 2 * h]),
                                            __uint_as_float(r[j][kH + 2 * h + 1]));
              out.o[h] = f32x2::fma(f32x2::add(hi, lo), f, out.o[h]);
            }
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(v.bar(S::kDEmpty));
      }
      wide = wide_now;
    }
    fail = fail || !wait(p, v, S::kLFull + (seg & 1), (seg >> 1) & 1);
    if (any_in_group(1, kValues, fail)) return false;
    if constexpr (D == 128) {   // the second page's sums to the first's
      float* x = reinterpret_cast<float*>(v.base + S::kX) + (warp & 3) * (32 * kMaxG + 2 * kMaxG);
      float4* mine = reinterpret_cast<float4*>(x + lane * kMaxG);
      if (half) {
#pragma unroll
        for (int h = 0; h < kH / 2; h += 2)
          mine[h / 2] = make_float4(out.o[h].x, out.o[h].y, out.o[h + 1].x, out.o[h + 1].y);
        if (lane < kH) {
          x[32 * kMaxG + lane] = out.m;
          x[33 * kMaxG + lane] = __int_as_float(out.top);
        }
      }
      ptx::named_barrier(1, kValues);
      if (!half) {
        float f = 1.f, more = 1.f;
        if (lane < kH) {
          const float mw = x[32 * kMaxG + lane];
          const int tw = __float_as_int(x[33 * kMaxG + lane]);
          if (mw != kNoRef) {
            int d = 1 << 20;
            if (out.m != kNoRef)
              d = max(min((int)(mw - out.m), 1 << 20), -(1 << 20)) + (out.top - tw);
            f = ptx::pow2i(min(-d, 0));
            more = ptx::pow2i(min(d, 0));
            if (d > 0) {
              out.m = mw;
              out.top = tw;
            }
          }
        }
        out.scale(f);
#pragma unroll
        for (int h = 0; h < kH / 2; h += 2) {
          const float4 y = mine[h / 2];
          auto add = [&](float2& o, float a, float b, int i) {
            o = f32x2::fma(make_float2(a, b), make_float2(__shfl_sync(0xffffffffu, more, i),
                                                          __shfl_sync(0xffffffffu, more, i + 1)), o);
          };
          add(out.o[h], y.x, y.y, 2 * h);
          add(out.o[h + 1], y.z, y.w, 2 * h + 2);
        }
      }
      ptx::named_barrier(1, kValues);   // read before the next segment's are written
    }
    // ---- the segment's sums, and its output or partial ----
    const size_t orow = (size_t)s.bt * p.Hq + s.g * p.G;
    float f1 = 0.f, f2 = 0.f;
    if (lane < kH) {
      float m = kNoRef, l = 0.f;
      const float* stats = reinterpret_cast<const float*>(v.base + S::kStats) +
                           (seg & 1) * kScoreWarps * 2 * kMaxG + lane;
#pragma unroll
      for (int k = 0; k < kScoreWarps; ++k) m = fmaxf(m, stats[2 * k * kMaxG]);
#pragma unroll
      for (int k = 0; k < kScoreWarps; ++k)
        l = fmaf(ref_weight(stats[2 * k * kMaxG], m), stats[(2 * k + 1) * kMaxG], l);
      // The output, or the partial, is relative to the sum's own magnitude 2^(m + k), with
      // l 2^-k in (2^-8, 1].  (Two factors, as the first may be as large as the largest V
      // scale.)
      const int k = l > 0.f ? ((__float_as_int(l) >> 23) - 127 + 8) >> 3 << 3 : 0;
      const int ref = max(min((int)(out.m - m), 512), -512);
      const int scale = max(-240, min(240, ref - out.top - kUp - k));
      l *= ptx::pow2i(max(-126, -k));
      m += (float)k;
      f1 = ptx::pow2i(scale >> 1);
      f2 = ptx::pow2i(scale - (scale >> 1));
      if (s.whole()) f2 /= l;
      if (l != l) f2 = l;
      if (warp == 0 && lane < p.G) {
        if (s.whole()) {
          const float x = lse_of(m, l);
          p.lse[orow + lane] = x;
          if (p.lse2) p.lse2[orow + lane] = x;
        } else {
          reinterpret_cast<float2*>(p.part_ml)[s.slot() * kMaxG + lane] =
              make_float2(l != l ? l : m, l);
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kLEmpty + (seg & 1)));
    out.scale(f1);
    out.scale(f2);
    const int d = group * kGroup + dim_of(lane);
    float* dst = (s.whole() ? p.out + orow * D : p.part_o + s.slot() * kMaxG * D) + d;
    float* dst2 = s.whole() && p.out2 ? p.out2 + orow * D + d : nullptr;
    if (!half) {
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        if (h >= p.G) break;
        const float y = h % 2 ? out.o[h / 2].y : out.o[h / 2].x;
        dst[h * D] = y;
        if (dst2) dst2[h * D] = y;
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

template <int D, int kH, int kMaxUnits>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q4_kernel(const __grid_constant__ CUtensorMap keys,
                     const __grid_constant__ CUtensorMap values,
                     const __grid_constant__ Params<kMaxUnits> p) {
  using S = Smem<D, kH>;
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
      if (i >= S::kKEmpty && i < S::kVFull) n = 1 + kGroupWarps;   // products and softmax
      if (i >= S::kVEmpty && i < S::kSfEmpty) n = kValueWarps;
      if (i >= S::kSFull && i < S::kSEmpty) n = 2;                 // products and scales
      if (i >= S::kSEmpty && i < S::kPEmpty) n = kGroupWarps;      // S empty, P full
      if (i >= S::kPEmpty && i < S::kAFull) n = kValueWarps + 1;   // and the product
      if (i >= S::kAFull && i < S::kAEmpty) n = kValueWarps;
      if (i >= S::kDEmpty && i < S::kQEmpty) n = kValueWarps;      // D empty, q full
      if (i >= S::kQEmpty && i < S::kLFull) n = kScoreWarps + 1;   // and the last product
      if (i >= S::kLFull && i < S::kDrain) n = kScoreWarps;        // and L empty: as many
      static_assert(kScoreWarps == kValueWarps, "arrivals at L");
      ptx::mbar_init(v.bar(i), n);
    }
    *v.abort_flag = 0;
    ptx::mbar_init_fence();
  }
  if (warp == kTmaWarp && lane == 0) {
    ptx::prefetch_tensormap(&keys);
    ptx::prefetch_tensormap(&values);
  }
  if (warp == kHelperWarp) {
    for (int i = 0; i < 4; ++i)   // scales of one
      reinterpret_cast<uint32_t*>(v.base + S::kOnes)[32 * i + lane] = 0x7f7f7f7fu;
    ptx::fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) tc::alloc(ptx::smem_addr(tmem_slot), kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile int*>(tmem_slot);
  if (warp < kScoreWarp) value_warps<D, kH>(p, v, tmem, warp, lane);
  else if (warp < kTmaWarp) score_warps<D, kH>(p, v, tmem, warp - kScoreWarp, lane);
  else if (warp == kTmaWarp) tma_warp<D, kH>(p, v, &keys, &values, lane);
  else if (warp == kMmaWarp) mma_warp<D, kH>(p, v, tmem, lane);
  else if (warp == kProductWarp) product_warp<D, kH>(p, v, tmem);
  else helper_warp<D, kH>(p, v, lane);
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

template <int D, int kH, int N>
int launch_units(const CUtensorMap* maps, const Plan& plan, const Launch& L,
                 const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  using Prm = Params<N>;
  static_assert(N >= kMaxUnitsSmall && offsetof(Prm, starts) == offsetof(Common, starts), "");
  Prm prm;
  std::memcpy(static_cast<void*>(&prm), &common, offsetof(Common, starts));
  fill_units(plan, L, order, &prm);
  static PerContext smem_limit;   // the attribute lives in the context
  cudaError_t e = smem_limit.apply([] {
    return cudaFuncSetAttribute(decode_q4_kernel<D, kH, N>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, kH>::kAlloc);
  });
  if (e == cudaSuccess)
    e = launch_dependent(decode_q4_kernel<D, kH, N>, dim3(L.grid), dim3(kThreads), Smem<D, kH>::kAlloc,
                         stream, maps[0], maps[1], prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "4-bit paged decode launch failed: %s", cudaGetErrorString(e));
  return PA_OK;
}

template <int D, int kH>
int launch(const CUtensorMap* maps, const Plan& plan, const Launch& L,
           const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  return L.n <= (size_t)kMaxUnitsSmall
             ? launch_units<D, kH, kMaxUnitsSmall>(maps, plan, L, order, common, stream)
             : launch_units<D, kH, kMaxUnitsLarge>(maps, plan, L, order, common, stream);
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
  const bool few = common.G <= 4;
  auto fn = D == 128 ? (few ? launch<128, 4> : launch<128, 8>)
                     : (few ? launch<256, 4> : launch<256, 8>);
  for (Launch& L : plan.launches) {
    const std::vector<int> order = pack(&plan, &L, sms, rules);
    rc = fn(maps, plan, L, order, common, stream);
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
