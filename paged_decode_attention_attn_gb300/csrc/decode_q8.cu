// Split-KV paged GQA decode attention over an 8-bit (e4m3) pool with a per-tile
// log-sum-exp, for sm_103a.
//
// The bytes of the codes bound it: 2 D bytes per token and kv head, half of the
// bf16 pool's, so each SM has half the time per token that the bf16 kernel has.
// Both products therefore run on the fifth-generation tensor cores straight
// from the codes as TMA leaves them in shared memory.  No thread reads a code; the
// softmax threads write some: rows of V outside the tile (a NaN code there would
// reach the product) are cleared in the stage, before the fence and the arrival
// that hand the product its P.
// Times beside a choice compare it with the alternative on one box at the time it
// was made; what whole launches take now is measured on the finished kernel.
//
//  * Work split and partials: as the bf16 kernel (split_units.cuh); a request's
//    tiles are merged by a kernel of its own.  A CTA streams its pages two at a
//    time: a step is 128 tokens of one kv head.
//  * S = K Q^T: M = 128 tokens, N = 32, K = D.  q (bf16, 8 significant bits) is
//    scaled by a power of two per head and held as four e4m3 parts (4 bits each, and
//    a sign between them): two hold all bits of values down to 2^-14 of the head's
//    largest, two more those down to 2^-24, and 2^-32 of the largest of any.  (Most
//    heads have nothing in the last two, but a K that is large where q is small
//    would show what they lack.)
//  * Softmax: a thread per token, two groups of threads taking every other step,
//    each with its own references and sum.  A head has two running references,
//    multiples of 8 (log2).  One, m, is near the largest score x_j and serves the
//    sum of e_j = 2^(x_j - m), whatever V's scales are.  The other, ref, bounds
//    x_j + log2 sv_j (sv the token's V scale), so w_j = 2^(x_j - ref) sv_j =
//    e_j sv_j 2^(m - ref) lies in [0, 1] and the largest in (2^-8, 1] whatever the
//    scales.  (One reference for both lost keys from the sum where V's scales lay
//    more than 2^126 apart, and small probabilities beside V scales near 2^100.)
//    They move rarely, and then by an exact power of two.  w is held as kParts e4m3
//    parts, each the rounding of what the parts before left, 32 times finer (that
//    stays below 256 = 2^8, as w 2^8 does): a part takes 5 bits (4 and a sign), so a w
//    is within 2^-19 of itself, 3.5e-7 on the root mean square, or within 2^-33 of the
//    row's bound.  What the last part leaves in the first case is summed too, as
//    left_j / sv_j, and taken from the sum that divides the outputs: numerator and
//    denominator have the same probabilities, and a row that hangs on few keys loses
//    nothing to the parts.  (Cutting w to the 19 bits that every w has did the same at
//    twice the error on long rows.)  The log-sum-exp takes the whole sum.
//  * O^T = V^T P^T: M = 128 dims (a step's V codes as they lie, M-major), N =
//    8 kParts (a token's row of P, N-major), K = 128 tokens.  Every step's
//    product starts from zero in tensor memory and is added to fp32 registers (a
//    thread per dim), so the long sum is rounded to nearest and rescaled there.
//  * Warps: 0-7 softmax, 8-11 output, 12 TMA, 13 scores, 14 products, 15 what is
//    done per segment (q, factors of the outputs, empty units); 16 warps leave
//    128 registers a thread, 17 would leave 96.  All waits are on mbarriers
//    with a time limit; S, P and the products have two buffers each.
//    Each product has a warp of its own: with one thread for both, a step of
//    256 dims took 1.4 us, 0.86 us of it the issue of its 16 instructions and
//    the rest waits that did not overlap.  K and V have a ring each, because a
//    K stage is free as soon as its scores are, a V stage a softmax and a
//    product later.
//  * A launch starts under programmatic dependent launch; only what reads or
//    writes global memory waits for the kernels before it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>
#include <vector>

#include "common.h"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "ptx.cuh"
#include "split_units.cuh"
#include "tc.cuh"

namespace pa {
namespace decode_q8 {

using namespace split;

constexpr int kBlock = PA_SCALE_TOKENS;
constexpr int kStep = 2 * kPage;            // tokens per step
constexpr int kStepBlocks = kStep / kBlock;
constexpr int kBlocksPerPage = kPage / kBlock;
constexpr int kParts = 4;                   // e4m3 parts of a probability
constexpr float kFirstPart = 256.f;         // scale of the first part
constexpr float kPartRatio = 32.f;          // of each further one
constexpr float kLastPart = 1.f / (kFirstPart * kPartRatio * kPartRatio * kPartRatio);
constexpr int kPCols = kParts * kMaxG;      // N of the second product
constexpr int kQParts = 4;                  // e4m3 parts of q, each scaled up from the
// one before by these: the second holds what the first leaves of 8 bits, and what
// these two leave, of values below 256, is at most 2^-15.
constexpr float kQScale1 = 32.f, kQScale2 = 1 << 18, kQScale3 = 32.f;
constexpr int kQCols = kQParts * kMaxG;     // N of the first product
// A product of codes of K and q lies below 2^25.  It is multiplied by K's scale (up to
// 2^120) and by a factor per head; this much of the one goes to the other, so that a
// score within range has every step of its product there too.
constexpr int kScaleShift = 17;
constexpr int kChunk = 128;                 // dims per 128-byte row
constexpr int kTmemCols = 256;
constexpr int kRefs = 4;                    // reference slots, two steps more than P buffers
constexpr int kGroups = 2;                  // softmax groups
constexpr int kGroupWarps = 4, kOutWarps = 4;
constexpr int kOut = kOutWarps * 32;
constexpr int kSoftmaxWarps = kGroups * kGroupWarps;
constexpr int kTmaWarp = 12, kScoreWarp = 13, kProductWarp = 14;
constexpr int kThreads = 32 * 16;           // the last warp: per segment
constexpr int kSegmentCharge = 6;           // pages charged per unit start
constexpr int kWholePages = 16;             // units this short are not split while SMs are idle
constexpr int kMinPages = 4;                // pages per CTA at least, where units are split
// A launch of this many pages per SM runs on kLongGridPct percent of the SMs:
// with HBM saturated, fewer and longer streams finish sooner (as the bf16
// kernel's do; 100 / 90 / 85 / 80 percent on one box: 1 x 262,144 tokens 85.3 /
// 84.4 / 83.7 / 83.2 us, 8 ragged of up to 131,072 247.5 / 245.5 / 244.5 / 242.1).
constexpr int kLongPages = 64, kLongGridPct = 85;
constexpr int kTwoPartsBytes = 400 << 10;   // worth what a CTA loses with parts of two units
constexpr int kWholeBytes = 1600 << 10;     // beyond an equal share, for units kept whole
constexpr int kUnitCharge = 3;              // pages that a whole unit costs beside its own
constexpr int kSnapPages = 4;               // how far a CTA's end moves to a unit's border
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kMinScaleExp = -100, kMaxScaleExp = 120;   // log2 of V scales
// e_j may lie above 1, up to 2^kSlack: a sum of 2^30 of them is still finite.
constexpr float kSlack = 96.f;
constexpr float kMaxUnder = 104.f;          // how far ref may lie below m
// A reference before the first score, and of a head whose scores are all -inf.
constexpr float kNoRef = -1e30f;

static_assert(kStep == kGroupWarps * 32 && kChunk == kOut, "a thread per token and per dim");

// A softmax group's references, per head; weight: 2^(m - ref) times the first part's
// scale; by, by_ref: what is relative to m, or ref, is multiplied by at a move; gap:
// ref - m.
struct State {
  float4 minus_m[kMaxG / 4], weight[kMaxG / 4], minus_ref[kMaxG / 4], ref[kMaxG / 4];
  float4 by[kMaxG / 4], by_ref[kMaxG / 4], gap[kMaxG / 4];
};
// Two heads of four.
__device__ __forceinline__ float2 half_of(const float4& x, int i) {
  return i ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
}
constexpr int kStateBytes = sizeof(State);

// Shared memory of a CTA; offsets from a 1024-byte boundary.
template <int D>
struct Smem {
  static constexpr int kChunks = D / kChunk;
  static constexpr int kPageBytes = kPage * kChunk;              // one page, one chunk
  static constexpr int kChunkBytes = 2 * kPageBytes;             // one step, one chunk
  static constexpr int kHalfBytes = kChunks * kChunkBytes;       // K (or V) of a step
  static constexpr int kStages = D == 256 ? 3 : 6;               // of K, and of V
  static constexpr int kV = kStages * kHalfBytes;
  static constexpr int kPBytes = kPCols * kStep;
  static constexpr int kQChunkBytes = kQCols * kChunk;
  static constexpr int kQBytes = kChunks * kQChunkBytes;
  static constexpr int kP = 2 * kV;
  static constexpr int kQ = kP + 2 * kPBytes;
  // Scales come for up to 16 steps at a time, a page of them per lane of the TMA
  // warp.  When those of steps i .. i + 15 are asked for, the K of step i - 1 is,
  // so the scores of step i - 1 - kStages are done, and the softmax of the step
  // two before it has read its scales: 32 slots hold them all.
  static constexpr int kSlots = 32;
  static_assert(kStages + 3 <= 17, "slots of scales");
  static constexpr int kQRaw = kQ + 2 * kQBytes;                 // [head][dim] of a later segment
  static constexpr int kScales = kQRaw + kMaxG * D * 2;          // [slot][K | V][block]
  static constexpr int kScaleBytes = 2 * kStepBlocks * 4;
  static constexpr int kQScale = kScales + kSlots * kScaleBytes;  // [2][kMaxG]
  static constexpr int kRef = kQScale + 2 * kMaxG * 4;             // [kRefs][kMaxG]
  static constexpr int kSegL = kRef + kRefs * kMaxG * 4;    // [2][warp][sums | left][kMaxG]
  // [2][group][m | ref][kMaxG]
  static constexpr int kSegRef = kSegL + 2 * kSoftmaxWarps * 2 * kMaxG * 4;
  // A group's references now (see State), and what a move of them looks at: log2 sv
  // of the step's blocks, and its scores [token][head].  At 256 dims the scores lie in
  // the group's buffer of P, once the product before is done with it; at 128 there is
  // room for one of their own (256 x 512 tokens in a buffer of P 56.4 us, so 54.7).
  static constexpr int kState = kSegRef + 2 * kGroups * 2 * kMaxG * 4;   // [group]
  static constexpr int kUp = kState + kGroups * kStateBytes;             // [group][block]
  static constexpr bool kOwnScores = D == 128;
  static constexpr int kScores = kOwnScores ? kUp + kGroups * kStepBlocks * 4 : kP;
  static constexpr int kScoreBytes = kStep * kMaxG * 4;
  static_assert(kOwnScores || kScoreBytes == kPBytes, "scores in a buffer of P");
  static constexpr int kQs =   // a softmax warp's scales of q: [warp][kMaxG]
      kUp + kGroups * (kStepBlocks * 4 + (kOwnScores ? kScoreBytes : 0));
  // [2][two factors | m | sum][kMaxG]
  static constexpr int kFactor = kQs + kSoftmaxWarps * kMaxG * 4;
  static constexpr int kBars = kFactor + 2 * 4 * kMaxG * 4;
  // mbarriers: full, empty per K and V stage; S, P, product, q, sums: full and
  // empty; all of a warp's products done; reference slots written; a segment's
  // factors: full and empty
  static constexpr int kKFull = 0, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages,
                       kVEmpty = kVFull + kStages, kSFull = kVEmpty + kStages,
                       kSEmpty = kSFull + 2, kPFull = kSEmpty + 2, kOFull = kPFull + 2,
                       kOEmpty = kOFull + 2, kQFull = kOEmpty + 2, kQEmpty = kQFull + 2,
                       kLFull = kQEmpty + 2, kLEmpty = kLFull + 2, kDrain = kLEmpty + 2,
                       kRefFull = kDrain + 2, kFFull = kRefFull + kRefs, kFEmpty = kFFull + 2,
                       kNumBars = kFEmpty + 2;
  static constexpr int kMisc = kBars + kNumBars * 8;               // ints, see View
  static constexpr int kUsed = kMisc + (kSlots + 2 * kGroups + 4) * 4;
  static constexpr int kAlloc = kUsed + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// A unit as the kernel reads it: three 8-byte loads.
struct alignas(8) DevUnit {
  int32_t page_first, bt, tok_start, tok_end, g;
  uint16_t part_base;
  uint8_t n_parts, first_cta;
};

template <int kMaxUnits>
struct Params {
  const __nv_bfloat16* q;
  const float* scales;
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
  float scale_log2;   // times 2^kScaleShift
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
  volatile int* poison;      // [slots] step holds a page that is not there
  volatile int* seg_poison;  // [2][group]
  volatile int* abort_flag;
  volatile int* merge_info;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
};

// A position in a ring of kN buffers and the parity of its barriers' phase: a
// reader waits for `full` with it, a writer for `empty` with the other parity
// (which a fresh barrier passes).
template <int kN>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == kN) {
      i = 0;
      phase ^= 1;
    }
  }
};

// The slow side of a wait, out of line: the roles' loops stay short (a warp on
// its own runs ~6 cycles per instruction, and every line of code is fetched
// cold in a launch).
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                       int32_t* status, volatile int* abort_flag) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > limit_ns) {
      atomicOr(status, PA_STATUS_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

// Waits for the phase of the given parity to be complete.  False once the time
// limit, or another warp's, has run out.
template <class P>
__device__ __forceinline__ bool wait(const P& p, const View& v, int bar, uint32_t parity) {
  const uint32_t b = v.bar(bar);
  return ptx::mbar_try_wait(b, parity) ||
         wait_long(b, parity, p.wait_limit_ns, p.status, v.abort_flag);
}
// The same for a converged warp, with one answer for all its lanes: false too if
// `ok` is false in one of them.  A warp skips tensor memory loads, and leaves its
// loop, by such an answer alone: lanes that gave up by themselves would be missed at
// the next instruction that takes the whole warp, by a wait without a limit.
template <class P>
__device__ __forceinline__ bool warp_wait(const P& p, const View& v, int bar, uint32_t parity,
                                          bool ok = true) {
  return __all_sync(0xffffffffu, ok && wait(p, v, bar, parity));
}

// A CTA's part of a unit: its pages [lo, hi).
struct Segment {
  DevUnit U;
  int u, pf, lo, hi, bt, g, first_tok;
  __device__ __forceinline__ int steps() const { return (hi - lo + 1) / 2; }
  __device__ __forceinline__ bool whole() const { return U.n_parts == 1; }
  // the segment's partial slot, where the unit has several
  __device__ __forceinline__ size_t slot() const {
    return U.part_base + (int)blockIdx.x - U.first_cta;
  }
};

// This CTA's segments, one after the other.
template <class P>
__device__ __forceinline__ int request_of(const P& p, int bt) {
  return p.T == 1 ? bt : bt / p.T;
}

template <class P>
struct Segments {
  const P& p;
  int start, end, u;
  __device__ __forceinline__ explicit Segments(const P& params)
      : p(params), start(params.starts[blockIdx.x]), end(params.starts[blockIdx.x + 1]),
        u(params.first_unit[blockIdx.x]) {}
  __device__ __forceinline__ bool next(Segment& s) {
    for (; u < p.n_full && p.units[u].page_first < end; ++u) {
      const DevUnit& from = p.units[u];
      s.U = from;
      const int np = unit_pages(s.U.tok_start, s.U.tok_end);
      s.pf = s.U.page_first;
      s.lo = max(start, s.pf) - s.pf;
      s.hi = min(end, s.pf + np) - s.pf;
      if (s.hi <= s.lo) continue;   // only its segment charge falls in this range
      s.u = u++;
      s.bt = s.U.bt;
      s.g = s.U.g;
      s.first_tok = s.U.tok_start / kPage * kPage;
      return true;
    }
    return false;
  }
};

// Calls f(segment, index) for every segment of this CTA until f returns false.
template <class P, class F>
__device__ __forceinline__ void for_segments(const P& p, F f) {
  Segments<P> segments(p);
  Segment s;
  for (int index = 0; segments.next(s); ++index)
    if (!f(s, index)) return;
}

__device__ __forceinline__ bool any_in_group(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// One lane of a converged warp.  What a whole warp computes alike stays in
// uniform registers, which TMA and tcgen05 instructions take their operands
// from; a branch on the lane index would cost a move for each.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 16 bytes (copy_own: a value of 8 or 16) from global to shared memory, and an
// arrival at `bar` once the thread's copies have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <class T>
__device__ __forceinline__ void copy_own(uint32_t dst, const T* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(sizeof(T))
               : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------------------
// Warp 12: the pages' K (with the scales) and V into their rings, V kLag steps
// behind K.  At 256 dims (three stages) V follows two steps behind, as a product
// does its scores, and one wait and one branch serve both; at 128 (six stages) it
// follows one step behind, with a wait of its own.  Together / apart: 1 x 262,144
// tokens 82.9 / 84.8 us, 64 x 2,048 41.1 / 41.8, 4 x 31,744 44.7 / 45.0, and at
// 128 dims 16 x 8,192 45.1 / 43.9, 256 x 512 58.2 / 55.9.  (At 128 dims a step
// lasts about as long as this warp's instructions for it.)
// ---------------------------------------------------------------------------
struct StepPages {
  int row0, row1, n, col;   // first rows of its pages in the pool, pages, V's column
};

template <int D, class P>
__device__ __forceinline__ void tma_warp(const P& p, const View& v, const CUtensorMap* tmap,
                                         int lane) {
  using S = Smem<D>;
  constexpr bool kTogether = D == 256;
  constexpr int kLag = kTogether ? 2 : 1;
  Ring<S::kStages> kr, vr;
  Ring<S::kSlots> slot;
  int keys = 0, values = 0;            // steps loaded
  StepPages late[kLag] = {};           // the steps whose V is next
  const uint64_t pol = ptx::policy_evict_first();   // every page is read once
  const int stall = blockIdx.x == 0 ? p.stall_iteration : -1;
  const int stall_values = stall - (int)PA_STALL_VALUES;   // (negative without the flag)
  auto boxes = [&](uint32_t dst, uint32_t full, int col, const StepPages& at) {
    ptx::mbar_arrive_expect_tx(full, at.n * S::kChunks * S::kPageBytes);
#pragma unroll
    for (int c = 0; c < S::kChunks; ++c)
      ptx::tma_load_2d_hint(dst + c * S::kChunkBytes, tmap, col + c * kChunk, at.row0, full, pol);
    if (at.n > 1) {
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
        ptx::tma_load_2d_hint(dst + c * S::kChunkBytes + S::kPageBytes, tmap, col + c * kChunk,
                              at.row1, full, pol);
    }
  };
  auto load_values = [&]() {   // by one lane, into a free stage
    if (values == stall_values) return;
    boxes(v.addr + S::kV + vr.i * S::kHalfBytes, v.bar(S::kVFull + vr.i), late[0].col, late[0]);
  };
  for_segments(p, [&](const Segment& s, int seg) {
    if (seg == 0) ptx::grid_dependency_wait();
    const int32_t* prow =
        p.page_table + (size_t)request_of(p, s.bt) * p.max_pages + s.U.tok_start / kPage;
    const float* scales = p.scales + s.g * kBlocksPerPage;   // K's; V's lie Hkv heads behind
    int next_pid = s.lo + lane < s.hi ? __ldg(prow + s.lo + lane) : 0;
    for (int base = s.lo; base < s.hi; base += 32) {
      const int cnt = min(32, s.hi - base);
      // a page that is not there: page 0 in its place, its step marked
      const bool bad = lane < cnt && (uint32_t)next_pid >= (uint32_t)p.pool_pages;
      const uint32_t bad_pages = __ballot_sync(0xffffffffu, bad);
      const int my_pid = bad ? 0 : next_pid;
      if (bad) atomicOr(p.status, PA_STATUS_BAD_PAGE);
      if (lane < cnt) {
        const float* src = scales + (size_t)my_pid * (2 * p.Hkv * kBlocksPerPage);
        const uint32_t dst = v.addr + S::kScales +
                             (keys + (lane >> 1)) % S::kSlots * S::kScaleBytes + (lane & 1) * 16;
        copy16(dst, src);
        copy16(dst + kStepBlocks * 4, src + p.Hkv * kBlocksPerPage);
      }
      if (base + 32 + lane < s.hi) next_pid = __ldg(prow + base + 32 + lane);
      for (int j = 0; j < cnt; j += 2) {
        const StepPages now = {__shfl_sync(0xffffffffu, my_pid, j) * kPage,
                               __shfl_sync(0xffffffffu, my_pid, (j + 1) & 31) * kPage,
                               min(2, cnt - j), (p.Hkv + s.g) * D};
        const bool with_values = keys >= kLag;
        if constexpr (kTogether) {
          const int kbar = S::kKEmpty + kr.i, vbar = with_values ? S::kVEmpty + vr.i : kbar;
          const uint32_t kpar = kr.phase ^ 1, vpar = with_values ? vr.phase ^ 1 : kpar;
          const bool kfree = ptx::mbar_try_wait(v.bar(kbar), kpar);
          const bool vfree = ptx::mbar_try_wait(v.bar(vbar), vpar);
          if (!__all_sync(0xffffffffu, kfree && vfree) &&
              (!warp_wait(p, v, kbar, kpar) || !warp_wait(p, v, vbar, vpar)))
            return false;
        } else {
          if (!warp_wait(p, v, S::kKEmpty + kr.i, kr.phase ^ 1)) return false;
        }
        const uint32_t full = v.bar(S::kKFull + kr.i);
        if (keys != stall) {
          if (elect()) {
            v.poison[slot.i] = (bad_pages >> j) & 3;   // set before the arrival that publishes it
            boxes(v.addr + kr.i * S::kHalfBytes, full, s.g * D, now);
            if (kTogether && with_values) load_values();
          }
        } else if (kTogether && with_values && elect()) {
          load_values();
        }
        arrive_after_copies(full);   // every lane's scales (of this step and earlier ones)
        __syncwarp();
        kr.next();
        slot.next();
        ++keys;
        if (with_values) {
          if constexpr (!kTogether) {
            if (!warp_wait(p, v, S::kVEmpty + vr.i, vr.phase ^ 1)) return false;
            if (elect()) load_values();
            __syncwarp();
          }
          vr.next();
          ++values;
        }
        if (kLag > 1) late[0] = late[kLag - 1];
        late[kLag - 1] = now;
      }
    }
    return true;
  });
  if (keys < kLag) late[0] = late[kLag - 1];
  while (values < keys && warp_wait(p, v, S::kVEmpty + vr.i, vr.phase ^ 1)) {
    if (elect()) load_values();
    __syncwarp();
    vr.next();
    ++values;
    late[0] = late[kLag - 1];
  }
  // Every page of this CTA is requested: the next kernel in the stream may
  // start its prologue.
  if (lane == 0) ptx::launch_dependents();
  // The copies issued land before the CTA can exit, whatever became of the
  // other warps.
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int k = max(0, keys - S::kStages); k < keys; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kKFull + k % S::kStages), (k / S::kStages) & 1,
                           p.wait_limit_ns);
  for (int k = max(0, values - S::kStages); k < values; ++k)
    ptx::mbar_wait_bounded(v.bar(S::kVFull + k % S::kStages), (k / S::kStages) & 1,
                           p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Warp 13: scores.  Warp 14: products with V.
// ---------------------------------------------------------------------------
// Every product this warp issued, and every arrival that follows from one,
// ends before the CTA can.
template <class P>
__device__ __forceinline__ void drain(const P& p, const View& v, int bar) {
  if (elect()) tc::commit(v.bar(bar));
  __syncwarp();
  ptx::mbar_wait_bounded(v.bar(bar), 0, p.wait_limit_ns);
}

template <int D, class P>
__device__ __forceinline__ void score_warp(const P& p, const View& v, uint32_t tmem) {
  using S = Smem<D>;
  constexpr uint32_t kIdesc = tc::idesc_e4m3(kStep, kQCols, false, false);
  Ring<S::kStages> kr;
  Ring<2> sr, qr;
  for_segments(p, [&](const Segment& s, int) {
    if (!warp_wait(p, v, S::kQFull + qr.i, qr.phase)) return false;
    const uint64_t b = tc::desc_sw128(v.addr + S::kQ + qr.i * S::kQBytes);
    for (int left = s.steps(); left > 0; --left) {
      if (!warp_wait(p, v, S::kSEmpty + sr.i, sr.phase ^ 1) ||
          !warp_wait(p, v, S::kKFull + kr.i, kr.phase))
        return false;
      tc::fence_after();
      const uint64_t a = tc::desc_sw128(v.addr + kr.i * S::kHalfBytes);
      if (elect()) {
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_e4m3(tmem + sr.i * kQCols, a + (c * S::kChunkBytes >> 4) + 2 * k,
                         b + (c * S::kQChunkBytes >> 4) + 2 * k, kIdesc, c + k > 0);
        }
        tc::commit(v.bar(S::kSFull + sr.i));
        tc::commit(v.bar(S::kKEmpty + kr.i));
        // and an arrival of its own: the scales and the mark that came with K,
        // whose barrier may be phases ahead by the time softmax looks
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

template <int D, class P>
__device__ __forceinline__ void product_warp(const P& p, const View& v, uint32_t tmem) {
  using S = Smem<D>;
  constexpr uint32_t kIdesc = tc::idesc_e4m3(kChunk, kPCols, true, true);
  // 32 tokens of a chunk, and of the probabilities, in descriptor units
  constexpr uint32_t kSlice = 32 * kChunk >> 4, kPSlice = 32 * kPCols >> 4;
  Ring<S::kStages> vr;
  Ring<2> pr;
  for_segments(p, [&](const Segment& s, int) {
    for (int page = s.lo; page < s.hi; page += 2) {
      const bool two = page + 1 < s.hi;   // both pages of the step are there
      if (!warp_wait(p, v, S::kOEmpty + pr.i, pr.phase ^ 1) ||
          !warp_wait(p, v, S::kVFull + vr.i, vr.phase) ||
          !warp_wait(p, v, S::kPFull + pr.i, pr.phase))
        return false;
      tc::fence_after();
      const uint64_t a = tc::desc_sw128(v.addr + S::kV + vr.i * S::kHalfBytes);
      const uint64_t b = tc::desc_sw32(v.addr + S::kP + pr.i * S::kPBytes);
      const uint32_t d = tmem + 2 * kQCols + pr.i * S::kChunks * kPCols;
      if (elect()) {
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c) {
          const uint64_t ac = a + (c * S::kChunkBytes >> 4);
          tc::mma_e4m3(d + c * kPCols, ac, b, kIdesc, false);
          tc::mma_e4m3(d + c * kPCols, ac + kSlice, b + kPSlice, kIdesc, true);
          if (two) {
            tc::mma_e4m3(d + c * kPCols, ac + 2 * kSlice, b + 2 * kPSlice, kIdesc, true);
            tc::mma_e4m3(d + c * kPCols, ac + 3 * kSlice, b + 3 * kPSlice, kIdesc, true);
          }
        }
        tc::commit(v.bar(S::kOFull + pr.i));
        tc::commit(v.bar(S::kVEmpty + vr.i));
      }
      __syncwarp();
      vr.next();
      pr.next();
    }
    return true;
  });
  drain(p, v, S::kDrain + 1);
}

// ---------------------------------------------------------------------------
// q of a segment as hi and lo parts, and its scales: by the output warps, two
// heads each, for a CTA's first segment (on one warp it takes 3.7 us, the
// longest part of a launch's start), by warp 15 ahead of time for the others.
// That warp loops over the heads, from shared memory: code that runs once per
// segment is fetched anew each time, and eight heads unrolled were 11 KB of it
// (252 requests of 103 / 256 tokens 27.2 / 30.8 -> 23.8 / 26.7 us).
// ---------------------------------------------------------------------------
template <int D>
using QVec = typename std::conditional<D == 256, uint4, uint2>::type;   // D / 32 dims per lane

// A lane's dims of head h of a segment.
template <int D, class P>
__device__ __forceinline__ const QVec<D>* q_of(const P& p, const Segment& s, int h, int lane) {
  return reinterpret_cast<const QVec<D>*>(
      p.q + ((size_t)request_of(p, s.bt) * p.Hq + s.g * p.G + h) * D + lane * (D / 32));
}

__device__ __forceinline__ void store_shared(uint32_t at, const uint32_t (&x)[1]) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x[0]) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint32_t (&x)[2]) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x[0]), "r"(x[1]) : "memory");
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
  return *reinterpret_cast<const __nv_bfloat162*>(&x);
}

// A head of q, as its four parts, into a buffer.  (All four of every head: most heads
// have nothing in the last two, but a test for that and its branch took as long, 252
// requests of 103 tokens 24.8 us with and 24.7 without.)
template <int D, class P>
__device__ __forceinline__ void convert_head(const P& p, const View& v, const QVec<D>& raw,
                                             int buffer, int h, int lane) {
  using S = Smem<D>;
  constexpr int kDims = D / 32;             // dims per lane
  const int col = lane * kDims;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
  __nv_bfloat162 most = __habs2(as_bf162(w[0]));   // NaN if there is one
#pragma unroll
  for (int k = 1; k < kDims / 2; ++k) most = __hmax2_nan(most, __habs2(as_bf162(w[k])));
  const unsigned amax = __reduce_max_sync(
      0xffffffffu, __bfloat16_as_ushort(__hmax_nan(__low2bfloat16(most), __high2bfloat16(most))));
  // Largest value to [128, 256).  A head with a NaN or an infinity becomes
  // NaN (its scores would be).
  const int e = amax ? min(7 - ((int)(amax >> 7) - 127), 120) : 0;
  const float up = amax < 0x7f80u ? ptx::pow2i(e) : __int_as_float(0x7fc00000);
  if (lane == 0)
    reinterpret_cast<float*>(v.base + S::kQScale)[buffer * kMaxG + h] =
        p.scale_log2 * ptx::pow2i(-e);
  // z = q * up is exact in fp16 down to steps of 2^-24, and so is what each part leaves.
  uint32_t code[kQParts][kDims / 4];
#pragma unroll
  for (int k = 0; k < kDims / 2; ++k) {
    auto take = [&](int part, __half2 x) {   // returns what the part leaves
      const uint32_t c = fp8::pack2(x);
      uint32_t& to = code[part][k / 2];
      to = k % 2 ? to | c << 16 : c;
      return __hsub2(x, fp8::unpack2_half(c));
    };
    __half2 z = __floats2half2_rn(ptx::bf16_lo_to_f32(w[k]) * up,
                                  ptx::bf16_hi_to_f32(w[k]) * up);
    z = take(1, __hmul2(take(0, z), __float2half2_rn(kQScale1)));
    const __half2 by = __float2half2_rn(512.f);   // 2^18 in two factors: fp16 ends at 2^16
    z = take(2, __hmul2(__hmul2(z, by), by));
    take(3, __hmul2(z, __float2half2_rn(kQScale3)));
  }
  const uint32_t at = v.addr + S::kQ + buffer * S::kQBytes + col / kChunk * S::kQChunkBytes +
                      (col & 15) + h * kChunk + (((col % kChunk >> 4) ^ h) << 4);
#pragma unroll
  for (int part = 0; part < kQParts; ++part)
    store_shared(at + part * kMaxG * kChunk, code[part]);
}

// ---------------------------------------------------------------------------
// Warp 15: what is not done per step: q ahead of its segment, the factors of a
// segment's outputs (and its log-sum-exp) from its sums, and empty units.
// ---------------------------------------------------------------------------
// slot: the segment's partial slot, negative where it is a whole unit.
template <int D, class P>
__device__ __forceinline__ bool segment_factors(const P& p, const View& v, int slot, Ring<2>& r,
                                                int lane) {
  using S = Smem<D>;
  if (!warp_wait(p, v, S::kFEmpty + r.i, r.phase ^ 1) ||
      !warp_wait(p, v, S::kLFull + r.i, r.phase))
    return false;
  const float* seg_l = reinterpret_cast<const float*>(v.base + S::kSegL) +
                       r.i * kSoftmaxWarps * 2 * kMaxG;
  const float* sr = reinterpret_cast<const float*>(v.base + S::kSegRef) +
                    r.i * kGroups * 2 * kMaxG;
  float* factor = reinterpret_cast<float*>(v.base + S::kFactor) + r.i * 4 * kMaxG;
  const bool nan = (v.seg_poison[r.i * kGroups] | v.seg_poison[r.i * kGroups + 1]) != 0;
  if (lane < kMaxG) {
    const float qnan = __int_as_float(0x7fc00000);
    float m = kNoRef, ref = kNoRef, l = 0.f, left = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      m = fmaxf(m, sr[g * 2 * kMaxG + lane]);
      ref = fmaxf(ref, sr[(g * 2 + 1) * kMaxG + lane]);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float* w = seg_l + g * kGroupWarps * 2 * kMaxG + lane;
      const float a = ref_weight(sr[g * 2 * kMaxG + lane], m);
      l = fmaf(a, (w[0] + w[2 * kMaxG]) + (w[4 * kMaxG] + w[6 * kMaxG]), l);
      w += kMaxG;
      left = fmaf(ref_weight(sr[(g * 2 + 1) * kMaxG + lane], ref),
                  (w[0] + w[2 * kMaxG]) + (w[4 * kMaxG] + w[6 * kMaxG]), left);
    }
    // The sum of products is relative to ref; the output, or the partial, to the sum's
    // own magnitude 2^(m + k), with l 2^-k in (2^-8, 1].  (Two factors: 2^(ref - m - k)
    // may be as large as the largest V scale.)
    const int k = l > 0.f ? ((__float_as_int(l) >> 23) - 127 + 8) >> 3 << 3 : 0;
    const int by = max(-240, min(240, (int)(ref - m) - k));
    l *= ptx::pow2i(max(-126, -k));
    const float f1 = ptx::pow2i(by >> 1), f2 = ptx::pow2i(by - (by >> 1));
    float f = f2 / (l - left * kLastPart * f1 * f2);
    if (slot < 0) {
      // for the log-sum-exp, which the output warps take from these
      factor[2 * kMaxG + lane] = m + (float)k;
      factor[3 * kMaxG + lane] = nan ? qnan : l;
    } else {
      reinterpret_cast<float2*>(p.part_ml)[(size_t)slot * kMaxG + lane] =
          make_float2(nan ? qnan : m + (float)k, l);
      f *= l;   // a partial's products belong to the sum that the merge divides by
    }
    factor[lane] = f1;
    factor[kMaxG + lane] = nan ? qnan : f;
  }
  __syncwarp();
  if (lane == 0) {
    ptx::mbar_arrive(v.bar(S::kLEmpty + r.i));
    ptx::mbar_arrive(v.bar(S::kFFull + r.i));
  }
  r.next();
  return true;
}

template <int D, class P>
__device__ __forceinline__ void helper_warp(const P& p, const View& v, int lane) {
  using S = Smem<D>;
  Ring<2> qr, fr;
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
  // q is loaded two segments ahead (a lane's dims by that lane, so no lane waits
  // for another) and converted one ahead (the first segment's by the output warps).
  constexpr int kNone = -2, kWholeUnit = -1;
  Segments<P> ahead(p);
  Segment s;
  QVec<D>* staged = reinterpret_cast<QVec<D>*>(v.base + S::kQRaw) + lane;   // [head][lane]
  // The next segment's partial slot.
  auto take = [&]() {
    if (!ahead.next(s)) return kNone;
    return s.whole() ? kWholeUnit : (int)s.slot();
  };
  auto take_and_load = [&]() {
    const int slot = take();
    if (slot == kNone) return slot;
#pragma unroll 1
    for (int h = 0; h < p.G; ++h)
      copy_own(ptx::smem_addr(staged + 32 * h), q_of<D>(p, s, h, lane));
    return slot;
  };
  int now = take();
  if (now == kNone) return;
  int next = take_and_load();
  for (int heads = kMaxG;;) {
    // q of `next`, and that of the segment behind it is asked for
    int later = kNone;
    qr.next();
    if (next != kNone) {
      const bool free = warp_wait(p, v, S::kQEmpty + qr.i, qr.phase ^ 1);
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!free) return;
#pragma unroll 1
      for (int h = 0; h < heads; ++h)
        convert_head<D>(p, v, h < p.G ? staged[32 * h] : QVec<D>{}, qr.i, h, lane);
      heads = p.G;   // the first conversion clears the columns without a head
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane < kOutWarps) ptx::mbar_arrive(v.bar(S::kQFull + qr.i));
      later = take_and_load();
    }
    const bool done = segment_factors<D>(p, v, now, fr, lane);
    if (!done || next == kNone) {   // (copies asked for may be in flight where it gave up)
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;
    }
    now = next;
    next = later;
  }
}

__device__ __forceinline__ float warp_max(float x) {   // (NaN ignored)
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// A word of x's bytes' bits 7, each copied through a byte (kSelect: prmt's, with its
// sign bits).
template <int kSelect>
__device__ __forceinline__ uint32_t sign_bytes(uint32_t x) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "n"(kSelect));
  return r;
}

// ---------------------------------------------------------------------------
// Warps 0-3 and 4-7: a thread per token of every other step.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void softmax_warps(const P& p, const View& v, uint32_t tmem, int group,
                                              int warp, int lane) {
  using S = Smem<D>;
  const int barrier = 2 + 2 * group;
  const int tok = warp * 32 + lane;
  int it = 0;
  bool fail = false;   // of this lane; the wait for a step's scores asks all of the warp
  State& st = reinterpret_cast<State*>(v.base + S::kState)[group];
  float* ups = reinterpret_cast<float*>(v.base + S::kUp) + group * kStepBlocks;
  float* scores = reinterpret_cast<float*>(v.base + S::kScores + group * S::kScoreBytes);
  float* qs = reinterpret_cast<float*>(v.base + S::kQs) + (group * kGroupWarps + warp) * kMaxG;
  for_segments(p, [&](const Segment& s, int seg) {
    // Tokens whose log2 sv is below `lowest` might lie above m by more than kSlack.
    float2 l[kMaxG / 2], left[kMaxG / 2];
    float lowest = 0.f;
    fail |= !wait(p, v, S::kQFull + (seg & 1), (seg >> 1) & 1);
    if (lane < kMaxG) {
      const float x = reinterpret_cast<const float*>(v.base + S::kQScale)[(seg & 1) * kMaxG + lane];
      qs[lane] = fminf(fmaxf(x, -FLT_MAX), FLT_MAX);   // (infinite for |q| above 2^113)
    }
#pragma unroll
    for (int h = 0; h < kMaxG / 2; ++h) l[h] = left[h] = f32x2::both(0.f);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQEmpty + (seg & 1)));
    int poisoned = 0;
    bool first = true;
    const int steps = s.steps();
    for (int i = 0; i < steps; ++i, ++it) {
      if ((it & 1) != group) continue;
      const uint32_t phase = (it >> 1) & 1;
      const int slot = it % S::kSlots;
      const int tok0 = s.first_tok + (s.lo + 2 * i) * kPage;
      const int pages = min(2, s.hi - (s.lo + 2 * i));
      const bool loaded = tok < pages * kPage;
      const bool live = loaded && tok0 + tok >= s.U.tok_start && tok0 + tok < s.U.tok_end;
      float2 x[kMaxG / 2];
      float sv = 0.f, up = 0.f;
      fail = !warp_wait(p, v, S::kSFull + group, phase, !fail);
      if (!fail) {
        const float* sc = reinterpret_cast<const float*>(v.base + S::kScales +
                                                         slot * S::kScaleBytes);
        const float sk = sc[tok / kBlock] * ptx::pow2i(-kScaleShift);
        sv = sc[kStepBlocks + tok / kBlock];
        if (tok == 0) poisoned |= v.poison[slot];
        tc::fence_after();
        uint32_t r[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          tc::ld16(tmem + group * kQCols + 16 * k + ((uint32_t)(warp * 32) << 16), r[k]);
#pragma unroll
        for (int k = 0; k < 2; ++k) tc::wait_ld(r[k]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(v.bar(S::kSEmpty + group));
        // 2^up >= |sv| (a scale of zero weighs nothing)
        const unsigned sb = __float_as_uint(sv) & 0x7fffffffu;
        up = (float)max(min((int)(sb >> 23) - 127 + ((sb & 0x7fffffu) ? 1 : 0), kMaxScaleExp),
                        kMinScaleExp);
        if (sb == 0) up = kNoRef;
        if (sb > __float_as_uint(ptx::pow2i(kMaxScaleExp))) sv = __int_as_float(0x7fc00000);
        if (!live) sv = 0.f;   // whatever its row holds
#pragma unroll
        for (int k = 0; k < kMaxG / 4; ++k) {
          const float4 q4 = reinterpret_cast<const float4*>(qs)[k];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = 2 * k + i;
            auto part = [&](int n) {
              const int col = n * kMaxG + 2 * h;
              return make_float2(__uint_as_float(r[col / 16][col % 16]),
                                 __uint_as_float(r[col / 16][col % 16 + 1]));
            };
            float2 d = f32x2::fma(part(3), f32x2::both(1.f / kQScale3), part(2));
            d = f32x2::fma(d, f32x2::both(1.f / kQScale2), part(1));
            d = f32x2::fma(d, f32x2::both(1.f / kQScale1), part(0));
            x[h] = f32x2::mul(f32x2::mul(d, f32x2::both(sk)), half_of(q4, i));
          }
        }
        if (pages < 2 || tok0 < s.U.tok_start || tok0 + kStep > s.U.tok_end) {
#pragma unroll
          for (int h = 0; h < kMaxG / 2; ++h)
            if (!live) x[h] = f32x2::both(-INFINITY);
        }
      }
      bool move = first;
      if (!move) {
        // A token above a ref, or one that might lie too far above an m?
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxG / 4; ++k) {
          const float4 r4 = st.minus_ref[k];
          const float2 a = f32x2::add(x[2 * k], half_of(r4, 0));
          const float2 b = f32x2::add(x[2 * k + 1], half_of(r4, 1));
          most = fmaxf(most, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)));
        }
        move = any_in_group(barrier, kStep, fail || most > -up || (live && up < lowest));
      }
      if (move) {
        // The references move.
        if (!S::kOwnScores) fail |= !wait(p, v, S::kOFull + group, phase ^ 1);
        if (tok % kBlock == 0) ups[tok / kBlock] = up;
#pragma unroll
        for (int k = 0; k < kMaxG / 4; ++k)
          reinterpret_cast<float4*>(scores + tok * kMaxG)[k] =
              make_float4(x[2 * k].x, x[2 * k].y, x[2 * k + 1].x, x[2 * k + 1].y);
        if (any_in_group(barrier + 1, kStep, fail)) return false;
        // A warp looks at two heads, a lane at every 32nd token.
        float a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = b[i] = -INFINITY;   // largest x, and x + log2 sv (NaN ignored)
#pragma unroll
          for (int k = 0; k < kStep / 32; ++k) {
            const float y = scores[(lane + 32 * k) * kMaxG + 2 * warp + i];
            a[i] = fmaxf(a[i], y);
            b[i] = fmaxf(b[i], y + ups[(lane + 32 * k) / kBlock]);
          }
          a[i] = warp_max(a[i]);
          b[i] = warp_max(b[i]);
        }
        if (lane < 2) {
          const int h = 2 * warp + lane;
          const float top = lane ? a[1] : a[0], top_sv = lane ? b[1] : b[0];
          auto at = [&](void* f) -> float& { return reinterpret_cast<float*>(f)[h]; };
          const float old = first ? kNoRef : -at(st.minus_m), m = fmaxf(old, ref_ceil(top));
          const float had = first ? kNoRef : -at(st.minus_ref);
          const float ref = fmaxf(fmaxf(had, ref_ceil(top_sv)), m - kMaxUnder);
          at(st.minus_m) = -m;
          at(st.minus_ref) = -ref;
          at(st.ref) = ref;
          at(st.weight) = kFirstPart * ptx::pow2i((int)(m - ref));
          at(st.by) = ref_weight(old, m);
          at(st.by_ref) = ref_weight(had, ref);
          // (a head without a reference yet looks at every token)
          at(st.gap) = m == kNoRef ? -kNoRef : ref - m;
        }
        ptx::named_barrier(barrier, kStep);
        lowest = kNoRef;
#pragma unroll
        for (int k = 0; k < kMaxG / 4; ++k) {
          const float4 g = st.gap[k], a = st.by[k], b = st.by_ref[k];
          lowest = fmaxf(lowest, fmaxf(fmaxf(g.x, g.y), fmaxf(g.z, g.w)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[2 * k + i] = f32x2::mul(l[2 * k + i], half_of(a, i));
            left[2 * k + i] = f32x2::mul(left[2 * k + i], half_of(b, i));
          }
        }
        lowest -= kSlack;
        first = false;
      }
      uint32_t codes[2 * kParts];   // this token's row: kParts times the eight heads
      __half2 last[kMaxG / 2];      // what the last part rounds
#pragma unroll
      for (int k = 0; k < kMaxG / 4; ++k) {
        const float4 m4 = st.minus_m[k], w4 = st.weight[k];
        float2 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = 2 * k + i;
          const float2 y = f32x2::add(x[h], half_of(m4, i));
          const float2 e = make_float2(ptx::ex2(y.x), ptx::ex2(y.y));
          l[h] = f32x2::add(l[h], e);
          w[i] = f32x2::mul(f32x2::mul(e, f32x2::both(sv)), half_of(w4, i));
        }
#pragma unroll
        for (int part = 0; part + 1 < kParts; ++part) {
          codes[2 * part + k] = fp8::pack4(w[0].x, w[0].y, w[1].x, w[1].y);
#pragma unroll
          for (int i = 0; i < 2; ++i)   // and w becomes (w - code) kPartRatio
            w[i] = f32x2::fma(fp8::unpack2(codes[2 * part + k] >> 16 * i), f32x2::both(-kPartRatio),
                              f32x2::mul(w[i], f32x2::both(kPartRatio)));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)     // (exact: 10 bits are left)
          last[2 * k + i] = __floats2half2_rn(w[i].x, w[i].y);
        codes[2 * kParts - 2 + k] = fp8::pack4(last[2 * k], last[2 * k + 1]);
      }
      // Step it - 2's product is done: its P buffer is free, and so is the
      // reference slot of step it - 4 (the product waited for the output warps
      // to be through with that step).
      fail = !wait(p, v, S::kOFull + group, phase ^ 1);
      const uint32_t prow = v.addr + S::kP + group * S::kPBytes + tok * kPCols;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                         prow + ((half << 4) ^ ((tok & 4) << 2))),
                     "r"(codes[4 * half]), "r"(codes[4 * half + 1]), "r"(codes[4 * half + 2]),
                     "r"(codes[4 * half + 3])
                     : "memory");
      if (loaded && !live) {
        // A NaN code in a row outside the tile would reach the product (0 x NaN).
        const int stage = it % S::kStages;
        fail |= !wait(p, v, S::kVFull + stage, (it / S::kStages) & 1);
        const uint32_t row = v.addr + S::kV + stage * S::kHalfBytes + tok * kChunk;
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c)
          for (int k = 0; k < kChunk; k += 16)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             row + c * S::kChunkBytes + k),
                         "r"(0u)
                         : "memory");
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(v.bar(S::kPFull + group));
      // What is left of the w that have all 19 bits, 2^-6 and more: their first part's
      // exponent is not zero.  (The parts of smaller ones end at a step of their own; where
      // V's scale is small that is a large share of a probability, which counts in full.)
      const float inv = fabsf(sv) >= ptx::pow2i(kMinScaleExp) ? __fdividef(1.f, sv) : 0.f;
#pragma unroll
      for (int k = 0; k < kMaxG / 4; ++k) {
        const uint32_t normal = (codes[k] & 0x78787878u) + 0x78787878u;   // in each byte's bit 7
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = 2 * k + i;
          const __half2 rest = __hsub2(
              last[h], fp8::unpack2_half(codes[2 * kParts - 2 + k] >> 16 * i));
          const uint32_t bits = *reinterpret_cast<const uint32_t*>(&rest) &
                                (i ? sign_bytes<0xbbaa>(normal) : sign_bytes<0x9988>(normal));
          left[h] = f32x2::fma(__half22float2(*reinterpret_cast<const __half2*>(&bits)),
                               f32x2::both(inv), left[h]);
        }
      }
      // (behind P, as the above: the output warps need it a product later)
      if (tok == 0) {
        float4* to = reinterpret_cast<float4*>(v.base + S::kRef) + (it % kRefs) * (kMaxG / 4);
#pragma unroll
        for (int k = 0; k < kMaxG / 4; ++k) to[k] = st.ref[k];
        ptx::mbar_arrive(v.bar(S::kRefFull + it % kRefs));
      }
    }
    // ---- the segment's sums, references and poison to the output warps ----
    fail |= !wait(p, v, S::kLEmpty + (seg & 1), ((seg >> 1) & 1) ^ 1);
    float* seg_l = reinterpret_cast<float*>(v.base + S::kSegL) +
                   ((seg & 1) * kSoftmaxWarps + group * kGroupWarps + warp) * 2 * kMaxG;
    // Eight sums of both kinds over 32 lanes: each exchange halves the heads a lane
    // holds, the last two add lanes of one head.
    float2 sum[kMaxG];
#pragma unroll
    for (int h = 0; h < kMaxG / 2; ++h) {
      sum[2 * h] = make_float2(l[h].x, left[h].x);
      sum[2 * h + 1] = make_float2(l[h].y, left[h].y);
    }
#pragma unroll
    for (int n = kMaxG / 2; n; n >>= 1) {
      const bool upper = lane & (4 * n);
#pragma unroll
      for (int h = 0; h < n; ++h) {
        const float2 give = upper ? sum[h] : sum[h + n], keep = upper ? sum[h + n] : sum[h];
        sum[h] = f32x2::add(keep, make_float2(__shfl_xor_sync(0xffffffffu, give.x, 4 * n),
                                              __shfl_xor_sync(0xffffffffu, give.y, 4 * n)));
      }
    }
#pragma unroll
    for (int n = 1; n < 4; n <<= 1)
      sum[0] = f32x2::add(sum[0], make_float2(__shfl_xor_sync(0xffffffffu, sum[0].x, n),
                                              __shfl_xor_sync(0xffffffffu, sum[0].y, n)));
    if ((lane & 3) == 0) {
      seg_l[lane >> 2] = sum[0].x;
      seg_l[kMaxG + (lane >> 2)] = sum[0].y;
    }
    if (tok == 0) {
      float4* sr = reinterpret_cast<float4*>(v.base + S::kSegRef) +
                   ((seg & 1) * kGroups + group) * 2 * (kMaxG / 4);
      const float4 none = make_float4(kNoRef, kNoRef, kNoRef, kNoRef);
#pragma unroll
      for (int k = 0; k < kMaxG / 4; ++k) {
        const float4 m = st.minus_m[k];
        sr[k] = first ? none : make_float4(-m.x, -m.y, -m.z, -m.w);
        sr[kMaxG / 4 + k] = first ? none : st.ref[k];
      }
      v.seg_poison[(seg & 1) * kGroups + group] = poisoned;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kLFull + (seg & 1)));
    return true;
  });
}

// ---------------------------------------------------------------------------
// Warps 8-11: a thread per dim of each chunk.
// ---------------------------------------------------------------------------
template <int D, class P>
__device__ __forceinline__ void output_warps(const P& p, const View& v, uint32_t tmem, int warp,
                                             int lane) {
  using S = Smem<D>;
  const int ct = warp * 32 + lane;
  ptx::grid_dependency_wait();   // earlier kernels write q and may still read the outputs
  for_segments(p, [&](const Segment& s, int) {
    constexpr int kHeads = kMaxG / kOutWarps;
    QVec<D> raw[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      raw[i] = QVec<D>{};
      if (warp * kHeads + i < p.G) raw[i] = __ldg(q_of<D>(p, s, warp * kHeads + i, lane));
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) convert_head<D>(p, v, raw[i], 0, warp * kHeads + i, lane);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kQFull));
    return false;   // the first segment's
  });
  int it = 0;
  for_segments(p, [&](const Segment& s, int seg) {
    float acc[S::kChunks][kMaxG], ref[kMaxG];
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
      ref[h] = kNoRef;
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c) acc[c][h] = 0.f;
    }
    bool fail = false;
    const int steps = s.steps();
    for (int i = 0; i < steps; ++i, ++it) {
      // A slot is written again four steps on, behind a product that waits
      // for this step's buffer.
      fail = !warp_wait(p, v, S::kOFull + (it & 1), (it >> 1) & 1,
                        wait(p, v, S::kRefFull + it % kRefs, (it / kRefs) & 1));
      if (fail) break;
      const float4* slot = reinterpret_cast<const float4*>(v.base + S::kRef) +
                           (it % kRefs) * (kMaxG / 4);
      const float4 lo = slot[0], hi = slot[1];
      float by[kMaxG] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      bool same = true;
#pragma unroll
      for (int h = 0; h < kMaxG; ++h) {
        if (i == 0) ref[h] = by[h];   // the segment's first
        same = same && by[h] == ref[h];
      }
      if (same) {
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) by[h] = 1.0f / kFirstPart;
      } else {
        // The two groups' references move apart: the sum keeps the largest seen
        // (a rescale where a slot is above it) and weighs each step's product.
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) {
          const float to = fmaxf(ref[h], by[h]);
          const float a = ref_weight(ref[h], to);
#pragma unroll
          for (int c = 0; c < S::kChunks; ++c) acc[c][h] *= a;
          by[h] = ref_weight(by[h], to) * (1.0f / kFirstPart);
          ref[h] = to;
        }
      }
      tc::fence_after();
      const uint32_t d = tmem + 2 * kQCols + (it & 1) * S::kChunks * kPCols +
                         ((uint32_t)(warp * 32) << 16);
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c) {
        uint32_t r[kPCols / 16][16];
#pragma unroll
        for (int k = 0; k < kPCols / 16; ++k) tc::ld16(d + c * kPCols + 16 * k, r[k]);
#pragma unroll
        for (int k = 0; k < kPCols / 16; ++k) tc::wait_ld(r[k]);
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) {
          float sum = 0.f;
#pragma unroll
          for (int part = kParts - 1; part >= 0; --part) {
            const int col = part * kMaxG + h;
            sum = fmaf(sum, 1.0f / kPartRatio, __uint_as_float(r[col / 16][col % 16]));
          }
          acc[c][h] = fmaf(sum, by[h], acc[c][h]);
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(v.bar(S::kOEmpty + (it & 1)));
    }
    fail = fail || !wait(p, v, S::kFFull + (seg & 1), (seg >> 1) & 1);
    if (any_in_group(1, kOut, fail)) return false;
    // ---- the segment's output or partial ----
    const float* factor = reinterpret_cast<const float*>(v.base + S::kFactor) +
                          (seg & 1) * 4 * kMaxG;
    float m = 0.f, l = 0.f;
    const bool has_lse = s.whole() && warp == 0 && lane < p.G;
    if (has_lse) {
      m = factor[2 * kMaxG + lane];
      l = factor[3 * kMaxG + lane];
    }
    const size_t orow = (size_t)s.bt * p.Hq + s.g * p.G;
    float* dst = (s.whole() ? p.out + orow * D : p.part_o + s.slot() * kMaxG * D) + ct;
    float* dst2 = s.whole() && p.out2 ? p.out2 + orow * D + ct : nullptr;
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
      if (h >= p.G) break;
      const float f = factor[h], f2 = factor[kMaxG + h];
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c) {
        const float y = acc[c][h] * f * f2;
        dst[h * D + c * kChunk] = y;
        if (dst2) dst2[h * D + c * kChunk] = y;
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(v.bar(S::kFEmpty + (seg & 1)));
    if (has_lse) {
      const float x = lse_of(m, l);
      p.lse[orow + lane] = x;
      if (p.lse2) p.lse2[orow + lane] = x;
    }
    if (!s.whole()) {
      Unit U{};
      U.n_parts = s.U.n_parts;
      U.part_base = s.U.part_base;
      finish_split_unit<D, kOut>(p, v, U, s.u, 0, s.bt, s.g, s.U.first_cta, ct, warp, lane);
      ptx::named_barrier(1, kOut);   // merge_info is read before it is written again
    }
    return true;
  });
}

template <int D, int kMaxUnits>
__global__ void __launch_bounds__(kThreads, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmap,
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
  misc += S::kSlots;
  v.seg_poison = misc;
  misc += 2 * kGroups;
  v.abort_flag = misc;
  v.merge_info = misc + 1;
  int* tmem_slot = misc + 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) {
      int n = 1;
      if (i < S::kKEmpty) n = 1 + 32;                                 // K full: and scales
      if (i >= S::kSFull && i < S::kSEmpty) n = 2;                    // products and scales
      if (i >= S::kSEmpty && i < S::kOFull) n = kGroupWarps;          // S empty, P full
      if (i >= S::kOEmpty && i < S::kQFull) n = kOutWarps;
      if (i >= S::kQFull && i < S::kQEmpty) n = kOutWarps;
      if (i >= S::kQEmpty && i < S::kLFull) n = kSoftmaxWarps + 1;    // and the last product
      if (i >= S::kLFull && i < S::kLEmpty) n = kSoftmaxWarps;
      if (i >= S::kFEmpty) n = kOutWarps;
      ptx::mbar_init(v.bar(i), n);
    }
    *v.abort_flag = 0;
    ptx::mbar_init_fence();
  }
  if (warp == kTmaWarp && lane == 0) ptx::prefetch_tensormap(&tmap);
  if (warp == kScoreWarp) tc::alloc(ptx::smem_addr(tmem_slot), kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile int*>(tmem_slot);
  if (warp < kSoftmaxWarps) {
    softmax_warps<D>(p, v, tmem, warp / kGroupWarps, warp % kGroupWarps, lane);
  } else if (warp < kSoftmaxWarps + kOutWarps) {
    output_warps<D>(p, v, tmem, warp - kSoftmaxWarps, lane);
  } else if (warp == kTmaWarp) {
    tma_warp<D>(p, v, &tmap, lane);
  } else if (warp == kScoreWarp) {
    score_warp<D>(p, v, tmem);
  } else if (warp == kProductWarp) {
    product_warp<D>(p, v, tmem);
  } else {
    helper_warp<D>(p, v, lane);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kScoreWarp) tc::dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// The merge of every request's T tiles, by the rule of lse_merge: a thread per
// float4 of an output row and every kTeams-th tile, kBatch tiles' values in
// flight with the LSEs that weigh them.  As a launch of its own it costs what
// its wait and a round of loads do, 1.5-2.5 us; inside the attention kernel, by
// the CTA that completed a request's tiles (as the bf16 kernel does it), such a
// CTA's stream stood still for an arrival and its answer and for code and values
// met cold: 262,144 tokens in 8 tiles 88.2 -> 85.4 us, 700 in 7 tiles 11.8 ->
// 7.4, 42 requests of 593 in 6 tiles 42.4 -> 33.0, 60 of up to 3,828 in 7 tiles
// 116.6 -> 82.9.  (Adding the partials of split units here too, in place of the
// attention kernel's slices, took 7 ragged requests in 5 tiles from 21.9 to 20.7
// us and 20,000 tokens in 20 tiles from 18.5 to 22.9: not kept.)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;
constexpr int kOneTeamTiles = 8;   // up to here one thread takes all tiles

template <int D, int kTeams>
__global__ void __launch_bounds__(kMergeThreads)
    merge_kernel(const float* out, const float* lse, int T, int Hq, int rows, float* m_out,
                 float* m_lse) {
  constexpr int kVec = D / 4, kRows = kMergeThreads / (kVec * kTeams);
  constexpr int kBatch = kTeams == 1 ? kOneTeamTiles : 4;
  __shared__ float4 s_acc[kTeams][kVec];
  __shared__ float s_m[kTeams], s_w[kTeams];
  ptx::launch_dependents();
  const int team = threadIdx.x / kVec % kTeams, c = threadIdx.x % kVec;
  const int row = blockIdx.x * kRows + threadIdx.x / (kVec * kTeams);
  if (row >= rows) return;   // (kTeams > 1: never, a block is a row)
  const size_t first = (size_t)(row / Hq) * T * Hq + row % Hq;   // of tile 0; tile t: + t Hq
  lse += first;
  const float4* src = reinterpret_cast<const float4*>(out) + first * kVec + c;
  const size_t step = (size_t)Hq * kVec;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, ws = 0.f;   // ws becomes NaN with a tile's LSE
  ptx::grid_dependency_wait();
  for (int t0 = team; t0 < T; t0 += kTeams * kBatch) {
    float4 x[kBatch];
    float l[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = t0 + i * kTeams;
      l[i] = -INFINITY;
      if (t < T) {
        l[i] = __ldcg(lse + (size_t)t * Hq);
        x[i] = __ldcg(src + t * step);
      }
    }
    float to = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) to = fmaxf(to, l[i]);
    const float f = m == -INFINITY ? 0.f : expf(m - to);
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
    ws = ws != ws ? ws : ws * f;
    m = to;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (l[i] == -INFINITY) continue;
      const float w = expf(l[i] - m);
      ws += w;
      acc.x = fmaf(w, x[i].x, acc.x);
      acc.y = fmaf(w, x[i].y, acc.y);
      acc.z = fmaf(w, x[i].z, acc.z);
      acc.w = fmaf(w, x[i].w, acc.w);
    }
  }
  if constexpr (kTeams > 1) {
    s_acc[team][c] = acc;
    if (c == 0) {
      s_m[team] = m;
      s_w[team] = ws;
    }
    __syncthreads();
    if (team != 0) return;
    for (int k = 1; k < kTeams; ++k) m = fmaxf(m, s_m[k]);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    ws = 0.f;
#pragma unroll
    for (int k = 0; k < kTeams; ++k) {
      const float f = s_m[k] == -INFINITY ? 0.f : expf(s_m[k] - m);
      const float4 x = s_acc[k][c];
      ws += s_w[k] != s_w[k] ? s_w[k] : f * s_w[k];
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
  }
  float4 y = make_float4(acc.x / ws, acc.y / ws, acc.z / ws, acc.w / ws);
  float z = m + logf(ws);
  if (ws != ws || m == -INFINITY) {
    z = ws != ws ? ws : -INFINITY;
    const float fill = ws != ws ? ws : 0.f;
    y = make_float4(fill, fill, fill, fill);
  }
  reinterpret_cast<float4*>(m_out + (size_t)row * D)[c] = y;
  if (c == 0) m_lse[row] = z;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// For units of one length, a grid (at least 80% of `grid`) that divides them, or
// that they divide: no CTA has parts of two units.  0 if there is none.
int even_grid(int count, int grid) {
  for (int g = grid; g * 5 >= grid * 4; --g)
    if (count % g == 0 || g % count == 0) return g;
  return 0;
}

// Pages that each CTA has at most if no CTA takes parts of two units (the fewest
// for which the units' CTAs fit the grid), or 0 where that is more than
// kTwoPartsBytes above an equal share.  A CTA with a part of a split unit before
// another segment is ~5 us behind the others: a table row, q, an arrival and its
// fence lie between the two.  (Against equal shares: 7 ragged requests in 5 tiles
// 24.9 -> 23.6 us, 20,000 tokens in 3 tiles 15.7 -> 14.5, 9,000 and 800 tokens 12.3
// -> 10.5, 3 x 54,748 in 4 tiles unchanged; 200 KB or 300 KB did as well but for 12
// x 9,000 in 3 tiles, 26.0 -> 25.4.)
int pages_alone(const int32_t* pages, size_t n, long long sum, int count, int grid, int d) {
  if (count > grid) return 0;
  auto fits = [&](long long most) {
    long long ctas = 0;
    for (size_t i = 0; i < n; ++i) ctas += (pages[i] + most - 1) / most;
    return ctas <= grid;
  };
  long long lo = (sum + grid - 1) / grid, hi = sum / grid + kTwoPartsBytes / (2 * kPage * d);
  if (!fits(hi)) return 0;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  return (int)lo;
}

// Cuts a launch's units into CTAs.  A unit on one CTA costs a step per two
// pages (0.5-0.65 us); a unit on several costs partials and their merge, about
// 2 us more.
void cut_pages(const Unit* units, const int32_t* pages, size_t n, long long total, int sms,
               int heads, int d, std::vector<int32_t>* starts) {
  int count = 0, most = 0, least = 1 << 30;   // units with pages
  long long sum = 0;
  for (size_t i = 0; i < n; ++i) {
    if (pages[i] == 0) continue;
    ++count;
    sum += pages[i];
    most = std::max(most, pages[i]);
    least = std::min(least, pages[i]);
  }
  starts->reserve(sms + 1);
  if (count == 0) {
    starts->assign({0, 1});
    return;
  }
  if (count <= sms && most <= kWholePages) {
    for (size_t i = 0; i < n; ++i)
      if (pages[i] != 0) starts->push_back(starts->empty() ? 0 : units[i].page_first);
    starts->push_back(static_cast<int32_t>(total));
    return;
  }
  int grid = sum >= (long long)kLongPages * sms ? sms * kLongGridPct / 100
                                                : (int)std::min<long long>(sms, sum / kMinPages);
  grid = std::max(grid, 1);
  // As the bf16 kernel's: the CTAs at the same offset of each kv head's block
  // of units stream the same pages at the same time.
  if (grid >= heads) grid -= grid % heads;
  const int alone = most == least ? 0 : pages_alone(pages, n, sum, count, grid, d);
  if (alone > 0) {
    for (size_t i = 0; i < n; ++i) {
      const int parts = (pages[i] + alone - 1) / alone;
      for (int k = 0; k < parts; ++k)
        starts->push_back(starts->empty() ? 0 : units[i].page_first +
                                                    (int)((long long)pages[i] * k / parts));
    }
    starts->push_back(static_cast<int32_t>(total));
    return;
  }
  if (const int even = most == least ? even_grid(count, grid) : 0) grid = even;
  starts->push_back(0);
  int at = 0;
  size_t i = 0;
  for (int k = 1; k < grid; ++k) {
    int to = at + ((int)total - at) / (grid - k + 1);
    // the unit that holds the border, if one does
    while (i < n && (pages[i] == 0 || units[i].page_first + pages[i] <= to)) ++i;
    if (i < n && to > units[i].page_first) {
      const int lo = units[i].page_first, hi = lo + pages[i];
      if (to - lo <= kSnapPages && to - lo <= hi - to && lo > at) to = lo;
      else if (hi - to <= kSnapPages) to = hi;
    }
    if (to <= at) continue;
    starts->push_back(to);
    at = to;
  }
  if (total > at) starts->push_back(static_cast<int32_t>(total));
}

// Adds CTAs that have no pages where units without pages (padded requests, tiles
// behind a request's end) outnumber the CTAs: those are dealt out to all CTAs, a
// warp each (4 requests of 700 tokens and 252 without any: 8.1 us, 24.8 without
// these CTAs; 1 and 63: 7.6, 21.2).
void deal_empty(size_t empty, int sms, std::vector<int32_t>* starts) {
  const size_t ctas = std::min<size_t>(sms, empty);
  if (starts->size() < ctas + 1) starts->resize(ctas + 1, starts->back());
}

void cut(const Unit* units, const int32_t* pages, size_t n, long long total, int sms, int heads,
         int d, std::vector<int32_t>* starts) {
  cut_pages(units, pages, n, total, sms, heads, d, starts);
  deal_empty(std::count(pages, pages + n, 0), sms, starts);
}

// Lays a launch's units out anew so that every CTA has whole ones, the longest
// first dealt to the CTA with the least, where that comes within kWholeBytes
// of equal shares: no unit is split, and nothing merged.  A CTA takes its
// shortest first, so that launches end in long streams.  (Shortest / longest
// first, and equal shares: 64 requests of up to 2,500 tokens 32.9 / 33.6 / 35.6
// us, at 256 dims 29.8 / 29.7 / 33.5, 256 of up to 600 33.9 / 37.6 / 37.1, 120 of
// up to 2,000 with 2 kv heads 14.5 / 14.9 / 19.3.  Giving each kv head CTAs of its
// own, which then read the same pages at the same time, made no difference; with
// 400 KB for kWholeBytes 42 of up to 4,000 took 34.4 us instead of 32.0, with 3.2
// MB nothing changed.)
// Linear in the units: a sort by counting, and CTAs kept in lists by their load
// (the least load only grows).  Returns the order of the units that have pages, or
// nothing if they stay as they are.
std::vector<int> pack(Plan* plan, Launch* L, int sms, int d) {
  const int32_t* pages = plan->pages.data() + L->u0;
  Unit* units = plan->units.data() + L->u0;
  const int n = (int)L->n;
  long long sum = 0;
  int count = 0, most = 0, least = 1 << 30;   // units with pages
  for (int i = 0; i < n; ++i) {
    if (pages[i] == 0) continue;
    ++count;
    sum += pages[i];
    most = std::max(most, pages[i]);
    least = std::min(least, pages[i]);
  }
  const int grid = sum >= (long long)kLongPages * sms ? sms * kLongGridPct / 100 : sms;
  if (count <= grid) return {};
  // (Units of one length stay in an even grid: 64 x 2,048 tokens 42.9 us, 43.9 dealt
  // out; 180 x 1,000 60.5 and 62.4.  Without one, 50 x 1,000 23.4 and 22.5.)
  if (most == least && even_grid(count, grid)) return {};
  // Loads are pages and a few more per unit.
  const long long limit =
      (sum + (long long)kUnitCharge * count) / grid + kWholeBytes / (2 * kPage * d);
  if (most + kUnitCharge > limit || limit > 1 << 20) return {};
  // Units by their pages, and CTAs by their loads: heads of lists.
  std::vector<int> of_pages(most + 1, -1), of_load(limit + 1, -1), next_unit(n), next_cta(grid),
      first(grid, -1);
  for (int i = n - 1; i >= 0; --i) {
    next_unit[i] = of_pages[pages[i]];
    of_pages[pages[i]] = i;
  }
  for (int k = 0; k < grid; ++k) next_cta[k] = k + 1 < grid ? k + 1 : -1;
  of_load[0] = 0;
  int load = 0;
  for (int p = most; p > 0; --p) {
    for (int i = of_pages[p]; i >= 0;) {
      while (of_load[load] < 0) ++load;
      const int k = of_load[load], to = load + p + kUnitCharge, next = next_unit[i];
      if (to > limit) return {};
      of_load[load] = next_cta[k];
      next_cta[k] = of_load[to];
      of_load[to] = k;
      next_unit[i] = first[k];   // the CTA's last comes first
      first[k] = i;
      i = next;
    }
  }
  std::vector<int> order;
  order.reserve(count);
  L->starts.clear();
  int32_t at = 0;
  for (int k = 0; k < grid; ++k) {
    L->starts.push_back(at);
    for (int i = first[k]; i >= 0; i = next_unit[i]) {
      order.push_back(i);
      units[i].page_first = at;
      units[i].n_parts = 1;
      units[i].first_cta = static_cast<uint8_t>(k);
      at += pages[i];
    }
  }
  L->starts.push_back(at);
  deal_empty(n - count, sms, &L->starts);
  L->grid = (int)L->starts.size() - 1;
  return order;
}

using Common = Params<kMaxUnitsSmall>;

template <int D, int N>
int launch_units(const CUtensorMap& tmap, const Plan& plan, const Launch& L,
                 const std::vector<int>& order, const Common& common, cudaStream_t stream) {
  using Prm = Params<N>;
  static_assert(N >= kMaxUnitsSmall && offsetof(Prm, starts) == offsetof(Common, starts), "");
  Prm prm;
  std::memcpy(static_cast<void*>(&prm), &common, offsetof(Common, starts));
  prm.n_units = static_cast<int>(L.n);
  prm.grid = L.grid;
  // Units without pages go last: every role walks its CTA's units, and skipping
  // one costs it ~0.2 us (4 requests of 700 tokens and 252 without any: 64.5 us
  // with the others among them).
  DevUnit* to = prm.units;
  auto add = [&](const Unit& u) {
    *to++ = {u.page_first, u.bt, u.tok_start, u.tok_end, u.g, u.part_base, u.n_parts, u.first_cta};
  };
  for (int i : order) add(plan.units[L.u0 + i]);
  for (size_t i = L.u0; order.empty() && i < L.u0 + L.n; ++i)
    if (plan.pages[i] != 0) add(plan.units[i]);
  prm.n_full = static_cast<int>(to - prm.units);
  for (size_t i = L.u0; i < L.u0 + L.n && to < prm.units + L.n; ++i)
    if (plan.pages[i] == 0) add(plan.units[i]);
  std::memcpy(prm.starts, L.starts.data(), L.starts.size() * sizeof(int32_t));
  for (int k = 0, u = 0; k < L.grid; ++k) {
    // the last unit that starts at or before the CTA's first page
    while (u + 1 < prm.n_full && prm.units[u + 1].page_first <= L.starts[k]) ++u;
    prm.first_unit[k] = static_cast<int16_t>(u);
  }
  static PerContext smem_limit;   // the attribute lives in the context
  cudaError_t e = smem_limit.apply([] {
    return cudaFuncSetAttribute(decode_q8_kernel<D, N>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc);
  });
  if (e == cudaSuccess)
    e = launch_dependent(decode_q8_kernel<D, N>, dim3(L.grid), dim3(kThreads), Smem<D>::kAlloc,
                         stream, tmap, prm);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(PA_ERR_CUDA, "8-bit paged decode launch failed: %s", cudaGetErrorString(e));
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

// One thread per float4 for up to kOneTeamTiles tiles (one round of loads), a
// block per row behind that (64 tiles: 19.8 -> 12.9 us for the whole call).
template <int D>
cudaError_t launch_merge(const float* out, const float* lse, int T, int Hq, int rows, float* m_out,
                         float* m_lse, cudaStream_t stream) {
  constexpr int kTeams = kMergeThreads / (D / 4);
  const bool one = T <= kOneTeamTiles;
  const dim3 grid(one ? (rows + kTeams - 1) / kTeams : rows);
  return launch_dependent(one ? merge_kernel<D, 1> : merge_kernel<D, kTeams>, grid,
                          dim3(kMergeThreads), 0, stream, out, lse, T, Hq, rows, m_out, m_lse);
}

int run(const void* q, const void* pool, const float* scales, int64_t pool_pages,
        const int32_t* page_table, int max_pages, const int32_t* tiles, int B, int T, int Hq,
        int Hkv, int D, float scale, float* out, float* lse, float* merged_out, float* merged_lse,
        void* workspace, size_t ws_bytes, cudaStream_t stream) {
  PA_REQUIRE(B >= 0 && T >= 0, "B and T must be >= 0 (got %d, %d)", B, T);
  if ((long long)B * T == 0) return PA_OK;
  if (D != 128 && D != 256)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 128, 256)", D);
  PA_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0,
             "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", Hq, Hkv);
  if (Hq / Hkv > kMaxG)
    return fail(PA_ERR_UNSUPPORTED, "group size %d above the supported %d", Hq / Hkv, kMaxG);
  PA_REQUIRE(q && pool && scales && page_table && tiles && out && lse && workspace,
             "null pointer argument");
  PA_REQUIRE(max_pages >= 1 && pool_pages >= 1, "max_pages and pool_pages must be >= 1");
  auto aligned = [](const void* ptr, int n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  PA_REQUIRE(aligned(q, 16), "q must be 16-byte aligned");
  PA_REQUIRE(aligned(pool, 16), "pool must be 16-byte aligned");
  PA_REQUIRE(aligned(scales, 16), "scales must be 16-byte aligned");
  PA_REQUIRE(aligned(out, 16), "out must be 16-byte aligned");
  PA_REQUIRE(aligned(workspace, 256), "workspace must be 256-byte aligned");
  PA_REQUIRE((merged_out == nullptr) == (merged_lse == nullptr),
             "merged_out and merged_lse go together");
  PA_REQUIRE(aligned(merged_out, 16), "merged_out must be 16-byte aligned");
  PA_REQUIRE(pool_pages < (1ll << 31) / kPage, "pool too large for 32-bit row coordinates");
  PA_REQUIRE((long long)B * T * Hq < (1ll << 31), "output too large");
  const size_t need = workspace_bytes(B, T, Hkv, D);
  PA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes,
             need);
  const long long max_tok = (long long)max_pages * kPage;
  for (long long i = 0; i < (long long)B * T; ++i) {
    const int s = tiles[2 * i], e = tiles[2 * i + 1];
    PA_REQUIRE(s >= 0 && s <= e && e <= max_tok,
               "tile %lld of request %lld is [%d, %d), outside [0, %lld]", i % T, i / T, s, e,
               max_tok);
  }
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  CUtensorMap tmap;
  {
    const int row = 2 * Hkv * D;
    const cuuint64_t dims[2] = {(cuuint64_t)row, (cuuint64_t)pool_pages * kPage};
    const cuuint64_t strides[1] = {(cuuint64_t)row};
    const cuuint32_t box[2] = {kChunk, kPage};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(&tmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  int sms = sm_count();
  if (sms <= 0) return fail(PA_ERR_CUDA, "cannot query the device's SM count");
  sms = std::min(sms, kMaxGrid);
  Plan plan;
  int rc = plan_units(
      tiles, B, T, Hkv, kSegmentCharge, false,
      [&](const Unit* units, const int32_t* pages, size_t n, long long total,
          std::vector<int32_t>* starts) { cut(units, pages, n, total, sms, Hkv, D, starts); },
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
  common.scale_log2 = std::ldexp(scale * kLog2e, kScaleShift);
  if (T == 1) {
    common.out2 = merged_out;
    common.lse2 = merged_lse;
  }
  const TestHooks hooks = take_test_hooks();
  common.wait_limit_ns = hooks.wait_limit_ns;
  common.stall_iteration = hooks.stall_iteration;
  common.slice_wait_ns = hooks.slice_wait_ns;
  for (Launch& L : plan.launches) {
    const std::vector<int> order = pack(&plan, &L, sms, D);
    rc = launch(D, tmap, plan, L, order, common, stream);
    if (rc != PA_OK) return rc;
  }
  if (T > 1 && merged_out != nullptr) {
    auto merge = D == 128 ? launch_merge<128> : launch_merge<256>;
    PA_CHECK_CUDA(merge(out, lse, T, Hq, B * Hq, merged_out, merged_lse, stream));
    PA_CHECK_CUDA(cudaGetLastError());
  }
  return PA_OK;
}

}  // namespace decode_q8
}  // namespace pa

extern "C" size_t paged_decode_attn_q8_workspace_bytes(int B, int T, int n_q_heads, int n_kv_heads,
                                                       int head_dim) {
  if (B < 0 || T < 0 || (head_dim != 128 && head_dim != 256) || n_kv_heads < 1 ||
      n_q_heads < n_kv_heads || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > pa::split::kMaxG)
    return 0;
  return pa::split::workspace_bytes(B, T, n_kv_heads, head_dim);
}

extern "C" int paged_decode_attn_q8_lse(const void* q, const void* pool, const float* scales,
                                        int64_t pool_pages, const int32_t* page_table,
                                        int max_pages, const int32_t* tiles, int B, int T,
                                        int n_q_heads, int n_kv_heads, int head_dim, float scale,
                                        float* out, float* lse, float* merged_out,
                                        float* merged_lse, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  pa::clear_error();
  try {
    return pa::decode_q8::run(q, pool, scales, pool_pages, page_table, max_pages, tiles, B, T,
                              n_q_heads, n_kv_heads, head_dim, scale, out, lse, merged_out,
                              merged_lse, workspace, workspace_bytes, stream);
  } catch (const std::exception& e) {
    return pa::fail(PA_ERR_INVALID, "host memory for the plan: %s", e.what());
  }
}
