// How the decode kernels split their work over CTAs, and how the parts of a
// unit that spans several CTAs come together: shared by the bf16 and the 8-bit
// pool's kernels.
//
// A unit is one (tile, kv head).  All units' pages are laid end to end and cut
// into one contiguous page range per CTA.  A kernel's parameter struct P has
// the fields these functions name (out, lse, status, arrivals, part_o, part_ml,
// T, Hq, Hkv, G, n_units, units, wait_limit_ns, slice_wait_ns; where kSecondOut
// says that outputs are written twice, out2 and lse2; where kMerge says that the
// kernel merges a request's tiles, m_out, m_lse and req_counters; kAllSlices,
// see split_slices); its shared-memory view Sh has merge_info and, with kMerge,
// fin_flag.  The kConsumers threads that call a function meet at named barrier 1.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "common.h"
#include "merge_row.cuh"
#include "ptx.cuh"

namespace pa {
namespace split {

constexpr int kPage = PA_PAGE_TOKENS;      // tokens per page
constexpr int kMaxG = 8;                   // query heads per kv head
constexpr int kMaxUnitsLarge = 1024;
constexpr int kMaxUnitsSmall = 64;
constexpr size_t kStatusBytes = 256;
constexpr size_t kPartMLBytes = size_t(kMaxG) * 2 * 4;   // per partial slot
// A split unit's merge reads up to kMaxPartsPerLane partials per lane of a
// 32-lane team, which bounds the CTAs a unit may span and so the grid.
constexpr int kMaxPartsPerLane = 5;
constexpr int kMaxGrid = 32 * kMaxPartsPerLane;
// How long a CTA that has stored its partial waits without seeing another
// CTA of the unit arrive before it leaves its share of the merge to the
// unit's last CTA.  The CTAs of a launch finish within ~25 us of each other
// (per-SM streaming speeds differ by up to ~10% over a long launch), with
// arrivals every few hundred ns; the limit matters only when some of them
// cannot be resident at the same time (other work holds SMs), where waiting
// longer would only delay them.
constexpr uint64_t kSliceWaitNs = 50000ull;
// A split unit's outputs are merged in at most this many slices, one per
// waiting CTA: enough to spread the partials' loads, few enough that most of
// a widely split unit's CTAs leave at once (their SMs then take the next
// launch's first page loads).
constexpr int kMaxSlices = 16;
constexpr int kMaxSlicesAll = 24;
constexpr uint64_t kWaitLimitNs = 2000000000ull;         // 2 s per bounded device wait
// Per unit: a 64-bit arrival word (count | leavers << 16 | generation << 32).
constexpr size_t kCounterBytes = 8 * kMaxUnitsLarge;
constexpr float kLn2Hi = 0.693145751953125f;        // ln 2, high bits (exact products)
constexpr float kLn2Lo = 1.428606765330187045e-06f; // ln 2 - kLn2Hi
// The running softmax reference is kept on multiples of kRefStep (log2 units):
// rescales and the weights between partials are then exact powers of two, and
// every probability is the same number (up to an exact power of two) however
// the tokens are split into tiles, chunks and warps.
constexpr float kRefStep = 8.0f;

static_assert(kMaxSlices <= kMaxGrid - 1, "slices per split unit");
static_assert(kMaxGrid <= 255 && kMaxUnitsLarge + 1024 <= 65536, "fields of Unit");

struct Unit {
  int32_t bt;          // b * T + t
  int32_t tok_start;
  int32_t tok_end;
  int32_t page_first;  // flattened index of the unit's first page in this launch
  int32_t g;           // kv head
  uint16_t part_base;  // first partial slot (units covered by several CTAs)
  uint8_t n_parts;     // CTAs covering the unit
  uint8_t first_cta;   // the first of them
  int32_t pair_total;  // completions the (request, kv head) tile counter reaches (fused merge)
};

// Slices a unit split over n >= 2 CTAs is merged in: half its CTAs wait and
// merge, the other half leave at once (their SMs take the next launch's first
// page loads).  Measured per launch against n - 1 slices (both capped at 16),
// one box: 4 x 31,744 tokens (n ~ 9) 77.76 -> 77.05 us, 2 x 32,768 (n ~ 19)
// 44.18 -> 43.37 us, 1 x 32,768 (n ~ 38) and 1 x 262,144 unchanged; a third
// of them cost 1 x 32,768 0.3 us, two thirds gained half as much.
// kAll (a kernel that merges with 128 threads): all the slices there can be (every
// CTA but the last ends in the unit), so that a slice takes one round of loads,
// about 1 us across the dies, where half of them took two (1 x 32,768 tokens
// 17.5 -> 16.5 us).
template <bool kAll>
__host__ __device__ __forceinline__ int split_slices(int n) {
  if (kAll) return n - 1 < kMaxSlicesAll ? n - 1 : kMaxSlicesAll;
  return n / 2 < kMaxSlices ? n / 2 : kMaxSlices;
}

__host__ __device__ __forceinline__ int unit_pages(int tok_start, int tok_end) {
  return tok_end > tok_start ? (tok_end + kPage - 1) / kPage - tok_start / kPage : 0;
}

// CTA whose page range [k P / grid, (k+1) P / grid) holds flattened page p.
__host__ __device__ __forceinline__ int cta_of(long long p, long long total, int grid) {
  return static_cast<int>(((p + 1) * grid - 1) / total);
}

template <class P>
__device__ __forceinline__ int first_unit(const P& p, long long start) {
  int lo = 0, hi = p.n_units - 1, ans = 0;
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (p.units[mid].page_first <= start) {
      ans = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  return ans;
}

// ln-domain LSE of a reference m (log2 units, a multiple of kRefStep) and a
// sum l > 0: (m + e) ln 2 + ln f with l = f 2^e, f in [0.5, 1).  m + e is an
// exact small integer, its product with the high part of ln 2 (a Cody-Waite
// split) is exact, and the small terms go into the last addition, so the
// result carries about one fp32 rounding, as a double evaluation rounded to
// fp32 would -- without FP64 arithmetic, which is slow on this part (a double
// log per row had cost microseconds of every launch's tail).
__device__ __forceinline__ float lse_of(float m, float l) {
  if (m == -INFINITY || !(l > 0.f)) return m * kLn2Hi + logf(l);   // -inf / degenerate
  int e;
  const float f = frexpf(l, &e);
  const float t = m + static_cast<float>(e);
  return t * kLn2Hi + fmaf(t, kLn2Lo, logf(f));
}

__device__ __forceinline__ float ref_ceil(float x) {
  return ceilf(x * (1.0f / kRefStep)) * kRefStep;
}

// Weight of a partial whose reference is m relative to the common reference
// big_m >= m (both multiples of kRefStep): exactly 2^(m - big_m), 0 for -inf.
__device__ __forceinline__ float ref_weight(float m, float big_m) {
  return (m == -INFINITY) ? 0.f : ptx::pow2i(static_cast<int>(m - big_m));
}

// Called by every consumer thread once it has stored `done` parts of the
// tile outputs of (request b, kv head g): a whole unsplit (or empty) unit
// counts 1, a slice of a split unit 1.  With the fused merge, the CTA whose
// parts complete the pair's count (`total`, over its T tiles) merges the T
// tiles for the G query heads of g with the merge kernel's own row routine
// (same bits as lse_merge over those partials), then resets the counter for
// the next call.
template <int kD, int kConsumers, class P, class Sh>
__device__ __forceinline__ void finish_unit(const P& p, const Sh& sh, int b,
                                            int g, int ct, int warp, int lane, int done,
                                            int total) {
  if constexpr (P::kMerge) {
    if (p.m_out == nullptr) return;
    ptx::named_barrier(1, kConsumers);       // this CTA's outputs are all stored
    if (ct == 0) {
      const int prev = ptx::atomic_add_acq_rel_gpu(p.req_counters + b * p.Hkv + g, done);
      *sh.fin_flag = (prev + done == total) ? 1 : 0;
    }
    ptx::named_barrier(1, kConsumers);
    if (*sh.fin_flag) {
      for (int r = warp; r < p.G; r += kConsumers / 32) {
        const int h = g * p.G + r;
        mergerow::merge_row<true>(p.out, p.lse, b * p.T, p.T, p.Hq, h, kD,
                                  p.m_out + ((size_t)b * p.Hq + h) * kD,
                                  p.m_lse + (size_t)b * p.Hq + h, lane);
      }
      if (ct == 0) p.req_counters[b * p.Hkv + g] = 0;
    }
    ptx::named_barrier(1, kConsumers);
  }
}

// Merges output float4s [o_lo, o_hi) of a split unit (o = row * kD/4 + float4
// column) from its n partials (slots part_base ..): the unit's tile output and,
// at column 0, its LSE.  The same merge rule as the tile merge: common
// reference = max partial reference, weights exactly 2^(m_c - max), output =
// weighted sum / summed weights.  Each output is taken by a team of t lanes
// (t a power of two, as large as one pass over the outputs allows); lane j
// adds partials j, j + t, ... in that order, and the team adds its lanes'
// sums by a butterfly.  The arithmetic depends only on n and the range, never
// on which CTA runs it, so slices merged by different CTAs, or twice, give
// the same bits.  All of a lane's loads are issued before its arithmetic.
template <int kD, int kConsumers, class P>
__device__ __forceinline__ void merge_split_slice(const P& p, int part_base, int n,
                                                  int o_lo, int o_hi, size_t orow0, int ct) {
  constexpr int kVec = kD / 4;
  const int len = o_hi - o_lo;
  int t = 32;
  while (t > 1 && kConsumers / t < len && (n + t / 2 - 1) / (t / 2) <= kMaxPartsPerLane) t >>= 1;
  const int n_teams = kConsumers / t;
  const int j = ct & (t - 1);
  const int team = ct / t;
  const float2* pml = reinterpret_cast<const float2*>(p.part_ml) + (size_t)part_base * kMaxG;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + (size_t)part_base * kMaxG * kVec;
  for (int base = o_lo; base < o_hi; base += n_teams) {
    const int o = base + team;
    const bool have = o < o_hi;
    const int row = have ? o / kVec : 0;
    const int dv = have ? o - row * kVec : 0;
    float2 ml[kMaxPartsPerLane];
    float4 v[kMaxPartsPerLane];
#pragma unroll
    for (int k = 0; k < kMaxPartsPerLane; ++k) {
      const int c = j + k * t;
      if (have && c < n) {
        ml[k] = __ldcg(pml + (size_t)c * kMaxG + row);
        v[k] = __ldcg(po + ((size_t)c * kMaxG + row) * kVec + dv);
      } else {
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float big_m = -INFINITY;
    int nan = 0;
#pragma unroll
    for (int k = 0; k < kMaxPartsPerLane; ++k) {
      big_m = fmaxf(big_m, ml[k].x);
      nan |= (ml[k].x != ml[k].x);
    }
    for (int off = t >> 1; off > 0; off >>= 1) {
      big_m = fmaxf(big_m, __shfl_xor_sync(0xffffffffu, big_m, off));
      nan |= __shfl_xor_sync(0xffffffffu, nan, off);
    }
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMaxPartsPerLane; ++k) {
      const float a = ref_weight(ml[k].x, big_m);
      l = fmaf(a, ml[k].y, l);
      acc.x = fmaf(a, v[k].x, acc.x);
      acc.y = fmaf(a, v[k].y, acc.y);
      acc.z = fmaf(a, v[k].z, acc.z);
      acc.w = fmaf(a, v[k].w, acc.w);
    }
    for (int off = t >> 1; off > 0; off >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
    }
    if (have && j == 0) {
      const size_t orow = orow0 + row;
      const float qnan = __int_as_float(0x7fc00000);
      const float4 v4 = nan ? make_float4(qnan, qnan, qnan, qnan)
                            : make_float4(acc.x / l, acc.y / l, acc.z / l, acc.w / l);
      reinterpret_cast<float4*>(p.out + orow * kD)[dv] = v4;
      const float x = dv == 0 ? (nan ? qnan : lse_of(big_m, l)) : 0.f;
      if (dv == 0) p.lse[orow] = x;
      if constexpr (P::kSecondOut) {
        if (p.out2) {
          reinterpret_cast<float4*>(p.out2 + orow * kD)[dv] = v4;
          if (dv == 0) p.lse2[orow] = x;
        }
      }
    }
  }
}

// Thread 0 of a CTA that has arrived at split unit `arrival` in generation
// `gen`, with this unit's segment as its last: waits until every CTA of the
// unit has arrived (the count reaches n, or the last CTA has already opened
// the next generation), so every partial is stored and visible.  If no other
// CTA of the unit arrives for slice_wait_ns while some have not, it records
// itself as a leaver (the last CTA then merges every slice) and returns false.
__device__ __forceinline__ bool wait_unit_complete(unsigned long long* arrival, unsigned gen,
                                                   int n, uint64_t slice_wait_ns,
                                                   uint64_t wait_limit_ns, int32_t* status) {
  const uint64_t t0 = ptx::globaltimer_ns();
  uint64_t t_seen = t0;
  int seen = -1;
  while (true) {
    // Acquire polls: the one that sees every arrival synchronises with all
    // of them (each arrival is an acquire-release add, and the opening add
    // is in the release sequence of each).  Measured against relaxed polls
    // followed by a fence: 25.33 -> 24.96 us per launch at 1 x 32,768 tokens,
    // 78.17 -> 77.84 us with 4 x 31,744.
    const unsigned long long v = ptx::load_acquire_gpu(arrival);
    const int count = (int)(v & 0xffffu);
    if ((unsigned)(v >> 32) != gen || count == n) return true;
    const uint64_t now = ptx::globaltimer_ns();
    if (count != seen) {
      seen = count;
      t_seen = now;
    }
    if (now - t_seen > slice_wait_ns && ptx::atomic_cas_gpu(arrival, v, v + (1ull << 16)) == v)
      return false;
    if (now - t0 > wait_limit_ns) {
      atomicOr(status, PA_STATUS_TIMEOUT);
      return false;
    }
  }
}

// Split unit u: CTAs k0 .. k1 each stored a partial.  The barrier orders
// every thread's partial before thread 0's acquire-release arrival,
// which publishes it at device scope.  CTAs k0 .. k0 + S - 1 (S <= n - 1:
// their page ranges end inside this unit, so it is their last segment)
// wait until all n have arrived and each merges one of S slices of the
// unit's outputs, so the merge is spread over S SMs instead of loading
// every partial into one; the last CTA to arrive resets the count and
// opens the word's next generation for the next call.  A CTA that gave
// up waiting leaves its slice to the last CTA, which then merges every
// slice (a slice merged twice gets the same bits).  The other CTAs
// leave at once.
template <int kD, int kConsumers, class P, class Sh>
__device__ __forceinline__ void finish_split_unit(const P& p, const Sh& sh, const Unit& U, int u,
                                                  int b, int bt, int g, int first_cta, int ct,
                                                  int warp, int lane) {
  const int n = U.n_parts;
  const int S = split_slices<P::kAllSlices>(n);
  const int rank = (int)blockIdx.x - first_cta;
  const bool participant = rank < S;
  unsigned long long* arrival = p.arrivals + u;
  ptx::named_barrier(1, kConsumers);
  if (ct == 0) {
    const unsigned long long prev = ptx::atomic_add_acq_rel_gpu(arrival, 1ull);
    const int arrived = (int)(prev & 0xffffu) + 1;
    int mode = 0;  // 0: no slice here, 1: this CTA's slice, 2: every slice
    int leavers = 0;
    if (arrived == n) {
      leavers = (int)((prev >> 16) & 0xffffu);
      // Count and leavers back to zero, generation + 1 (a plain add: a
      // waiting CTA that reads it still acquires every arrival, which
      // it follows in the word's order of modifications).
      ptx::red_add_relaxed_gpu(arrival, (1ull << 32) -
                                            ((unsigned long long)leavers << 16) -
                                            (unsigned long long)n);
      mode = leavers ? 2 : (participant ? 1 : 0);
      if (leavers) atomicAdd(p.status + 1, leavers);   // diagnostic count, not an error
    } else if (participant) {
      mode = wait_unit_complete(arrival, (unsigned)(prev >> 32), n, p.slice_wait_ns,
                                p.wait_limit_ns, p.status) ? 1 : 0;
    }
    sh.merge_info[0] = mode;
    sh.merge_info[1] = leavers;
  }
  ptx::named_barrier(1, kConsumers);
  const int mode = sh.merge_info[0];
  if (mode != 0) {
    const int n_out = p.G * (kD / 4);
    for (int sl = mode == 2 ? 0 : rank; sl < (mode == 2 ? S : rank + 1); ++sl) {
      merge_split_slice<kD, kConsumers>(
          p, U.part_base, n, (int)((long long)sl * n_out / S),
          (int)((long long)(sl + 1) * n_out / S), (size_t)bt * p.Hq + g * p.G, ct);
    }
    // Each slice counts once toward the pair's tile count (the slices
    // of leavers are counted by the last CTA, which merged them).
    const int done = mode == 2 ? sh.merge_info[1] + (participant ? 1 : 0) : 1;
    finish_unit<kD, kConsumers>(p, sh, b, g, ct, warp, lane, done, U.pair_total);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Settings of the test hooks (paged_decode_attn_test_stall and
// _test_slice_wait): consumed by the next decode call on the calling thread.
struct TestHooks {
  int stall_iteration = -1;
  unsigned long long wait_limit_ns = kWaitLimitNs;
  unsigned long long slice_wait_ns = kSliceWaitNs;
};
extern thread_local TestHooks t_hooks;
inline TestHooks take_test_hooks() {
  const TestHooks h = t_hooks;
  t_hooks = TestHooks();
  return h;
}

// Partial slots reserved: one per unit of a launch plus one per CTA (a CTA
// adds at most one split point), with room for grids up to 1,024 CTAs.
inline size_t part_slots(int B, int T, int Hkv) {
  const long long units = (long long)B * T * Hkv;
  return (size_t)std::min<long long>(units, kMaxUnitsLarge) + 1024;
}

// Per (request, kv head) counters of finished tiles for the fused merge.
inline size_t request_counter_bytes(int B, int Hkv) {
  return ((size_t)B * Hkv * 4 + 255) / 256 * 256;
}

inline size_t workspace_bytes(int B, int T, int Hkv, int D) {
  return kStatusBytes + kCounterBytes + request_counter_bytes(B, Hkv) +
         part_slots(B, T, Hkv) * ((size_t)kMaxG * D * 4 + kPartMLBytes);
}

// The parts of a caller's workspace.
struct Workspace {
  int32_t* status;
  unsigned long long* arrivals;
  int32_t* req_counters;
  float* part_o;
  float* part_ml;
  Workspace(void* base, int B, int T, int Hkv, int D) {
    uint8_t* ws = static_cast<uint8_t*>(base);
    status = reinterpret_cast<int32_t*>(ws);
    ws += kStatusBytes;
    arrivals = reinterpret_cast<unsigned long long*>(ws);
    ws += kCounterBytes;
    req_counters = reinterpret_cast<int32_t*>(ws);
    ws += request_counter_bytes(B, Hkv);
    part_o = reinterpret_cast<float*>(ws);
    part_ml = reinterpret_cast<float*>(ws + part_slots(B, T, Hkv) * kMaxG * D * 4);
  }
};

struct Launch {
  size_t u0, n;       // units [u0, u0 + n)
  long long total;    // flattened pages, at least 1
  int grid;
  std::vector<int32_t> starts;   // [grid + 1] CTA k takes flattened pages [k], [k + 1)
};
struct Plan {
  std::vector<Unit> units;
  std::vector<int32_t> pages;      // of each unit
  std::vector<Launch> launches;
};

// CTA boundaries that give `grid` CTAs equal shares.
inline void equal_starts(long long total, int grid, std::vector<int32_t>* starts) {
  starts->resize(grid + 1);
  for (int k = 0; k <= grid; ++k) (*starts)[k] = static_cast<int32_t>(k * total / grid);
}

// Lays a call's tiles out as units and launches.  shape(units, their pages, n,
// total, starts) cuts a launch's n units, laid out over `total` flattened
// pages, into CTAs; segment_charge is the number of pages that hold no data
// charged per unit start; merge: the kernel merges every request's tiles.
template <class Shape>
int plan_units(const int32_t* tiles, int B, int T, int n_kv_heads, int segment_charge, bool merge,
               Shape shape, Plan* plan) {
  const size_t n_tiles = (size_t)B * T, n_units = n_tiles * n_kv_heads;
  std::vector<Unit>& units = plan->units;
  std::vector<int32_t>& pages = plan->pages;
  units.resize(n_units);
  pages.resize(n_units);
  // Kv-head-major order: the units of one kv head form a block of the page
  // sequence, and every block has the same unit sizes, so the CTAs at the
  // same offset of the n_kv_heads blocks stream the same physical pages (each
  // its head's slice of every row) at about the same time.
  for (size_t bt = 0; bt < n_tiles; ++bt)
    pages[bt] = unit_pages(tiles[2 * bt], tiles[2 * bt + 1]);
  for (int g = 0; g < n_kv_heads; ++g) {
    Unit* u = units.data() + g * n_tiles;
    if (g > 0) std::copy_n(pages.data(), n_tiles, pages.data() + g * n_tiles);
    for (size_t bt = 0; bt < n_tiles; ++bt) {
      u[bt].bt = static_cast<int32_t>(bt);
      u[bt].g = g;
      u[bt].tok_start = tiles[2 * bt];
      u[bt].tok_end = tiles[2 * bt + 1];
    }
  }

  // Launches of at most kMaxUnitsLarge units each; every launch partitions its
  // own pages and reuses the workspace after the previous one (same stream).
  // All launches are laid out first: the fused merge's per-(request, kv
  // head) count spans every launch that holds a tile of the pair.
  const size_t slots = part_slots(B, T, n_kv_heads);
  for (size_t u0 = 0; u0 < n_units; u0 += kMaxUnitsLarge) {
    const size_t n = std::min<size_t>(kMaxUnitsLarge, n_units - u0);
    // The CTAs' shares are cut from the units' pages laid end to end, each unit
    // preceded by segment_charge pages that hold no data: a segment (one unit's
    // part on one CTA) costs a Q load, a combine and a partial whatever its
    // length, so a CTA whose range holds a unit start (one more segment) gets
    // that many fewer pages to stream.
    long long total = 0;
    for (size_t i = u0; i < u0 + n; ++i) {
      if (pages[i] > 0) total += segment_charge;
      units[i].page_first = static_cast<int32_t>(total);
      total += pages[i];
      PA_REQUIRE(total < (1ll << 31), "too many pages in one launch");
    }
    Launch L{u0, n, total > 0 ? total : 1, 1, {}};
    shape(units.data() + u0, pages.data() + u0, n, total, &L.starts);
    L.grid = (int)L.starts.size() - 1;
    int part_cursor = 0, k = 0;
    for (size_t i = u0; i < u0 + n; ++i) {
      Unit& u = units[i];
      if (pages[i] == 0) continue;     // no parts
      while (L.starts[k + 1] <= u.page_first) ++k;
      const int k0 = k;
      while (L.starts[k + 1] < u.page_first + pages[i]) ++k;
      u.n_parts = static_cast<uint8_t>(k - k0 + 1);
      u.first_cta = static_cast<uint8_t>(k0);
      if (k > k0) {
        u.part_base = static_cast<uint16_t>(part_cursor);
        part_cursor += k - k0 + 1;
      }
    }
    if ((size_t)part_cursor > slots)
      return fail(PA_ERR_INVALID, "internal: %d partial slots exceed the %zu reserved",
                  part_cursor, slots);
    plan->launches.push_back(std::move(L));
  }
  if (!merge) return PA_OK;
  // Completions each (request, kv head) pair's tile count reaches: one per
  // unsplit or empty unit, one per merge slice of a split unit.
  for (int g = 0; g < n_kv_heads; ++g) {
    for (int b = 0; b < B; ++b) {
      Unit* u = units.data() + (g * (size_t)B + b) * T;
      int count = 0;
      for (int t = 0; t < T; ++t) count += u[t].n_parts > 1 ? split_slices<false>(u[t].n_parts) : 1;
      for (int t = 0; t < T; ++t) u[t].pair_total = count;
    }
  }
  return PA_OK;
}

}  // namespace split
}  // namespace pa
