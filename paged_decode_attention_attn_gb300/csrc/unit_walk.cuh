// What the warps of the decode kernels over the 8-bit and the 4-bit pool do alike: walk
// their CTA's units, wait on mbarriers with a time limit, move small things to shared
// memory.  A kernel's parameter struct P has, beside what split_units.cuh names, n_full,
// grid, starts and first_unit (see unit_plan.h); its view V of shared memory bar(i), the
// address of barrier i, and abort_flag.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "split_units.cuh"

namespace pa {
namespace split {

// A unit as the kernel reads it: three 8-byte loads.
struct alignas(8) DevUnit {
  int32_t page_first, bt, tok_start, tok_end, g;
  uint16_t part_base;
  uint8_t n_parts, first_cta;
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

// The slow side of a wait, out of line: the roles' loops stay short (a warp on its own runs ~6
// cycles per instruction, and every line of code is fetched cold in a launch).
inline __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns,
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
template <class P, class V>
__device__ __forceinline__ bool wait(const P& p, const V& v, int bar, uint32_t parity) {
  const uint32_t b = v.bar(bar);
  if (ptx::mbar_try_wait(b, parity)) return true;
  return wait_long(b, parity, p.wait_limit_ns, p.status, v.abort_flag);
}
// The same for a converged warp, with one answer for all its lanes: false too if
// `ok` is false in one of them.  A warp skips tensor memory loads, and leaves its
// loop, by such an answer alone: lanes that gave up by themselves would be missed at
// the next instruction that takes the whole warp, by a wait without a limit.
template <class P, class V>
__device__ __forceinline__ bool warp_wait(const P& p, const V& v, int bar, uint32_t parity,
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

}  // namespace split
}  // namespace pa
