// q of a segment as e4m3 operands of the first product: shared by the 8-bit and the 4-bit
// pool's decode kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8.cuh"
#include "ptx.cuh"
#include "split_units.cuh"
#include "unit_walk.cuh"

namespace pa {
namespace split {

constexpr int kQParts = 4;                  // e4m3 parts of q, each scaled up from the
// one before by these: the second holds what the first leaves of 8 bits, and what
// these two leave, of values below 256, is at most 2^-15.
constexpr float kQScale1 = 32.f, kQScale2 = 1 << 18, kQScale3 = 32.f;
constexpr int kQCols = kQParts * kMaxG;     // N of the first product
constexpr int kChunk = 128;                 // dims per 128-byte row

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
// S: the kernel's layout of shared memory, with kQ, kQBytes, kQChunkBytes and kQScale (the
// heads' factors); p.scale_log2 is the scores' scale.
template <class S, int D, class P, class V>
__device__ __forceinline__ void convert_head(const P& p, const V& v, const QVec<D>& raw,
                                             int buffer, int h, int lane) {
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

}  // namespace split
}  // namespace pa
