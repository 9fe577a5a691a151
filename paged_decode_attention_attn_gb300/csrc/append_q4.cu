// Appends of a step's new tokens to a 4-bit pool (e2m1 codes, a power of two as the
// scale of each 32 values of a token's head) with the norms of q and k heads and the
// position rotation on the way, and the gather that reads rows back as bf16 values.
//
// A token's codes and scales depend on no other token, so a row is stored by the warp
// that takes it, whatever its request: no block is shared, nothing is read back.  A lane
// takes 8 neighbouring values of a head, so four lanes hold a scale's group (two
// shuffles find its largest value) and a lane stores a word of codes.  Pairs that lie
// half a rotation apart are in another lane's values: those are loaded a second time
// (from L1) instead of exchanged.  q rows go as in the appends to the other pools, by
// CTAs of their own.
//
// Decode sizes are bound by the latency of dependent loads (request, position, page, row:
// 1-96 tokens 3.7-4.5 us and 2 us for the gather); prompts by instructions and their loads'
// latency (8,000 tokens of 24 q and 4 kv heads of 256 dims with norms 63.3 us where the bytes
// take 35, their gather 7.4 where they take 6.2).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "common.h"
#include "fp4.cuh"
#include "ptx.cuh"
#include "rope_rows.cuh"

namespace pa {
namespace rope {

constexpr int kGroup = PA_Q4_GROUP;

// A key near a border between two codes may go either way by the rounding of its norm and
// turn.  Which way is fixed here as that of one form in plain fp32, an array library's for a
// GPU, so that a pool filled here and one filled by such a form agree code by code:
// x * rsqrt(sum / D + eps) * w with each product rounded, sines and cosines the nearest floats,
// a c - b s with both products and the difference rounded, and the squares of a row of D
// summed as written at sum_of_squares().

// A product of two sums of two floats each, the second of each the small part.
__device__ __forceinline__ float2 times_fine(float2 a, float2 b) {
  const float h = __fmul_rn(a.x, b.x);
  return make_float2(h, fmaf(a.x, b.x, -h) + fmaf(a.x, b.y, a.y * b.x));
}
// a + b for |b| <= |a|, rounded once.
__device__ __forceinline__ float add_fine(float a, float2 b, float a_lo) {
  const float s = __fadd_rn(a, b.x), rest = __fadd_rn(__fsub_rn(a, s), b.x);
  return __fadd_rn(s, rest + (b.y + a_lo));
}
// c + q z, |q z| <= |c| / 2.
__device__ __forceinline__ float2 fma_fine(float q, float2 z, float2 c) {
  const float h = fmaf(q, z.x, c.x);
  return make_float2(h, fmaf(q, z.x, __fsub_rn(c.x, h)) + fmaf(q, z.y, c.y));
}

// Sine and cosine at position p (see turn()), the nearest floats but for 2 in 100,000 (at most
// 0.5003 units in the last place): the angle's rest x, and the series' terms behind x and 1 -
// x^2 / 2, in two floats each.
__device__ __forceinline__ void turn_fine(long long p, unsigned long long step, float nan,
                                          float* s, float* c) {
  const unsigned long long at = step * (unsigned long long)p;
  const unsigned quarter = (unsigned)((at + (1ull << 61)) >> 62);
  const long long rest = (long long)(at - ((unsigned long long)quarter << 62));
  constexpr float kHi = 3.40612167e-19f, kLo = -9.47839643e-27f;   // 2 pi 2^-64
  const float hi = __ll2float_rn(rest), lo = __ll2float_rn(rest - __float2ll_rn(hi));
  float2 x, z;
  x.x = __fmul_rn(hi, kHi);
  x.y = fmaf(hi, kHi, -x.x) + fmaf(hi, kLo, lo * kHi);
  z.x = __fmul_rn(x.x, x.x);
  z.y = fmaf(x.x, x.x, -z.x) + 2.f * x.x * x.y;
  constexpr float kLo6 = 4.967054e-09f, kLo24 = -1.2417635e-09f, kLo120 = -4.346172e-10f;
  float a = fmaf(z.x, -1.0f / 39916800.0f, 1.0f / 362880.0f);
  a = fmaf(a, z.x, -1.0f / 5040.0f);
  const float2 a2 = fma_fine(a, z, make_float2(1.0f / 120.0f, kLo120));
  float2 a3 = fma_fine(a2.x, z, make_float2(-1.0f / 6.0f, kLo6));
  a3.y = fmaf(a2.y, z.x, a3.y);
  const float sx = add_fine(x.x, times_fine(x, times_fine(z, a3)), x.y);
  float b = fmaf(z.x, 1.0f / 479001600.0f, -1.0f / 3628800.0f);
  b = fmaf(b, z.x, 1.0f / 40320.0f);
  b = fmaf(b, z.x, -1.0f / 720.0f);
  const float2 b2 = fma_fine(b, z, make_float2(1.0f / 24.0f, kLo24));
  const float h = __fsub_rn(1.f, 0.5f * z.x), h_lo = __fsub_rn(1.f, h) - 0.5f * z.x - 0.5f * z.y;
  const float cx = add_fine(h, times_fine(times_fine(z, z), b2), h_lo);
  const bool odd = quarter & 1;
  const float ss = odd ? cx : sx, cc = odd ? sx : cx;
  *s = (quarter & 2 ? -ss : ss) + nan;
  *c = ((quarter + 1) & 2 ? -cc : cc) + nan;
}

// The sum of a head's squares: a lane has 8 neighbours, the head D / 8 lanes.  All lanes call.
// Of 256: those of dims i and i + 128, then of four neighbours in turn, then of neighbouring
// sums pair by pair; of 128: of dims i, i + 32, i + 64 and i + 96 in turn, then pair by pair.
template <int D>
__device__ __forceinline__ float sum_of_squares(const float (&y)[8], float by) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = y[j] * by;
    t[j] = __fmul_rn(x, x);
  }
  float ss;
  if constexpr (D == 256) {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __fadd_rn(t[j], __shfl_xor_sync(0xffffffffu, t[j], 16));
    ss = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), t[2]), t[3]),
                   __fadd_rn(__fadd_rn(__fadd_rn(t[4], t[5]), t[6]), t[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = threadIdx.x & 0x13;
      float u = __shfl_sync(0xffffffffu, t[j], at);
#pragma unroll
      for (int k = 1; k < 4; ++k) u = __fadd_rn(u, __shfl_sync(0xffffffffu, t[j], at + 4 * k));
      t[j] = u;
    }
    ss = __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                   __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7])));
  }
#pragma unroll
  for (int off = 1; off < (D == 256 ? 16 : 4); off *= 2)
    ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
  return ss;
}

// A head's 1 / sqrt(mean + eps) of its D squares, and `pre`, the power of two that its
// values are multiplied by first (1, unless squares pass the range of fp32: bf16 values
// reach 2^128, and x 2^-70 has a square and a sum in range, beside which eps is nothing).
// sum(by): of the squares of the values times `by`, in all lanes of the head.  All lanes of
// the warp call.
template <int D, class Sum>
__device__ __forceinline__ float norm_of(Sum sum, float eps, float* pre) {
  float ss = sum(1.f);
  *pre = 1.f;
  const bool large = !(ss <= FLT_MAX);
  if (__any_sync(0xffffffffu, large)) {
    const float again = sum(ptx::pow2i(-70));
    if (large) {
      ss = again;
      eps = 0.f;
      *pre = ptx::pow2i(-70);
    }
  }
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

// The k and v heads of a row into the 4-bit pool.  `share` warps to a row, this one the
// w-th; cs: the row's cosines and sines.
template <int D, bool kNorm>
__device__ __forceinline__ void store_row_q4(const Tokens& t, const Norm& norm,
                                             const float (*weights)[D],
                                             const float (*cs)[D / 2], int row, uint8_t* pool,
                                             uint8_t* scales, long long page, int at, int w,
                                             int share, int lane) {
  constexpr int kN = 8;                      // values per lane
  constexpr int kLanes = D / kN;             // lanes per head
  constexpr int kHeads = 32 / kLanes;        // heads a warp takes at once
  constexpr int kUnroll = 4;
  const int sub = lane / kLanes, l = lane % kLanes, d0 = kN * l;
  const int heads = 2 * t.Hkv, step = share * kHeads;
  const __nv_bfloat16* k = t.k + row * t.k_stride + d0;
  const __nv_bfloat16* v = t.v + row * t.v_stride + d0;
  // Two runs of four values; of each, where its pairs are (multiples of four all) and
  // the sign of the partner's part.
  int other[2], pair[2];
  float sign[2];
  bool turns[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = d0 + 4 * j;
    turns[j] = c < 2 * t.half;
    const bool second = !t.interleaved && c >= t.half;
    pair[j] = t.interleaved ? c / 2 : second ? c - t.half : c;
    other[j] = !turns[j] || t.interleaved ? 0 : second ? -t.half : t.half;
    sign[j] = second ? 1.f : -1.f;
  }
  for (int h0 = w * kHeads; h0 < heads; h0 += kUnroll * step) {
    uint4 own[kUnroll];
    uint2 far[kUnroll][2];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + sub + i * step;
      own[i] = make_uint4(0u, 0u, 0u, 0u);
      far[i][0] = far[i][1] = make_uint2(0u, 0u);
      if (h >= heads) continue;
      const __nv_bfloat16* src = h < t.Hkv ? k + h * D : v + (h - t.Hkv) * D;
      own[i] = *reinterpret_cast<const uint4*>(src);
      if (h >= t.Hkv) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (other[j] != 0) far[i][j] = *reinterpret_cast<const uint2*>(src + 4 * j + other[j]);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + sub + i * step;
      if (h0 + i * step >= heads) break;   // (of the whole warp)
      const bool key = h < t.Hkv;
      float y[kN];
      const uint32_t word[4] = {own[i].x, own[i].y, own[i].z, own[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = ptx::bf16_lo_to_f32(word[j]);
        y[2 * j + 1] = ptx::bf16_hi_to_f32(word[j]);
      }
      float r = 1.f, pre = 1.f;
      if (kNorm && h - sub < t.Hkv) {   // (of the whole warp: a k head is among its)
        r = norm_of<D>([&](float by) { return sum_of_squares<D>(y, by); }, norm.eps, &pre);
        if (key) {
#pragma unroll
          for (int j = 0; j < kN; ++j) y[j] = y[j] * pre * r * weights[1][d0 + j];
        }
      }
      if (key) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!turns[j]) continue;
          float* x = y + 4 * j;
          if (t.interleaved) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const float c = cs[0][pair[j] + m], s = cs[1][pair[j] + m];
              const float a = x[2 * m], b = x[2 * m + 1];
              x[2 * m] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
              x[2 * m + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
            }
          } else {
            float z[4] = {ptx::bf16_lo_to_f32(far[i][j].x), ptx::bf16_hi_to_f32(far[i][j].x),
                          ptx::bf16_lo_to_f32(far[i][j].y), ptx::bf16_hi_to_f32(far[i][j].y)};
            const float4 c4 = *reinterpret_cast<const float4*>(&cs[0][pair[j]]);
            const float4 s4 = *reinterpret_cast<const float4*>(&cs[1][pair[j]]);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              if constexpr (kNorm)
                z[m] = z[m] * pre * r * weights[1][d0 + 4 * j + other[j] + m];
              x[m] = __fadd_rn(__fmul_rn(x[m], c[m]), sign[j] * __fmul_rn(z[m], s[m]));
            }
          }
        }
      }
      // (as integers the bits of NaN lie above infinity's, and those above all others)
      unsigned amax = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) amax = max(amax, __float_as_uint(y[j]) & 0x7fffffffu);
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const bool finite = amax < 0x7f800000u;
      const int e = finite ? fp4::scale_exp(amax) : 0;
      const float inv = finite ? ptx::pow2i(-e) : 0.f;   // exact
#pragma unroll
      for (int j = 0; j < kN; ++j) y[j] *= inv;
      const uint32_t codes = finite ? fp4::pack8(y) : 0u;
      if (h >= heads) continue;
      const size_t place = ((size_t)page * heads + h) * kPage + at;
      *reinterpret_cast<uint32_t*>(pool + place * (D / 2) + 4 * l) = codes;
      if (l % 4 == 0)
        scales[place * (D / kGroup) + l / 4] =
            static_cast<uint8_t>(finite ? e + fp4::kScaleBias : fp4::kNanScale);
    }
  }
}

// CTA kv_cta's rows of k and v.
template <int D, bool kNorm>
__device__ __forceinline__ void store_rows_q4(const Tokens& t, const Norm& norm, uint8_t* pool,
                                              uint8_t* scales, int kv_cta, int share) {
  __shared__ __align__(16) float cs[kWarps][2][D / 2];
  __shared__ __align__(16) float weights[kNorm ? 2 : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = kv_cta * (kWarps / share) + warp / share;
  if constexpr (kNorm) {
    load_weights<D, true>(norm, false, weights);
    __syncthreads();
  }
  if (row >= t.n_tokens) return;
  int b = 0, first, end;
  long long pos = 0;
  if (!locate(t.cu, t.positions, t.B, t.n_tokens, row, lane, &b, &pos, &first, &end)) return;
  const long long page = page_of(t.page_table, t.max_pages, t.pool_pages, b, pos);
  if (page < 0) {
    if (lane == 0 && t.status) atomicOr(t.status, PA_STATUS_BAD_ROW);
    return;
  }
  for (int i = lane; i < t.half; i += 32) {
    const float f = __ldg(t.inv_freq + i);
    turn_fine(pos, turn_step(f), not_finite(f), &cs[warp][1][i], &cs[warp][0][i]);
  }
  __syncwarp();
  store_row_q4<D, kNorm>(t, norm, weights, cs[warp], row, pool, scales, page, (int)(pos % kPage),
                         warp % share, share, lane);
}

// kv_ctas CTAs store rows of k and v, the others rotate q rows; the kinds alternate, so
// that an SM has both.
template <int D, int V, bool kNorm>
__global__ void __launch_bounds__(kThreads, kNorm ? 3 : 2)
    append_rope_q4_kernel(const Tokens t, const Norm norm, uint8_t* pool, uint8_t* scales,
                          int kv_ctas, int kv_share, int q_share) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int pairs = min(kv_ctas, (int)gridDim.x - kv_ctas);
  const bool paired = (int)blockIdx.x < 2 * pairs;
  const int cta = paired ? blockIdx.x / 2 : blockIdx.x - pairs;
  if (paired ? blockIdx.x & 1 : pairs == kv_ctas) {
    if constexpr (kNorm) norm_rows<D, V, false>(t, norm, nullptr, cta, q_share);
    else rotate_rows<D, V, false>(t, nullptr, cta, q_share);
  } else {
    store_rows_q4<D, kNorm>(t, norm, pool, scales, cta, kv_share);
  }
}

// Rows of a 4-bit pool as bf16 values: `share` warps to a row, a lane turns 16 codes of
// one head at a time and stores them whole.
template <int D>
__global__ void __launch_bounds__(kThreads)
    gather_q4_kernel(const uint8_t* pool, const uint8_t* scales, long long pool_pages,
                     const int32_t* page_table, int max_pages, const int32_t* cu,
                     const int32_t* positions, int n_tokens, int B, int heads, int share,
                     __nv_bfloat16* out, int32_t* status) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kWarps / share) + warp / share;
  if (row >= n_tokens) return;
  int b = 0, first, end;
  long long pos = 0;
  if (!locate(cu, positions, B, n_tokens, row, lane, &b, &pos, &first, &end)) return;
  const long long page = page_of(page_table, max_pages, pool_pages, b, pos);
  if (page < 0 && lane == 0 && status) atomicOr(status, PA_STATUS_BAD_ROW);
  const size_t place = page < 0 ? 0 : (size_t)page * heads * kPage + pos % kPage;   // of head 0
  uint4* dst = reinterpret_cast<uint4*>(out + (size_t)row * heads * D);
  constexpr int kPer = D / 16, kUnroll = 4;
  const int per_row = heads * kPer, step = 32 * share;
  for (int c0 = (warp % share) * 32 + lane; c0 < per_row; c0 += kUnroll * step) {
    uint2 codes[kUnroll];
    unsigned byte[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * step;
      codes[i] = make_uint2(0u, 0u);
      byte[i] = fp4::kNanScale;
      if (c < per_row && page >= 0) {
        const size_t head = place + (size_t)(c / kPer) * kPage;
        codes[i] = __ldg(reinterpret_cast<const uint2*>(pool + head * (D / 2)) + c % kPer);
        byte[i] = __ldg(scales + head * (D / kGroup) + c % kPer / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * step;
      if (c >= per_row) break;
      const float s = fp4::scale_of(byte[i]);
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float y[8];
        fp4::unpack8(j ? codes[i].y : codes[i].x, y);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          o[4 * j + m] = ptx::round_bf16x2(y[2 * m] * s, y[2 * m + 1] * s);
      }
      store32(dst + 2 * c, o);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <int D, int V, bool kNorm>
cudaError_t launch_append_q4(const Tokens& t, const Norm& norm, void* pool, uint8_t* scales,
                             cudaStream_t stream) {
  int kv_share, kv, q_share = 1, q = 0;
  row_grid(t.n_tokens, &kv_share, &kv);
  if (t.q) row_grid(t.n_tokens, &q_share, &q);
  return launch_dependent(append_rope_q4_kernel<D, V, kNorm>, dim3(kv + q), dim3(kThreads), 0,
                          stream, t, norm, static_cast<uint8_t*>(pool), scales, kv, kv_share,
                          q_share);
}

// (q rows with norms go by 4 pairs of a lane, three CTAs to an SM: two prompts of 8,054 tokens with
// 24 q and 4 kv heads of 256 dims 63.6 us, 32 and 8 of 128 50.4; by 8, two CTAs: 66.5 and 53.6.
// 1-96 tokens alike.)
template <int D>
cudaError_t launch_append_q4(const Tokens& t, const Norm& norm, bool normed, void* pool,
                             uint8_t* scales, cudaStream_t stream) {
  return normed    ? launch_append_q4<D, 4, true>(t, norm, pool, scales, stream)
         : wide(t) ? launch_append_q4<D, 8, false>(t, norm, pool, scales, stream)
                   : launch_append_q4<D, 4, false>(t, norm, pool, scales, stream);
}

}  // namespace rope
}  // namespace pa

extern "C" int kv_append_rope_q4(const void* q, const void* k, const void* v, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, void* q_out,
                                 int64_t q_out_stride, const int32_t* cu_tokens,
                                 const int32_t* positions, int n_tokens, int B, int n_q_heads,
                                 int n_kv_heads, int head_dim, const float* q_weight,
                                 const float* k_weight, float eps, const float* inv_freq,
                                 int rot_dim, unsigned flags, void* pool, uint8_t* scales,
                                 int64_t pool_pages, const int32_t* page_table, int max_pages,
                                 int32_t* status, cudaStream_t stream) {
  using namespace pa::rope;
  pa::clear_error();
  const Tokens t = tokens_of(q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, cu_tokens,
                             positions, n_tokens, B, n_q_heads, n_kv_heads, inv_freq, rot_dim,
                             flags, pool_pages, page_table, max_pages, status);
  const Norm norm{q_weight, k_weight, eps};
  const bool normed = q_weight || k_weight;
  if (head_dim != 128 && head_dim != 256)
    return pa::fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 128, 256)", head_dim);
  int rc = check_tokens(t, head_dim, rot_dim, flags, pool);
  if (rc != PA_OK || n_tokens == 0 || B == 0) return rc;
  PA_REQUIRE(scales != nullptr && aligned16(scales), "scales must be non-null, 16-byte aligned");
  if (normed && (rc = check_norm(t, norm)) != PA_OK) return rc;
  PA_CHECK_CUDA(head_dim == 128 ? launch_append_q4<128>(t, norm, normed, pool, scales, stream)
                                : launch_append_q4<256>(t, norm, normed, pool, scales, stream));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}

extern "C" int kv_gather_q4(const void* pool, const uint8_t* scales, int64_t pool_pages,
                            const int32_t* page_table, int max_pages, const int32_t* cu_tokens,
                            const int32_t* positions, int n_tokens, int B, int n_kv_heads,
                            int head_dim, void* out, int32_t* status, cudaStream_t stream) {
  using namespace pa::rope;
  pa::clear_error();
  PA_REQUIRE(n_tokens >= 0 && B >= 0, "n_tokens and B must be >= 0 (got %d, %d)", n_tokens, B);
  if (head_dim != 128 && head_dim != 256)
    return pa::fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 128, 256)", head_dim);
  if (n_tokens == 0 || B == 0) return PA_OK;
  PA_REQUIRE(n_tokens <= kMaxTokens, "n_tokens (%d) above %d", n_tokens, kMaxTokens);
  PA_REQUIRE(n_kv_heads >= 1 && n_kv_heads <= 4096, "n_kv_heads (%d) must be in 1..4096",
             n_kv_heads);
  PA_REQUIRE(pool && scales && page_table && positions && out, "null pointer argument");
  PA_REQUIRE(cu_tokens || n_tokens == B, "without cu_tokens there is one row per request");
  PA_REQUIRE(aligned16(pool) && aligned16(scales), "pool and scales must be 16-byte aligned");
  PA_REQUIRE(reinterpret_cast<uintptr_t>(out) % 32 == 0, "out must be 32-byte aligned");
  PA_REQUIRE(pool_pages >= 1 && max_pages >= 1, "pool_pages and max_pages must be >= 1");
  int share, ctas;
  row_grid(n_tokens, &share, &ctas);
  PA_CHECK_CUDA(pa::launch_dependent(
      head_dim == 128 ? gather_q4_kernel<128> : gather_q4_kernel<256>, dim3(ctas), dim3(kThreads),
      0, stream, static_cast<const uint8_t*>(pool), scales, (long long)pool_pages, page_table,
      max_pages, cu_tokens, positions, n_tokens, B, 2 * n_kv_heads, share,
      static_cast<__nv_bfloat16*>(out), status));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}
