// Appends of a step's new tokens to a paged cache with the position rotation
// applied on the way, for bf16 pools and for 8-bit (e4m3) pools, and the
// gather that reads 8-bit rows back as bf16 values.
//
// Rotation: pair i of a head turns by the angle p * inv_freq[i] (p the token's
// position).  The angle is needed modulo one turn only, so inv_freq[i] / 2 pi
// is held as a 64-bit binary fraction of a turn and multiplied by the position
// in integers: the product wraps modulo one turn by itself and keeps its low
// bits at any position (fp32 angles lose all of them near 2^24).  No fp64 is
// used (its rate on this part made a prompt's angles cost more than its
// bytes).  A token's sines and cosines are computed once for all its heads.
//
// Rows (bf16 pool, and q of both kinds): a warp takes a token row, or a share
// of its heads when there are few rows; a lane keeps its pairs' sines and
// cosines in registers and moves 16 (or 8) bytes per load.
//
// 8-bit blocks: kBlock consecutive tokens of one head share one fp32 scale, a
// power of two, so rows that were already there are requantised exactly (but
// for codes that become subnormal) when a larger row makes the scale grow.
// One warp takes one (block, head), once for the largest value and once for
// the codes; the second reading of more than four rows comes from L1 (16 rows
// in registers left two CTAs per SM and half the rate of the launch).
//
// All of it is bound by HBM at prompt sizes and by the latency of its
// dependent loads (request, position, page, row) at decode sizes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "fp8.cuh"
#include "ptx.cuh"
#include "rope_rows.cuh"

namespace pa {
namespace rope {

constexpr int kBlock = PA_SCALE_TOKENS;
constexpr int kBlocks = kPage / kBlock;   // scale blocks per page

template <int D, int V>
__global__ void __launch_bounds__(kThreads, 3)
    append_rope_kernel(const Tokens t, __nv_bfloat16* pool, int share) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  rotate_rows<D, V, true>(t, pool, blockIdx.x, share);
}

template <int D, int V>
__global__ void __launch_bounds__(kThreads, 2)
    append_norm_rope_kernel(const Tokens t, const Norm norm, __nv_bfloat16* pool, int share) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  norm_rows<D, V, true>(t, norm, pool, blockIdx.x, share);
}

// Smallest power of two s >= 2^-60 with amax <= 448 s (448 = 1.75 * 2^8 is the
// largest e4m3 value), from the bits of a finite amax >= 0.
__device__ __forceinline__ float block_scale(unsigned amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return ptx::pow2i(max(e, -60));
}

// One (block, head) by one warp: rows [row, row + n_new) of the step go to the
// block's rows [first, first + n_new).  h counts K heads, then V heads.
template <int D, bool kKey>
__device__ __forceinline__ void store_block(const Tokens& t, uint8_t* pool, float* scales,
                                            const float (*cs)[2][D / 2], int row, int n_new,
                                            int first, long long page, int blk, int h, int lane) {
  constexpr int V = 4;
  constexpr int kLanes = D / (2 * V);
  constexpr int kRows = 32 / kLanes;         // token rows a warp takes at once
  constexpr int kUnroll = 4;
  const int sub = lane / kLanes;
  const Lane ln = lane_of<V>(lane % kLanes, kKey ? t.half : 0, t.interleaved);
  const long long stride = kKey ? t.k_stride : t.v_stride;
  const __nv_bfloat16* src =
      (kKey ? t.k + h * D : t.v + (h - t.Hkv) * D) + (row + sub) * stride;
  const int row_bytes = 2 * t.Hkv * D;
  uint8_t* base = pool + ((size_t)page * kPage + blk * kBlock) * row_bytes + (size_t)h * D;
  float* scale = scales + ((size_t)page * 2 * t.Hkv + h) * kBlocks + blk;
  const float old = first > 0 ? *scale : 0.f;
  Vec<V> a[kUnroll], b[kUnroll];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = r0 + i * kRows;
      if (r + sub < n_new) {
        a[i] = *reinterpret_cast<const Vec<V>*>(src + r * stride + ln.oa);
        b[i] = *reinterpret_cast<const Vec<V>*>(src + r * stride + ln.ob);
      } else {
        a[i] = b[i] = Vec<V>{};
      }
    }
  };
  auto values = [&](int i, int r, float (&y)[2 * V]) {   // of row r0 + r, held at i
    unpack<V>(a[i], b[i], y);
    if (kKey && ln.turns) {
      float c[V], s[V];
      *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(&cs[r][0][ln.pair]);
      *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(&cs[r][1][ln.pair]);
      rotate<V>(t.interleaved, c, s, y);
    }
  };
  // Largest magnitude but for NaN (finite: and infinities).
  auto largest = [&](bool finite) {
    float m = 0.f;
    for (int r0 = 0; r0 < n_new; r0 += kUnroll * kRows) {
      if (!finite || n_new > kUnroll * kRows) load(r0);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        float y[2 * V];
        // (rows behind the last are zeros, whatever they turn by)
        values(i, (r0 + i * kRows + sub) % kBlock, y);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
          if (finite && fabsf(y[j]) > FLT_MAX) y[j] = 0.f;
          m = fmaxf(m, fabsf(y[j]));
        }
      }
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  };
  float amax = largest(false);
  const bool infinite = amax > FLT_MAX;
  if (infinite) amax = largest(true);
  const float need = block_scale(__float_as_uint(amax));
  const float s = first > 0 ? fmaxf(old, need) : need;
  if (first > 0 && s != old) {
    // The scale grows: the block's older rows are requantised.
    const float ratio = old / s;
    for (int r = sub; r < first; r += kRows) {
      uint32_t* pa = reinterpret_cast<uint32_t*>(base + r * row_bytes + ln.oa);
      uint32_t* pb = reinterpret_cast<uint32_t*>(base + r * row_bytes + ln.ob);
      const uint32_t ca = *pa, cb = *pb;
      *pa = fp8::scale4(ca, ratio);
      *pb = fp8::scale4(cb, ratio);
    }
  }
  const float inv = 1.0f / s;   // exact for a power of two
  uint8_t* dst = base + (first + sub) * row_bytes;
  for (int r0 = 0; r0 < n_new; r0 += kUnroll * kRows) {
    if (n_new > kUnroll * kRows) load(r0);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = r0 + i * kRows;
      if (r + sub >= n_new) break;
      float y[2 * V];
      values(i, r + sub, y);
      if (infinite) {   // (a NaN stays one by itself)
#pragma unroll
        for (int j = 0; j < 2 * V; ++j)
          if (fabsf(y[j]) > FLT_MAX) y[j] = __int_as_float(0x7fc00000);
      }
#pragma unroll
      for (int j = 0; j < 2 * V; ++j) y[j] *= inv;
      *reinterpret_cast<uint32_t*>(dst + r * row_bytes + ln.oa) =
          fp8::pack4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint32_t*>(dst + r * row_bytes + ln.ob) =
          fp8::pack4(y[4], y[5], y[6], y[7]);
    }
  }
  if (lane == 0 && (first == 0 || s != old)) *scale = s;
}

// kv_ctas CTAs take `chunk` token rows each and store the blocks whose first
// new row lies among them (a request's first new row, or a row on a block
// border); the others rotate q rows.  The two kinds alternate, so that an SM
// has CTAs that wait for their loads beside CTAs that stream.
template <int D, int V>
__global__ void __launch_bounds__(kThreads, 3)
    append_rope_q8_kernel(const Tokens t, uint8_t* pool, float* scales, int kv_ctas, int chunk,
                          int share) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int pairs = min(kv_ctas, (int)gridDim.x - kv_ctas);
  const bool paired = (int)blockIdx.x < 2 * pairs;
  const int cta = paired ? blockIdx.x / 2 : blockIdx.x - pairs;
  if (paired ? blockIdx.x & 1 : pairs == kv_ctas) {
    rotate_rows<D, V, false>(t, nullptr, cta, share);
    return;
  }
  __shared__ __align__(16) float cs[kBlock][2][D / 2];
  __shared__ long long s_pos[kBlock], s_page[kBlock];
  __shared__ int s_new[kBlock];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = cta * chunk;
  for (int r = warp; r < chunk; r += kWarps) {
    const int row = row0 + r;
    int b, first, end, n = 0;
    long long pos = 0, page = -1;
    if (row < t.n_tokens &&
        locate(t.cu, t.positions, t.B, t.n_tokens, row, lane, &b, &pos, &first, &end) &&
        (row == first || pos % kBlock == 0)) {
      page = page_of(t.page_table, t.max_pages, t.pool_pages, b, pos);
      if (page >= 0) n = min(kBlock - (int)(pos % kBlock), end - row);
      else if (lane == 0 && t.status) atomicOr(t.status, PA_STATUS_BAD_ROW);
    }
    if (lane == 0) {
      s_pos[r] = pos;
      s_page[r] = page;
      s_new[r] = n;
    }
  }
  __syncthreads();
  for (int r = 0; r < chunk; ++r) {
    const int n = s_new[r];
    if (n <= 0) continue;
    const long long pos = s_pos[r];
    const int in_page = (int)(pos % kPage);
    // Half the warps take K heads, after they made the table of angles; the
    // others V heads, which need none.
    constexpr int kKWarps = kWarps / 2, kKThreads = 32 * kKWarps;
    int h = warp;
    if (warp < kKWarps) {
      for (int j = threadIdx.x; j < t.half; j += kKThreads) {
        const float f = __ldg(t.inv_freq + j), nan = not_finite(f);
        const unsigned long long step = turn_step(f);
        for (int k = 0; k < n; ++k) turn(pos + k, step, nan, &cs[k][1][j], &cs[k][0][j]);
      }
      ptx::named_barrier(1, kKThreads);
    } else {
      h = t.Hkv + warp - kKWarps;
    }
    if (warp < kKWarps) {
      for (; h < t.Hkv; h += kKWarps)
        store_block<D, true>(t, pool, scales, cs, row0 + r, n, in_page % kBlock, s_page[r],
                             in_page / kBlock, h, lane);
      // (the table is not made again before every K warp is done with it)
      ptx::named_barrier(1, kKThreads);
    } else {
      for (; h < 2 * t.Hkv; h += kKWarps)
        store_block<D, false>(t, pool, scales, cs, row0 + r, n, in_page % kBlock, s_page[r],
                              in_page / kBlock, h, lane);
    }
  }
}

// Rows of an 8-bit pool as bf16 values: `share` warps to a row, a lane turns 16
// codes of one head at a time and stores them whole (two 16-byte stores a lane
// took 13.8 us where this takes 10.7, for 8,000 rows of 2,048 codes).
__global__ void __launch_bounds__(kThreads)
    gather_q8_kernel(const uint8_t* pool, const float* scales, long long pool_pages,
                     const int32_t* page_table, int max_pages, const int32_t* cu,
                     const int32_t* positions, int n_tokens, int B, int heads, int d, int share,
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
  const int at = (int)(pos % kPage);
  const uint4* src = reinterpret_cast<const uint4*>(
      pool + ((size_t)(page < 0 ? 0 : page) * kPage + (page < 0 ? 0 : at)) * heads * d);
  const float* sc = scales + (size_t)(page < 0 ? 0 : page) * heads * kBlocks +
                    (page < 0 ? 0 : at / kBlock);
  uint4* dst = reinterpret_cast<uint4*>(out + (size_t)row * heads * d);
  const int per_row = heads * d / 16, step = 32 * share;
  constexpr int kUnroll = 4;
  for (int c0 = (warp % share) * 32 + lane; c0 < per_row; c0 += kUnroll * step) {
    uint4 codes[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * step;
      codes[i] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);   // NaN
      s[i] = 1.f;
      if (c < per_row && page >= 0) {
        codes[i] = __ldg(src + c);
        s[i] = __ldg(sc + c * 16 / d * kBlocks);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * step;
      if (c >= per_row) break;
      const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y[4];
        fp8::unpack4(w[j], y);
        o[2 * j] = ptx::pack_bf16x2(__float2bfloat16_rn(y[0] * s[i]),
                                     __float2bfloat16_rn(y[1] * s[i]));
        o[2 * j + 1] = ptx::pack_bf16x2(__float2bfloat16_rn(y[2] * s[i]),
                                        __float2bfloat16_rn(y[3] * s[i]));
      }
      store32(dst + 2 * c, o);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

template <int D, int V>
cudaError_t launch_append(const Tokens& t, void* pool, cudaStream_t stream) {
  int share, ctas;
  row_grid(t.n_tokens, &share, &ctas);
  return launch_dependent(append_rope_kernel<D, V>, dim3(ctas), dim3(kThreads), 0, stream, t,
                          static_cast<__nv_bfloat16*>(pool), share);
}

template <int D, int V>
cudaError_t launch_append_norm(const Tokens& t, const Norm& norm, void* pool,
                               cudaStream_t stream) {
  int share, ctas;
  row_grid(t.n_tokens, &share, &ctas);
  return launch_dependent(append_norm_rope_kernel<D, V>, dim3(ctas), dim3(kThreads), 0, stream, t,
                          norm, static_cast<__nv_bfloat16*>(pool), share);
}

// Token rows a CTA looks through for blocks to store: a power of two that leaves
// about two waves of CTAs (one that finds none leaves at once; one that finds
// several takes them one after the other), but no more than a request has on
// average, or 2 where most rows are a request, and so a block, of their own.  (1 / 2 / 4 / 8 / 16 rows, with q:
// 40 requests of up to 71 tokens 17.5 / 16.1 / 15.9 / 18.0 / 22.6 us; 3 of 600
// 20.5 / 17.9 / 17.1 / 17.9 / 20.8; 2 of 4,050 57.8 / 51.5 / 48.4 / 46.6 / 45.8;
// 1,200 of one 19.4 / 16.6 / 19.8 / 23.4 / 41.6.)
int rows_per_cta(int n_tokens, int B) {
  int rows = 1;
  while (rows < kBlock && rows * 760ll < n_tokens) rows *= 2;
  return std::min(rows, std::max(2, n_tokens / B));
}

template <int D, int V>
cudaError_t launch_append_q8(const Tokens& t, void* pool, float* scales, cudaStream_t stream) {
  const int chunk = rows_per_cta(t.n_tokens, t.B);
  const int kv = (t.n_tokens + chunk - 1) / chunk;
  int share = 1, q = 0;
  if (t.q) row_grid(t.n_tokens, &share, &q);
  return launch_dependent(append_rope_q8_kernel<D, V>, dim3(kv + q), dim3(kThreads), 0, stream, t,
                          static_cast<uint8_t*>(pool), scales, kv, chunk, share);
}

}  // namespace rope
}  // namespace pa

extern "C" int kv_append_rope(const void* q, const void* k, const void* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, void* q_out,
                              int64_t q_out_stride, const int32_t* cu_tokens,
                              const int32_t* positions, int n_tokens, int B, int n_q_heads,
                              int n_kv_heads, int head_dim, const float* inv_freq, int rot_dim,
                              unsigned flags, void* pool, int64_t pool_pages,
                              const int32_t* page_table, int max_pages, int32_t* status,
                              cudaStream_t stream) {
  using namespace pa::rope;
  pa::clear_error();
  const Tokens t = tokens_of(q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, cu_tokens,
                             positions, n_tokens, B, n_q_heads, n_kv_heads, inv_freq, rot_dim,
                             flags, pool_pages, page_table, max_pages, status);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return pa::fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 64, 128, 256)",
                    head_dim);
  const int rc = check_tokens(t, head_dim, rot_dim, flags, pool);
  if (rc != PA_OK || n_tokens == 0 || B == 0) return rc;
  const bool w = wide(t);
  PA_CHECK_CUDA(head_dim == 64 ? (w ? launch_append<64, 8>(t, pool, stream)
                                    : launch_append<64, 4>(t, pool, stream))
                : head_dim == 128 ? (w ? launch_append<128, 8>(t, pool, stream)
                                       : launch_append<128, 4>(t, pool, stream))
                                  : (w ? launch_append<256, 8>(t, pool, stream)
                                       : launch_append<256, 4>(t, pool, stream)));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}

extern "C" int kv_append_norm_rope(const void* q, const void* k, const void* v, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, void* q_out,
                                   int64_t q_out_stride, const int32_t* cu_tokens,
                                   const int32_t* positions, int n_tokens, int B, int n_q_heads,
                                   int n_kv_heads, int head_dim, const float* q_weight,
                                   const float* k_weight, float eps, const float* inv_freq,
                                   int rot_dim, unsigned flags, void* pool, int64_t pool_pages,
                                   const int32_t* page_table, int max_pages, int32_t* status,
                                   cudaStream_t stream) {
  using namespace pa::rope;
  pa::clear_error();
  const Tokens t = tokens_of(q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, cu_tokens,
                             positions, n_tokens, B, n_q_heads, n_kv_heads, inv_freq, rot_dim,
                             flags, pool_pages, page_table, max_pages, status);
  const Norm norm{q_weight, k_weight, eps};
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return pa::fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 64, 128, 256)",
                    head_dim);
  int rc = check_tokens(t, head_dim, rot_dim, flags, pool);
  if (rc != PA_OK || n_tokens == 0 || B == 0) return rc;
  rc = check_norm(t, norm);
  if (rc != PA_OK) return rc;
  const bool w = wide(t);
  PA_CHECK_CUDA(head_dim == 64 ? (w ? launch_append_norm<64, 8>(t, norm, pool, stream)
                                    : launch_append_norm<64, 4>(t, norm, pool, stream))
                : head_dim == 128 ? (w ? launch_append_norm<128, 8>(t, norm, pool, stream)
                                       : launch_append_norm<128, 4>(t, norm, pool, stream))
                                  : (w ? launch_append_norm<256, 8>(t, norm, pool, stream)
                                       : launch_append_norm<256, 4>(t, norm, pool, stream)));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}

extern "C" int kv_append_rope_q8(const void* q, const void* k, const void* v, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, void* q_out,
                                 int64_t q_out_stride, const int32_t* cu_tokens,
                                 const int32_t* positions, int n_tokens, int B, int n_q_heads,
                                 int n_kv_heads, int head_dim, const float* inv_freq, int rot_dim,
                                 unsigned flags, void* pool, float* scales, int64_t pool_pages,
                                 const int32_t* page_table, int max_pages, int32_t* status,
                                 cudaStream_t stream) {
  using namespace pa::rope;
  pa::clear_error();
  const Tokens t = tokens_of(q, k, v, q_stride, k_stride, v_stride, q_out, q_out_stride, cu_tokens,
                             positions, n_tokens, B, n_q_heads, n_kv_heads, inv_freq, rot_dim,
                             flags, pool_pages, page_table, max_pages, status);
  if (head_dim != 128 && head_dim != 256)
    return pa::fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 128, 256)", head_dim);
  const int rc = check_tokens(t, head_dim, rot_dim, flags, pool);
  if (rc != PA_OK || n_tokens == 0 || B == 0) return rc;
  PA_REQUIRE(scales != nullptr && aligned16(scales), "scales must be non-null, 16-byte aligned");
  const bool w = wide(t);
  PA_CHECK_CUDA(head_dim == 128 ? (w ? launch_append_q8<128, 8>(t, pool, scales, stream)
                                     : launch_append_q8<128, 4>(t, pool, scales, stream))
                                : (w ? launch_append_q8<256, 8>(t, pool, scales, stream)
                                     : launch_append_q8<256, 4>(t, pool, scales, stream)));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}

extern "C" int kv_gather_q8(const void* pool, const float* scales, int64_t pool_pages,
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
      gather_q8_kernel, dim3(ctas), dim3(kThreads), 0, stream,
      static_cast<const uint8_t*>(pool), scales, (long long)pool_pages, page_table, max_pages,
      cu_tokens, positions, n_tokens, B, 2 * n_kv_heads, head_dim, share,
      static_cast<__nv_bfloat16*>(out), status));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}
