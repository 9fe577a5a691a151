// Appends of a step's new tokens to a paged cache with the position rotation
// applied on the way, for bf16 pools and for 8-bit (e4m3) pools, and the
// gather that reads 8-bit rows back as bf16 values.
//
// Rotation: pair i of a head turns by the angle p * inv_freq[i] (p the token's
// position).  The angle is needed modulo one turn only, so inv_freq[i] / 2 pi
// is held as a 64-bit binary fraction of a turn and multiplied by the position
// in integers: the product wraps modulo one turn by itself and keeps its low
// bits at any position (fp32 angles lose all of them near 2^24).  The sine and
// cosine of a token's pairs are computed once per CTA and shared by its heads.
//
// 8-bit blocks: kBlock consecutive tokens of one head share one fp32 scale, a
// power of two, so rows that were already there are requantised exactly (but
// for codes that become subnormal) when a larger row makes the scale grow.
// One warp takes one (block, head): it holds the block's new rows in
// registers, so the amax and the store read them once.
//
// All of it is bound by HBM at prompt sizes and by the latency of its
// dependent loads (request, position, page, row) at decode sizes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace pa {
namespace rope {

constexpr int kPage = PA_PAGE_TOKENS;
constexpr int kBlock = PA_SCALE_TOKENS;
constexpr int kBlocks = kPage / kBlock;   // scale blocks per page
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 8;               // token rows per CTA of the row-wise kernels

struct Tokens {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  long long q_stride, k_stride, v_stride, q_out_stride;   // elements per token
  const int32_t* cu;          // [B + 1] or null: one token per request
  const int32_t* positions;   // [B] position of each request's first new token
  const float* inv_freq;      // [half]
  const int32_t* page_table;
  int32_t* status;
  long long pool_pages;
  int n_tokens, B, Hq, Hkv, half, interleaved, max_pages;
};

// Request of token row `row` (all lanes of a warp): the first whose end lies
// behind the row.  B or more if there is none.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int row, int lane) {
  if (cu == nullptr) return row;
  int n = 0;
  for (int b = lane; b < B; b += 32) n += __ldg(cu + b + 1) <= row ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, n);
}

// Position of row `row` and the rows of its request [first, end); false if no
// request holds the row.
__device__ __forceinline__ bool locate(const int32_t* cu, const int32_t* positions, int B,
                                       int n_tokens, int row, int lane, int* request,
                                       long long* pos, int* first, int* end) {
  const int b = request_of(cu, B, row, lane);
  if (b >= B) return false;
  *request = b;
  *first = cu ? __ldg(cu + b) : row;
  *end = cu ? min(__ldg(cu + b + 1), n_tokens) : row + 1;
  if (row < *first) return false;
  *pos = (long long)__ldg(positions + b) + (row - *first);
  return true;
}

// Physical page of a token, -1 if its position or page is outside the table
// or the pool.
__device__ __forceinline__ long long page_of(const int32_t* page_table, int max_pages,
                                             long long pool_pages, int b, long long pos) {
  if (pos < 0 || pos / kPage >= max_pages) return -1;
  const long long page = __ldg(page_table + (size_t)b * max_pages + pos / kPage);
  return page < pool_pages ? page : -1;
}

// (cos, sin) of position p at inverse frequency f.
__device__ __forceinline__ float2 turn(long long pos, float f) {
  const double turns = (double)f * 0.15915494309189535;   // 1 / (2 pi)
  const double part = turns - floor(turns);
  const unsigned long long step = (unsigned long long)(part * 18446744073709551616.0);
  const unsigned long long at = step * (unsigned long long)pos;
  float2 cs;
  sincospif((float)(int)(at >> 32) * 4.656612873077393e-10f, &cs.y, &cs.x);   // 2^-31
  return cs;
}

// A lane holds four pairs of one head row as two 4-element vectors a and b at
// element offsets oa and ob of the head: pairs 4l .. 4l+3, which lie half a
// rotation apart (a holds the first, b the second of each pair) or next to
// each other (interleaved; a holds pairs 0 and 1, b pairs 2 and 3).  Lanes
// behind the rotated part hold the elements that pass.
struct Lane {
  int oa, ob, pair;
  bool turns;
};
__device__ __forceinline__ Lane lane_of(int l, int half, int interleaved) {
  Lane x;
  x.pair = 4 * l;
  x.turns = x.pair < half;
  const bool apart = x.turns && !interleaved;
  x.oa = apart ? x.pair : 2 * x.pair;
  x.ob = apart ? x.pair + half : 2 * x.pair + 4;
  return x;
}

// The lane's eight values, rotated in fp32: y[0..3] for a, y[4..7] for b.
__device__ __forceinline__ void rotate(uint2 a, uint2 b, const Lane& ln, int interleaved,
                                       const float2* cs, float (&y)[8]) {
  y[0] = ptx::bf16_lo_to_f32(a.x);
  y[1] = ptx::bf16_hi_to_f32(a.x);
  y[2] = ptx::bf16_lo_to_f32(a.y);
  y[3] = ptx::bf16_hi_to_f32(a.y);
  y[4] = ptx::bf16_lo_to_f32(b.x);
  y[5] = ptx::bf16_hi_to_f32(b.x);
  y[6] = ptx::bf16_lo_to_f32(b.y);
  y[7] = ptx::bf16_hi_to_f32(b.y);
  if (!ln.turns) return;
  const float4 c01 = *reinterpret_cast<const float4*>(cs + ln.pair);
  const float4 c23 = *reinterpret_cast<const float4*>(cs + ln.pair + 2);
  const float c[4] = {c01.x, c01.z, c23.x, c23.z};
  const float s[4] = {c01.y, c01.w, c23.y, c23.w};
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = y[2 * i], w = y[2 * i + 1];
      y[2 * i] = u * c[i] - w * s[i];
      y[2 * i + 1] = w * c[i] + u * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = y[i], w = y[i + 4];
      y[i] = u * c[i] - w * s[i];
      y[i + 4] = w * c[i] + u * s[i];
    }
  }
}

__device__ __forceinline__ uint2 pack4(const float* y) {
  return make_uint2(ptx::pack_bf16x2(__float2bfloat16_rn(y[0]), __float2bfloat16_rn(y[1])),
                    ptx::pack_bf16x2(__float2bfloat16_rn(y[2]), __float2bfloat16_rn(y[3])));
}

// Rotates the q heads of token rows [row0, row0 + rows) into q_out and, with
// kKv, stores their k (rotated) and v heads in the bf16 pool.
template <int D, bool kKv>
__device__ __forceinline__ void rotate_rows(const Tokens& t, __nv_bfloat16* pool, int row0,
                                            int rows) {
  constexpr int kLanes = D / 8;              // lanes per head row
  constexpr int kHeads = 32 / kLanes;        // head rows a warp takes at once
  constexpr int kUnroll = 4;
  __shared__ __align__(16) float2 cs[kMaxRows][D / 2];
  __shared__ long long s_pos[kMaxRows];
  __shared__ long long s_dst[kMaxRows];      // pool element of the row; -1: not stored
  __shared__ int s_live[kMaxRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  rows = min(rows, t.n_tokens - row0);
  for (int r = warp; r < rows; r += kWarps) {
    int b = 0, first, end;
    long long pos = 0, dst = -1;
    const bool live = locate(t.cu, t.positions, t.B, t.n_tokens, row0 + r, lane, &b, &pos, &first,
                             &end);
    if (kKv && live) {
      const long long page = page_of(t.page_table, t.max_pages, t.pool_pages, b, pos);
      if (page >= 0) dst = (page * kPage + pos % kPage) * (2ll * t.Hkv * D);
      else if (lane == 0 && t.status) atomicOr(t.status, PA_STATUS_BAD_ROW);
    }
    if (lane == 0) {
      s_pos[r] = pos;
      s_dst[r] = dst;
      s_live[r] = live;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * t.half; i += kThreads) {
    const int r = i / t.half, j = i - r * t.half;
    if (s_live[r]) cs[r][j] = turn(s_pos[r], __ldg(t.inv_freq + j));
  }
  __syncthreads();
  const Lane ln = lane_of(lane % kLanes, t.half, t.interleaved);
  const int heads = t.Hq + (kKv ? 2 * t.Hkv : 0);
  const int total = rows * heads;
  for (int u0 = warp * kHeads + lane / kLanes; u0 < total; u0 += kUnroll * kWarps * kHeads) {
    uint2 a[kUnroll], b[kUnroll];
    __nv_bfloat16* dst[kUnroll];
    int row[kUnroll];
    bool turns[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int u = u0 + i * kWarps * kHeads;
      const int r = u < total ? u / heads : 0;
      const int h = u - r * heads;
      const __nv_bfloat16* src;
      dst[i] = nullptr;
      row[i] = r;
      turns[i] = true;
      if (u >= total || !s_live[r]) continue;
      if (h < t.Hq) {
        src = t.q + (row0 + r) * t.q_stride + h * D;
        dst[i] = t.q_out + (row0 + r) * t.q_out_stride + h * D;
      } else {
        const int g = h - t.Hq;
        if (s_dst[r] < 0) continue;
        turns[i] = g < t.Hkv;
        src = turns[i] ? t.k + (row0 + r) * t.k_stride + g * D
                       : t.v + (row0 + r) * t.v_stride + (g - t.Hkv) * D;
        dst[i] = pool + s_dst[r] + g * D;
      }
      a[i] = *reinterpret_cast<const uint2*>(src + ln.oa);
      b[i] = *reinterpret_cast<const uint2*>(src + ln.ob);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (dst[i] == nullptr) continue;
      if (turns[i] && ln.turns) {
        float y[8];
        rotate(a[i], b[i], ln, t.interleaved, cs[row[i]], y);
        a[i] = pack4(y);
        b[i] = pack4(y + 4);
      }
      *reinterpret_cast<uint2*>(dst[i] + ln.oa) = a[i];
      *reinterpret_cast<uint2*>(dst[i] + ln.ob) = b[i];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_rope_kernel(const Tokens t, __nv_bfloat16* pool, int rows) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  rotate_rows<D, true>(t, pool, blockIdx.x * rows, rows);
}

// Smallest power of two s >= 2^-60 with amax <= 448 s (448 = 1.75 * 2^8 is the
// largest e4m3 value), from the bits of a finite amax >= 0.
__device__ __forceinline__ float block_scale(unsigned amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return ptx::pow2i(max(e, -60));
}

// One (block, head) by one warp: rows [row, row + n_new) of the step go to the
// block's rows [first, first + n_new).
template <int D>
__device__ __forceinline__ void store_block(const Tokens& t, uint8_t* pool, float* scales,
                                            const float2 (*cs)[D / 2], int row, int n_new,
                                            int first, long long page, int blk, int h, int lane) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;         // token rows a warp takes at once
  constexpr int kSteps = kBlock / kRows;
  const int sub = lane / kLanes;
  const Lane ln = lane_of(lane % kLanes, t.half, t.interleaved);
  const bool is_k = h < t.Hkv;
  const long long stride = is_k ? t.k_stride : t.v_stride;
  const __nv_bfloat16* src =
      (is_k ? t.k + h * D : t.v + (h - t.Hkv) * D) + (long long)row * stride;
  const size_t row_bytes = (size_t)2 * t.Hkv * D;
  uint8_t* base = pool + ((size_t)page * kPage + blk * kBlock) * row_bytes + (size_t)h * D;
  float* scale = scales + ((size_t)page * 2 * t.Hkv + h) * kBlocks + blk;
  const float old = first > 0 ? *scale : 0.f;
  uint2 a[kSteps], b[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRows + sub;
    if (r < n_new) {
      a[i] = *reinterpret_cast<const uint2*>(src + r * stride + ln.oa);
      b[i] = *reinterpret_cast<const uint2*>(src + r * stride + ln.ob);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRows + sub;
    if (r < n_new) {
      float y[8];
      Lane l2 = ln;
      l2.turns = ln.turns && is_k;
      rotate(a[i], b[i], l2, t.interleaved, cs[r], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(y[j]);
        amax = fmaxf(amax, m <= FLT_MAX ? m : 0.f);   // infinities and NaN set no scale
      }
    }
  }
  const float need = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
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
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRows + sub;
    if (r < n_new) {
      float y[8];
      Lane l2 = ln;
      l2.turns = ln.turns && is_k;
      rotate(a[i], b[i], l2, t.interleaved, cs[r], y);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = fabsf(y[j]) <= FLT_MAX ? y[j] * inv : __int_as_float(0x7fc00000);
      uint8_t* dst = base + (size_t)(first + r) * row_bytes;
      *reinterpret_cast<uint32_t*>(dst + ln.oa) = fp8::pack4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint32_t*>(dst + ln.ob) = fp8::pack4(y[4], y[5], y[6], y[7]);
    }
  }
  if (lane == 0 && (first == 0 || s != old)) *scale = s;
}

// CTAs [0, kv_ctas) take `chunk` token rows each and store the blocks whose
// first new row lies among them (a request's first new row, or a row on a
// block border); the other CTAs rotate q rows.
template <int D>
__global__ void __launch_bounds__(kThreads)
    append_rope_q8_kernel(const Tokens t, uint8_t* pool, float* scales, int kv_ctas, int chunk,
                          int q_rows) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  if ((int)blockIdx.x >= kv_ctas) {
    rotate_rows<D, false>(t, nullptr, (blockIdx.x - kv_ctas) * q_rows, q_rows);
    return;
  }
  __shared__ __align__(16) float2 cs[kBlock][D / 2];
  __shared__ long long s_pos[kBlock], s_page[kBlock];
  __shared__ int s_new[kBlock];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * chunk;
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
    for (int i = threadIdx.x; i < n * t.half; i += kThreads) {
      const int k = i / t.half, j = i - k * t.half;
      cs[k][j] = turn(pos + k, __ldg(t.inv_freq + j));
    }
    __syncthreads();
    const int in_page = (int)(pos % kPage);
    for (int h = warp; h < 2 * t.Hkv; h += kWarps)
      store_block<D>(t, pool, scales, cs, row0 + r, n, in_page % kBlock, s_page[r],
                     in_page / kBlock, h, lane);
    __syncthreads();
  }
}

// Rows of an 8-bit pool as bf16 values: a thread turns 16 codes of one head.
__global__ void __launch_bounds__(kThreads)
    gather_q8_kernel(const uint8_t* pool, const float* scales, long long pool_pages,
                     const int32_t* page_table, int max_pages, const int32_t* cu,
                     const int32_t* positions, int n_tokens, int B, int heads, int d, int rows,
                     __nv_bfloat16* out, int32_t* status) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  __shared__ long long s_pos[kMaxRows], s_page[kMaxRows];
  __shared__ int s_live[kMaxRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * rows;
  rows = min(rows, n_tokens - row0);
  for (int r = warp; r < rows; r += kWarps) {
    int b = 0, first, end;
    long long pos = 0, page = -1;
    const bool live = locate(cu, positions, B, n_tokens, row0 + r, lane, &b, &pos, &first, &end);
    if (live) {
      page = page_of(page_table, max_pages, pool_pages, b, pos);
      if (page < 0 && lane == 0 && status) atomicOr(status, PA_STATUS_BAD_ROW);
    }
    if (lane == 0) {
      s_pos[r] = pos;
      s_page[r] = page;
      s_live[r] = live;
    }
  }
  __syncthreads();
  const int per_row = heads * d / 16;
  for (int i = threadIdx.x; i < rows * per_row; i += kThreads) {
    const int r = i / per_row, c = i - r * per_row;
    if (!s_live[r]) continue;
    uint4 codes = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);   // NaN
    float s = 1.f;
    if (s_page[r] >= 0) {
      const int at = (int)(s_pos[r] % kPage);
      codes = __ldg(reinterpret_cast<const uint4*>(
                        pool + ((size_t)s_page[r] * kPage + at) * heads * d) + c);
      s = __ldg(scales + ((size_t)s_page[r] * heads + c * 16 / d) * kBlocks + at / kBlock);
    }
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint4 o[2];
    uint32_t* ow = reinterpret_cast<uint32_t*>(o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y[4];
      fp8::unpack4(w[j], y);
      ow[2 * j] = ptx::pack_bf16x2(__float2bfloat16_rn(y[0] * s), __float2bfloat16_rn(y[1] * s));
      ow[2 * j + 1] =
          ptx::pack_bf16x2(__float2bfloat16_rn(y[2] * s), __float2bfloat16_rn(y[3] * s));
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (size_t)(row0 + r) * heads * d) + 2 * c;
    dst[0] = o[0];
    dst[1] = o[1];
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Token rows per CTA of the row-wise kernels: one while the launch is small
// (every CTA's dependent loads then run at the same time), more once there
// are several CTAs per SM.
int rows_per_cta(int n_tokens) { return std::max(1, std::min(kMaxRows, n_tokens / 1024)); }

int check_tokens(const Tokens& t, int head_dim, int rot_dim, unsigned flags, const void* pool) {
  PA_REQUIRE(t.n_tokens >= 0 && t.B >= 0, "n_tokens and B must be >= 0 (got %d, %d)", t.n_tokens,
             t.B);
  if (t.n_tokens == 0 || t.B == 0) return PA_OK;
  PA_REQUIRE(t.Hkv >= 1 && t.Hkv <= 4096, "n_kv_heads (%d) must be in 1..4096", t.Hkv);
  PA_REQUIRE((t.q == nullptr) == (t.q_out == nullptr), "q and q_out go together");
  PA_REQUIRE(t.q == nullptr || (t.Hq >= 1 && t.Hq <= 65536), "n_q_heads (%d) must be in 1..65536",
             t.Hq);
  PA_REQUIRE(t.k && t.v && t.positions && t.page_table && pool, "null pointer argument");
  PA_REQUIRE(t.cu || t.n_tokens == t.B, "without cu_tokens there is one token per request");
  PA_REQUIRE(rot_dim >= 0 && rot_dim <= head_dim && rot_dim % 8 == 0,
             "rot_dim (%d) must be a multiple of 8 in [0, %d]", rot_dim, head_dim);
  PA_REQUIRE(rot_dim == 0 || t.inv_freq, "inv_freq is required");
  PA_REQUIRE((flags & ~PA_ROPE_INTERLEAVED) == 0, "unknown flags %#x", flags);
  PA_REQUIRE(aligned16(t.q) && aligned16(t.q_out) && aligned16(t.k) && aligned16(t.v) &&
                 aligned16(pool),
             "q, q_out, k, v and pool must be 16-byte aligned");
  const long long kv = (long long)t.Hkv * head_dim, qd = (long long)t.Hq * head_dim;
  PA_REQUIRE(t.k_stride % 8 == 0 && t.v_stride % 8 == 0 && t.q_stride % 8 == 0 &&
                 t.q_out_stride % 8 == 0,
             "token strides must be multiples of 8 elements");
  PA_REQUIRE((t.n_tokens == 1 || (t.k_stride >= kv && t.v_stride >= kv)) &&
                 (t.q == nullptr || t.n_tokens == 1 ||
                  (t.q_stride >= qd && t.q_out_stride >= qd)),
             "token strides are smaller than a token's heads");
  PA_REQUIRE(t.pool_pages >= 1 && t.max_pages >= 1, "pool_pages and max_pages must be >= 1");
  return PA_OK;
}

Tokens tokens_of(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                 int64_t v_stride, void* q_out, int64_t q_out_stride, const int32_t* cu_tokens,
                 const int32_t* positions, int n_tokens, int B, int n_q_heads, int n_kv_heads,
                 const float* inv_freq, int rot_dim, unsigned flags, int64_t pool_pages,
                 const int32_t* page_table, int max_pages, int32_t* status) {
  Tokens t{};
  t.q = static_cast<const __nv_bfloat16*>(q);
  t.k = static_cast<const __nv_bfloat16*>(k);
  t.v = static_cast<const __nv_bfloat16*>(v);
  t.q_out = static_cast<__nv_bfloat16*>(q_out);
  t.q_stride = q_stride;
  t.k_stride = k_stride;
  t.v_stride = v_stride;
  t.q_out_stride = q_out_stride;
  t.cu = cu_tokens;
  t.positions = positions;
  t.inv_freq = inv_freq;
  t.page_table = page_table;
  t.status = status;
  t.pool_pages = pool_pages;
  t.n_tokens = n_tokens;
  t.B = B;
  t.Hq = q ? n_q_heads : 0;
  t.Hkv = n_kv_heads;
  t.half = rot_dim / 2;
  t.interleaved = (flags & PA_ROPE_INTERLEAVED) ? 1 : 0;
  t.max_pages = max_pages;
  return t;
}

template <int D>
cudaError_t launch_append(const Tokens& t, void* pool, cudaStream_t stream) {
  const int rows = rows_per_cta(t.n_tokens);
  return launch_dependent(append_rope_kernel<D>, dim3((t.n_tokens + rows - 1) / rows),
                          dim3(kThreads), 0, stream, t, static_cast<__nv_bfloat16*>(pool), rows);
}

template <int D>
cudaError_t launch_append_q8(const Tokens& t, void* pool, float* scales, cudaStream_t stream) {
  const int rows = rows_per_cta(t.n_tokens);
  // A CTA of one row is either one block's or leaves at once, which is the
  // shortest path while all rows' CTAs fit the GPU together; behind that, 16
  // rows (one block's worth) a CTA.
  const int chunk = t.cu == nullptr || t.n_tokens <= 1024 ? 1 : kBlock;
  const int kv = (t.n_tokens + chunk - 1) / chunk;
  const int q = t.q ? (t.n_tokens + rows - 1) / rows : 0;
  return launch_dependent(append_rope_q8_kernel<D>, dim3(kv + q), dim3(kThreads), 0, stream, t,
                          static_cast<uint8_t*>(pool), scales, kv, chunk, rows);
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
  PA_CHECK_CUDA(head_dim == 64    ? launch_append<64>(t, pool, stream)
                : head_dim == 128 ? launch_append<128>(t, pool, stream)
                                  : launch_append<256>(t, pool, stream));
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
  PA_CHECK_CUDA(head_dim == 128 ? launch_append_q8<128>(t, pool, scales, stream)
                                : launch_append_q8<256>(t, pool, scales, stream));
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
  PA_REQUIRE(n_kv_heads >= 1 && n_kv_heads <= 4096, "n_kv_heads (%d) must be in 1..4096",
             n_kv_heads);
  PA_REQUIRE(pool && scales && page_table && positions && out, "null pointer argument");
  PA_REQUIRE(cu_tokens || n_tokens == B, "without cu_tokens there is one row per request");
  PA_REQUIRE(aligned16(pool) && aligned16(scales) && aligned16(out),
             "pool, scales and out must be 16-byte aligned");
  PA_REQUIRE(pool_pages >= 1 && max_pages >= 1, "pool_pages and max_pages must be >= 1");
  const int rows = rows_per_cta(n_tokens);
  PA_CHECK_CUDA(pa::launch_dependent(
      gather_q8_kernel, dim3((n_tokens + rows - 1) / rows), dim3(kThreads), 0, stream,
      static_cast<const uint8_t*>(pool), scales, (long long)pool_pages, page_table, max_pages,
      cu_tokens, positions, n_tokens, B, 2 * n_kv_heads, head_dim, rows,
      static_cast<__nv_bfloat16*>(out), status));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}
