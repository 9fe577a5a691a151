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

namespace pa {
namespace rope {

constexpr int kPage = PA_PAGE_TOKENS;
constexpr int kBlock = PA_SCALE_TOKENS;
constexpr int kBlocks = kPage / kBlock;   // scale blocks per page
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 1 << 30;       // rows of a call: CTA and row numbers stay in 32 bits
constexpr int kRowCtas = 304;             // CTAs up to which rows are shared by several warps

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

// Turns per position, modulo one, in units of 2^-64: f / (2 pi) from f's 24
// significant bits and 1 / (2 pi) to 66 bits.
__device__ __forceinline__ unsigned long long turn_step(float f) {
  constexpr unsigned long long kInvTwoPi = 0xa2f9836e4e44152aull;  // 2^66 / (2 pi)
  const unsigned bits = __float_as_uint(f);
  const int e = (bits >> 23) & 255;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const unsigned long long lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  // f = m 2^(max(e, 1) - 150): the product is 2^(shift - 64) times the result
  const int shift = 152 - max(e, 1);
  unsigned long long x;
  if (shift >= 64) x = shift < 128 ? hi >> (shift - 64) : 0ull;
  else if (shift > 0) x = (hi << (64 - shift)) | (lo >> shift);
  else x = shift > -64 ? lo << -shift : 0ull;
  return (bits >> 31) ? 0ull - x : x;
}

// 0, or NaN for a frequency that is not finite, whose pairs become NaN.
__device__ __forceinline__ float not_finite(float f) { return f - f; }

// Sine and cosine at position p: the turn's nearest quarter, and the Taylor
// polynomials of the rest (|x| <= pi / 4: the first terms left out are below
// 2e-9 and 3e-10).  Half the instructions of sincospif, which reduces a float.
__device__ __forceinline__ void turn(long long p, unsigned long long step, float nan, float* s,
                                     float* c) {
  const uint32_t at = (uint32_t)((step * (unsigned long long)p) >> 32);
  const uint32_t quarter = (at + 0x20000000u) >> 30;
  const float x = (float)(int)(at - (quarter << 30)) * 1.4629180792671596e-09f;   // 2 pi 2^-32
  const float z = x * x;
  float a = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  a = fmaf(a, z, 1.0f / 120.0f);
  a = fmaf(a, z, -1.0f / 6.0f);
  const float sx = fmaf(a * z, x, x);
  float b = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  b = fmaf(b, z, -1.0f / 720.0f);
  b = fmaf(b, z, 1.0f / 24.0f);
  b = fmaf(b, z, -0.5f);
  const float cx = fmaf(b, z, 1.0f);
  const bool odd = quarter & 1;
  const float ss = odd ? cx : sx, cc = odd ? sx : cx;
  *s = (quarter & 2 ? -ss : ss) + nan;
  *c = ((quarter + 1) & 2 ? -cc : cc) + nan;
}

template <int V>
using Vec = typename std::conditional<V == 8, uint4, uint2>::type;

// A lane holds V pairs of one head row as two V-element vectors a and b at
// element offsets oa and ob of the head: pairs Vl .. Vl + V-1, which lie half a
// rotation apart (a holds the first, b the second of each pair) or next to
// each other (interleaved; a holds the first V/2 pairs, b the others).  Lanes
// behind the rotated part hold the elements that pass.
struct Lane {
  int oa, ob, pair;
  bool turns;
};
template <int V>
__device__ __forceinline__ Lane lane_of(int l, int half, int interleaved) {
  Lane x;
  x.pair = V * l;
  x.turns = x.pair < half;
  const bool apart = x.turns && !interleaved;
  x.oa = apart ? x.pair : 2 * x.pair;
  x.ob = apart ? x.pair + half : 2 * x.pair + V;
  return x;
}

// The lane's 2 V values in fp32; the first V are a's.
template <int V>
__device__ __forceinline__ void unpack(const Vec<V>& a, const Vec<V>& b, float (&y)[2 * V]) {
  const uint32_t* wa = reinterpret_cast<const uint32_t*>(&a);
  const uint32_t* wb = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    y[2 * i] = ptx::bf16_lo_to_f32(wa[i]);
    y[2 * i + 1] = ptx::bf16_hi_to_f32(wa[i]);
    y[V + 2 * i] = ptx::bf16_lo_to_f32(wb[i]);
    y[V + 2 * i + 1] = ptx::bf16_hi_to_f32(wb[i]);
  }
}

// They turned by their pairs' c and s.
template <int V>
__device__ __forceinline__ void rotate(int interleaved, const float* c, const float* s,
                                       float (&y)[2 * V]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float u = y[2 * i], w = y[2 * i + 1];
      y[2 * i] = u * c[i] - w * s[i];
      y[2 * i + 1] = w * c[i] + u * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float u = y[i], w = y[i + V];
      y[i] = u * c[i] - w * s[i];
      y[i + V] = w * c[i] + u * s[i];
    }
  }
}

template <int V>
__device__ __forceinline__ Vec<V> pack(const float* y) {
  Vec<V> r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    w[i] = ptx::pack_bf16x2(__float2bfloat16_rn(y[2 * i]), __float2bfloat16_rn(y[2 * i + 1]));
  return r;
}

// Rotates the q heads of the token rows of CTA cta into q_out and, with kKv,
// stores their k (rotated) and v heads in the bf16 pool: `share` (1, 2, 4 or 8)
// warps to a row.  Warps do not wait for each other; a warp issues its row's
// first loads before it looks the row up.  (Fewer CTAs whose warps take several
// rows each, the next one's loads ahead, measured slower: 44.6 against 40.4 us
// for 11 prompts of up to 2,500 tokens.)
template <int D, int V, bool kKv>
__device__ __forceinline__ void rotate_rows(const Tokens& t, __nv_bfloat16* pool, int cta,
                                            int share) {
  constexpr int kLanes = D / (2 * V);        // lanes per head row
  constexpr int kHeads = 32 / kLanes;        // head rows a warp takes at once
  constexpr int kUnroll = 4;
  __shared__ __align__(16) float table[kWarps][2][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = kWarps / share;
  const Lane ln = lane_of<V>(lane % kLanes, t.half, t.interleaved);
  const int heads = t.Hq + (kKv ? 2 * t.Hkv : 0);
  const int step = share * kHeads;
  const int first_h = (warp % share) * kHeads + lane / kLanes;
  Vec<V> va[kUnroll], vb[kUnroll];
  const int row = cta * per_cta + warp / share;
  if (row >= t.n_tokens) return;
  auto load = [&](int h0) {
    const __nv_bfloat16* q = t.q + row * t.q_stride;
    const __nv_bfloat16* k = t.k + row * t.k_stride;
    const __nv_bfloat16* v = t.v + row * t.v_stride;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * step, g = h - t.Hq;
      if (h >= heads) continue;
      const __nv_bfloat16* src = !kKv || g < 0 ? q + h * D
                                 : g < t.Hkv   ? k + g * D
                                               : v + (g - t.Hkv) * D;
      va[i] = *reinterpret_cast<const Vec<V>*>(src + ln.oa);
      vb[i] = *reinterpret_cast<const Vec<V>*>(src + ln.ob);
    }
  };
  load(first_h);
  int b = 0, first, end;
  long long pos = 0;
  if (!locate(t.cu, t.positions, t.B, t.n_tokens, row, lane, &b, &pos, &first, &end)) return;
  for (int i = lane; i < t.half; i += 32) {
    const float f = __ldg(t.inv_freq + i);
    turn(pos, turn_step(f), not_finite(f), &table[warp][1][i], &table[warp][0][i]);
  }
  __nv_bfloat16* q_out = t.q_out + row * t.q_out_stride;
  __nv_bfloat16* kv_out = nullptr;
  if (kKv) {
    const long long page = page_of(t.page_table, t.max_pages, t.pool_pages, b, pos);
    if (page >= 0) kv_out = pool + (page * kPage + pos % kPage) * (2ll * t.Hkv * D);
    else if (lane == 0 && t.status) atomicOr(t.status, PA_STATUS_BAD_ROW);
  }
  __syncwarp();
  float c[V], s[V];
  if (ln.turns) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      *reinterpret_cast<float4*>(c + i) =
          *reinterpret_cast<const float4*>(&table[warp][0][ln.pair + i]);
      *reinterpret_cast<float4*>(s + i) =
          *reinterpret_cast<const float4*>(&table[warp][1][ln.pair + i]);
    }
  }
  for (int h0 = first_h;;) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * step, g = h - t.Hq;
      if (h >= heads || (kKv && g >= 0 && kv_out == nullptr)) continue;
      if (ln.turns && (!kKv || g < t.Hkv)) {   // v and what passes keep their bits
        float y[2 * V];
        unpack<V>(va[i], vb[i], y);
        rotate<V>(t.interleaved, c, s, y);
        va[i] = pack<V>(y);
        vb[i] = pack<V>(y + V);
      }
      __nv_bfloat16* dst = !kKv || g < 0 ? q_out + h * D : kv_out + g * D;
      *reinterpret_cast<Vec<V>*>(dst + ln.oa) = va[i];
      *reinterpret_cast<Vec<V>*>(dst + ln.ob) = vb[i];
    }
    h0 += kUnroll * step;
    if (h0 >= heads) break;
    load(h0);
  }
}

template <int D, int V>
__global__ void __launch_bounds__(kThreads, 3)
    append_rope_kernel(const Tokens t, __nv_bfloat16* pool, int share) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  rotate_rows<D, V, true>(t, pool, blockIdx.x, share);
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

// 32 bytes (aligned) in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Warps per row and CTAs of the row-wise kernels: a CTA per row while there are
// few (its warps share the row's heads), up to a row per warp.
void row_grid(int n_tokens, int* share, int* ctas) {
  *share = kWarps;
  while (*share > 1 && (long long)n_tokens * *share > (long long)kRowCtas * kWarps) *share /= 2;
  const int per_cta = kWarps / *share;
  *ctas = (n_tokens + per_cta - 1) / per_cta;
}

int check_tokens(const Tokens& t, int head_dim, int rot_dim, unsigned flags, const void* pool) {
  PA_REQUIRE(t.n_tokens >= 0 && t.B >= 0, "n_tokens and B must be >= 0 (got %d, %d)", t.n_tokens,
             t.B);
  if (t.n_tokens == 0 || t.B == 0) return PA_OK;
  PA_REQUIRE(t.n_tokens <= kMaxTokens, "n_tokens (%d) above %d", t.n_tokens, kMaxTokens);
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

template <int D, int V>
cudaError_t launch_append(const Tokens& t, void* pool, cudaStream_t stream) {
  int share, ctas;
  row_grid(t.n_tokens, &share, &ctas);
  return launch_dependent(append_rope_kernel<D, V>, dim3(ctas), dim3(kThreads), 0, stream, t,
                          static_cast<__nv_bfloat16*>(pool), share);
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

// Pairs per lane: 8 (16-byte accesses) unless the rotated half is no multiple.
bool wide(const Tokens& t) { return t.half % 8 == 0; }

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
