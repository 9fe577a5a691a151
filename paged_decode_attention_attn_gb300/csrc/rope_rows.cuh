// What the appends to the three kinds of pools share: the rows of a step's new
// tokens, their places in the pool, the position rotation with the norm of a head
// before it, and the checks of the calls' arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <type_traits>

#include "common.h"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace pa {
namespace rope {

constexpr int kPage = PA_PAGE_TOKENS;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 1 << 30;       // rows of a call: CTA and row numbers stay in 32 bits
constexpr float kMinEps = 1.f / (1ll << 60);   // (a square's last bit in fp32 is far below)
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

// kPairs: two values by one conversion.  (The rows without norms stream at the copy's rate and
// measured slower so: 11 prompts of up to 2,500 tokens 42.0 us, 40.6 without; with norms 13 of
// up to 2,100 take 56.0 us so, 60.1 without.)
template <int V, bool kPairs = false>
__device__ __forceinline__ Vec<V> pack(const float* y) {
  Vec<V> r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    w[i] = kPairs ? ptx::round_bf16x2(y[2 * i], y[2 * i + 1])
                  : ptx::pack_bf16x2(__float2bfloat16_rn(y[2 * i]), __float2bfloat16_rn(y[2 * i + 1]));
  return r;
}

// 32 bytes (aligned) in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The norm of q and k heads ahead of the rotation: y = x w / sqrt(mean x^2 + eps).
struct Norm {
  const float* q_weight;   // [D]
  const float* k_weight;
  float eps;
};

// The weights of both norms into shared memory: every thread of the CTA, a barrier
// before they are read.
template <int D, bool kKey>
__device__ __forceinline__ void load_weights(const Norm& norm, bool q, float (*w)[D]) {
  for (int i = threadIdx.x; i < D; i += kThreads) {
    if (q) w[0][i] = __ldg(norm.q_weight + i);
    if (kKey) w[1][i] = __ldg(norm.k_weight + i);
  }
}

// Rotates the q heads of the token rows of CTA cta into q_out and, with kKv,
// stores their k (rotated) and v heads in the bf16 pool: `share` (1, 2, 4 or 8)
// warps to a row.  Warps do not wait for each other; a warp issues its row's first
// loads before it looks the row up.  (Fewer CTAs whose warps take several rows each,
// the next one's loads ahead, measured slower: 44.6 against 40.4 us for 11 prompts of
// up to 2,500 tokens.)
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

// The same with the norm of q and k heads ahead of the rotation.  A row's weights and
// turns meet once, y[j] = x[j] r p[j] + x'[j] r q[j] with x' the pair's other, for all its
// q heads and again for its k heads.  Slots of a row go through the warp one after the
// other, q heads, k heads, v heads, the load of a slot four ahead.  (With the turn after
// the norm of each head, weights from shared memory, and a batch's loads after the one
// before it: 252 instructions for 16 values of a lane, 87.7 us for 13 prompts of up to
// 2,100 tokens; 56.0 so.)
template <int D, int V, bool kKv>
__device__ __forceinline__ void norm_rows(const Tokens& t, const Norm& norm, __nv_bfloat16* pool,
                                          int cta, int share) {
  constexpr int kLanes = D / (2 * V);        // lanes per head row
  constexpr int kHeads = 32 / kLanes;        // head rows a warp takes at once
  constexpr int kAhead = 4;
  __shared__ __align__(16) float table[kWarps][2][D / 2];
  __shared__ __align__(16) float weights[2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = kWarps / share;
  const Lane ln = lane_of<V>(lane % kLanes, t.half, t.interleaved);
  const int step = share * kHeads, h0 = (warp % share) * kHeads + lane / kLanes;
  const int q_slots = (t.Hq + step - 1) / step, k_slots = kKv ? (t.Hkv + step - 1) / step : 0;
  const int slots = q_slots + 2 * k_slots;
  const long long row = (long long)cta * per_cta + warp / share;
  Vec<V> va[kAhead], vb[kAhead];
  // (a lane without a head of its own takes the last one's values and stores nothing)
  auto load = [&](int slot, Vec<V>& a, Vec<V>& b) {
    const __nv_bfloat16* src = t.q + row * t.q_stride;
    int h = h0 + slot * step, last = t.Hq - 1;
    if (kKv && slot >= q_slots) {
      const bool value = slot >= q_slots + k_slots;
      h -= (value ? q_slots + k_slots : q_slots) * step;
      last = t.Hkv - 1;
      src = value ? t.v + row * t.v_stride : t.k + row * t.k_stride;
    }
    if (slot >= slots) return;
    src += min(h, last) * D + ln.oa;
    a = *reinterpret_cast<const Vec<V>*>(src);
    b = *reinterpret_cast<const Vec<V>*>(src + (ln.ob - ln.oa));
  };
  if (row < t.n_tokens) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, va[i], vb[i]);
  }
  load_weights<D, kKv>(norm, t.Hq > 0, weights);
  __syncthreads();
  if (row >= t.n_tokens) return;
  int b = 0, first, end;
  long long pos = 0;
  if (!locate(t.cu, t.positions, t.B, t.n_tokens, (int)row, lane, &b, &pos, &first, &end)) return;
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
  float2 p[V], q[V];
  auto meet = [&](const float* w) {          // q 0 where nothing turns
    float x[2 * V], c[V] = {}, s[V] = {};
    auto four = [](float* to, const float* from) {
      *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(from);
    };
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      four(x + j, w + ln.oa + j);
      four(x + V + j, w + ln.ob + j);
      if (ln.turns) {
        four(c + j, &table[warp][0][ln.pair + j]);
        four(s + j, &table[warp][1][ln.pair + j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * V; ++j) {
      // its pair, and whether it is the first of it, in the two layouts
      const float cj = t.interleaved ? c[j / 2] : c[j % V], sj = t.interleaved ? s[j / 2] : s[j % V];
      const float other = t.interleaved ? x[j ^ 1] : x[(j + V) % (2 * V)];
      const bool is_first = t.interleaved ? j % 2 == 0 : j < V;
      (j % 2 ? p[j / 2].y : p[j / 2].x) = ln.turns ? x[j] * cj : x[j];
      (j % 2 ? q[j / 2].y : q[j / 2].x) = ln.turns ? (is_first ? -other : other) * sj : 0.f;
    }
  };
  meet(weights[q_slots ? 0 : 1]);
  auto slot_of = [&](int slot, Vec<V>& a, Vec<V>& b2) {
    Vec<V> oa = a, ob = b2;
    const bool value = slot >= q_slots + k_slots, key = !value && slot >= q_slots;
    const int h = h0 + (slot - (key ? q_slots : value ? q_slots + k_slots : 0)) * step;
    if (key && slot == q_slots && q_slots) meet(weights[1]);
    if (!value) {
      float2 y[V];
      {
        float x[2 * V];
        unpack<V>(a, b2, x);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = make_float2(x[2 * j], x[2 * j + 1]);
      }
      load(slot + kAhead, a, b2);
      auto sum_of_squares = [&]() {
        float2 z = f32x2::mul(y[0], y[0]);
#pragma unroll
        for (int j = 1; j < V; ++j) z = f32x2::fma(y[j], y[j], z);
        float ss = z.x + z.y;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        return ss;
      };
      float ss = sum_of_squares(), eps = norm.eps;
      // Squares beyond the range of fp32 (bf16 values reach 2^128): x 2^-70 has a square and
      // a sum in range, beside which eps is nothing.
      if (__any_sync(0xffffffffu, !(ss <= FLT_MAX))) {
        const bool large = !(ss <= FLT_MAX);
        if (large) eps = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = f32x2::mul(y[j], f32x2::both(large ? ptx::pow2i(-70) : 1.f));
        ss = sum_of_squares();
      }
      const float2 r = f32x2::both(rsqrtf(fmaf(ss, 1.f / D, eps)));
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = f32x2::mul(y[j], r);
      float2 z[V];
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] = f32x2::mul(y[j], p[j]);
      if (ln.turns) {
        if (t.interleaved) {
#pragma unroll
          for (int j = 0; j < V; ++j) z[j] = f32x2::fma(make_float2(y[j].y, y[j].x), q[j], z[j]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) z[j] = f32x2::fma(y[(j + V / 2) % V], q[j], z[j]);
        }
      }
      float x[2 * V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[2 * j] = z[j].x;
        x[2 * j + 1] = z[j].y;
      }
      oa = pack<V, true>(x);
      ob = pack<V, true>(x + V);
    } else {
      load(slot + kAhead, a, b2);
    }
    if (h >= (key || value ? t.Hkv : t.Hq) || (kv_out == nullptr && (key || value))) return;
    __nv_bfloat16* dst = key ? kv_out + h * D : value ? kv_out + (t.Hkv + h) * D : q_out + h * D;
    dst += ln.oa;
    *reinterpret_cast<Vec<V>*>(dst) = oa;
    *reinterpret_cast<Vec<V>*>(dst + (ln.ob - ln.oa)) = ob;
  };
  for (int s0 = 0; s0 < slots; s0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i >= slots) break;            // (of the whole warp)
      slot_of(s0 + i, va[i], vb[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Warps per row and CTAs of the row-wise kernels: a CTA per row while there are
// few (its warps share the row's heads), up to a row per warp.
inline void row_grid(int n_tokens, int* share, int* ctas) {
  *share = kWarps;
  while (*share > 1 && (long long)n_tokens * *share > (long long)kRowCtas * kWarps) *share /= 2;
  const int per_cta = kWarps / *share;
  *ctas = (n_tokens + per_cta - 1) / per_cta;
}

inline int check_tokens(const Tokens& t, int head_dim, int rot_dim, unsigned flags, const void* pool) {
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

inline Tokens tokens_of(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
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

// Pairs per lane: 8 (16-byte accesses) unless the rotated half is no multiple.
inline bool wide(const Tokens& t) { return t.half % 8 == 0; }

// The norms' arguments (of a call that has them).
inline int check_norm(const Tokens& t, const Norm& norm) {
  PA_REQUIRE(norm.k_weight && (t.q == nullptr || norm.q_weight),
             "q_weight and k_weight are required");
  PA_REQUIRE(reinterpret_cast<uintptr_t>(norm.q_weight) % 4 == 0 &&
                 reinterpret_cast<uintptr_t>(norm.k_weight) % 4 == 0,
             "q_weight and k_weight must be 4-byte aligned");
  PA_REQUIRE(norm.eps >= kMinEps && norm.eps <= 1.f, "eps (%g) must be in [2^-60, 1]",
             (double)norm.eps);
  return PA_OK;
}

}  // namespace rope
}  // namespace pa
