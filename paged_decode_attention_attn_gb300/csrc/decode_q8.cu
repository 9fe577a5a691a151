// Paged GQA decode attention over an 8-bit pool, per tile, with its
// log-sum-exp: the definition written out in FP32, one CTA per (tile, kv head).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <vector>

#include "common.h"
#include "fp8.cuh"
#include "merge_row.cuh"
#include "ptx.cuh"

namespace pa {
namespace decode_q8 {

constexpr int kPage = PA_PAGE_TOKENS;
constexpr int kMaxG = 8;
constexpr int kWarps = 8;
constexpr int kMaxTiles = 1024;            // tiles per launch
constexpr size_t kStatusBytes = 256;

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* pool;
  const float* scales;
  const int32_t* page_table;
  float* out;
  float* lse;
  int32_t* status;
  long long pool_pages;
  int max_pages, T, Hq, Hkv, G, bt0;
  float scale;
  int2 tiles[kMaxTiles];
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const __grid_constant__ Params p) {
  constexpr int kDims = D / 32;
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  __shared__ float xo[kWarps][kMaxG][D];
  __shared__ float xm[kWarps][kMaxG], xl[kWarps][kMaxG];
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x / p.Hkv, g = blockIdx.x - i * p.Hkv;
  const int bt = p.bt0 + i, b = bt / p.T;
  const int2 tile = p.tiles[i];
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  float q[kMaxG][kDims], o[kMaxG][kDims], m[kMaxG], l[kMaxG];
#pragma unroll
  for (int h = 0; h < kMaxG; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      o[h][d] = 0.f;
      q[h][d] = h < p.G ? __bfloat162float(
                              p.q[((size_t)b * p.Hq + g * p.G + h) * D + lane * kDims + d])
                        : 0.f;
    }
  }
  for (int j = tile.x + warp; j < tile.y; j += kWarps) {
    const long long page = p.page_table[(size_t)b * p.max_pages + j / kPage];
    if (page < 0 || page >= p.pool_pages) {
      if (lane == 0) {
        atomicOr(p.status, PA_STATUS_BAD_PAGE);
        s_bad = 1;
      }
      continue;
    }
    const uint8_t* row = p.pool + ((size_t)page * kPage + j % kPage) * (2 * p.Hkv * D) + g * D +
                         lane * kDims;
    const float* sc = p.scales + ((size_t)page * 2 * p.Hkv + g) * 4 + j % kPage / PA_SCALE_TOKENS;
    float k[kDims], v[kDims];
#pragma unroll
    for (int d = 0; d < kDims; d += 4) {
      float y[4];
      fp8::unpack4(*reinterpret_cast<const uint32_t*>(row + d), y);
#pragma unroll
      for (int e = 0; e < 4; ++e) k[d + e] = y[e];
      fp8::unpack4(*reinterpret_cast<const uint32_t*>(row + p.Hkv * D + d), y);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[d + e] = y[e] * sc[p.Hkv * 4];
    }
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
      float x = 0.f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) x = fmaf(q[h][d], k[d], x);
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      x *= p.scale * sc[0];
      const float m_new = fmaxf(m[h], x);
      const float a = expf(m[h] - m_new), w = expf(x - m_new);
      l[h] = l[h] * a + w;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[h][d] = o[h][d] * a + w * v[d];
      m[h] = m_new;
    }
  }
#pragma unroll
  for (int h = 0; h < kMaxG; ++h) {
#pragma unroll
    for (int d = 0; d < kDims; ++d) xo[warp][h][lane * kDims + d] = o[h][d];
    xm[warp][h] = m[h];
    xl[warp][h] = l[h];
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < p.G * D; idx += kWarps * 32) {
    const int h = idx / D, d = idx - h * D;
    float big = -INFINITY, acc = 0.f, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) big = fmaxf(big, xm[w][h]);
    for (int w = 0; w < kWarps; ++w) {
      if (xm[w][h] == -INFINITY && xl[w][h] == 0.f) continue;
      const float a = expf(xm[w][h] - big);
      acc += a * xo[w][h][d];
      sum += a * xl[w][h];
    }
    const size_t r = (size_t)bt * p.Hq + g * p.G + h;
    const bool empty = tile.y <= tile.x;
    const float nan = __int_as_float(0x7fc00000);
    p.out[r * D + d] = s_bad ? nan : empty ? 0.f : acc / sum;
    if (d == 0) p.lse[r] = s_bad ? nan : empty ? -INFINITY : big + logf(sum);
  }
}

__global__ void merge_kernel(const float* out, const float* lse, int T, int H, int D, float* m_out,
                             float* m_lse) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
  mergerow::merge_row<false>(out, lse, b * T, T, H, h, D, m_out + (size_t)blockIdx.x * D,
                             m_lse + blockIdx.x, threadIdx.x);
}

size_t workspace_bytes() { return kStatusBytes; }

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
  auto aligned = [](const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
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
  PA_REQUIRE(ws_bytes >= workspace_bytes(), "workspace of %zu bytes is smaller than the %zu needed",
             ws_bytes, workspace_bytes());
  const long long max_tok = (long long)max_pages * kPage;
  for (long long i = 0; i < (long long)B * T; ++i) {
    const int s = tiles[2 * i], e = tiles[2 * i + 1];
    PA_REQUIRE(s >= 0 && s <= e && e <= max_tok,
               "tile %lld of request %lld is [%d, %d), outside [0, %lld]", i % T, i / T, s, e,
               max_tok);
  }
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.scales = scales;
  p.page_table = page_table;
  p.out = out;
  p.lse = lse;
  p.status = static_cast<int32_t*>(workspace);
  p.pool_pages = pool_pages;
  p.max_pages = max_pages;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.scale = scale;
  for (int bt0 = 0; bt0 < B * T; bt0 += kMaxTiles) {
    const int n = B * T - bt0 < kMaxTiles ? B * T - bt0 : kMaxTiles;
    p.bt0 = bt0;
    for (int i = 0; i < n; ++i)
      p.tiles[i] = make_int2(tiles[2 * (bt0 + i)], tiles[2 * (bt0 + i) + 1]);
    if (D == 128)
      PA_CHECK_CUDA(launch_dependent(decode_kernel<128>, dim3(n * Hkv), dim3(kWarps * 32), 0,
                                     stream, p));
    else
      PA_CHECK_CUDA(launch_dependent(decode_kernel<256>, dim3(n * Hkv), dim3(kWarps * 32), 0,
                                     stream, p));
  }
  if (merged_out)
    PA_CHECK_CUDA(launch_dependent(merge_kernel, dim3(B * Hq), dim3(32), 0, stream, out, lse, T,
                                   Hq, D, merged_out, merged_lse));
  PA_CHECK_CUDA(cudaGetLastError());
  return PA_OK;
}

}  // namespace decode_q8
}  // namespace pa

extern "C" size_t paged_decode_attn_q8_workspace_bytes(int B, int T, int n_q_heads, int n_kv_heads,
                                                       int head_dim) {
  if (B < 0 || T < 0 || (head_dim != 128 && head_dim != 256) || n_kv_heads < 1 ||
      n_q_heads < n_kv_heads || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > pa::decode_q8::kMaxG)
    return 0;
  return pa::decode_q8::workspace_bytes();
}

extern "C" int paged_decode_attn_q8_lse(const void* q, const void* pool, const float* scales,
                                        int64_t pool_pages, const int32_t* page_table,
                                        int max_pages, const int32_t* tiles, int B, int T,
                                        int n_q_heads, int n_kv_heads, int head_dim, float scale,
                                        float* out, float* lse, float* merged_out,
                                        float* merged_lse, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  pa::clear_error();
  return pa::decode_q8::run(q, pool, scales, pool_pages, page_table, max_pages, tiles, B, T,
                            n_q_heads, n_kv_heads, head_dim, scale, out, lse, merged_out,
                            merged_lse, workspace, workspace_bytes, stream);
}
