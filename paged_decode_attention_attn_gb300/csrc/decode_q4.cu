// Paged GQA decode attention over a 4-bit pool (e2m1 codes, a power of two as the scale
// of each 32 values of a token's head) with a per-tile log-sum-exp.
//
// The simplest form: a CTA per (tile, kv head), a warp per token, fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "common.h"
#include "fp4.cuh"
#include "ptx.cuh"
#include "split_units.cuh"
#include "tile_merge.cuh"

namespace pa {
namespace decode_q4 {

using namespace split;

constexpr int kGroup = PA_Q4_GROUP;
constexpr int kThreads = 128, kWarps = kThreads / 32;

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* pool;
  const uint8_t* scales;
  const int32_t* page_table;
  float* out;
  float* lse;
  float* out2;
  float* lse2;
  int32_t* status;
  long long pool_pages;
  int max_pages, T, Hq, Hkv, G;
  float scale;
  Unit units[kMaxUnitsLarge];
};
static_assert(sizeof(Params) <= 32764, "kernel parameters too large");

// A lane's dims of a row: N codes from byte N / 2 * lane of its codes.
template <int N>
__device__ __forceinline__ void load_row(const uint8_t* codes, const uint8_t* scales, int lane,
                                         float (&y)[N]) {
  uint32_t w;
  if constexpr (N == 8) w = __ldg(reinterpret_cast<const uint32_t*>(codes) + lane);
  else w = __ldg(reinterpret_cast<const uint16_t*>(codes) + lane);
  float x[8];
  fp4::unpack8(w, x);
  const float s = fp4::scale_of(__ldg(scales + lane * N / kGroup));
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = x[i] * s;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    decode_q4_kernel(const __grid_constant__ Params p) {
  constexpr int N = D / 32;
  __shared__ float s_m[kWarps][kMaxG], s_l[kWarps][kMaxG];
  __shared__ float s_o[kWarps][kMaxG][D];
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  const Unit& U = p.units[blockIdx.x];
  const int b = U.bt / p.T;
  float q[kMaxG][N], o[kMaxG][N] = {}, m[kMaxG], l[kMaxG] = {};
#pragma unroll
  for (int h = 0; h < kMaxG; ++h) {
    m[h] = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      q[h][i] = h < p.G ? __bfloat162float(p.q[((size_t)b * p.Hq + U.g * p.G + h) * D + lane * N + i])
                        : 0.f;
  }
  for (int j = U.tok_start + warp; j < U.tok_end; j += kWarps) {
    const int page = p.page_table[(size_t)b * p.max_pages + j / kPage];
    if (page < 0 || page >= p.pool_pages) {
      if (lane == 0) {
        atomicOr(p.status, PA_STATUS_BAD_PAGE);
        s_bad = 1;
      }
      continue;
    }
    const size_t k_at = ((size_t)page * 2 * p.Hkv + U.g) * kPage + j % kPage;
    const size_t v_at = k_at + (size_t)p.Hkv * kPage;
    float k[N], v[N];
    load_row<N>(p.pool + k_at * (D / 2), p.scales + k_at * (D / kGroup), lane, k);
    load_row<N>(p.pool + v_at * (D / 2), p.scales + v_at * (D / kGroup), lane, v);
    for (int h = 0; h < kMaxG; ++h) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) x = fmaf(q[h][i], k[i], x);
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      x *= p.scale;
      const float to = fmaxf(m[h], x);
      const float a = m[h] == -INFINITY ? 0.f : expf(m[h] - to);
      const float e = to == -INFINITY && x == x ? 0.f : expf(x - to);
      m[h] = to;
      l[h] = fmaf(l[h], a, e);
#pragma unroll
      for (int i = 0; i < N; ++i) o[h][i] = fmaf(o[h][i], a, e * v[i]);
    }
  }
#pragma unroll
  for (int h = 0; h < kMaxG; ++h) {
    if (lane == 0) {
      s_m[warp][h] = m[h];
      s_l[warp][h] = l[h];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[warp][h][lane * N + i] = o[h][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * D; i += kThreads) {
    const int h = i / D, d = i % D;
    float top = -INFINITY, sum = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][h]);
    for (int w = 0; w < kWarps; ++w) {
      const float a = s_m[w][h] == -INFINITY ? (s_l[w][h] == s_l[w][h] ? 0.f : s_l[w][h])
                                             : expf(s_m[w][h] - top);
      sum = fmaf(a, s_l[w][h], sum);
      y = fmaf(a, s_o[w][h][d], y);
    }
    float x = top + logf(sum);
    y = sum == 0.f ? 0.f : y / sum;
    if (sum == 0.f) x = -INFINITY;
    if (s_bad) x = y = __int_as_float(0x7fc00000);
    const size_t row = (size_t)U.bt * p.Hq + U.g * p.G + h;
    p.out[row * D + d] = y;
    if (p.out2) p.out2[row * D + d] = y;
    if (d == 0) p.lse[row] = x;
    if (d == 0 && p.lse2) p.lse2[row] = x;
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int run(const void* q, const void* pool, const uint8_t* scales, int64_t pool_pages,
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
  PA_REQUIRE(pool_pages < (1ll << 31) / (2 * Hkv), "pool too large for 32-bit page coordinates");
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
  Plan plan;
  const int rc = plan_units(
      tiles, B, T, Hkv, 0, false,
      [&](const Unit*, const int32_t*, size_t, long long total, std::vector<int32_t>* starts) {
        equal_starts(std::max(total, 1ll), 1, starts);
      },
      &plan);
  if (rc != PA_OK) return rc;
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.scales = scales;
  p.page_table = page_table;
  p.out = out;
  p.lse = lse;
  p.out2 = T == 1 ? merged_out : nullptr;
  p.lse2 = T == 1 ? merged_lse : nullptr;
  p.status = Workspace(workspace, B, T, Hkv, D).status;
  p.pool_pages = pool_pages;
  p.max_pages = max_pages;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.scale = scale;
  for (const Launch& L : plan.launches) {
    std::copy_n(plan.units.data() + L.u0, L.n, p.units);
    PA_CHECK_CUDA(launch_dependent(D == 128 ? decode_q4_kernel<128> : decode_q4_kernel<256>,
                                   dim3(L.n), dim3(kThreads), 0, stream, p));
    PA_CHECK_CUDA(cudaGetLastError());
  }
  if (T > 1 && merged_out != nullptr) {
    auto merge = D == 128 ? tilemerge::launch_merge<128> : tilemerge::launch_merge<256>;
    PA_CHECK_CUDA(merge(out, lse, T, Hq, B * Hq, merged_out, merged_lse, stream));
    PA_CHECK_CUDA(cudaGetLastError());
  }
  return PA_OK;
}

}  // namespace decode_q4
}  // namespace pa

extern "C" size_t paged_decode_attn_q4_workspace_bytes(int B, int T, int n_q_heads, int n_kv_heads,
                                                       int head_dim) {
  if (B < 0 || T < 0 || (head_dim != 128 && head_dim != 256) || n_kv_heads < 1 ||
      n_q_heads < n_kv_heads || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > pa::split::kMaxG)
    return 0;
  return pa::split::workspace_bytes(B, T, n_kv_heads, head_dim);
}

extern "C" int paged_decode_attn_q4_lse(const void* q, const void* pool, const uint8_t* scales,
                                        int64_t pool_pages, const int32_t* page_table,
                                        int max_pages, const int32_t* tiles, int B, int T,
                                        int n_q_heads, int n_kv_heads, int head_dim, float scale,
                                        float* out, float* lse, float* merged_out,
                                        float* merged_lse, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  pa::clear_error();
  try {
    return pa::decode_q4::run(q, pool, scales, pool_pages, page_table, max_pages, tiles, B, T,
                              n_q_heads, n_kv_heads, head_dim, scale, out, lse, merged_out,
                              merged_lse, workspace, workspace_bytes, stream);
  } catch (const std::exception& e) {
    return pa::fail(PA_ERR_INVALID, "host memory for the plan: %s", e.what());
  }
}
