// The merge of every request's tiles as a launch of its own: the second launch of a
// decode call over the 8-bit and the 4-bit pool.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "common.h"
#include "ptx.cuh"

namespace pa {
namespace tilemerge {

// ---------------------------------------------------------------------------
// The merge of every request's T tiles, by the rule of lse_merge: a thread per
// float4 of an output row and every kTeams-th tile, kBatch tiles' values in
// flight with the LSEs that weigh them.  As a launch of its own it costs what
// its wait and a round of loads do, 1.5-2.5 us; inside the attention kernel, by
// the CTA that completed a request's tiles (as the bf16 kernel does it), such a
// CTA's stream stood still for an arrival and its answer and for code and values
// met cold: 262,144 tokens in 8 tiles 88.2 -> 85.4 us, 700 in 7 tiles 11.8 ->
// 7.4, 42 requests of 593 in 6 tiles 42.4 -> 33.0, 60 of up to 3,828 in 7 tiles
// 116.6 -> 82.9.  (Adding the partials of split units here too, in place of the
// attention kernel's slices, took 7 ragged requests in 5 tiles from 21.9 to 20.7
// us and 20,000 tokens in 20 tiles from 18.5 to 22.9: not kept.)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;
constexpr int kOneTeamTiles = 8;   // up to here one thread takes all tiles

template <int D, int kTeams>
__global__ void __launch_bounds__(kMergeThreads)
    merge_kernel(const float* out, const float* lse, int T, int Hq, int rows, float* m_out,
                 float* m_lse) {
  constexpr int kVec = D / 4, kRows = kMergeThreads / (kVec * kTeams);
  constexpr int kBatch = kTeams == 1 ? kOneTeamTiles : 4;
  __shared__ float4 s_acc[kTeams][kVec];
  __shared__ float s_m[kTeams], s_w[kTeams];
  ptx::launch_dependents();
  const int team = threadIdx.x / kVec % kTeams, c = threadIdx.x % kVec;
  const int row = blockIdx.x * kRows + threadIdx.x / (kVec * kTeams);
  if (row >= rows) return;   // (kTeams > 1: never, a block is a row)
  const size_t first = (size_t)(row / Hq) * T * Hq + row % Hq;   // of tile 0; tile t: + t Hq
  lse += first;
  const float4* src = reinterpret_cast<const float4*>(out) + first * kVec + c;
  const size_t step = (size_t)Hq * kVec;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, ws = 0.f;   // ws becomes NaN with a tile's LSE
  ptx::grid_dependency_wait();
  for (int t0 = team; t0 < T; t0 += kTeams * kBatch) {
    float4 x[kBatch];
    float l[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = t0 + i * kTeams;
      l[i] = -INFINITY;
      if (t < T) {
        l[i] = __ldcg(lse + (size_t)t * Hq);
        x[i] = __ldcg(src + t * step);
      }
    }
    float to = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) to = fmaxf(to, l[i]);
    const float f = m == -INFINITY ? 0.f : expf(m - to);
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
    ws = ws != ws ? ws : ws * f;
    m = to;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (l[i] == -INFINITY) continue;
      const float w = expf(l[i] - m);
      ws += w;
      acc.x = fmaf(w, x[i].x, acc.x);
      acc.y = fmaf(w, x[i].y, acc.y);
      acc.z = fmaf(w, x[i].z, acc.z);
      acc.w = fmaf(w, x[i].w, acc.w);
    }
  }
  if constexpr (kTeams > 1) {
    s_acc[team][c] = acc;
    if (c == 0) {
      s_m[team] = m;
      s_w[team] = ws;
    }
    __syncthreads();
    if (team != 0) return;
    for (int k = 1; k < kTeams; ++k) m = fmaxf(m, s_m[k]);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    ws = 0.f;
#pragma unroll
    for (int k = 0; k < kTeams; ++k) {
      const float f = s_m[k] == -INFINITY ? 0.f : expf(s_m[k] - m);
      const float4 x = s_acc[k][c];
      ws += s_w[k] != s_w[k] ? s_w[k] : f * s_w[k];
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
  }
  float4 y = make_float4(acc.x / ws, acc.y / ws, acc.z / ws, acc.w / ws);
  float z = m + logf(ws);
  if (ws != ws || m == -INFINITY) {
    z = ws != ws ? ws : -INFINITY;
    const float fill = ws != ws ? ws : 0.f;
    y = make_float4(fill, fill, fill, fill);
  }
  reinterpret_cast<float4*>(m_out + (size_t)row * D)[c] = y;
  if (c == 0) m_lse[row] = z;
}

// One thread per float4 for up to kOneTeamTiles tiles (one round of loads), a
// block per row behind that (64 tiles: 19.8 -> 12.9 us for the whole call).
template <int D>
cudaError_t launch_merge(const float* out, const float* lse, int T, int Hq, int rows, float* m_out,
                         float* m_lse, cudaStream_t stream) {
  constexpr int kTeams = kMergeThreads / (D / 4);
  const bool one = T <= kOneTeamTiles;
  const dim3 grid(one ? (rows + kTeams - 1) / kTeams : rows);
  return launch_dependent(one ? merge_kernel<D, 1> : merge_kernel<D, kTeams>, grid,
                          dim3(kMergeThreads), 0, stream, out, lse, T, Hq, rows, m_out, m_lse);
}

}  // namespace tilemerge
}  // namespace pa
