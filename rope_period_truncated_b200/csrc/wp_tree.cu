// Attention of a tree of drafted tokens over a cache (simple form: one warp
// per node and query head).
//
// Node t of sequence b stands at position len + depth(t) and sees the keys
// 0..len-1 of the context, its ancestors and itself (node u's K/V row is slot
// len + u of the cache, at position len + depth(u)):
//   s_tj = scale * sum_{g : dist <= W_g} q_t[g] . k_j[g],  dist = pos_t - pos_j,
// then softmax over the visible keys and O = sum_j p_j v_j.
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_device.cuh"
#include "wp_serve.h"

namespace wp {
namespace {

constexpr int WARPS = 4;

template <int D>
__global__ void __launch_bounds__(WARPS * 32) tree_simple_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;  // dims per lane, all of one group
  __shared__ int32_t par[TREE_MAX_NODES], depth[TREE_MAX_NODES];
  const int b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = a.lens[b], n = a.n_nodes != nullptr ? a.n_nodes[b] : a.T;
  const CacheGeom &g = a.cache;
  bool bad = len < 0 || n < 0 || n > a.T || static_cast<int64_t>(len) + n > cache_capacity(g);
  if (!bad && threadIdx.x < n) {
    par[threadIdx.x] = a.parents[static_cast<int64_t>(b) * a.T + threadIdx.x];
    bad = par[threadIdx.x] < -1 || par[threadIdx.x] >= static_cast<int>(threadIdx.x);
  }
  if (!bad && g.block_table != nullptr)
    for (int64_t s = static_cast<int64_t>(threadIdx.x) * g.page_size; s < len + n;
         s += static_cast<int64_t>(WARPS) * 32 * g.page_size)
      bad = bad || cache_page(g, b, static_cast<int>(s)) < 0;
  bad = __syncthreads_or(bad);
  if (!bad && threadIdx.x < n) {
    int e = 0;
    for (int t = par[threadIdx.x]; t >= 0; t = par[t]) ++e;
    depth[threadIdx.x] = e;
  }
  __syncthreads();
  const int idx = blockIdx.x * WARPS + warp;  // node * Hq + head
  if (idx >= a.T * a.Hq) return;
  const int t = idx / a.Hq, h = idx % a.Hq, hk = h / (a.Hq / g.Hkv);
  const int64_t row = (static_cast<int64_t>(b) * a.T + t) * a.Hq + h;
  float *lse = a.lse == nullptr ? nullptr : a.lse + (static_cast<int64_t>(b) * a.Hq + h) * a.T + t;
  float acc[E];
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  if (!bad && t < n) {
    uint64_t seen = 0;
    for (int u = t; u >= 0; u = par[u]) seen |= 1ull << u;
    const int W = a.cut[lane * E / 16];
    float q[E];
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row * D + lane * E + e]);
    const int64_t pos = static_cast<int64_t>(len) + depth[t];
    for (int j = 0; j < len + n; ++j) {
      if (j >= len && !((seen >> (j - len)) & 1)) continue;
      const int64_t page = cache_page(g, b, j);
      const int r = j % g.page_size, d0 = lane * E;
      const int64_t ko = k_offset(g, page, hk, r, d0 & ~7) + (d0 & 7), vo = v_offset(g, page, hk, r, d0 & ~7) + (d0 & 7);
      const int64_t dist = pos - (j < len ? j : len + depth[j - len]);
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += q[e] * __bfloat162float(g.kc[ko + e]);
      s = dist <= W ? s : 0.f;
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s);
      const float f = exp2f(m - mn), p = exp2f(s - mn);
      l = l * f + p;
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * __bfloat162float(g.vc[vo + e]);
      m = mn;
    }
  }
  const float nan = __int_as_float(0x7fc00000);
  for (int e = 0; e < E; ++e)
    a.o[row * D + lane * E + e] = __float2bfloat16_rn(bad ? nan : t < n ? acc[e] / l : 0.f);
  if (lane == 0 && lse != nullptr)
    *lse = bad ? nan : t < n ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
  const dim3 grid((a.T * a.Hq + WARPS - 1) / WARPS, a.B);
  if (a.cache.D == 128)
    tree_simple_kernel<128><<<grid, WARPS * 32, 0, stream>>>(a);
  else
    tree_simple_kernel<64><<<grid, WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace wp
