// What the two tree-attention kernels share: a sequence's plan, the classes of
// its key tiles, the loads of a tile's K, the nodes' masks. Inline device code
// only.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_device.cuh"
#include "wp_prefill_common.cuh"
#include "wp_serve.h"

namespace wp {
namespace {

constexpr float LOWEST = -3.4028234663852886e38f;  // of a running maximum: finite, so that m - m is 0

// Cycles to wait for the CTA's own copies and products before it gives back its
// shared memory and TMEM: they end by themselves, and a caller's short wait
// limit must not let the CTA go before them.
constexpr long long DRAIN_LIMIT = 2000000000;
__device__ __forceinline__ long long drain_limit(const TreeArgs &a) { return max(a.wait_limit, DRAIN_LIMIT); }

// Position in a ring of stages: slot, and the parity of its current round.
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++slot == stages) {
      slot = 0;
      round ^= 1u;
    }
  }
};

// 5-D tiled TMA load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_5d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barrier `id` over `n` threads of the CTA (whole warps), and whether any of
// them brings a true value.
__device__ __forceinline__ bool named_any(int id, int n, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(y)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(n)
      : "memory");
  return y != 0;
}

struct Plan {
  int len, n, total, tiles;  // context keys, nodes, keys, key tiles
  bool ok;
};

template <int TILE>
__device__ __forceinline__ Plan sequence_plan(const TreeArgs &a, int b) {
  Plan p;
  p.len = a.lens[b];
  p.n = a.n_nodes != nullptr ? a.n_nodes[b] : a.T;
  p.ok = p.len >= 0 && p.n >= 0 && p.n <= a.T && static_cast<int64_t>(p.len) + p.n <= cache_capacity(a.cache);
  p.total = p.ok ? p.len + p.n : 0;
  p.tiles = (p.total + TILE - 1) / TILE;
  return p;
}

// Where row `row` (node * R + head) of KV head hk writes.
__device__ __forceinline__ int64_t out_row(const TreeArgs &a, int b, int hk, int R, int row) {
  return (static_cast<int64_t>(b) * a.T + row / R) * a.Hq + hk * R + row % R;
}
__device__ __forceinline__ float *out_lse(const TreeArgs &a, int b, int hk, int R, int row) {
  return a.lse == nullptr ? nullptr : a.lse + (static_cast<int64_t>(b) * a.Hq + hk * R + row % R) * a.T + row / R;
}

// Smallest distance of a tile's pairs that count (0 with drafted keys in it).
template <int TILE>
__device__ __forceinline__ int64_t tile_dmin(int len, int k0) {
  return k0 + TILE > len ? 0 : static_cast<int64_t>(len) - (k0 + TILE - 1);
}

// Groups that some pair of the tile at key k0 keeps; group g's cutoff W in lane g.
template <int TILE>
__device__ __forceinline__ uint32_t live_groups(int W, int G, int len, int k0, int lane) {
  return __ballot_sync(FULL, lane < G && tile_dmin<TILE>(len, k0) <= W);
}

// Full groups (bits 0-7: every pair keeps them) and boundary groups (8-15).
template <int TILE>
__device__ __forceinline__ uint32_t tile_classes(int W, int G, int len, int deepest, int k0, int lane) {
  const int64_t dmax = static_cast<int64_t>(len) + deepest - min(k0, len);
  const bool live = lane < G && tile_dmin<TILE>(len, k0) <= W;
  const bool full = live && dmax <= W;
  return __ballot_sync(FULL, full) | (__ballot_sync(FULL, live && !full) << 8);
}

// Where a box of keys lies: page and row in it; page < 0: behind the last key.
// An entry that is no page reaches TMA as a coordinate outside the tensor
// (zeros, nothing read); the pages are checked apart from the loads.
struct Place {
  int page, row;
};
__device__ __forceinline__ Place place_of(const CacheGeom &g, int b, int key, int end) {
  if (key >= end) return Place{-1, 0};
  if (g.block_table == nullptr) return Place{b, key};
  const int j = key / g.page_size;
  return Place{g.block_table[static_cast<int64_t>(b) * g.max_pages + j], key - j * g.page_size};
}

// Copies of one tile's K that `need` names: groups (group-major K) or 64-dim
// chunks (K in rows). One elected lane issues them; an issue costs about 100
// cycles, whatever its size, so where a tile is one box high a run of groups
// goes in boxes of 4, 2 and 1. The loops stay rolled: a CTA's warps run five
// different loops at a time, and unrolled ones do not fit the instruction cache
// (16 sequences of 16K to 32K keys in pages of 32, 32 rows: 259 us unrolled, 222
// rolled).
template <int D, bool KGM, int TILE>
__device__ __forceinline__ void issue_k(const TreeMaps &tm, const Place &here, int have, uint32_t need, int box, int hk,
                                        uint8_t *dst, uint64_t *full, bool leader) {
  constexpr uint32_t GROUP = TILE * 32, CHUNK = TILE * 128;
  if (box == TILE) {
    const int page = __shfl_sync(FULL, here.page, 0), row = __shfl_sync(FULL, here.row, 0);
    if (leader && have) {
      for (uint32_t left = need; left;) {
        const int g = __ffs(left) - 1;
        const uint32_t run = left >> g;
        const int wide = KGM && (run & 0xfu) == 0xfu ? 2 : (run & 3u) == 3u ? 1 : 0;  // log2 of the box
        tma_load_5d(dst + g * (KGM ? GROUP : CHUNK), &tm.k[wide], full, 0, row, g, hk, page);
        left &= ~(((1u << (1 << wide)) - 1) << g);
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < have; ++i) {  // the boxes that exist come first
      const int page = __shfl_sync(FULL, here.page, i), row = __shfl_sync(FULL, here.row, i);
      uint8_t *at = dst + i * box * (KGM ? 32 : 128);
      if (leader) {
#pragma unroll 1
        for (uint32_t left = need; left; left &= left - 1) {
          const int g = __ffs(left) - 1;
          tma_load_5d(at + g * (KGM ? GROUP : CHUNK), &tm.k[0], full, 0, row, g, hk, page);
        }
      }
    }
  }
  __syncwarp();
}

// Offset, in 16-byte units, of 16 keys kk of a V tile from its start.
template <int D>
__device__ __forceinline__ uint32_t v_step(int kk, int box) {
  const int i = kk * 16 / box;
  return static_cast<uint32_t>(i * box * D * 2 + (kk * 16 - i * box) * 128) >> 4;
}

// The nodes, by one warp: what each one sees (itself and its ancestors, bit per
// node) and its depth, by pointer doubling: after step i a node has joined 2^i
// of its ancestors. Returns whether a parent is out of range (then every node
// sees only itself). `jump`: 64 words of scratch.
__device__ __forceinline__ bool node_masks(const TreeArgs &a, const Plan &plan, int b, uint64_t *sees, int32_t *depth,
                                           int32_t *jump, int *deepest) {
  const int lane = threadIdx.x % 32;
  int j[2];
  uint64_t m[2];
  bool bad = !plan.ok;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    const bool there = plan.ok && t < plan.n;
    j[e] = -1;
    m[e] = there ? 1ull << t : 0ull;
    const int p = there ? a.parents[static_cast<int64_t>(b) * a.T + t] : -1;
    if (p < -1 || p >= t)
      bad = bad || there;
    else
      j[e] = p;
  }
  bad = __any_sync(FULL, bad);
  if (bad) j[0] = j[1] = -1;
  while (__any_sync(FULL, j[0] >= 0 || j[1] >= 0)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sees[lane + 32 * e] = m[e];
      jump[lane + 32 * e] = j[e];
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (j[e] >= 0) {
        m[e] |= sees[j[e]];
        j[e] = jump[j[e]];
      }
    __syncwarp();
  }
  int deep = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = m[e] ? __popcll(m[e]) - 1 : 0;
    sees[lane + 32 * e] = m[e];
    depth[lane + 32 * e] = d;
    deep = max(deep, d);
  }
  deep = __reduce_max_sync(FULL, deep);
  if (lane == 0) *deepest = deep;
  return bad;
}

// A warp merges `count` partial results of one row, partial i in slot(i): O =
// sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M), E dims per lane. Eight at a time,
// their LSE and rows loaded together, each time brought to the maximum so far: a
// load takes as long as the arithmetic of all of them. M = infinity: spoilt.
template <int D, class Slot>
__device__ __forceinline__ void merge_row(const TreeArgs &a, int count, Slot slot, float (&acc)[D / 32], float &sum, float &M) {
  constexpr int E = D / 32, BATCH = 8;
  const int lane = threadIdx.x % 32;
  M = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i = 0; i < count; i += BATCH) {
    float l[BATCH], v[BATCH][E];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const bool in = i + k < count;
      const int64_t s = in ? slot(i + k) : 0;
      l[k] = in ? a.lse_part[s] : -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = in ? a.o_part[s * D + lane * E + e] : 0.f;
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) m = fmaxf(m, l[k]);
    const float scale = M == -INFINITY ? 0.f : fast_exp2(M - m);
    sum *= scale;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= scale;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float w = l[k] == -INFINITY ? 0.f : fast_exp2(l[k] - m);
      sum += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * v[k][e];
    }
    M = m;
  }
}

}  // namespace
}  // namespace wp
