// What the two tree-attention kernels share: a sequence's plan, the classes of
// its key tiles, the TMA producers, the nodes' masks. Inline device code only.
//
// Warps of a CTA: 0-3 softmax, 4 and 5 producers of K (and Q) and V, 6 issuer of
// the S products, 7 issuer of the P V products.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_device.cuh"
#include "wp_prefill_common.cuh"
#include "wp_serve.h"

namespace wp {
namespace {

constexpr int NTHREADS = 256;
constexpr int K_WARP = 4, V_WARP = 5, QK_WARP = 6, PV_WARP = 7;
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

// Barrier `id` over `n` threads of the CTA (whole warps).
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// The same, and whether any of them brings a true value.
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

// Splits of a sequence: at most a.nsplit, each of at least MIN_KEYS keys.
constexpr int MIN_KEYS = 256;
template <int TILE>
__device__ __forceinline__ int sequence_splits(const TreeArgs &a, int tiles) {
  constexpr int least = MIN_KEYS / TILE;
  return max(1, min(a.nsplit, (tiles + least - 1) / least));
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

// Does a page of the keys [begin, end) lie outside the pool? Threads share the
// entries, every one of them returns for its own.
__device__ __forceinline__ bool bad_page(const CacheGeom &g, int b, int begin, int end, int thread, int threads) {
  if (g.block_table == nullptr || begin >= end) return false;
  bool bad = false;
  for (int64_t j = begin / g.page_size + thread; j <= (end - 1) / g.page_size; j += threads)
    bad = bad || cache_page(g, b, static_cast<int>(j * g.page_size)) < 0;
  return bad;
}

// Keys of one TMA box: the largest of 16, 32, .. TILE that never crosses a page.
struct Work {
  int b, hk, k_begin, k_end, ntiles;  // sequence, KV head, the CTA's keys and key tiles
  int first_row, nodes;               // first node of the CTA's rows; nodes of one Q box
};

// Copies of one tile's K that `need` names: groups (group-major K) or 64-dim
// chunks (K in rows). One elected lane issues them; an issue costs about 100
// cycles, whatever its size, so where a tile is one box high a run of groups
// goes in boxes of 4, 2 and 1.
template <int D, bool KGM, int TILE>
__device__ __forceinline__ void issue_k(const TreeMaps &tm, const Place &here, int have, uint32_t need, int box, int hk,
                                        uint8_t *dst, uint64_t *full, bool leader) {
  constexpr uint32_t GROUP = TILE * 32, CHUNK = TILE * 128;
  constexpr int PIECES = KGM ? D / 16 : D / 64;
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
    for (int i = 0; i < have; ++i) {  // the boxes that exist come first
      const int page = __shfl_sync(FULL, here.page, i), row = __shfl_sync(FULL, here.row, i);
      uint8_t *at = dst + i * box * (KGM ? 32 : 128);
      if (leader) {
#pragma unroll
        for (int g = 0; g < PIECES; ++g)
          if (need & (1u << g)) tma_load_5d(at + g * (KGM ? GROUP : CHUNK), &tm.k[0], full, 0, row, g, hk, page);
      }
    }
  }
  __syncwarp();
}

// Producer of Q and K. Lane i looks up box i % boxes one tile ahead of its
// loads (a block table's entry arrives meanwhile).
template <int D, bool KGM, int TILE>
__device__ __forceinline__ void produce_k(const TreeMaps &tm, const TreeArgs &a, const Work &w, int len, uint8_t *q_smem,
                                          uint32_t q_tile, uint64_t *q_full, uint8_t *ring_smem, uint64_t *k_full,
                                          uint64_t *k_empty, volatile int *abort_flag) {
  constexpr int G = D / 16;
  constexpr uint32_t STAGE = TILE * D * 2;
  const CacheGeom &cg = a.cache;
  const int lane = threadIdx.x % 32, R = a.Hq / cg.Hkv;
  const int box = a.box_rows, boxes = TILE / box, stages = a.k_stages;
  const int my_cut = lane < G ? a.cut[lane] : 0;
  const int key0 = w.k_begin + (lane & (boxes - 1)) * box;
  const long long lim = a.wait_limit;
  const bool leader = elect_one();
  Ring ring;  // of the next load; a slot is free once its previous round was consumed
  int issued = 0;
  if (w.ntiles > 0 && leader) {
    mbar_arrive_expect_tx(q_full, G * 32u * R * w.nodes);
    for (int g = 0; g < G; ++g) tma_load_4d(q_smem + g * q_tile, &tm.q, q_full, 16 * g, w.hk * R, w.first_row, w.b);
  }
  __syncwarp();
  Place here = place_of(cg, w.b, key0, w.k_end);
  for (int u = 0; u < w.ntiles; ++u) {
    const Place next = place_of(cg, w.b, key0 + (u + 1) * TILE, w.k_end);
    uint64_t *full = &k_full[ring.slot];
    uint8_t *dst = ring_smem + ring.slot * STAGE;
    uint32_t need = live_groups<TILE>(my_cut, G, len, w.k_begin + u * TILE, lane);
    if (!KGM) need = ((need & 0xfu) ? 1u : 0u) | ((need >> 4) ? 2u : 0u);  // 64-dim chunks
    if (u >= stages && !warp_wait_idle(&k_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) break;
    const int have = __popc(__ballot_sync(FULL, lane < boxes && here.page >= 0));
    if (leader) mbar_arrive_expect_tx(full, have * __popc(need) * box * (KGM ? 32u : 128u));
    issue_k<D, KGM, TILE>(tm, here, have, need, box, w.hk, dst, full, leader);
    ++issued;
    ring.next(stages);
    here = next;
  }
  // no bulk copy may still be in flight when this CTA's shared memory goes
  if (w.ntiles > 0) warp_wait_idle(q_full, 0, drain_limit(a), nullptr);
  for (int s = 0; s < stages && s < issued; ++s) {
    const int last = s + ((issued - 1 - s) / stages) * stages;
    warp_wait_idle(&k_full[s], (last / stages) & 1, drain_limit(a), nullptr);
  }
}

// Producer of V: whole rows, one box after the other; within a box the 64-dim
// chunks lie box * 128 bytes apart.
template <int D, int TILE>
__device__ __forceinline__ void produce_v(const TreeMaps &tm, const TreeArgs &a, const Work &w, uint8_t *ring_smem,
                                          uint64_t *v_full, uint64_t *v_empty, volatile int *abort_flag) {
  constexpr uint32_t STAGE = TILE * D * 2;
  const CacheGeom &cg = a.cache;
  const int lane = threadIdx.x % 32;
  const int box = a.box_rows, boxes = TILE / box, stages = a.v_stages;
  const int key0 = w.k_begin + (lane & (boxes - 1)) * box;
  const long long lim = a.wait_limit;
  const bool leader = elect_one();
  Ring ring;
  int issued = 0;
  Place here = place_of(cg, w.b, key0, w.k_end);
  for (int u = 0; u < w.ntiles; ++u) {
    const Place next = place_of(cg, w.b, key0 + (u + 1) * TILE, w.k_end);
    uint64_t *full = &v_full[ring.slot];
    if (u >= stages && !warp_wait_idle(&v_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) break;
    const int have = __popc(__ballot_sync(FULL, lane < boxes && here.page >= 0));
    if (leader) mbar_arrive_expect_tx(full, have * box * D * 2u);
    for (int i = 0; i < have; ++i) {
      const int page = __shfl_sync(FULL, here.page, i), row = __shfl_sync(FULL, here.row, i);
      if (leader) tma_load_5d(ring_smem + ring.slot * STAGE + i * box * D * 2, &tm.v, full, 0, row, 0, w.hk, page);
      __syncwarp();
    }
    ++issued;
    ring.next(stages);
    here = next;
  }
  for (int s = 0; s < stages && s < issued; ++s) {
    const int last = s + ((issued - 1 - s) / stages) * stages;
    warp_wait_idle(&v_full[s], (last / stages) & 1, drain_limit(a), nullptr);
  }
}

// Lane i gets the sum over the warp of every lane's v[i]: at each step a lane
// keeps half of its values and gives the other half away.
__device__ __forceinline__ float warp_sums(float (&v)[32]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(FULL, give, o);
    }
  return v[0];
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

}  // namespace
}  // namespace wp
