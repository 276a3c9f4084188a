// Attention of a tree of drafted tokens over a cache, on sm_100a: TMA +
// tcgen05 + TMEM, split over the keys.
//
// Node t of sequence b stands at position len + depth(t) and sees the keys
// 0..len-1 of the context, its ancestors and itself (node u's K/V row is key
// len + u of the cache, at position len + depth(u)):
//   s_tj = scale * sum_{g : dist <= W_g} q_t[g] . k_j[g],  dist = pos_t - pos_j,
// then softmax over the visible keys and O = sum_j p_j v_j. A group out of
// window adds 0; an invisible key is left out of the softmax.
//
// The rows of one KV head are its R = Hq/Hkv query heads of every node, row
// m = node * R + head: they share every K/V tile. One CTA takes up to 128 rows
// (whole nodes) and one range of keys, in sub-tiles of 64:
//   warps 4-5 TMA producers: Q once, and per sub-tile the K pieces that a live
//             group needs (group-major K: 16-dim groups; K in rows: 64-dim
//             chunks of four groups); V. A box never crosses a page: it has
//             gcd(page size, 64) rows.
//   warp 6    issuer of S = sum of one M128 N64 K16 product per live group. S
//             has two 64-column halves, so the softmax of u runs beside the
//             products of u + 1.
//   warp 7    issuer of O += P V (P bf16 in S's place, V MN-major). One warp
//             for both was what bounded the kernel: issuing a sub-tile's 12
//             products and their commits took it about 1800 cycles.
//   warps 0-3 softmax, a row per thread, online in base 2; O is rescaled only
//             when a maximum grows by more than 2^8. P rounds to bf16 (2^-8 of
//             each weight, as in the package's prefill and decode): both
//             operands of a product have one type, and V is bf16. Maxima, sums,
//             O and partial results are fp32; the sums take P unrounded.
// Groups whose cutoff falls inside a sub-tile's distances go first, one cutoff
// at a time in ascending order, and S is masked in place after each (windows
// of ascending cutoffs are nested, so later masks keep what earlier ones did).
//
// Sub-tiles that hold drafted keys are the last one or two: there a row takes
// a 64-bit word of what it sees (context keys, its ancestors' bits), and rows
// of V behind the last key are zeroed in shared memory before the product, so
// that P = 0 meets no NaN that an unused slot may hold.
//
// Splits write O (fp32) and LSE to the workspace; a second kernel merges them
// (4 to 7 us; merging in a cluster through its shared memory took 7 and more).
//
// What bounds it. Short caches: latency. 4 sequences of 2.5K to 4K keys, 64
// rows: 25 us a call. By length (4 x 512, 1K, 2K, 4K, 8K keys: 15.5, 16.4, 19.2,
// 23.7, 35 us) a CTA's eighth of 4K keys, 8 sub-tiles one after the other, is 9
// us of that (1.1 us each, from 8K keys on 1.4); launches, first keys, last rows
// and the merge are 11, the partial rows of 8 splits instead of 2 about 4. 16
// sequences of 16K to 32K keys, 64 rows: 245 us, 5.1 TB/s. 252 rows over 128K
// keys, most groups live: 143 us back to back (612 TFLOP/s), 170 us a call among
// calls on other inputs; no pipe is full (tensor 33 %, XU 50 %, DRAM 33 %), a
// sub-tile takes about 1760 cycles per CTA: P V(u) to S(u + 2) to P(u + 2) is a
// chain through two issuers and their barriers, and the two row tiles of a KV
// head run as separate CTAs that each load all keys (one of them from L2). wp_prefill.cu runs products
// of the same shape at 980 TFLOP/s with two row tiles on one K/V stage, one
// issuer per tile whose order spares those barriers, and part of the exponentials
// on the FMA pipe; that arrangement has not been built here.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_tree.cuh"

namespace wp {
namespace {

constexpr int NTHREADS = 256;
constexpr int K_WARP = 4, V_WARP = 5, QK_WARP = 6, PV_WARP = 7;
constexpr int SUB = 64;  // keys per sub-tile
constexpr int SMEM_PER_CTA = 115712;  // (228 KB - 2 x 1 KB reserved) / 2
constexpr uint32_t TMEM_COLS = 256;  // two CTAs per SM share 512
constexpr uint32_t COL_S = 0, COL_O = 128;
constexpr uint32_t K_TILE = SUB * 32;  // 64 keys x 16 bf16 (group-major K)
constexpr uint32_t CHUNK = SUB * 128;  // 64 keys x 64 bf16 (V, and K in rows)

// Shared memory: the K and V rings, then Q (one tile of `rows` rows per group,
// rows rounded up to 8), then the nodes and barriers. The products read 128
// rows from each Q tile: what lies beyond a tile's rows (the next tile, or the
// space behind the last) only makes rows of S and O that nobody reads.
constexpr uint32_t NUM_BARS = 1 + 4 * TREE_MAX_STAGES + 3 * 2 + 5;

template <int D>
struct Layout {
  static constexpr int G = D / 16;
  static constexpr uint32_t STAGE = SUB * D * 2;  // one K or V sub-tile
  static constexpr uint32_t PITCH = D * 4 + 16;   // of a row of O (fp32), in the end, over the rings and Q
  uint32_t v_off, q_off, q_tile, node_off, bar_off, misc_off;
  __host__ __device__ Layout(int kst, int vst, int rows) {
    v_off = kst * STAGE;
    q_off = v_off + vst * STAGE;
    q_tile = ((rows + 7) & ~7) * 32;
    node_off = q_off + (G - 1) * q_tile + 128 * 32;  // uint64 sees[64], int32 depth[64], jump[64]
    bar_off = node_off + 64 * 16;
    misc_off = bar_off + NUM_BARS * 8;  // abort flag, TMEM base, deepest node
  }
  __host__ __device__ uint32_t bytes() const { return misc_off + 16 + 1024; }  // + alignment
};

// Columns c of su whose bit is clear become `fill`.
__device__ __forceinline__ void keep_columns(uint32_t (&su)[64], uint64_t bits, uint32_t fill) {
  const uint32_t lo = static_cast<uint32_t>(bits), hi = static_cast<uint32_t>(bits >> 32);
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    if (!(lo & (1u << c))) su[c] = fill;
    if (!(hi & (1u << c))) su[32 + c] = fill;
  }
}

// Splits of a sequence: at most a.nsplit, each of at least MIN_KEYS keys.
constexpr int MIN_KEYS = 256;
__device__ __forceinline__ int sequence_splits(const TreeArgs &a, int tiles) {
  constexpr int least = MIN_KEYS / SUB;
  return max(1, min(a.nsplit, (tiles + least - 1) / least));
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

struct Work {
  int b, hk, k_begin, k_end, ntiles;  // sequence, KV head, the CTA's keys and key tiles
  int first_row, nodes;               // first node of the CTA's rows; nodes of one Q box
};

// Producer of Q and K. Lane i looks up box i % boxes one tile ahead of its
// loads (a block table's entry arrives meanwhile).
template <int D, bool KGM>
__device__ __forceinline__ void produce_k(const TreeMaps &tm, const TreeArgs &a, const Work &w, int len, uint8_t *q_smem,
                                          uint32_t q_tile, uint64_t *q_full, uint8_t *ring_smem, uint64_t *k_full,
                                          uint64_t *k_empty, volatile int *abort_flag) {
  constexpr int G = D / 16;
  constexpr uint32_t STAGE = SUB * D * 2;
  const CacheGeom &cg = a.cache;
  const int lane = threadIdx.x % 32, R = a.Hq / cg.Hkv;
  const int box = a.box_rows, boxes = SUB / box, stages = a.k_stages;
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
    const Place next = place_of(cg, w.b, key0 + (u + 1) * SUB, w.k_end);
    uint64_t *full = &k_full[ring.slot];
    uint8_t *dst = ring_smem + ring.slot * STAGE;
    uint32_t need = live_groups<SUB>(my_cut, G, len, w.k_begin + u * SUB, lane);
    if (!KGM) need = ((need & 0xfu) ? 1u : 0u) | ((need >> 4) ? 2u : 0u);  // 64-dim chunks
    if (u >= stages && !warp_wait_idle(&k_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) break;
    const int have = __popc(__ballot_sync(FULL, lane < boxes && here.page >= 0));
    if (leader) mbar_arrive_expect_tx(full, have * __popc(need) * box * (KGM ? 32u : 128u));
    issue_k<D, KGM, SUB>(tm, here, have, need, box, w.hk, dst, full, leader);
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
template <int D>
__device__ __forceinline__ void produce_v(const TreeMaps &tm, const TreeArgs &a, const Work &w, uint8_t *ring_smem,
                                          uint64_t *v_full, uint64_t *v_empty, volatile int *abort_flag) {
  constexpr uint32_t STAGE = SUB * D * 2;
  const CacheGeom &cg = a.cache;
  const int lane = threadIdx.x % 32;
  const int box = a.box_rows, boxes = SUB / box, stages = a.v_stages;
  const int key0 = w.k_begin + (lane & (boxes - 1)) * box;
  const long long lim = a.wait_limit;
  const bool leader = elect_one();
  Ring ring;
  int issued = 0;
  Place here = place_of(cg, w.b, key0, w.k_end);
  for (int u = 0; u < w.ntiles; ++u) {
    const Place next = place_of(cg, w.b, key0 + (u + 1) * SUB, w.k_end);
    uint64_t *full = &v_full[ring.slot];
    if (u >= stages && !warp_wait_idle(&v_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) break;
    const int have = __popc(__ballot_sync(FULL, lane < boxes && here.page >= 0));
    if (leader) mbar_arrive_expect_tx(full, have * box * D * 2u);
#pragma unroll 1
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

template <int D, bool KGM>
__global__ void __launch_bounds__(NTHREADS, 2)
    tree_kernel(const __grid_constant__ TreeMaps tm, const __grid_constant__ TreeArgs a) {
  cudaGridDependencySynchronize();
  constexpr int G = D / 16;
  constexpr uint32_t STAGE = Layout<D>::STAGE;
  constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, SUB, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int KST = a.k_stages, VST = a.v_stages;
  const Layout<D> L(KST, VST, a.tile_nodes * (a.Hq / a.cache.Hkv));
  uint64_t *sees = reinterpret_cast<uint64_t *>(smem + L.node_off);
  int32_t *depth = reinterpret_cast<int32_t *>(smem + L.node_off + 64 * 8);
  int32_t *jump = depth + 64;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L.bar_off);
  uint64_t *q_full = bars, *k_full = q_full + 1, *k_empty = k_full + TREE_MAX_STAGES, *v_full = k_empty + TREE_MAX_STAGES,
           *v_empty = v_full + TREE_MAX_STAGES, *s_ready = v_empty + TREE_MAX_STAGES, *p_ready = s_ready + 2, *o_ready = p_ready + 2, *o_final = o_ready + 2,
           *bnd_ready = o_final + 1, *bnd_done = bnd_ready + 1, *drain = bnd_done + 1;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L.misc_off);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L.misc_off + 4);
  int *s_deepest = reinterpret_cast<int *>(smem + L.misc_off + 8);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheGeom &cg = a.cache;
  const int R = a.Hq / cg.Hkv;
  const int mt = static_cast<int>(blockIdx.x) % a.row_tiles, split = static_cast<int>(blockIdx.x) / a.row_tiles;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int row0 = mt * a.tile_nodes * R;                            // first row of this CTA
  const int rows = min(a.tile_nodes, a.T - mt * a.tile_nodes) * R;  // up to 128
  const int warps = (rows + 31) / 32;                               // softmax warps with rows
  const Plan plan = sequence_plan<SUB>(a, b);
  const int splits = sequence_splits(a, plan.tiles);
  if (split >= splits) return;
  const int t_begin = static_cast<int>(static_cast<int64_t>(plan.tiles) * split / splits);
  const int nsub_all = static_cast<int>(static_cast<int64_t>(plan.tiles) * (split + 1) / splits) - t_begin;
  const int k_begin = t_begin * SUB;
  const int k_end = min(k_begin + nsub_all * SUB, plan.total);
  const long long lim = a.wait_limit;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(q_full, 1);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_ready[s], 1);
      mbar_init(&p_ready[s], warps);
      mbar_init(&o_ready[s], 1);
    }
    mbar_init(o_final, 1);
    mbar_init(bnd_ready, 1);
    mbar_init(bnd_done, warps);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_barrier_init();
  }
  if (warp == QK_WARP) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int box = a.box_rows;
  const Work work{b, hk, k_begin, k_end, nsub_all, mt * a.tile_nodes, a.tile_nodes};
  // The producers need no more than the lengths; the others look at the nodes
  // and the pages meanwhile. A bad sequence raises the abort flag for them.
  bool bad = !plan.ok;
  if (warp == PV_WARP) bad = node_masks(a, plan, b, sees, depth, jump, s_deepest);
  if (warp < 4) bad = bad || bad_page(cg, b, k_begin, k_end, threadIdx.x, 128);
  if (warp != K_WARP && warp != V_WARP) {
    bad = named_any(1, NTHREADS - 64, bad);
    if (bad) *abort_flag = 1;
  }
  const uint32_t tmem = *tmem_slot;
  const int deepest = warp != K_WARP && warp != V_WARP ? *s_deepest : 0;
  const int nsub = bad ? 0 : nsub_all;
  const int my_cut = lane < G ? a.cut[lane] : 0;
  // The rows' place among the 128 lanes. A warp reaches the lanes of its own
  // quarter only, and warps w of both CTAs of an SM share a scheduler: few rows
  // go to other quarters in the CTA that got the upper half of TMEM, one warp of
  // rows to the quarters whose schedulers the producers' warps share, not the
  // issuers'.
  const int half = (tmem & 0xffffu) >= TMEM_COLS ? 1 : 0;
  const int warp0 = warps == 1 ? half : warps == 2 ? 2 * half : 0;

  if (warp == K_WARP) {
    produce_k<D, KGM>(tm, a, work, plan.len, smem + L.q_off, L.q_tile, q_full, smem, k_full, k_empty, abort_flag);
  } else if (warp == V_WARP) {
    produce_v<D>(tm, a, work, smem + L.v_off, v_full, v_empty, abort_flag);
  } else if (warp == QK_WARP) {
    // --------------------------------------------------------- issuer of S
    // S(u) into half u & 1, once P V(u - 2) has read the P that lies there.
    const bool leader = elect_one();
    // row 0 of Q stands in lane 32 * warp0: the tile begins that many rows earlier
    const uint64_t q_desc = smem_desc(smem_u32(smem + L.q_off) - warp0 * 1024, 16, 256, SMEM_SWIZZLE_32B);
    const uint64_t k_desc = KGM ? smem_desc(smem_u32(smem), 16, 256, SMEM_SWIZZLE_32B)
                                : smem_desc(smem_u32(smem), 16, 1024, SMEM_SWIZZLE_128B);
    Ring ring;
    int bnd_cnt = 0;
    bool ok = nsub > 0 && warp_wait(q_full, 0, lim, abort_flag);
    const auto issue_groups = [&](uint32_t s_col, uint64_t kst_desc, uint32_t groups, uint32_t acc) {
#pragma unroll 1
      for (int g = 0; g < G; ++g)
        if (groups & (1u << g)) {
          // K in rows: group g is 32 bytes into the 128-byte rows of chunk g / 4
          const uint32_t koff = KGM ? g * K_TILE : (g / 4) * CHUNK + (g % 4) * 32;
          umma_ss(s_col, q_desc + g * (L.q_tile >> 4), kst_desc + (koff >> 4), IDESC_QK, acc);
          acc = 1;
        }
    };
    for (int u = 0; ok && u < nsub; ++u) {
      const int hh = u & 1;
      const uint32_t cls = tile_classes<SUB>(my_cut, G, plan.len, deepest, k_begin + u * SUB, lane);
      const uint32_t s_col = tmem + COL_S + SUB * hh;
      const uint64_t kst_desc = k_desc + ((ring.slot * STAGE) >> 4);
      ok = warp_wait(&k_full[ring.slot], ring.round, lim, abort_flag) &&
           (u < 2 || warp_wait(&o_ready[hh], ((u >> 1) - 1) & 1, lim, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t acc = 0;
      const uint32_t bnd = cls >> 8;
      if (bnd) {
        // boundary classes first, ascending cutoff; each one masked in place
        int64_t prev = -1;
        int32_t W;
        uint32_t groups;
        while (ok && next_boundary_class(a.cut, bnd, prev, &W, &groups)) {
          if (leader) {
            issue_groups(s_col, kst_desc, groups, acc);
            umma_commit(bnd_ready);
          }
          acc = 1;
          __syncwarp();
          ok = warp_wait(bnd_done, bnd_cnt & 1, lim, abort_flag);
          tc_fence_after();
          ++bnd_cnt;
          prev = W;
        }
        if (!ok) break;
      }
      if (leader) {
        issue_groups(s_col, kst_desc, cls & 0xffu, acc);
        umma_commit(&s_ready[hh]);
        umma_commit(&k_empty[ring.slot]);
      }
      __syncwarp();
      ring.next(KST);
    }
    // every product must have finished before TMEM is given back
    if (leader) umma_commit(&drain[0]);
    __syncwarp();
    warp_wait(&drain[0], 0, drain_limit(a), nullptr);
  } else if (warp == PV_WARP) {
    // --------------------------------------------------------- issuer of O
    const bool leader = elect_one();
    // V: dims contiguous (MN-major), one box after the other; in a box 8-key row
    // groups lie 1024 B apart and 64-dim chunks box * 128 B
    const uint64_t v_desc = smem_desc(smem_u32(smem + L.v_off), box * 128, 1024, SMEM_SWIZZLE_128B);
    Ring ring;
    for (int u = 0; u < nsub; ++u) {
      const int hh = u & 1;
      const uint64_t vst_desc = v_desc + ((ring.slot * STAGE) >> 4);
      if (!warp_wait(&v_full[ring.slot], ring.round, lim, abort_flag) || !warp_wait(&p_ready[hh], (u >> 1) & 1, lim, abort_flag))
        break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < SUB / 16; ++kk)
          umma_ts(tmem + COL_O, tmem + COL_S + SUB * hh + kk * 8, vst_desc + v_step<D>(kk, box), IDESC_PV,
                  (u > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&o_ready[hh]);
        umma_commit(&v_empty[ring.slot]);
        if (u == nsub - 1) umma_commit(o_final);
      }
      __syncwarp();
      ring.next(VST);
    }
    if (leader) umma_commit(&drain[1]);
    __syncwarp();
    warp_wait(&drain[1], 0, drain_limit(a), nullptr);
  } else if (warp >= warp0 && warp < warp0 + warps) {
    // ------------------------------------------------------------- softmax
    const int r = (warp - warp0) * 32 + lane;  // row of the tile, in TMEM lane 32 * warp + lane
    const int node = min(row0 + r, a.T * R - 1) / R;
    const uint64_t my_sees = sees[node];  // 0 for a node that is not there
    const int64_t pos = static_cast<int64_t>(plan.len) + depth[node];
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t o_addr = lane_addr + COL_O;
    const float c2 = a.scale_log2;
    const uint64_t c2x2 = pack_f2(c2, c2);
    // A lane without a row, or with the row of a node that is not there, has no
    // say in when the warp moves its maxima: the products read shared memory
    // behind Q for the one, a q that may be anything for the other, and a present
    // row's roundings must not depend on either. No logit exceeds infinity.
    float m_run = my_sees != 0 && r < rows ? LOWEST : INFINITY, l_run = 0.f;  // base-2 units
    int bnd_cnt = 0;
    bool ok = nsub > 0;
    for (int u = 0; ok && u < nsub; ++u) {
      const int hh = u & 1;
      const int k0 = k_begin + u * SUB;
      const uint32_t s_addr = lane_addr + COL_S + SUB * hh;
      const uint32_t cls = tile_classes<SUB>(my_cut, G, plan.len, deepest, k0, lane);
      const bool drafts = k0 + SUB > plan.len;
      if (cls >> 8) {
        int64_t prev = -1;
        int32_t W;
        uint32_t groups;
        while (next_boundary_class(a.cut, cls >> 8, prev, &W, &groups)) {
          // keys within the window: dist = pos - key position <= W
          const int64_t first = pos - W - k0;  // first column of the context inside
          uint64_t keep = first <= 0 ? ~0ull : first >= 64 ? 0ull : ~0ull << first;
          if (drafts) {
            const int c0 = max(plan.len - k0, 0);  // first drafted column
            const uint64_t drafted = ~0ull << c0;  // c0 < 64 here
            keep &= ~drafted;
            if (W >= deepest) {  // no two nodes are further apart
              keep |= drafted;
            } else {
              const int c1 = min(plan.total - k0, 64);
#pragma unroll 1
              for (int c = c0; c < c1; ++c)
                if (pos - (plan.len + depth[k0 + c - plan.len]) <= W) keep |= 1ull << c;
            }
          }
          ok = warp_wait(bnd_ready, bnd_cnt & 1, lim, abort_flag);
          if (!ok) break;
          tc_fence_after();
          uint32_t su[64];
          tmem_ld64(s_addr, su);
          keep_columns(su, keep, 0u);
          tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&su[0]));
          tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&su[32]));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bnd_done);
          ++bnd_cnt;
          prev = W;
        }
        if (!ok) break;
      }
      if (!warp_wait(&s_ready[hh], (u >> 1) & 1, lim, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t su[64];
      load_half(s_addr, cls != 0, su);
      if (drafts) {
        // context columns, then the bits of the nodes this row sees
        const int c0 = plan.len - k0;  // column of node 0
        const uint64_t ctx = c0 <= 0 ? 0ull : (1ull << c0) - 1;  // c0 < 64 here
        const uint64_t own = c0 >= 0 ? my_sees << c0 : c0 > -64 ? my_sees >> -c0 : 0ull;
        keep_columns(su, ctx | own, 0xff800000u);
      }
      const float m_half = half_max(su) * c2;
      if (__any_sync(FULL, m_half > m_run + RESCALE_THRESHOLD)) {
        const float m_new = fmaxf(m_run, m_half);
        if (u > 0) {
          const float alpha = fast_exp2(m_run - m_new);
          if (!warp_wait(&o_ready[hh ^ 1], ((u - 1) >> 1) & 1, lim, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          scale_cols_f32(o_addr, D / 32, alpha);
          l_run *= alpha;
        }
        m_run = m_new;
      }
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      exp_half<false>(su, c2x2, m_run, acc, s_addr);
      float s0, s1, s2, s3, s4, s5, s6, s7;
      unpack_f2(acc[0], s0, s1);
      unpack_f2(acc[1], s2, s3);
      unpack_f2(acc[2], s4, s5);
      unpack_f2(acc[3], s6, s7);
      l_run += ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
      tmem_wait_st();
      if (k0 + SUB > plan.total) {
        // rows of V behind the last key: unused slots may hold anything
        if (!warp_wait(&v_full[u % VST], (u / VST) & 1, lim, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t *v = smem + L.v_off + (u % VST) * STAGE;
        const int first = plan.total - k0;
        for (int e = r; e < (SUB - first) * (D / 8); e += warps * 32) {
          // 16-byte piece p of row rr; the swizzle stays within a row's 128 bytes
          const int rr = first + e / (D / 8), p = e % (D / 8), i = rr / box;
          *reinterpret_cast<uint4 *>(v + i * box * D * 2 + (p / 8) * box * 128 + (rr - i * box) * 128 + (p % 8) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_shared();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[hh]);
    }
    const int row = row0 + r;
    const bool mine = r < rows;
    const bool there = plan.ok && row / R < plan.n;
    const int64_t part = ((static_cast<int64_t>(b) * cg.Hkv + hk) * (a.T * R) + row) * a.nsplit + split;
    const bool done = ok && warp_wait(o_final, 0, lim, abort_flag);
    if (done) {
      tc_fence_after();
      const float inv_l = l_run != 0.f ? 1.f / l_run : 0.f;
      // A partial row goes through shared memory (the rings and Q have been
      // read) and leaves as one bulk copy; few instructions, since this code
      // runs once and has to be fetched. 4 x 1152 keys 22.4 -> 21.2 us, 16 x 16K
      // to 32K keys 265 -> 262 us (64 rows) against 16-byte stores from here.
      uint8_t *stage = smem + r * Layout<D>::PITCH;
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        uint32_t ov[32];
        tmem_ld32(o_addr + 32 * c4, ov);
        tmem_wait_ld(ov);
        if (a.nsplit > 1) {
          float4 *dst = reinterpret_cast<float4 *>(stage + 128 * c4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(__uint_as_float(ov[4 * k]) * inv_l, __uint_as_float(ov[4 * k + 1]) * inv_l,
                                 __uint_as_float(ov[4 * k + 2]) * inv_l, __uint_as_float(ov[4 * k + 3]) * inv_l);
        } else if (mine) {
          uint4 *dst = reinterpret_cast<uint4 *>(a.o + out_row(a, b, hk, R, row) * D + 32 * c4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (there)
              w = make_uint4(pack_bf16x2(__uint_as_float(ov[8 * k]) * inv_l, __uint_as_float(ov[8 * k + 1]) * inv_l),
                             pack_bf16x2(__uint_as_float(ov[8 * k + 2]) * inv_l, __uint_as_float(ov[8 * k + 3]) * inv_l),
                             pack_bf16x2(__uint_as_float(ov[8 * k + 4]) * inv_l, __uint_as_float(ov[8 * k + 5]) * inv_l),
                             pack_bf16x2(__uint_as_float(ov[8 * k + 6]) * inv_l, __uint_as_float(ov[8 * k + 7]) * inv_l));
            dst[k] = w;
          }
        }
      }
      if (a.nsplit > 1) {
        fence_async_shared();
        if (mine) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.o_part + part * D), "r"(smem_u32(stage)), "r"(D * 4)
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
        }
      }
    } else if (nsub > 0) {
      *abort_flag = 1;
    }
    if (mine) {
      const float lse2 = m_run + __log2f(l_run);  // -inf where no key of this range is visible
      // not done: no keys at all (every row is empty), or a bad sequence, page or wait: NaN rows
      const bool spoilt = !done && (bad || nsub > 0);
      if (a.nsplit > 1) {
        if (!done && !spoilt)
          for (int k = 0; k < D; ++k) a.o_part[part * D + k] = 0.f;
        a.lse_part[part] = spoilt ? INFINITY : done ? lse2 : -INFINITY;
      } else {
        if (!done) {
          const uint32_t w = spoilt ? 0x7FC07FC0u : 0u;
          uint4 *dst = reinterpret_cast<uint4 *>(a.o + out_row(a, b, hk, R, row) * D);
          for (int k = 0; k < D / 8; ++k) dst[k] = make_uint4(w, w, w, w);
        }
        float *lse = out_lse(a, b, hk, R, row);
        if (lse != nullptr)
          *lse = spoilt ? __int_as_float(0x7FC00000) : done && there ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == QK_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Merges the splits, one warp per row.
constexpr int COMBINE_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(COMBINE_WARPS * 32) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;
  cudaGridDependencySynchronize();
  const int R = a.Hq / a.cache.Hkv, rows = a.T * R;
  const int row = static_cast<int>(blockIdx.x) * COMBINE_WARPS + static_cast<int>(threadIdx.x) / 32, hk = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  const int64_t id = (static_cast<int64_t>(b) * a.cache.Hkv + hk) * rows + row;
  const Plan plan = sequence_plan<SUB>(a, b);
  const int splits = sequence_splits(a, plan.tiles);
  float acc[E], sum = 1.f, M = 0.f;
  bool spoilt = !plan.ok;
  const bool there = plan.ok && row / R < plan.n;
  if (there) {
    merge_row<D>(a, splits, [&](int i) { return id * a.nsplit + i; }, acc, sum, M);
    spoilt = M == INFINITY;
  }
  __nv_bfloat16 *o = a.o + out_row(a, b, hk, R, row) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = spoilt ? __int_as_float(0x7fc00000) : there ? acc[e] / sum : 0.f;
    const float y = spoilt ? __int_as_float(0x7fc00000) : there ? acc[e + 1] / sum : 0.f;
    *reinterpret_cast<uint32_t *>(o + e) = pack_bf16x2(x, y);
  }
  float *lse = out_lse(a, b, hk, R, row);
  if (lane == 0 && lse != nullptr)
    *lse = spoilt ? __int_as_float(0x7fc00000) : there ? (M + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool KGM>
cudaError_t launch(const TreeMaps &tm, TreeArgs a, cudaStream_t stream) {
  // as many stages as let two CTAs share an SM, one more of K than of V where
  // the number is odd
  const int rows = a.tile_nodes * (a.Hq / a.cache.Hkv);
  const int stages = min(2 * TREE_MAX_STAGES, (SMEM_PER_CTA - static_cast<int>(Layout<D>(0, 0, rows).bytes())) / static_cast<int>(Layout<D>::STAGE));
  a.v_stages = stages / 2;
  a.k_stages = stages - a.v_stages;
  const int smem = static_cast<int>(Layout<D>(a.k_stages, a.v_stages, rows).bytes());
  const cudaError_t e = allow_shared_memory<tree_kernel<D, KGM>>(SMEM_PER_CTA);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.row_tiles * a.nsplit, a.cache.Hkv, a.B);
  return launch_after(tree_kernel<D, KGM>, grid, NTHREADS, smem, stream, 1, tm, a);
}

template <int D>
cudaError_t combine(const TreeArgs &a, cudaStream_t stream) {
  const dim3 grid((a.T * (a.Hq / a.cache.Hkv) + COMBINE_WARPS - 1) / COMBINE_WARPS, a.cache.Hkv, a.B);
  return launch_after(tree_combine_kernel<D>, grid, COMBINE_WARPS * 32, 0, stream, 1, a);
}

}  // namespace

cudaError_t launch_tree(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream) {
  if (tree_few_rows(a.T, a.Hq / a.cache.Hkv)) return launch_tree_few(tm, a, stream);
  cudaError_t e;
  if (a.cache.D == 128)
    e = a.cache.k_group_major ? launch<128, true>(tm, a, stream) : launch<128, false>(tm, a, stream);
  else
    e = a.cache.k_group_major ? launch<64, true>(tm, a, stream) : launch<64, false>(tm, a, stream);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return a.cache.D == 128 ? combine<128>(a, stream) : combine<64>(a, stream);
}

}  // namespace wp
