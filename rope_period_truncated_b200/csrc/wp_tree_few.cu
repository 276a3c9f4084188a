// Tree attention for few rows (nodes x query heads of a KV head <= 32), with
// the products turned round: S^T = K Q^T and O^T = V^T P^T.
//
// The mathematics is that of wp_tree.cu. With few rows an M = 128 tile of
// query rows would be mostly padding, and its exponentials would sit in one
// warp, 64 per thread and sub-tile. Here the 128 rows of a product are keys
// (S^T) or head dims (O^T) and the query rows are its N = 32: the tensor
// work shrinks with the rows, a softmax thread has one key and all rows, and
// the four warps share a tile's exponentials evenly.
//
// What bounds it: HBM over long caches (16 sequences of 16K to 32K keys, 32 rows,
// pages of 64 keys: 211 us back to back, 5.9 TB/s, 218 us a call among calls on
// other inputs; K in rows, whose 64-dim chunks are read whole, 258), the issue of
// the copies from one lane where pages of group-major K are small (32 keys 222
// us, 16 keys 342), latency over short ones (4 sequences of 2.5K to 4K keys: 26
// us; one of 200 keys, a CTA per KV head: 9, with 8 heads of 128 11). One
// sequence of 128K keys, 32 rows: 81 us back to back where its bytes take 63; some
// 10 of the 18 between are what a short call takes, the rest was not taken apart.
//
// One CTA per SM. All (sequence, KV head) units lie end to end as a line of
// 128-key tiles, cut evenly among the CTAs, whatever the lengths: a CTA walks
// over its stretch in segments (what of one unit falls into it), and its loads
// run ahead across them. Warps 8 and 9 fetch K, and Q and V, warp 10 issues S^T
// (M = 128 keys, N = rows, one K = 16 product per live group), warps 0-3 turn it
// into P^T for the even tiles and warps 4-7 for the odd ones (bf16, since V is: 2^-8
// of each weight, as in the package's prefill; the sums take it unrounded; in shared
// memory: B of the second product, rows contiguous), warp 11 issues O^T (M = 128
// dims, V read as it lies, MN-major). Even and odd tiles have maxima, sums and
// an O^T of their own: a softmax warp alone on its scheduler waits for its own
// latencies, about 1900 cycles a tile; two of them overlap. A segment that is a
// whole unit writes its rows; the others, at most the first and the last of a
// CTA, write O (fp32) and LSE to the workspace, and a second kernel merges
// them.
//
// The running maxima are one per row and stream, kept in shared memory,
// and stay as they are while no logit exceeds them by more than 2^8: a tile
// then needs only one vote. Otherwise (the first tile, and rarely later) the
// exact maxima are formed with warp reductions and O^T and the sums rescaled.
// Sums are kept per thread (its keys') and reduced once, at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_tree.cuh"

namespace wp {
namespace {

constexpr int TILE = 128;
constexpr int NR = TREE_FEW_ROWS;  // query rows of a product
constexpr int FEW_THREADS = 384;
constexpr int FEW_K_WARP = 8, FEW_V_WARP = 9, FEW_QK_WARP = 10, FEW_PV_WARP = 11;
constexpr int SMEM_CAP = 232448;  // dynamic shared memory of one CTA
constexpr uint32_t GROUP = TILE * 32;   // 128 keys x 16 bf16 (group-major K)
constexpr uint32_t CHUNK = TILE * 128;  // 128 keys x 64 bf16 (K in rows)
constexpr int PAGE_FLAGS = 16;  // of segments: V is loaded up to TREE_MAX_STAGES tiles ahead of the softmax
constexpr int TABLES = 4;  // of segments in flight: S runs at most two tiles ahead of the softmax
constexpr uint32_t NUM_BARS = 2 + 4 * TREE_MAX_STAGES + 4 * 2 + TABLES + 7;

// The nodes of one segment's sequence.
struct NodeTable {
  uint32_t seen_by[64];  // per node: the rows that see it
  uint32_t upto[64];     // per depth: the rows no deeper
  int32_t depth[64];
  int deepest, bad, pad[2];
};

// Shared memory: K ring, V ring, two P tiles, Q (NR rows per group), then
// the small tables and the barriers.
template <int D>
struct FewLayout {
  static constexpr int G = D / 16;
  static constexpr uint32_t STAGE = TILE * D * 2;
  static constexpr uint32_t P_TILE = TILE * NR * 2;
  static constexpr uint32_t Q_TILE = NR * 32;
  static constexpr uint32_t Q_BYTES = G * Q_TILE;
  // node tables, scratch, and per row and stream: -max, a factor, 4 warps' values
  static constexpr uint32_t SMALL = TABLES * sizeof(NodeTable) + 64 * 8 + 64 * 4 + 2 * NR * 4 * 6;
  static constexpr uint32_t FIXED = 2 * P_TILE + Q_BYTES + SMALL + NUM_BARS * 8 + 32 + PAGE_FLAGS * 4 + 1024;  // + alignment
  uint32_t v_off, p_off, q_off, small_off, bar_off, misc_off;
  __host__ __device__ FewLayout(int kst, int vst) {
    v_off = kst * STAGE;
    p_off = v_off + vst * STAGE;
    q_off = p_off + 2 * P_TILE;
    small_off = q_off + Q_BYTES;
    bar_off = small_off + SMALL;
    misc_off = bar_off + NUM_BARS * 8;  // abort flag, TMEM base, start of the stretch; from 32: page flags
  }
};

// The line of tiles. Sequence b has plan.tiles tiles per KV head; prefix[b] is
// the sum over the sequences before it. CTA c of G takes the tiles [cut(c),
// cut(c + 1)).
// (fewer than 2^55 tiles: the products stay within 64 bits.)
__device__ __forceinline__ int64_t cut(int64_t tiles, int c, int G) { return tiles * c / G; }
// The CTA of tile x: the largest c with cut(c) <= x.
__device__ __forceinline__ int cta_of(int64_t tiles, int64_t x, int G) {
  return static_cast<int>(((x + 1) * G - 1) / tiles);
}

// A sequence with no nodes has nothing to attend; one with bad lengths is left
// to the merging kernel.
__device__ __forceinline__ Plan few_plan(const TreeArgs &a, int b) {
  Plan p = sequence_plan<TILE>(a, b);
  if (!p.ok || p.n == 0) p.tiles = 0;
  return p;
}

struct Segment {
  Plan plan;
  int b, hk, k_begin, tiles, index;  // index: count of the CTA's segments
  int slot;                          // of its partial result; -1: the whole unit
};

// One warp's walk over the CTA's segments.
struct Walk {
  int64_t x, x1;
  int b, hk, t, cta, index;
  bool first;
  Plan plan;
  __device__ __forceinline__ bool next(const TreeArgs &a, Segment &s) {
    if (x >= x1) return false;
    while (t >= plan.tiles) {  // on to the next unit that has tiles
      t = 0;
      if (plan.tiles > 0 && ++hk < a.cache.Hkv) break;
      hk = 0;
      plan = few_plan(a, ++b);
    }
    const int64_t left = x1 - x;
    s.plan = plan;
    s.b = b;
    s.hk = hk;
    s.tiles = static_cast<int>(left < plan.tiles - t ? left : plan.tiles - t);
    s.k_begin = t * TILE;
    s.index = index++;
    s.slot = t == 0 && s.tiles == plan.tiles ? -1 : 2 * cta + (first ? 0 : 1);
    first = false;
    t += s.tiles;
    x += s.tiles;
    return true;
  }
};

// TMEM -> registers, 32 lanes x 32 bit, 16 consecutive columns, and the wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 TMEM columns of this warp's lanes.
__device__ __forceinline__ void load_rows(uint32_t taddr, uint32_t (&r)[NR]) {
  tmem_ld32(taddr, r);
  tmem_wait_ld(r);
}
__device__ __forceinline__ void store_rows(uint32_t taddr, const uint32_t (&r)[NR]) {
  tmem_st32(taddr, r);
  tmem_wait_st();
}

// Columns whose bit is clear become `fill`.
__device__ __forceinline__ void keep_rows(uint32_t (&r)[NR], uint32_t bits, uint32_t fill) {
#pragma unroll
  for (int c = 0; c < NR; ++c)
    if (!(bits & (1u << c))) r[c] = fill;
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

// Barrier `id` over `n` threads of the CTA (whole warps).
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// Floats as integers of the same order (and back).
__device__ __forceinline__ int ordered(uint32_t x) {
  const int i = static_cast<int>(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}

template <int D, bool KGM>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    tree_few_kernel(const __grid_constant__ TreeMaps tm, const __grid_constant__ TreeArgs a) {
  using L = FewLayout<D>;
  constexpr int G = D / 16;
  constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, NR, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, NR, true, true);
  constexpr uint32_t TMEM_COLS = 4 * NR;  // S^T and O^T of both streams
  constexpr uint32_t COL_O = 2 * NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const L lay(a.k_stages, a.v_stages);
  NodeTable *tables = reinterpret_cast<NodeTable *>(smem + lay.small_off);
  uint64_t *sees = reinterpret_cast<uint64_t *>(tables + TABLES);  // per node: the nodes it sees (scratch of the S^T issuer)
  int32_t *jump = reinterpret_cast<int32_t *>(sees + 64);
  float *all_negm = reinterpret_cast<float *>(jump + 64);  // [2][NR] minus the running maxima
  float *all_alpha = all_negm + 2 * NR;                    // [2][NR] rescaling, at the end the streams' factors
  float *all_part = all_alpha + 2 * NR;                    // [2][4][NR] of the warps
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bar_off);
  uint64_t *q_full = bars, *q_empty = q_full + 1, *k_full = q_empty + 1, *k_empty = k_full + TREE_MAX_STAGES,
           *v_full = k_empty + TREE_MAX_STAGES, *v_empty = v_full + TREE_MAX_STAGES, *s_ready = v_empty + TREE_MAX_STAGES,
           *s_free = s_ready + 2, *p_ready = s_free + 2, *o_ready = p_ready + 2, *t_ready = o_ready + 2,
           *o_final = t_ready + TABLES, *bnd_ready = o_final + 1, *bnd_done = bnd_ready + 2, *drain = bnd_done + 2;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + lay.misc_off);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + lay.misc_off + 4);
  volatile int *bad_pages = reinterpret_cast<volatile int *>(smem + lay.misc_off + 32);  // set by the V producer
  int *start = reinterpret_cast<int *>(smem + lay.misc_off + 8);                         // sequence, KV head, tile

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheGeom &cg = a.cache;
  const int R = a.Hq / cg.Hkv, rows = a.T * R;
  const long long lim = a.wait_limit;
  const int my_cut = lane < G ? a.cut[lane] : 0;
  if (threadIdx.x == FEW_K_WARP * 32) {
    tma_prefetch_desc(&tm.k[0]);
    tma_prefetch_desc(&tm.k[1]);
    tma_prefetch_desc(&tm.k[2]);
    tma_prefetch_desc(&tm.v);
    tma_prefetch_desc(&tm.q);
  }

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < TABLES; ++s) mbar_init(&t_ready[s], 1);
    for (int s = 0; s < a.k_stages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < a.v_stages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_ready[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&p_ready[s], 4);
      mbar_init(&o_ready[s], 1);
      mbar_init(&bnd_ready[s], 1);
      mbar_init(&bnd_done[s], 4);
      mbar_init(&drain[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_final, 1);
    fence_barrier_init();
  }
  cudaGridDependencySynchronize();  // nothing of global memory before it, nor of TMEM, which the kernel before may hold
  if (warp == FEW_QK_WARP) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  // rows of Q beyond the last one, as zeros (their columns of S^T take part in the votes)
  const int pad = (NR - rows) * 2;  // 16-byte pieces per group
  for (int e = threadIdx.x; e < pad * G; e += FEW_THREADS)
    *reinterpret_cast<uint4 *>(smem + lay.q_off + (e / pad) * L::Q_TILE + rows * 32 + (e % pad) * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_async_shared();

  // The line of tiles: each thread takes a run of sequences; the sums before
  // them by a scan over the block. CTA 0 writes them down for the merge.
  Walk walk;
  walk.cta = blockIdx.x;
  walk.index = 0;
  walk.first = true;
  if (a.prefix == nullptr) {
    // a unit of its own
    walk.b = blockIdx.x / cg.Hkv;
    walk.hk = blockIdx.x - walk.b * cg.Hkv;
    walk.t = 0;
    walk.plan = few_plan(a, walk.b);
    walk.x = 0;
    walk.x1 = walk.plan.tiles;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (walk.x1 == 0)  // nothing to attend: zeros, or NaN where the lengths are bad
      for (int e = threadIdx.x; e < rows * D; e += FEW_THREADS) {
        const int r = e / D;
        a.o[out_row(a, walk.b, walk.hk, R, r) * D + e % D] = __float2bfloat16_rn(walk.plan.ok ? 0.f : __int_as_float(0x7FC00000));
        float *lse = out_lse(a, walk.b, walk.hk, R, r);
        if (e % D == 0 && lse != nullptr) *lse = walk.plan.ok ? -INFINITY : __int_as_float(0x7FC00000);
      }
  } else {
    const int run = (a.B + FEW_THREADS - 1) / FEW_THREADS, b0 = min(static_cast<int>(threadIdx.x) * run, a.B), b1 = min(b0 + run, a.B);
    int64_t mine = 0;
    int own = 0;  // tiles of the last one
    for (int b = b0; b < b1; ++b) mine += own = few_plan(a, b).tiles;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, inc, o);
      if (lane >= o) inc += y;
    }
    int64_t *sums = reinterpret_cast<int64_t *>(all_part);  // of the warps
    if (lane == 31) sums[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t before = inc - mine, total = 0;
    #pragma unroll
    for (int w = 0; w < FEW_THREADS / 32; ++w) {
      before += w < warp ? sums[w] : 0;
      total += sums[w];
    }
    const int64_t tiles = total * cg.Hkv;
    walk.x = cut(tiles, blockIdx.x, gridDim.x);
    walk.x1 = cut(tiles, blockIdx.x + 1, gridDim.x);
    for (int b = b0; b < b1; ++b) {
      const int t = run == 1 ? own : few_plan(a, b).tiles;
      if (blockIdx.x == 0) a.prefix[b] = before;
      const int64_t at = walk.x - before * cg.Hkv;  // the stretch's start within sequence b
      if (at >= 0 && at < static_cast<int64_t>(t) * cg.Hkv) {
        start[0] = b;
        int h = 0;
        int64_t rest = at;
        for (; rest >= t; rest -= t) ++h;
        start[1] = h;
        start[2] = static_cast<int>(rest);
      }
      before += t;
    }
    if (blockIdx.x == 0 && threadIdx.x == FEW_THREADS - 1) a.prefix[a.B] = total;
    __syncthreads();
    if (walk.x < walk.x1) {
      walk.b = start[0];
      walk.hk = start[1];
      walk.t = start[2];
      walk.plan = few_plan(a, walk.b);
    }
  }
  const uint32_t tmem = *tmem_slot;
  const int box = a.box_rows, boxes = TILE / box;
  Segment seg;

  if (warp == FEW_K_WARP) {
    // ------------------------------------------------------- producer of K
    // Lane i looks up box i % boxes one tile ahead.
    const bool leader = elect_one();
    Ring ring;
    int issued = 0;
    bool ok = true;
    while (ok && walk.next(a, seg)) {
      const int end = min(seg.k_begin + seg.tiles * TILE, seg.plan.total);
      const int key0 = seg.k_begin + (lane & (boxes - 1)) * box;
      Place here = place_of(cg, seg.b, key0, end);
#pragma unroll 1
      for (int u = 0; u < seg.tiles; ++u) {
        const Place next = place_of(cg, seg.b, key0 + (u + 1) * TILE, end);
        uint64_t *full = &k_full[ring.slot];
        uint8_t *dst = smem + ring.slot * L::STAGE;
        uint32_t need = live_groups<TILE>(my_cut, G, seg.plan.len, seg.k_begin + u * TILE, lane);
        if (!KGM) need = ((need & 0xfu) ? 1u : 0u) | ((need >> 4) ? 2u : 0u);  // 64-dim chunks
        if (issued >= a.k_stages && !warp_wait_idle(&k_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        const int have = __popc(__ballot_sync(FULL, lane < boxes && key0 + u * TILE < end));
        if (leader) mbar_arrive_expect_tx(full, have * __popc(need) * box * (KGM ? 32u : 128u));
        issue_k<D, KGM, TILE>(tm, here, have, need, box, seg.hk, dst, full, leader);
        ++issued;
        ring.next(a.k_stages);
        here = next;
      }
    }
    // no bulk copy may still be in flight when this CTA's shared memory goes
    for (int s = 0; s < a.k_stages && s < issued; ++s) {
      const int last = s + ((issued - 1 - s) / a.k_stages) * a.k_stages;
      warp_wait_idle(&k_full[s], (last / a.k_stages) & 1, drain_limit(a), nullptr);
    }
  } else if (warp == FEW_V_WARP) {
    // -------------------------------------------------- producer of Q and V
    // It also looks at the pages: an entry outside the pool spoils the segment
    // (TMA reads nothing there and gives zeros).
    const bool leader = elect_one();
    Ring ring;
    int issued = 0, q_issued = 0;
    bool ok = true;
    while (ok && walk.next(a, seg)) {
      const int end = min(seg.k_begin + seg.tiles * TILE, seg.plan.total);
      const int key0 = seg.k_begin + (lane & (boxes - 1)) * box;
      Place here = place_of(cg, seg.b, key0, end);
      // one buffer: after the last S^T product of the segment before
      if (seg.index >= 1 && !warp_wait_idle(q_empty, (seg.index - 1) & 1, lim, abort_flag)) break;
      if (leader) {
        mbar_arrive_expect_tx(q_full, G * 32u * rows);
#pragma unroll
        for (int g = 0; g < G; ++g)
          tma_load_4d(smem + lay.q_off + g * L::Q_TILE, &tm.q, q_full, 16 * g, seg.hk * R, 0, seg.b);
      }
      ++q_issued;
      if (leader) bad_pages[seg.index % PAGE_FLAGS] = 0;
      __syncwarp();
#pragma unroll 1
      for (int u = 0; u < seg.tiles; ++u) {
        const Place next = place_of(cg, seg.b, key0 + (u + 1) * TILE, end);
        uint64_t *full = &v_full[ring.slot];
        if (issued >= a.v_stages && !warp_wait_idle(&v_empty[ring.slot], ring.round ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        const bool mine = lane < boxes && key0 + u * TILE < end;
        const int have = __popc(__ballot_sync(FULL, mine));
        const bool bad = __any_sync(FULL, mine && (here.page < 0 || here.page >= cg.n_pages));
        if (leader) {
          if (bad) bad_pages[seg.index % PAGE_FLAGS] = 1;
          mbar_arrive_expect_tx(full, have * box * D * 2u);
        }
#pragma unroll 1
        for (int i = 0; i < have; ++i) {
          const int page = __shfl_sync(FULL, here.page, i), row = __shfl_sync(FULL, here.row, i);
          if (leader) tma_load_5d(smem + lay.v_off + ring.slot * L::STAGE + i * box * D * 2, &tm.v, full, 0, row, 0, seg.hk, page);
          __syncwarp();
        }
        ++issued;
        ring.next(a.v_stages);
        here = next;
      }
    }
    if (q_issued > 0) warp_wait_idle(q_full, (q_issued - 1) & 1, drain_limit(a), nullptr);
    for (int s = 0; s < a.v_stages && s < issued; ++s) {
      const int last = s + ((issued - 1 - s) / a.v_stages) * a.v_stages;
      warp_wait_idle(&v_full[s], (last / a.v_stages) & 1, drain_limit(a), nullptr);
    }
  } else if (warp == FEW_QK_WARP) {
    // ------------------------------------------------------- issuer of S^T
    const bool leader = elect_one();
    const uint64_t q_desc = smem_desc(smem_u32(smem + lay.q_off), 16, 256, SMEM_SWIZZLE_32B);
    const uint64_t k_desc = KGM ? smem_desc(smem_u32(smem), 16, 256, SMEM_SWIZZLE_32B)
                                : smem_desc(smem_u32(smem), 16, 1024, SMEM_SWIZZLE_128B);
    Ring ring;
    int bnd_cnt[2] = {0, 0}, it = 0;  // it: tiles of all segments
    bool ok = true;
    while (ok && walk.next(a, seg)) {
      const auto issue_groups = [&](uint32_t s_col, uint64_t kst_desc, uint32_t groups, uint32_t acc) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (groups & (1u << g)) {
            // K in rows: group g is 32 bytes into the 128-byte rows of chunk g / 4
            const uint32_t koff = KGM ? g * GROUP : (g / 4) * CHUNK + (g % 4) * 32;
            umma_ss(s_col, kst_desc + (koff >> 4), q_desc + g * (L::Q_TILE >> 4), IDESC_QK, acc);
            acc = 1;
          }
      };
      // The nodes' table. Tile it - 2 has been taken by its softmax warps, and
      // they are past tile it - 4 then; tile it - 3 belongs to the others. So
      // three segments back is the oldest table in use.
      ok = it < 2 || warp_wait(&s_free[it & 1], ((it >> 1) - 1) & 1, lim, abort_flag);
      if (!ok) break;
      NodeTable &tab = tables[seg.index % TABLES];
      const bool bad = node_masks(a, seg.plan, seg.b, sees, tab.depth, jump, &tab.deepest);
      __syncwarp();
      const int deepest = tab.deepest;
      {
        const uint64_t mine = lane < rows ? sees[lane / R] : 0ull;
        const int my_depth = lane < rows ? tab.depth[lane / R] : 64;
#pragma unroll 1
        for (int u = 0; u < seg.plan.n; ++u) {
          const uint32_t set = __ballot_sync(FULL, (mine >> u) & 1);
          if (lane == 0) tab.seen_by[u] = set;
        }
#pragma unroll 1
        for (int u = 0; u <= deepest; ++u) {
          const uint32_t set = __ballot_sync(FULL, my_depth <= u);
          if (lane == 0) tab.upto[u] = set;
        }
        if (lane == 0) tab.bad = bad;
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_ready[seg.index % TABLES]);
      }
      ok = warp_wait(q_full, seg.index & 1, lim, abort_flag);
      if (ok && seg.plan.n < a.T) {
        // The q of nodes that are not there may be anything, and its logits would
        // take part in the votes on the maxima: zeros instead.
        const int first = seg.plan.n * R, pieces = (rows - first) * 2;  // 16-byte pieces per group
        for (int e = lane; e < pieces * G; e += 32)
          *reinterpret_cast<uint4 *>(smem + lay.q_off + (e / pieces) * L::Q_TILE + first * 32 + (e % pieces) * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_shared();
        __syncwarp();
      }
      for (int u = 0; ok && u < seg.tiles; ++u, ++it) {
        const int hh = it & 1;
        const uint32_t cls = tile_classes<TILE>(my_cut, G, seg.plan.len, deepest, seg.k_begin + u * TILE, lane);
        const uint32_t s_col = tmem + NR * hh;
        const uint64_t kst_desc = k_desc + ((ring.slot * L::STAGE) >> 4);
        ok = warp_wait(&k_full[ring.slot], ring.round, lim, abort_flag) &&
             (it < 2 || u == 0 || warp_wait(&s_free[hh], ((it >> 1) - 1) & 1, lim, abort_flag));
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
              umma_commit(&bnd_ready[hh]);
            }
            acc = 1;
            __syncwarp();
            const int round = hh ? bnd_cnt[1]++ : bnd_cnt[0]++;
            ok = warp_wait(&bnd_done[hh], round & 1, lim, abort_flag);
            tc_fence_after();
            prev = W;
          }
          if (!ok) break;
        }
        if (leader) {
          issue_groups(s_col, kst_desc, cls & 0xffu, acc);
          umma_commit(&s_ready[hh]);
          umma_commit(&k_empty[ring.slot]);
          if (u == seg.tiles - 1) umma_commit(q_empty);
        }
        __syncwarp();
        ring.next(a.k_stages);
      }
    }
    // every product must have finished before TMEM is given back
    if (leader) umma_commit(&drain[0]);
    __syncwarp();
    warp_wait(&drain[0], 0, drain_limit(a), nullptr);
  } else if (warp == FEW_PV_WARP) {
    // ------------------------------------------------------- issuer of O^T
    const bool leader = elect_one();
    // A = V^T: dims contiguous (MN-major); 8-key row groups 1024 B and 64-dim
    // chunks box * 128 B apart. At d = 64 there is one chunk, and the upper 64
    // rows of O^T repeat the lower ones. B = P^T: rows contiguous.
    const uint64_t v_desc = smem_desc(smem_u32(smem + lay.v_off), D == 128 ? box * 128 : 0, 1024, SMEM_SWIZZLE_128B);
    const uint64_t p_desc = smem_desc(smem_u32(smem + lay.p_off), 0, 8 * NR * 2, SMEM_SWIZZLE_64B);
    Ring ring;
    int it = 0;
    bool ok = true;
    while (ok && walk.next(a, seg)) {
      for (int u = 0; u < seg.tiles; ++u, ++it) {
        const int hh = it & 1;
        const uint64_t vst_desc = v_desc + ((ring.slot * L::STAGE) >> 4);
        const uint64_t pst_desc = p_desc + ((hh * L::P_TILE) >> 4);
        ok = warp_wait(&v_full[ring.slot], ring.round, lim, abort_flag) && warp_wait(&p_ready[hh], (it >> 1) & 1, lim, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll 2
          for (int kk = 0; kk < TILE / 16; ++kk)
            umma_ss(tmem + COL_O + NR * hh, vst_desc + v_step<D>(kk, box), pst_desc + kk * ((16 * NR * 2) >> 4), IDESC_PV,
                    (u > 1 || kk > 0) ? 1u : 0u);  // each stream's first tile of the segment starts O^T
          umma_commit(&o_ready[hh]);
          umma_commit(&v_empty[ring.slot]);
          if (u == seg.tiles - 1) umma_commit(o_final);
        }
        __syncwarp();
        ring.next(a.v_stages);
      }
    }
    if (leader) umma_commit(&drain[1]);
    __syncwarp();
    warp_wait(&drain[1], 0, drain_limit(a), nullptr);
  } else {
    // ------------------------------------------------------------- softmax
    // The four warps meet in a vote on every tile, so none leaves the loop by
    // itself: one whose wait gave up goes on to the vote and says so there.
    const int hh = warp / 4, w4 = warp % 4, st = threadIdx.x % 128;  // stream; warp and thread within it
    const int kt = w4 * 32 + lane;  // key of the tile == TMEM lane; head dim == lane of O^T
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t s_addr = lane_addr + NR * hh, o_addr = lane_addr + COL_O + NR * hh;
    const int bar = 2 + hh;  // the stream's named barrier; 1: both streams
    float *negm = all_negm + hh * NR, *alpha = all_alpha + hh * NR, *part4 = all_part + hh * 4 * NR;
    const float c2 = a.scale_log2;
    const uint64_t c2x2 = pack_f2(c2, c2);
    uint64_t l2[NR / 2];  // this thread's sums, two rows each
    int bnd_cnt = 0, it = 0;
    bool ok = true;
    Ring vr;  // the V stage of the tile
    while (walk.next(a, seg)) {
      const Plan &plan = seg.plan;
      if (st < NR) negm[st] = -LOWEST;
#pragma unroll
      for (int i = 0; i < NR / 2; ++i) l2[i] = 0ull;
      const NodeTable &tab = tables[seg.index % TABLES];
      ok = ok && warp_wait(&t_ready[seg.index % TABLES], (seg.index / TABLES) & 1, lim, abort_flag);
      named_sync(bar, 128);
      const int deepest = tab.deepest;
      bool fresh = true;  // no tile of this stream in the segment yet
      for (int u = 0; u < seg.tiles; ++u, ++it) {
        if ((it & 1) != hh) {
          vr.next(a.v_stages);
          continue;
        }
        const int k0 = seg.k_begin + u * TILE, key = k0 + kt;
        const uint32_t cls = tile_classes<TILE>(my_cut, G, plan.len, deepest, k0, lane);
        const bool drafts = k0 + TILE > plan.len;
        const bool context = key < plan.len, there = key < plan.total;
        if (cls >> 8) {
          const int64_t kpos = context || !there ? key : plan.len + tab.depth[key - plan.len];
          int64_t prev = -1;
          int32_t W;
          uint32_t groups;
          while (ok && next_boundary_class(a.cut, cls >> 8, prev, &W, &groups)) {
            // rows within the window: len + depth - kpos <= W
            const int64_t most = W + kpos - plan.len;
            const uint32_t keep = most < 0 ? 0u : tab.upto[static_cast<int>(min(most, static_cast<int64_t>(deepest)))];
            ok = warp_wait(&bnd_ready[hh], bnd_cnt & 1, lim, abort_flag);
            if (!ok) break;
            tc_fence_after();
            uint32_t su[NR];
            load_rows(s_addr, su);
            keep_rows(su, keep, 0u);
            store_rows(s_addr, su);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bnd_done[hh]);
            ++bnd_cnt;
            prev = W;
          }
        }
        ok = ok && warp_wait(&s_ready[hh], (it >> 1) & 1, lim, abort_flag);
        tc_fence_after();
        const uint32_t visible = !drafts || context ? ~0u : there ? tab.seen_by[key - plan.len] : 0u;
        uint8_t *p_row = smem + lay.p_off + hh * L::P_TILE + kt * (NR * 2);
        const int turn = (kt >> 1) & 3;  // the swizzle of the row's 16-byte pieces
        uint32_t su[NR];
        if (cls == 0) {  // no product: zeros, by the same load
#pragma unroll
          for (int c = 0; c < NR; ++c) su[c] = 0u;
          store_rows(s_addr, su);
        }
        load_rows(s_addr, su);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[hh]);
        if (drafts) keep_rows(su, visible, 0xff800000u);
        // Does any logit exceed its row's maximum by more than 2^8?
        float over = -INFINITY;
#pragma unroll
        for (int c = 0; c < NR; c += 4) {
          const float4 m4 = *reinterpret_cast<const float4 *>(negm + c);
          float x0, x1, x2, x3;
          unpack_f2(ffma2(pack_f2(__uint_as_float(su[c]), __uint_as_float(su[c + 1])), c2x2, pack_f2(m4.x, m4.y)), x0, x1);
          unpack_f2(ffma2(pack_f2(__uint_as_float(su[c + 2]), __uint_as_float(su[c + 3])), c2x2, pack_f2(m4.z, m4.w)), x2, x3);
          over = max3(over, max3(x0, x1, x2), x3);
        }
        if (named_any(bar, 128, over > RESCALE_THRESHOLD || !ok)) {
          if (named_any(bar, 128, !ok)) {
            ok = false;
            break;
          }
          int *warp_max = reinterpret_cast<int *>(part4) + w4 * NR;
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            const int mx = __reduce_max_sync(FULL, ordered(su[c]));
            if (lane == c) warp_max[c] = mx;
          }
          named_sync(bar, 128);
          if (st < NR) {
            const int *p = reinterpret_cast<const int *>(part4) + st;
            const int mx = max(max(p[0], p[NR]), max(p[2 * NR], p[3 * NR]));
            const float m_old = -negm[st];
            const float m_new = fmaxf(m_old, __int_as_float(ordered(static_cast<uint32_t>(mx))) * c2);
            alpha[st] = fast_exp2(m_old - m_new);
            negm[st] = -m_new;
          }
          named_sync(bar, 128);
          if (!fresh) {
#pragma unroll
            for (int c = 0; c < NR; c += 2) {
              float l0, l1;
              unpack_f2(l2[c / 2], l0, l1);
              l2[c / 2] = pack_f2(l0 * alpha[c], l1 * alpha[c + 1]);
            }
            ok = warp_wait(&o_ready[hh], ((it >> 1) - 1) & 1, lim, abort_flag);  // the stream's last P V
            tc_fence_after();
            uint32_t ov[NR];
            load_rows(o_addr, ov);
#pragma unroll
            for (int c = 0; c < NR; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha[c]);
            store_rows(o_addr, ov);
          }
        }
        // P^T of two tiles ago must have been read before its place is written again
        if (it >= 2) ok = warp_wait(&o_ready[hh], ((it >> 1) - 1) & 1, lim, abort_flag) && ok;
#pragma unroll
        for (int c = 0; c < NR; c += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = c + 2 * e;
            const uint64_t m2 = *reinterpret_cast<const uint64_t *>(negm + i);
            float x0, x1;
            unpack_f2(ffma2(pack_f2(__uint_as_float(su[i]), __uint_as_float(su[i + 1])), c2x2, m2), x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            l2[i / 2] = fadd2(l2[i / 2], pack_f2(p0, p1));
            w[e] = pack_bf16x2(p0, p1);
          }
          *reinterpret_cast<uint4 *>(p_row + (((c >> 3) ^ turn) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fresh = false;
        if (u == seg.tiles - 1) {
          // The last tile: V has landed (so have the V producer's words on the
          // pages), and its rows behind the last key become zeros: unused slots
          // may hold anything.
          ok = warp_wait(&v_full[vr.slot], vr.round, lim, abort_flag) && ok;
          if (!there) {
            const int i = kt / box;
            uint8_t *v = smem + lay.v_off + vr.slot * L::STAGE + i * box * D * 2 + (kt - i * box) * 128;
#pragma unroll
            for (int p = 0; p < D / 8; ++p)
              *reinterpret_cast<uint4 *>(v + (p / 8) * box * 128 + (p % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        vr.next(a.v_stages);
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&p_ready[hh]);
      }
      // ---------------------------------------------------------- epilogue
      // Both streams together: the sums of the rows over the four warps' keys,
      // the factors that bring the two accumulators to one maximum, and half
      // of the rows' results each.
      ok = ok && warp_wait(o_final, seg.index & 1, lim, abort_flag);
      float l[NR];
#pragma unroll
      for (int c = 0; c < NR; c += 2) unpack_f2(l2[c / 2], l[c], l[c + 1]);
      part4[w4 * NR + lane] = warp_sums(l);
      ok = !named_any(1, 256, !ok);  // all eight warps or none
      if (!ok) *abort_flag = 1;
      tc_fence_after();
      const bool spoilt = !ok || tab.bad || bad_pages[seg.index % PAGE_FLAGS];
      if (threadIdx.x < rows) {
        const int r = threadIdx.x, node = r / R;
        const auto sum4 = [&](const float *p) { return (p[r] + p[NR + r]) + (p[2 * NR + r] + p[3 * NR + r]); };
        const float m0 = -all_negm[r], m1 = -all_negm[NR + r], m = fmaxf(m0, m1);
        const float f0 = fast_exp2(m0 - m), f1 = fast_exp2(m1 - m);
        const float l0 = sum4(all_part), l1 = sum4(all_part + 4 * NR), l = l0 * f0 + l1 * f1;
        const bool live = node < plan.n;
        // a stream without a visible key adds nothing, whatever its accumulator
        // holds; rows of nodes that are not there are 0, chosen and not multiplied
        // to it: their q may be anything, and so may the factors be. A spoilt
        // segment's rows are NaN.
        const float inv = spoilt ? __int_as_float(0x7FC00000) : l != 0.f ? 1.f / l : 0.f;
        all_alpha[r] = !spoilt && (!live || l0 == 0.f) ? 0.f : f0 * inv;
        all_alpha[NR + r] = !spoilt && (!live || l1 == 0.f) ? 0.f : f1 * inv;
        if (seg.slot >= 0)
          a.lse_part[static_cast<int64_t>(seg.slot) * rows + r] = spoilt ? INFINITY : m + __log2f(l);
        else if (a.lse != nullptr)
          a.lse[(static_cast<int64_t>(seg.b) * a.Hq + seg.hk * R + r - node * R) * a.T + node] =
              spoilt ? __int_as_float(0x7FC00000) : live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
      named_sync(1, 256);
      // Lanes are head dims: 32 contiguous values of a row per warp.
      constexpr int HALF = NR / 2;
      uint32_t ov[2][HALF];
      const uint32_t half_addr = lane_addr + COL_O + hh * HALF;
      tmem_ld16(half_addr, ov[0]);
      tmem_ld16(half_addr + NR, ov[1]);
#pragma unroll
      for (int c = 0; c < HALF; ++c) {
        const float f0 = all_alpha[hh * HALF + c], f1 = all_alpha[NR + hh * HALF + c];
        ov[0][c] = __float_as_uint((f0 == 0.f ? 0.f : __uint_as_float(ov[0][c]) * f0) + (f1 == 0.f ? 0.f : __uint_as_float(ov[1][c]) * f1));
      }
      if (kt < D) {
        const int r0 = hh * HALF;
        if (seg.slot >= 0) {  // the rows follow one another
          float *dst = a.o_part + (static_cast<int64_t>(seg.slot) * rows + r0) * D + kt;
#pragma unroll
          for (int c = 0; c < HALF; ++c)
            if (r0 + c < rows) dst[c * D] = __uint_as_float(ov[0][c]);
        } else {  // a node's R heads do
          __nv_bfloat16 *dst = a.o + (static_cast<int64_t>(seg.b) * a.T * a.Hq + seg.hk * R) * D + kt;
          int node = r0 / R, head = r0 - node * R;
#pragma unroll
          for (int c = 0; c < HALF; ++c) {
            if (r0 + c < rows) dst[(static_cast<int64_t>(node) * a.Hq + head) * D] = __float2bfloat16_rn(__uint_as_float(ov[0][c]));
            if (++head == R) {
              head = 0;
              ++node;
            }
          }
        }
      }
      tc_fence_before();
      named_sync(1, 256);  // O^T, the sums and the factors are free again
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == FEW_QK_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Merges the partial results of the units that more than one CTA worked on, one
// warp per row. It also writes the rows that no CTA had: of sequences without
// nodes, or with bad lengths.
constexpr int MERGE_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(MERGE_WARPS * 32) tree_few_merge_kernel(const __grid_constant__ TreeArgs a, int G) {
  constexpr int E = D / 32;
  cudaGridDependencySynchronize();
  const int R = a.Hq / a.cache.Hkv, rows = a.T * R;
  const int row = static_cast<int>(blockIdx.x) * MERGE_WARPS + static_cast<int>(threadIdx.x) / 32, hk = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  const int64_t before = a.prefix[b], own = a.prefix[b + 1] - before, tiles = a.prefix[a.B] * a.cache.Hkv;
  float acc[E], sum = 1.f, M = 0.f;
  bool spoilt = false, live = false;
  if (own == 0) {
    spoilt = !sequence_plan<TILE>(a, b).ok;
  } else {
    const int64_t x0 = before * a.cache.Hkv + own * hk;
    const int c0 = cta_of(tiles, x0, G), c1 = cta_of(tiles, x0 + own - 1, G);
    if (c0 == c1) return;  // that CTA wrote the rows
    // CTA c's slot: its first segment, or for a unit that begins within c0 its last
    const int late = cut(tiles, c0, G) < x0 ? 1 : 0;
    live = row / R < (a.n_nodes != nullptr ? a.n_nodes[b] : a.T);
    // with fewer tiles than CTAs some of them have none: then each of the unit's tiles is a part
    const bool each = tiles < G;
    const auto slot_of = [&](int i) {
      const int c = each ? cta_of(tiles, x0 + i, G) : c0 + i;
      return static_cast<int64_t>(2 * c + (c == c0 ? late : 0)) * rows + row;
    };
    merge_row<D>(a, each ? static_cast<int>(own) : c1 - c0 + 1, slot_of, acc, sum, M);
    spoilt = M == INFINITY;
  }
  __nv_bfloat16 *o = a.o + out_row(a, b, hk, R, row) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = spoilt ? __int_as_float(0x7fc00000) : live ? acc[e] / sum : 0.f;
    const float y = spoilt ? __int_as_float(0x7fc00000) : live ? acc[e + 1] / sum : 0.f;
    *reinterpret_cast<uint32_t *>(o + e) = pack_bf16x2(x, y);
  }
  float *lse = out_lse(a, b, hk, R, row);
  if (lane == 0 && lse != nullptr)
    *lse = spoilt ? __int_as_float(0x7fc00000) : live ? (M + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool KGM>
cudaError_t launch(const TreeMaps &tm, TreeArgs a, cudaStream_t stream) {
  using L = FewLayout<D>;
  // as many stages as fit, one more of K than of V where the number is odd
  const int fit = (SMEM_CAP - static_cast<int>(L::FIXED)) / static_cast<int>(L::STAGE);
  const int stages = fit < 2 * TREE_MAX_STAGES ? fit : 2 * TREE_MAX_STAGES;
  a.v_stages = stages / 2;
  a.k_stages = stages - a.v_stages;
  const int smem = static_cast<int>(L::FIXED + stages * L::STAGE);
  const cudaError_t e = allow_shared_memory<tree_few_kernel<D, KGM>>(SMEM_CAP);
  if (e != cudaSuccess) return e;
  return launch_after(tree_few_kernel<D, KGM>, dim3(a.nsplit), FEW_THREADS, smem, stream, 1, tm, a);
}

template <int D>
cudaError_t launch_both(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream) {
  const cudaError_t e = a.cache.k_group_major ? launch<D, true>(tm, a, stream) : launch<D, false>(tm, a, stream);
  if (e != cudaSuccess || a.prefix == nullptr) return e;
  const int rows = a.T * (a.Hq / a.cache.Hkv);
  const dim3 grid((rows + MERGE_WARPS - 1) / MERGE_WARPS, a.cache.Hkv, a.B);
  return launch_after(tree_few_merge_kernel<D>, grid, MERGE_WARPS * 32, 0, stream, 1, a, a.nsplit);
}

}  // namespace

cudaError_t launch_tree_few(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream) {
  return a.cache.D == 128 ? launch_both<128>(tm, a, stream) : launch_both<64>(tm, a, stream);
}

}  // namespace wp
