// Pages of a paged K/V cache: one transaction on the block tables of a batch
// (fork, grow, copy on write, free), the row copies it asks for, and the
// compaction of an accepted path of drafted rows.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <climits>
#include <cstdint>

#include "wp_serve.h"
#include "waveprune.h"

namespace wp {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ update
//
// For row b: drop its pages (ceil(lens/P)), take the first ceil(keep/P) pages
// of row parent[b], copy the last of them if it is partly filled, will be
// written (new_lens > keep) and is held by somebody else, and extend to
// ceil(new_lens/P) pages with the lowest free ones, row after row. Counts are
// integer atomics, so their order cannot change the result.
//
// A page that several rows of the call would write: if they are its only
// holders, the lowest of them keeps it. So a copied page keeps at least one
// holder and is never handed out in the same call: its copy reads rows that
// no other copy writes.
//
// One cluster of up to 8 blocks does it all: its steps are ordered by the
// hardware's cluster barrier instead of by launches or by waiting on flags. It
// is a chain of a dozen dependent memory accesses and four barriers, so its
// time is latency (256 rows, a pool of 40000 pages: 21 us, with the scratch of 8
// blocks in global memory, where every atomic and dependent read goes to L2): few
// steps, and no more blocks than have work.
constexpr int PG_THREADS = 1024;
constexpr int MAX_CLUSTER = 8;
constexpr int ONE_BLOCK = 8192;  // fewer pages and table entries: one block, its scratch in shared memory
constexpr int PER_BLOCK = 4096;
constexpr int PER_LANE = 8;  // a warp ranks 32 x 8 pages at a time

__device__ __forceinline__ int pages_of(int tokens, int P) { return tokens / P + (tokens % P != 0); }

// Exclusive sum over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // warp_sums free
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s - w;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  *total = warp_sums[32];
  return warp_sums[warp] + inc - x;
}

constexpr unsigned long long DROP = 1ull, TAKE = 1ull << 32;

// Holders of a page after drops and takes.
__device__ __forceinline__ int holders(int refs, unsigned long long counts) {
  return refs - static_cast<int>(counts & 0xffffffffu) + static_cast<int>(counts >> 32);
}

// Copies of a page with r holders, w of them rows that will write into it.
__device__ __forceinline__ int copies_of(int r, int w) { return r > 1 ? (w == r ? w - 1 : w) : 0; }

__global__ void __launch_bounds__(PG_THREADS) pages_update_kernel(const __grid_constant__ PagesArgs a) {
  cudaGridDependencySynchronize();
  // One block: its scratch and the holders' counts are in shared memory, for the
  // atomics and for the reads that wait for them. 16 rows, a pool of 640 pages:
  // 11.5 -> 7.5 us.
  extern __shared__ unsigned long long scratch[];
  const bool own = a.in_shared;
  unsigned long long *counts = own ? scratch : a.counts;
  int32_t *writers = own ? reinterpret_cast<int32_t *>(scratch + a.n_pages) : a.writers;
  int32_t *first_of = own ? writers + a.n_pages : a.first, *order = own ? first_of + a.n_pages : a.order;
  int32_t *off_of = own ? order + a.n_pages : a.off, *copying = own ? off_of + a.B : a.copying;
  int32_t *held_refs = own ? copying + a.B : nullptr;
  const int32_t *refs = own ? held_refs : a.refs;
  __shared__ int warp_sums[33];
  __shared__ int s_bad, s_lost, s_free, s_out, s_copies;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
  const int tid = rank * PG_THREADS + threadIdx.x;
  const int NT = blocks * PG_THREADS;
  const int P = a.page_size, MP = a.max_pages;
  const int64_t cap = static_cast<int64_t>(MP) * P;
  const int warp = tid / 32, lane = tid % 32, warps = NT / 32;  // a warp takes a row of the tables
  if (threadIdx.x == 0) s_bad = s_lost = s_free = s_out = s_copies = 0;
  __syncthreads();

  // 1. The counts to work on, and the rows' arguments.
#pragma unroll 4
  for (int i = tid; i < a.n_pages; i += NT) {
    const int r = a.refs[i];
    if (r < 0) s_bad = 1;
    if (own) held_refs[i] = r;
    counts[i] = 0;
    writers[i] = 0;
    first_of[i] = INT_MAX;
  }
  for (int b = tid; b < a.B; b += NT) {
    const int len = a.lens[b], k = a.keep[b], nl = a.new_lens[b], p = a.parent[b];
    bool ok = len >= 0 && len <= cap && k >= 0 && nl >= k && nl <= cap;
    if (ok && k > 0) {
      ok = p >= 0 && p < a.B;
      if (ok) ok = k <= a.lens[p] && a.lens[p] <= cap;
    }
    if (!ok) s_bad = 1;
  }
  // Row threadIdx.x for step 3 (every block forms that sum): what it needs is
  // known now but for the counts.
  int my_kept = 0, my_wanted = 0, my_last = -1;
  const auto row_of = [&](int b) {
    my_kept = my_wanted = 0;
    my_last = -1;
    if (b >= a.B) return;
    const int k = a.keep[b], nl = a.new_lens[b], p = a.parent[b];
    my_kept = pages_of(k, P);
    my_wanted = pages_of(nl, P);
    if (k > 0 && k <= cap && nl > k && k % P != 0 && p >= 0 && p < a.B) my_last = a.table[static_cast<int64_t>(p) * MP + k / P];
  };
  row_of(threadIdx.x);
  // Every block's copy of a variable, one lane per block.
  const auto of_blocks = [&](int *v) { return lane < blocks ? *cluster.map_shared_rank(v, lane) : 0; };
  cluster.sync();
  bool bad = __any_sync(0xffffffffu, of_blocks(&s_bad));

  // 2. Drop the rows' pages and take up the kept ones: drops in the low half of
  // a page's count, takes in the high half, one atomic for both where a row
  // goes on with its own page (the scattered atomics bound this step). More
  // drops than holders: handing such a page out would give it two owners.
  if (!bad)
    for (int b = warp; b < a.B; b += warps) {
      const int k = a.keep[b], held = pages_of(a.lens[b], P), kept = pages_of(k, P);
      const int32_t *row = a.table + static_cast<int64_t>(b) * MP;
      const int32_t *from = kept ? a.table + static_cast<int64_t>(a.parent[b]) * MP : row;
      const int partial = a.new_lens[b] > k && k % P != 0 ? kept - 1 : -1;  // the page that row b will write into
#pragma unroll 2
      for (int j = lane; j < max(held, kept); j += 32) {
        const int p = j < held ? row[j] : -1, q = j < kept ? from[j] : -1;
        const bool p_ok = p >= 0 && p < a.n_pages, q_ok = q >= 0 && q < a.n_pages;
        if (j < held && !p_ok) s_lost = 1;  // a parent's bad page is flagged where its own row drops it
        if (p_ok) atomicAdd(&counts[p], p == q ? DROP + TAKE : DROP);
        if (q_ok) {
          if (p != q) atomicAdd(&counts[q], TAKE);
          if (j == partial) {
            atomicAdd(&writers[q], 1);
            atomicMin(&first_of[q], b);
          }
        }
      }
    }
  cluster.sync();
  bad = __any_sync(0xffffffffu, of_blocks(&s_lost)) || bad;

  // 3. Free pages of this block's share of the pool, and what each row needs
  // (every block forms that sum; block 0 writes it down).
  const int share = (a.n_pages + blocks - 1) / blocks;
  const int p0 = min(rank * share, a.n_pages), p1 = min(p0 + share, a.n_pages);
  int mine = 0;
#pragma unroll 4
  for (int i = p0 + threadIdx.x; i < p1; i += PG_THREADS) {
    const int r = refs[i];
    const unsigned long long c = counts[i];
    mine += holders(r, c) == 0;
    // more drops than holders, or more holders than 32 bits hold (a page that the caller has pinned by a huge count)
    const unsigned drops = static_cast<unsigned>(c & 0xffffffffu), takes = static_cast<unsigned>(c >> 32);
    if (drops > static_cast<unsigned>(r) || takes > static_cast<unsigned>(INT_MAX) - static_cast<unsigned>(r) + drops) s_out = 1;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) atomicAdd(&s_free, mine);
  int64_t total = 0;
  if (!bad)
    for (int b0 = 0; b0 < a.B; b0 += PG_THREADS) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      if (b0 > 0) row_of(b);
      int copy = 0;
      if (my_last >= 0) {
        const int r = holders(refs[my_last], counts[my_last]);
        copy = r > 1 && !(writers[my_last] == r && first_of[my_last] == b);
      }
      const int copies = __reduce_add_sync(0xffffffffu, copy);
      if (lane == 0) atomicAdd(&s_copies, copies);
      int sum;
      const int off = block_scan(my_wanted - my_kept + copy, warp_sums, &sum);
      if (rank == 0 && b < a.B) {
        off_of[b] = static_cast<int>(min(total + off, static_cast<int64_t>(INT_MAX)));
        copying[b] = copy;
      }
      total += sum;
    }
  cluster.sync();
  const int theirs = of_blocks(&s_free);
  bad = __any_sync(0xffffffffu, of_blocks(&s_out)) || bad;
  const int free_before = __reduce_add_sync(0xffffffffu, lane < rank ? theirs : 0);
  const int free_all = __reduce_add_sync(0xffffffffu, theirs);
  const bool refused = bad || total > free_all;

  // 4. The new counts; the lowest `total` free pages are taken, in order.
  {
    int64_t at = free_before;
    constexpr int STEP = PG_THREADS * PER_LANE;
    for (int i0 = p0; i0 < p1; i0 += STEP) {
      const int first = i0 + (threadIdx.x / 32) * 32 * PER_LANE + lane;  // this lane's pages: first + 32 e
      int r[PER_LANE], w[PER_LANE];
      unsigned free_lanes[PER_LANE];
#pragma unroll
      for (int e = 0; e < PER_LANE; ++e) {
        const int i = first + 32 * e;
        const bool in = i < p1;
        r[e] = !in ? 1 : refused ? refs[i] : holders(refs[i], counts[i]);
        w[e] = in && !refused ? writers[i] : 0;
      }
      int f = 0;
#pragma unroll
      for (int e = 0; e < PER_LANE; ++e) {
        free_lanes[e] = __ballot_sync(0xffffffffu, r[e] == 0);
        f += __popc(free_lanes[e]);
      }
      int sum;
      // lane 0 brings the warp's count into the sum; every lane gets what lies before the warp
      int64_t rank_of = at + __shfl_sync(0xffffffffu, block_scan(lane == 0 ? f : 0, warp_sums, &sum), 0);
#pragma unroll
      for (int e = 0; e < PER_LANE; ++e) {
        const int i = first + 32 * e;
        if (i < p1) {
          int now = r[e] - copies_of(r[e], w[e]);
          const int64_t k = rank_of + __popc(free_lanes[e] & ((1u << lane) - 1));
          if (r[e] == 0 && !refused && k < total) {
            order[k] = i;
            now = 1;
          }
          a.refs_out[i] = now;
        }
        rank_of += __popc(free_lanes[e]);
      }
      at += sum;
    }
  }
  cluster.sync();  // also: nobody reads another block's shared memory from here on

  // 5. The new rows.
  for (int b = warp; b < a.B; b += warps) {
    const int64_t at = static_cast<int64_t>(b) * MP;
    const int kept = pages_of(a.keep[b], P), base = refused ? MP : kept - copying[b];
    const int wanted = refused ? MP : pages_of(a.new_lens[b], P);
    const int32_t *from = refused || kept == 0 ? a.table + at : a.table + static_cast<int64_t>(a.parent[b]) * MP;
    const int32_t *fresh = order + (refused ? 0 : off_of[b] - base);
#pragma unroll 2
    for (int j = lane; j < MP; j += 32) a.table_out[at + j] = j < base ? from[j] : j < wanted ? fresh[j] : -1;
  }
  for (int b = tid; b < a.B; b += NT) {
    int src = -1, dst = -1, rows = 0;
    if (!refused && copying[b]) {
      const int k = a.keep[b];
      src = a.table[static_cast<int64_t>(a.parent[b]) * MP + k / P];
      dst = order[off_of[b]];
      rows = k % P;
    }
    a.copies[3 * b] = src;
    a.copies[3 * b + 1] = dst;
    a.copies[3 * b + 2] = rows;
    a.lens_out[b] = refused ? a.lens[b] : a.new_lens[b];
  }
  if (tid == 0) {
    a.info[0] = bad ? WP_PAGES_BAD_ARGUMENT : refused ? WP_PAGES_SHORT : WP_PAGES_OK;
    a.info[1] = bad ? 0 : static_cast<int>(min(total, static_cast<int64_t>(INT_MAX)));
    a.info[2] = bad ? 0 : free_all;
    a.info[3] = refused ? 0 : s_copies;
  }
}

// -------------------------------------------------------------------- copy
//
// Rows [0, rows) of every KV head from one page to another, K and V: bound by
// memory (read + write) where there is much, by latency else. One block per
// (copy, KV head); 16-byte pieces.
constexpr int COPY_THREADS = 256;

__global__ void __launch_bounds__(COPY_THREADS) pages_copy_kernel(const __grid_constant__ PagesCopyArgs a) {
  cudaGridDependencySynchronize();
  const CacheGeom &g = a.cache;
  const int i = blockIdx.x, h = blockIdx.y;
  const int32_t *c = a.copies + 3 * static_cast<int64_t>(i);
  const int src = c[0], dst = c[1], rows = c[2];
  if (src < 0 || src >= g.n_pages || dst < 0 || dst >= g.n_pages || rows < 1 || rows > g.page_size || src == dst) return;
  const int per_row = g.D / 8;
  const int n = rows * per_row;
  // group-major K: the rows of a group are contiguous, so walk group by group
  for (int e = threadIdx.x; e < n; e += COPY_THREADS) {
    int row, dim;
    if (g.k_group_major) {
      const int grp = e / (2 * rows), r = e - grp * 2 * rows;
      row = r >> 1;
      dim = 16 * grp + 8 * (r & 1);
    } else {
      row = e / per_row;
      dim = 8 * (e - row * per_row);
    }
    const int vr = e / per_row, vd = 8 * (e - vr * per_row);
    const uint4 k = *reinterpret_cast<const uint4 *>(g.kc + k_offset(g, src, h, row, dim));
    const uint4 v = *reinterpret_cast<const uint4 *>(g.vc + v_offset(g, src, h, vr, vd));
    *reinterpret_cast<uint4 *>(g.kc + k_offset(g, dst, h, row, dim)) = k;
    *reinterpret_cast<uint4 *>(g.vc + v_offset(g, dst, h, vr, vd)) = v;
  }
}

// ----------------------------------------------------------------- compact
//
// Row lens + path[i] moves to row lens + i, i < n_keep, in place. The path
// increases, so i <= path[i]: a move never overwrites the source of a later
// one, and a thread that carries its 16-byte column of the rows in order needs
// nobody else. One block per sequence; a bad path, length or page moves
// nothing and gives lens_out = -1. A chain of dependent loads (length, path,
// page, row), 8 rows in flight per thread. 16 paths of 16 nodes, 8 KV heads of
// 128: 3.4 us; 256 of 31: 6.3 us.
constexpr int COMPACT_THREADS = 256;
constexpr int BATCH = 8;

__global__ void __launch_bounds__(COMPACT_THREADS) compact_kernel(const __grid_constant__ CompactArgs a) {
  cudaGridDependencySynchronize();
  // element offsets of head 0, dim 0: of V; of K the same in rows, else apart
  __shared__ int64_t s_from[COMPACT_MAX_PATH], s_to[COMPACT_MAX_PATH];
  __shared__ int s_row_from[COMPACT_MAX_PATH], s_row_to[COMPACT_MAX_PATH];
  __shared__ int s_moves;
  const CacheGeom &g = a.cache;
  const int b = blockIdx.x;
  const int len = a.lens[b], n = a.n_keep[b];
  if (threadIdx.x == 0) s_moves = 0;
  bool bad = len < 0 || len > cache_capacity(g) || n < 0 || n > a.A;
  int first = INT_MAX;  // rows before it stay where they are
  for (int i = threadIdx.x; i < a.A; i += COMPACT_THREADS) {
    const int p = a.path[static_cast<int64_t>(b) * a.A + i];
    const int before = i == 0 ? -1 : a.path[static_cast<int64_t>(b) * a.A + i - 1];
    if (bad || i >= n) break;
    const int64_t from = static_cast<int64_t>(len) + p;
    // p >= i follows from a whole path that increases from 0 or more, but each
    // thread sees two entries of it: without this, an entry before a bad one
    // elsewhere could lead it to a key below 0 or a target behind the capacity,
    // and to a page looked up outside the block table.
    if (p < i || p <= before || from >= cache_capacity(g)) {
      bad = true;
      break;
    }
    const int to = len + i;
    const int64_t fp = cache_page(g, b, static_cast<int>(from)), tp = cache_page(g, b, to);
    if (fp < 0 || tp < 0) {
      bad = true;
      break;
    }
    if (p != i) first = min(first, i);
    s_row_from[i] = static_cast<int>(from) % g.page_size;
    s_row_to[i] = to % g.page_size;
    s_from[i] = fp * g.Hkv * g.page_size * g.D;
    s_to[i] = tp * g.Hkv * g.page_size * g.D;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.lens_out[b] = bad ? -1 : len + n;
  if (bad) return;
  // the path increases, so path[i] = i up to some i and never again
  if (first != INT_MAX) atomicMax(&s_moves, n - first);
  __syncthreads();
  const int start = n - s_moves;
  const int pieces = g.D / 8;
  const int cols = g.Hkv * pieces * 2;  // K and V
  for (int e = threadIdx.x; e < cols; e += COMPACT_THREADS) {
    const bool is_v = e >= g.Hkv * pieces;
    const int x = is_v ? e - g.Hkv * pieces : e;
    const int h = x / pieces, dim = 8 * (x - h * pieces);
    const bool split = !is_v && g.k_group_major;
    const int64_t col = is_v ? v_offset(g, 0, h, 0, dim) : k_offset(g, 0, h, 0, dim);
    const int row_step = split ? 16 : g.D;
    __nv_bfloat16 *base = (is_v ? g.vc : g.kc) + col;
    for (int i0 = start; i0 < n; i0 += BATCH) {
      uint4 v[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j < n) v[j] = *reinterpret_cast<const uint4 *>(base + s_from[i0 + j] + static_cast<int64_t>(s_row_from[i0 + j]) * row_step);
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j < n) *reinterpret_cast<uint4 *>(base + s_to[i0 + j] + static_cast<int64_t>(s_row_to[i0 + j]) * row_step) = v[j];
    }
  }
}

}  // namespace

cudaError_t launch_pages_update(PagesArgs a, cudaStream_t stream) {
  // one block with its scratch in shared memory (24 bytes a page, 8 a row) while
  // that holds it, else four from 8192 pages and table entries on and eight, the
  // portable cluster size, from 16384. 64 rows of 40 pages, a pool of 5000: 11.8 us
  // with one block, 14.6 with two that have their scratch in memory.
  const int64_t work = a.n_pages + static_cast<int64_t>(a.B) * a.max_pages;
  int blocks = 1;
  while (work >= ONE_BLOCK && blocks < MAX_CLUSTER && blocks <= work / PER_BLOCK) blocks *= 2;
  size_t smem = 0;
  a.in_shared = blocks == 1;
  if (a.in_shared) {
    smem = static_cast<size_t>(a.n_pages) * 24 + static_cast<size_t>(a.B) * 8;
    const cudaError_t e = allow_shared_memory<pages_update_kernel>(ONE_BLOCK * 24);  // n_pages + B < ONE_BLOCK
    if (e != cudaSuccess) return e;
  }
  return launch_after(pages_update_kernel, dim3(blocks), PG_THREADS, smem, stream, blocks, a);
}

cudaError_t launch_pages_copy(const PagesCopyArgs &a, cudaStream_t stream) {
  return launch_after(pages_copy_kernel, dim3(a.n, a.cache.Hkv), COPY_THREADS, 0, stream, 1, a);
}

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream) {
  return launch_after(compact_kernel, dim3(a.cache.B), COMPACT_THREADS, 0, stream, 1, a);
}

}  // namespace wp
