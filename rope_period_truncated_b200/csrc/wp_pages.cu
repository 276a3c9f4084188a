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
// One cluster of CLUSTER blocks does it all: the steps are ordered by the
// hardware's cluster barrier instead of by launches or by waiting on flags.
constexpr int PG_THREADS = 1024;
constexpr int CLUSTER = 8;

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

__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(PG_THREADS)
    pages_update_kernel(const __grid_constant__ PagesArgs a) {
  __shared__ int warp_sums[33];
  __shared__ int s_bad, s_free;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = rank * PG_THREADS + threadIdx.x;
  constexpr int NT = CLUSTER * PG_THREADS;
  const int P = a.page_size, MP = a.max_pages;
  const int64_t cap = static_cast<int64_t>(MP) * P;
  if (threadIdx.x == 0) s_bad = s_free = 0;
  __syncthreads();

  // 1. The counts to work on, and the rows' arguments.
  for (int i = tid; i < a.n_pages; i += NT) {
    const int r = a.refs[i];
    if (r < 0) s_bad = 1;
    a.refs_out[i] = r;
    a.writers[i] = 0;
    a.first[i] = INT_MAX;
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
  cluster.sync();
  bool bad = false;
  for (int c = 0; c < CLUSTER; ++c) bad = bad || *cluster.map_shared_rank(&s_bad, c) != 0;
  cluster.sync();  // s_bad is written again below

  // 2. Drop the rows' pages. A count that would fall below 0 has fewer holders
  // than there are rows: handing such a page out would give it two owners.
  const int64_t n = static_cast<int64_t>(a.B) * MP;
  if (!bad)
    for (int64_t e = tid; e < n; e += NT) {
      const int b = static_cast<int>(e / MP), j = static_cast<int>(e - static_cast<int64_t>(b) * MP);
      if (j < pages_of(a.lens[b], P)) {
        const int p = a.table[e];
        if (p < 0 || p >= a.n_pages || atomicSub(&a.refs_out[p], 1) < 1) s_bad = 1;
      }
    }
  cluster.sync();
  for (int c = 0; c < CLUSTER; ++c) bad = bad || *cluster.map_shared_rank(&s_bad, c) != 0;

  // 3. Take up the kept pages, and count who writes into partly filled ones.
  if (!bad)
    for (int64_t e = tid; e < n; e += NT) {
      const int b = static_cast<int>(e / MP), j = static_cast<int>(e - static_cast<int64_t>(b) * MP);
      if (j < pages_of(a.keep[b], P)) atomicAdd(&a.refs_out[a.table[static_cast<int64_t>(a.parent[b]) * MP + j]], 1);
    }
  // Who writes into which partly filled page.
  if (!bad)
    for (int b = tid; b < a.B; b += NT) {
      const int k = a.keep[b];
      if (a.new_lens[b] > k && k % P != 0) {
        const int last = a.table[static_cast<int64_t>(a.parent[b]) * MP + k / P];
        atomicAdd(&a.writers[last], 1);
        atomicMin(&a.first[last], b);
      }
    }
  cluster.sync();
  // Free pages of this block's share of the pool.
  const int share = (a.n_pages + CLUSTER - 1) / CLUSTER;
  const int p0 = min(rank * share, a.n_pages), p1 = min(p0 + share, a.n_pages);
  int mine = 0;
  for (int i = p0 + threadIdx.x; i < p1; i += PG_THREADS) mine += a.refs_out[i] == 0;
  int free_here;
  block_scan(mine, warp_sums, &free_here);
  if (threadIdx.x == 0) s_free = free_here;
  cluster.sync();
  int free_before = 0, free_all = 0;
  for (int c = 0; c < CLUSTER; ++c) {
    const int f = *cluster.map_shared_rank(&s_free, c);
    free_before += c < rank ? f : 0;
    free_all += f;
  }

  // 4. What each row needs (every block forms the sum; block 0 writes it down).
  int64_t total = 0;
  int n_copies = 0;
  if (!bad)
    for (int b0 = 0; b0 < a.B; b0 += PG_THREADS) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      int need = 0, copy = 0;
      if (b < a.B) {
        const int k = a.keep[b], nl = a.new_lens[b];
        if (nl > k && k % P != 0) {
          const int last = a.table[static_cast<int64_t>(a.parent[b]) * MP + k / P];
          const int r = a.refs_out[last];
          copy = r > 1 && !(a.writers[last] == r && a.first[last] == b);
        }
        need = pages_of(nl, P) - pages_of(k, P) + copy;
      }
      int sum, copies;
      const int off = block_scan(need, warp_sums, &sum);
      block_scan(copy, warp_sums, &copies);
      if (rank == 0 && b < a.B) {
        a.off[b] = static_cast<int>(min(total + off, static_cast<int64_t>(INT_MAX)));
        a.copying[b] = copy;
      }
      total += sum;
      n_copies += copies;
    }
  const bool refused = bad || total > free_all;
  // refs_out was read by every block above; the ranking below writes it
  cluster.sync();

  // 5. Rank the free pages; the lowest `total` of them are taken.
  if (!refused) {
    int64_t at = free_before;
    for (int i0 = p0; i0 < p1 && at < total; i0 += PG_THREADS) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      const int f = i < p1 && a.refs_out[i] == 0;
      int sum;
      const int64_t r = at + block_scan(f, warp_sums, &sum);
      if (f && r < total) {
        a.order[r] = i;
        a.refs_out[i] = 1;
      }
      at += sum;
    }
  }
  cluster.sync();

  // 6. The new rows.
  if (refused)
    for (int i = tid; i < a.n_pages; i += NT) a.refs_out[i] = a.refs[i];
  for (int64_t e = tid; e < n; e += NT) {
    const int b = static_cast<int>(e / MP), j = static_cast<int>(e - static_cast<int64_t>(b) * MP);
    int p = -1;
    if (refused) {
      p = a.table[e];
    } else {
      const int base = pages_of(a.keep[b], P) - a.copying[b];
      if (j < base)
        p = a.table[static_cast<int64_t>(a.parent[b]) * MP + j];
      else if (j < pages_of(a.new_lens[b], P))
        p = a.order[a.off[b] + j - base];
    }
    a.table_out[e] = p;
  }
  for (int b = tid; b < a.B; b += NT) {
    int src = -1, dst = -1, rows = 0;
    if (!refused && a.copying[b]) {
      const int k = a.keep[b];
      src = a.table[static_cast<int64_t>(a.parent[b]) * MP + k / P];
      dst = a.order[a.off[b]];
      rows = k % P;
      atomicSub(&a.refs_out[src], 1);
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
    a.info[3] = refused ? 0 : n_copies;
  }
  cluster.sync();  // no block leaves while another may still read its shared memory
}

// -------------------------------------------------------------------- copy
//
// Rows [0, rows) of every KV head from one page to another, K and V: bound by
// memory (read + write). One block per (copy, KV head); 16-byte pieces.
constexpr int COPY_THREADS = 256;

__global__ void __launch_bounds__(COPY_THREADS) pages_copy_kernel(const __grid_constant__ PagesCopyArgs a) {
  const CacheGeom &g = a.cache;
  const int i = blockIdx.x, h = blockIdx.y;
  const int src = a.copies[3 * i], dst = a.copies[3 * i + 1], rows = a.copies[3 * i + 2];
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
// nothing and gives lens_out = -1.
constexpr int COMPACT_THREADS = 256;
constexpr int BATCH = 8;

__global__ void __launch_bounds__(COMPACT_THREADS) compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int64_t s_from[COMPACT_MAX_PATH], s_to[COMPACT_MAX_PATH];  // page * page_size + row
  const CacheGeom &g = a.cache;
  const int b = blockIdx.x;
  const int len = a.lens[b], n = a.n_keep[b];
  bool bad = len < 0 || n < 0 || n > a.A;
  if (!bad)
    for (int i = threadIdx.x; i < n; i += COMPACT_THREADS) {
      const int p = a.path[static_cast<int64_t>(b) * a.A + i];
      const int before = i == 0 ? -1 : a.path[static_cast<int64_t>(b) * a.A + i - 1];
      const int64_t from = static_cast<int64_t>(len) + p;
      if (p <= before || from >= cache_capacity(g)) {
        bad = true;
        break;
      }
      const int to = len + i;
      const int64_t fp = cache_page(g, b, static_cast<int>(from)), tp = cache_page(g, b, to);
      if (fp < 0 || tp < 0) {
        bad = true;
        break;
      }
      s_from[i] = fp * g.page_size + from % g.page_size;
      s_to[i] = tp * g.page_size + to % g.page_size;
    }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.lens_out[b] = bad ? -1 : len + n;
  if (bad) return;
  const int pieces = g.D / 8;
  const int cols = g.Hkv * pieces * 2;  // K and V
  for (int e = threadIdx.x; e < cols; e += COMPACT_THREADS) {
    const bool is_v = e >= g.Hkv * pieces;
    const int x = is_v ? e - g.Hkv * pieces : e;
    const int h = x / pieces, dim = 8 * (x - h * pieces);
    __nv_bfloat16 *base = is_v ? g.vc : g.kc;
    auto at = [&](int64_t pr) {
      const int64_t page = pr / g.page_size;
      const int row = static_cast<int>(pr - page * g.page_size);
      return base + (is_v ? v_offset(g, page, h, row, dim) : k_offset(g, page, h, row, dim));
    };
    for (int i0 = 0; i0 < n; i0 += BATCH) {
      uint4 v[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j < n) v[j] = *reinterpret_cast<const uint4 *>(at(s_from[i0 + j]));
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j < n && s_from[i0 + j] != s_to[i0 + j]) *reinterpret_cast<uint4 *>(at(s_to[i0 + j])) = v[j];
    }
  }
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs &a, cudaStream_t stream) {
  pages_update_kernel<<<CLUSTER, PG_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PagesCopyArgs &a, cudaStream_t stream) {
  pages_copy_kernel<<<dim3(a.n, a.cache.Hkv), COPY_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream) {
  compact_kernel<<<a.cache.B, COMPACT_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace wp
