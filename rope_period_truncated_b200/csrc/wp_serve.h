// Internal launch interface of the rotary, cache-append, tree-attention,
// compaction and page kernels (not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace wp {

// Defined beside the other calls' tensor maps and wait limit.
long long wait_limit();
bool encode_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                const cuuint32_t *box, CUtensorMapSwizzle sw, CUtensorMapL2promotion promotion);

// A K/V cache, contiguous or paged. Both are pools of pages of page_size keys:
// K [n_pages, Hkv, page_size, D] or (group-major) [n_pages, Hkv, D/16,
// page_size, 16], V [n_pages, Hkv, page_size, D]. Contiguous: no block table,
// page b is sequence b and page_size = Lmax.
struct CacheGeom {
  __nv_bfloat16 *kc, *vc;
  const int32_t *block_table;  // [B, max_pages], or null: contiguous
  int B, Hkv, D, page_size, max_pages, n_pages;
  int k_group_major;
};

// Capacity in keys of one sequence.
__host__ __device__ inline int64_t cache_capacity(const CacheGeom &g) {
  return static_cast<int64_t>(g.max_pages) * g.page_size;
}

// Page of key `slot` of sequence b (slot within the capacity), -1 where the
// block table holds none.
__device__ __forceinline__ int64_t cache_page(const CacheGeom &g, int b, int slot) {
  if (g.block_table == nullptr) return b;
  const int p = g.block_table[static_cast<int64_t>(b) * g.max_pages + slot / g.page_size];
  return p >= 0 && p < g.n_pages ? p : -1;
}

// Element offsets of dims [dim, dim + 8) of row `row` of KV head h in `page`
// (dim a multiple of 8).
__device__ __forceinline__ int64_t v_offset(const CacheGeom &g, int64_t page, int h, int row, int dim) {
  return ((page * g.Hkv + h) * g.page_size + row) * g.D + dim;
}
__device__ __forceinline__ int64_t k_offset(const CacheGeom &g, int64_t page, int h, int row, int dim) {
  if (!g.k_group_major) return v_offset(g, page, h, row, dim);
  return (((page * g.Hkv + h) * (g.D / 16) + (dim >> 4)) * g.page_size + row) * 16 + (dim & 15);
}

// A strided [B, N, H, D] tensor, strides in elements, dims contiguous.
struct RowsArg {
  __nv_bfloat16 *data;
  int64_t sb, sn, sh;
};

struct RotaryArgs {
  RowsArg q, q_out, k, k_out, v;  // k_out / v unused when appending / not appending
  int Hq, Hk;                     // heads of q (0: none) and of k
  int64_t tokens;                 // B * N
  int N, D, rot;
  const int32_t *pos;             // [tokens], or null: pos0 + n
  int64_t pos0;
  float amp;                      // amplitude of the rotated dims
  float sign;                     // -1: the inverse rotation
  const int32_t *seq, *slot;      // appending: sequence and slot of each token
  CacheGeom cache;
  double freq[64];                // per channel, rot/2 entries
};

// layout as in the C ABI; append: K and V rows go to the cache.
cudaError_t launch_rotary(const RotaryArgs &a, int layout, bool inverse, bool append, cudaStream_t stream);

struct CompactArgs {
  CacheGeom cache;
  const int32_t *lens, *path, *n_keep;
  int32_t *lens_out;
  int A;  // entries per row of path
};
constexpr int COMPACT_MAX_PATH = 1024;
cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream);

struct PagesArgs {
  const int32_t *refs, *table, *lens, *parent, *keep, *new_lens;
  int32_t *refs_out, *table_out, *lens_out, *copies, *info;
  unsigned long long *counts;                // scratch [n_pages]
  int32_t *writers, *first, *order;          // scratch [n_pages] each
  int32_t *off, *copying;            // scratch [B] each
  int B, max_pages, n_pages, page_size;
};
cudaError_t launch_pages_update(const PagesArgs &a, cudaStream_t stream);

struct PagesCopyArgs {
  CacheGeom cache;
  const int32_t *copies;  // [n, 3]: source page, target page, rows
  int n;
};
cudaError_t launch_pages_copy(const PagesCopyArgs &a, cudaStream_t stream);

constexpr int TREE_MAX_NODES = 64;
constexpr int TREE_MAX_STAGES = 6;  // of K and of V
constexpr int TREE_MAX_GROUP = 16;  // query heads per KV head

struct TreeArgs {
  CacheGeom cache;
  const int32_t *lens, *parents, *n_nodes;  // [B], [B, T], [B] or null
  __nv_bfloat16 *o;                         // [B, T, Hq, D]
  float *lse;                               // [B, Hq, T] or null
  float *o_part, *lse_part;                 // [B, Hkv, T * R, nsplit(, D)], lse base 2
  int B, T, Hq;
  int tile_nodes, row_tiles;                // nodes per CTA, CTAs per KV head and split
  int nsplit, box_rows;                     // splits of the keys; rows of one TMA box
  int k_stages, v_stages;                   // ring depths, set at the launch
  int32_t cut[8];
  float scale_log2;
  long long wait_limit;
};

// How the work is cut. Nodes per CTA: as many whole nodes (R rows each) as 128
// rows hold. Splits: one batch entry fills the 148 SMs x 2 CTAs once, since
// its splits are equal; several entries have lengths of their own, so their
// CTAs are cut to fill them about four times over and the SMs even out.
inline int tree_tile_nodes(int T, int R) { return T < 128 / R ? T : 128 / R; }
inline int tree_splits(int B, int T, int Hkv, int R, int64_t capacity) {
  const int tile = tree_tile_nodes(T, R), tiles = (T + tile - 1) / tile;
  const int64_t units = static_cast<int64_t>(B) * Hkv * tiles;
  const int64_t want = (B == 1 ? 296 : 4 * 296) / units;
  const int64_t most = (capacity + 255) / 256;
  const int64_t n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n);
}
inline size_t tree_partial_o_bytes(int B, int T, int Hq, int nsplit, int D) {
  return (static_cast<size_t>(B) * T * Hq * nsplit * D * sizeof(float) + 255) & ~static_cast<size_t>(255);
}
inline size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int64_t capacity) {
  const int nsplit = tree_splits(B, T, Hkv, Hq / Hkv, capacity);
  if (nsplit == 1) return 256;
  return tree_partial_o_bytes(B, T, Hq, nsplit, D) + static_cast<size_t>(B) * T * Hq * nsplit * sizeof(float);
}

// Tensor maps. Q: 16 dims of the R heads of tile_nodes nodes. V: box_rows keys
// whole. K in boxes of box_rows keys: group-major 1, 2 or 4 groups, in rows 1
// or 2 chunks of 64 dims.
struct TreeMaps {
  CUtensorMap q, v, k[3];
};
cudaError_t launch_tree(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream);

}  // namespace wp
