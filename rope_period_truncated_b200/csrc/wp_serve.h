// Internal launch interface of the rotary, cache-append, tree-attention,
// compaction and page kernels (not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>

namespace wp {

// Lets `kernel` have `bytes` of dynamic shared memory, once per device.
template <auto kernel>
inline cudaError_t allow_shared_memory(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// Launches `kernel`, which calls cudaGridDependencySynchronize() before it touches
// global memory: its blocks are set up while the kernel before it in the stream
// ends, and wait there until that one's results are in place. Saves about 2 us a
// kernel (a page step of two 14.5 -> 10.7 us, a tree of 4 nodes 10.4 -> 8.9, one
// over 4 x 4K keys, with its merge, 26.9 -> 25.3). Not with a cluster: a page
// transaction of 8 blocks took 54 us so, 28 without.
template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  if (cluster > 1) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  } else {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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
  int32_t *off, *copying;                    // scratch [B] each
  int B, max_pages, n_pages, page_size;
  int in_shared;                             // the scratch is the block's shared memory; set at the launch
};
cudaError_t launch_pages_update(PagesArgs a, cudaStream_t stream);

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
  float *o_part, *lse_part;                 // partial results, lse base 2
  int64_t *prefix;                          // few rows: [B + 1] key tiles (per head) before each sequence,
                                            // or null: a CTA per (sequence, KV head)
  int B, T, Hq;
  int tile_nodes, row_tiles;                // nodes per CTA, CTAs per KV head and split
  int nsplit, box_rows;                     // splits of the keys (few rows: CTAs); rows of one TMA box
  int k_stages, v_stages;                   // ring depths, set at the launch
  int32_t cut[8];
  float scale_log2;
  long long wait_limit;
};

// How the work is cut. Up to 32 rows per KV head (R query heads of T nodes) go
// to the kernel whose products have keys and dims as their 128 rows (16
// sequences of 16K to 32K keys, 32 rows: 211 us, 239 with the other; with 64
// rows, which it then took, 318 against 264): tiles of 128 keys, one CTA per SM,
// the tiles of all sequences and KV heads dealt out evenly; or, where no sequence
// can exceed 512 keys and the (sequence, KV head) units are no more than the
// SMs, a CTA per unit, which needs no merge (its launch and run cost 5 us, a
// tile about 1). More rows go to the one that has query rows there: tiles of
// whole nodes, 64 keys, two CTAs per SM, each
// (sequence, KV head) split on its own: so that the CTAs fill the SMs once (all
// 296 places where a CTA then has at least 1024 keys: 252 rows over 128K keys,
// back to back, 146 us, 159 with 256 CTAs; else 256, with less to merge: 4 x 2.5K to 4K keys
// 30.7 us with 9 splits, 28.4 with 8), or,
// for several sequences, whose lengths may differ, up to twice as long as a CTA
// keeps 1024 keys (16 x 16K to 32K keys, 64 rows: 248 us, 261 with twice as many).
constexpr int TREE_FEW_ROWS = 32;
constexpr int TREE_SMS = 148;
__host__ __device__ inline bool tree_few_rows(int T, int R) { return T * R <= TREE_FEW_ROWS; }
inline bool tree_whole_units(int B, int T, int Hkv, int R, int64_t capacity) {
  return tree_few_rows(T, R) && capacity <= 512 && static_cast<int64_t>(B) * Hkv <= TREE_SMS;
}
inline int tree_key_tile(int T, int R) { return tree_few_rows(T, R) ? 128 : 64; }
inline int tree_tile_nodes(int T, int R) { return T < 128 / R ? T : 128 / R; }
inline int tree_splits(int B, int T, int Hkv, int R, int64_t capacity) {
  const int64_t units = static_cast<int64_t>(B) * Hkv;
  if (tree_whole_units(B, T, Hkv, R, capacity)) return static_cast<int>(units);
  if (tree_few_rows(T, R)) {
    const int64_t tiles = units * ((capacity + 127) / 128);
    return static_cast<int>(tiles < TREE_SMS ? tiles : TREE_SMS);
  }
  const int tile = tree_tile_nodes(T, R), row_tiles = (T + tile - 1) / tile;
  int64_t once = 2 * TREE_SMS / (units * row_tiles);
  if (once * 1024 > capacity) once = 256 / (units * row_tiles);
  int64_t n = B == 1 ? 0 : 4 * TREE_SMS / (units * row_tiles);
  if (n > capacity / 1024) n = capacity / 1024;
  if (n < once) n = once;
  if (n > (capacity + 255) / 256) n = (capacity + 255) / 256;
  return static_cast<int>(n < 1 ? 1 : n);
}
// The workspace: partial O, partial LSE, prefix sums, each from a multiple of
// 256; nothing where nothing is merged.
struct TreeWorkspace {
  size_t lse, prefix, bytes;  // offsets, and the whole
};
inline TreeWorkspace tree_workspace(int B, int T, int Hq, int Hkv, int D, int64_t capacity) {
  const int nsplit = tree_splits(B, T, Hkv, Hq / Hkv, capacity);
  const bool few = tree_few_rows(T, Hq / Hkv);
  if (few ? tree_whole_units(B, T, Hkv, Hq / Hkv, capacity) : nsplit == 1) return TreeWorkspace{0, 0, 0};
  // few rows: two partial results per CTA, of the rows of one KV head
  const size_t n = few ? static_cast<size_t>(nsplit) * 2 * T * (Hq / Hkv) : static_cast<size_t>(B) * T * Hq * nsplit;
  const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  TreeWorkspace w;
  w.lse = up(n * D * sizeof(float));
  w.prefix = w.lse + up(n * sizeof(float));
  w.bytes = w.prefix + up(few ? (static_cast<size_t>(B) + 1) * sizeof(int64_t) : 0);
  return w;
}

// Tensor maps. Q: 16 dims of the R heads of tile_nodes nodes. V: box_rows keys
// whole. K in boxes of box_rows keys: group-major 1, 2 or 4 groups, in rows 1
// or 2 chunks of 64 dims.
struct TreeMaps {
  CUtensorMap q, v, k[3];
};
cudaError_t launch_tree(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream);
cudaError_t launch_tree_few(const TreeMaps &tm, const TreeArgs &a, cudaStream_t stream);

}  // namespace wp
