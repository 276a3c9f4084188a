// C ABI of the rotary, cache-append, tree-attention, compaction and page
// calls: argument checks and launches. Contracts: waveprune.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "waveprune.h"
#include "wp_serve.h"

namespace wp {
namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr double kLog2e = 1.4426950408889634074;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int head_dim_status(int d_h) {
  if (d_h == 64 || d_h == 128) return WP_OK;
  return d_h > 0 && d_h % 16 == 0 ? WP_ERR_UNSUPPORTED : WP_ERR_ARG;
}

bool rotary_args_ok(int d_h, int rot_dim, double theta, const double *freq_scale, double scale_all) {
  if (rot_dim < 16 || rot_dim > d_h || rot_dim % 16 != 0) return false;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(scale_all > 0.0) || !std::isfinite(scale_all)) return false;
  if (freq_scale != nullptr)
    for (int c = 0; c < rot_dim / 2; ++c)
      if (!(freq_scale[c] > 0.0) || !std::isfinite(freq_scale[c])) return false;
  return true;
}

// f_c = theta^(-2c/rot) * freq_scale[c] * scale_all
double channel_freq(int c, int rot_dim, double theta, const double *freq_scale, double scale_all) {
  return std::pow(theta, -2.0 * c / rot_dim) * (freq_scale != nullptr ? freq_scale[c] : 1.0) * scale_all;
}

// One [B, N, H, d] tensor's strides and where its elements lie.
struct Extent {
  uintptr_t lo, hi;  // bytes [lo, hi)
};

// Base, alignment and sign of the strides; `writes`: no element twice.
bool rows_ok(const wp_rows *x, int B, int N, int H, int d, bool writes, Extent *ext) {
  if (x == nullptr || x->data == nullptr || !aligned(x->data, 16)) return false;
  const int64_t stride[3] = {x->stride_b, x->stride_n, x->stride_h};
  const int size[3] = {B, N, H};
  int64_t last = 0;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (stride[i] < 0 || stride[i] % 8 != 0 || stride[i] > (int64_t(1) << 46) / size[i]) return false;
    last += stride[i] * (size[i] - 1);
  }
  if (writes) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return stride[i] < stride[j]; });
    int64_t inner = d;
    for (int i : order) {
      if (size[i] == 1) continue;
      if (stride[i] < inner) return false;
      inner += stride[i] * (size[i] - 1);
    }
  }
  ext->lo = reinterpret_cast<uintptr_t>(x->data);
  ext->hi = ext->lo + (static_cast<uintptr_t>(last) + d) * 2;
  return true;
}

// Do two tensors over the same B and N share an element? Exact where one
// lies outside the other's range and where both are slices of one fused row
// (same strides per token); true wherever it cannot be excluded.
bool may_overlap(const wp_rows *x, int Hx, const Extent &ex, const wp_rows *y, int Hy, const Extent &ey, int B, int N,
                 int d) {
  if (ex.hi <= ey.lo || ey.hi <= ex.lo) return false;
  if ((B > 1 && x->stride_b != y->stride_b) || (N > 1 && x->stride_n != y->stride_n)) return true;
  const int64_t in_x = (Hx > 1 ? x->stride_h * (Hx - 1) : 0) + d, in_y = (Hy > 1 ? y->stride_h * (Hy - 1) : 0) + d;
  const int64_t at = (static_cast<int64_t>(ey.lo) - static_cast<int64_t>(ex.lo)) / 2;  // y relative to x
  const bool apart = at >= in_x || -at >= in_y;
  const int64_t span = std::max(in_x, at + in_y) - std::min<int64_t>(0, at);  // both, within one token
  // from token to token at least the span, from run to run of tokens at least a whole run
  struct {
    int64_t stride;
    int size;
  } in = {x->stride_n, N}, out = {x->stride_b, B};
  if (N == 1 || (B > 1 && in.stride > out.stride)) std::swap(in, out);
  const int64_t run = span + (in.size > 1 ? in.stride * (in.size - 1) : 0);
  const bool fits = (in.size == 1 || in.stride >= span) && (out.size == 1 || out.stride >= run);
  return !(apart && fits);
}

bool same_rows(const wp_rows *x, const wp_rows *y, int B, int N, int H) {
  return x->data == y->data && (B == 1 || x->stride_b == y->stride_b) && (N == 1 || x->stride_n == y->stride_n) &&
         (H == 1 || x->stride_h == y->stride_h);
}

RowsArg rows_arg(const wp_rows *x) {
  if (x == nullptr) return RowsArg{nullptr, 0, 0, 0};
  return RowsArg{static_cast<__nv_bfloat16 *>(x->data), x->stride_b, x->stride_n, x->stride_h};
}

// Checks of a cache's arguments, and its geometry.
int cache_args(void *kcache, int k_layout, void *vcache, int B, int Lmax, const int32_t *block_table, int max_pages,
               int page_size, int n_pages, int H_kv, int d_h, CacheGeom *g) {
  if (kcache == nullptr || vcache == nullptr || !aligned(kcache, 16) || !aligned(vcache, 16)) return WP_ERR_ARG;
  if (k_layout == WP_KCACHE_WINDOWED) return WP_ERR_UNSUPPORTED;
  if (k_layout != WP_KCACHE_ROWS && k_layout != WP_KCACHE_GROUP_MAJOR) return WP_ERR_ARG;
  if (B <= 0 || H_kv <= 0) return WP_ERR_ARG;
  const int rc = head_dim_status(d_h);
  if (rc != WP_OK) return rc;
  if (block_table == nullptr) {
    if (Lmax <= 0) return WP_ERR_ARG;
    max_pages = 1;
    page_size = Lmax;
    n_pages = B;
  } else {
    if (!aligned(block_table, 4) || max_pages <= 0 || n_pages <= 0 || page_size < 16 || page_size % 16 != 0)
      return WP_ERR_ARG;
  }
  if (static_cast<int64_t>(max_pages) * page_size > (1ll << 30)) return WP_ERR_UNSUPPORTED;
  if (B > 65535 || H_kv > 65535) return WP_ERR_UNSUPPORTED;
  *g = CacheGeom{static_cast<__nv_bfloat16 *>(kcache), static_cast<__nv_bfloat16 *>(vcache), block_table, B, H_kv, d_h,
                 page_size, max_pages, n_pages, k_layout == WP_KCACHE_GROUP_MAJOR ? 1 : 0};
  return WP_OK;
}

// Bytes of a K or V pool from its base.
Extent pool_extent(const CacheGeom &g, const void *base) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
  return Extent{lo, lo + static_cast<uintptr_t>(g.n_pages) * g.Hkv * g.page_size * g.D * 2};
}
Extent extent(const void *p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Extent{lo, p == nullptr ? lo : lo + bytes};
}
bool meets(const Extent &x, const Extent &y) { return x.lo < y.hi && y.lo < x.hi; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? WP_OK : WP_ERR_CUDA; }

bool layout_ok(int layout) {
  return layout == WP_ROPE_INTERLEAVED || layout == WP_ROPE_HALF_SPLIT || layout == WP_ROPE_HALF_SPLIT_PAIRED;
}

void fill_freqs(RotaryArgs *a, int rot_dim, double theta, const double *freq_scale, double scale_all) {
  for (int c = 0; c < 64; ++c) a->freq[c] = c < rot_dim / 2 ? channel_freq(c, rot_dim, theta, freq_scale, scale_all) : 0.0;
}

}  // namespace
}  // namespace wp

using namespace wp;

extern "C" {

int wp_cutoffs_partial(int d_h, int rot_dim, double theta, const double *freq_scale, double scale_all, double alpha,
                       int layout, int32_t *chan_cut, int32_t *group_cut) {
  if (d_h < 16 || d_h % 16 != 0 || d_h > 1024) return WP_ERR_ARG;
  if (layout != WP_ROPE_INTERLEAVED && layout != WP_ROPE_HALF_SPLIT) return WP_ERR_ARG;
  if (!rotary_args_ok(d_h, rot_dim, theta, freq_scale, scale_all) || !(alpha > 0.0)) return WP_ERR_ARG;
  const int C = rot_dim / 2;
  int32_t wc[512];
  for (int c = 0; c < C; ++c) {
    const double fl = std::floor(alpha * kPi / channel_freq(c, rot_dim, theta, freq_scale, scale_all));
    wc[c] = fl < 2147483647.0 ? static_cast<int32_t>(fl) : WP_CUTOFF_INF;
  }
  if (chan_cut != nullptr) std::memcpy(chan_cut, wc, sizeof(int32_t) * C);
  if (group_cut != nullptr)
    for (int g = 0; g < d_h / 16; ++g) {
      int32_t m = 0;
      for (int k = 16 * g; k < 16 * g + 16; ++k) {
        const int32_t w = k >= rot_dim ? WP_CUTOFF_INF : wc[layout == WP_ROPE_INTERLEAVED ? k / 2 : k % C];
        m = w > m ? w : m;
      }
      group_cut[g] = m;
    }
  return WP_OK;
}

int wp_rope_scaling(int rot_dim, double theta, double factor, int original_len, double turns_slow, double turns_fast,
                    double *freq_scale, double *amplitude) {
  if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > 1024 || freq_scale == nullptr || amplitude == nullptr) return WP_ERR_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor) || original_len <= 0)
    return WP_ERR_ARG;
  if (!(turns_slow >= 0.0) || !(turns_fast > turns_slow) || !std::isfinite(turns_fast)) return WP_ERR_ARG;
  for (int c = 0; c < rot_dim / 2; ++c) {
    const double turns = original_len * std::pow(theta, -2.0 * c / rot_dim) / (2.0 * kPi);
    const double keep = std::min(1.0, std::max(0.0, (turns - turns_slow) / (turns_fast - turns_slow)));
    freq_scale[c] = (1.0 - keep) / factor + keep;
  }
  *amplitude = 0.1 * std::log(factor) + 1.0;
  return WP_OK;
}

int wp_rope_qk(const wp_rows *q, const wp_rows *q_out, int H_q, const wp_rows *k, const wp_rows *k_out, int H_k, int B,
               int N, int d_h, int rot_dim, const int32_t *pos, int pos0, double theta, const double *freq_scale,
               double scale_all, double amplitude, int layout, int inverse, void *stream) {
  if (B <= 0 || N <= 0 || H_q < 0 || H_k < 0 || H_q + static_cast<int64_t>(H_k) == 0) return WP_ERR_ARG;
  if (!layout_ok(layout)) return WP_ERR_ARG;
  const int rc = head_dim_status(d_h);
  if (rc != WP_OK) return rc;
  if (!rotary_args_ok(d_h, rot_dim, theta, freq_scale, scale_all) || !std::isfinite(static_cast<float>(amplitude))) return WP_ERR_ARG;
  if (!aligned(pos, 4)) return WP_ERR_ARG;
  if (H_q > 65535 || H_k > 65535 || static_cast<int64_t>(B) * N > 0x7fffffff) return WP_ERR_UNSUPPORTED;
  const bool paired = layout == WP_ROPE_HALF_SPLIT_PAIRED;
  const wp_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
  const int H[2] = {H_q, H_k};
  Extent ei[2], eo[2];
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0) continue;
    if (!rows_ok(in[i], B, N, H[i], d_h, false, &ei[i]) || !rows_ok(out[i], B, N, H[i], d_h, true, &eo[i]))
      return WP_ERR_ARG;
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      if (H[i] == 0 || H[j] == 0) continue;
      // an output over its own input: only in place, element by element
      if (i == j && same_rows(in[i], out[i], B, N, H[i])) {
        if (paired) return WP_ERR_ARG;
      } else if (may_overlap(in[i], H[i], ei[i], out[j], H[j], eo[j], B, N, d_h)) {
        return WP_ERR_ARG;
      }
    }
  if (H_q > 0 && H_k > 0 && may_overlap(q_out, H_q, eo[0], k_out, H_k, eo[1], B, N, d_h)) return WP_ERR_ARG;
  // positions are read by blocks that start after others have stored
  const Extent positions = extent(pos, static_cast<size_t>(B) * N * 4);
  for (int i = 0; i < 2; ++i)
    if (H[i] > 0 && meets(positions, eo[i])) return WP_ERR_ARG;
  RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  if (H_q > 0) a.q = rows_arg(q), a.q_out = rows_arg(q_out);
  if (H_k > 0) a.k = rows_arg(k), a.k_out = rows_arg(k_out);
  a.Hq = H_q;
  a.Hk = H_k;
  a.tokens = static_cast<int64_t>(B) * N;
  a.N = N;
  a.D = d_h;
  a.rot = rot_dim;
  a.pos = pos;
  a.pos0 = pos0;
  a.amp = static_cast<float>(amplitude);
  a.sign = inverse ? -1.f : 1.f;
  fill_freqs(&a, rot_dim, theta, freq_scale, scale_all);
  return from_cuda(launch_rotary(a, layout, inverse != 0, false, static_cast<cudaStream_t>(stream)));
}

int wp_rope_append(const wp_rows *q, const wp_rows *q_out, int H_q, const wp_rows *k, const wp_rows *v, int H_kv, int T,
                   int d_h, int rot_dim, const int32_t *pos, const int32_t *seq, const int32_t *slot, void *kcache,
                   int k_layout, void *vcache, int B, int Lmax, const int32_t *block_table, int max_pages,
                   int page_size, int n_pages, double theta, const double *freq_scale, double scale_all,
                   double amplitude, int layout, void *stream) {
  if (T <= 0 || H_q < 0 || pos == nullptr || seq == nullptr || slot == nullptr) return WP_ERR_ARG;
  if (!aligned(pos, 4) || !aligned(seq, 4) || !aligned(slot, 4) || !layout_ok(layout)) return WP_ERR_ARG;
  RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  const int rc = cache_args(kcache, k_layout, vcache, B, Lmax, block_table, max_pages, page_size, n_pages, H_kv, d_h, &a.cache);
  if (rc != WP_OK) return rc;
  if (!rotary_args_ok(d_h, rot_dim, theta, freq_scale, scale_all) || !std::isfinite(static_cast<float>(amplitude))) return WP_ERR_ARG;
  if (H_q > 65535) return WP_ERR_UNSUPPORTED;
  Extent ek, ev, eq, eo;
  if (!rows_ok(k, 1, T, H_kv, d_h, false, &ek) || !rows_ok(v, 1, T, H_kv, d_h, false, &ev)) return WP_ERR_ARG;
  const Extent cache[2] = {pool_extent(a.cache, kcache), pool_extent(a.cache, vcache)};
  if (meets(cache[0], cache[1])) return WP_ERR_ARG;
  // read by blocks that start after others have stored
  const size_t nt = static_cast<size_t>(T) * 4;
  const Extent index[4] = {extent(pos, nt), extent(seq, nt), extent(slot, nt), extent(block_table, static_cast<size_t>(B) * max_pages * 4)};
  for (const Extent &c : cache) {
    if (meets(ek, c) || meets(ev, c)) return WP_ERR_ARG;
    for (const Extent &i : index)
      if (meets(i, c)) return WP_ERR_ARG;
  }
  if (H_q > 0) {
    if (!rows_ok(q, 1, T, H_q, d_h, false, &eq) || !rows_ok(q_out, 1, T, H_q, d_h, true, &eo)) return WP_ERR_ARG;
    if (same_rows(q, q_out, 1, T, H_q)) {
      if (layout == WP_ROPE_HALF_SPLIT_PAIRED) return WP_ERR_ARG;
    } else if (may_overlap(q, H_q, eq, q_out, H_q, eo, 1, T, d_h)) {
      return WP_ERR_ARG;
    }
    if (may_overlap(k, H_kv, ek, q_out, H_q, eo, 1, T, d_h) || may_overlap(v, H_kv, ev, q_out, H_q, eo, 1, T, d_h))
      return WP_ERR_ARG;
    for (const Extent &c : cache)
      if (meets(eq, c) || meets(eo, c)) return WP_ERR_ARG;
    for (const Extent &i : index)
      if (meets(i, eo)) return WP_ERR_ARG;
    a.q = rows_arg(q), a.q_out = rows_arg(q_out);
  }
  a.k = rows_arg(k);
  a.v = rows_arg(v);
  a.Hq = H_q;
  a.Hk = H_kv;
  a.tokens = T;
  a.N = T;
  a.D = d_h;
  a.rot = rot_dim;
  a.pos = pos;
  a.seq = seq;
  a.slot = slot;
  a.amp = static_cast<float>(amplitude);
  a.sign = 1.f;
  fill_freqs(&a, rot_dim, theta, freq_scale, scale_all);
  return from_cuda(launch_rotary(a, layout, false, true, static_cast<cudaStream_t>(stream)));
}

size_t wp_decode_tree_workspace_bytes(int B, int T, int H_q, int H_kv, int d_h, int Lmax) {
  if (B <= 0 || T <= 0 || T > TREE_MAX_NODES || H_q <= 0 || H_kv <= 0 || d_h <= 0 || Lmax <= 0) return 0;
  if (H_q % H_kv != 0 || H_q / H_kv > TREE_MAX_GROUP) return 0;
  return tree_workspace(B, T, H_q, H_kv, d_h, Lmax).bytes;
}

int wp_decode_tree(const void *q, const void *kcache, int k_layout, const void *vcache, const int32_t *lens,
                   const int32_t *parents, const int32_t *n_nodes, int T, int Lmax, const int32_t *block_table,
                   int max_pages, int page_size, int n_pages, int B, int H_q, int H_kv, int d_h,
                   const int32_t *group_cut, float softmax_scale, void *o, float *lse, void *workspace,
                   size_t ws_bytes, void *stream) {
  if (q == nullptr || lens == nullptr || parents == nullptr || o == nullptr) return WP_ERR_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(lens, 4) || !aligned(parents, 4) ||
      !aligned(n_nodes, 4) || !aligned(workspace, 256))
    return WP_ERR_ARG;
  if (T <= 0 || H_q <= 0) return WP_ERR_ARG;
  TreeArgs a;
  std::memset(&a, 0, sizeof(a));
  const int rc = cache_args(const_cast<void *>(kcache), k_layout, const_cast<void *>(vcache), B, Lmax, block_table,
                            max_pages, page_size, n_pages, H_kv, d_h, &a.cache);
  if (rc != WP_OK) return rc;
  if (H_q % H_kv != 0 || !std::isfinite(softmax_scale)) return WP_ERR_ARG;
  if (T > TREE_MAX_NODES || H_q / H_kv > TREE_MAX_GROUP) return WP_ERR_UNSUPPORTED;
  const int64_t cap = cache_capacity(a.cache);
  const TreeWorkspace w = tree_workspace(B, T, H_q, H_kv, d_h, cap);
  if (w.bytes > 0 && (workspace == nullptr || ws_bytes < w.bytes)) return WP_ERR_ARG;
  for (int g = 0; g < 8; ++g) {
    a.cut[g] = (group_cut == nullptr || g >= d_h / 16) ? WP_CUTOFF_INF : group_cut[g];
    if (a.cut[g] < 0) return WP_ERR_ARG;
  }
  // the outputs and the workspace are written while the inputs are still read
  const size_t nq = static_cast<size_t>(B) * T * H_q, nb = static_cast<size_t>(B) * 4;
  const Extent parts[] = {extent(q, nq * d_h * 2),    extent(lens, nb),       extent(parents, nb * T), extent(n_nodes, nb),
                          pool_extent(a.cache, kcache), pool_extent(a.cache, vcache), extent(block_table, nb * max_pages),
                          extent(o, nq * d_h * 2),    extent(lse, nq * 4),    extent(w.bytes > 0 ? workspace : nullptr, w.bytes)};
  for (int out = 7; out < 10; ++out)
    for (int i = 0; i < out; ++i)
      if (meets(parts[out], parts[i])) return WP_ERR_ARG;
  const int R = H_q / H_kv, D = d_h;
  a.lens = lens;
  a.parents = parents;
  a.n_nodes = n_nodes;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.lse = lse;
  a.B = B;
  a.T = T;
  a.Hq = H_q;
  a.tile_nodes = tree_tile_nodes(T, R);
  a.row_tiles = (T + a.tile_nodes - 1) / a.tile_nodes;
  a.nsplit = tree_splits(B, T, H_kv, R, cap);
  const int key_tile = tree_key_tile(T, R);
  a.box_rows = key_tile;  // of one box: never across a page, which holds a multiple of 16 keys
  while (block_table != nullptr && page_size % a.box_rows != 0) a.box_rows /= 2;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.o_part = reinterpret_cast<float *>(ws);
  a.lse_part = reinterpret_cast<float *>(ws + w.lse);
  a.prefix = w.bytes > 0 ? reinterpret_cast<int64_t *>(ws + w.prefix) : nullptr;
  a.wait_limit = wait_limit();
  const float scale = softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(double(d_h)));
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  if (!std::isfinite(a.scale_log2)) return WP_ERR_ARG;
  // Q [B, T, Hq, D]; V and K in rows [pages, Hkv, P, D] with the dims as
  // chunks of 64; group-major K [pages, Hkv, G, P, 16]. K is promoted in L2 no
  // further than a line: its neighbours in memory may be out of window.
  const CacheGeom &g = a.cache;
  const cuuint64_t P = g.page_size, H = H_kv, n = g.n_pages, G = D / 16, C = D / 64, row = 2 * D;
  const cuuint32_t box = a.box_rows;
  TreeMaps tm;
  const cuuint64_t dq[4] = {cuuint64_t(D), cuuint64_t(H_q), cuuint64_t(T), cuuint64_t(B)}, sq[3] = {row, row * H_q, row * H_q * T};
  const cuuint32_t bq[4] = {16, cuuint32_t(R), cuuint32_t(a.tile_nodes), 1};
  const cuuint64_t dr[5] = {64, P, C, H, n}, sr[4] = {row, 128, row * P, row * P * H};
  const cuuint64_t dg[5] = {16, P, G, H, n}, sg[4] = {32, 32 * P, row * P, row * P * H};
  const cuuint32_t bv[5] = {64, box, cuuint32_t(C), 1, 1};
  bool ok = encode_map(&tm.q, q, 4, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
            encode_map(&tm.v, vcache, 5, dr, sr, bv, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  for (int w = 0; ok && w < 3; ++w) {
    // boxes of several groups only where one box holds a whole tile of keys
    const cuuint32_t wide = a.box_rows == key_tile ? 1u << w : 1u;
    const cuuint32_t bg[5] = {16, box, wide, 1, 1}, br[5] = {64, box, wide < C ? wide : cuuint32_t(C), 1, 1};
    ok = g.k_group_major
             ? encode_map(&tm.k[w], kcache, 5, dg, sg, bg, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B)
             : encode_map(&tm.k[w], kcache, 5, dr, sr, br, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  }
  if (!ok) return WP_ERR_CUDA;
  return from_cuda(launch_tree(tm, a, static_cast<cudaStream_t>(stream)));
}

int wp_kv_compact(void *kcache, int k_layout, void *vcache, const int32_t *lens, const int32_t *path, int A,
                  const int32_t *n_keep, int32_t *lens_out, int Lmax, const int32_t *block_table, int max_pages,
                  int page_size, int n_pages, int B, int H_kv, int d_h, void *stream) {
  if (lens == nullptr || path == nullptr || n_keep == nullptr || lens_out == nullptr || A <= 0) return WP_ERR_ARG;
  if (!aligned(lens, 4) || !aligned(path, 4) || !aligned(n_keep, 4) || !aligned(lens_out, 4)) return WP_ERR_ARG;
  CompactArgs a;
  const int rc = cache_args(kcache, k_layout, vcache, B, Lmax, block_table, max_pages, page_size, n_pages, H_kv, d_h, &a.cache);
  if (rc != WP_OK) return rc;
  if (A > COMPACT_MAX_PATH) return WP_ERR_UNSUPPORTED;
  // sequences run side by side: what one of them writes, none may read
  const size_t nb = static_cast<size_t>(B) * 4;
  const Extent parts[] = {extent(path, nb * A), extent(n_keep, nb), extent(block_table, nb * max_pages), extent(lens, nb),
                          extent(lens_out, nb), pool_extent(a.cache, kcache), pool_extent(a.cache, vcache)};
  for (int out = 4; out < 7; ++out)
    for (int i = 0; i < out; ++i)
      if (meets(parts[out], parts[i]) && !(out == 4 && i == 3 && lens_out == lens)) return WP_ERR_ARG;
  a.lens = lens;
  a.path = path;
  a.n_keep = n_keep;
  a.lens_out = lens_out;
  a.A = A;
  return from_cuda(launch_compact(a, static_cast<cudaStream_t>(stream)));
}

size_t wp_pages_update_workspace_bytes(int B, int n_pages) {
  if (B <= 0 || n_pages <= 0) return 0;
  return (static_cast<size_t>(n_pages) * 5 + static_cast<size_t>(B) * 2) * sizeof(int32_t);
}

int wp_pages_update(const int32_t *refs, const int32_t *block_table, const int32_t *lens, const int32_t *parent,
                    const int32_t *keep, const int32_t *new_lens, int32_t *refs_out, int32_t *block_table_out,
                    int32_t *lens_out, int32_t *copies, int32_t *info, int B, int max_pages, int page_size, int n_pages,
                    void *workspace, size_t ws_bytes, void *stream) {
  const void *ptrs[] = {refs, block_table, lens, parent, keep, new_lens, refs_out, block_table_out, lens_out, copies, info, workspace};
  for (const void *p : ptrs)
    if (p == nullptr || !aligned(p, p == workspace ? 8 : 4)) return WP_ERR_ARG;
  if (B <= 0 || max_pages <= 0 || page_size < 16 || page_size % 16 != 0 || n_pages <= 0) return WP_ERR_ARG;
  if (static_cast<int64_t>(max_pages) * page_size > (1ll << 30) || B > 65535 || n_pages > (1 << 30)) return WP_ERR_UNSUPPORTED;
  // the pages that all rows need, and a page's drops and takes, are counted in 32 bits
  if (static_cast<int64_t>(B) * max_pages > 0x7fffffff) return WP_ERR_UNSUPPORTED;
  if (ws_bytes < wp_pages_update_workspace_bytes(B, n_pages)) return WP_ERR_ARG;
  // the outputs are written while the inputs are still read
  const size_t nb = static_cast<size_t>(B) * 4, nt = nb * max_pages, np = static_cast<size_t>(n_pages) * 4;
  const size_t size[] = {np, nt, nb, nb, nb, nb, np, nt, nb, 3 * nb, 16, wp_pages_update_workspace_bytes(B, n_pages)};
  for (int o = 6; o < 12; ++o)
    for (int i = 0; i < o; ++i) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(ptrs[o]), y = reinterpret_cast<uintptr_t>(ptrs[i]);
      if (x < y + size[i] && y < x + size[o]) return WP_ERR_ARG;
    }
  PagesArgs a;
  a.refs = refs;
  a.table = block_table;
  a.lens = lens;
  a.parent = parent;
  a.keep = keep;
  a.new_lens = new_lens;
  a.refs_out = refs_out;
  a.table_out = block_table_out;
  a.lens_out = lens_out;
  a.copies = copies;
  a.info = info;
  a.counts = static_cast<unsigned long long *>(workspace);
  a.writers = reinterpret_cast<int32_t *>(a.counts + n_pages);
  a.first = a.writers + n_pages;
  a.order = a.first + n_pages;
  a.off = a.order + n_pages;
  a.copying = a.off + B;
  a.B = B;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  return from_cuda(launch_pages_update(a, static_cast<cudaStream_t>(stream)));
}

int wp_pages_copy(void *k_pages, int k_layout, void *v_pages, const int32_t *copies, int n, int n_pages, int page_size,
                  int H_kv, int d_h, void *stream) {
  if (copies == nullptr || !aligned(copies, 4) || n <= 0) return WP_ERR_ARG;
  PagesCopyArgs a;
  // any non-null block table: the pools are paged, the copies name their pages
  const int rc = cache_args(k_pages, k_layout, v_pages, 1, 0, copies, 1, page_size, n_pages, H_kv, d_h, &a.cache);
  if (rc != WP_OK) return rc;
  if (static_cast<int64_t>(page_size) * (d_h / 8) > (1ll << 30)) return WP_ERR_UNSUPPORTED;  // 16-byte pieces of a head's page, in 32 bits
  const Extent k = pool_extent(a.cache, k_pages), v = pool_extent(a.cache, v_pages), c = extent(copies, static_cast<size_t>(n) * 12);
  if (meets(k, v) || meets(k, c) || meets(v, c)) return WP_ERR_ARG;
  a.copies = copies;
  a.n = n;
  return from_cuda(launch_pages_copy(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
