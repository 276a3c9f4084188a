// Rotation of Q and K in one launch (training, both directions), and the same
// rotation with the new K and V rows placed in a cache (serving).
//
// Channel c of a token at position p turns the pair of dims it owns by
// p * f_c, f_c = s_c * theta^(-2c/rot), c < rot/2, and multiplies it by the
// amplitude; dims from rot on pass through. Which dims a channel owns is the
// layout: (2c, 2c+1) interleaved, (c, c + rot/2) half-split; half-split paired
// reads the one and writes the other. The rotation is orthogonal, so the
// inverse (the gradient of the forward) is the same with -p * f_c, and swaps
// the paired layout's two sides.
//
// Bound by memory: 2 bytes read and 2 written per element. A block takes a few
// tokens; their angles are formed once, in fp64 (a far position times a
// frequency near 1 loses its phase in fp32), reduced modulo 2 pi and shared as
// (cos, sin). The work is in units of 16 dims (8 whole channels in every
// layout): two 16-byte loads, 8 rotations in fp32, two 16-byte stores. A
// thread keeps one token and one unit and walks over the heads, two in flight,
// its 8 (cos, sin) in registers; read from shared memory for every unit they
// were what bounded the kernel (131 us against 112).
// Q and K of 32768 tokens, 32 + 8 heads of 128: 105 us, 6.4 TB/s. Appending 20005
// tokens of the same heads, half of each head rotated, to pages of 16 keys: 70
// us, 5.8 TB/s; 128 tokens: 4 us.
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_serve.h"

namespace wp {
namespace {

constexpr int THREADS = 128;
constexpr int MAX_TOKENS = 4;  // per block

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float2 v = __bfloat1622float2(h[t]);
    f[2 * t] = v.x;
    f[2 * t + 1] = v.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 u;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
  for (int t = 0; t < 4; ++t) h[t] = __floats2bfloat162_rn(f[2 * t], f[2 * t + 1]);
  return u;
}

// The pieces (8 dims each) of unit u: [16u, +8) and [16u + 8, +8) where the
// pairs are adjacent, [8u, +8) and [rot/2 + 8u, +8) where they are split.
template <bool PAIRS>
__device__ __forceinline__ void unit_dims(int u, int rot, int &d0, int &d1) {
  d0 = PAIRS ? 16 * u : 8 * u;
  d1 = PAIRS ? d0 + 8 : rot / 2 + 8 * u;
}

// Element offsets of one token's rows: inputs and outputs of head 0, and of the
// cache rows it goes to (-1: nowhere).
struct TokenPlace {
  int64_t q, q_out, k, k_out, v, v_out;
};

// One unit in flight: its 16 dims and where they go (d0 null: nowhere).
struct Unit {
  uint4 lo, hi;
  __nv_bfloat16 *d0, *d1;
  bool turns;
};

template <bool PAIRS_IN, bool PAIRS_OUT>
__device__ __forceinline__ void rotate_unit(Unit &x, const float2 (&w)[8]) {
  float f[8], g[8], x0[8], x1[8], y0[8], y1[8];
  unpack8(x.lo, f);
  unpack8(x.hi, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x0[j] = PAIRS_IN ? (j < 4 ? f[2 * (j & 3)] : g[2 * (j & 3)]) : f[j];
    x1[j] = PAIRS_IN ? (j < 4 ? f[2 * (j & 3) + 1] : g[2 * (j & 3) + 1]) : g[j];
    y0[j] = x0[j] * w[j].x - x1[j] * w[j].y;
    y1[j] = x0[j] * w[j].y + x1[j] * w[j].x;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = PAIRS_OUT ? ((j & 1) ? y1[j >> 1] : y0[j >> 1]) : y0[j];
    g[j] = PAIRS_OUT ? ((j & 1) ? y1[4 + (j >> 1)] : y0[4 + (j >> 1)]) : y1[j];
  }
  x.lo = pack8(f);
  x.hi = pack8(g);
}

// A thread keeps its token and unit, and with them its 8 (cos, sin) in
// registers, and walks over heads: units run fastest over the lanes, then
// heads, then tokens.
template <int D, bool PAIRS_IN, bool PAIRS_OUT, bool APPEND>
__global__ void __launch_bounds__(THREADS, 6) rotary_kernel(const __grid_constant__ RotaryArgs a, int log_tokens) {
  cudaGridDependencySynchronize();
  constexpr int ULOG = D == 128 ? 3 : 2, U = 1 << ULOG;  // units per head
  extern __shared__ float2 cs[];                        // [tokens][rot / 2]
  __shared__ TokenPlace places[MAX_TOKENS];
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) << log_tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(1) << log_tokens, a.tokens - token0));
  const int C = a.rot / 2;
  const CacheGeom &cg = a.cache;
  if (threadIdx.x < nt) {
    const int64_t token = token0 + threadIdx.x;
    const int64_t b = token / a.N, n = token - b * a.N;
    TokenPlace p;
    p.q = b * a.q.sb + n * a.q.sn;
    p.q_out = b * a.q_out.sb + n * a.q_out.sn;
    p.k = b * a.k.sb + n * a.k.sn;
    if (APPEND) {
      p.v = b * a.v.sb + n * a.v.sn;
      p.k_out = p.v_out = -1;
      const int sq = a.seq[token], sl = a.slot[token];
      // padding, or outside the batch, the capacity or the pool: nothing written
      if (sq >= 0 && sq < cg.B && sl >= 0 && sl < cache_capacity(cg)) {
        const int64_t page = cache_page(cg, sq, sl);
        if (page >= 0) {
          const int row = sl % cg.page_size;
          p.k_out = k_offset(cg, page, 0, row, 0);
          p.v_out = v_offset(cg, page, 0, row, 0);
        }
      }
    } else {
      p.k_out = b * a.k_out.sb + n * a.k_out.sn;
    }
    places[threadIdx.x] = p;
  }
  __syncthreads();
  const int u = threadIdx.x & (U - 1);
  const int lanes = (THREADS >> ULOG) >> log_tokens;  // heads side by side
  const int t = (threadIdx.x >> ULOG) / lanes;
  int h = (threadIdx.x >> ULOG) - t * lanes;
  const int heads = t < nt ? a.Hq + a.Hk * (APPEND ? 2 : 1) : 0;  // q, k, and v when appending
  const TokenPlace p = places[t < nt ? t : 0];
  const bool rotated = 16 * u < a.rot;
  int i0 = 16 * u, i1 = i0 + 8, o0 = i0, o1 = i1;
  if (rotated) {
    unit_dims<PAIRS_IN>(u, a.rot, i0, i1);
    unit_dims<PAIRS_OUT>(u, a.rot, o0, o1);
  }
  const int64_t head_out = static_cast<int64_t>(cg.page_size) * D;  // from head to head of a cache page, K and V
  const auto load = [&](Unit &x) {
    const __nv_bfloat16 *src;
    __nv_bfloat16 *dst;
    bool split = false;  // group-major rows
    x.turns = rotated;
    int i = i0, j = i1, o = o0, e = o1;
    if (h < a.Hq) {
      src = a.q.data + p.q + h * a.q.sh;
      dst = a.q_out.data + p.q_out + h * a.q_out.sh;
    } else if (h < a.Hq + a.Hk) {
      const int hk = h - a.Hq;
      src = a.k.data + p.k + hk * a.k.sh;
      if (APPEND) {
        dst = p.k_out < 0 ? nullptr : cg.kc + p.k_out + hk * head_out;
        split = cg.k_group_major;
      } else {
        dst = a.k_out.data + p.k_out + hk * a.k_out.sh;
      }
    } else {
      const int hv = h - a.Hq - a.Hk;
      x.turns = false;
      src = a.v.data + p.v + hv * a.v.sh;
      dst = p.v_out < 0 ? nullptr : cg.vc + p.v_out + hv * head_out;
      i = o = 16 * u;
      j = e = i + 8;
    }
    x.lo = __ldcg(reinterpret_cast<const uint4 *>(src + i));
    x.hi = __ldcg(reinterpret_cast<const uint4 *>(src + j));
    // group-major rows: 16 dims in a row, the groups page_size rows apart
    x.d0 = dst == nullptr ? nullptr : dst + (split ? static_cast<int64_t>(o >> 4) * cg.page_size * 16 + (o & 15) : o);
    x.d1 = dst + (split ? static_cast<int64_t>(e >> 4) * cg.page_size * 16 + (e & 15) : e);
    h += lanes;
  };
  // Two units in flight per thread; the first two load while the angles form.
  Unit x, y;
  bool one = h < heads;
  if (one) load(x);
  bool two = one && h < heads;
  if (two) load(y);
  for (int e = threadIdx.x; e < nt * C; e += THREADS) {
    const int te = e / C, c = e - te * C;
    const int64_t token = token0 + te;
    const double pos = a.pos != nullptr ? static_cast<double>(a.pos[token]) : static_cast<double>(a.pos0 + token % a.N);
    constexpr double TWO_PI = 6.283185307179586476925286766559;
    constexpr double INV_TWO_PI = 0.15915494309189533576888376337251;
    const double ang = pos * a.freq[c];
    const float r = static_cast<float>(fma(-rint(ang * INV_TWO_PI), TWO_PI, ang));
    float s, co;
    sincosf(r, &s, &co);
    cs[e] = make_float2(co * a.amp, s * a.amp * a.sign);
  }
  __syncthreads();
  float2 w[8];
  if (rotated && t < nt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = cs[t * C + 8 * u + j];
  }
  const auto store = [&](Unit &x) {
    if (x.turns) rotate_unit<PAIRS_IN, PAIRS_OUT>(x, w);
    if (x.d0 != nullptr) {
      *reinterpret_cast<uint4 *>(x.d0) = x.lo;
      *reinterpret_cast<uint4 *>(x.d1) = x.hi;
    }
  };
  while (one) {
    store(x);
    if (two) store(y);
    one = two && h < heads;
    if (one) load(x);
    two = one && h < heads;
    if (two) load(y);
  }
}

template <int D, bool PAIRS_IN, bool PAIRS_OUT>
cudaError_t launch(const RotaryArgs &a, bool append, cudaStream_t stream) {
  // 4 tokens per block where that leaves blocks for every SM (10 heads per
  // thread for 32 + 8 heads), else 1. Q and K of 32768 tokens: 105 us with 4,
  // 110 us with 2, 110 us with 8; 5.5K appended tokens: 32 us with 4, 42 us with
  // 1; 128 tokens: 4.0 us with 1.
  const int log_tokens = a.tokens >= 2048 ? 2 : 0;
  const int64_t blocks = (a.tokens + (1 << log_tokens) - 1) >> log_tokens;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const size_t smem = (static_cast<size_t>(a.rot / 2) << log_tokens) * sizeof(float2);
  const auto kernel = append ? rotary_kernel<D, PAIRS_IN, PAIRS_OUT, true> : rotary_kernel<D, PAIRS_IN, PAIRS_OUT, false>;
  return launch_after(kernel, dim3(static_cast<unsigned>(blocks)), THREADS, smem, stream, 1, a, log_tokens);
}

template <int D>
cudaError_t launch_layout(const RotaryArgs &a, int layout, bool inverse, bool append, cudaStream_t stream) {
  if (layout == 0) return launch<D, true, true>(a, append, stream);
  if (layout == 1) return launch<D, false, false>(a, append, stream);
  return inverse ? launch<D, true, false>(a, append, stream) : launch<D, false, true>(a, append, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, int layout, bool inverse, bool append, cudaStream_t stream) {
  return a.D == 128 ? launch_layout<128>(a, layout, inverse, append, stream)
                    : launch_layout<64>(a, layout, inverse, append, stream);
}

}  // namespace wp
