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
// frequency near 1 loses its phase in fp32), reduced modulo 2 pi and kept as
// (cos, sin) in shared memory. Then the threads walk over the tokens' heads
// in units of 16 dims (8 whole channels in every layout): two 16-byte loads,
// 8 rotations in fp32, two 16-byte stores.
#include <cuda_bf16.h>
#include <cstdint>

#include "wp_serve.h"

namespace wp {
namespace {

constexpr int THREADS = 256;

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

template <bool PAIRS_IN, bool PAIRS_OUT, bool APPEND>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a, int tokens_per_block) {
  extern __shared__ float2 cs[];  // [tokens_per_block][rot / 2]
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), a.tokens - token0));
  const int C = a.rot / 2;
  for (int e = threadIdx.x; e < nt * C; e += THREADS) {
    const int t = e / C, c = e % C;
    const int64_t token = token0 + t;
    const double p = a.pos != nullptr ? static_cast<double>(a.pos[token]) : static_cast<double>(a.pos0 + token % a.N);
    constexpr double TWO_PI = 6.283185307179586476925286766559;
    constexpr double INV_TWO_PI = 0.15915494309189533576888376337251;
    const double ang = p * a.freq[c];
    const float r = static_cast<float>(fma(-rint(ang * INV_TWO_PI), TWO_PI, ang));
    float s, co;
    sincosf(r, &s, &co);
    cs[e] = make_float2(co * a.amp, s * a.amp * a.sign);
  }
  __syncthreads();
  const int U = a.D / 16;                                   // units per head
  const int per_token = (a.Hq + a.Hk * (APPEND ? 2 : 1)) * U;  // q heads, k heads, v heads when appending
  for (int e = threadIdx.x; e < nt * per_token; e += THREADS) {
    const int t = e / per_token;
    int h = (e - t * per_token) / U;
    const int u = e % U;  // per_token is a multiple of U
    const int64_t token = token0 + t;
    const int64_t b = token / a.N, n = token - b * a.N;
    const int what = h < a.Hq ? 0 : h < a.Hq + a.Hk ? 1 : 2;  // q, k, v
    const RowsArg &x = what == 0 ? a.q : what == 1 ? a.k : a.v;
    h -= what == 0 ? 0 : what == 1 ? a.Hq : a.Hq + a.Hk;
    const __nv_bfloat16 *src = x.data + b * x.sb + n * x.sn + h * x.sh;
    const bool turns = what != 2 && 16 * u < a.rot;
    int i0 = 16 * u, i1 = 16 * u + 8, o0 = i0, o1 = i1;
    if (turns) {
      unit_dims<PAIRS_IN>(u, a.rot, i0, i1);
      unit_dims<PAIRS_OUT>(u, a.rot, o0, o1);
    }
    uint4 lo = *reinterpret_cast<const uint4 *>(src + i0), hi = *reinterpret_cast<const uint4 *>(src + i1);
    if (turns) {
      float f[8], g[8], x0[8], x1[8], y0[8], y1[8];
      unpack8(lo, f);
      unpack8(hi, g);
      const float2 *w = cs + t * C + 8 * u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // channel 8u + j
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
      lo = pack8(f);
      hi = pack8(g);
    }
    __nv_bfloat16 *d0, *d1;
    if (APPEND && what != 0) {
      const CacheGeom &cg = a.cache;
      const int sq = a.seq[token], sl = a.slot[token];
      if (sq < 0 || sq >= cg.B || sl < 0 || sl >= cache_capacity(cg)) continue;  // padding, or outside: nothing written
      const int64_t page = cache_page(cg, sq, sl);
      if (page < 0) continue;
      const int row = sl % cg.page_size;
      if (what == 1) {
        d0 = cg.kc + k_offset(cg, page, h, row, o0);
        d1 = cg.kc + k_offset(cg, page, h, row, o1);
      } else {
        d0 = cg.vc + v_offset(cg, page, h, row, o0);
        d1 = cg.vc + v_offset(cg, page, h, row, o1);
      }
    } else {
      const RowsArg &y = what == 0 ? a.q_out : a.k_out;
      __nv_bfloat16 *dst = y.data + b * y.sb + n * y.sn + h * y.sh;
      d0 = dst + o0;
      d1 = dst + o1;
    }
    *reinterpret_cast<uint4 *>(d0) = lo;
    *reinterpret_cast<uint4 *>(d1) = hi;
  }
}

template <bool PAIRS_IN, bool PAIRS_OUT>
cudaError_t launch(const RotaryArgs &a, bool append, cudaStream_t stream) {
  const int tpb = a.tokens >= 8192 ? 8 : a.tokens >= 2048 ? 2 : 1;
  const int64_t blocks = (a.tokens + tpb - 1) / tpb;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const size_t smem = static_cast<size_t>(tpb) * (a.rot / 2) * sizeof(float2);
  if (append)
    rotary_kernel<PAIRS_IN, PAIRS_OUT, true><<<static_cast<unsigned>(blocks), THREADS, smem, stream>>>(a, tpb);
  else
    rotary_kernel<PAIRS_IN, PAIRS_OUT, false><<<static_cast<unsigned>(blocks), THREADS, smem, stream>>>(a, tpb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, int layout, bool inverse, bool append, cudaStream_t stream) {
  if (layout == 0) return launch<true, true>(a, append, stream);
  if (layout == 1) return launch<false, false>(a, append, stream);
  return inverse ? launch<true, false>(a, append, stream) : launch<false, true>(a, append, stream);
}

}  // namespace wp
