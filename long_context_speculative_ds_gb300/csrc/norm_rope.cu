// RMS norm of every query and key head with the position rotation in the
// same pass (include/ds.h, ds_qk_norm_rope).
//
// Eight lanes hold one head (head_dim 128; four at 64): lane l the eight
// values from 8l of the head's first half and the eight opposite them in the
// second, so that a lane owns whole rotation pairs, reads and writes 16-byte
// vectors, and the sum of squares is a sum over the eight lanes.  A warp
// takes four (eight) heads at a time.  A block works on one row, whose D / 2
// sines and cosines it forms once.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dev_common.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace ds {

struct NormRopeKArgs {
  const uint16_t* x[2];           // q, k
  uint16_t* out[2];
  const uint16_t* weight[2];
  int64_t stride[2], out_stride[2];
  const int32_t* positions;
  int32_t n_rows, hq, heads;      // heads = query + key heads
  float eps;
  int32_t rotate;
  uint32_t* status;
  // frequency j as a 64-bit fraction of a turn
  unsigned long long turn[64];
};

template <int D>
__global__ void __launch_bounds__(256) qk_norm_rope(const NormRopeKArgs a) {
  constexpr int HALF = D / 2;
  constexpr int LPH = HALF / 8;           // lanes of a head
  constexpr int HPW = 32 / LPH;           // heads of a warp
  __shared__ __align__(16) float2 cs[HALF];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int row = blockIdx.x;
  const int pos = __ldg(a.positions + row);
  if (pos < 0) {
    if (threadIdx.x == 0) flag(a.status, DS_DEV_BAD_LENGTH);
    return;
  }
  // position * frequency wraps modulo one turn in 64 bits; its upper half,
  // read as a signed number, is the angle in units of pi / 2^31
  for (int j = threadIdx.x; j < HALF; j += blockDim.x) {
    const unsigned long long t = (unsigned long long)pos * a.turn[j];
    float sn = 0.f, c = 1.f;
    if (a.rotate) sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &sn, &c);
    cs[j] = make_float2(c, sn);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, l = lane % LPH;
  const int nw = blockDim.x >> 5;
  for (int h0 = (threadIdx.x >> 5) * HPW; h0 < a.heads; h0 += nw * HPW) {
    const int hh = h0 + lane / LPH;
    const bool ok = hh < a.heads;
    const int t = hh >= a.hq, h = t ? hh - a.hq : hh;
    float x[8], y[8];
    if (ok) {
      const uint16_t* p = a.x[t] + (int64_t)row * a.stride[t] + h * D + l * 8;
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint4 v = *reinterpret_cast<const uint4*>(p + HALF);
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(uw[i] << 16);
        x[2 * i + 1] = __uint_as_float(uw[i] & 0xffff0000u);
        y[2 * i] = __uint_as_float(vw[i] << 16);
        y[2 * i + 1] = __uint_as_float(vw[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!ok) continue;
    if (a.weight[t]) {
      const float r = 1.f / sqrtf(sum * (1.f / D) + a.eps);
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(a.weight[t] + l * 8));
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.weight[t] + HALF + l * 8));
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] *= r * __uint_as_float(uw[i] << 16);
        x[2 * i + 1] *= r * __uint_as_float(uw[i] & 0xffff0000u);
        y[2 * i] *= r * __uint_as_float(vw[i] << 16);
        y[2 * i + 1] *= r * __uint_as_float(vw[i] & 0xffff0000u);
      }
    }
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = *reinterpret_cast<const float4*>(&cs[l * 8 + 2 * i]);
      const float a0 = x[2 * i], b0 = y[2 * i], a1 = x[2 * i + 1], b1 = y[2 * i + 1];
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(lo[i]) : "f"(a1 * c.z - b1 * c.w), "f"(a0 * c.x - b0 * c.y));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(hi[i]) : "f"(a1 * c.w + b1 * c.z), "f"(a0 * c.y + b0 * c.x));
    }
    uint16_t* p = a.out[t] + (int64_t)row * a.out_stride[t] + h * D + l * 8;
    *reinterpret_cast<uint4*>(p) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(p + HALF) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

cudaError_t launch_norm_rope(const ds_norm_rope_args& g, cudaStream_t stream) {
  NormRopeKArgs a;
  a.x[0] = static_cast<const uint16_t*>(g.q);
  a.x[1] = static_cast<const uint16_t*>(g.k);
  a.out[0] = static_cast<uint16_t*>(g.q_out);
  a.out[1] = static_cast<uint16_t*>(g.k_out);
  a.weight[0] = static_cast<const uint16_t*>(g.q_weight);
  a.weight[1] = static_cast<const uint16_t*>(g.k_weight);
  a.stride[0] = g.q_row_stride;
  a.stride[1] = g.k_row_stride;
  a.out_stride[0] = g.q_out_row_stride;
  a.out_stride[1] = g.k_out_row_stride;
  a.positions = g.positions;
  a.n_rows = g.n_rows;
  a.hq = g.num_q_heads;
  a.heads = g.num_q_heads + g.num_kv_heads;
  a.eps = g.eps;
  a.rotate = g.rope_base > 0.f || g.inv_freq != nullptr;
  a.status = static_cast<uint32_t*>(g.workspace);
  // a double's 53 bits leave each frequency (at most a radian in use) off by
  // less than 2^-54 of a turn, and the angle, at positions below 2^31, by
  // less than 2^-23 of one; at 2^17 by less than 2^-37
  for (int j = 0; j < 64; ++j) {
    a.turn[j] = 0ull;
    if (a.rotate && j < g.head_dim / 2) {
      const double f = g.inv_freq ? g.inv_freq[j]
                                  : std::pow((double)g.rope_base, -2.0 * j / g.head_dim);
      const double turns = f / 6.283185307179586;
      const double frac = turns - std::floor(turns);   // whole turns drop out
      a.turn[j] = frac < 1.0 ? (unsigned long long)std::ldexp(frac, 64) : 0ull;
    }
  }
  const int hpw = 32 / (g.head_dim / 16);
  const int warps = std::max(1, std::min(8, (a.heads + hpw - 1) / hpw));
  const dim3 grid(g.n_rows), block(32 * warps);
  if (g.head_dim == 128) return launch_dependent(qk_norm_rope<128>, grid, block, 0, stream, a);
  return launch_dependent(qk_norm_rope<64>, grid, block, 0, stream, a);
}

}  // namespace ds
