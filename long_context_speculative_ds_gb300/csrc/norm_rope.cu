// RMS norm of every query and key head with the position rotation in the
// same pass (include/ds.h, ds_qk_norm_rope).
//
// y = x w / sqrt(mean(x^2) + eps), then each pair (a, b) half a head apart to
// (a cos - b sin, a sin + b cos), in float32 with one rounding to bf16.
//
// Bound by memory when there are many rows, by latency when there are few:
// with 32 + 8 heads of 128, 32,768 rows take 112 us, 6.0 TB/s of the 6.70 a
// copy reaches; 331 rows 4.5 us and one row 3.3 us, a launch and two round
// trips.  (A warp per row and one head at a time took 161, 10 and 9 us.)
//
// Eight lanes hold one head (head_dim 128; four at 64): lane l the eight
// values from 8l of the head's first half and the eight opposite them in the
// second, so that a lane owns whole rotation pairs, reads and writes 16-byte
// vectors, and the sum of squares is a sum over the eight lanes.  A warp
// takes a row and works on four (eight) heads at a time, the next ones' loads
// on their way; the row's D / 2 sines and cosines are formed once, two a
// lane, and shared through the warp's corner of shared memory.  With few rows
// a row's heads are spread over more warps.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dev_common.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

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
  int32_t per;                    // head groups of a warp
  uint32_t* status;
  // frequency j as a 64-bit fraction of a turn
  unsigned long long turn[64];
};

constexpr int kNormWarps = 8;             // warps of a block
// Head groups of a warp, their loads together; at three blocks an SM (80
// registers) a few words spill, 16 bytes stored and 48 loaded a thread.
constexpr int kNormBatch = 5;

template <int D>
__global__ void __launch_bounds__(32 * kNormWarps, 3) qk_norm_rope(const NormRopeKArgs a) {
  constexpr int HALF = D / 2;
  constexpr int LPH = HALF / 8;           // lanes of a head
  constexpr int HPW = 32 / LPH;           // heads of a warp at a time
  __shared__ __align__(16) float2 s_cs[kNormWarps][HALF];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row64 = (int64_t)blockIdx.x * kNormWarps + warp;
  if (row64 >= a.n_rows) return;
  const int row = (int)row64;
  const int groups = (a.heads + HPW - 1) / HPW;
  const int g0 = blockIdx.y * a.per, g1 = min(groups, g0 + a.per);
  if (g0 >= g1) return;
  const int pos = __ldg(a.positions + row);
  const int l = lane % LPH, sub = lane / LPH;
  // lane's part of head hh (query heads first, then key heads)
  auto src = [&](int hh) {
    const bool t = hh >= a.hq;
    return (t ? a.x[1] + (int64_t)row * a.stride[1] - (int64_t)a.hq * D
              : a.x[0] + (int64_t)row * a.stride[0]) + (int64_t)hh * D + l * 8;
  };
  auto dst = [&](int hh) {
    const bool t = hh >= a.hq;
    return (t ? a.out[1] + (int64_t)row * a.out_stride[1] - (int64_t)a.hq * D
              : a.out[0] + (int64_t)row * a.out_stride[0]) + (int64_t)hh * D + l * 8;
  };
  uint4 u[kNormBatch], v[kNormBatch];
#pragma unroll
  for (int k = 0; k < kNormBatch; ++k) {
    const int hh = (g0 + k) * HPW + sub;
    u[k] = v[k] = make_uint4(0, 0, 0, 0);
    if (g0 + k < g1 && hh < a.heads) {
      // plain loads: with q_out = q the same bytes are written below
      const uint16_t* p = src(hh);
      u[k] = *reinterpret_cast<const uint4*>(p);
      v[k] = *reinterpret_cast<const uint4*>(p + HALF);
    }
  }
  if (pos < 0) {
    if (lane == 0) flag(a.status, DS_DEV_BAD_LENGTH);
    return;
  }
  // position * frequency wraps modulo one turn in 64 bits; its upper half,
  // read as a signed number, is the angle in units of pi / 2^31
  float2* const cs = s_cs[warp];
#pragma unroll
  for (int k = 0; k < HALF / 32; ++k) {
    const int j = lane + 32 * k;
    const unsigned long long t = (unsigned long long)pos * a.turn[j];
    float sn = 0.f, c = 1.f;
    if (a.rotate) sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &sn, &c);
    cs[j] = make_float2(c, sn);
  }
  __syncwarp();
  float4 rot[4];                          // cosine and sine of two pairs each
#pragma unroll
  for (int i = 0; i < 4; ++i) rot[i] = *reinterpret_cast<const float4*>(&cs[l * 8 + 2 * i]);
#pragma unroll
  for (int k = 0; k < kNormBatch; ++k) {
    if (g0 + k < g1) {
      const int hh = (g0 + k) * HPW + sub;
      const uint32_t uw[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      const uint32_t vw[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      float x[8], y[8], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(uw[i] << 16);
        x[2 * i + 1] = __uint_as_float(uw[i] & 0xffff0000u);
        y[2 * i] = __uint_as_float(vw[i] << 16);
        y[2 * i + 1] = __uint_as_float(vw[i] & 0xffff0000u);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const uint16_t* const w = hh >= a.hq ? a.weight[1] : a.weight[0];
      if (w) {
        const float r = 1.f / sqrtf(sum * (1.f / D) + a.eps);
        const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(w + l * 8));
        const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(w + HALF + l * 8));
        const uint32_t p0[4] = {w0.x, w0.y, w0.z, w0.w}, p1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] *= r * __uint_as_float(p0[i] << 16);
          x[2 * i + 1] *= r * __uint_as_float(p0[i] & 0xffff0000u);
          y[2 * i] *= r * __uint_as_float(p1[i] << 16);
          y[2 * i + 1] *= r * __uint_as_float(p1[i] & 0xffff0000u);
        }
      }
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 c = rot[i];
        lo[i] = ptx::pack_bf16x2(x[2 * i] * c.x - y[2 * i] * c.y,
                                 x[2 * i + 1] * c.z - y[2 * i + 1] * c.w);
        hi[i] = ptx::pack_bf16x2(x[2 * i] * c.y + y[2 * i] * c.x,
                                 x[2 * i + 1] * c.w + y[2 * i + 1] * c.z);
      }
      if (hh < a.heads) {
        uint16_t* p = dst(hh);
        *reinterpret_cast<uint4*>(p) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(p + HALF) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
    }
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
  // less than 2^-53 of a turn, and the angle, at positions below 2^31, by
  // less than 2^-22 of one; at 2^17 by less than 2^-36
  // (base^(-2j/D) as a product of two powers: sixteen calls of pow, not 64)
  double lo[8], hi[8];
  if (a.rotate && !g.inv_freq)
    for (int k = 0; k < 8; ++k) {
      lo[k] = std::pow((double)g.rope_base, -2.0 * k / g.head_dim);
      hi[k] = std::pow((double)g.rope_base, -16.0 * k / g.head_dim) / 6.283185307179586;
    }
  for (int j = 0; j < 64; ++j) {
    a.turn[j] = 0ull;
    if (a.rotate && j < g.head_dim / 2) {
      const double turns =
          g.inv_freq ? g.inv_freq[j] / 6.283185307179586 : lo[j & 7] * hi[j >> 3];
      const double frac = turns - std::floor(turns);   // whole turns drop out
      a.turn[j] = frac < 1.0 ? (unsigned long long)(frac * 18446744073709551616.0) : 0ull;
    }
  }
  // at most kNormBatch head groups a warp, fewer (down to one) while that
  // fills the machine (152 SMs of 24 warps)
  const int hpw = 32 / (g.head_dim / 16), groups = (a.heads + hpw - 1) / hpw;
  const int slices = std::max((groups + kNormBatch - 1) / kNormBatch,
                              std::min(groups, 152 * 24 / g.n_rows));
  a.per = (groups + slices - 1) / slices;
  const dim3 grid((unsigned)(((int64_t)g.n_rows + kNormWarps - 1) / kNormWarps),
                  (unsigned)((groups + a.per - 1) / a.per));
  const dim3 block(32 * kNormWarps);
  if (g.head_dim == 128) return launch_dependent(qk_norm_rope<128>, grid, block, 0, stream, a);
  return launch_dependent(qk_norm_rope<64>, grid, block, 0, stream, a);
}

}  // namespace ds
