// Attention of one new token per sequence over the draft's cache, with every
// key's weight added to its running sum (include/ds.h, ds_decode_attn).
//
// Two kernels.  The split pass cuts every segment (a sequence's kv head) into
// pieces; a block forms a piece's running maximum m, sum l and output o in one
// pass over its keys, o and l scaled by 2^-m, and, when weights are asked for,
// leaves every logit in the workspace.  The finish joins the pieces:
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) o_i / l,
// and turns logits s into weights 2^(s - M - log2 l), summed over heads.
// Logits carry the factor log2 e, so that exponentials are powers of two.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dev_common.cuh"
#include "draft_cache.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace ds {
namespace decode {

constexpr int kTile = 64;       // keys of a tile

struct KArgs {
  const uint16_t* q;
  int64_t q_stride;
  DraftCache cache;
  const int32_t* lens;
  int32_t batch, hq, hkv, group, splits;
  int32_t window, sinks;
  float scale;                  // softmax scale times log2 e
  void* out;
  int32_t out_type;             // 0 bf16, 1 f16, 2 f32
  float* lse;
  const float* w_in;
  float* w_out;
  float decay;
  int32_t slot_heads;
  int64_t slot_stride;
  int2* desc;
  float2* part_ml;
  float* part_o;
  float* logits;                // NULL: no weights
  uint32_t* status;
};

// The slots that a sequence of n attends to: t < sinks and t >= n - window, as
// tiles of 64 slots, those that hold none left out.
struct Range {
  int n, sinks, start;          // t < sinks or t >= start
  int head, skip, tiles;        // tiles before the gap, tiles in it, tiles in all
};
DS_DEV Range range_of(int n, int window, int sinks) {
  Range r;
  r.n = n;
  r.sinks = sinks;
  r.start = window > 0 && window < n ? n - window : 0;
  const int w0 = r.start / kTile;
  r.head = min((int)(((int64_t)min(sinks, n) + kTile - 1) / kTile), w0);
  r.skip = w0 - r.head;
  r.tiles = (int)(((int64_t)n + kTile - 1) / kTile) - r.skip;
  return r;
}
DS_DEV int tile_slot(const Range& r, int i) { return (i < r.head ? i : i + r.skip) * kTile; }
DS_DEV bool visible(const Range& r, int t) {
  return t < r.n && (t < r.sinks || t >= r.start);
}

template <bool BF>
DS_DEV float up(uint16_t x) {
  if constexpr (BF) return __uint_as_float((uint32_t)x << 16);
  return __half2float(__ushort_as_half(x));
}

// A piece of a segment, key by key on the ordinary units.
template <int D, bool BF>
__global__ void __launch_bounds__(128) split(const KArgs a) {
  __shared__ float s_p[16][kTile];
  __shared__ float s_q[16][D];
  __shared__ int64_t s_at[kTile];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, b = seg / a.hkv, h = seg % a.hkv, G = a.group;
  const int n = checked_len(__ldg(a.lens + b), a.cache.slots, a.status,
                            threadIdx.x == 0 && h == 0 && blockIdx.y == 0);
  const Range r = range_of(n, a.window, a.sinks);
  const int pieces = max(1, min(a.splits, r.tiles));
  if (blockIdx.y == 0 && threadIdx.x == 0) a.desc[seg] = make_int2(seg * a.splits, pieces);
  if ((int)blockIdx.y >= pieces) return;
  const int t0 = (int)((int64_t)r.tiles * blockIdx.y / pieces);
  const int t1 = (int)((int64_t)r.tiles * (blockIdx.y + 1) / pieces);
  const int piece = seg * a.splits + blockIdx.y;
  for (int i = threadIdx.x; i < G * D; i += 128)
    s_q[i / D][i % D] = up<BF>(a.q[(int64_t)b * a.q_stride + (int64_t)(h * G) * D + i]);
  float m[16], l[16], o[16];
  for (int g = 0; g < G; ++g) { m[g] = -CUDART_INF_F; l[g] = 0.f; o[g] = 0.f; }
  for (int t = t0; t < t1; ++t) {
    const int slot0 = tile_slot(r, t);
    __syncthreads();
    if (threadIdx.x < kTile) {
      const int slot = slot0 + threadIdx.x;
      int64_t at = -1;                    // -1: not attended to, -2: no page
      if (visible(r, slot)) {
        const int pg = slot_page(a.cache, b, slot);
        if (pg < 0) flag(a.status, DS_DEV_BAD_PAGE);
        at = pg < 0 ? -2 : slot_at(a.cache, pg, slot) + (int64_t)h * a.cache.head_stride;
      }
      s_at[threadIdx.x] = at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * kTile; i += 128) {
      const int g = i / kTile, k = i % kTile;
      const int64_t at = s_at[k];
      float s = 0.f;
      if (at >= 0)
        for (int d = 0; d < D; ++d) s = fmaf(s_q[g][d], up<BF>(a.cache.pool[0][at + d]), s);
      s = at == -1 ? -CUDART_INF_F : s * a.scale;
      s_p[g][k] = s;
      if (a.logits && at != -1)
        a.logits[((int64_t)seg * a.cache.slots + slot0 + k) * G + g] = s;
    }
    __syncthreads();
    for (int g = 0; g < G; ++g) {
      float mx = m[g];
      for (int k = 0; k < kTile; ++k) mx = fmaxf(mx, s_p[g][k]);
      const float ref = mx == -CUDART_INF_F ? 0.f : mx;
      const float f = exp2f(m[g] - ref);
      m[g] = mx;
      l[g] *= f;
      o[g] *= f;
      for (int k = 0; k < kTile; ++k) {
        if (s_at[k] == -1) continue;
        const float p = exp2f(s_p[g][k] - ref);
        l[g] += p;
        if (threadIdx.x < D && s_at[k] >= 0)
          o[g] = fmaf(p, up<BF>(a.cache.pool[1][s_at[k] + threadIdx.x]), o[g]);
      }
    }
  }
  for (int g = 0; g < G; ++g) {
    if (threadIdx.x < D) a.part_o[((int64_t)piece * G + g) * D + threadIdx.x] = o[g];
    if (threadIdx.x == 0) a.part_ml[(int64_t)piece * G + g] = make_float2(m[g], l[g]);
  }
}

// Joins (max, sum) pairs over the warp.
DS_DEV float2 join_ml(float2 x) {
  const float M = warp_max(x.x);
  const float ref = M == -CUDART_INF_F ? 0.f : M;
  return make_float2(M, warp_sum(x.y * exp2f(x.x - ref)));
}
// (max, sum) of a row over its pieces; all lanes of a warp.
DS_DEV float2 row_ml(const KArgs& a, int2 d, int row) {
  float2 ml = make_float2(-CUDART_INF_F, 0.f);
  for (int i = threadIdx.x & 31; i < d.y; i += 32) {
    const float2 x = a.part_ml[(int64_t)(d.x + i) * a.group + row];
    const float M = fmaxf(ml.x, x.x), ref = M == -CUDART_INF_F ? 0.f : M;
    ml = make_float2(M, ml.y * exp2f(ml.x - ref) + x.y * exp2f(x.x - ref));
  }
  return join_ml(ml);
}

constexpr int kFinishWarps = 8;
constexpr int kSpan = 1024;     // slots of a weights item

template <int D>
__global__ void __launch_bounds__(32 * kFinishWarps) finish(const KArgs a, int row_blocks,
                                                            int spans) {
  __shared__ float s_ref[16];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group;
  if ((int)blockIdx.x < row_blocks) {     // a warp per output row
    const int64_t row = (int64_t)blockIdx.x * kFinishWarps + warp;
    if (row >= (int64_t)a.batch * a.hq) return;
    const int b = (int)(row / a.hq), hq = (int)(row % a.hq), h = hq / G, g = hq % G;
    const int n = checked_len(__ldg(a.lens + b), a.cache.slots, nullptr, false);
    float o[D / 32];
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
    if (n > 0) {
      const int2 d = a.desc[b * a.hkv + h];
      ml = row_ml(a, d, g);
      const float ref = ml.x == -CUDART_INF_F ? 0.f : ml.x;
      for (int i = 0; i < d.y; ++i) {
        const int64_t p = (int64_t)(d.x + i) * G + g;
        const float f = exp2f(a.part_ml[p].x - ref);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          o[k] = fmaf(f, a.part_o[p * D + lane * (D / 32) + k], o[k]);
      }
      const float inv = 1.f / ml.y;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) o[k] *= inv;
    }
    if (a.lse && lane == 0)
      a.lse[row] = n > 0 ? (ml.x + log2f(ml.y)) * 0.6931471805599453f : -CUDART_INF_F;
    const int64_t at = row * D + lane * (D / 32);
#pragma unroll
    for (int k = 0; k < D / 32; k += 2) {
      if (a.out_type == 2)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + k) =
            make_float2(o[k], o[k + 1]);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + k) =
            a.out_type == 0 ? ptx::pack_bf16x2(o[k], o[k + 1]) : ptx::pack_f16x2(o[k], o[k + 1]);
    }
    return;
  }
  // the others: weights of up to kSpan slots of a (sequence, slot head)
  const int64_t items = (int64_t)a.batch * a.slot_heads * spans;
  for (int64_t it = blockIdx.x - row_blocks; it < items; it += gridDim.x - row_blocks) {
    const int64_t bw = it / spans;
    const int b = (int)(bw / a.slot_heads), w = (int)(bw % a.slot_heads);
    const int n = checked_len(__ldg(a.lens + b), a.cache.slots, nullptr, false);
    const int64_t t0 = (it % spans) * kSpan;
    if (t0 >= n) continue;
    const Range r = range_of(n, a.window, a.sinks);
    float sum[kSpan / (32 * kFinishWarps)];
    const int64_t at = bw * a.slot_stride + t0;
#pragma unroll
    for (int k = 0; k < kSpan / (32 * kFinishWarps); ++k) {
      const int t = k * 32 * kFinishWarps + threadIdx.x;
      sum[k] = a.w_in && t0 + t < n ? a.w_in[at + t] * a.decay : 0.f;
    }
    for (int h = a.slot_heads == 1 ? 0 : w; h < (a.slot_heads == 1 ? a.hkv : w + 1); ++h) {
      const int seg = b * a.hkv + h;
      __syncthreads();
      const int2 d = a.desc[seg];
      for (int g = warp; g < G; g += kFinishWarps) {
        const float2 ml = row_ml(a, d, g);
        if (lane == 0) s_ref[g] = ml.x + log2f(ml.y);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSpan / (32 * kFinishWarps); ++k) {
        const int t = (int)t0 + k * 32 * kFinishWarps + threadIdx.x;
        if (!visible(r, t)) continue;
        const float* s = a.logits + ((int64_t)seg * a.cache.slots + t) * G;
        for (int g = 0; g < G; ++g) sum[k] += exp2f(s[g] - s_ref[g]);
      }
    }
#pragma unroll
    for (int k = 0; k < kSpan / (32 * kFinishWarps); ++k) {
      const int t = k * 32 * kFinishWarps + threadIdx.x;
      if (t0 + t < n) a.w_out[at + t] = sum[k];
    }
  }
}

}  // namespace decode

cudaError_t launch_decode_attn(const ds_decode_args& g, const DecodeLayout& L,
                               cudaStream_t stream) {
  using namespace decode;
  KArgs a = {};
  a.q = static_cast<const uint16_t*>(g.q);
  a.q_stride = g.q_row_stride;
  a.cache = draft_cache(g);
  a.lens = g.lens;
  a.batch = g.batch;
  a.hq = g.num_q_heads;
  a.hkv = g.num_kv_heads;
  a.group = a.hq / a.hkv;
  a.window = g.window;
  a.sinks = g.sinks;
  a.scale = (g.scale > 0.f ? g.scale : 1.f / std::sqrt((float)g.head_dim)) * kLog2e;
  a.out = g.out;
  a.out_type = g.out_f32 ? 2 : g.dtype == DS_KV_BF16 ? 0 : 1;
  a.lse = g.lse;
  a.w_in = g.weights_in;
  a.w_out = g.weights_out;
  a.decay = g.decay;
  a.slot_heads = g.slot_heads;
  a.slot_stride = g.slot_stride;
  unsigned char* ws = static_cast<unsigned char*>(g.workspace);
  a.desc = reinterpret_cast<int2*>(ws + L.desc);
  a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.logits = g.weights_out ? reinterpret_cast<float*>(ws + L.logits) : nullptr;
  a.status = reinterpret_cast<uint32_t*>(ws);
  const int segs = g.batch * g.num_kv_heads;
  a.splits = std::max(1, L.ctas / segs);
  const bool bf = g.dtype == DS_KV_BF16;
  auto k = g.head_dim == 128 ? (bf ? split<128, true> : split<128, false>)
                             : (bf ? split<64, true> : split<64, false>);
  cudaError_t e = launch_dependent(k, dim3(segs, a.splits), dim3(128), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int row_blocks = (int)(((int64_t)g.batch * a.hq + kFinishWarps - 1) / kFinishWarps);
  const int spans = (int)((a.cache.slots + kSpan - 1) / kSpan);
  const int64_t items = g.weights_out ? (int64_t)g.batch * g.slot_heads * spans : 0;
  const int grid = row_blocks + (int)std::min<int64_t>(items, 152 * 8);
  return launch_dependent(g.head_dim == 128 ? finish<128> : finish<64>, dim3(grid),
                          dim3(32 * kFinishWarps), 0, stream, a, row_blocks, spans);
}

}  // namespace ds
