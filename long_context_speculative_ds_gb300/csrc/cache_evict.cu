// Eviction from the draft's cache by accumulated attention weight, in place
// (include/ds.h, ds_cache_evict).
//
// A slot's rank is a 32-bit key: all ones for the first and recent tokens,
// else the weight's bits in an order that is the floats' (a NaN 0).  `select`
// finds the budget-th largest key of a segment (a sequence's slot head) digit
// by digit, how many of that very key stay (the lower slots), and lists the
// kept slots behind the budget and the free ones below it, both ascending;
// `move` copies one to the other.  No move's source is another's target
// (sources lie behind the budget, targets below it), so it works in place.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "draft_cache.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace ds {
namespace evict {

struct KArgs {
  DraftCache cache;
  const int32_t* lens;
  int32_t batch, slot_heads, head_dim;
  int64_t slot_stride, moves;
  float *weights, *weights_out;
  int32_t *positions, *positions_out;
  const int32_t* next_positions;
  int32_t budget, limit;         // cut when a sequence has more than `limit`
  int32_t recent, sinks;
  int32_t* new_lens;
  int32_t *count, *src, *dst;
  uint32_t* status;
};

constexpr int kThreads = 1024;

DS_DEV uint32_t rank_key(float w, int pos, int sinks, int64_t recent_from, bool& nan) {
  if (pos < sinks || pos >= recent_from) return ~0u;
  if (w != w) {
    nan = true;
    return 0u;
  }
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
  // (the largest key of a weight, +inf, is 0xff800000)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of one value per thread over the block, and the total.
DS_DEV int block_prefix(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int w = s_warp[lane];
  int wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += x;
  }
  total = __shfl_sync(0xffffffffu, wi, 31);
  return __shfl_sync(0xffffffffu, wi - w, warp) + incl - v;
}

__global__ void __launch_bounds__(kThreads) select(const KArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_prefix, s_left;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int len = __ldg(a.lens + b), tid = threadIdx.x;
  const int n = checked_len(len, a.cache.slots, a.status, tid == 0 && w == 0);
  const bool cut = n > a.limit;
  const int keep = cut ? a.budget : n;
  if (tid == 0 && w == 0) a.new_lens[b] = cut ? keep : len;
  const int64_t base = (int64_t)seg * a.slot_stride;
  const float* wt = a.weights + base;
  const int32_t* ps = a.positions + base;
  float* wo = a.weights_out ? a.weights_out + base : nullptr;
  int32_t* po = a.positions_out ? a.positions_out + base : nullptr;
  if (!cut) {
    if (tid == 0) a.count[seg] = 0;
    for (int i = tid; i < n; i += kThreads) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
    return;
  }
  const int64_t from = (int64_t)__ldg(a.next_positions + b) - a.recent;
  bool nan = false;
  if (tid == 0) { s_prefix = 0; s_left = keep; }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, left = s_left;
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t k = rank_key(wt[i], ps[i], a.sinks, from, nan);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {                       // from the largest digit down
      uint32_t above = 0;
      int d = 255;
      while (d > 0 && above + hist[d] < left) above += hist[d--];
      s_prefix = prefix << 8 | d;
      s_left = left - above;
    }
    __syncthreads();
  }
  if (nan) flag(a.status, DS_DEV_BAD_VALUE);
  const uint32_t at = s_prefix;           // the budget-th largest key
  const int ties = (int)s_left;           // how many of it stay
  int tie0 = 0, src0 = 0, dst0 = 0;
  int32_t* src = a.src + (int64_t)seg * a.moves;
  int32_t* dst = a.dst + (int64_t)seg * a.moves;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    uint32_t k = 0;
    if (i < n) k = rank_key(wt[i], ps[i], a.sinks, from, nan);
    const bool tie = i < n && k == at;
    int total;
    const int before = tie0 + block_prefix(tie, s_warp, total);
    tie0 += total;
    const bool stay = i < n && (k > at || (tie && before < ties));
    const bool come = stay && i >= keep, free = i < keep && !stay;
    const int si = src0 + block_prefix(come, s_warp, total);
    src0 += total;
    const int di = dst0 + block_prefix(free, s_warp, total);
    dst0 += total;
    if (come) src[si] = i;
    if (free) dst[di] = i;
    if (stay && i < keep) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
  }
  if (tid == 0) a.count[seg] = src0;
}

// A warp per move and kv head.
__global__ void __launch_bounds__(256) move(const KArgs a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int lane = threadIdx.x & 31;
  const int heads = a.slot_heads == 1 ? a.cache.num_kv_heads : 1;
  const int64_t items = (int64_t)a.count[seg] * heads;
  const int vecs = a.head_dim / 8;        // 16-byte vectors of a head's row
  for (int64_t it = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); it < items;
       it += (int64_t)gridDim.y * 8) {
    const int64_t i = it / heads;
    const int h = a.slot_heads == 1 ? (int)(it % heads) : w;
    const int s = a.src[(int64_t)seg * a.moves + i], d = a.dst[(int64_t)seg * a.moves + i];
    if (it % heads == 0 && lane == 0) {
      const int64_t base = (int64_t)seg * a.slot_stride;
      (a.weights_out ? a.weights_out : a.weights)[base + d] = a.weights[base + s];
      (a.positions_out ? a.positions_out : a.positions)[base + d] = a.positions[base + s];
    }
    const int ps = slot_page(a.cache, b, s), pd = slot_page(a.cache, b, d);
    if (ps < 0 || pd < 0) {
      if (lane == 0) flag(a.status, DS_DEV_BAD_PAGE);
      continue;
    }
    const int64_t from = slot_at(a.cache, ps, s) + (int64_t)h * a.cache.head_stride;
    const int64_t to = slot_at(a.cache, pd, d) + (int64_t)h * a.cache.head_stride;
    if (lane < 2 * vecs) {
      uint16_t* pool = a.cache.pool[lane >= vecs];
      const int v = lane % vecs;
      *reinterpret_cast<uint4*>(pool + to + v * 8) =
          *reinterpret_cast<const uint4*>(pool + from + v * 8);
    }
  }
}

}  // namespace evict

cudaError_t launch_cache_evict(const ds_evict_args& g, const EvictLayout& L,
                               cudaStream_t stream) {
  using namespace evict;
  KArgs a = {};
  a.cache = draft_cache(g);
  a.lens = g.lens;
  a.batch = g.batch;
  a.slot_heads = g.slot_heads;
  a.head_dim = g.head_dim;
  a.slot_stride = g.slot_stride;
  a.moves = L.moves;
  a.weights = g.weights;
  a.positions = g.positions;
  a.weights_out = g.weights_out == g.weights ? nullptr : g.weights_out;
  a.positions_out = g.positions_out == g.positions ? nullptr : g.positions_out;
  a.next_positions = g.next_positions;
  a.budget = g.budget;
  a.limit = std::max(g.budget, g.trigger);
  a.recent = g.recent;
  a.sinks = g.sinks;
  a.new_lens = g.new_lens;
  unsigned char* ws = static_cast<unsigned char*>(g.workspace);
  a.count = reinterpret_cast<int32_t*>(ws + L.count);
  a.src = reinterpret_cast<int32_t*>(ws + L.src);
  a.dst = reinterpret_cast<int32_t*>(ws + L.dst);
  a.status = reinterpret_cast<uint32_t*>(ws);
  const int segs = g.batch * g.slot_heads;
  cudaError_t e = launch_dependent(select, dim3(segs), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess || L.moves == 0) return e;
  const int64_t warps = L.moves * (g.slot_heads == 1 ? g.num_kv_heads : 1);
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8,
                                                               152 * 8 / segs + 1));
  return launch_dependent(move, dim3(segs, rows), dim3(256), 0, stream, a);
}

}  // namespace ds
