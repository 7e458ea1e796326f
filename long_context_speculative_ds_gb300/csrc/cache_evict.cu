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
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "draft_cache.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace cg = cooperative_groups;

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

// A cluster of blocks per segment, a contiguous part of its slots to each, and
// of that a contiguous part to each warp: its slots i0 + 32 j + lane, j < per.
// Keys of the first kKeep of these stay in registers; beyond (segments of more
// than kKeep 1024 slots a block) they are formed anew from memory.
constexpr int kKeep = 16;
constexpr int kBins = 2048;               // of a digit: 11, 11 and 10 bits

struct Shared {
  uint32_t hist[3][kBins];
  uint32_t forced;                        // slots that must stay
  int warp_sum[2][32];
  int block_sum[2][2];                    // [ties | come and free][...]: of this block
  uint32_t prefix, left, count;
};

// Exclusive prefix of one value per warp (the same on all its lanes) over the
// block's warps, and the total.
DS_DEV int warps_prefix(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  const int w = s_warp[lane];
  int incl = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  total = __shfl_sync(0xffffffffu, incl, 31);
  return __shfl_sync(0xffffffffu, incl - w, warp);
}

__global__ void __launch_bounds__(kThreads) select(const KArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.forced = 0;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x / C, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int len = __ldg(a.lens + b);
  const int n = checked_len(len, a.cache.slots, a.status, tid == 0 && rank == 0 && w == 0);
  const bool cut = n > a.limit;
  const int keep = cut ? a.budget : n;
  if (tid == 0 && rank == 0 && w == 0) a.new_lens[b] = cut ? keep : len;
  const int64_t base = (int64_t)seg * a.slot_stride;
  const float* wt = a.weights + base;
  const int32_t* ps = a.positions + base;
  float* wo = a.weights_out ? a.weights_out + base : nullptr;
  int32_t* po = a.positions_out ? a.positions_out + base : nullptr;
  if (!cut) {                             // (the whole cluster)
    if (tid == 0 && rank == 0) a.count[seg] = 0;
    for (int i = rank * kThreads + tid; i < n; i += C * kThreads) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
    return;
  }
  const int64_t from = (int64_t)__ldg(a.next_positions + b) - a.recent;
  // rows of 32 slots: of the segment, of a warp
  const int rows = (n + 31) / 32, per = (rows + C * 32 - 1) / (C * 32);
  const int i0 = ((rank * 32 + warp) * per) * 32 + lane;
  bool nan = false;
  auto read = [&](int j) {                // 0: no slot (no key of a slot is ranked by it
    const int i = i0 + 32 * j;            // before the slot's own bounds are looked at)
    return i < n ? rank_key(wt[i], ps[i], a.sinks, from, nan) : 0u;
  };
  uint32_t kept[kKeep];
#pragma unroll
  for (int j = 0; j < kKeep; ++j) kept[j] = j < per ? read(j) : 0u;
  // f(key, slot) for each of the warp's rows of slots in order
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (j < per) f(kept[j], i0 + 32 * j);
    for (int j = kKeep; j < per; ++j) f(read(j), i0 + 32 * j);
  };
  __syncthreads();                        // the histograms are empty
  // ---- the keep-th largest key, digit by digit
  uint32_t prefix = 0, left = keep, same = 0;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
    uint32_t* const hist = sh.hist[round];
    uint32_t must = 0;
    each([&](uint32_t k, int i) {
      const bool in = i < n && (round == 0 || (k >> (shift + bits)) == prefix);
      // (slots that must stay are many of one key: counted apart)
      if (in && k != ~0u) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
      if (in && k == ~0u) ++must;
    });
    must = __reduce_add_sync(0xffffffffu, must);
    if (lane == 0 && must) atomicAdd(&hist[(1u << bits) - 1], must);
    cl.sync();
    // thread t holds bins kBins - 1 - 2 t and the one below, of all blocks
    uint32_t x0 = 0, x1 = 0;
    for (int c = 0; c < C; ++c) {
      const uint2 v = *reinterpret_cast<const uint2*>(
          cl.map_shared_rank(hist, c) + kBins - 2 - 2 * tid);
      x0 += v.y;
      x1 += v.x;
    }
    uint32_t incl = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int unused;
    const uint32_t above =
        warps_prefix(__shfl_sync(0xffffffffu, incl, 31), sh.warp_sum[round & 1], unused) + incl -
        x0 - x1;
    if (above < left && left <= above + x0 + x1) {   // one thread
      const bool first = left <= above + x0;
      sh.prefix = prefix << bits | (kBins - 1 - 2 * tid - (first ? 0 : 1));
      sh.left = left - above - (first ? 0 : x0);
      sh.count = first ? x0 : x1;
    }
    __syncthreads();
    prefix = sh.prefix;
    left = sh.left;
    same = sh.count;
  }
  if (nan) flag(a.status, DS_DEV_BAD_VALUE);
  // `left` of the `same` slots with key `prefix` stay, the lower ones
  int ties0 = 0;                          // ties before this warp's slots
  if (left < same) {
    int ties = 0, total;
    each([&](uint32_t k, int i) {
      ties += __popc(__ballot_sync(0xffffffffu, i < n && k == prefix));
    });
    ties0 = warps_prefix(ties, sh.warp_sum[1], total);
    if (tid == 0) sh.block_sum[0][0] = total;
    cl.sync();
    for (int c = 0; c < rank; ++c) ties0 += *cl.map_shared_rank(&sh.block_sum[0][0], c);
  }
  const uint32_t below = (1u << lane) - 1;
  // the row's slots that stay (ballot), with the ties counted on
  auto stays = [&](uint32_t k, int i, int& seen) {
    const uint32_t tie = __ballot_sync(0xffffffffu, i < n && k == prefix);
    const bool stay = i < n && (k > prefix || ((tie >> lane & 1) &&
                                               seen + __popc(tie & below) < (int)left));
    seen += __popc(tie);
    return stay;
  };
  int come = 0, freed = 0, seen = ties0;
  each([&](uint32_t k, int i) {
    const bool stay = stays(k, i, seen);
    come += __popc(__ballot_sync(0xffffffffu, stay && i >= keep));
    freed += __popc(__ballot_sync(0xffffffffu, !stay && i < keep));
  });
  int total;
  int come0 = warps_prefix(come, sh.warp_sum[0], total);
  if (tid == 0) sh.block_sum[1][0] = total;
  __syncthreads();
  int freed0 = warps_prefix(freed, sh.warp_sum[1], total);
  if (tid == 0) sh.block_sum[1][1] = total;
  cl.sync();
  int all = 0;
  for (int c = 0; c < C; ++c) {
    const int* x = cl.map_shared_rank(&sh.block_sum[1][0], c);
    if (c < rank) {
      come0 += x[0];
      freed0 += x[1];
    }
    all += x[0];
  }
  int32_t* src = a.src + (int64_t)seg * a.moves;
  int32_t* dst = a.dst + (int64_t)seg * a.moves;
  seen = ties0;
  each([&](uint32_t k, int i) {
    const bool stay = stays(k, i, seen);
    const uint32_t c = __ballot_sync(0xffffffffu, stay && i >= keep);
    const uint32_t f = __ballot_sync(0xffffffffu, !stay && i < keep);
    if (c >> lane & 1) src[come0 + __popc(c & below)] = i;
    if (f >> lane & 1) dst[freed0 + __popc(f & below)] = i;
    come0 += __popc(c);
    freed0 += __popc(f);
    if (stay && i < keep) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
  });
  if (tid == 0 && rank == 0) a.count[seg] = all;
  cl.sync();                              // others may still read this block's sums
}

// A warp takes 32 moves of a segment and one kv head: a lane looks up one
// move's places, then the rows go four at a time, a lane 16 bytes of K or V.
template <int D>
__global__ void __launch_bounds__(256) move(const KArgs a) {
  constexpr int VECS = D / 8;             // 16-byte vectors of a head's row
  constexpr int AT = 32 / (2 * VECS);     // moves (their K and V) of a warp at once
  constexpr int BATCH = 8;                // loads on their way
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int lane = threadIdx.x & 31;
  const int heads = a.slot_heads == 1 ? a.cache.num_kv_heads : 1;
  const int count = a.count[seg];
  const int64_t items = (int64_t)((count + 31) / 32) * heads;
  const int32_t* src = a.src + (int64_t)seg * a.moves;
  const int32_t* dst = a.dst + (int64_t)seg * a.moves;
  uint16_t* const pool = lane % (2 * VECS) < VECS ? a.cache.pool[0] : a.cache.pool[1];
  const int col = lane % VECS * 8, mine = lane / (2 * VECS);
  for (int64_t it = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); it < items;
       it += (int64_t)gridDim.y * 8) {
    const int i0 = (int)(it / heads) * 32, i = i0 + lane;
    const int h = a.slot_heads == 1 ? (int)(it % heads) : w;
    int64_t from = -1, to = -1;           // -1: nothing to move
    if (i < count) {
      const int s = src[i], d = dst[i];
      if (it % heads == 0) {
        const int64_t base = (int64_t)seg * a.slot_stride;
        (a.weights_out ? a.weights_out : a.weights)[base + d] = a.weights[base + s];
        (a.positions_out ? a.positions_out : a.positions)[base + d] = a.positions[base + s];
      }
      const int pf = slot_page(a.cache, b, s), pt = slot_page(a.cache, b, d);
      if (pf >= 0 && pt >= 0) {
        from = slot_at(a.cache, pf, s) + (int64_t)h * a.cache.head_stride;
        to = slot_at(a.cache, pt, d) + (int64_t)h * a.cache.head_stride;
      } else {
        flag(a.status, DS_DEV_BAD_PAGE);
      }
    }
    const int rows = min(32, count - i0);
    for (int r0 = 0; r0 < rows; r0 += AT * BATCH) {
      uint4 x[BATCH];
      int64_t at[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int r = (r0 + k * AT + mine) & 31;
        const int64_t f = __shfl_sync(0xffffffffu, from, r);
        at[k] = __shfl_sync(0xffffffffu, to, r);
        if (r0 + k * AT + mine >= rows) at[k] = -1;
        if (at[k] >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(pool + f + col));
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (at[k] >= 0) *reinterpret_cast<uint4*>(pool + at[k] + col) = x[k];
    }
  }
}

// Blocks of a segment's cluster: as many as fill the machine (two blocks of
// 1024 threads on each of 152 SMs), but 2048 slots or more to each, where
// another block costs more than it saves.
int cluster_size(int segs, int64_t slots) {
  int c = 1;
  while (c < 8 && (int64_t)segs * 2 * c <= 304 && slots / (2 * c) >= 2048) c *= 2;
  // more while a block's slots do not fit in its registers
  while (c < 8 && slots > (int64_t)c * kKeep * kThreads) c *= 2;
  return c;
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
  const int cluster = cluster_size(segs, a.cache.slots);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select, a);
  if (e != cudaSuccess || L.moves == 0) return e;
  // eight blocks an SM, as far as there can be moves
  const int64_t warps = (L.moves + 31) / 32 * (g.slot_heads == 1 ? g.num_kv_heads : 1);
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8,
                                                               152 * 8 / segs + 1));
  return launch_dependent(g.head_dim == 128 ? move<128> : move<64>, dim3(segs, rows), dim3(256),
                          0, stream, a);
}

}  // namespace ds
