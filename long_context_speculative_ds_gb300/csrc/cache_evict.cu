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

// (without branches, so that the loads of many slots go out together)
DS_DEV uint32_t rank_key(float w, int pos, int sinks, int64_t recent_from, bool& nan) {
  const bool must = pos < sinks || pos >= recent_from, none = w != w;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
  // (the largest key of a weight, +inf, is 0xff800000)
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  nan |= none && !must;
  return must ? ~0u : none ? 0u : k;
}

// A cluster of blocks per segment, a contiguous part of its slots to each, and
// of that a contiguous part to each warp: its slots i0 + 32 j + lane, j < per.
// Keys of the first kKeep of these stay in registers; beyond (segments of more
// than kKeep 1024 slots a block) they are formed anew from memory.
constexpr int kKeep = 16;
constexpr int kBins = 2048;               // of a digit: 11, 11 and 10 bits

struct Shared {
  uint32_t hist[3][kBins];
  int2 warp_sum[2][32];
  int2 block_sum[2];                      // of this block: ties; slots that come, that are freed
  uint32_t prefix, left, count;
};

// Exclusive prefix of two values per warp (the same on all its lanes) over the
// block's warps, and the totals.
DS_DEV int2 warps_prefix(int2 v, int2* s_warp, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  const int2 w = s_warp[lane];
  int2 incl = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o);
    const int y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  total.x = __shfl_sync(0xffffffffu, incl.x, 31);
  total.y = __shfl_sync(0xffffffffu, incl.y, 31);
  return make_int2(__shfl_sync(0xffffffffu, incl.x - w.x, warp),
                   __shfl_sync(0xffffffffu, incl.y - w.y, warp));
}

__global__ void __launch_bounds__(kThreads) select(const KArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  auto meet = [&] {                       // a barrier of the cluster
    if (C == 1) __syncthreads(); else cl.sync();
  };
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
  auto read = [&](int j) {                // (slots past the end: some key, never looked at)
    const int i = min(i0 + 32 * j, n - 1);
    return rank_key(__ldg(wt + i), __ldg(ps + i), a.sinks, from, nan);
  };
  uint32_t kept[kKeep];
#pragma unroll
  for (int j0 = 0; j0 < kKeep; j0 += 8)
    if (j0 < per) {
      float w[8];
      int p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = min(i0 + 32 * (j0 + j), n - 1);
        w[j] = __ldg(wt + i);
        p[j] = __ldg(ps + i);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) kept[j0 + j] = rank_key(w[j], p[j], a.sinks, from, nan);
    }
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
    meet();
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
    int2 unused;
    const int2 whole = make_int2(__shfl_sync(0xffffffffu, incl, 31), 0);
    const uint32_t above =
        warps_prefix(whole, sh.warp_sum[round & 1], unused).x + incl - x0 - x1;
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
    if (left == same && round < 2) {      // all of the bin stay: what lies above it and these
      prefix = (prefix << shift) - 1;     // (bin 0 cannot: more slots than stay)
      left = same = 0;
      break;
    }
  }
  if (nan) flag(a.status, DS_DEV_BAD_VALUE);
  // above `prefix` all stay, and `left` of the `same` slots at it, the lower ones
  const bool ties = left < same;
  int ties0 = 0;                 // ties before this warp's slots
  if (ties) {
    int2 v = make_int2(0, 0), total;
    each([&](uint32_t k, int i) {
      v.x += __popc(__ballot_sync(0xffffffffu, i < n && k == prefix));
    });
    ties0 = warps_prefix(v, sh.warp_sum[1], total).x;
    if (tid == 0) sh.block_sum[0] = total;
    meet();
    for (int c = 0; c < rank; ++c) ties0 += cl.map_shared_rank(&sh.block_sum[0], c)->x;
  } else if (left > 0) {
    --prefix;                             // (all at it stay; 0 cannot be)
  }
  const uint32_t below = (1u << lane) - 1;
  auto stays = [&](uint32_t k, int i, int& seen) {
    bool stay = i < n && k > prefix;
    if (ties) {
      const bool tie = i < n && k == prefix;
      const uint32_t all = __ballot_sync(0xffffffffu, tie);
      stay |= tie && seen + __popc(all & below) < (int)left;
      seen += __popc(all);
    }
    return stay;
  };
  int2 sum = make_int2(0, 0), total;
  int seen = ties0;
  each([&](uint32_t k, int i) {
    const bool stay = stays(k, i, seen);
    sum.x += __popc(__ballot_sync(0xffffffffu, stay && i >= keep));
    sum.y += __popc(__ballot_sync(0xffffffffu, !stay && i < keep));
  });
  int2 before = warps_prefix(sum, sh.warp_sum[0], total);
  if (tid == 0) sh.block_sum[1] = total;
  meet();
  int all = 0;
  for (int c = 0; c < C; ++c) {
    const int2 x = *cl.map_shared_rank(&sh.block_sum[1], c);
    if (c < rank) {
      before.x += x.x;
      before.y += x.y;
    }
    all += x.x;
  }
  int32_t* src = a.src + (int64_t)seg * a.moves;
  int32_t* dst = a.dst + (int64_t)seg * a.moves;
  seen = ties0;
  each([&](uint32_t k, int i) {
    const bool stay = stays(k, i, seen);
    const uint32_t c = __ballot_sync(0xffffffffu, stay && i >= keep);
    const uint32_t f = __ballot_sync(0xffffffffu, !stay && i < keep);
    if (c >> lane & 1) src[before.x + __popc(c & below)] = i;
    if (f >> lane & 1) dst[before.y + __popc(f & below)] = i;
    before.x += __popc(c);
    before.y += __popc(f);
    if (stay && i < keep) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
  });
  if (tid == 0 && rank == 0) a.count[seg] = all;
  if (C > 1) cl.sync();                   // others may still read this block's sums
}

// A warp takes the moves of a segment 32 kv heads' rows at a time (32 moves of
// one head, or 4 of eight that move together): a lane looks up one move's
// places, then the rows go eight (sixteen) at once, a lane 16 bytes of K or V,
// a move's heads one behind the other.
template <int D>
__global__ void __launch_bounds__(256) move(const KArgs a, const int per) {
  constexpr int VECS = D / 8;             // 16-byte vectors of a head's row
  constexpr int AT = 32 / (2 * VECS);     // rows (their K and V) of a warp at once
  constexpr int BATCH = 8;                // loads on their way
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int lane = threadIdx.x & 31;
  const bool shared = a.slot_heads == 1;
  const int heads = shared ? a.cache.num_kv_heads : 1, h0 = shared ? 0 : w;
  const int count = a.count[seg];
  const int32_t* src = a.src + (int64_t)seg * a.moves;
  const int32_t* dst = a.dst + (int64_t)seg * a.moves;
  uint16_t* const pool = lane % (2 * VECS) < VECS ? a.cache.pool[0] : a.cache.pool[1];
  const int col = lane % VECS * 8, mine = lane / (2 * VECS);
  for (int64_t m0 = ((int64_t)blockIdx.y * 8 + (threadIdx.x >> 5)) * per; m0 < count;
       m0 += (int64_t)gridDim.y * 8 * per) {
    const int moves = (int)min((int64_t)per, count - m0);
    int64_t from = -1, to = -1;           // -1: nothing to move
    if (lane < moves) {
      const int s = src[m0 + lane], d = dst[m0 + lane];
      const int64_t base = (int64_t)seg * a.slot_stride;
      (a.weights_out ? a.weights_out : a.weights)[base + d] = a.weights[base + s];
      (a.positions_out ? a.positions_out : a.positions)[base + d] = a.positions[base + s];
      const int pf = slot_page(a.cache, b, s), pt = slot_page(a.cache, b, d);
      if (pf >= 0 && pt >= 0) {
        from = slot_at(a.cache, pf, s) + (int64_t)h0 * a.cache.head_stride;
        to = slot_at(a.cache, pt, d) + (int64_t)h0 * a.cache.head_stride;
      } else {
        flag(a.status, DS_DEV_BAD_PAGE);
      }
    }
    const int rows = moves * heads;
    int m = mine / heads, h = mine % heads;       // of this lane's next row
    for (int r0 = 0; r0 < rows; r0 += AT * BATCH) {
      uint4 x[BATCH];
      int64_t at[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int64_t f = __shfl_sync(0xffffffffu, from, m & 31);
        at[k] = __shfl_sync(0xffffffffu, to, m & 31);
        const int64_t off = (int64_t)h * a.cache.head_stride + col;
        if (r0 + k * AT + mine >= rows || at[k] < 0)
          at[k] = -1;
        else
          at[k] += off;
        if (at[k] >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(pool + f + off));
        for (h += AT; h >= heads; h -= heads) ++m;
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (at[k] >= 0) *reinterpret_cast<uint4*>(pool + at[k]) = x[k];
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
  // moves of a warp at a time, and eight blocks an SM as far as there can be moves
  const int per = std::max(1, 32 / (g.slot_heads == 1 ? g.num_kv_heads : 1));
  const int64_t warps = (L.moves + per - 1) / per;
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8,
                                                               152 * 8 / segs + 1));
  return launch_dependent(g.head_dim == 128 ? move<128> : move<64>, dim3(segs, rows), dim3(256),
                          0, stream, a, per);
}

}  // namespace ds
