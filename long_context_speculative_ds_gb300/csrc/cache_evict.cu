// Eviction from the draft's cache by accumulated attention weight, in place
// (include/ds.h, ds_cache_evict).
//
// A slot's rank is a 32-bit key: all ones for the first and recent tokens,
// else the weight's bits in an order that is the floats' (a NaN 1).  `select`
// finds the budget-th largest key of a segment (a sequence's slot head) digit
// by digit, how many of that very key stay (the lower slots), and lists the
// kept slots behind the budget and the free ones below it, both ascending;
// `move` (or `select` itself, where there are few) copies one to the other.  No
// move's source is another's target (sources lie behind the budget, targets below
// it), so it works in place, and moves no more than has to move.
//
// The moves are bound by memory: 6.2 TB/s for rows of 256 bytes here and there
// (heads by themselves), 6.5 where a token's heads move together.  The selection
// is bound by the latency of its passes over the keys in shared memory and of the
// cluster's barriers: 32 of 101 us for 16 segments of 128K slots cut to 32K, 16
// of 66 for eight of 18K cut to half; one slot of 2,049 4.1 us in all, one launch.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <climits>

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
  int32_t alone;                 // no second kernel: `select` moves the rows itself
  uint32_t* status;
};

// Segments that can have no more moves than this are moved by `select`: a token
// given up per call by a cache with a few slots above its budget saves a launch.
// One slot of 2,049, in a graph: 4.1 us in one launch and 5.9 in two (heads that
// move together 4.5 and 6.0), of 18,433 5.8 and 7.4, whatever the room.  But all the
// moves that there is room for take, 32 of them, 8.0 and 9.6 us (together 11.3 and
// 9.0), 64 8.7 and 9.8 (15.9 and 9.8), 128 9.8 and 10.0 (24 and 9.8), 256 11.9 and
// 10.1 (38 and 10.0).  The room, not the length, is what the host knows.
constexpr int kFewMoves = 64;

// (without branches, so that the loads of many slots go out together)
DS_DEV uint32_t rank_key(float w, int pos, int sinks, int recent_from, bool& nan) {
  const bool must = pos < sinks || pos >= recent_from, none = w != w;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
  // (the largest key of a weight, +inf, is 0xff800000)
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  nan |= none && !must;
  return must ? ~0u : none ? 1u : k;      // (-inf is 0x007fffff; 0: no slot)
}

// Moves m0 .. m0 + moves - 1 (at most 32) of a segment, by a warp: a lane looks up
// one move's places, then the rows go BATCH (twice as many at 64-wide heads) at
// once, a lane 16 bytes of K or V, a move's heads one behind the other.
template <int D, int BATCH>
DS_DEV void move_rows(const KArgs& a, const int seg, const int64_t m0, const int moves) {
  constexpr int VECS = D / 8;             // 16-byte vectors of a head's row
  constexpr int AT = 32 / (2 * VECS);     // rows (their K and V) of a warp at once
  const int b = seg / a.slot_heads, lane = threadIdx.x & 31;
  const bool shared = a.slot_heads == 1;
  const int heads = shared ? a.cache.num_kv_heads : 1, h0 = shared ? 0 : seg % a.slot_heads;
  uint16_t* const pool = lane % (2 * VECS) < VECS ? a.cache.pool[0] : a.cache.pool[1];
  const int col = lane % VECS * 8, mine = lane / (2 * VECS);
  int64_t from = -1, to = -1;             // -1: nothing to move
  if (lane < moves) {
    const int s = a.src[(int64_t)seg * a.moves + m0 + lane];
    const int d = a.dst[(int64_t)seg * a.moves + m0 + lane];
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
  __syncwarp();
  const int rows = moves * heads;
  int m = mine / heads, h = mine % heads; // of this lane's next row
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

// A cluster of blocks per segment; its rows of 32 slots in equal runs to the
// warps, one behind the other.  Keys of a warp's first rows stay in shared
// memory, as many as the launch has room for; beyond (segments of more than some
// 400,000 slots, 800,000 for few of them) they are formed anew from memory.
constexpr int kMaxKeyBytes = 200 * 1024;
constexpr int kBins = 2048;               // of a digit: 11, 11 and 10 bits

struct Shared {
  uint32_t hist[3][kBins];
  uint32_t part[3][32];                   // sums of 64 bins
  int2 warp_sum[2][32];
  int2 block_sum[2];                      // of this block: ties; slots that come, that are freed
  uint32_t prefix, left, count;
  unsigned long long least[32];           // of each warp
};

// Exclusive prefix of two values per warp (the same on all its lanes) over the
// block's NW warps, and the totals.
template <int NW>
DS_DEV int2 warps_prefix(int2 v, int2* s_warp, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  const int2 w = lane < NW ? s_warp[lane] : make_int2(0, 0);
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

DS_DEV void few_rows(const KArgs& a, const int seg, const int64_t m0, const int moves) {
  if (a.head_dim == 128) move_rows<128, 4>(a, seg, m0, moves);
  else move_rows<64, 4>(a, seg, m0, moves);
}

// Mask of the first k of 32.
DS_DEV uint32_t first_bits(int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1; }

// T threads; clusters of up to MAXC blocks (see shape_of)
template <int T, int MAXC>
__global__ void __launch_bounds__(T, 1024 / T) select(const KArgs a, const int room) {
  constexpr int NW = T / 32;
  extern __shared__ uint32_t s_keys[];    // [warp][room rows][32]
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins / 4; i += T)
    reinterpret_cast<uint4*>(&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  auto meet = [&] {                       // a barrier of the cluster
    if (C == 1) __syncthreads(); else cl.sync();
  };
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x / C, b = seg / a.slot_heads, w = seg % a.slot_heads;
  const int64_t base = (int64_t)seg * a.slot_stride;
  const float* wt = a.weights + base;
  const int32_t* ps = a.positions + base;
  // Eight rows' loads on their way together, the next eight's behind them.  A
  // segment of one block has its rows dealt by the slots there are, so that the
  // first ones' loads go out beside the length's.
  float x[8];
  int p[8];
  auto fetch = [&](const int slot0, const int end) {
    const int i0 = slot0 + lane;
    const float* const xs = wt + i0;
    const int32_t* const qs = ps + i0;
    if (slot0 + 32 * 8 <= end) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = xs[32 * j];
        p[j] = qs[32 * j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < end) {
          x[j] = xs[32 * j];
          p[j] = qs[32 * j];
        }
    }
  };
  const bool single = T == 256 && C == 1;
  const int len = a.lens[b], next = a.next_positions[b];
  int per = single ? ((int)a.cache.slots + 32 * NW - 1) / (32 * NW) : 0;   // rows of a warp
  if (single) fetch(warp * per * 32, (int)a.cache.slots);
  const int n = checked_len(len, a.cache.slots, a.status, tid == 0 && rank == 0 && w == 0);
  const bool cut = n > a.limit;
  const int keep = cut ? a.budget : n;
  if (tid == 0 && rank == 0 && w == 0) a.new_lens[b] = cut ? keep : len;
  float* wo = a.weights_out ? a.weights_out + base : nullptr;
  int32_t* po = a.positions_out ? a.positions_out + base : nullptr;
  if (!cut) {                             // (the whole cluster)
    if (tid == 0 && rank == 0) a.count[seg] = 0;
    for (int i = rank * T + tid; i < n; i += C * T) {
      if (wo) wo[i] = wt[i];
      if (po) po[i] = ps[i];
    }
    return;
  }
  const int from = (int)max((int64_t)next - a.recent, (int64_t)INT_MIN);
  if (!single) per = ((n + 31) / 32 + C * NW - 1) / (C * NW);
  const int row0 = (rank * NW + warp) * per * 32;       // slot of the warp's first row
  bool nan = false;
  auto read = [&](int j) {
    const int i = row0 + 32 * j + lane, at = min(i, n - 1);
    const uint32_t k = rank_key(wt[at], ps[at], a.sinks, from, nan);
    return i < n ? k : 0u;
  };
  uint32_t* const mine = s_keys + warp * room * 32 + lane;
  const int kept = min(per, room);
  // What is below the budget goes into arrays of its own at once (the moves
  // overwrite the slots that are given up).
  if (!single) fetch(row0, n);
  for (int j0 = 0; j0 < per; j0 += 8) {
    const int i0 = row0 + 32 * j0 + lane;
    uint32_t k[8];
    if ((wo || po) && row0 + 32 * j0 < keep) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < per && i0 + 32 * j < keep) {
          if (wo) wo[i0 + 32 * j] = x[j];
          if (po) po[i0 + 32 * j] = p[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = j0 + j < per && i0 + 32 * j < n;
      bool none = false;
      k[j] = rank_key(x[j], p[j], a.sinks, from, none);
      nan |= none && in;
      if (!in) k[j] = 0u;
    }
    if (j0 + 8 < per) fetch(row0 + 32 * (j0 + 8), n);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < kept) mine[32 * (j0 + j)] = k[j];
  }
  // f(key, row) for each of the warp's rows in order
  auto each = [&](auto f) {
#pragma unroll 8
    for (int j = 0; j < kept; ++j) f(mine[32 * j], j);
    for (int j = kept; j < per; ++j) f(read(j), j);
  };
  // ---- one slot to give up, as a cache at its budget does every token: the
  // lightest, of equal ones the last; the one behind the budget takes its place
  // (a call on 2,049 slots 6.3 us instead of 11.4, and 4.1 without a second kernel)
  if (n - keep == 1) {
    unsigned long long least = ~0ull;     // key, then slot from the end
    each([&](uint32_t k, int j) {
      const unsigned long long x =
          (unsigned long long)k << 32 | (uint32_t)~(row0 + 32 * j + lane);
      if (k != 0u) least = min(least, x);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) sh.least[warp] = least;
    meet();
    if (warp == 0 && rank == 0) {
      least = ~0ull;
      for (int c = 0; c < C; ++c)
        if (lane < NW) least = min(least, cl.map_shared_rank(&sh.least[0], c)[lane]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      const int gone = (int)~(uint32_t)least;
      if (lane == 0) {
        a.count[seg] = gone < keep;
        a.src[(int64_t)seg * a.moves] = keep;
        a.dst[(int64_t)seg * a.moves] = gone;
      }
      __syncwarp();
      if (a.alone && gone < keep) few_rows(a, seg, 0, 1);
    }
    if (nan) flag(a.status, DS_DEV_BAD_VALUE);
    if (C > 1) cl.sync();                 // others may still be read
    return;
  }
  __syncthreads();                        // the histograms are empty
  // ---- the keep-th largest key, digit by digit
  uint32_t prefix = 0, left = keep, same = 0;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
    uint32_t* const hist = sh.hist[round];
    const uint32_t mask = (1u << bits) - 1;
    uint32_t must = 0;
    each([&](uint32_t k, int) {
      // (slots that must stay are many of one key: counted apart)
      const bool in = k != 0u && (round == 0 || (k >> (shift + bits)) == prefix);
      if (in && k != ~0u) atomicAdd(&hist[(k >> shift) & mask], 1u);
      must += in && k == ~0u;
    });
    must = __reduce_add_sync(0xffffffffu, must);
    if (lane == 0 && must) atomicAdd(&hist[mask], must);
    __syncthreads();
    // sums of 64 bins first: blocks read one another's 32 of these and 64 bins
    // (all bins of 16 blocks took 5 us a digit)
    for (int c = warp; c < 32; c += NW) {
      const uint2 v = *reinterpret_cast<const uint2*>(hist + 64 * c + 2 * lane);
      const uint32_t x = __reduce_add_sync(0xffffffffu, v.x + v.y);
      if (lane == 0) sh.part[round][c] = x;
    }
    meet();
    if (warp == 0) {
      uint32_t x = sh.part[round][31 - lane];   // lane l: part 31 - l, of all blocks
      if (C > 1) {                        // (their loads on their way together)
        uint32_t v[MAXC];
#pragma unroll
        for (int c = 1; c < MAXC; ++c)
          v[c] = cl.map_shared_rank(&sh.part[round][0], (rank + c) & (C - 1))[31 - lane];
#pragma unroll
        for (int c = 1; c < MAXC; ++c) x += c < C ? v[c] : 0;
      }
      uint32_t incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int at = __ffs(__ballot_sync(0xffffffffu, left <= incl)) - 1;   // the first that reaches it
      const uint32_t above = __shfl_sync(0xffffffffu, incl - x, at);
      const int bin0 = 64 * (31 - at) + 62 - 2 * lane;  // lane's two bins, from the top down
      const uint2 own = *reinterpret_cast<const uint2*>(hist + bin0);
      uint32_t x0 = own.y, x1 = own.x;
      if (C > 1) {
        uint2 v[MAXC];
#pragma unroll
        for (int c = 1; c < MAXC; ++c)
          v[c] = *reinterpret_cast<const uint2*>(
              cl.map_shared_rank(hist, (rank + c) & (C - 1)) + bin0);
#pragma unroll
        for (int c = 1; c < MAXC; ++c) {
          x0 += c < C ? v[c].y : 0;
          x1 += c < C ? v[c].x : 0;
        }
      }
      incl = x0 + x1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      incl += above;
      at = __ffs(__ballot_sync(0xffffffffu, left <= incl)) - 1;
      if (lane == at) {
        const uint32_t over = incl - x0 - x1;
        const bool first = left <= over + x0;
        sh.prefix = prefix << bits | (bin0 + (first ? 1 : 0));
        sh.left = left - over - (first ? 0 : x0);
        sh.count = first ? x0 : x1;
      }
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
  int ties0 = 0;                          // ties before this warp's slots
  if (ties) {
    int2 v = make_int2(0, 0), total;
    each([&](uint32_t k, int) { v.x += __popc(__ballot_sync(0xffffffffu, k == prefix)); });
    ties0 = warps_prefix<NW>(v, sh.warp_sum[1], total).x;
    if (tid == 0) sh.block_sum[0] = total;
    meet();
    ties0 += __reduce_add_sync(
        0xffffffffu, lane < rank ? cl.map_shared_rank(&sh.block_sum[0], lane)->x : 0);
  } else if (left > 0) {
    --prefix;                             // (all at it stay; 0 cannot be)
  }
  const uint32_t below = (1u << lane) - 1;
  // the row's slots that stay, as a mask
  auto stays = [&](uint32_t k, int& seen) {
    uint32_t m = __ballot_sync(0xffffffffu, k > prefix);
    if (ties) {
      const uint32_t at = __ballot_sync(0xffffffffu, k == prefix);
      m |= __ballot_sync(0xffffffffu, k == prefix && seen + __popc(at & below) < (int)left);
      seen += __popc(at);
    }
    return m;
  };
  // (a row's mask takes the place of its first key)
  int2 sum = make_int2(0, 0), total;
  int seen = ties0, seen_kept = ties0;
  each([&](uint32_t k, int j) {
    const uint32_t m = stays(k, seen), low = first_bits(keep - row0 - 32 * j);
    sum.x += __popc(m & ~low);
    sum.y += __popc(~m & low);
    if (j < kept) {
      if (lane == 0) mine[32 * j] = m;
      seen_kept = seen;
    }
  });
  __syncwarp();
  int2 before = warps_prefix<NW>(sum, sh.warp_sum[0], total);
  if (tid == 0) sh.block_sum[1] = total;
  meet();
  const int2 other =
      lane < C ? *cl.map_shared_rank(&sh.block_sum[1], lane) : make_int2(0, 0);
  const int all = __reduce_add_sync(0xffffffffu, other.x);
  before.x += __reduce_add_sync(0xffffffffu, lane < rank ? other.x : 0);
  before.y += __reduce_add_sync(0xffffffffu, lane < rank ? other.y : 0);
  int32_t* src = a.src + (int64_t)seg * a.moves;
  int32_t* dst = a.dst + (int64_t)seg * a.moves;
  src += before.x;
  dst += before.y;
  auto list = [&](uint32_t m, int j) {
    const int i = row0 + 32 * j;
    const uint32_t low = first_bits(keep - i), come = m & ~low, free = ~m & low;
    if (come >> lane & 1) src[__popc(come & below)] = i + lane;
    if (free >> lane & 1) dst[__popc(free & below)] = i + lane;
    src += __popc(come);
    dst += __popc(free);
  };
#pragma unroll 8
  for (int j = 0; j < kept; ++j) list(mine[32 * j - lane], j);
  seen = seen_kept;
  for (int j = kept; j < per; ++j) list(stays(read(j), seen), j);
  if (tid == 0 && rank == 0) a.count[seg] = all;
  if (C > 1) cl.sync();                   // others may still read this block's sums
  if (a.alone) {
    if (C == 1) __syncthreads();          // the lists are whole
    const int share = (all + C * NW - 1) / (C * NW), m0 = (rank * NW + warp) * share;
    if (m0 < all) few_rows(a, seg, m0, min(share, all - m0));
  }
}

// The moves of a segment go 32 kv heads' rows to a warp at a time (32 moves of
// one head, or 4 of eight that move together).
template <int D>
__global__ void __launch_bounds__(256) move(const KArgs a, const int per) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int seg = blockIdx.x, count = a.count[seg];
  for (int64_t m0 = ((int64_t)blockIdx.y * 8 + (threadIdx.x >> 5)) * per; m0 < count;
       m0 += (int64_t)gridDim.y * 8 * per)
    move_rows<D, 8>(a, seg, m0, (int)min((int64_t)per, count - m0));
}

// Threads of a block and blocks of a segment's cluster.  Segments of up to 4,096
// slots take one block of 256 threads, whose barriers cost less.  Longer ones
// take up to eight blocks of 512, as many as fill the machine, but with 2,048
// slots or more to each, and more while a block's keys do not fit beside two
// others'.  Few segments beyond 65,536 slots take 16 blocks of 256: cut to half,
// 8 of 128K 48 us instead of 54, 16 77 instead of 82, 20 92 instead of 97, but 24
// 121 instead of 110; 8 of 70,000 31 instead of 34, 16 48.6 instead of 49.3, 20 57.3
// instead of 56.7, 32 89 instead of 80; 8 of 40,000 21.3 instead of 20.5.  Blocks of which only one fits an SM leave no place
// for 16 clusters at once (two waves, 44 us for the selection instead of 35).
struct Shape {
  int threads, cluster;
};
Shape shape_of(int segs, int64_t slots, bool sixteen) {
  if (slots <= 4096) return {256, 1};
  if (slots > 65536 && segs <= 16 && sixteen) return {256, 16};
  int c = 1;
  while (c < 8 && (int64_t)segs * 2 * c <= 152 && slots / (2 * c) >= 2048) c *= 2;
  while (c < 8 && slots * 4 > (int64_t)c * kMaxKeyBytes / 3) c *= 2;
  return {512, c};
}

// Whether the current device can place a cluster of 16 blocks with all the shared
// memory that they may ask for: not every one has 16 SMs side by side.  What a
// device has does not change, so it is asked once for each.
bool sixteen_fit() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];              // 0: not yet, 1: no, 2: yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < kDevices && known[dev].load(std::memory_order_relaxed))
    return known[dev].load(std::memory_order_relaxed) == 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = kMaxKeyBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*const kernel)(KArgs, int) = select<256, 16>;
  int clusters = 0;
  const bool fit =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
          cudaSuccess &&
      allow_smem(kernel, kMaxKeyBytes) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters >= 1;
  if (!fit) cudaGetLastError();
  if (dev < kDevices) known[dev].store(fit ? 2 : 1, std::memory_order_relaxed);
  return fit;
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
  a.alone = L.moves <= kFewMoves;
  const int segs = g.batch * g.slot_heads;
  const Shape shape = shape_of(segs, a.cache.slots, a.cache.slots > 65536 && sixteen_fit());
  const int cluster = shape.cluster, warps_of = shape.threads / 32;
  void (*const kernel)(KArgs, int) = shape.threads == 256 ? select<256, 16> : select<512, 8>;
  if (cluster > 8) {                      // more than every device has to take, sixteen_fit asked
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  // rows of 32 keys that a warp has room for
  const int64_t need = (a.cache.slots + 32 * cluster * warps_of - 1) / (32 * cluster * warps_of);
  const int room = (int)std::min<int64_t>(need, kMaxKeyBytes / (128 * warps_of));
  const size_t smem = (size_t)room * 128 * warps_of;
  // (always the most, not this call's share: the permission is the kernel's, and
  // another thread may be between its own and its launch)
  cudaError_t e = allow_smem(kernel, kMaxKeyBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * cluster));
  cfg.blockDim = dim3(warps_of * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, room);
  if (e != cudaSuccess || a.alone) return e;
  // Rows of a warp at a time: 8, that go at once, up to 32 when there are enough to
  // fill the machine with warps all the same; and eight blocks an SM as far as
  // there can be moves.
  const int heads = g.slot_heads == 1 ? g.num_kv_heads : 1;
  const int64_t fill = (int64_t)segs * L.moves * heads / (152 * 24);
  const int per = (int)std::max<int64_t>(1, std::min<int64_t>(32, std::max<int64_t>(8, fill)) / heads);
  const int64_t warps = (L.moves + per - 1) / per;
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8,
                                                               152 * 8 / segs + 1));
  return launch_dependent(g.head_dim == 128 ? move<128> : move<64>, dim3(segs, rows), dim3(256),
                          0, stream, a, per);
}

}  // namespace ds
