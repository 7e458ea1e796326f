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
//
// Bound by the stream of K and V.  With 32 query heads on 8 of 128: one token
// over 128K 97 us, the split pass 86 of them (537 MB, 6.2 TB/s of the 6.8 that a
// copy reaches; without weights the call takes 85); 96 ragged contexts of 33 to
// 8K 75 us (457 MB, 6.1 TB/s); eight compact caches of 9K to 18K 82 us; 512
// slots with 4 heads of 64 on 2 8.0 us, two launches of four dependent reads
// each.  Logits cost 4 bytes a slot and query head, written and read: 3 % of the
// bytes at 4 query heads a kv head, a quarter at 16 (128K: 122 us, 87 without
// weights).
//
// Split pass: blocks of four warps that compute and one that loads, two blocks
// an SM, each with a ring of three (six at 64-wide heads) tiles of 64 slots.
// The loader brings a tile's K and V as copies of 16 slots of one head through
// the page table, works out the pieces, and runs ahead over their ends, so that
// the stream does not stop where one segment ends and the next begins; the other
// block's ring covers what is left.  (One block of eight warps and six tiles an
// SM took 88 us for the 96 ragged contexts; with pieces worked out by the
// computing warps 206 sequences of up to 4 slots took 21.7 us, not 14.)  A warp
// takes 16 slots of a tile, with the cache as the larger operand of m16n8k16
// products and up to eight query heads as the smaller (16 as two):
//   S^T[16 slots, 8 heads] += K[16 slots, 16 channels] Q^T[16 channels, 8 heads]
//   O^T[16 dims, 8 heads]  += V^T[16 dims, 16 slots]   P^T[16 slots, 8 heads]
// P^T is S^T's fragment transposed (movmatrix), and enters as the sum of two
// values of the cache's type, so that its rounding (2^-9 of a weight in bf16)
// does not show beside the output's own: 2^-17 of a weight is left, in f16 2^-22
// of it or 2^-32 of the largest.  The tensor pipe is at 13 % of its rate, issue
// slots at 20 %.  The finish with 16 slots a thread spills 32 bytes of each, the one
// by warps at 64-wide heads 8.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
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
  int32_t batch, hq, hkv, group;
  int32_t window, sinks;
  float scale;                  // softmax scale times log2 e
  void* out;
  int32_t out_type;             // 0 bf16, 1 f16, 2 f32
  int32_t f16;                  // of q and the cache; 0: bf16
  float* lse;
  const float* w_in;
  float* w_out;
  float decay;
  int32_t slot_heads;
  int64_t slot_stride;
  int2* desc;
  int32_t ranges;               // blocks of the split pass
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

// The axis on which the segments' tiles lie one behind the other, each segment
// behind a lead-in that stands for what its start and end cost, is cut into
// equal ranges, one a block, two blocks an SM.  (SMs differ by some 10 % in what
// they get of the memory's bandwidth, but small ranges behind the large ones,
// for those that are done first, cost more in starts than they gave: a token
// over 128K 93.7 us instead of 91.5, 96 ragged contexts 77 instead of 72.)
constexpr int kLead = 1;
constexpr int kWarps = 4;                     // warps that compute
constexpr int kThreads = 32 * (kWarps + 1);   // and one that loads

struct Walk {
  int64_t pos, left;            // start of the segment on the axis; units of the range to go
  int b, h;                     // the segment
  int64_t off;                  // units of it before the range
};

struct Plan {
  Walk first;
  int64_t units;
  int ranges;
};

// First unit of range i, and the range that unit u lies in.
DS_DEV int64_t range_start(const Plan& p, int i) { return p.units * i / p.ranges; }
DS_DEV int range_with(const Plan& p, int64_t u) {     // the last i with units i / ranges <= u
  return (int)min(((u + 1) * p.ranges - 1) / p.units, (int64_t)p.ranges - 1);
}

struct Piece {
  Range r;
  int b, h;
  int t0, t1;                   // tiles; t1 0: no more pieces
  int64_t pos;                  // of the segment
};
constexpr int kPieces = 8;

DS_DEV Range seq_range(const KArgs& a, int b, bool report) {
  return range_of(checked_len(a.lens[b], a.cache.slots, a.status, report), a.window,
                  a.sinks);
}

// The block's range, formed by all of its threads; false when it has none.
DS_DEV bool make_plan(const KArgs& a, Plan& plan, int64_t (*s_sum)[2]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  int64_t units = 0, tiles = 0;               // of this thread's sequences
  for (int b = b0; b < b1; ++b) {
    const int t = seq_range(a, b, blockIdx.x == 0).tiles;
    tiles += t;
    units += t > 0 ? t + kLead : 0;
  }
  units *= a.hkv;
  tiles *= a.hkv;
  if (tid == 0) plan.first.left = 0;
  int64_t incl = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  }
  if (lane == 31) { s_sum[warp][0] = incl; s_sum[warp][1] = tiles; }
  __syncthreads();
  int64_t before = incl - units, all = 0, all_tiles = 0;
  for (int w = 0; w <= kWarps; ++w) {
    if (w < warp) before += s_sum[w][0];
    all += s_sum[w][0];
    all_tiles += s_sum[w][1];
  }
  Plan p;
  p.units = all;
  p.ranges = (int)min((int64_t)gridDim.x, all_tiles);
  if ((int)blockIdx.x >= p.ranges) return false;
  const int64_t lo = range_start(p, blockIdx.x);
  if (before <= lo && lo < before + units) {  // one thread
    int b = b0;
    int64_t len = 0, off = lo - before;
    for (; b < b1; ++b) {
      const int t = seq_range(a, b, false).tiles;
      len = t > 0 ? t + kLead : 0;
      if (off < len * a.hkv) break;
      off -= len * a.hkv;
    }
    len = max(len, (int64_t)1);
    plan.first.b = b;
    plan.first.h = (int)(off / len);
    plan.first.off = off - plan.first.h * len;
    plan.first.pos = lo - plan.first.off;
    plan.first.left = range_start(p, blockIdx.x + 1) - lo;
    plan.units = p.units;
    plan.ranges = p.ranges;
  }
  __syncthreads();
  return true;
}

// The next piece of the walk; false at its end.
DS_DEV bool next_piece(const KArgs& a, Walk& w, Piece& p) {
  while (w.left > 0 && w.b < a.batch) {
    const Range r = seq_range(a, w.b, false);
    if (r.tiles == 0) {
      ++w.b;
      w.h = 0;
      continue;
    }
    const int64_t len = r.tiles + kLead;
    const int64_t take = min(w.left, len - w.off);
    p.r = r;
    p.b = w.b;
    p.h = w.h;
    p.pos = w.pos;
    p.t0 = (int)max(w.off - kLead, (int64_t)0);
    p.t1 = (int)(w.off + take - kLead);
    w.left -= take;
    w.pos += len;
    w.off = 0;
    if (++w.h == a.hkv) {
      w.h = 0;
      ++w.b;
    }
    if (p.t1 > p.t0) return true;             // else only part of the lead-in
  }
  return false;
}

DS_DEV void tma_load_4d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                             int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}
DS_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
DS_DEV void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
DS_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF>
DS_DEV void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF>
DS_DEV uint32_t pack2(float lo, float hi) {
  return BF ? ptx::pack_bf16x2(lo, hi) : ptx::pack_f16x2(lo, hi);
}
// (lo, hi) as a pair of the cache's type, and what that rounding left.
template <bool BF>
DS_DEV void split2(float lo, float hi, uint32_t& big, uint32_t& rest) {
  big = pack2<BF>(lo, hi);
  float2 b;
  if constexpr (BF)
    b = make_float2(__uint_as_float(big << 16), __uint_as_float(big & 0xffff0000u));
  else
    b = __half22float2(*reinterpret_cast<const __half2*>(&big));
  rest = pack2<BF>(lo - b.x, hi - b.y);
}

// A barrier of the warps that compute; whether x holds for all of them.
DS_DEV bool all_warps(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}

template <int D>
struct Cfg {
  static constexpr int kSubBytes = 16 * D * 2;          // 16 keys of K or V
  static constexpr int kStage = 2 * 4 * kSubBytes;      // a tile's K and V
  static constexpr int kStages = D == 128 ? 3 : 6;
  // ring, and the warps' outputs of eight rows
  static constexpr size_t smem = (size_t)kStages * kStage + kWarps * 8 * D * 4;
  // where value d of a row lies among the D of a warp's output row (rows turned
  // so that the four rows that a warp writes at once fall into different banks)
  static DS_DEV int turned(int row, int d) { return (d + 8 * (row >> 1)) & (D - 1); }
};

struct Shared {
  alignas(8) uint64_t full[6], empty[6];
  Plan plan;
  int64_t sum[kWarps + 1][2];
  float m[kWarps][8], l[kWarps][8];
  // Pieces, from the loader to the warps that compute.  It is at most a ring of
  // tiles ahead of them, and a piece has a tile or more: eight places are enough
  // (a piece is copied out before its first tile is waited for).
  uint64_t told[kPieces];
  Piece piece[kPieces];
  int abort;
};
static_assert(sizeof(Shared) <= 1024 && 2 * (Cfg<128>::smem + 1024 + 1024) <= 233472,
              "two blocks an SM (1 KB a block is the system's)");
static_assert(Cfg<64>::kStages + 2 <= kPieces && Cfg<128>::kStages + 2 <= kPieces, "");

template <int D, bool BF, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    split(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
          const KArgs a, const int hnd) {
  using namespace ptx;
  using C = Cfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t ring = smem_addr(raw);
  float* const merge = reinterpret_cast<float*>(raw + S * C::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 4);
    }
    for (int i = 0; i < kPieces; ++i) mbar_init(smem_addr(&sh.told[i]), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (tid == kThreads - 1) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (!make_plan(a, sh.plan, sh.sum)) return;
  volatile int* const abort = &sh.abort;
  Walk walk = sh.plan.first;
  Piece pc;
  int stage = 0, phase = 0;                   // of the next tile

  if (warp == kWarps) {
    // ---- the loader: lanes 0 to 3 bring the tile's K, 4 to 7 its V, a box of
    // 16 slots each; page ids are read eight tiles ahead
    const uint64_t policy = l2_evict_first();
    const int sub = lane & 3, kind = (lane >> 2) & 1;
    int64_t issued = 0;
    bool ok = true;
    for (int np = 0; ok; np = (np + 1) % kPieces) {
      if (!next_piece(a, walk, pc)) pc.t1 = 0;
      const Range r = pc.r;
      if (lane == 0) {
        sh.piece[np] = pc;
        mbar_arrive(smem_addr(&sh.told[np]));
        if (pc.t1 > 0 && pc.t0 == 0) {        // numbered by range and segment, which never
          const int64_t u = pc.pos + kLead, seg = (int64_t)pc.b * a.hkv + pc.h;
          const int f = range_with(sh.plan, u);   // both stand still, pieces have places of
          a.desc[seg] = make_int2((int)(f + seg),  // their own (u: the segment's first tile)
                                  range_with(sh.plan, u + r.tiles - 1) - f + 1);
        }
      }
      __syncwarp();
      if (pc.t1 == 0) break;
      auto sub_visible = [&](int t, int s) {
        const int k0 = tile_slot(r, t) + 16 * s;
        return t < pc.t1 && k0 < r.n && (k0 < r.sinks || k0 + 16 > r.start);
      };
      auto page_of = [&](int t, int s) {
        return a.cache.page_table && sub_visible(t, s)
                   ? a.cache.page_table[(int64_t)pc.b * a.cache.max_pages +
                                        ((tile_slot(r, t) + 16 * s) >> a.cache.page_shift)]
                   : pc.b;
      };
      int ids = 0, next = page_of(pc.t0 + (lane >> 2), sub);
      for (int t = pc.t0; t < pc.t1; ++t) {
        const int k = (t - pc.t0) & 7;
        if (k == 0) {
          ids = next;
          next = page_of(t + 8 + (lane >> 2), sub);
        }
        int pg = __shfl_sync(0xffffffffu, ids, k * 4 + sub);
        if ((uint32_t)pg >= (uint32_t)a.cache.num_pages) {
          // (a page past the pool reads as zeros)
          if (lane < 4 && sub_visible(t, sub)) flag(a.status, DS_DEV_BAD_PAGE);
          pg = a.cache.num_pages;
        }
        const bool vis = sub_visible(t, sub);
        const int boxes = __popc(__ballot_sync(0xffffffffu, vis && lane < 8));
        ok = mbar_wait(smem_addr(&sh.empty[stage]), phase ^ 1, abort);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_addr(&sh.full[stage]);
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * C::kSubBytes);
        __syncwarp();
        if (lane < 8 && vis) {
          const int slot = tile_slot(r, t) + 16 * sub;
          const int row = a.cache.page_table ? slot & (a.cache.page_size - 1) : slot;
          const uint32_t dst = ring + stage * C::kStage + (kind * 4 + sub) * C::kSubBytes;
          tma_load_4d_hint(dst, kind ? &tv : &tk, bar, 0, row, hnd ? 0 : pc.h * (D / 64),
                           hnd ? pg * a.hkv + pc.h : pg, policy);
        }
        ++issued;
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
    }
    // No copy may land behind the block's end, whoever gave up: the loader stays
    // until the last ones are here.
    for (int i = 0; i < S && i < issued; ++i) {
      if (--stage < 0) { stage = S - 1; phase ^= 1; }
      drain_wait(smem_addr(&sh.full[stage]), phase);
    }
    if (!ok && lane == 0) flag(a.status, DS_DEV_TIMEOUT);
    return;
  }

  // ---- the others: a warp takes 16 keys of every tile
  const int g = lane >> 2, t4 = lane & 3, G = a.group;
  const int sub = warp;
  // ldmatrix: this lane's row of K (keys 0-15, 8 channels a chunk) and of V
  const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kchunk = lane >> 4;
  const int vrow = (lane & 7) + (lane >> 4) * 8, vchunk = (lane >> 3) & 1;
  // a box is [64-channel half][16 slots][128 bytes], chunks swizzled by row
  auto chunk_at = [&](uint32_t base, int row, int chunk) {
    return base + (chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
  };
  // m lies this far below the maximum that it follows (f16's range, see below).
  constexpr float kBelow = BF ? 0.f : 7.f;
  // The next piece and its queries, which are read while the last one is joined.
  uint32_t q[NT][D / 16][2];
  int np = 0, told = 0;
  auto fetch = [&] {
    const bool ok = mbar_wait(smem_addr(&sh.told[np]), told, abort);
    if (!__all_sync(0xffffffffu, ok)) return false;
    pc = sh.piece[np];
    if (++np == kPieces) { np = 0; told ^= 1; }
    if (pc.t1 == 0) return false;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        q[i][ks][0] = q[i][ks][1] = 0u;
        if (8 * i + g < G) {
          const uint16_t* p = a.q + (int64_t)pc.b * a.q_stride +
                              (int64_t)(pc.h * G + 8 * i + g) * D + ks * 16 + 2 * t4;
          q[i][ks][0] = *reinterpret_cast<const uint32_t*>(p);
          q[i][ks][1] = *reinterpret_cast<const uint32_t*>(p + 8);
        }
      }
    return true;
  };
  // (a warp whose wait gave up takes the others with it: they meet at barriers)
  bool more = all_warps(fetch());
  while (more) {
    const Range r = pc.r;
    const int64_t seg = (int64_t)pc.b * a.hkv + pc.h;
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      m[i][0] = m[i][1] = -CUDART_INF_F;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][d][j] = 0.f;
    }
    for (int t = pc.t0; t < pc.t1; ++t) {
      const int st = stage, ph = phase;
      if (++stage == S) { stage = 0; phase ^= 1; }
      const bool ok = mbar_wait(smem_addr(&sh.full[st]), ph, abort);
      const int k0 = tile_slot(r, t) + 16 * sub;
      if (__all_sync(0xffffffffu, ok) && k0 < r.n && (k0 < r.sinks || k0 + 16 > r.start)) {
        const uint32_t kb = ring + st * C::kStage + sub * C::kSubBytes;
        const uint32_t vb = kb + 4 * C::kSubBytes;
        float s[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t x[4];
          ldmatrix4(x, chunk_at(kb, krow, 2 * ks + kchunk));
#pragma unroll
          for (int i = 0; i < NT; ++i) mma<BF>(s[i], x, q[i][ks][0], q[i][ks][1]);
        }
        const bool whole = k0 + 16 <= r.n && (k0 >= r.start || k0 + 16 <= r.sinks);
        const bool va = whole || visible(r, k0 + g), vc = whole || visible(r, k0 + g + 8);
        float mx[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s[i][j] = va ? s[i][j] * a.scale : -CUDART_INF_F;
            s[i][2 + j] = vc ? s[i][2 + j] * a.scale : -CUDART_INF_F;
            const int row = 8 * i + 2 * t4 + j;
            if (a.logits && row < G) {
              float* x = a.logits + (seg * a.cache.slots + k0 + g) * G + row;
              if (va) x[0] = s[i][j];
              if (vc) x[8 * G] = s[i][2 + j];
            }
            mx[i][j] = fmaxf(s[i][j], s[i][2 + j]);
          }
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              mx[i][j] = fmaxf(mx[i][j], __shfl_xor_sync(0xffffffffu, mx[i][j], x));
        // the reference point m follows the maximum only when that has grown by
        // more than 2^8, so that outputs are rarely scaled; in f16 it lies 2^7
        // below: weights reach 2^15 of the 2^16 that there are, and those that
        // the type's smallest step cuts short (2^-25 of its unit) lie 2^7 lower
        // (the difference is exact where it is near the limit; of logits beyond
        // 2^24 m plus the limit is not, and a weight of 2^16 has no value)
        bool grow = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) grow |= mx[i][j] - m[i][j] > 8.f + kBelow;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float now = fmaxf(m[i][j], mx[i][j] - kBelow);
              const float f = m[i][j] == now ? 1.f : ex2(m[i][j] - now);
              m[i][j] = now;
              l[i][j] *= f;
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                o[i][d][j] *= f;
                o[i][d][2 + j] *= f;
              }
            }
          }
        }
        uint32_t big[NT][2], rest[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ref = m[i][j & 1] == -CUDART_INF_F ? 0.f : m[i][j & 1];
            p[j] = ex2(s[i][j] - ref);
            l[i][j & 1] += p[j];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            split2<BF>(p[2 * j], p[2 * j + 1], big[i][j], rest[i][j]);
            big[i][j] = transpose8x8(big[i][j]);
            rest[i][j] = transpose8x8(rest[i][j]);
          }
        }
        // slots that are not attended to may hold anything: their V is zeroed
        uint32_t keep[2] = {~0u, ~0u};
        if (!whole)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            keep[j] = (visible(r, k0 + 8 * j + 2 * t4) ? 0xffffu : 0u) |
                      (visible(r, k0 + 8 * j + 2 * t4 + 1) ? 0xffff0000u : 0u);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t x[4];
          ldmatrix4_trans(x, chunk_at(vb, vrow, 2 * d + vchunk));
          x[0] &= keep[0];
          x[1] &= keep[0];
          x[2] &= keep[1];
          x[3] &= keep[1];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma<BF>(o[i][d], x, big[i][0], big[i][1]);
            mma<BF>(o[i][d], x, rest[i][0], rest[i][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.empty[st]));
    }
    // ---- the warps' outputs joined, eight rows at a time, into the piece's place
    more = fetch();
    const int64_t piece = blockIdx.x + seg;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) l[i][j] += __shfl_xor_sync(0xffffffffu, l[i][j], x);
    float* const mine = merge + warp * 8 * D;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const bool all = all_warps(more);       // and the last rows have been read
      if (i == 0) more = all;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 2 * t4 + j;
        if (g == 0) {
          sh.m[warp][row] = m[i][j];
          sh.l[warp][row] = l[i][j];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          mine[row * D + C::turned(row, d * 16 + g)] = o[i][d][j];
          mine[row * D + C::turned(row, d * 16 + g + 8)] = o[i][d][2 + j];
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      for (int x = tid; x < min(8, G - 8 * i) * D / 4; x += 32 * kWarps) {
        const int row = x / (D / 4), c = x % (D / 4);
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][row]);
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(sh.m[w][row] - ref);
          const float4 y = *reinterpret_cast<const float4*>(
              merge + (w * 8 + row) * D + C::turned(row, c * 4));
          sum.x = fmaf(f, y.x, sum.x);
          sum.y = fmaf(f, y.y, sum.y);
          sum.z = fmaf(f, y.z, sum.z);
          sum.w = fmaf(f, y.w, sum.w);
          total = fmaf(f, sh.l[w][row], total);
        }
        *reinterpret_cast<float4*>(a.part_o + ((piece * G + 8 * i + row) * D + c * 4)) = sum;
        if (c == 0) a.part_ml[piece * G + 8 * i + row] = make_float2(M, total);
      }
    }
  }
  if (tid == 0 && *abort) flag(a.status, DS_DEV_TIMEOUT);
}

// (max, sum) of two parts of a row.
DS_DEV float2 join_ml(float2 x, float2 y) {
  const float M = fmaxf(x.x, y.x), ref = M == -CUDART_INF_F ? 0.f : M;
  return make_float2(M, x.y * ptx::ex2(x.x - ref) + y.y * ptx::ex2(y.x - ref));
}
// Joined over N neighbouring lanes.
template <int N>
DS_DEV float2 join_lanes(float2 x) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
    x = join_ml(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o),
                               __shfl_xor_sync(0xffffffffu, x.y, o)));
  return x;
}

constexpr int kFinishWarps = 8;
constexpr int kFinishThreads = 32 * kFinishWarps;

// First piece and pieces of a segment with slots; none where the split pass gave up
// before it told them (it has set the status bit), whose rows are 0 and whose slots
// get no weight.
DS_DEV int2 pieces_of(const KArgs& a, const int64_t seg) {
  const int2 d = a.desc[seg];
  return pieces_usable((int)seg, d.x, d.y, a.ranges) ? d : make_int2(0, 0);
}

// Lane l's values of a row of the cache or of q, 4 l .. 4 l + 3 or 2 l and 2 l + 1,
template <int V>
DS_DEV void row_words(uint32_t (&w)[V / 2], const uint16_t* row) {
  if constexpr (V == 4) {
    const uint2 y = *reinterpret_cast<const uint2*>(row + (threadIdx.x & 31) * V);
    w[0] = y.x;
    w[1] = y.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(row + (threadIdx.x & 31) * V);
  }
}
// as float32.
DS_DEV float2 word_values(uint32_t w, int f16) {
  return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
             : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// The signs' bits of the values that are infinite or NaN (an exponent of ones
// carries into the sign).
DS_DEV uint32_t not_finite(uint32_t w, int f16) {
  return ((w & 0x7fff7fffu) + (f16 ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// An output row with NaN, looked at once more by its `parts` warps.  A weight is
// above 0 and an infinite value times it infinite, but the split pass multiplies V
// with the two values that make up a weight: the second, what rounding left, may be
// 0 or below, and either too small for its type, and inf - inf and 0 inf are NaN.
// So what the infinite and NaN values that the row attends to add up to by
// themselves takes the output's place, each times 1, or times 0 where its logit is
// -inf.  Only a row with NaN pays for it (32 rows of 128K slots 2.8 ms in all), the
// others a vote, 0.1 to 0.2 us a call.  (Taken out of the products tile by tile
// they cost every call: 128K 0.5 % more, with 16 query heads a kv head 1.8.)
template <int D>
DS_DEV void put_endless(const KArgs& a, int64_t row, int part, int parts, float (*s_o)[D]) {
  constexpr int V = D / 32;
  const int b = (int)(row / a.hq), hq = (int)(row % a.hq), lane = threadIdx.x & 31;
  const int n = checked_len(a.lens[b], a.cache.slots, nullptr, false);
  const Range r = range_of(n, a.window, a.sinks);
  const int64_t head = (int64_t)(hq / a.group) * a.cache.head_stride;
  const int t1 = (int)((int64_t)n * (part + 1) / parts);
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.f;
  // 16 bytes a lane of as many rows as that gives a warp, four times, are looked
  // through; only rows that have something are gone into
  constexpr int LPR = D / 8, AT = 32 / LPR;
#pragma unroll 1
  for (int t0 = (int)((int64_t)n * part / parts); t0 < t1; t0 += 4 * AT) {
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = min(t0 + j * AT + lane / LPR, t1 - 1);
      const int pg = visible(r, t) ? slot_page(a.cache, b, t) : -1;
      w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (pg >= 0)
        w[j] = *reinterpret_cast<const uint4*>(a.cache.pool[1] + slot_at(a.cache, pg, t) + head +
                                               lane % LPR * 8);
    }
    uint32_t any = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      any |= not_finite(w[j].x, a.f16) | not_finite(w[j].y, a.f16) | not_finite(w[j].z, a.f16) |
             not_finite(w[j].w, a.f16);
    if (!__any_sync(0xffffffffu, any != 0u)) continue;
#pragma unroll 1
    for (int t = t0; t < min(t0 + 4 * AT, t1); ++t) {
      const int pg = visible(r, t) ? slot_page(a.cache, b, t) : -1;
      if (pg < 0) continue;
      const int64_t at = slot_at(a.cache, pg, t) + head;
      uint32_t q[V / 2], x[V / 2], v[V / 2];
      row_words<V>(q, a.q + (int64_t)b * a.q_stride + (int64_t)hq * D);
      row_words<V>(x, a.cache.pool[0] + at);
      row_words<V>(v, a.cache.pool[1] + at);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 y = word_values(q[i], a.f16), z = word_values(x[i], a.f16);
        s = fmaf(y.x, z.x, fmaf(y.y, z.y, s));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float p = s * a.scale == -CUDART_INF_F ? 0.f : 1.f;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 y = word_values(v[i], a.f16);
        const uint32_t bad = not_finite(v[i], a.f16);
        if (bad & 0xffffu) sum[2 * i] = fmaf(p, y.x, sum[2 * i]);
        if (bad >> 16) sum[2 * i + 1] = fmaf(p, y.y, sum[2 * i + 1]);
      }
    }
  }
  if (parts > 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_o[part][lane * V + k] = sum[k];
    __syncthreads();
    if (part > 0) return;
    for (int w = 1; w < parts; ++w)
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += s_o[w][lane * V + k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t at = row * D + lane * V + k;
    if (sum[k] == 0.f) continue;          // (nothing infinite here)
    if (a.out_type == 2) static_cast<float*>(a.out)[at] = sum[k];
    else static_cast<uint16_t*>(a.out)[at] =
        (uint16_t)(a.out_type == 0 ? ptx::pack_bf16x2(sum[k], 0.f) : ptx::pack_f16x2(sum[k], 0.f));
  }
}

// An output row by `parts` warps, which share its pieces: lane l has values 4 l ..
// 4 l + 3 (2 l at D = 64) of eight pieces on their way at once.
template <int D>
DS_DEV void finish_row(const KArgs& a, const int64_t row, const int part, const int parts,
                       float (*s_o)[D], float2* s_ml) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, G = a.group;
  const bool real = row < (int64_t)a.batch * a.hq;
  const int b = real ? (int)(row / a.hq) : 0, hq = real ? (int)(row % a.hq) : 0;
  const int h = hq / G, g = hq % G;
  const int n = real ? checked_len(__ldcg(a.lens + b), a.cache.slots, nullptr, false) : 0;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int2 d = pieces_of(a, b * a.hkv + h);   // (not looked at without slots)
  const bool some = n > 0 && d.y > 0;
  float o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = 0.f;
  float2 all = make_float2(-CUDART_INF_F, 0.f);
  if (some) {
    const int p0 = (int)((int64_t)d.y * part / parts), p1 = (int)((int64_t)d.y * (part + 1) / parts);
    const float2* ml = a.part_ml + (int64_t)d.x * G + g;
    const float* po = a.part_o + ((int64_t)d.x * G + g) * D + lane * V;
    for (int i0 = p0; i0 < p1; i0 += 32) {        // 32 pieces, a lane each
      const int m = min(32, p1 - i0);
      float2 x = make_float2(-CUDART_INF_F, 0.f);
      if (lane < m) x = ml[(int64_t)(i0 + lane) * G];
      float v[8][V];
      auto load = [&](int i) {            // (past the last: the last one's, unused)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* p = po + (int64_t)(i0 + min(i + j, m - 1)) * G * D;
          if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4*>(p);
            v[j][0] = y.x; v[j][1] = y.y; v[j][2] = y.z; v[j][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(p);
            v[j][0] = y.x; v[j][1] = y.y;
          }
        }
      };
      load(0);
      const float2 now = join_ml(all, join_lanes<32>(x));
      const float ref = now.x == -CUDART_INF_F ? 0.f : now.x;
      const float f = ptx::ex2(x.x - ref), old = ptx::ex2(all.x - ref);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] *= old;
      for (int i = 0; i < m; i += 8) {
        if (i > 0) load(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = __shfl_sync(0xffffffffu, f, (i + j) & 31);
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (i + j < m) o[k] = fmaf(w, v[j][k], o[k]);
        }
      }
      all = now;
    }
  }
  if (parts > 1) {                        // the whole block works on this row
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < V; ++k) s_o[warp][lane * V + k] = o[k];
    if (lane == 0) s_ml[warp] = all;
    __syncthreads();
    for (int w = 1; part == 0 && w < parts; ++w) {
      const float2 x = s_ml[w], now = join_ml(all, x);
      const float ref = now.x == -CUDART_INF_F ? 0.f : now.x;
      const float f = ptx::ex2(x.x - ref), old = ptx::ex2(all.x - ref);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = fmaf(f, s_o[w][lane * V + k], o[k] * old);
      all = now;
    }
  }
  bool nan = false;                       // in the row, but not in its sum of weights
  if (real && part == 0) {
    if (some) {
      const float inv = 1.f / all.y;
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] *= inv;
    }
    if (a.lse && lane == 0)
      a.lse[row] = some ? (all.x + log2f(all.y)) * 0.6931471805599453f : -CUDART_INF_F;
    const int64_t at = row * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      if (a.out_type == 2)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + k) =
            make_float2(o[k], o[k + 1]);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + k) =
            a.out_type == 0 ? ptx::pack_bf16x2(o[k], o[k + 1]) : ptx::pack_f16x2(o[k], o[k + 1]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) nan |= o[k] != o[k];
    nan &= all.y == all.y;
  }
  nan = parts > 1 ? __syncthreads_or(nan) : __any_sync(0xffffffffu, nan);
  if (nan) put_endless<D>(a, row, part, parts, s_o);
}

// Logits of rows g0 .. g0 + 3 of a slot's G, in a piece as wide as G allows;
// rows past the last repeat it.
DS_DEV void load_logits(float (&s)[4], const float* p, int g0, int G) {
  if ((G & 3) == 0) {
    const float4 v = *reinterpret_cast<const float4*>(p + g0);
    s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = p[min(g0 + j, G - 1)];
  }
}

// The weights of 128 slots of a (sequence, kv head), by a warp: four query heads
// at a time, eight lanes to the sums of each.
DS_DEV void warp_weights(const KArgs& a, const int64_t item) {
  const int lane = threadIdx.x & 31, G = a.group, l = lane % 8;
  const int64_t spans = (a.cache.slots + 127) / 128, seg = item / spans;
  const bool real = seg < (int64_t)a.batch * a.hkv;
  const int n = real ? checked_len(__ldcg(a.lens + seg / a.hkv), a.cache.slots, nullptr, false) : 0;
  const int t0 = (int)(item - seg * spans) * 128 + lane;
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (t0 - lane >= n) return;
  const int2 d = pieces_of(a, seg);
  const Range r = range_of(n, a.window, a.sinks);
  const int64_t at = seg * a.slot_stride;
  float old[4], sum[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    old[k] = a.w_in ? a.w_in[at + min(t0 + 32 * k, n - 1)] : 0.f;
    sum[k] = 0.f;
  }
  for (int g0 = 0; g0 < G; g0 += 4) {
    float s[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      load_logits(s[k], a.logits + (seg * a.cache.slots + min(t0 + 32 * k, n - 1)) * G, g0, G);
    const int row = g0 + lane / 8;
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (row < G)
      for (int j = l; j < d.y; j += 8) ml = join_ml(ml, a.part_ml[(int64_t)(d.x + j) * G + row]);
    ml = join_lanes<8>(ml);
    // (no pieces: a sum of infinity, weights of zero)
    const float ref = d.y > 0 ? ml.x + log2f(ml.y) : CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float rj = __shfl_sync(0xffffffffu, ref, 8 * j);
      if (g0 + j < G && rj != CUDART_INF_F) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sum[k] += visible(r, t0 + 32 * k) ? ptx::ex2(s[k][j] - rj) : 0.f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t0 + 32 * k < n) a.w_out[at + t0 + 32 * k] = fmaf(old[k], a.decay, sum[k]);
}

// Output rows (the first blocks), and the weights of SLOTS x 256 slots of a
// (sequence, slot head) a time: the rows whose weights a slot sums go in chunks
// of up to four of one kv head, CHUNKS at once, so that a thread has 16 loads
// on its way beside the rows' own sums, which 8 to 32 lanes join a row.  With
// SLOTS 0 a warp works by itself, or (CHUNKS 0) there are output rows only.
template <int D, int SLOTS, int CHUNKS>
__global__ void __launch_bounds__(kFinishThreads, SLOTS == 0 ? 4 : 2)
    finish(const KArgs a, const int row_blocks, const int parts) {
  __shared__ float s_ref[32];
  __shared__ float s_o[kFinishWarps][D];
  __shared__ float2 s_ml[kFinishWarps];
  const int tid = threadIdx.x, G = a.group;
  // Every block of the split pass has waited for what came before it when it lets
  // this kernel's blocks start, so lengths and input weights are read, and places
  // worked out, before this kernel's own wait.  These reads go past the L1, which the
  // wait alone promises to hold nothing older than the kernels in front.
  if (CHUNKS == 0 || (int)blockIdx.x < row_blocks) {      // `parts` warps per output row
    const int w = blockIdx.x * kFinishWarps + (tid >> 5);
    finish_row<D>(a, w / parts, w % parts, parts, s_o, s_ml);
    return;
  }
  if constexpr (SLOTS == 0 && CHUNKS == 1) {
    warp_weights(a, ((int64_t)blockIdx.x - row_blocks) * kFinishWarps + (tid >> 5));
    return;
  } else if constexpr (CHUNKS > 0) {
    constexpr int SPAN = SLOTS * kFinishThreads;
    constexpr int LPR = kFinishThreads / (4 * CHUNKS) < 32 ? kFinishThreads / (4 * CHUNKS) : 32;
    const int64_t spans = (a.cache.slots + SPAN - 1) / SPAN;
    const int64_t items = (int64_t)a.batch * a.slot_heads * spans;
    const int per_head = (G + 3) / 4;       // chunks
    const int chunks = per_head * (a.slot_heads == 1 ? a.hkv : 1);
    // this thread's part of a row's sum: row i % 4 of chunk i / 4, pieces from l on
    const int i = tid / LPR, l = tid % LPR;
    int64_t seg0, at;                       // the item: first segment, place of its weights
    int n, t0;                              // slots of its sequence, this thread's first
    float old[SLOTS];
    // slots past the end: the thread's first again (or the last one), unused
    auto slot = [&](int k) { return t0 + k * kFinishThreads < n ? k * kFinishThreads : 0; };
    auto item = [&](int64_t it) {
      const int64_t bw = it / spans;
      const int b = (int)(bw / a.slot_heads);
      seg0 = (int64_t)b * a.hkv + (a.slot_heads == 1 ? 0 : (int)(bw % a.slot_heads));
      at = bw * a.slot_stride;
      n = checked_len(__ldcg(a.lens + b), a.cache.slots, nullptr, false);
      const int64_t start = (it - bw * spans) * SPAN;
      t0 = (int)start + tid;
      if (start >= n) return false;
      const float* p = a.w_in + at + min(t0, n - 1);
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) old[k] = a.w_in ? __ldcg(p + slot(k)) : 0.f;
      return true;
    };
    int64_t it = blockIdx.x - row_blocks;
    bool work = it < items && item(it);
    grid_dep_wait();
    grid_dep_launch_dependents();
    while (it < items) {
      if (work) {
        const Range r = range_of(n, a.window, a.sinks);
        const int first = min(t0, n - 1);
        float sum[SLOTS];
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) sum[k] = 0.f;
        for (int c0 = 0; c0 < chunks; c0 += CHUNKS) {
          const int mine = min(c0 + i / 4, chunks - 1), g = mine % per_head * 4 + i % 4;
          const bool row = i < 4 * CHUNKS && c0 + i / 4 < chunks && g < G;
          const int2 d = pieces_of(a, seg0 + mine / per_head);
          float s[CHUNKS][SLOTS][4];
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            const int ch = min(c0 + c, chunks - 1);
            const float* p = a.logits + ((seg0 + ch / per_head) * a.cache.slots + first) * G;
#pragma unroll
            for (int k = 0; k < SLOTS; ++k)
              load_logits(s[c][k], p + slot(k) * G, ch % per_head * 4, G);
          }
          const float2* const p_ml = a.part_ml + (int64_t)d.x * G + g;
          float2 ml = make_float2(-CUDART_INF_F, 0.f), ml2 = ml;
          if (row && l < d.y) ml = p_ml[(int64_t)l * G];
          if (row && l + LPR < d.y) ml2 = p_ml[(int64_t)(l + LPR) * G];
          __syncthreads();                  // the last ones' sums are used
          ml = join_ml(ml, ml2);
          if (row)
            for (int j = l + 2 * LPR; j < d.y; j += LPR) ml = join_ml(ml, p_ml[(int64_t)j * G]);
          ml = join_lanes<LPR>(ml);
          // (no row, no pieces: a sum of infinity, weights of zero)
          if (i < 4 * CHUNKS && l == 0)
            s_ref[i] = row && d.y > 0 ? ml.x + log2f(ml.y) : CUDART_INF_F;
          __syncthreads();
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float ref = s_ref[4 * c + j];
              if (ref != CUDART_INF_F) {
#pragma unroll
                for (int k = 0; k < SLOTS; ++k) {
                  const float p = ptx::ex2(s[c][k][j] - ref);
                  sum[k] += visible(r, first + slot(k)) ? p : 0.f;
                }
              }
            }
        }
#pragma unroll
        for (int k = 0; k < SLOTS; ++k)
          if (t0 + k * kFinishThreads < n)
            a.w_out[at + t0 + k * kFinishThreads] = fmaf(old[k], a.decay, sum[k]);
      }
      it += gridDim.x - row_blocks;
      work = it < items && item(it);
    }
  }
}

template <int D, int SLOTS, int CHUNKS>
cudaError_t launch_finish(const KArgs& a, int pieces, cudaStream_t stream) {
  // a block per row when a segment may have many pieces, else a warp
  const int parts = pieces > 16 ? kFinishWarps : 1;
  const int row_blocks =
      (int)(((int64_t)a.batch * a.hq * parts + kFinishWarps - 1) / kFinishWarps);
  int64_t items = 0;                      // blocks for the weights
  if constexpr (CHUNKS > 0 && SLOTS > 0) {
    const int span = SLOTS * kFinishThreads;
    items = std::min<int64_t>(
        (int64_t)a.batch * a.slot_heads * ((a.cache.slots + span - 1) / span), 152 * 4 * 2);
  } else if constexpr (CHUNKS > 0) {
    items = ((int64_t)a.batch * a.hkv * ((a.cache.slots + 127) / 128) + kFinishWarps - 1) /
            kFinishWarps;
  }
  const int grid = (int)(row_blocks + items);
  return launch_dependent(finish<D, SLOTS, CHUNKS>, dim3(grid), dim3(kFinishThreads), 0, stream, a,
                          row_blocks, parts);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// (the driver's, the same on every device; looked for again when it was not found)
EncodeFn encode_fn() {
  static std::atomic<void*> found{nullptr};
  void* ptr = found.load(std::memory_order_relaxed);
  cudaDriverEntryPointQueryResult q;
  if (!ptr && cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                               cudaEnableDefault, &q) == cudaSuccess) {
    if (q != cudaDriverEntryPointSuccess) ptr = nullptr;
    found.store(ptr, std::memory_order_relaxed);
  }
  return reinterpret_cast<EncodeFn>(ptr);
}

// K or V as [64 channels][slots of a page][halves of heads][pages] (heads
// before slots: the head is part of the page's coordinate): a box is 16 slots
// of one head, [half][16][128 bytes], its chunks swizzled.
bool cache_map(CUtensorMap* map, const void* base, const ds_decode_args& g) {
  const cuuint64_t D = g.head_dim, P = g.page_size, H = g.num_kv_heads, N = g.num_pages;
  const bool hnd = g.kv_layout == DS_KV_HND;
  const cuuint64_t dims[4] = {64, P, (D / 64) * (hnd ? 1 : H), N * (hnd ? H : 1)};
  const cuuint64_t strides[3] = {(hnd ? 1 : H) * D * 2, 128, P * (hnd ? 1 : H) * D * 2};
  const cuuint32_t box[4] = {64, 16, (cuuint32_t)(D / 64), 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  // (lines of 128 bytes are fetched as they are: asking the L2 for 256 brings the
  // neighbouring head's too, 61 us instead of 43 for eight contexts of 16K with
  // eight heads of 64, slots before heads)
  const EncodeFn fn = encode_fn();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF, int NT>
cudaError_t launch_split(const KArgs& a, const ds_decode_args& g, int blocks,
                         cudaStream_t stream) {
  CUtensorMap tk, tv;
  if (!cache_map(&tk, g.k_cache, g) || !cache_map(&tv, g.v_cache, g))
    return cudaErrorInvalidValue;
  const size_t smem = Cfg<D>::smem;
  const cudaError_t e = allow_smem(split<D, BF, NT>, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(split<D, BF, NT>, dim3(blocks), dim3(kThreads), smem, stream, tk, tv, a,
                          g.kv_layout == DS_KV_HND ? 1 : 0);
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
  a.f16 = g.dtype == DS_KV_F16;
  a.out_type = g.out_f32 ? 2 : g.dtype == DS_KV_BF16 ? 0 : 1;
  a.lse = g.lse;
  a.w_in = g.weights_in;
  a.w_out = g.weights_out;
  a.decay = g.decay;
  a.slot_heads = g.slot_heads;
  a.slot_stride = g.slot_stride;
  unsigned char* ws = static_cast<unsigned char*>(g.workspace);
  a.desc = reinterpret_cast<int2*>(ws + L.desc);
  a.ranges = L.ranges;
  a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.logits = g.weights_out ? reinterpret_cast<float*>(ws + L.logits) : nullptr;
  a.status = reinterpret_cast<uint32_t*>(ws);
  const bool bf = g.dtype == DS_KV_BF16;
  cudaError_t e;
  if (a.group <= 8)
    e = g.head_dim == 128 ? (bf ? launch_split<128, true, 1>(a, g, L.ranges, stream)
                                : launch_split<128, false, 1>(a, g, L.ranges, stream))
                          : (bf ? launch_split<64, true, 1>(a, g, L.ranges, stream)
                                : launch_split<64, false, 1>(a, g, L.ranges, stream));
  else
    e = g.head_dim == 128 ? (bf ? launch_split<128, true, 2>(a, g, L.ranges, stream)
                                : launch_split<128, false, 2>(a, g, L.ranges, stream))
                          : (bf ? launch_split<64, true, 2>(a, g, L.ranges, stream)
                                : launch_split<64, false, 2>(a, g, L.ranges, stream));
  if (e != cudaSuccess) return e;
  // chunks of up to four rows whose weights a slot sums; pieces of a segment
  const int chunks = !a.w_out ? 0 : (a.group + 3) / 4 * (a.slot_heads == 1 ? a.hkv : 1);
  const int pieces = L.ranges / (a.batch * a.hkv) + 1;
  // A warp to 128 slots, each with the rows' own sums (weights per head): 24
  // sequences of 8,000 slots and eight heads of a group of 7 139 us instead of 150,
  // 300 of 200 in room for 2,000 68 instead of 100, of a group of 4 59 instead of
  // 88.  A segment of many pieces makes these sums long (one head's token over
  // 16,384 slots, 257 pieces, 15.3 instead of 10.7; four sequences of it, 77 pieces,
  // 13.1 instead of 12.8), and a few warps with many heads take longer than blocks
  // that share them (16 heads of 1,000 slots 13.2 instead of 11.5).  The rule goes
  // by the capacity all the same, and where pieces are few it stops too early: one
  // sequence of 18,432 slots and eight heads of a group of 4 (39 pieces) 21.5 where a
  // warp to 128 slots takes 20.0, eight of them 107 and 104, one of 32,768 31.2 and
  // 29.6, two of 70,000 of a group of 7 120 and 111.
  const int64_t spans = (int64_t)((a.cache.slots + 127) / 128) * a.batch * a.hkv;
  const bool few = a.w_out && a.slot_heads == a.hkv &&
                   (a.group <= 4 ? a.cache.slots <= 16384
                                 : a.cache.slots <= 65536 && spans >= 8 * 152);
  if (g.head_dim == 128)
    return chunks == 0   ? launch_finish<128, 0, 0>(a, pieces, stream)
           : few         ? launch_finish<128, 0, 1>(a, pieces, stream)
           : chunks == 1 ? launch_finish<128, 16, 1>(a, pieces, stream)
           : chunks < 8  ? launch_finish<128, 4, 4>(a, pieces, stream)
                         : launch_finish<128, 2, 8>(a, pieces, stream);
  return chunks == 0   ? launch_finish<64, 0, 0>(a, pieces, stream)
         : few         ? launch_finish<64, 0, 1>(a, pieces, stream)
         : chunks == 1 ? launch_finish<64, 16, 1>(a, pieces, stream)
         : chunks < 8  ? launch_finish<64, 4, 4>(a, pieces, stream)
                       : launch_finish<64, 2, 8>(a, pieces, stream);
}

}  // namespace ds
