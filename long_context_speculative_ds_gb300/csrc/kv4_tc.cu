// Split pass of ds_kv4_verify_attn for trees, on the 5th-generation tensor
// cores (tcgen05) of sm_103a, and the pass that joins the splits.
//
// softmax(scale Q K^T) V by one pass over the keys with a running reference
// point and sum per row, as in the bf16 cache's split pass (verify_tc.cu:
// work items, softmax groups, P V / Q K order, split outputs), over tiles of
// 128 keys that arrive in 4 bits and are brought to f16 in shared memory,
// where code x scale is exact.  P is f16 too, with a reference point 2^7
// below the row's maximum (verify_softmax.cuh).
//
// The two products of 256 query rows with 128K keys of eight heads (137
// GFLOP) are 70 us of the tensor pipe at its measured rate; the 151 MB of the
// cache are 23 us.  A call over 64 nodes and 32 query heads takes 122 us, 1.13
// PFLOP/s or 57 %: about 22 us go into the start (plan 2.5, Q 2.5, first
// tile), the split outputs (2.5) and the join (8), and in between a tile takes
// 1.8 us: 1.2 of products, 1.2 of softmax (0.9 with nothing beside it) and 0.7
// of conversion share issue slots and wait for one another.
//
// More than 128 rows ("row mode"): each of two softmax groups has a tile of
// 128 rows and goes through all keys.  Up to 128 rows ("key mode"): both
// groups have the same rows and take every other tile of keys; their outputs
// are merged in the end.  A tile takes 1.2 us in key mode, 1.8 in row mode.
//
// 16 warps:
//   warp 0      loader: page blocks (codes and scales of one page of one kv
//               head, contiguous) into a ring of raw tiles by bulk copies;
//               pages past the sequence end are not copied (no byte of the
//               cache format reads as NaN or infinity, and their weights are
//               zero), bad pages are marked and read as zeros.
//   warp 1      tensor-memory allocator and ancestor masks; in key mode then
//               V's loader, with a ring of its own (one loader for both was
//               the slowest part there: 106 us against 99 for 8 nodes over
//               128K).  In row mode one keeps up, and there is no room.
//   warps 2, 3  MMA issuers of softmax groups 0 and 1.
//   warps 4-7, 8-11   softmax groups; at the start they also bring Q to f16.
//   warps 12-15 converters, 32 keys of a tile a warp.  Four warps do: a
//               second team, with 20 warps and fewer registers each, made a
//               row-mode call 152 us instead of 125, and reading the cache
//               into registers without the raw ring a key-mode call 148
//               instead of 106.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "dev_common.cuh"
#include "internal.h"
#include "kv4_common.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"
#include "verify_common.cuh"
#include "verify_softmax.cuh"

namespace ds {
namespace kv4tc {

constexpr int kThreads = 512;
constexpr uint32_t kHalfBytes = 128 * 128;
constexpr int kTmemCols = 512;
constexpr int kRing = 3;         // raw slots of a ring: one for K and V in row mode, one
                                 // for each in key mode (V's in the unused second Q tile)

// The products complete two kinds of barrier: one per 64-key unit of a group,
// when its P V and the next tile's S are done, and one per tile, when with the
// tile's last S its K and an earlier tile's V are free.
enum Bar {
  kQFull = 0,
  kKFull = 1,      // 2 slots
  kVFull = 3,
  kFree = 5,       // [t % 2]: S of tile t is done and with it, in row mode, P V
                   // of tile t - 1 (in key mode, of the group's: t - 2)
  kRawFull = 7,    // 6 slots
  kRawEmpty = 13,
  kSFull = 19,     // [group][half]: S is ready, and P V of the half before done
  kPFull = 23,     // [group][half]
  kOFinal = 27,    // [group]
  kAnc = 29,
  kNumBars = 30
};

struct Ctrl {
  uint64_t bar[kNumBars];
  uint32_t tmem_base;
  int abort;
  Plan plan;
  int kvh, rgi, t0, t1, rows;    // of the item: kv head, row group, tiles, rows; 0 without one
  int32_t parents[DS_MAX_TREE_NODES];
  uint64_t anc[DS_MAX_TREE_NODES];
  uint32_t bad[2 * kRing];       // bad pages of each raw tile, one bit a page
  uint32_t where[6];             // last wait site of loader, issuers, softmax groups, converters
  int last;
};

template <int D>
struct Cfg {
  static constexpr int TB = 128 * D * 2;            // bytes of one 128-row f16 tile
  static constexpr int NH = D / 64;
  static constexpr uint32_t RG = NH * 1024;
  static constexpr int RAW = DS_KV4_BLOCK_BYTES(128, D);
  // Q (2 tiles), K and V (2 slots each), raw tiles, control block
  static constexpr size_t smem = 6 * TB + kRing * RAW + sizeof(Ctrl) + 1024;
  static_assert(smem <= 232448, "dynamic shared memory above the 227 KB a block can have");
  static_assert(4 * 32 * 32 * 4 <= TB, "output staging must fit in a Q tile");
  static_assert(kRing * RAW <= TB, "extra raw slots must fit in a Q tile");
  static_assert(1024 <= kRing * RAW, "the merge's maxima and sums must fit in the raw ring");
};

// Cost of a tile: 1.28 us in key mode, 1.87 us in row mode (128K, 32 heads of
// 128; calls over heads of 64 take 70 and 117 us there, 5 : 8, with the same)
DS_DEV int tile_cost(const SeqPlan& s) { return s.rows <= 128 ? 5 : 7; }

// The work item of this block, by one warp: near-equal ranges of tiles per
// row group, of a cost of at most q (but for the rounding to tiles) each.  q
// is the even share when its items fit one block per SM; else the smallest of
// 32 candidates that does, tried at once, a lane each; and when that would
// cost more than 15 % and the grid has room, the smallest that fits two.
__device__ __noinline__ Plan kv4_plan(const PlanArgs& a, int item) {
  const int lane = threadIdx.x & 31;
  // tiles and row groups of the first 32 sequences, a lane each
  SeqPlan s0{0, 0, 0, 0, 0, 0, 0, 0};
  if (lane < a.batch) s0 = seq_sizes(a, lane, item == 0);
  auto seq = [&](int b0) {
    if (b0 == 0) return s0;
    SeqPlan s{0, 0, 0, 0, 0, 0, 0, 0};
    if (b0 + lane < a.batch) s = seq_sizes(a, b0 + lane, item == 0);
    return s;
  };
  auto splits = [](int tiles, int cost, int q) {
    const int t = (q + cost - 1) / cost;
    return (tiles + t - 1) / t;
  };
  int64_t total = 0;
  int most = 1;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const SeqPlan s = seq(b0);
    const int cost = s.tiles * tile_cost(s);
    const int64_t u = (int64_t)cost * a.num_kv_heads * s.rg;
    total += ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)(u >> 24)) << 24) +
             __reduce_add_sync(0xffffffffu, (unsigned)u & 0xffffffu);
    most = max(most, (int)__reduce_max_sync(0xffffffffu, (unsigned)cost));
  }
  const int ctas = max(1, a.target_ctas);
  const int64_t up = total + ctas - 1;
  const int64_t share = up >> 32 ? up / ctas : (int64_t)((uint32_t)up / (uint32_t)ctas);
  int q = (int)max((int64_t)1, min((int64_t)most, share));
  int fits = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const SeqPlan s = seq(b0);
    fits += (int)__reduce_add_sync(
        0xffffffffu, (unsigned)(a.num_kv_heads * s.rg * splits(s.tiles, tile_cost(s), q)));
  }
  if (fits > a.target_ctas) {
    // items at q, each lane its own q
    auto items_at = [&](int q) {
      int it = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const SeqPlan s = seq(b0);
        const int groups = a.num_kv_heads * s.rg, cost = tile_cost(s), n = min(32, a.batch - b0);
        for (int k = 0; k < n; ++k)
          it += __shfl_sync(0xffffffffu, groups, k) *
                splits(__shfl_sync(0xffffffffu, s.tiles, k), __shfl_sync(0xffffffffu, cost, k), q);
      }
      return it;
    };
    // the smallest of 32 candidates from q0 up, in steps of a sixteenth, whose
    // items fit; the longest sequence's cost when none does
    auto smallest = [&](int q0, int fit) {
      const int x = (int)min((int64_t)most, q0 + ((int64_t)q0 * lane + 15) / 16);
      const uint32_t ok = __ballot_sync(0xffffffffu, items_at(x) <= fit);
      return ok ? __shfl_sync(0xffffffffu, x, __ffs(ok) - 1) : most;
    };
    const int even = q;
    q = smallest(even, a.target_ctas);
    if (a.wave_ctas > a.target_ctas && (int64_t)q * 100 > (int64_t)even * 115)
      q = min(q, smallest(max(1, even / 2), a.wave_ctas));
  }
  // the sequence that owns the item
  Plan p;
  p.tps = q;
  p.b = -1;
  p.seq = SeqPlan{0, 0, 0, 0, 0, 0, 0, 0};
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    SeqPlan s = seq(b0);
    s.splits = splits(s.tiles, tile_cost(s), q);
    const int items = a.num_kv_heads * s.rg * s.splits;
    int incl = items;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    s.item_base = base + incl - items;
    const uint32_t m =
        __ballot_sync(0xffffffffu, item >= s.item_base && item < s.item_base + items);
    if (m) {
      const int src = __ffs(m) - 1;
      p.b = b0 + src;
      p.seq.L = __shfl_sync(0xffffffffu, s.L, src);
      p.seq.T = __shfl_sync(0xffffffffu, s.T, src);
      p.seq.node0 = __shfl_sync(0xffffffffu, s.node0, src);
      p.seq.tiles = __shfl_sync(0xffffffffu, s.tiles, src);
      p.seq.rows = __shfl_sync(0xffffffffu, s.rows, src);
      p.seq.rg = __shfl_sync(0xffffffffu, s.rg, src);
      p.seq.splits = __shfl_sync(0xffffffffu, s.splits, src);
      p.seq.item_base = __shfl_sync(0xffffffffu, s.item_base, src);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  p.total_items = base;
  return p;
}

// Output of one softmax thread after its last tile: O / l and the row's
// log2-sum-exp.  In key mode group 1 leaves its O, maximum and sum in shared
// memory and group 0 merges them.  A warp's rows go through a staging tile of
// 32 rows x 32 columns (idle by then), so that a store instruction covers
// whole sectors; 16-byte chunk c of row r is staged where eight lanes of an
// access, eight rows' or a row's, touch all banks.
template <int D>
__device__ __noinline__ void write_split(const bool row_mode, const int g, const bool ok,
                                         const int nt1, const uint32_t tO, const int lrow,
                                         const int rows_left, const float m2, const float l,
                                         float* __restrict__ merge_buf, float* m1buf,
                                         float* l1buf, unsigned char* __restrict__ stage,
                                         const bool f32, void* __restrict__ dst,
                                         float* __restrict__ lse_out, const float out_mult) {
  using namespace ptx;
  const int lane = threadIdx.x & 31;
  const bool merge = !row_mode && nt1 > 0;
  if (!row_mode && g == 1) {
    if (ok && merge) {
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        uint32_t r[32];
        tmem_ld32(tO + c4 * 32, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) merge_buf[(c4 * 32 + i) * 128 + lrow] = __uint_as_float(r[i]);
      }
      m1buf[lrow] = m2;
      l1buf[lrow] = l;
    }
    if (merge) asm volatile("bar.sync 1, 256;" ::: "memory");
    return;
  }
  float k0 = 1.f, k1 = 0.f, lt = l, mt = m2;
  if (merge) {
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float m1 = m1buf[lrow], l1 = l1buf[lrow];
    mt = fmaxf(m2, m1);
    const float mb = mt == -CUDART_INF_F ? 0.f : mt;
    k0 = l > 0.f ? ex2(m2 - mb) : 0.f;
    k1 = l1 > 0.f ? ex2(m1 - mb) : 0.f;
    lt = l * k0 + l1 * k1;
  }
  if (lane < rows_left) *lse_out = lt > 0.f ? mt + __log2f(lt) : -CUDART_INF_F;
  const float inv = lt > 0.f ? __fdividef(out_mult, lt) : 0.f;
  k0 *= inv;
  k1 *= inv;
#pragma unroll 1
  for (int c4 = 0; c4 < D / 32; ++c4) {
    uint32_t r[32];
    if (ok) {
      tmem_ld32(tO + c4 * 32, r);
      tmem_ld_wait(r);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * k0);
    if (merge && k1 != 0.f) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(
            fmaf(merge_buf[(c4 * 32 + i) * 128 + lrow], k1, __uint_as_float(r[i])));
    }
    if (!f32) {
      // four 16-byte chunks a row, chunk c in place c ^ ((row / 2) % 4)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_f16x2(__uint_as_float(r[8 * c + 2 * e]),
                            __uint_as_float(r[8 * c + 2 * e + 1]));
        *reinterpret_cast<uint4*>(stage + lane * 64 + 16 * (c ^ ((lane >> 1) & 3))) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = 8 * k + (lane >> 2), cc = lane & 3;
        if (rr < rows_left)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + (int64_t)rr * D + c4 * 32 +
                                    cc * 8) =
              *reinterpret_cast<const uint4*>(stage + rr * 64 + 16 * (cc ^ ((rr >> 1) & 3)));
      }
    } else {
      // eight chunks a row, chunk c in place c ^ (row % 8)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * (c ^ (lane & 7))) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rr = 4 * k + (lane >> 3), cc = lane & 7;
        if (rr < rows_left)
          *reinterpret_cast<uint4*>(static_cast<float*>(dst) + (int64_t)rr * D + c4 * 32 +
                                    cc * 4) =
              *reinterpret_cast<const uint4*>(stage + rr * 128 + 16 * (cc ^ (rr & 7)));
      }
    }
    __syncwarp();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_split_tc(const Kv4KArgs ka) {
  using namespace ptx;
  using tc::softmax_unit;
  const VerifyKArgs& a = ka.v;
  constexpr int TB = Cfg<D>::TB;
  constexpr uint32_t RG = Cfg<D>::RG;
  constexpr int RAW = Cfg<D>::RAW;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t sQ = sbase;
  const uint32_t sK = sbase + 2 * TB;
  const uint32_t sV = sbase + 4 * TB;
  const uint32_t sR = sbase + 6 * TB;
  // key-mode merge scratch, used once all MMAs have completed: O of group 1
  // over the V slots, its row maxima and sums over the raw ring
  float* merge_buf = reinterpret_cast<float*>(smem + 4 * TB);
  float* m1buf = reinterpret_cast<float*>(smem + 6 * TB);
  float* l1buf = m1buf + 128;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + 6 * TB + kRing * RAW);
  volatile int* abort_flag = &ctrl->abort;
  uint32_t* diag = a.plan.status + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return smem_addr(&ctrl->bar[i]); };

  // ---------------------------------------------------------------- set-up
  if (warp == 1 && lane == 0) {
    mbar_init(bar(kQFull), 256);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kKFull + s), 4);      // one arrival per converter warp
      mbar_init(bar(kVFull + s), 4);
      mbar_init(bar(kOFinal + s), 1);
    }
    for (int s = 0; s < 2 * kRing; ++s) {
      mbar_init(bar(kRawFull + s), 1);
      mbar_init(bar(kRawEmpty + s), 4);
    }
    for (int s = 0; s < 4; ++s) mbar_init(bar(kSFull + s), 1);
    for (int s = 0; s < 4; ++s) mbar_init(bar(kPFull + s), 128);
    mbar_init(bar(kAnc), 32);
    ctrl->abort = 0;
    for (int i = 0; i < 6; ++i) ctrl->where[i] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctrl->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  // the item, and the barriers whose arrivals depend on it
  auto find_item = [&]() {
    const Plan p = kv4_plan(a.plan, blockIdx.x);
    int kvh = 0, rgi = 0, t0 = 0, t1 = 0, rows = 0;
    if ((int)blockIdx.x < p.total_items && p.b >= 0) {
      const SeqPlan& sq = p.seq;
      const int local = blockIdx.x - sq.item_base;
      const int grp = local / sq.splits, split = local - grp * sq.splits;
      kvh = grp / sq.rg;
      rgi = grp - kvh * sq.rg;
      const int base = sq.tiles / sq.splits, rem = sq.tiles - base * sq.splits;
      t0 = split * base + min(split, rem);
      t1 = t0 + base + (split < rem ? 1 : 0);
      rows = min(kRowsPerGroup, sq.rows - rgi * kRowsPerGroup);
    }
    if (lane == 0) {
      ctrl->plan = p;
      ctrl->kvh = kvh; ctrl->rgi = rgi; ctrl->t0 = t0; ctrl->t1 = t1; ctrl->rows = rows;
      // both groups' arrivals in row mode, the tile's own group's in key mode
      for (int s = 0; s < 2; ++s) mbar_init(bar(kFree + s), rows > 128 ? 2 : 1);
      fence_mbar_init();
    }
  };
  const bool early_plan = a.accumulate != 0;
  if (early_plan && warp == 0) find_item();
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (!early_plan && warp == 0) find_item();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  const Plan& p = ctrl->plan;           // stays in shared memory: registers are scarce
  const SeqPlan& sq = p.seq;
  const int kvh = ctrl->kvh, rgi = ctrl->rgi, t0 = ctrl->t0, rows_here = ctrl->rows;
  const int G = a.plan.group, nt = ctrl->t1 - t0;
  const bool active = nt > 0, row_mode = rows_here > 128;
  const int L = sq.L, T = sq.T;
  const bool need_anc = active && (t0 + nt) * kTileKeys > L;
  auto raw_addr = [&](int s) -> uint32_t {
    return s < kRing ? sR + s * RAW : sQ + TB + (s - kRing) * RAW;
  };
  // Tiles are loaded and converted in the order the MMAs need them: K runs
  // one tile ahead of V (two in key mode, where both groups start at once).
  // In row mode K and V share a ring of raw slots; in key mode each has one,
  // and a loader.  The walk keeps counters instead of dividing: a single warp
  // follows it, and every instruction adds its latency to each tile's turn.
  enum { kAll = 0, kOnlyK = 1, kOnlyV = 2 };
  struct Walk {
    int what, lead, nt;
    int k = 0, v = 0;              // K and V tiles taken so far
    bool is_v = false;             // the tile at hand
    int n = 0;
    int slot = 0, phase = 0;       // its raw slot, and the parity of that slot's uses
    int other_slot, other_phase = 0;             // of the ring that is not at hand
    bool other_v = true, two;
    __device__ bool take() {       // false at the end
      if ((what == kOnlyK ? k : v) == nt) return false;
      is_v = what == kOnlyV || (what == kAll && (k >= nt || k >= v + lead));
      n = is_v ? v++ : k++;
      if (two && is_v == other_v) {
        const int s = slot, p = phase;
        slot = other_slot; phase = other_phase;
        other_slot = s; other_phase = p;
        other_v = !other_v;
      }
      return true;
    }
    __device__ void release() {    // on to the next raw slot of the ring
      if (++slot == kRing || slot == 2 * kRing) {
        slot -= kRing;
        phase ^= 1;
      }
    }
  };
  auto walk = [&](int what) {
    Walk w;
    w.what = what;
    w.lead = row_mode ? 1 : 2;
    w.nt = nt;
    w.two = !row_mode;
    w.other_slot = kRing;
    return w;
  };
  // tiles of group g: row mode every tile, key mode every other tile (so
  // slot n % 2 is then always group n % 2's)
  auto ntiles = [&](int g) { return row_mode ? nt : (nt - g + 1) / 2; };
  auto tile_of = [&](int g, int j) { return row_mode ? j : 2 * j + g; };

  // registers move from the loader's and the converters' warpgroups to the
  // softmax groups: 128 (88 + 88) + 256 x 168 = the launch's 512 x 128.  At 80
  // the issuers spill.  With 128-wide heads nothing spills then; with 64-wide
  // ones the paired conversion does (48 bytes stored, 296 loaded), and is
  // faster all the same.
  static_assert(128 * (88 + 88) + 256 * 168 <= kThreads * 128, "more than the launch has");
  if (warp < 4) {
    regs_release<88>();
    if (!active) {
    } else if (warp < 2) {
      // ---------------------------------------------------- ancestor masks
      if (warp == 1 && need_anc) {
        tc::tree_ancestors(a.parents + sq.node0, T, ctrl->parents, ctrl->anc, a.plan.status);
        mbar_arrive(bar(kAnc));
      }
      if (warp == 0 || !row_mode) {
        // ------------------------------------------------------------ loader
        const int P = a.plan.page_size;
        const int npg = kTileKeys / P;
        const uint32_t blk = DS_KV4_BLOCK_BYTES(P, D);
        const int32_t* ptab = a.page_table + (int64_t)p.b * a.plan.max_pages;
        const uint64_t policy = l2_evict_first();
        // Page ids come 32 at a time, a run of 32 / npg tiles, the next run on
        // its way (a load per tile would put its latency into every tile's
        // turn), and are checked together; lane r of a run holds page r of it.
        // K and V walk their own runs.
        const int rshift = __ffs(P) - 1 - 2;       // log2 of the tiles of a run, P / 4
        const int run = 1 << rshift, pend = (L + T + P - 1) / P;
        const uint32_t page_bytes = a.plan.num_kv_heads * blk;
        struct Side {                              // of K, of V
          const uint8_t* head;
          int ids, next;
          uint32_t bad;
        } side[2];
        auto ids_of = [&](int r) {
          const int pi = (t0 + r * run) * npg + lane;
          return pi < pend ? __ldg(ptab + pi) : 0;
        };
        auto check = [&](Side& x) {
          const bool bad = (uint32_t)x.ids >= (uint32_t)a.num_pages;
          if (bad) flag(a.plan.status, DS_DEV_BAD_PAGE);
          x.bad = __ballot_sync(0xffffffffu, bad);
        };
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          side[v].head = (v ? ka.v4 : ka.k4) + (int64_t)kvh * blk;
          side[v].ids = ids_of(0);
          side[v].next = ids_of(1);
          check(side[v]);
        }
        bool ok = true;
        const uint32_t pmask = npg == 8 ? 0xffu : (1u << npg) - 1u;
        Walk w = walk(row_mode ? kAll : warp == 0 ? kOnlyK : kOnlyV);
        auto load = [&](Side& x) {
          const int in_run = w.n & (run - 1);
          if (w.n > 0 && in_run == 0) {
            x.ids = x.next;
            x.next = ids_of((w.n >> rshift) + 1);
            check(x);
          }
          const uint32_t pg = __shfl_sync(0xffffffffu, x.ids, (in_run * npg + lane) & 31);
          const uint32_t badm = (x.bad >> (in_run * npg)) & pmask;
          const int left = pend - (t0 + w.n) * npg;          // pages of the sequence from here on
          const bool have = lane < min(npg, left) && !((badm >> lane) & 1u);
          const int n = min(npg, left) - __popc(badm);
          const uint32_t full = bar(kRawFull + w.slot);
          const uint32_t tag = 10000 + 2 * w.n + (w.is_v ? 1 : 0);
          if (lane == 0 && warp == 0) ctrl->where[0] = tag;
          if (!__all_sync(0xffffffffu, mbar_wait(bar(kRawEmpty + w.slot), w.phase ^ 1, abort_flag,
                                                 diag, tag)))
            return false;
          if (lane == 0) {
            ctrl->bad[w.slot] = badm;
            mbar_arrive_expect_tx(full, n * blk);
          }
          __syncwarp();
          if (have)
            bulk_load_hint(raw_addr(w.slot) + lane * blk, x.head + (uint64_t)pg * page_bytes, blk,
                           full, policy);
          return true;
        };
        while (w.take()) {
          ok = w.is_v ? load(side[1]) : load(side[0]);
          if (!ok) break;
          w.release();
        }
        if (lane == 0 && warp == 0) ctrl->where[0] = ok ? 19999 : 19998;
        // copies still in flight must land before the CTA can exit: each slot's
        // last phase (a slot not used yet passes at once)
        if (!ok && lane == 0)
          for (int s0 = w.slot < kRing ? 0 : kRing, i = s0; i < s0 + kRing; ++i)
            drain_wait(bar(kRawFull + i), i >= w.slot ? w.phase ^ 1 : w.phase);
      }
    } else {
      // ------------------------------------------------------ MMA issuers
      const int g = warp - 2;
      if (lane == 0) {
        constexpr uint32_t idesc_qk = idesc_f16_f32(128, 64, false);
        constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
        const uint64_t qd0 = sdesc_sw128(sQ, 16, 1024);
        const uint64_t qb = (row_mode && g == 1) ? qd0 + (TB >> 4) : qd0;
        const uint64_t kd0 = sdesc_sw128(sK, 16, RG);
        const uint64_t vd0 = sdesc_sw128(sV, 1024, RG);
        const uint32_t tG = tmem + (uint32_t)(256 * g);
        auto qk = [&](int t, int h) {
          const uint64_t kb = kd0 + (uint64_t)((t & 1) * (TB >> 4) + h * ((8 * RG) >> 4));
          const uint32_t d = tG + (uint32_t)(64 * h);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qoff = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
            const uint32_t koff = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
            mma_ss(d, qb + qoff, kb + koff, idesc_qk, kk > 0);
          }
        };
        auto pv = [&](int t, int h, bool acc) {
          const uint64_t vb = vd0 + (uint64_t)((t & 1) * (TB >> 4) + h * ((8 * RG) >> 4));
          const uint32_t pa = tG + (uint32_t)(64 * h);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tG + 128, pa + kk * 8, vb + (uint64_t)(kk * ((2 * RG) >> 4)), idesc_pv,
                   (acc || kk > 0) ? 1u : 0u);
        };
        const int wi = 1 + g;
        auto wait = [&](int b, uint32_t par, uint32_t tag) {
          ctrl->where[wi] = tag;
          return mbar_wait(bar(b), par, abort_flag, diag, tag);
        };
        auto wait_k = [&](int t) {
          return wait(kKFull + (t & 1), (t >> 1) & 1, 20000 + kKFull * 100 + t);
        };
        auto wait_v = [&](int t) {
          return wait(kVFull + (t & 1), (t >> 1) & 1, 20000 + kVFull * 100 + t);
        };
        const int my_nt = ntiles(g);
        bool ok = wait(kQFull, 0, 20000 + kQFull * 100);
        if (ok && my_nt > 0) {
          const int t = tile_of(g, 0);
          if ((ok = wait_k(t))) {
            tc_fence_after();
            for (int h = 0; h < 2; ++h) {
              qk(t, h);
              mma_commit(bar(kSFull + 2 * g + h));
            }
            mma_commit(bar(kFree + (t & 1)));
          }
        }
        for (int j = 0; ok && j < my_nt; ++j) {
          const int n = tile_of(g, j);
          const int tn = row_mode ? n + 1 : n + 2;
          const bool more = j + 1 < my_nt;
          for (int h = 0; h < 2; ++h) {
            if (!(ok = wait(kPFull + 2 * g + h, j & 1,
                            20000 + (kPFull + 2 * g + h) * 100 + 2 * j + h)))
              break;
            if (h == 0 && !(ok = wait_v(n))) break;
            // K is looked at before the products are issued: afterwards a
            // look at a barrier waits until they have drained
            const bool k_there =
                h == 1 || !more || mbar_try_wait(bar(kKFull + (tn & 1)), (tn >> 1) & 1);
            tc_fence_after();
            pv(n, h, j > 0 || h > 0);
            if (more) {
              if (!k_there) {
                if (!(ok = wait_k(tn))) break;
                tc_fence_after();
              }
              qk(tn, h);
            }
            mma_commit(bar(kSFull + 2 * g + h));
            if (h == 1) mma_commit(bar(kFree + (tn & 1)));
          }
        }
        if (ok) ctrl->where[wi] = 29999;
        mma_commit(bar(kOFinal + g));
      }
    }
  } else if (warp < 12) {
    regs_claim<168>();
    if (active) {
      // ------------------------------------------------------------ softmax
      const int g = (warp - 4) >> 2;
      const int q4 = warp & 3;
      const int lrow = q4 * 32 + lane;
      const int grow_local = row_mode ? g * 128 + lrow : lrow;
      const bool row_ok = grow_local < rows_here;
      const bool idle = grow_local - lane >= rows_here;        // a warp without rows
      const int grow = rgi * kRowsPerGroup + grow_local;
      const int jn = grow / G;
      // the group's query rows as f16 into its Q tile (key mode: one tile,
      // group 0's): 16-byte chunks, a row's by consecutive lanes, all of a
      // thread's on their way at once
      if (row_mode || g == 0) {
        constexpr int CPR = D / 8;                   // chunks of a row
        constexpr int RPI = 32 / CPR;                // rows of a warp's load
        const int ch = lane % CPR;
        const uint32_t dst = sQ + (row_mode ? g * TB : 0) + (ch >> 3) * kHalfBytes;
        // row / G as a product: exact, as rows times G stay below 2^32
        const uint32_t inv = G > 1 ? 0xffffffffu / G + 1u : 0u;
        uint4 x[32 / RPI];
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
          const int rl = q4 * 32 + i * RPI + lane / CPR;          // row of the tile
          const int rr = (row_mode ? g * 128 : 0) + rl;
          const int gr = rgi * kRowsPerGroup + rr;
          x[i] = make_uint4(0, 0, 0, 0);
          const int node = G > 1 ? (int)__umulhi((uint32_t)gr, inv) : gr;
          if (rr < rows_here)
            x[i] = __ldg(reinterpret_cast<const uint4*>(
                             a.q + ((int64_t)(sq.node0 + node) * a.num_q_heads + kvh * G +
                                    (gr - node * G)) * D) + ch);
        }
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
          const int rl = q4 * 32 + i * RPI + lane / CPR;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           dst + rl * 128 + (((ch & 7) ^ (rl & 7)) << 4)),
                       "r"(bf16x2_to_f16x2(x[i].x)), "r"(bf16x2_to_f16x2(x[i].y)),
                       "r"(bf16x2_to_f16x2(x[i].z)), "r"(bf16x2_to_f16x2(x[i].w))
                       : "memory");
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(bar(kQFull));
      uint64_t anc = 0ull;
      bool anc_ready = !need_anc;
      const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
      const uint32_t tG = tmem + lane_addr + 256 * g;
      const uint32_t tO = tG + 128;
      const float c2 = a.scale_log2;
      const int C = a.plan.chunk_size;
      const int cshift = __ffs(C) - 1;
      const int n_ch = a.scores ? (L + C - 1) / C : 0;
      float* clse_row = a.clse +
                        (((int64_t)p.b * a.plan.num_kv_heads + kvh) * a.plan.rg_max + rgi) *
                            a.plan.max_chunks * kRowsPerGroup +
                        grow_local;
      float m2 = -CUDART_INF_F, l = 0.f, cs = 0.f;
      bool ok = true;
      const int my_nt = ntiles(g);
      const int wi = 3 + g;
      for (int j = 0; ok && j < my_nt; ++j) {
        const int n = tile_of(g, j);
        const int tile_slot0 = (t0 + n) * kTileKeys;
        for (int hb = 0; hb < 2; ++hb) {
          const int u = 2 * j + hb;
          if (lrow == 0) ctrl->where[wi] = 30000 + (kSFull + 2 * g + hb) * 100 + j;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kSFull + 2 * g + hb), j & 1, abort_flag,
                                                 diag, 30000 + (kSFull + 2 * g + hb) * 100 + j));
          if (!ok) break;
          if (idle) {                    // its part of P is never read back
            mbar_arrive(bar(kPFull + 2 * g + hb));
            continue;
          }
          tc_fence_after();
          const uint32_t tS = tG + 64 * hb;
          const int unit_slot0 = tile_slot0 + 64 * hb;
          float alpha;
          bool rescale;
          if (unit_slot0 + 64 <= L) {
            softmax_unit<false, true>(tS, tS, ~0u, ~0u, ~0u, ~0u, c2, u == 0, m2, l, cs, alpha,
                                      rescale, tile_slot0, 4 * hb, cshift, n_ch, row_ok,
                                      clse_row);
          } else if (unit_slot0 >= L + T && u > 0) {
            // past the end: zero weights; a chunk of the context may end here
            alpha = 1.f;
            rescale = false;
            const int c = unit_slot0 >> cshift;
            if (row_ok && c < n_ch)
              clse_row[(int64_t)c * kRowsPerGroup] = cs > 0.f ? m2 + __log2f(cs) : -CUDART_INF_F;
            cs = 0.f;
            uint32_t zero[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) zero[i] = 0u;
            tmem_st32(tS, zero);
          } else {
            if (!anc_ready) {
              if (lrow == 0) ctrl->where[wi] = 30000 + kAnc * 100;
              ok = __all_sync(0xffffffffu, mbar_wait(bar(kAnc), 0, abort_flag, diag,
                                                     30000 + kAnc * 100));
              if (!ok) break;
              anc = (row_ok && jn < T) ? ctrl->anc[jn] : 0ull;
              anc_ready = true;
            }
            const int off = L - unit_slot0;
            const uint64_t ctx = off >= 64 ? ~0ull : (off <= 0 ? 0ull : ((1ull << off) - 1));
            const uint64_t tr = off >= 0 ? (off >= 64 ? 0ull : (anc << off))
                                         : (-off >= 64 ? 0ull : (anc >> (-off)));
            const uint64_t vis = ctx | tr;
            softmax_unit<true, true>(tS, tS, (uint32_t)vis, (uint32_t)(vis >> 32),
                                     (uint32_t)ctx, (uint32_t)(ctx >> 32), c2, u == 0, m2, l, cs,
                                     alpha, rescale, tile_slot0, 4 * hb, cshift, n_ch, row_ok,
                                     clse_row);
          }
          if (rescale) {
            // O must hold every earlier half: the half before this one is
            // done with the other half's next S
            if (lrow == 0) ctrl->where[wi] = 35000 + u;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(bar(kSFull + 2 * g + 1 - hb), (hb ? j + 1 : j) & 1,
                                      abort_flag, diag, 35000 + u));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int c4 = 0; c4 < D / 32; ++c4) {
                uint32_t r[32];
                tmem_ld32(tO + c4 * 32, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                tmem_st32(tO + c4 * 32, r);
              }
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(kPFull + 2 * g + hb));
          if (!ok) break;
        }
      }
      // ------------------------------------------------------------ epilogue
      if (lrow == 0) ctrl->where[wi] = 30000 + (kOFinal + g) * 100;
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kOFinal + g), 0, abort_flag, diag,
                                               30000 + (kOFinal + g) * 100));
      if (ok && !row_mode)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kOFinal + 1 - g), 0, abort_flag, diag,
                                               30000 + (kOFinal + 1 - g) * 100));
      else __syncwarp();
      if (ok) tc_fence_after();
      const int nt1 = row_mode ? 0 : ntiles(1);
      unsigned char* stage = smem + (row_mode ? g * TB : 0) + q4 * 4096;
      const int warp_row0 = grow_local - lane;
      const int64_t orow = ((int64_t)blockIdx.x * kRowsPerGroup + warp_row0) * D;
      void* op_warp = a.out_f32 ? static_cast<void*>(a.o_part + orow)
                                : static_cast<void*>(
                                      reinterpret_cast<uint16_t*>(a.o_part) + orow);
      // A split's output is a weighted mean of code x scale, at most 2688: f16
      // holds it with three more bits than bf16, to 2^-25 at worst; the
      // cache's exponent is applied where the splits meet.
      write_split<D>(row_mode, g, ok, nt1, tO, lrow, rows_here - warp_row0, m2, l, merge_buf,
                     m1buf, l1buf, stage, a.out_f32, op_warp,
                     a.lse_part + (int64_t)blockIdx.x * kRowsPerGroup + grow_local,
                     a.out_f32 ? ka.out_mult : 1.f);
    }
  } else {
    regs_release<88>();
    if (active) {
      // ---------------------------------------------------------- converters
      // A lane takes one 16-byte piece pc (32 channels) of a key per round, a
      // warp 8 keys (16 at head_dim 64), and the rounds of a warp's 32 keys are
      // a constant apart but for a page's end.  Of eight lanes, four keys with
      // the low bits r, the reads (piece pc of key r) and the writes (chunk
      // 4 pc + k in place of chunk (4 pc + k) ^ key % 8) touch all banks once.
      constexpr int NJ = D / 32;                       // rounds
      constexpr int KPR = 32 / NJ;                     // keys of a round
      const int P = a.plan.page_size;
      const int r = (lane >> 1) & 3, ph = lane >> 3;
      const int pc = D == 128 ? (lane & 1) + 2 * (((lane >> 2) ^ ph) & 1) : lane & 1;
      const int key = (warp - 12) * 32 + r + 4 * (D == 128 ? ph >> 1 : ph);
      const int pidx = key / P, off = key % P;
      // the first key's piece and scales inside a raw tile; the second half of
      // the rounds is a page further on when pages have 16 keys
      const uint32_t blk = DS_KV4_BLOCK_BYTES(P, D);
      const uint32_t ccode = pidx * blk + off * (D / 2) + pc * 16;
      const uint32_t cscale = pidx * blk + P * (D / 2) + off * (D / 16) + pc * 2;
      const uint32_t code_hop = P == 16 ? blk - 16 * (D / 2) : 0;
      const uint32_t scale_hop = P == 16 ? blk - 16 * (D / 16) : 0;
      const int bad_hop = P == 16 ? 1 : 0;
      // chunk 4 pc + k of key % 8 is at drow ^ 16 k
      const uint32_t drow = (key >> 3) * RG + (key & 7) * 128 + (pc >> 1) * 1024 +
                            ((((pc & 1) * 4) ^ (key & 7)) << 4);
      const bool rep = warp == 12 && lane == 0;
      // a tile's pieces and scales of this lane, from its raw slot
      auto read = [&](int slot, uint4 (&c)[NJ], uint32_t (&sb)[NJ]) {
        const uint32_t badm = ctrl->bad[slot] >> pidx;
        const uint32_t raw = raw_addr(slot);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const bool far = j >= NJ / 2;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(c[j].x), "=r"(c[j].y), "=r"(c[j].z), "=r"(c[j].w)
                       : "r"(raw + ccode + j * KPR * (D / 2) + (far ? code_hop : 0)));
          uint16_t h;
          asm volatile("ld.shared.u16 %0, [%1];"
                       : "=h"(h)
                       : "r"(raw + cscale + j * KPR * (D / 16) + (far ? scale_hop : 0)));
          sb[j] = (badm >> (far ? bad_hop : 0)) & 1u ? 0u : h;     // a bad page: scales of zero
        }
      };
      auto put = [&](uint32_t dst, const uint4 (&c)[NJ], const uint32_t (&sb)[NJ]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const uint32_t s2 = kv4_scales_f16(sb[j]);
          const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {      // 16-byte chunk 4 pc + k of the key
            uint32_t v[4];
            kv4_codes_f16(w[k], v);
            const uint32_t s = __byte_perm(s2, s2, k < 2 ? 0x1010 : 0x3232);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             (dst ^ (16 * k)) + j * (KPR / 8) * RG),
                         "r"(hmul2(v[0], s)), "r"(hmul2(v[1], s)), "r"(hmul2(v[2], s)),
                         "r"(hmul2(v[3], s))
                         : "memory");
          }
        }
      };
      // The K behind a V becomes free with it: with 64-wide heads, where waits
      // and fences take more of a tile's time than its conversion, both go at
      // once (8 nodes over 128K: 78 us instead of 84; with 128-wide heads 98
      // either way and 133 instead of 131 for 64 nodes).
      constexpr bool kPair = D == 64;
      bool ok = true;
      Walk w = walk(kAll);
      uint4 c[NJ], c2[NJ];
      uint32_t sb[NJ], sb2[NJ];
      while (w.take()) {
        const int slot = w.slot, n = w.n;
        const bool is_v = w.is_v;
        const uint32_t tag = 40000 + 2 * n + (is_v ? 1 : 0);
        if (rep) ctrl->where[5] = tag;
        ok = mbar_wait(bar(kRawFull + slot), w.phase, abort_flag, diag, tag);
        if (ok && n >= 2) {                // the tile two before has been used
          const int t = is_v ? (row_mode ? n - 1 : n) : n - 2;
          ok = mbar_wait(bar(kFree + (t & 1)), (t >> 1) & 1, abort_flag, diag, tag + 100000);
        }
        if (!__all_sync(0xffffffffu, ok)) break;
        read(slot, c, sb);
        w.release();
        const bool pair = kPair && is_v && n >= 2 && w.k < nt;
        int slot2 = 0, n2 = 0;
        if (pair) {
          w.take();
          slot2 = w.slot;
          n2 = w.n;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kRawFull + slot2), w.phase, abort_flag,
                                                 diag, tag + 200000));
          if (!ok) break;
          read(slot2, c2, sb2);
          w.release();
        }
        put((is_v ? sV : sK) + (n & 1) * TB + drow, c, sb);
        if (pair) put(sK + (n2 & 1) * TB + drow, c2, sb2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar((is_v ? kVFull : kKFull) + (n & 1)));
          mbar_arrive(bar(kRawEmpty + slot));
          if (pair) {
            mbar_arrive(bar(kKFull + (n2 & 1)));
            mbar_arrive(bar(kRawEmpty + slot2));
          }
        }
      }
    }
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    flag(a.plan.status, DS_DEV_TIMEOUT);
    if (diag[1] == blockIdx.x)
      for (int i = 0; i < 6; ++i) diag[2 + i] = ctrl->where[i];
  }
  if (active) {
    // the last split of the row group forms the rows' final log2-sum-exp
    // (see verify_tc.cu)
    const int64_t cidx = ((int64_t)p.b * a.plan.num_kv_heads + kvh) * a.plan.rg_max + rgi;
    const int64_t base = (int64_t)sq.item_base + (kvh * sq.rg + rgi) * sq.splits;
    if (threadIdx.x == 0) {
      __threadfence();
      const uint32_t prev = atomicAdd(a.counters + cidx, 1u);
      const int last = prev + 1 == (uint32_t)sq.splits;
      if (last) {
        a.counters[cidx] = 0u;
        a.gdesc[cidx] = make_int4((int)base, sq.splits, 0, 0);
        __threadfence();
      }
      ctrl->last = last;
    }
    __syncthreads();
    if (ctrl->last)
      for (int r = threadIdx.x; r < rows_here; r += kThreads)
        a.row_lse[cidx * kRowsPerGroup + r] =
            tc::row_lse_from_splits(a.lse_part + base * kRowsPerGroup + r, sq.splits);
  }
  if (warp == 1) {
    if (active && lane == 0) {
      drain_wait(bar(kOFinal), 0);
      drain_wait(bar(kOFinal + 1), 0);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Second launch, bound by the round trips to the L2 (8 us of a 64-node call):
// the first n_comb blocks merge the splits of the output rows,
// a warp per (node, query head); the rest form the chunk scores, a warp per
// (chunk, sequence), four rows a lane, kFinCombos (kv head, row group)
// combinations per round trip.  What only depends on the call's inputs is
// worked out before the wait for the split pass, which has itself waited for
// whatever wrote them.
constexpr int kFinCombos = 2;

template <int D, bool HALF>
DS_DEV void merge_row(const VerifyKArgs& a, int blk, float out_mult) {
  const int lane = threadIdx.x & 31;
  const int64_t x = (int64_t)blk * 8 + (threadIdx.x >> 5);
  const int node = (int)(x / a.num_q_heads), qh = (int)(x - (int64_t)node * a.num_q_heads);
  const int G = a.plan.group, kvh = qh / G;
  // the sequence that owns the node: the last whose offset is at most it
  int b = -1;
  for (int b0 = 0; b0 < a.plan.batch; b0 += 32) {
    const bool in = b0 + lane < a.plan.batch && __ldg(a.plan.tree_offsets + b0 + lane) <= node;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (m) b = b0 + 31 - __clz(m);
  }
  SeqPlan sq{0, 0, 0, 0, 0, 0, 0, 0};
  if (b >= 0 && node < a.plan.n_nodes) sq = seq_sizes(a.plan, b, false);
  const int row = (node - sq.node0) * G + qh % G;
  const int rgi = row / kRowsPerGroup, r = row % kRowsPerGroup;
  const int64_t grp = ((int64_t)max(b, 0) * a.plan.num_kv_heads + kvh) * a.plan.rg_max + rgi;
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (row < 0 || row >= sq.rows) return;          // not a row of a usable sequence
  const int4 gd = __ldcg(a.gdesc + grp);
  const float lse = __ldcg(a.row_lse + grp * kRowsPerGroup + r);
  combine_row_splits<D, HALF, HALF ? (D == 128 ? 20 : 32) : 8, HALF>(a, gd.x, gd.y, r, lse, x,
                                                                     out_mult);
}

DS_DEV void chunk_score(const VerifyKArgs& a, int blk) {
  const int per_b = (a.plan.max_chunks + 7) / 8;
  const int b = blk / per_b, c = blk % per_b * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const SeqPlan sq = seq_sizes(a.plan, b, false);
  const int rg = sq.rg, combos = a.plan.num_kv_heads * rg;
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (c >= (sq.L + a.plan.chunk_size - 1) / a.plan.chunk_size) return;
  float sum = 0.f;
  for (int cb0 = 0; cb0 < combos; cb0 += kFinCombos) {
    float4 v[kFinCombos][2], w[kFinCombos][2];
    int n[kFinCombos];                             // rows from this lane's first on
#pragma unroll
    for (int k = 0; k < kFinCombos; ++k) {
      const int h = (cb0 + k) / max(rg, 1), rgi = (cb0 + k) - h * rg;
      const int64_t g =
          ((int64_t)b * a.plan.num_kv_heads + h) * a.plan.rg_max + rgi;
      n[k] = cb0 + k < combos ? min(kRowsPerGroup, sq.rows - rgi * kRowsPerGroup) - 4 * lane : 0;
      const float4* m =
          reinterpret_cast<const float4*>(a.clse + (g * a.plan.max_chunks + c) * kRowsPerGroup);
      const float4* l = reinterpret_cast<const float4*>(a.row_lse + g * kRowsPerGroup);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (n[k] > 128 * q) {
          v[k][q] = __ldcg(m + lane + 32 * q);
          w[k][q] = __ldcg(l + lane + 32 * q);
        }
    }
#pragma unroll
    for (int k = 0; k < kFinCombos; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int left = n[k] - 128 * q;
        if (left > 0) sum += exp2f(v[k][q].x - w[k][q].x);
        if (left > 1) sum += exp2f(v[k][q].y - w[k][q].y);
        if (left > 2) sum += exp2f(v[k][q].z - w[k][q].z);
        if (left > 3) sum += exp2f(v[k][q].w - w[k][q].w);
      }
  }
  sum = warp_sum(sum);
  if (lane == 0) {
    float* dst = a.scores + (int64_t)b * a.plan.max_chunks + c;
    *dst = a.accumulate ? *dst + sum : sum;
  }
}

// Four blocks an SM leave 64 registers: 72 bytes spilled and 100 loaded at
// head_dim 128, 28 and 32 at 64.
template <int D>
__global__ void __launch_bounds__(256, 4) kv4_finish(const __grid_constant__ VerifyKArgs a,
                                                     int n_comb, float out_mult) {
  if ((int)blockIdx.x >= n_comb) chunk_score(a, blockIdx.x - n_comb);
  else if (a.out_f32) merge_row<D, false>(a, blockIdx.x, out_mult);
  else merge_row<D, true>(a, blockIdx.x, out_mult);
}

}  // namespace kv4tc

template <int D>
static cudaError_t launch_tc(const Kv4KArgs& k, const VerifyLayout& L, cudaStream_t stream) {
  const size_t smem = kv4tc::Cfg<D>::smem;
  cudaError_t e = allow_smem(kv4tc::kv4_split_tc<D>, smem);
  if (e != cudaSuccess) return e;
  const VerifyKArgs& v = k.v;
  // The plan makes at most one item per SM, two in its two-wave form, or one
  // per row group.  No blocks beyond that: one without work still takes an
  // SM's turn, behind the last items when those end together.
  const int64_t groups = (int64_t)v.plan.batch * v.plan.num_kv_heads * v.plan.rg_max;
  const int64_t blocks = std::max<int64_t>(groups, std::max(L.target_ctas, L.wave_ctas));
  e = launch_dependent(kv4tc::kv4_split_tc<D>, dim3((unsigned)blocks), dim3(kv4tc::kThreads),
                       smem, stream, k);
  if (e != cudaSuccess) return e;
  const int64_t n_comb = ((int64_t)v.plan.n_nodes * v.num_q_heads + 7) / 8;
  const int64_t n_fin = v.scores ? (int64_t)v.plan.batch * ((v.plan.max_chunks + 7) / 8) : 0;
  return launch_dependent(kv4tc::kv4_finish<D>, dim3((unsigned)(n_comb + n_fin)), dim3(256), 0,
                          stream, v, (int)n_comb, k.out_mult);
}

// The whole call for trees.
cudaError_t launch_kv4_tc(const Kv4KArgs& k, int head_dim, const VerifyLayout& L,
                          cudaStream_t stream) {
  return head_dim == 128 ? launch_tc<128>(k, L, stream) : launch_tc<64>(k, L, stream);
}

}  // namespace ds
