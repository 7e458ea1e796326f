// Split pass of ds_kv4_verify_attn for few query rows per kv head: decoding
// and small trees.
//
// With few rows the pass is a stream of K and V, 72 bytes a key and head, and
// a tcgen05 tile of 128 rows would convert every tile through shared memory
// for products that are nearly all padding.  Here each warp works alone on
// blocks of 32 keys, from its own ring of asynchronous copies, with
// m16n8k16 products whose 16-row operand is the cache and whose 8-column
// operand the queries, so that codes go from shared memory to registers to
// the product:
//
//   S^T[16 keys, 8 rows] += K[16 keys, 16 channels] Q^T[16 channels, 8 rows]
//   O^T[16 dims, 8 rows] += V^T[16 dims, 16 keys]  P^T[16 keys, 8 rows]
//
// One token over 128K (32 query heads on 8 of the cache, 151 MB) takes 43.8
// us, 3.4 TB/s of the 6.70 a copy reaches.  An earlier form of 48 took 39
// without the products and 44 without the loads: conversions and products
// (issue slots 58 % busy) and the stream overlap, and some 12 us go into the
// start, the merge, the join and the salience.  A ragged batch of eight (4K to
// 128K, no salience) takes 84 us, 4.7 TB/s; one token over 512 keys, with 4
// heads of 64 on 2, 9.0 us.
//
// Which channels make up a step of the first product, and which dims a tile
// of the second, is free as long as both operands agree.  Lane 4g + t takes
// the channels from 32t on of its two keys (two scale groups), and dims 16g
// .. 16g + 15 of its four keys (one scale group of each), both as whole
// vectors (16t and 8g at head_dim 64).  For the second product codes of two
// keys are interleaved nibble by nibble before the conversion, which then
// yields the pairs over keys that the operand holds.  P^T is S^T's fragment
// transposed (movmatrix).
//
// Of 16 keys, fragment row i holds key i ^ ((i >> 1) & 1), and keys 4-7 and
// 12-15 have the halves of their 16-byte pieces exchanged: then eight lanes
// of a 16-byte read and 16 lanes of an 8-byte read touch every bank once.
//
// Work: every (sequence, kv head, group of 8 NT query rows) is a segment of
// 32-key units, and the units of all segments, in order, are dealt to the
// blocks in equal contiguous ranges, each segment behind a lead-in that
// stands for what its start and end cost, so that a ragged batch balances.
// A block works its range segment by segment: the units of one go to
// its warps in turn, whose outputs are merged in shared memory.  When a
// segment was cut between blocks, the last of them to finish merges the
// pieces into the output (with few rows that costs less than a launch); only
// the salience takes a second kernel.  Each warp works the plan out by
// itself, from the lengths, in one pass over the batch, and again for every
// piece: with a thousand sequences that is what takes the time (8 heads over
// 1K keys each: 64 sequences 55 us, 256 264, 1,024 2,450).
//
// Chunk masses are kept per 32 keys or less ("subchunks"), so that a unit
// never shares one: [kv head][sequence's rows x subchunks][subchunk][row],
// rows numbered through the batch.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "dev_common.cuh"
#include "internal.h"
#include "kv4_common.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"
#include "verify_common.cuh"
#include "verify_softmax.cuh"

namespace ds {
namespace kv4few {

constexpr int kStages = 3;      // blocks of 32 keys in a warp's ring
constexpr int kBlock = 32;                       // keys of a block, and of a unit
// A piece's start (plan, page ids, first copies) and end (merge) take about
// as long as 40 units do in a block of 16 warps: 5 us against 0.13 us a unit
// (heads of 128; the other forms were not measured for it and share it)
constexpr int kPieceUnits = 40;

template <int D, int NT>
struct Cfg {
  static constexpr int W = NT == 1 ? 16 : 12;       // warps of a block
  static constexpr int R = 8 * NT;                  // query rows of one pass
  static constexpr int kTensor = kBlock * (D / 2 + D / 16);   // bytes of a block's K or V
  static constexpr int kRing = kStages * 2 * kTensor;     // bytes of a warp's ring
  // With two tiles of queries the fragments of both do not fit beside their
  // outputs in the registers of 12 warps: the queries stay in shared memory,
  // in fragment order, and the scores are not formed a block ahead.
  static constexpr bool kQShared = NT > 1;
  static constexpr size_t smem = (size_t)W * kRing + (kQShared ? R * D * 2 : 0);
  static_assert(kStages == 3, "a block in use, the next one's scores, one on its way");
  static constexpr int kOutStride = D + 8;          // floats of a row of a warp's output
  static_assert(R * kOutStride * 4 <= kRing, "a warp's output must fit in its ring");
};

// One piece of a segment: units [u0, u1).
struct Piece {
  int L, T, node0, rows;         // the sequence's
  int b, kvh, rgi;               // sequence, kv head, row group
  int u0, u1;
  int slot;                      // of this piece's partial output
  int first_slot, n_slots;       // of the segment's pieces
  int seg;                       // number of the segment in the batch
  int next;                      // unit after the piece; -1 when the block's range ends
};

struct Ctrl {
  Piece piece[16];               // [warp]
  int32_t parents[DS_MAX_TREE_NODES];
  uint64_t anc[DS_MAX_TREE_NODES];
  float m[16][16], l[16][16];    // [warp][row]
  Piece cut[2];                  // pieces of cut segments: at most the range's two ends
  int n_cut, last[2];
};

DS_DEV void cp16(uint32_t dst, const void* src, uint32_t bytes) {   // bytes 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes)
               : "memory");
}
DS_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DS_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

DS_DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DS_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
DS_DEV uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
DS_DEV uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
DS_DEV uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a));
  return r;
}
DS_DEV uint32_t lds_u16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
DS_DEV uint32_t lds_u8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

// The piece of this block's range that begins at unit x (x < 0: its first);
// false when the block has none.  One warp, which writes *pc: the plan is
// worked out again for every piece, so that nothing of it stays in registers.
// Offsets that go up and down can describe more nodes than there are, and
// more segments than there are counters: then there is no work (*overlap).
template <int R, int W>
__device__ __noinline__ bool find_piece(const PlanArgs& pa, int x, Piece* pc,
                                        int32_t* overlap) {
  const int lane = threadIdx.x & 31;
  // units and segments of sequence b (lane-parallel)
  struct Seq { int L, T, node0, rows, nu, segs; };
  auto seq_of = [&](int b, bool report) {
    Seq s = {0, 0, 0, 0, 0, 0};
    if (b < pa.batch) {
      const SeqPlan q = seq_sizes(pa, b, report);
      s.L = q.L; s.T = q.T; s.node0 = q.node0; s.rows = q.rows;
      s.nu = (q.L + q.T + kBlock - 1) / kBlock;
      s.segs = pa.num_kv_heads * ((q.rows + R - 1) / R);
    }
    return s;
  };
  const bool report = blockIdx.x == 0 && x < 0;
  int U = 0, S = 0, nodes = 0;
  unsigned most = 0, least = ~0u;                 // units of a segment
  const Seq first = seq_of(lane, report);
  for (int b0 = 0; b0 < pa.batch; b0 += 32) {
    const Seq s = b0 == 0 ? first : seq_of(b0 + lane, report);
    U += __reduce_add_sync(0xffffffffu, s.segs * s.nu);
    S += __reduce_add_sync(0xffffffffu, s.segs);
    nodes += __reduce_add_sync(0xffffffffu, s.T);
    most = max(most, __reduce_max_sync(0xffffffffu, s.segs ? (unsigned)s.nu : 0u));
    least = min(least, __reduce_min_sync(0xffffffffu, s.segs ? (unsigned)s.nu : ~0u));
  }
  if (report && lane == 0) *overlap = nodes > pa.n_nodes;
  if (nodes > pa.n_nodes) return false;
  // at most one block per segment or, for long segments, per 2 W units
  const int N = min((int)gridDim.x, max(S, (U + 2 * W - 1) / (2 * W)));
  const int i = blockIdx.x;
  // Segments of one length: cut evenly, a piece a block, down to a unit a
  // warp (but not for the second unit: the join costs as much), unless that
  // leaves more blocks idle than the cuts of the general way cost.  One token
  // over 1K, 2K, 8K: 12, 12 and 14 us; the general way had 20, 18 and 18.
  const int each =
      S > 0 ? min((int)gridDim.x / S, (int)most <= 2 * W ? 1 : ((int)most + W - 1) / W) : 0;
  const bool even = each > 0 && most == least &&
                    (int64_t)((most + each - 1) / each) * N <= (int64_t)U + S * kPieceUnits;
  if (even ? i >= S * each : i >= N) return false;
  if (even) {
    int sbase = 0;
    const int seg = i / each, j = i - seg * each;
    for (int b0 = 0; b0 < pa.batch; b0 += 32) {
      const Seq s = b0 == 0 ? first : seq_of(b0 + lane, false);
      int ps = s.segs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, ps, o);
        if (lane >= o) ps += v;
      }
      const int all_s = __shfl_sync(0xffffffffu, ps, 31);
      ps += sbase - s.segs;
      if (seg >= ps && seg < ps + s.segs) {       // one lane
        const int rg = (s.rows + R - 1) / R;
        pc->L = s.L; pc->T = s.T; pc->node0 = s.node0; pc->rows = s.rows;
        pc->b = b0 + lane;
        pc->kvh = (seg - ps) / rg;
        pc->rgi = seg - ps - pc->kvh * rg;
        pc->u0 = (int)((int64_t)s.nu * j / each);
        pc->u1 = (int)((int64_t)s.nu * (j + 1) / each);
        pc->seg = seg;
        pc->slot = i;
        pc->first_slot = seg * each;
        pc->n_slots = each;
        pc->next = -1;
      }
      sbase += all_s;
    }
    __syncwarp();
    return true;
  }
  U += S * kPieceUnits;                           // the axis: units behind their lead-ins
  const int q = U / N, rem = U - q * N;           // the first rem blocks: q + 1 of it
  const int lo = i * q + min(i, rem), hi = lo + q + (i < rem ? 1 : 0);
  auto block_of = [&](int u) {
    return u < rem * (q + 1) ? u / (q + 1) : rem + (u - rem * (q + 1)) / q;
  };
  if (x < 0) x = lo;
  int ubase = 0, sbase = 0;                       // axis and segments before the 32
  for (int b0 = 0; b0 < pa.batch; b0 += 32) {
    const Seq s = b0 == 0 ? first : seq_of(b0 + lane, false);
    const int len = s.nu + kPieceUnits;           // of a segment
    int pu = s.segs * len, ps = s.segs;           // inclusive prefixes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, pu, o), v = __shfl_up_sync(0xffffffffu, ps, o);
      if (lane >= o) { pu += u; ps += v; }
    }
    const int all_u = __shfl_sync(0xffffffffu, pu, 31), all_s = __shfl_sync(0xffffffffu, ps, 31);
    pu += ubase - s.segs * len;                   // where the sequence begins
    ps += sbase - s.segs;
    if (x < ubase + all_u) {
      if (s.segs > 0 && pu <= x && x < pu + s.segs * len) {             // one lane
        const int rg = (s.rows + R - 1) / R;
        const int seg = (x - pu) / len;
        const int u = pu + seg * len + kPieceUnits;                     // its first unit
        pc->L = s.L; pc->T = s.T; pc->node0 = s.node0; pc->rows = s.rows;
        pc->b = b0 + lane;
        pc->kvh = seg / rg;
        pc->rgi = seg - pc->kvh * rg;
        pc->u0 = max(x - u, 0);
        pc->u1 = min(s.nu, hi - u);               // <= u0: only part of the lead-in
        pc->seg = ps + seg;
        // numbered by block and segment, which never both stand still, the
        // pieces have slots of their own, a segment's in a row
        pc->slot = i + ps + seg;
        const int f = block_of(u);
        pc->first_slot = f + ps + seg;
        pc->n_slots = block_of(u + s.nu - 1) - f + 1;
        pc->next = u + s.nu < hi ? u + s.nu : -1;
      }
      __syncwarp();
      return true;
    }
    ubase += all_u;
    sbase += all_s;
  }
  return false;
}

template <int D, int NT>
__device__ __forceinline__ void work_piece(const Kv4KArgs& ka, const Piece& pc, Ctrl& ctrl,
                                           unsigned char* smem, const int warp) {
  using namespace ptx;
  using C_ = Cfg<D, NT>;
  constexpr int W = C_::W, R = C_::R;
  constexpr int NS = D / 16;              // product steps of Q K^T, dim tiles of O
  constexpr int CB = D / 2, SB = D / 16;  // bytes of a key's codes and scales
  const VerifyKArgs& a = ka.v;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = a.plan.group, L = pc.L, T = pc.T, P = a.plan.page_size;
  const int rows = min(R, pc.rows - pc.rgi * R);                // of this segment
  const int C = a.scores ? min(kBlock, a.plan.chunk_size) : 0;      // keys of a subchunk
  const int64_t row0 = (int64_t)pc.node0 * G;                   // first row of the sequence
  const int64_t n_rows = (int64_t)a.plan.n_nodes * G;
  const int64_t n_sub = C ? (int64_t)a.plan.max_chunks * (a.plan.chunk_size / C) : 0;
  float* const mass = a.clse + ((int64_t)pc.kvh * n_rows + row0) * n_sub + pc.rgi * R;
  float* const row_lse = a.row_lse + (int64_t)pc.kvh * n_rows + row0 + pc.rgi * R;
  const int32_t* ptab = a.page_table + (int64_t)pc.b * a.plan.max_pages;

  // this warp's units u0 + warp, + W, ... of the piece, a block each; nh is
  // their number of 16-key halves that hold keys of the sequence
  const int nh_piece = (min(pc.u1 * kBlock, L + T) - pc.u0 * kBlock + 15) / 16;
  const int n_units = pc.u1 - pc.u0;
  const int nblk = n_units > warp ? (n_units - warp - 1) / W + 1 : 0;
  const int nh = nblk > 0 ? (nblk - 1) * 2 + min(2, nh_piece - (warp + (nblk - 1) * W) * 2) : 0;
  const int first_key = (pc.u0 + warp) * kBlock;
  const int pshift = __ffs(P) - 1;
  // first key of half i
  auto key_of = [&](int i) { return first_key + (i >> 1) * (W * kBlock) + (i & 1) * 16; };
  // page ids of this warp's halves, 32 at a time, the next 32 on their way
  auto ids_of = [&](int i) { return i < nh ? __ldg(ptab + (key_of(i) >> pshift)) : 0; };
  int ids = ids_of(lane), next_ids = ids_of(32 + lane);
  // output row of row r of this segment
  auto out_row = [&](int r) {
    const int grow = pc.rgi * R + r;
    return ((int64_t)pc.node0 + grow / G) * a.num_q_heads + pc.kvh * G + grow % G;
  };
  // queries: column g of tile n is row 8 n + g; the fragments of step s are
  // channels t D/4 + 4 s .. + 3
  constexpr bool QS = C_::kQShared;
  constexpr int QT = QS ? 1 : NT;                   // tiles kept in registers
  uint4 qx[QT][D / 32];
  if constexpr (!QS) {
#pragma unroll
    for (int n = 0; n < QT; ++n) {
      const int r = 8 * n + g;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + out_row(r) * D + t * (D / 4));
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
        qx[n][w] = r < rows ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
    }
  }
  // ancestor masks, when the piece holds tree keys; a tree of one node has
  // only itself
  const bool need_anc = pc.u1 * kBlock > L;
  uint64_t anc[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) anc[n][0] = anc[n][1] = 1ull;

  const uint32_t ring = smem_addr(smem) + warp * C_::kRing;
  const uint32_t blk = DS_KV4_BLOCK_BYTES(P, D);
  const uint32_t page_bytes = a.plan.num_kv_heads * blk;
  const uint8_t* const k_head = ka.k4 + (int64_t)pc.kvh * blk;
  const uint8_t* const v_head = ka.v4 + (int64_t)pc.kvh * blk;
  const float c2 = a.scale_log2;
  // pieces this lane copies: one or two of the codes of each tensor and
  // half, and one of the scales (one of two lanes at head_dim 64)
  constexpr int PPK = CB / 16;                      // 16-byte pieces of a key
  constexpr int SP = SB;                            // pieces of 16 keys' scales
  const int pk = lane / PPK;                        // key of the first piece
  const uint32_t dcode =
      ring + pk * CB + ((D == 128 ? lane % PPK ^ (((pk >> 2) & 1) << 1) : lane % PPK) << 4);
  const int s_t = lane / SP & 1, s_h = lane / (2 * SP);        // tensor and half
  const uint32_t dscale =
      ring + s_t * C_::kTensor + kBlock * CB + s_h * 16 * SB + (lane % SP) * 16;
  const uint8_t* const k_lane = k_head + lane * 16;
  const uint8_t* const v_lane = v_head + lane * 16;
  const uint8_t* const s_lane =
      (s_t ? v_head : k_head) + (P << (D == 128 ? 6 : 5)) + (lane % SP) * 16;
  // bad page ids among the 32 at hand: page 0 stands in, and copies nothing
  auto check = [&]() {
    const bool bad = (uint32_t)ids >= (uint32_t)a.num_pages;
    if (bad) {
      flag(a.plan.status, DS_DEV_BAD_PAGE);
      ids = 0;
    }
    return __ballot_sync(0xffffffffu, bad);
  };
  uint32_t bad_ids = check();
  uint32_t slot_in = 0;                             // ring offset of the next block
  auto issue = [&](int i) {
    if (i < nblk) {
      if (i > 0 && (i & 15) == 0) {
        ids = next_ids;
        next_ids = ids_of(2 * i + 32 + lane);
        bad_ids = check();
      }
      const int off = key_of(2 * i) & (P - 1);
      const int off1 = (off + 16) & (P - 1);
      const int j = (2 * i) & 31;
      const uint32_t pg0 = __shfl_sync(0xffffffffu, ids, j);
      const uint32_t pg1 = __shfl_sync(0xffffffffu, ids, j + 1);
      const uint32_t n0 = (bad_ids >> j) & 1u ? 0u : 16u, n1 = (bad_ids >> j) & 2u ? 0u : 16u;
      const uint32_t d = dcode + slot_in;
      const uint8_t* kp = k_lane + ((uint64_t)pg0 * page_bytes + off * CB);
      const uint8_t* vp = v_lane + ((uint64_t)pg0 * page_bytes + off * CB);
#pragma unroll
      for (int c = 0; c < PPK / 2; ++c) {           // keys pk and, at 128, pk + 8
        cp16(d + c * 512, kp + c * 512, n0);
        cp16(d + C_::kTensor + c * 512, vp + c * 512, n0);
      }
      const bool in1 = 2 * i + 1 < nh;   // past the end: whatever is there is masked
      if (in1) {
        kp = k_lane + ((uint64_t)pg1 * page_bytes + off1 * CB);
        vp = v_lane + ((uint64_t)pg1 * page_bytes + off1 * CB);
#pragma unroll
        for (int c = 0; c < PPK / 2; ++c) {
          cp16(d + 16 * CB + c * 512, kp + c * 512, n1);
          cp16(d + 16 * CB + C_::kTensor + c * 512, vp + c * 512, n1);
        }
      }
      if (lane < (in1 ? 4 * SP : 2 * SP))
        cp16(dscale + slot_in,
             s_lane + ((uint64_t)(s_h ? pg1 : pg0) * page_bytes + (s_h ? off1 : off) * SB),
             s_h ? n1 : n0);
    }
    cp_commit();
    slot_in = slot_in == (kStages - 1) * 2 * C_::kTensor ? 0u : slot_in + 2 * C_::kTensor;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  if (need_anc && warp == 0) {
    if (T > 1)
      tc::tree_ancestors(a.parents + pc.node0, T, ctrl.parents, ctrl.anc, a.plan.status);
    else if (lane == 0 && __ldg(a.parents + pc.node0) != -1)
      flag(a.plan.status, DS_DEV_BAD_TREE);
  }
  uint32_t q[QT][NS][2];
  const uint32_t q_smem = smem_addr(smem) + W * C_::kRing + lane * 8;
  if constexpr (QS) {
    for (int x = threadIdx.x; x < NT * NS * 32; x += 32 * W) {      // (tile, step, lane)
      const int r = 8 * (x / (NS * 32)) + ((x & 31) >> 2);
      const int c = (x & 3) * (D / 4) + (x >> 5) % NS * 4;
      uint2 v = make_uint2(0, 0);
      if (r < rows) v = __ldg(reinterpret_cast<const uint2*>(a.q + out_row(r) * D + c));
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(
                       smem_addr(smem) + W * C_::kRing + x * 8),
                   "r"(bf16x2_to_f16x2(v.x)), "r"(bf16x2_to_f16x2(v.y))
                   : "memory");
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int n = 0; n < QT; ++n)
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {            // 8 channels: steps 2w, 2w + 1
        q[n][2 * w][0] = bf16x2_to_f16x2(qx[n][w].x);
        q[n][2 * w][1] = bf16x2_to_f16x2(qx[n][w].y);
        q[n][2 * w + 1][0] = bf16x2_to_f16x2(qx[n][w].z);
        q[n][2 * w + 1][1] = bf16x2_to_f16x2(qx[n][w].w);
      }
  }
  if (need_anc && T > 1) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        anc[n][e] = r < rows ? ctrl.anc[(pc.rgi * R + r) / G] : 0ull;
      }
  }
  float o[NT][NS][4];
  float m[NT][2], mb[NT][2], l[NT][2], cs[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[n][e] = -CUDART_INF_F;
      l[n][e] = cs[n][e] = mb[n][e] = 0.f;
    }
  }

  // fragment row g of a block, and the lane's four keys of the second product
  const int krow = g ^ ((g >> 1) & 1);
  const uint32_t kcode =
      ring + krow * CB + (D == 128 ? (t ^ (((krow >> 2) & 1) << 1)) << 4 : t * 8);
  const uint32_t kscale = ring + kBlock * CB + krow * SB + (D == 128 ? 2 * t : t);
  uint32_t vcode[2], vscale[2];                   // keys of fragment rows 2t and 2t + 1
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int key = 2 * t + (e ^ (t & 1));
    vcode[e] = ring + C_::kTensor + key * CB +
               (D == 128 ? (((g >> 1) ^ (((key >> 2) & 1) << 1)) << 4) + (g & 1) * 8 : g * 4);
    vscale[e] = ring + C_::kTensor + kBlock * CB + key * SB + (D == 128 ? g : g >> 1);
  }
  const int cshift = C ? __ffs(C) - 1 : 0;
  // Scores of the block at ring offset `at`: s[n][hf][2h + e] is key 16 hf +
  // 8h + krow, row 8n + 2t + e.
  auto scores = [&](uint32_t at, float (&s)[NT][2][4]) {
    uint32_t w[4][D / 32], sc[4][2];                // of the lane's four keys 8 x + krow
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (D == 128) {
        const uint4 y = lds128(kcode + at + x * 8 * CB);
        w[x][0] = y.x; w[x][1] = y.y; w[x][2] = y.z; w[x][3] = y.w;
        const uint32_t s2 = kv4_scales_f16(lds_u16(kscale + at + x * 8 * SB));
        sc[x][0] = __byte_perm(s2, s2, 0x1010);
        sc[x][1] = __byte_perm(s2, s2, 0x3232);
      } else {
        const uint2 y = lds64(kcode + at + x * 8 * CB);
        w[x][0] = y.x; w[x][1] = y.y;
        const uint32_t b = lds_u8(kscale + at + x * 8 * SB);
        sc[x][0] = sc[x][1] = kv4_scales_f16(b | b << 8);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 8; ++x) s[n][x >> 2][x & 3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {              // 8 channels: steps 2k, 2k + 1
      uint2 qs[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (QS) qs[n][e] = lds64(q_smem + (n * NS + 2 * k + e) * 256);
          else qs[n][e] = make_uint2(q[n][2 * k + e][0], q[n][2 * k + e][1]);
        }
      const int si = D == 128 ? k >> 1 : 0;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t v0[4], v1[4];
        kv4_codes_f16(w[2 * hf][k], v0);
        kv4_codes_f16(w[2 * hf + 1][k], v1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v0[e] = hmul2(v0[e], sc[2 * hf][si]);
          v1[e] = hmul2(v1[e], sc[2 * hf + 1][si]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t fa[4] = {v0[2 * e], v1[2 * e], v0[2 * e + 1], v1[2 * e + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(s[n][hf], fa, qs[n][e].x, qs[n][e].y);
        }
      }
    }
  };
  // Software pipeline (queries in registers): the scores of block i + 1 are
  // formed beside the softmax and the second product of block i, which depend
  // on nothing of it, while block i + 2 is on its way.
  constexpr bool AHEAD = !QS;
  float s[NT][2][4];
  if constexpr (AHEAD) {
    cp_wait<kStages - 2>();
    __syncwarp();
    scores(0, s);
  }
  uint32_t st = 0;
#pragma unroll 1
  for (int i = 0; i < nblk; ++i) {
    if constexpr (!AHEAD) cp_wait<kStages - 2>();
    __syncwarp();                  // all lanes are done with block i - 1
    issue(i + kStages - 1);
    const uint32_t st_next = st == (kStages - 1) * 2 * C_::kTensor ? 0u : st + 2 * C_::kTensor;
    float s_next[NT][2][4];
    if constexpr (AHEAD) {
      cp_wait<kStages - 2>();
      __syncwarp();
      scores(st_next, s_next);     // after the last block: not used
    } else {
      scores(st, s);
    }
    const int key0 = key_of(2 * i);
    // ---------------------------------------------------------- softmax
    const bool tail = key0 + kBlock > L;
    if (tail) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int d = key0 + 8 * (x >> 1) + krow - L;        // tree slot when >= 0
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (d >= 0 && !(d < T && ((anc[n][x & 1] >> d) & 1)))
            s[n][x >> 2][x & 3] = -CUDART_INF_F;
      }
    }
    // lazy maximum, 2^7 above the reference so that P fills f16's range
    bool need = false;
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[n][e] = fmaf(fmax3(fmaxf(s[n][0][e], s[n][0][2 + e]), s[n][1][e], s[n][1][2 + e]),
                        c2, -7.f);
        need |= mx[n][e] > m[n][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[n][e];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
          x = fmaxf(m[n][e], x);
          const float al = x == -CUDART_INF_F ? 1.f : ex2(m[n][e] - x);
          m[n][e] = x;
          mb[n][e] = x == -CUDART_INF_F ? 0.f : -x;      // a row that has seen nothing
          l[n][e] *= al;
          cs[n][e] *= al;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            o[n][j][e] *= al;
            o[n][j][e + 2] *= al;
          }
        }
    }
    uint32_t pb[NT][2][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum[2][2];                            // [half][e]
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float pr[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) pr[x] = ex2(fmaf(s[n][hf][x], c2, mb[n][x & 1]));
        sum[hf][0] = pr[0] + pr[2];
        sum[hf][1] = pr[1] + pr[3];
        pb[n][hf][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
        pb[n][hf][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
#pragma unroll
        for (int e = 0; e < 2; ++e) l[n][e] += sum[hf][e];
        if (C) {
          if (tail) {                             // context keys only
            const bool c0 = key0 + 16 * hf + krow < L, c1 = key0 + 16 * hf + 8 + krow < L;
            sum[hf][0] = (c0 ? pr[0] : 0.f) + (c1 ? pr[2] : 0.f);
            sum[hf][1] = (c0 ? pr[1] : 0.f) + (c1 ? pr[3] : 0.f);
          }
        }
      }
      // log2 of a chunk's mass at a half that ends the chunk or the context
      if (C) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int k0 = key0 + 16 * hf;
#pragma unroll
          for (int e = 0; e < 2; ++e) cs[n][e] += sum[hf][e];
          if (k0 < L && (((k0 + 16) & (C - 1)) == 0 || k0 + 16 >= L)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = cs[n][e];
              cs[n][e] = 0.f;
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
              const int r = 8 * n + 2 * t + e;
              if (g == 0 && r < rows)
                mass[(int64_t)(k0 >> cshift) * pc.rows + r] =
                    x > 0.f ? m[n][e] + __log2f(x) : -CUDART_INF_F;
            }
          }
        }
      }
    }
    // -------------------------------------------------------------- P V
    // fragment rows 2t + e and 8 + 2t + e are keys 2t + (e ^ (t & 1))
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      constexpr int VW = D / 64;                  // words of 8 dims of a key
      uint32_t w[4][VW], b[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int k8 = 2 * hf + (x >> 1);
        if constexpr (D == 128) {
          const uint2 y = lds64(vcode[x & 1] + st + k8 * 8 * CB);
          w[x][0] = y.x;
          w[x][VW - 1] = y.y;
        } else {
          w[x][0] = lds32(vcode[x & 1] + st + k8 * 8 * CB);
        }
        b[x] = lds_u8(vscale[x & 1] + st + k8 * 8 * SB);
      }
      const uint32_t s01 = kv4_scales_f16(b[0] | b[1] << 8);
      const uint32_t s23 = kv4_scales_f16(b[2] | b[3] << 8);
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        constexpr uint32_t M = 0x0f0f0f0fu;
        uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, pairs over keys
        kv4_codes_f16((w[0][k] & M) | ((w[1][k] << 4) & ~M), e01);
        kv4_codes_f16(((w[0][k] >> 4) & M) | (w[1][k] & ~M), o01);
        kv4_codes_f16((w[2][k] & M) | ((w[3][k] << 4) & ~M), e23);
        kv4_codes_f16(((w[2][k] >> 4) & M) | (w[3][k] & ~M), o23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t fa[4] = {hmul2(e01[j], s01), hmul2(o01[j], s01), hmul2(e23[j], s23),
                                  hmul2(o23[j], s23)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(o[n][4 * k + j], fa, pb[n][hf][0], pb[n][hf][1]);
        }
      }
    }
    st = st_next;
    if constexpr (AHEAD) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 8; ++x) s[n][x >> 2][x & 3] = s_next[n][x >> 2][x & 3];
    }
  }
  cp_wait<0>();
  __syncwarp();

  // --------------------------------------------- merge of the block's warps
  // A warp's output in its ring: rows of D + 8 floats, dims 2j and 2j + 1 of
  // lane group g at 16 j + 2 g, so that a store's 32 lanes touch all banks.
  constexpr int ST = C_::kOutStride;
  float* ow = reinterpret_cast<float*>(smem + warp * C_::kRing);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      float x = l[n][e];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
      if (g == 0) {
        ctrl.m[warp][r] = m[n][e];
        ctrl.l[warp][r] = x;
      }
      // tile j: dims g D/8 + 2j (elements 0, 1) and the next (2, 3)
#pragma unroll
      for (int j = 0; j < NS; ++j)
        *reinterpret_cast<float2*>(ow + r * ST + 16 * j + 2 * g) =
            make_float2(o[n][j][e], o[n][j][e + 2]);
    }
  __syncthreads();
  // a warp per row: the warps' weights (in place of their maxima) and the
  // row's log2-sum-exp
  const int used = min(W, n_units);                 // warps that had a unit
  for (int r = warp; r < rows; r += W) {
    const float mw = lane < used ? ctrl.m[lane][r] : -CUDART_INF_F;
    const float lw = lane < used ? ctrl.l[lane][r] : 0.f;
    const float mm = warp_max(mw);
    const float f = ex2(mw - (mm == -CUDART_INF_F ? 0.f : mm));
    const float sum = warp_sum(f * lw);
    if (lane < used) ctrl.m[lane][r] = f * (sum > 0.f ? ka.out_mult / sum : 0.f);
    if (lane == 0) {
      const float lse = sum > 0.f ? mm + __log2f(sum) : -CUDART_INF_F;
      if (pc.n_slots == 1) row_lse[r] = lse;
      else a.lse_part[(int64_t)pc.slot * R + r] = lse;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * (D / 2); x += 32 * W) {
    const int r = x / (D / 2), c = x % (D / 2);     // columns 2c and 2c + 1
    const float* src = reinterpret_cast<const float*>(smem) + r * ST +
                       c % (D / 16) * 16 + c / (D / 16) * 2;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int w = 0; w < used; ++w) {
      const float f = ctrl.m[w][r];
      const float2 v = *reinterpret_cast<const float2*>(src + w * (C_::kRing / 4));
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
    }
    const bool whole = pc.n_slots == 1;
    const int64_t at = (whole ? out_row(r) : (int64_t)pc.slot * R + r) * D + 2 * c;
    if (!whole)
      *reinterpret_cast<float2*>(a.o_part + at) = acc;
    else if (a.out_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = acc;
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
          pack_bf16x2(acc.x, acc.y);
  }
  if (pc.n_slots > 1 && threadIdx.x == 0) ctrl.cut[ctrl.n_cut++] = pc;
  __syncthreads();                 // the ring and ctrl are the next piece's
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * Cfg<D, NT>::W, 1)
kv4_split_few(const __grid_constant__ Kv4KArgs ka) {
  constexpr int W = Cfg<D, NT>::W, R = Cfg<D, NT>::R;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Ctrl ctrl;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // known uniform
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0) ctrl.n_cut = 0;
  Piece& pc = ctrl.piece[warp];
  // the row groups' table is the tree pass's: its first word tells the
  // salience's launch that there is nothing to sum
  int32_t* const overlap = reinterpret_cast<int32_t*>(ka.v.gdesc);
  bool more = find_piece<R, W>(ka.v.plan, -1, &pc, overlap), worked = false;
  while (more) {                   // the same for every warp of the block
    if (pc.u1 > pc.u0) {
      work_piece<D, NT>(ka, pc, ctrl, smem, warp);
      worked = true;
    }
    const int next = pc.next;
    __syncwarp();
    more = next >= 0 && find_piece<R, W>(ka.v.plan, next, &pc, overlap);
  }
  // Only the barriers of a piece order n_cut's first value before its read by
  // the other warps: a block without a piece leaves here, in every warp.
  if (!worked) return;
  // The last piece of a cut segment to finish merges them.
  const int n_cut = ctrl.n_cut;
  if (n_cut == 0) return;
  const VerifyKArgs& a = ka.v;
  __threadfence();                 // this block's pieces before its arrivals
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 0; k < n_cut; ++k) {
      const int seg = ctrl.cut[k].seg;
      ctrl.last[k] = atomicAdd(a.counters + seg, 1u) + 1 == (uint32_t)ctrl.cut[k].n_slots;
      if (ctrl.last[k]) a.counters[seg] = 0u;
    }
    __threadfence();               // the others' pieces before reading them
  }
  __syncthreads();
  // rows of the segments to merge, one after the other
  auto rows_of = [&](int k) {
    return k < n_cut && ctrl.last[k] ? min(R, ctrl.cut[k].rows - ctrl.cut[k].rgi * R) : 0;
  };
  const int n0 = rows_of(0), n1 = rows_of(1);
  if (n0 + n1 == 0) return;
  // a thread per two columns of a row; the pieces' log2-sum-exps and outputs
  // come in one round trip, NB at a time
  const int G = a.plan.group;
  constexpr int NB = 20;
  for (int x = threadIdx.x; x < (n0 + n1) * (D / 2); x += 32 * W) {
    const int y = x / (D / 2), col = x % (D / 2) * 2;
    const Piece& c = ctrl.cut[y >= n0];
    const int r = y >= n0 ? y - n0 : y, grow = c.rgi * R + r, ns = c.n_slots;
    const float* lp = a.lse_part + (int64_t)c.first_slot * R + r;
    const int64_t o = ((int64_t)c.first_slot * R + r) * D + col;
    float mm = -CUDART_INF_F, sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
    for (int k0 = 0; k0 < ns; k0 += NB) {
      float w[NB];
      float2 v[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        w[k] = -CUDART_INF_F;
        v[k] = make_float2(0.f, 0.f);
        if (k0 + k >= ns) continue;
        const int64_t at = o + (int64_t)(k0 + k) * R * D;
        w[k] = __ldcg(lp + (int64_t)(k0 + k) * R);
        v[k] = __ldcg(reinterpret_cast<const float2*>(a.o_part + at));
      }
      float nm = mm;
#pragma unroll
      for (int k = 0; k < NB; ++k) nm = fmaxf(nm, w[k]);
      const float mb = nm == -CUDART_INF_F ? 0.f : nm, f = ptx::ex2(mm - mb);
      mm = nm;
      sum *= f;
      acc.x *= f;
      acc.y *= f;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float e = ptx::ex2(w[k] - mb);
        sum += e;
        // a piece that saw nothing wrote zeros, or NaN for a query that is
        // not a number; that stays
        acc.x = fmaf(e, v[k].x, acc.x);
        acc.y = fmaf(e, v[k].y, acc.y);
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t row = ((int64_t)c.kvh * a.plan.n_nodes + c.node0) * G + grow;
    if (col == 0) a.row_lse[row] = sum > 0.f ? mm + __log2f(sum) : -CUDART_INF_F;
    const int64_t at =
        (((int64_t)c.node0 + grow / G) * a.num_q_heads + c.kvh * G + grow % G) * D + col;
    if (a.out_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) =
          make_float2(acc.x * inv, acc.y * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
          ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
  }
}

// Chunk scores: the sum over kv heads and rows of 2^(mass - the row's
// log2-sum-exp).  A warp per chunk; a lane has one (subchunk, row) of several
// heads, whose loads are on their way together: the launch is bound by one
// round trip (2 to 4 us behind the split pass).
__global__ void __launch_bounds__(256) kv4_scores_few(const __grid_constant__ VerifyKArgs a) {
  constexpr int NB = 8;
  // sequences and chunks share the grid's long axis: the others end at 65,535
  const int per_b = (a.plan.max_chunks + 7) / 8;
  const int b = blockIdx.x / per_b, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = (blockIdx.x - b * per_b) * 8 + warp;
  // the lengths (and the sums so far) are inputs of the call: the split pass,
  // which this launch follows, has itself waited for whatever wrote them
  const SeqPlan sq = seq_sizes(a.plan, b, false);
  const int sub = min(kBlock, a.plan.chunk_size), per = a.plan.chunk_size / sub;
  const int k0 = c * per, n_k = min(per, (sq.L + sub - 1) / sub - k0);
  const bool work = n_k > 0 && c < a.plan.max_chunks;
  const int per_head = work ? n_k * sq.rows : 0;  // a head's masses, consecutive
  const int span = min(32, max(1, per_head));     // lanes of a head
  const int hp = 32 / span;                       // heads side by side in the warp
  const int hl = per_head < 32 ? lane / span : 0;
  const int e0 = lane - hl * span;
  const int64_t n_rows = (int64_t)a.plan.n_nodes * a.plan.group;
  const int64_t n_sub = (int64_t)a.plan.max_chunks * per;
  const float* const mass = a.clse + (int64_t)sq.node0 * a.plan.group * n_sub +
                            (int64_t)k0 * sq.rows;
  const float* const lse = a.row_lse + (int64_t)sq.node0 * a.plan.group;
  float* const dst = a.scores + (int64_t)b * a.plan.max_chunks + c;
  const float before = work && a.accumulate && lane == 0 ? *dst : 0.f;
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (!work) return;
  const int overlap = __ldcg(reinterpret_cast<const int32_t*>(a.gdesc));
  float sum = 0.f;
  for (int e = hl < hp ? e0 : per_head; e < per_head; e += 32) {
    const int r = e % sq.rows;
    for (int h0 = hl; h0 < a.plan.num_kv_heads; h0 += hp * NB) {
      float m[NB], l[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int h = h0 + k * hp;
        m[k] = -CUDART_INF_F;
        l[k] = 0.f;
        if (h < a.plan.num_kv_heads) {
          m[k] = __ldcg(mass + h * n_rows * n_sub + e);
          l[k] = __ldcg(lse + h * n_rows + r);
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) sum += ptx::ex2(m[k] - l[k]);
    }
  }
  sum = warp_sum(sum);
  if (lane == 0 && !overlap) *dst = before + sum;
}

template <int D, int NT>
static cudaError_t launch(const Kv4KArgs& k, const VerifyLayout& L, cudaStream_t stream) {
  const size_t smem = Cfg<D, NT>::smem;
  cudaError_t e = allow_smem(kv4_split_few<D, NT>, smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv4_split_few<D, NT>, dim3(L.target_ctas), dim3(32 * Cfg<D, NT>::W), smem,
                       stream, k);
  if (e != cudaSuccess || !k.v.scores || k.v.plan.max_chunks == 0) return e;
  const int64_t blocks = (int64_t)k.v.plan.batch * ((k.v.plan.max_chunks + 7) / 8);
  return launch_dependent(kv4_scores_few, dim3((unsigned)blocks), dim3(256), 0, stream, k.v);
}

}  // namespace kv4few

// Up to 8 rows a segment the queries stay in registers beside 16 warps (a
// single call of 2 nodes of 4 rows over 128K: 54 us); above, two tiles of 8
// need the shared memory and leave room for 12 (3 nodes: 68, with 52 bytes a
// thread spilled and 64 loaded at head_dim 128; with 16 warps and
// the queries in registers, spilled, an earlier form of 4 nodes took 99
// instead of 76).
cudaError_t launch_kv4_few(const Kv4KArgs& k, int head_dim, int rows, const VerifyLayout& L,
                           cudaStream_t stream) {
  using kv4few::launch;
  if (rows <= 8)
    return head_dim == 128 ? launch<128, 1>(k, L, stream) : launch<64, 1>(k, L, stream);
  return head_dim == 128 ? launch<128, 2>(k, L, stream) : launch<64, 2>(k, L, stream);
}

}  // namespace ds
