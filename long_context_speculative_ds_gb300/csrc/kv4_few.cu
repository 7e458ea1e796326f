// Split pass of ds_kv4_verify_attn for few query rows per kv head: decoding
// and small trees.
//
// With few rows the pass is a stream of K and V, 72 bytes a key and head, and
// a tcgen05 tile of 128 rows would convert every tile through shared memory
// for products that are nearly all padding.  Here each warp works alone on
// blocks of 16 keys, from its own ring of asynchronous copies, with
// m16n8k16 products whose 16-row operand is the cache and whose 8-column
// operand the queries, so that codes go from shared memory to registers to
// the product:
//
//   S^T[16 keys, 8 rows] += K[16 keys, 16 channels] Q^T[16 channels, 8 rows]
//   O^T[16 dims, 8 rows] += V^T[16 dims, 16 keys]  P^T[16 keys, 8 rows]
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
// A block's 16 keys sit in fragment row i as key i ^ ((i >> 1) & 1), and the
// 16-byte pieces of keys 4-7 and 12-15 with their halves exchanged: then
// eight lanes of a 16-byte read and 16 lanes of an 8-byte read touch every
// bank once.
//
// A work item (the plan of the tree pass: sequence, kv head, row group, range
// of 128-key tiles) is cut into units of 64 keys, dealt to the block's warps
// in turn; the warps' outputs are merged in shared memory.  Rows beyond 8 NT
// make the block go over its keys again.  The last split of a row group to
// finish merges the splits into the output (with few rows that is less than
// a launch); only the salience takes a second kernel.
//
// Chunk masses are kept per 64 keys or less ("subchunks"), so that a unit
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

constexpr int kStages = 4;

template <int D, int NT>
struct Cfg {
  static constexpr int W = NT == 1 ? 16 : 8;        // warps of a block
  static constexpr int R = 8 * NT;                  // query rows of one pass
  static constexpr int kTensor = 16 * (D / 2 + D / 16);   // bytes of 16 keys
  static constexpr int kRing = kStages * 2 * kTensor;     // bytes of a warp's ring
  static constexpr size_t smem = (size_t)W * kRing;
  static_assert(R * D * 4 <= kRing, "a warp's output must fit in its ring");
};

struct Ctrl {
  Plan plan;
  int32_t parents[DS_MAX_TREE_NODES];
  uint64_t anc[DS_MAX_TREE_NODES];
  float m[16][16], l[16][16];    // [warp][row]
  int last;
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

template <int D, int NT>
__global__ void __launch_bounds__(32 * Cfg<D, NT>::W, 1) kv4_split_few(const Kv4KArgs ka) {
  using namespace ptx;
  using C_ = Cfg<D, NT>;
  constexpr int W = C_::W, R = C_::R;
  constexpr int NS = D / 16;              // product steps of Q K^T, dim tiles of O
  constexpr int CB = D / 2, SB = D / 16;  // bytes of a key's codes and scales
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Ctrl ctrl;
  const VerifyKArgs& a = ka.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const bool early_plan = a.accumulate != 0;    // as in the tree pass
  if (early_plan && warp == 0) {
    const Plan p = plan_find(a.plan, -1, blockIdx.x);
    if (lane == 0) ctrl.plan = p;
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (!early_plan && warp == 0) {
    const Plan p = plan_find(a.plan, -1, blockIdx.x);
    if (lane == 0) ctrl.plan = p;
  }
  __syncthreads();
  const Plan p = ctrl.plan;
  if ((int)blockIdx.x >= p.total_items || p.b < 0) return;
  const SeqPlan& sq = p.seq;
  const int G = a.plan.group;
  const int local = blockIdx.x - sq.item_base;
  const int kvh = local / (sq.rg * sq.splits);
  const int rgi = local % (sq.rg * sq.splits) / sq.splits;
  const int split = local % sq.splits;
  const int tb = sq.tiles / sq.splits, rem = sq.tiles % sq.splits;
  const int t0 = split * tb + min(split, rem), t1 = t0 + tb + (split < rem ? 1 : 0);
  const int rows = min(kRowsPerGroup, sq.rows - rgi * kRowsPerGroup);
  const int L = sq.L, T = sq.T, P = a.plan.page_size;
  const int C = a.scores ? min(64, a.plan.chunk_size) : 0;      // keys of a subchunk
  const int64_t row0 = (int64_t)sq.node0 * G;                    // first row of the sequence
  const int64_t n_rows = (int64_t)a.plan.n_nodes * G;
  const int64_t n_sub = C ? (int64_t)a.plan.max_chunks * (a.plan.chunk_size / C) : 0;
  float* const mass = a.clse + ((int64_t)kvh * n_rows + row0) * n_sub + rgi * kRowsPerGroup;
  float* const row_lse = a.row_lse + (int64_t)kvh * n_rows + row0 + rgi * kRowsPerGroup;
  const int64_t cidx = ((int64_t)p.b * a.plan.num_kv_heads + kvh) * a.plan.rg_max + rgi;
  const int32_t* ptab = a.page_table + (int64_t)p.b * a.plan.max_pages;
  const bool need_anc = t1 * kTileKeys > L;
  if (need_anc && warp == 0)
    tc::tree_ancestors(a.parents + sq.node0, T, ctrl.parents, ctrl.anc, a.plan.status);
  __syncthreads();

  // this warp's blocks of 16 keys: units warp, warp + W, ... of the item;
  // block i is block i % 4 of its unit i / 4
  constexpr int kUnit = 4;
  const int nb_item = (min(t1 * kTileKeys, L + T) - t0 * kTileKeys + 15) / 16;
  const int n_units = (nb_item + kUnit - 1) / kUnit;
  const int mine = n_units > warp ? (n_units - warp - 1) / W + 1 : 0;
  const int last_unit = warp + (mine - 1) * W;
  const int nblk = mine > 0 ? (mine - 1) * kUnit + min(kUnit, nb_item - last_unit * kUnit) : 0;
  const int first_key = t0 * kTileKeys + warp * kUnit * 16;
  const int pshift = __ffs(P) - 1;
  auto key_of = [&](int i) { return first_key + (i >> 2) * (W * kUnit * 16) + (i & 3) * 16; };
  const uint32_t ring = smem_addr(smem) + warp * C_::kRing;
  const uint32_t blk = DS_KV4_BLOCK_BYTES(P, D);
  const uint8_t* k_head = ka.k4 + (int64_t)kvh * blk;
  const uint8_t* v_head = ka.v4 + (int64_t)kvh * blk;
  const int64_t page_bytes = (int64_t)a.plan.num_kv_heads * blk;
  const float c2 = a.scale_log2;

  // output row of row r of this row group
  auto out_row = [&](int r) {
    const int grow = rgi * kRowsPerGroup + r;
    return ((int64_t)sq.node0 + grow / G) * a.num_q_heads + kvh * G + grow % G;
  };
  auto put = [&](void* dst, int64_t at, float x) {
    if (a.out_f32) static_cast<float*>(dst)[at] = x;
    else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(x);
  };

  for (int r0 = 0; r0 < rows; r0 += R) {
    // queries of rows r0 .. r0 + R - 1: column g of tile nt is row r0 + 8 nt + g
    uint32_t q[NT][NS][2];
    uint64_t anc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r0 + 8 * n + g;
      const int grow = rgi * kRowsPerGroup + r;
      const __nv_bfloat16* src =
          a.q + (((int64_t)sq.node0 + grow / G) * a.num_q_heads + kvh * G + grow % G) * D +
          t * (D / 4);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {            // 8 channels: steps 2w, 2w + 1
        const uint4 x = r < rows ? __ldg(reinterpret_cast<const uint4*>(src) + w)
                                 : make_uint4(0, 0, 0, 0);
        q[n][2 * w][0] = bf16x2_to_f16x2(x.x);
        q[n][2 * w][1] = bf16x2_to_f16x2(x.y);
        q[n][2 * w + 1][0] = bf16x2_to_f16x2(x.z);
        q[n][2 * w + 1][1] = bf16x2_to_f16x2(x.w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = r0 + 8 * n + 2 * t + e;
        anc[n][e] = need_anc && rr < rows ? ctrl.anc[(rgi * kRowsPerGroup + rr) / G] : 0ull;
      }
    }
    float o[NT][NS][4];
    float m[NT][2], l[NT][2], cs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -CUDART_INF_F;
        l[n][e] = cs[n][e] = 0.f;
      }
    }

    // page ids of this warp's blocks, 32 at a time, the next 32 on their way
    auto ids_of = [&](int i) { return i < nblk ? __ldg(ptab + (key_of(i) >> pshift)) : 0; };
    int ids = ids_of(lane), next_ids = ids_of(32 + lane);
    // pieces this lane copies: one or two of the codes of each tensor, and
    // for the first lanes one of the scales
    constexpr int PPK = CB / 16;                    // 16-byte pieces of a key
    constexpr int SP = SB;                          // pieces of 16 keys' scales
    const int pk = lane / PPK;                      // key of the first piece
    const uint32_t dcode =
        ring + pk * CB + ((D == 128 ? lane % PPK ^ (((pk >> 2) & 1) << 1) : lane % PPK) << 4);
    const uint32_t dscale = ring + (lane / SP) * C_::kTensor + 16 * CB + (lane % SP) * 16;
    const uint8_t* const s_head =
        (lane / SP ? v_head : k_head) + (P << (D == 128 ? 6 : 5)) + (lane % SP) * 16;
    auto issue = [&](int i) {
      if (i < nblk) {
        if (i > 0 && (i & 31) == 0) {
          ids = next_ids;
          next_ids = ids_of(i + 32 + lane);
        }
        const int pg = __shfl_sync(0xffffffffu, ids, i & 31);
        const bool ok = (uint32_t)pg < (uint32_t)a.num_pages;
        if (!ok && lane == 0) flag(a.plan.status, DS_DEV_BAD_PAGE);
        const uint32_t n = ok ? 16u : 0u;
        const int64_t at = (int64_t)(ok ? pg : 0) * page_bytes;
        const int off = key_of(i) & (P - 1);
        const uint32_t st = (i % kStages) * 2 * C_::kTensor;
        const int64_t code = at + (off * CB + lane * 16);
#pragma unroll
        for (int c = 0; c < PPK / 2; ++c) {         // keys pk and, at 128, pk + 8
          cp16(dcode + st + c * 512, k_head + code + c * 512, n);
          cp16(dcode + st + C_::kTensor + c * 512, v_head + code + c * 512, n);
        }
        if (lane < 2 * SP) cp16(dscale + st, s_head + at + off * SB, n);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // fragment row g of a block, and the lane's four keys of the second product
    const int krow = g ^ ((g >> 1) & 1);
    const uint32_t kcode =
        ring + krow * CB + (D == 128 ? (t ^ (((krow >> 2) & 1) << 1)) << 4 : t * 8);
    const uint32_t kscale = ring + 16 * CB + krow * SB + (D == 128 ? 2 * t : t);
    uint32_t vcode[2], vscale[2];                   // keys of fragment rows 2t and 2t + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int key = 2 * t + (e ^ (t & 1));
      vcode[e] = ring + C_::kTensor + key * CB +
                 (D == 128 ? (((g >> 1) ^ (((key >> 2) & 1) << 1)) << 4) + (g & 1) * 8 : g * 4);
      vscale[e] = ring + C_::kTensor + 16 * CB + key * SB + (D == 128 ? g : g >> 1);
    }
#pragma unroll 1
    for (int i = 0; i < nblk; ++i) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(i + kStages - 1);
      const uint32_t st = (i % kStages) * 2 * C_::kTensor;
      const int key0 = key_of(i);
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      // ------------------------------------------------------------ Q K^T
      {
        uint32_t w[2][D / 32], sc[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {               // keys krow and 8 + krow
          if constexpr (D == 128) {
            const uint4 x = lds128(kcode + st + h * 8 * CB);
            w[h][0] = x.x; w[h][1] = x.y; w[h][2] = x.z; w[h][3] = x.w;
            const uint32_t s2 = kv4_scales_f16(lds_u16(kscale + st + h * 8 * SB));
            sc[h][0] = __byte_perm(s2, s2, 0x1010);
            sc[h][1] = __byte_perm(s2, s2, 0x3232);
          } else {
            const uint2 x = lds64(kcode + st + h * 8 * CB);
            w[h][0] = x.x; w[h][1] = x.y;
            const uint32_t b = lds_u8(kscale + st + h * 8 * SB);
            sc[h][0] = sc[h][1] = kv4_scales_f16(b | b << 8);
          }
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {          // 8 channels of each key
          uint32_t v0[4], v1[4];
          kv4_codes_f16(w[0][k], v0);
          kv4_codes_f16(w[1][k], v1);
          const int si = D == 128 ? k >> 1 : 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v0[e] = hmul2(v0[e], sc[0][si]);
            v1[e] = hmul2(v1[e], sc[1][si]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t fa[4] = {v0[2 * e], v1[2 * e], v0[2 * e + 1], v1[2 * e + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[n], fa, q[n][2 * k + e][0], q[n][2 * k + e][1]);
          }
        }
      }
      // ---------------------------------------------------------- softmax
      // element 2h + e of tile n: key 8h + krow, row 8n + 2t + e
      const bool tail = key0 + 16 > L;
      if (tail) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int d = key0 + 8 * (x >> 1) + krow - L;        // tree slot when >= 0
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (d >= 0 && !(d < T && ((anc[n][x & 1] >> d) & 1))) s[n][x] = -CUDART_INF_F;
        }
      }
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[n][e] = fmaf(fmaxf(s[n][e], s[n][2 + e]), c2, -7.f);
      // lazy maximum, 2^7 above the reference so that P fills f16's range
      bool need = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) need |= mx[n][e] > m[n][e] + 8.f;
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
            l[n][e] *= al;
            cs[n][e] *= al;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              o[n][j][e] *= al;
              o[n][j][e + 2] *= al;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float pr[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // a row that has seen nothing: 2^(-inf - 0)
          const float mb = m[n][x & 1] == -CUDART_INF_F ? 0.f : m[n][x & 1];
          pr[x] = ex2(fmaf(s[n][x], c2, -mb));
        }
        l[n][0] += pr[0] + pr[2];
        l[n][1] += pr[1] + pr[3];
        if (C) {
          const bool c0 = !tail || key0 + krow < L, c1 = !tail || key0 + 8 + krow < L;
          cs[n][0] += (c0 ? pr[0] : 0.f) + (c1 ? pr[2] : 0.f);
          cs[n][1] += (c0 ? pr[1] : 0.f) + (c1 ? pr[3] : 0.f);
        }
        pb[n][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
        pb[n][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
      }
      // log2 of the chunk's mass when this block ends the chunk or the context
      if (C && key0 < L && (((key0 + 16) & (C - 1)) == 0 || key0 + 16 >= L)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = cs[n][e];
            cs[n][e] = 0.f;
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
            const int r = r0 + 8 * n + 2 * t + e;
            if (g == 0 && r < rows)
              mass[(int64_t)(key0 / C) * sq.rows + r] =
                  x > 0.f ? m[n][e] + __log2f(x) : -CUDART_INF_F;
          }
      }
      // -------------------------------------------------------------- P V
      // fragment rows 2t + e and 8 + 2t + e are keys 2t + (e ^ (t & 1))
      {
        constexpr int VW = D / 64;                  // words of 8 dims of a key
        uint32_t w[4][VW], b[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (D == 128) {
            const uint2 y = lds64(vcode[x & 1] + st + (x >> 1) * 8 * CB);
            w[x][0] = y.x;
            w[x][VW - 1] = y.y;
          } else {
            w[x][0] = lds32(vcode[x & 1] + st + (x >> 1) * 8 * CB);
          }
          b[x] = lds_u8(vscale[x & 1] + st + (x >> 1) * 8 * SB);
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
            for (int n = 0; n < NT; ++n) mma16816(o[n][4 * k + j], fa, pb[n][0], pb[n][1]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();

    // ------------------------------------------- merge of the block's warps
    float* ow = reinterpret_cast<float*>(smem + warp * C_::kRing);   // [row][D]
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
          *reinterpret_cast<float2*>(ow + r * D + g * (D / 8) + 2 * j) =
              make_float2(o[n][j][e], o[n][j][e + 2]);
      }
    __syncthreads();
    for (int x = threadIdx.x; x < R * D; x += 32 * W) {
      const int r = x / D;
      if (r0 + r >= rows) break;
      float mm = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < W; ++w) mm = fmaxf(mm, ctrl.m[w][r]);
      const float mb = mm == -CUDART_INF_F ? 0.f : mm;
      float sum = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2(ctrl.m[w][r] - mb);
        sum = fmaf(f, ctrl.l[w][r], sum);
        acc = fmaf(f, reinterpret_cast<const float*>(smem + w * C_::kRing)[x], acc);
      }
      const float inv = sum > 0.f ? ka.out_mult / sum : 0.f;
      const float lse = sum > 0.f ? mm + __log2f(sum) : -CUDART_INF_F;
      if (sq.splits == 1) {
        put(a.out, out_row(r0 + r) * D + x % D, acc * inv);
        if (x % D == 0) row_lse[r0 + r] = lse;
      } else {
        const int64_t row = (int64_t)blockIdx.x * kRowsPerGroup + r0 + r;
        put(a.o_part, row * D + x % D, acc * inv);
        if (x % D == 0) a.lse_part[row] = lse;
      }
    }
    __syncthreads();
  }
  if (sq.splits == 1) return;

  // The last split to finish merges them: one warp per row, the log2-sum-exp
  // of the row from its splits' (lane-parallel), then the outputs.
  const int64_t base = (int64_t)sq.item_base + (kvh * sq.rg + rgi) * sq.splits;
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t prev = atomicAdd(a.counters + cidx, 1u);
    ctrl.last = prev + 1 == (uint32_t)sq.splits;
    if (ctrl.last) {
      a.counters[cidx] = 0u;
      __threadfence();
    }
  }
  __syncthreads();
  if (!ctrl.last) return;
  for (int r = warp; r < rows; r += W) {
    const float* lp = a.lse_part + base * kRowsPerGroup + r;
    float mm = -CUDART_INF_F, sum = 0.f;
    for (int k = lane; k < sq.splits; k += 32)
      mm = fmaxf(mm, __ldcg(lp + (int64_t)k * kRowsPerGroup));
    mm = warp_max(mm);
    const float mb = mm == -CUDART_INF_F ? 0.f : mm;
    for (int k = lane; k < sq.splits; k += 32)
      sum += ex2(__ldcg(lp + (int64_t)k * kRowsPerGroup) - mb);
    sum = warp_sum(sum);
    const float lse = sum > 0.f ? mm + __log2f(sum) : -CUDART_INF_F;
    if (lane == 0) row_lse[r] = lse;
    if (a.out_f32) combine_row_splits<D, false, 8>(a, base, sq.splits, r, lse, out_row(r));
    else combine_row_splits<D, true, D == 128 ? 20 : 32>(a, base, sq.splits, r, lse, out_row(r));
  }
}

// Chunk scores: the sum over kv heads and rows of 2^(mass - the row's
// log2-sum-exp).  A block covers 32 chunks of a sequence, a lane each; warp w
// the kv heads w, w + 8, ..., whose sums are added in that order.
__global__ void __launch_bounds__(256) kv4_scores_few(const VerifyKArgs a) {
  __shared__ float part[8][32];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const SeqPlan sq = seq_sizes(a.plan, b, false);
  const int sub = min(64, a.plan.chunk_size), per = a.plan.chunk_size / sub;
  const int n_sub = (sq.L + sub - 1) / sub;       // of this sequence
  const int64_t n_rows = (int64_t)a.plan.n_nodes * a.plan.group;
  const int64_t row0 = (int64_t)sq.node0 * a.plan.group;
  const int64_t stride = (int64_t)a.plan.max_chunks * per;
  float sum = 0.f;
  for (int h = warp; h < a.plan.num_kv_heads; h += 8) {
    const float* lse = a.row_lse + h * n_rows + row0;
    const float* mass = a.clse + (h * n_rows + row0) * stride;
    for (int k = c * per; k < min((c + 1) * per, n_sub); ++k) {
      const float* mk = mass + (int64_t)k * sq.rows;
#pragma unroll 4
      for (int r = 0; r < sq.rows; ++r) sum += exp2f(__ldcg(mk + r) - __ldcg(lse + r));
    }
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp > 0 || c >= (sq.L + a.plan.chunk_size - 1) / a.plan.chunk_size) return;
  sum = part[0][lane];
#pragma unroll
  for (int w = 1; w < 8; ++w) sum += part[w][lane];
  float* dst = a.scores + (int64_t)b * a.plan.max_chunks + c;
  *dst = a.accumulate ? *dst + sum : sum;
}

template <int D, int NT>
static cudaError_t launch(const Kv4KArgs& k, const VerifyLayout& L, cudaStream_t stream) {
  const size_t smem = Cfg<D, NT>::smem;
  cudaError_t e = cudaFuncSetAttribute(kv4_split_few<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv4_split_few<D, NT>, dim3(L.max_items), dim3(32 * Cfg<D, NT>::W), smem,
                       stream, k);
  if (e != cudaSuccess || !k.v.scores || k.v.plan.max_chunks == 0) return e;
  return launch_dependent(kv4_scores_few,
                          dim3((k.v.plan.max_chunks + 31) / 32, k.v.plan.batch), dim3(256), 0,
                          stream, k.v);
}

}  // namespace kv4few

cudaError_t launch_kv4_few(const Kv4KArgs& k, int head_dim, int rows, const VerifyLayout& L,
                                 cudaStream_t stream) {
  using kv4few::launch;
  if (rows <= 8) return head_dim == 128 ? launch<128, 1>(k, L, stream) : launch<64, 1>(k, L, stream);
  return head_dim == 128 ? launch<128, 2>(k, L, stream) : launch<64, 2>(k, L, stream);
}

}  // namespace ds
