// Softmax, output and split-merge pieces of the tcgen05 split passes (the
// bf16 cache's in verify_tc.cu, the 4-bit cache's in kv4_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "dev_common.cuh"
#include "tc_ptx.cuh"
#include "verify_common.cuh"

namespace ds {
namespace tc {

// One 64-key unit of one softmax thread (one query row): loads the row's 64
// scores from tensor memory, applies the tree/tail mask (TAIL only), updates
// the running maximum lazily, writes the exponentials as bf16 P over the
// first 32 columns of the buffer, and emits the log2 attention mass of every
// context chunk that ends in this unit.  `cs` carries the context mass of a
// chunk that started in the previous unit of the same tile.  Returns the
// factor by which O must be scaled (alpha) and whether any row of the warp
// needs it.
//
// F16: P is f16 instead (with f16 V).  f16 has three more bits than bf16 but
// little range, so the reference point m2 sits 2^7 below the row's maximum:
// P reaches up to 2^15 and loses bits only below 2^-21 of the maximum.
template <bool TAIL, bool F16 = false>
DS_DEV void softmax_unit(const uint32_t tS, const uint32_t tP, const uint32_t vw0,
                         const uint32_t vw1,
                         const uint32_t cw0, const uint32_t cw1, const float c2, const bool first,
                         float& m2, float& l, float& cs, float& alpha, bool& rescale,
                         const int tile_slot0, const int kbase, const int cshift, const int n_ch,
                         const bool row_ok, float* __restrict__ clse_row) {
  using namespace ptx;
  float s[64];
  {
    uint32_t r0[32], r1[32];
    tmem_ld32(tS, r0);
    tmem_ld32(tS + 32, r1);
    tmem_ld_wait(r0);
    tmem_ld_wait(r1);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      s[i] = __uint_as_float(r0[i]);
      s[32 + i] = __uint_as_float(r1[i]);
    }
  }
  if constexpr (TAIL) {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (!((vw0 >> c) & 1u)) s[c] = -CUDART_INF_F;
      if (!((vw1 >> c) & 1u)) s[32 + c] = -CUDART_INF_F;
    }
  }
  // row maximum: three-input max, four independent chains of 16
  float mx4[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float m = fmax3(s[16 * k], s[16 * k + 1], s[16 * k + 2]);
#pragma unroll
    for (int i = 3; i < 15; i += 2) m = fmax3(m, s[16 * k + i], s[16 * k + i + 1]);
    mx4[k] = fmaxf(m, s[16 * k + 15]);
  }
  float mx2 = fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3])) * c2;
  if constexpr (F16) mx2 -= 7.f;
  alpha = 1.f;
  rescale = false;
  if (first) {
    m2 = mx2;
  } else {
    const bool need = mx2 > m2 + 8.f;
    rescale = __any_sync(0xffffffffu, need);
    if (need) {
      alpha = ex2(m2 - mx2);
      m2 = mx2;
    }
  }
  const float mb = (m2 == -CUDART_INF_F) ? 0.f : m2;
  // exponentials (masked columns: ex2(-inf) = 0) and per-16-column sums of
  // the context columns; tree columns of a tail unit go to tsum
  float cg[4];
  float tsum = 0.f;
  if constexpr (TAIL) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int c = 16 * k + i;
        const float e0 = ex2(fmaf(s[c], c2, -mb));
        const float e1 = ex2(fmaf(s[c + 1], c2, -mb));
        s[c] = e0;
        s[c + 1] = e1;
        const uint32_t w = c < 32 ? cw0 : cw1;
        const bool k0 = (w >> (c & 31)) & 1u;
        const bool k1 = (w >> ((c + 1) & 31)) & 1u;
        a0 += k0 ? e0 : 0.f;
        a1 += k1 ? e1 : 0.f;
        tsum += (k0 ? 0.f : e0) + (k1 ? 0.f : e1);
      }
      cg[k] = a0 + a1;
    }
  } else {
    // pairs of columns in f32x2 arithmetic: (s c2 - mb) and the running sums
    const uint64_t c2x2 = f2pack(c2, c2), nmb2 = f2pack(-mb, -mb);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint64_t acc = f2pack(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int c = 16 * k + i;
        float x0, x1;
        f2unpack(ffma2(f2pack(s[c], s[c + 1]), c2x2, nmb2), x0, x1);
        s[c] = ex2(x0);
        s[c + 1] = ex2(x1);
        acc = fadd2(acc, f2pack(s[c], s[c + 1]));
      }
      float lo, hi;
      f2unpack(acc, lo, hi);
      cg[k] = lo + hi;
    }
  }
  l = l * alpha + (tsum + ((cg[0] + cg[1]) + (cg[2] + cg[3])));
  // chunk log2-mass at chunk boundaries (C/16 sixteen-column groups a chunk)
  {
    const int per_mask = (1 << (cshift - 4)) - 1;
    cs *= alpha;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      cs += cg[k];
      const int kg = kbase + k;          // 16-column group index in the tile
      if (((kg + 1) & per_mask) == 0) {
        const int cidx = (tile_slot0 + kg * 16) >> cshift;
        if (row_ok && cidx < n_ch)
          clse_row[(int64_t)cidx * kRowsPerGroup] = cs > 0.f ? mb + __log2f(cs) : -CUDART_INF_F;
        cs = 0.f;
      }
    }
  }
  // P as bf16 (f16) pairs (keys 2i, 2i+1 -> column i of tP)
  uint32_t pk[32];
#pragma unroll
  for (int i = 0; i < 32; ++i)
    pk[i] = F16 ? pack_f16x2(s[2 * i], s[2 * i + 1]) : pack_bf16x2(s[2 * i], s[2 * i + 1]);
  tmem_st32(tP, pk);
}

// Output of one softmax thread after its last tile: O / l (merged with the
// other group's partial result in key mode) and the row's log2-sum-exp.
// The rows are written through a per-warp staging tile in shared memory
// (`stage`, 32 rows x 32 floats = 4 KB, idle by then; 16-byte chunk c of row
// r stored at chunk c ^ (r % 8), so that eight consecutive lanes touch all
// 32 banks both when a thread writes its row and when a lane reads a row
// segment): each thread writes its row's 32-column slice, then each warp
// store writes four rows' 128-byte segments, so the global writes are whole
// segments instead of 32 rows' scattered 16 bytes.
constexpr int kStageStride = 32;   // floats per staged row

template <int D>
__device__ __noinline__ void write_row_output(const bool row_mode, const int g, const bool ok,
                                              const int nt1, const uint32_t tO, const int lrow,
                                              const int rows_left, const float m2,
                                              const float l, float* __restrict__ merge_buf,
                                              float* m1buf, float* l1buf,
                                              float* __restrict__ stage,
                                              const bool part_bf16,
                                              void* __restrict__ op_warp,
                                              float* __restrict__ lse_out) {
  using namespace ptx;
  const int lane = threadIdx.x & 31;
  const bool row_ok = (lrow & 31) < rows_left;
  if (!row_mode && g == 1) {
    if (ok && nt1 > 0) {
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        uint32_t r[32];
        tmem_ld32(tO + c4 * 32, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) merge_buf[(c4 * 32 + i) * 128 + lrow] = __uint_as_float(r[i]);
      }
    }
    m1buf[lrow] = m2;
    l1buf[lrow] = l;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    return;
  }
  float sc0 = 1.f, sc1 = 0.f, lt = l, mt = m2;
  if (!row_mode) {
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (nt1 > 0) {
      const float m1 = m1buf[lrow], l1 = l1buf[lrow];
      mt = fmaxf(m2, m1);
      const float mb2 = (mt == -CUDART_INF_F) ? 0.f : mt;
      sc0 = l > 0.f ? ex2(m2 - mb2) : 0.f;
      sc1 = l1 > 0.f ? ex2(m1 - mb2) : 0.f;
      lt = l * sc0 + l1 * sc1;
    }
  }
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
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
    for (int i = 0; i < 32; ++i) {
      float o = __uint_as_float(r[i]) * sc0;
      if (sc1 != 0.f) o += merge_buf[(c4 * 32 + i) * 128 + lrow] * sc1;
      r[i] = __float_as_uint(o * inv);
    }
    if (part_bf16) {
      // bf16 pairs: a row's 32 columns are 64 bytes, four 16-byte chunks;
      // chunk c of row q sits in the row's slot c ^ ((q / 2) % 4), so that
      // eight lanes of one access (eight rows, or two rows' four chunks)
      // touch distinct 16-byte bank groups
      uint32_t* st = reinterpret_cast<uint32_t*>(stage) + lane * 16;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16x2(__uint_as_float(r[8 * c + 2 * e]),
                             __uint_as_float(r[8 * c + 2 * e + 1]));
        *reinterpret_cast<uint4*>(st + 4 * (c ^ ((lane >> 1) & 3))) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
      // rows 8k + lane / 4, 16-byte chunk lane % 4 of the slice
      __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(op_warp);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = 8 * k + (lane >> 2), cc = lane & 3;
        if (rr < rows_left) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              reinterpret_cast<const uint32_t*>(stage) + rr * 16 + 4 * (cc ^ ((rr >> 1) & 3)));
          *reinterpret_cast<uint4*>(ob + (int64_t)rr * D + c4 * 32 + cc * 8) = v;
        }
      }
      __syncwarp();
      continue;
    }
    // f32: this thread's row, 32 columns, into the staging tile
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(stage + lane * kStageStride + 4 * ((i >> 2) ^ (lane & 7))) =
          make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]),
                      __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
    __syncwarp();
    // rows 4k + lane / 8, columns 4 (lane % 8) .. + 3 of the slice
    float* of = reinterpret_cast<float*>(op_warp);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int rr = 4 * k + (lane >> 3), cc = 4 * (lane & 7);
      if (rr < rows_left) {
        const float4 v = *reinterpret_cast<const float4*>(
            stage + rr * kStageStride + 4 * ((lane & 7) ^ (rr & 7)));
        *reinterpret_cast<float4*>(of + (int64_t)rr * D + c4 * 32 + cc) = v;
      }
    }
    __syncwarp();
  }
  if (row_ok) *lse_out = lt > 0.f ? mt + __log2f(lt) : -CUDART_INF_F;
}

// Ancestor masks (bit i of anc[j]: i is j or an ancestor of j) of all T nodes
// of a tree, by pointer doubling; one warp.  `parents` and `anc` are the
// block's arrays in shared memory.
DS_DEV void tree_ancestors(const int32_t* parents_seq, int T, int32_t* parents, uint64_t* anc,
                           uint32_t* status) {
  const int lane = threadIdx.x & 31;
  for (int j = lane; j < T; j += 32) parents[j] = __ldg(parents_seq + j);
  __syncwarp();
  uint64_t m[2] = {0, 0};
  int up[2] = {-1, -1};
  for (int k = 0; k < 2; ++k) {
    const int j = lane + 32 * k;
    if (j < T) {
      int pj = parents[j];
      bool ok = (j == 0) ? (pj == -1) : (pj >= 0 && pj < j);
      if (!ok) {
        flag(status, DS_DEV_BAD_TREE);
        pj = -1;
      }
      m[k] = (1ull << j) | (pj >= 0 ? (1ull << pj) : 0ull);
      up[k] = pj;
      anc[j] = m[k];
      parents[j] = pj;   // sanitised jump pointer
    }
  }
  __syncwarp();
  for (int round = 0; round < 6; ++round) {
    uint64_t add[2] = {0, 0};
    int nup[2] = {-1, -1};
    for (int k = 0; k < 2; ++k) {
      const int j = lane + 32 * k;
      if (j < T && up[k] >= 0) {
        add[k] = anc[up[k]];
        nup[k] = parents[up[k]];
      }
    }
    __syncwarp();
    for (int k = 0; k < 2; ++k) {
      const int j = lane + 32 * k;
      if (j < T) {
        m[k] |= add[k];
        up[k] = nup[k];
        anc[j] = m[k];
        parents[j] = nup[k];
      }
    }
    __syncwarp();
  }
}

// Final log2-sum-exp of one row from its ns splits' (lp[s * 256]): 32 loads
// at a time, merged as a running (max, sum of 2^(x - max)).
DS_DEV float row_lse_from_splits(const float* lp, int ns) {
  constexpr int kB = 32;
  float mx = -CUDART_INF_F, sum = 0.f;
  for (int s0 = 0; s0 < ns; s0 += kB) {
    float v[kB];
#pragma unroll
    for (int k = 0; k < kB; ++k)
      v[k] = s0 + k < ns ? __ldcg(lp + (int64_t)(s0 + k) * kRowsPerGroup) : -CUDART_INF_F;
    float bm = v[0];
#pragma unroll
    for (int k = 1; k < kB; ++k) bm = fmaxf(bm, v[k]);
    const float nm = fmaxf(mx, bm);
    if (nm == -CUDART_INF_F) continue;
    float add = 0.f;
#pragma unroll
    for (int k = 0; k < kB; ++k) add += exp2f(v[k] - nm);
    sum = (mx == -CUDART_INF_F ? 0.f : sum * exp2f(mx - nm)) + add;
    mx = nm;
  }
  return sum > 0.f ? mx + log2f(sum) : -CUDART_INF_F;
}

}  // namespace tc
}  // namespace ds
