// Tree-verify attention over the 4-bit paged cache (include/ds.h,
// ds_kv4_verify_attn): the work plan, the split outputs and the finish kernel
// of ds_verify_attn, with a split pass that reads e2m1 codes and e4m3 scales.
//
// Split pass: one block of 256 threads per work item (sequence, kv head, row
// group of up to 256 query rows, range of 128-key tiles).  Each tile's K and
// V are brought to f16 in shared memory, where they are exact; one warp takes
// a query row at a time: a key per lane for the scores, a column per lane for
// the output.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <cmath>

#include "dev_common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "pdl.cuh"
#include "verify_common.cuh"

namespace ds {

struct Kv4KArgs {
  VerifyKArgs v;                  // k, v and the strides are not used
  const uint8_t* k4;
  const uint8_t* v4;
  float out_mult;                 // 2^v_exp
};

template <int D>
struct Kv4Smem {
  float o[kRowsPerGroup][D];
  __half k[kTileKeys][D + 2];
  __half v[kTileKeys][D];
  float m[kRowsPerGroup], l[kRowsPerGroup];
  float p[8][kTileKeys];
  uint64_t anc[DS_MAX_TREE_NODES];
  Plan plan;
  int last;
};

template <int D>
__global__ void __launch_bounds__(256) kv4_split(const Kv4KArgs ka) {
  extern __shared__ __align__(16) unsigned char raw[];
  Kv4Smem<D>& s = *reinterpret_cast<Kv4Smem<D>*>(raw);
  const VerifyKArgs& a = ka.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (warp == 0) {
    Plan p = plan_find(a.plan, -1, blockIdx.x);
    if (lane == 0) s.plan = p;
  }
  __syncthreads();
  const Plan p = s.plan;
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
  const int L = sq.L, T = sq.T, P = a.plan.page_size, C = a.plan.chunk_size;
  const int n_ch = a.scores ? (L + C - 1) / C : 0;
  const int64_t cidx = ((int64_t)p.b * a.plan.num_kv_heads + kvh) * a.plan.rg_max + rgi;
  const int32_t* ptab = a.page_table + (int64_t)p.b * a.plan.max_pages;
  for (int j = threadIdx.x; j < T; j += 256)
    s.anc[j] = ancestor_mask(a.parents + sq.node0, j, T, a.plan.status);
  for (int i = threadIdx.x; i < rows * D; i += 256) (&s.o[0][0])[i] = 0.f;
  for (int i = threadIdx.x; i < rows; i += 256) {
    s.m[i] = -CUDART_INF_F;
    s.l[i] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * kTileKeys * (D / 8); e += 256) {
      const int tensor = e / (kTileKeys * (D / 8)), i = e % (kTileKeys * (D / 8));
      const int key = i / (D / 8), w = i % (D / 8);
      const int slot = t * kTileKeys + key;
      uint32_t v[4] = {0, 0, 0, 0};
      if (slot < L + T) {
        const int pg = __ldg(ptab + slot / P);
        if (pg < 0 || pg >= a.num_pages) {
          flag(a.plan.status, DS_DEV_BAD_PAGE);
        } else {
          const uint8_t* blk = (tensor ? ka.v4 : ka.k4) +
                               ((int64_t)pg * a.plan.num_kv_heads + kvh) *
                                   DS_KV4_BLOCK_BYTES(P, D);
          const int off = slot % P;
          kv4_codes_f16(__ldg(reinterpret_cast<const uint32_t*>(blk + off * (D / 2)) + w), v);
          const uint32_t sb = __ldg(blk + P * (D / 2) + off * (D / 16) + w / 2);
          const uint32_t sc = kv4_scales_f16(sb | sb << 8);
          for (int k = 0; k < 4; ++k) v[k] = hmul2(v[k], sc);
        }
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(tensor ? &s.v[key][8 * w] : &s.k[key][8 * w]);
      for (int k = 0; k < 4; ++k) dst[k] = v[k];
    }
    __syncthreads();
    for (int r = warp; r < rows; r += 8) {
      const int grow = rgi * kRowsPerGroup + r;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) +
                          (((int64_t)sq.node0 + grow / G) * a.num_q_heads + kvh * G + grow % G) *
                              (D / 2);
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int d = 0; d < D / 2; ++d) {
        const uint32_t qw = bf16x2_to_f16x2(__ldg(q + d));
        const float2 qf = __half22float2(*reinterpret_cast<const __half2*>(&qw));
        for (int i = 0; i < 4; ++i) {
          const float2 kf =
              __half22float2(*reinterpret_cast<const __half2*>(&s.k[32 * i + lane][2 * d]));
          x[i] = fmaf(qf.x, kf.x, fmaf(qf.y, kf.y, x[i]));
        }
      }
      float mx = s.m[r];
      const float m0 = mx;
      for (int i = 0; i < 4; ++i) {
        const int slot = t * kTileKeys + 32 * i + lane;
        const bool seen = slot < L || (slot < L + T && ((s.anc[grow / G] >> (slot - L)) & 1));
        x[i] = seen ? x[i] * a.scale_log2 : -CUDART_INF_F;
        mx = fmaxf(mx, x[i]);
      }
      mx = warp_max(mx);
      const float mb = mx == -CUDART_INF_F ? 0.f : mx;
      float sum = 0.f;
      for (int i = 0; i < 4; ++i) {
        const float e = exp2f(x[i] - mb);
        s.p[warp][32 * i + lane] = e;
        sum += e;
      }
      const float alpha = exp2f(m0 - mb);
      sum = warp_sum(sum);
      __syncwarp();
      if (lane == 0) {
        s.m[r] = mx;
        s.l[r] = s.l[r] * alpha + sum;
      }
      for (int d = lane; d < D; d += 32) {
        float o = s.o[r][d] * alpha;
        for (int k = 0; k < kTileKeys; ++k) o = fmaf(s.p[warp][k], __half2float(s.v[k][d]), o);
        s.o[r][d] = o;
      }
      // log2 of every chunk's mass: context keys only
      if (lane < kTileKeys / C) {
        const int c = t * (kTileKeys / C) + lane;
        if (c < n_ch) {
          float cs = 0.f;
          for (int k = 0; k < C; ++k)
            if (c * C + k < L) cs += s.p[warp][lane * C + k];
          a.clse[(cidx * a.plan.max_chunks + c) * kRowsPerGroup + r] =
              cs > 0.f ? mb + log2f(cs) : -CUDART_INF_F;
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += 256) {
    const int r = i / D;
    const float o = s.l[r] > 0.f ? s.o[r][i % D] / s.l[r] * ka.out_mult : 0.f;
    const int64_t at = ((int64_t)blockIdx.x * kRowsPerGroup) * D + i;
    if (a.out_f32) a.o_part[at] = o;
    else reinterpret_cast<__nv_bfloat16*>(a.o_part)[at] = __float2bfloat16_rn(o);
  }
  for (int r = threadIdx.x; r < rows; r += 256)
    a.lse_part[(int64_t)blockIdx.x * kRowsPerGroup + r] =
        s.l[r] > 0.f ? s.m[r] + log2f(s.l[r]) : -CUDART_INF_F;
  // the last split of the row group to finish forms the rows' final
  // log2-sum-exp and the descriptor the finish kernel reads
  __threadfence();
  __syncthreads();
  const int64_t base = (int64_t)sq.item_base + (kvh * sq.rg + rgi) * sq.splits;
  if (threadIdx.x == 0) {
    s.last = atomicAdd(a.counters + cidx, 1u) + 1 == (uint32_t)sq.splits;
    if (s.last) {
      a.counters[cidx] = 0u;
      a.gdesc[cidx] = make_int4((int)base, sq.splits, 0, 0);
    }
    __threadfence();
  }
  __syncthreads();
  if (!s.last) return;
  for (int r = threadIdx.x; r < rows; r += 256) {
    const float* lp = a.lse_part + base * kRowsPerGroup + r;
    float mx = -CUDART_INF_F, sum = 0.f;
    for (int k = 0; k < sq.splits; ++k) mx = fmaxf(mx, __ldcg(lp + (int64_t)k * kRowsPerGroup));
    for (int k = 0; k < sq.splits && mx > -CUDART_INF_F; ++k)
      sum += exp2f(__ldcg(lp + (int64_t)k * kRowsPerGroup) - mx);
    a.row_lse[cidx * kRowsPerGroup + r] = sum > 0.f ? mx + log2f(sum) : -CUDART_INF_F;
  }
}

template <int D>
static cudaError_t launch_split(const Kv4KArgs& k, const VerifyLayout& L, cudaStream_t stream) {
  const size_t smem = sizeof(Kv4Smem<D>);
  static_assert(sizeof(Kv4Smem<D>) <= 232448, "above the 227 KB a block can have");
  cudaError_t e = cudaFuncSetAttribute(kv4_split<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv4_split<D>, dim3(L.max_items), dim3(256), smem, stream, k);
}

cudaError_t launch_kv4_attn(const ds_kv4_attn_args& a, const VerifyLayout& L,
                            cudaStream_t stream) {
  const ds_verify_args va = kv4_as_verify(a);
  Kv4KArgs ka = {};
  VerifyKArgs& k = ka.v;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  k.q = static_cast<const __nv_bfloat16*>(a.q);
  k.page_table = a.page_table;
  k.parents = a.parents;
  k.plan.ctx_lens = a.ctx_lens;
  k.plan.tree_offsets = a.tree_offsets;
  k.plan.batch = a.batch;
  k.plan.n_nodes = a.n_nodes;
  k.plan.num_kv_heads = a.num_kv_heads;
  k.plan.group = L.group;
  k.plan.page_size = a.page_size;
  k.plan.max_pages = a.max_pages;
  // without salience the chunk bound on the lengths must not bind
  k.plan.chunk_size = a.chunk_scores ? va.chunk_size : 128;
  k.plan.max_chunks = a.chunk_scores ? va.max_chunks : kKv4MaxSlots / 128;
  k.plan.target_ctas = L.target_ctas;
  k.plan.wave_ctas = L.wave_ctas;
  k.plan.rg_max = L.rg_max;
  k.plan.status = reinterpret_cast<uint32_t*>(ws);
  k.num_q_heads = a.num_q_heads;
  k.num_pages = a.num_pages;
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf((float)a.head_dim);
  k.scale_log2 = ldexpf(scale * kLog2e, a.k_exp);
  k.counters = reinterpret_cast<uint32_t*>(ws + L.counters);
  k.gdesc = reinterpret_cast<int4*>(ws + L.gdesc);
  k.o_part = reinterpret_cast<float*>(ws + L.o_part);
  k.lse_part = reinterpret_cast<float*>(ws + L.lse_part);
  k.clse = reinterpret_cast<float*>(ws + L.clse);
  k.row_lse = reinterpret_cast<float*>(ws + L.row_lse);
  k.out = a.out;
  k.out_f32 = a.out_dtype == DS_OUT_F32;
  k.scores = a.chunk_scores;
  k.accumulate = va.accumulate_scores;
  ka.k4 = static_cast<const uint8_t*>(a.k_cache);
  ka.v4 = static_cast<const uint8_t*>(a.v_cache);
  ka.out_mult = ldexpf(1.f, a.v_exp);
  cudaError_t e = a.head_dim == 128 ? launch_split<128>(ka, L, stream)
                                    : launch_split<64>(ka, L, stream);
  if (e != cudaSuccess) return e;
  return launch_finish(k, a.head_dim, L.rg_max, a.batch, stream);
}

}  // namespace ds
