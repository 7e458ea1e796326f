// Tree-verify attention over the 4-bit paged cache (include/ds.h,
// ds_kv4_verify_attn): a pass for few query rows per sequence and kv head
// (kv4_few.cu) and one for trees (kv4_tc.cu).
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

#include "dev_common.cuh"
#include "internal.h"
#include "kv4_common.cuh"
#include "verify_common.cuh"

namespace ds {

int kv4_few_rows(const ds_kv4_attn_args& a) {
  // Rows per sequence and kv head on average: the trees' sizes are on the
  // device, and both passes handle any.  The tree pass takes as long for any
  // number up to its tile of 128, this one in proportion to tiles of 8 from
  // the second on.  Single calls with the cache not in the L2, 8 kv heads, 4
  // rows a node, 128K keys: 2 nodes 54 us, 4 nodes 68, 5 to 32 nodes in the
  // tree pass 95 to 99.  8 sequences of 2K: 4 nodes 31, 5 nodes there 44;
  // head_dim 64, 128K: 50 and 80.  All trees of these batches are alike: in a
  // mixed one the rule may give some sequences the slower pass.
  const int64_t group = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = ((int64_t)a.n_nodes + a.batch - 1) / a.batch * group;
  if (rows > 16) return 0;
  // the few-row pass counts its work (32-key units, and segments) in 32 bits
  const int64_t segs = a.num_kv_heads * (a.batch + a.n_nodes * group / 8 + 1);
  const int64_t units = segs * ((int64_t)a.max_pages * a.page_size / 32 + 64);
  return units < ((int64_t)1 << 31) ? (int)rows : 0;
}

size_t kv4_counters(const ds_kv4_attn_args& a) {
  // The few-row pass counts arrivals by segment: at most 8 rows each but for
  // a sequence's last, and it takes calls of at most 16 rows a sequence and kv
  // head on average, so 3 a sequence and kv head.  Neither the number of
  // nodes nor the pass goes into it: what lies behind the counters stays where
  // it is when a workspace serves calls of other trees, and no call finds
  // anything but the zeros that the last one left in them.
  return (size_t)a.num_kv_heads * (3 * (size_t)a.batch + 1);
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
  // never zero: a hidden slot's score is -inf, and -inf times zero no number.
  // Products with the keys stay below 2^35, so that every weight is the same either way.
  k.scale_log2 = fmaxf(ldexpf(scale * kLog2e, a.k_exp), FLT_MIN);
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
  if (const int rows = kv4_few_rows(a)) return launch_kv4_few(ka, a.head_dim, rows, L, stream);
  return launch_kv4_tc(ka, a.head_dim, L, stream);
}

}  // namespace ds
