// Rows of K and V into the paged 4-bit cache and back (include/ds.h,
// ds_kv4_write and ds_kv4_read).
//
// One thread handles one scale group: 16 channels of one row's head, 32 bytes
// of bf16 on one side, 8 bytes of codes and one scale byte on the other.
// Nothing is shared between threads: the maximum over the group, the scale
// and the codes are the thread's own.  A warp covers consecutive rows of one
// head (4 rows at head_dim 128, 8 at 64), whose slots are consecutive in the
// page block, so that its codes are one run of 256 bytes and its scales one
// of 32.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dev_common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "pdl.cuh"

namespace ds {

struct Kv4RowsKArgs {
  uint16_t* rows[2];              // K, V
  uint8_t* cache[2];
  int64_t row_stride[2];
  const int32_t* page_table;
  const int32_t* from_lens;
  const int32_t* row_offsets;
  const int32_t* path;
  const int32_t* n_accepted;
  int32_t batch, n_rows, num_kv_heads, page_size, num_pages, max_pages;
  float mult[2];                  // write: 2^-exp, read: 2^exp
  int32_t* new_lens;
  uint32_t* status;
};

// The sequence that owns row r: the last b with row_offsets[b] <= r.
DS_DEV int row_sequence(const int32_t* offs, int batch, int r) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offs + mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Sizes of sequence b: false (and a status bit) when they cannot be used.
DS_DEV bool rows_of(const Kv4RowsKArgs& a, int b, int& n0, int& n, int& from) {
  n0 = __ldg(a.row_offsets + b);
  const int n1 = __ldg(a.row_offsets + b + 1);
  from = __ldg(a.from_lens + b);
  n = n1 - n0;
  const bool ok = n0 >= 0 && n1 >= n0 && n1 <= a.n_rows && from >= 0 &&
                  (int64_t)from + n <= (int64_t)a.max_pages * a.page_size &&
                  (a.path == nullptr || n <= DS_MAX_TREE_NODES);
  if (!ok) flag(a.status, DS_DEV_BAD_LENGTH);
  return ok;
}

// Whether sequence b's path is strictly increasing inside (0, n).
DS_DEV bool path_ok(const Kv4RowsKArgs& a, int b, int n, int acc) {
  if (acc < 0 || acc > n - 1) return false;
  const int32_t* p = a.path + (int64_t)b * DS_MAX_TREE_NODES;
  int prev = 0;
  for (int i = 0; i < acc; ++i) {
    const int c = __ldg(p + i);
    if (c <= prev || c >= n) return false;
    prev = c;
  }
  return true;
}

template <int D, bool WRITE>
__global__ void __launch_bounds__(256) kv4_rows(const Kv4RowsKArgs a) {
  constexpr int NG = D / kKv4Group;       // scale groups of a head
  constexpr int RW = 32 / NG;             // rows of a warp
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int units = 2 * a.num_kv_heads;   // (tensor, head) pairs
  const int unit = (int)(w % units);
  // with a path, "rows" are the path's entries: DS_MAX_TREE_NODES a sequence
  const int total = a.path ? a.batch * DS_MAX_TREE_NODES : a.n_rows;
  const int64_t e = w / units * RW + lane / NG;
  // new lengths: the first thread of each sequence's number in the grid
  if (WRITE && a.new_lens) {
    const int64_t tid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t b = tid; b < a.batch; b += (int64_t)gridDim.x * 256) {
      int n0, n, from, add = 0;
      if (rows_of(a, (int)b, n0, n, from)) {
        add = n;
        if (a.path && n > 0) {
          const int acc = __ldg(a.n_accepted + b);
          add = 1 + (path_ok(a, (int)b, n, acc) ? acc : 0);
        }
      }
      a.new_lens[b] = from + add;
    }
  }
  if (e >= total) return;
  int row, slot, b, n0, n, from;
  if (WRITE && a.path) {
    b = (int)(e / DS_MAX_TREE_NODES);
    const int i = (int)(e % DS_MAX_TREE_NODES);
    if (!rows_of(a, b, n0, n, from) || n == 0) return;
    const int acc = __ldg(a.n_accepted + b);
    if (!path_ok(a, b, n, acc)) {
      flag(a.status, DS_DEV_BAD_TREE);
      return;
    }
    if (i >= acc) return;
    row = n0 + __ldg(a.path + (int64_t)b * DS_MAX_TREE_NODES + i);
    slot = from + 1 + i;
  } else {
    row = (int)e;
    b = row_sequence(a.row_offsets, a.batch, row);
    if (!rows_of(a, b, n0, n, from) || row < n0 || row >= n0 + n) return;
    slot = from + (row - n0);
  }
  const int P = a.page_size;
  const int pg = __ldg(a.page_table + (int64_t)b * a.max_pages + slot / P);
  const bool page_ok = pg >= 0 && pg < a.num_pages;
  if (!page_ok) flag(a.status, DS_DEV_BAD_PAGE);
  const int t = unit & 1, h = unit >> 1, g = lane % NG;
  uint16_t* x = a.rows[t] + (int64_t)row * a.row_stride[t] + h * D + g * kKv4Group;
  uint8_t* blk = a.cache[t] + ((int64_t)pg * a.num_kv_heads + h) * DS_KV4_BLOCK_BYTES(P, D);
  const int off = slot % P;
  uint8_t* cp = blk + off * kv4_code_bytes(D) + g * 8;
  uint8_t* sp = blk + P * kv4_code_bytes(D) + off * kv4_scale_bytes(D) + g;
  if constexpr (WRITE) {
    if (!page_ok) return;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(x));
    const uint4 hi = __ldg(reinterpret_cast<const uint4*>(x) + 1);
    const uint32_t r[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = __uint_as_float(r[i] << 16) * a.mult[t];
      y[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u) * a.mult[t];
    }
    uint32_t sb;
    uint2 codes;
    bool bad;
    kv4_quantise16(y, sb, codes, bad);
    if (bad) flag(a.status, DS_DEV_BAD_VALUE);
    *reinterpret_cast<uint2*>(cp) = codes;
    *sp = (uint8_t)sb;
  } else {
    uint32_t r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (page_ok) {
      const uint2 codes = __ldg(reinterpret_cast<const uint2*>(cp));
      const uint32_t s2 = kv4_scales_f16(__ldg(sp));
      const float s = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu))) * a.mult[t];
      const uint32_t cw[2] = {codes.x, codes.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[4];
        kv4_codes_f16(cw[k], v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[4 * k + i]) : "f"(f.y * s), "f"(f.x * s));
        }
      }
    }
    reinterpret_cast<uint4*>(x)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(x)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

template <bool WRITE>
static cudaError_t launch_rows(const ds_kv4_rows_args& g, cudaStream_t stream) {
  Kv4RowsKArgs a;
  a.rows[0] = static_cast<uint16_t*>(g.k_rows);
  a.rows[1] = static_cast<uint16_t*>(g.v_rows);
  a.cache[0] = static_cast<uint8_t*>(g.k_cache);
  a.cache[1] = static_cast<uint8_t*>(g.v_cache);
  a.row_stride[0] = g.k_row_stride;
  a.row_stride[1] = g.v_row_stride;
  a.page_table = g.page_table;
  a.from_lens = g.from_lens;
  a.row_offsets = g.row_offsets;
  a.path = g.path;
  a.n_accepted = g.n_accepted;
  a.batch = g.batch;
  a.n_rows = g.n_rows;
  a.num_kv_heads = g.num_kv_heads;
  a.page_size = g.page_size;
  a.num_pages = g.num_pages;
  a.max_pages = g.max_pages;
  a.mult[0] = ldexpf(1.f, WRITE ? -g.k_exp : g.k_exp);
  a.mult[1] = ldexpf(1.f, WRITE ? -g.v_exp : g.v_exp);
  a.new_lens = g.new_lens;
  a.status = static_cast<uint32_t*>(g.workspace);
  const int rw = 32 / (g.head_dim / kKv4Group);
  const int64_t total = g.path ? (int64_t)g.batch * DS_MAX_TREE_NODES : g.n_rows;
  const int64_t warps = (total + rw - 1) / rw * 2 * g.num_kv_heads;
  const dim3 grid((unsigned)std::max<int64_t>(1, (warps + 7) / 8));
  if (g.head_dim == 128)
    return launch_dependent(kv4_rows<128, WRITE>, grid, dim3(256), 0, stream, a);
  return launch_dependent(kv4_rows<64, WRITE>, grid, dim3(256), 0, stream, a);
}

cudaError_t launch_kv4_write(const ds_kv4_rows_args& g, cudaStream_t stream) {
  return launch_rows<true>(g, stream);
}

cudaError_t launch_kv4_read(const ds_kv4_rows_args& g, cudaStream_t stream) {
  return launch_rows<false>(g, stream);
}

}  // namespace ds
