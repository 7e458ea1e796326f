// Rows of K and V into the paged 4-bit cache and back (include/ds.h,
// ds_kv4_write and ds_kv4_read).
//
// Bound by memory when there are many rows, by latency when there are few:
// with 8 heads of 128, 131,072 rows read back in 108.7 us, 6.3 TB/s of the
// 6.70 a copy reaches; a ragged batch of eight prompts (88,518 rows) is written
// and read back in 158 us, 5.9 TB/s (writing alone was 128 us before the
// quantiser worked in packed maxima and products with a reciprocal, 79 after,
// 10 above its bytes: its arithmetic overlaps the loads only in part); 64 rows
// written and read back 5.3 us.  A warp takes a few consecutive rows and walks over (tensor, kv head) units,
// several units' loads on their way at once; with few rows the units of a row
// are spread over more warps.  Which sequence a row belongs to, its slot and
// its page are looked up once per lane, for all units.
//
// Writing, a lane holds one scale group: 16 channels, whose maximum, scale and
// codes are its own.  A warp covers 4 rows of one head (8 at head_dim 64),
// whose slots follow each other in the page block: its codes are one run of
// 256 bytes and its scales one of 32.  Reading, a lane makes 8 channels (one
// 16-byte store), so that a store instruction covers whole sectors.
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
  int32_t batch, n_rows, num_kv_heads, page_size, page_shift, num_pages, max_pages;
  int32_t slices;                 // warps that share a row group's units
  int32_t row_blocks;             // the blocks behind these look at the sequences
  float mult[2];                  // write: 2^-exp, read: 2^exp
  int32_t* new_lens;
  uint32_t* status;
};

constexpr int64_t kRowWarps = 152 * 32;

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
  constexpr int CH = WRITE ? 16 : 8;      // channels of a lane
  constexpr int LPH = D / CH;             // lanes of a head
  constexpr int RW = 32 / LPH;            // rows of a warp
  constexpr int NB = WRITE ? 3 : 8;       // units on their way at once
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  // The last blocks have a thread per sequence, which checks its offsets and
  // length even when no row is mapped to it (offsets that decrease or leave
  // the rows), and writes the length that follows.
  if ((int)blockIdx.x >= a.row_blocks) {
    const int b = (blockIdx.x - a.row_blocks) * 256 + threadIdx.x;
    if (b >= a.batch) return;
    int n0, n, from, add = 0;
    const bool usable = rows_of(a, b, n0, n, from);
    if (WRITE && a.new_lens) {
      if (usable) {
        add = n;
        if (a.path && n > 0) {
          const int acc = __ldg(a.n_accepted + b);
          add = 1 + (path_ok(a, b, n, acc) ? acc : 0);
        }
      }
      a.new_lens[b] = from + add;
    }
    return;
  }
  // with a path, "rows" are the path's entries: DS_MAX_TREE_NODES a sequence
  const int total = a.path ? a.batch * DS_MAX_TREE_NODES : a.n_rows;
  const int64_t e = w / a.slices * RW + lane / LPH;
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
  const int P = a.page_size, off = slot & (P - 1);
  const int pg = __ldg(a.page_table + (int64_t)b * a.max_pages + (slot >> a.page_shift));
  const bool page_ok = (uint32_t)pg < (uint32_t)a.num_pages;
  if (!page_ok) flag(a.status, DS_DEV_BAD_PAGE);
  if (WRITE && !page_ok) return;
  const int g = lane % LPH;
  const int blk = DS_KV4_BLOCK_BYTES(P, D);
  // this lane's codes and scale in head 0's block, and its channels in the row
  const int64_t page0 = (int64_t)(page_ok ? pg : 0) * a.num_kv_heads * blk;
  const int64_t code0 = page0 + off * kv4_code_bytes(D) + g * (CH / 2);
  const int64_t scale0 =
      page0 + P * kv4_code_bytes(D) + off * kv4_scale_bytes(D) + g * CH / kKv4Group;
  const int units = 2 * a.num_kv_heads;   // unit u: tensor u % 2 of head u / 2
  const int per = (units + a.slices - 1) / a.slices;
  const int u0 = (int)(w % a.slices) * per, u1 = min(units, u0 + per);
  uint16_t* const x0[2] = {a.rows[0] + (int64_t)row * a.row_stride[0] + g * CH,
                           a.rows[1] + (int64_t)row * a.row_stride[1] + g * CH};
  if constexpr (WRITE) {
    bool any_bad = false;
    for (int u = u0; u < u1; u += NB) {
      uint4 lo[NB], hi[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (u + k < u1) {
          const int t = (u + k) & 1, h = (u + k) >> 1;
          const uint4* x = reinterpret_cast<const uint4*>((t ? x0[1] : x0[0]) + h * D);
          lo[k] = __ldg(x);
          hi[k] = __ldg(x + 1);
        }
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (u + k < u1) {
          const int t = (u + k) & 1, h = (u + k) >> 1;
          uint32_t r[8] = {lo[k].x, lo[k].y, lo[k].z, lo[k].w,
                           hi[k].x, hi[k].y, hi[k].z, hi[k].w};
          uint32_t sb;
          uint2 codes;
          bool bad;
          kv4_quantise16(r, t ? a.mult[1] : a.mult[0], sb, codes, bad);
          any_bad |= bad;
          uint8_t* const c = (t ? a.cache[1] : a.cache[0]) + (int64_t)h * blk;
          *reinterpret_cast<uint2*>(c + code0) = codes;
          c[scale0] = (uint8_t)sb;
        }
    }
    if (any_bad) flag(a.status, DS_DEV_BAD_VALUE);
  } else {
    for (int u = u0; u < u1; u += NB) {
      uint32_t codes[NB], sb[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        codes[k] = sb[k] = 0u;
        if (u + k < u1 && page_ok) {
          const int t = (u + k) & 1, h = (u + k) >> 1;
          const uint8_t* const c = (t ? a.cache[1] : a.cache[0]) + (int64_t)h * blk;
          codes[k] = __ldg(reinterpret_cast<const uint32_t*>(c + code0));
          sb[k] = __ldg(c + scale0);
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (u + k < u1) {
          const int t = (u + k) & 1, h = (u + k) >> 1;
          const uint32_t s2 = kv4_scales_f16(sb[k]);
          const float s = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu))) *
                          (t ? a.mult[1] : a.mult[0]);
          uint32_t v[4], r[4];
          kv4_codes_f16(codes[k], v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
            r[i] = ptx::pack_bf16x2(f.x * s, f.y * s);
          }
          *reinterpret_cast<uint4*>((t ? x0[1] : x0[0]) + h * D) =
              make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
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
  a.page_shift = __builtin_ctz((unsigned)g.page_size);
  a.num_pages = g.num_pages;
  a.max_pages = g.max_pages;
  a.mult[0] = ldexpf(1.f, WRITE ? -g.k_exp : g.k_exp);
  a.mult[1] = ldexpf(1.f, WRITE ? -g.v_exp : g.v_exp);
  a.new_lens = g.new_lens;
  a.status = static_cast<uint32_t*>(g.workspace);
  const int rw = 32 / (g.head_dim / (WRITE ? 16 : 8));
  const int64_t total = g.path ? (int64_t)g.batch * DS_MAX_TREE_NODES : g.n_rows;
  const int64_t groups = (total + rw - 1) / rw;
  // enough warps to fill the machine (152 SMs of 32), one unit a warp at least
  const int units = 2 * g.num_kv_heads;
  const int64_t spread = kRowWarps / std::max<int64_t>(1, groups);
  a.slices = (int)std::max<int64_t>(1, std::min<int64_t>(units, spread));
  a.row_blocks = (int)((groups * a.slices + 7) / 8);
  const dim3 grid((unsigned)(a.row_blocks + (g.batch + 255) / 256));
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
