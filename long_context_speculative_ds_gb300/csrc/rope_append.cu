// Rotation by position of queries and keys, and the new tokens' keys and
// values into the draft's cache (include/ds.h, ds_rope_append).
//
// (x, y) -> m (x cos a - y sin a, x sin a + y cos a) for every pair, a =
// position * frequency; float32 with one rounding.
//
// Bound by memory when there are many rows, by latency when there are few: with
// 32 + 8 heads of 128, 32,768 rows rotated and written into a paged cache take
// 123 us, 6.6 TB/s of the 6.8 that a copy reaches; the gradient of 8,191 rows
// 29 us (5.7 TB/s); one row, or one of each of 96 sequences, 3.0 us in a graph
// (4.3 called one by one, the host's time).
//
// D / 16 lanes hold one head, each two vectors of eight values that make up
// whole pairs: the eight from 8l and their partners r/2 on (half), or the
// sixteen from 16l (interleaved); heads' values past r the same way, unturned.
// A warp takes a row and works on four groups of heads at a time, the first
// ones' loads on their way while it forms the sines and cosines; these stay in
// registers for all heads (read from shared memory for each head they conflict
// in its banks four ways: 131 and 40 us).  With few rows a row's heads are
// spread over more warps.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "dev_common.cuh"
#include "draft_cache.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace ds {

struct RopeKArgs {
  const uint16_t* x[3];           // q, k, v
  int64_t stride[3];
  uint16_t* out[2];               // q, k (NULL: none)
  int64_t out_stride[2];
  const int32_t* positions;
  const int32_t* from_lens;
  const int32_t* row_offsets;
  int32_t* slot_positions;
  float* slot_weights;
  int32_t* new_lens;
  uint32_t* status;
  DraftCache cache;
  int64_t slot_stride;
  int32_t n_rows, batch, hq, hkv, heads;   // heads = query + key (+ value) heads
  int32_t slot_heads, rotary, write;       // write: there is a cache
  int32_t per;                    // head groups of a warp
  uint64_t heads_magic;           // 2^32 / heads, rounded up
  int32_t row_blocks;             // the blocks behind these look at the sequences
  float magnitude, sin_sign;
  unsigned long long turn[64];    // frequency j as a 64-bit fraction of a turn
};

constexpr int kRopeWarps = 4;             // warps of a block
constexpr int kRopeBatch = 4;             // head groups of a warp, their loads together
// Rows of few heads go several to a warp, when there are enough of them to fill
// the machine all the same: up to 12 heads from kManyRows on, up to 20 of 64 or 16
// of 128 from kMoreRows on, four rows, and eight from kMostRows on (of 1,536 values
// and more from twice that).
constexpr int kFewHeads = 12, kManyRows = 16384, kMoreRows = 32768, kMostRows = 65536;

// A row's sequence is where a binary search of the offsets ends, the number's bits
// from the highest down: a bit is set when the offset of the number with it lies at
// or below the row.  Whatever the offsets are, the search finds sequence b for each
// of its rows [n0, n1) just when, of the offsets on the way to b, those that set a
// bit lie at or below n0 and the others at or above n1.  Offsets that decrease
// somewhere can put that in doubt; such a sequence is left out like one whose own
// offsets are wrong.
struct Owner {
  int b, low, high;               // sequence; the largest that set a bit, the least that did not
};
DS_DEV bool sure(const Owner& o, int n0, int n1) { return o.low <= n0 && o.high >= n1; }

DS_DEV Owner row_owner(const int32_t* offs, int batch, int row) {
  Owner o = {0, INT_MIN, INT_MAX};
  for (int bit = 1 << (31 - __clz(max(batch - 1, 1))); bit > 0; bit >>= 1) {
    if (o.b + bit >= batch) continue;
    const int at = offs[o.b + bit];
    if (at <= row) {
      o.b += bit;
      o.low = max(o.low, at);
    } else {
      o.high = min(o.high, at);
    }
  }
  return o;
}
// Bit i's part of the way to sequence b.
DS_DEV Owner way_to(const int32_t* offs, int batch, int b, int i) {
  const uint32_t node = ((uint32_t)b >> i | 1u) << i;
  const bool set = (uint32_t)b >> i & 1, there = node < (uint32_t)batch;
  const int at = there ? offs[node] : 0;
  return {b, set ? at : INT_MIN, there && !set ? at : INT_MAX};
}
// The sequence before the first of 32 offsets at a time that lies above the row, by
// all lanes of a warp: where the search ends too when offsets increase.
DS_DEV int guess_owner(const int32_t* offs, int batch, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, i < n && offs[lo + min(i, n - 1)] <= row);
    const int k = max(__ffs(~at) - 2, at == ~0u ? 31 : 0);   // last of the run from lane 0
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Rows [n0, n0 + n) and first slot of sequence b; false when they cannot be used
// (whatever the other offsets are).
DS_DEV bool rope_rows_of(const RopeKArgs& a, int b, int& n0, int& n, int& from) {
  n0 = a.row_offsets[b];
  const int n1 = a.row_offsets[b + 1];
  from = a.from_lens[b];
  n = n1 - n0;
  return n0 >= 0 && n1 >= n0 && n1 <= a.n_rows && from >= 0 && (int64_t)from + n <= a.cache.slots;
}

template <bool BF>
DS_DEV float2 unpack2(uint32_t w) {
  if constexpr (BF)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF>
DS_DEV uint32_t pack2(float lo, float hi) {
  return BF ? ptx::pack_bf16x2(lo, hi) : ptx::pack_f16x2(lo, hi);
}

// A lane's eight pairs of a head: (u, v) value by value (half), or neighbours
// in u and in v; cs: their cosines and sines, two pairs an entry.
template <bool BF, bool HALVES>
DS_DEV void turn(uint4& u, uint4& v, const float4 (&cs)[4]) {
  uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF>(uw[i]), y = unpack2<BF>(vw[i]);
    if constexpr (HALVES) {
      const float4 c = cs[i];
      uw[i] = pack2<BF>(x.x * c.x - y.x * c.y, x.y * c.z - y.y * c.w);
      vw[i] = pack2<BF>(x.x * c.y + y.x * c.x, x.y * c.w + y.y * c.z);
    } else {
      const float cx = i & 1 ? cs[i / 2].z : cs[i / 2].x, sx = i & 1 ? cs[i / 2].w : cs[i / 2].y;
      const float cy = i & 1 ? cs[2 + i / 2].z : cs[2 + i / 2].x;
      const float sy = i & 1 ? cs[2 + i / 2].w : cs[2 + i / 2].y;
      uw[i] = pack2<BF>(x.x * cx - x.y * sx, x.x * sx + x.y * cx);
      vw[i] = pack2<BF>(y.x * cy - y.y * sy, y.x * sy + y.y * cy);
    }
  }
  u = make_uint4(uw[0], uw[1], uw[2], uw[3]);
  v = make_uint4(vw[0], vw[1], vw[2], vw[3]);
}

// Kind (query, key, value) and number of a row's head hh.
DS_DEV int head_of(const RopeKArgs& a, int hh, int& h) {
  const int ty = hh < a.hq ? 0 : hh < a.hq + a.hkv ? 1 : 2;
  h = hh - (ty > 0 ? a.hq : 0) - (ty > 1 ? a.hkv : 0);
  return ty;
}
DS_DEV const uint16_t* head_row(const RopeKArgs& a, int ty, int64_t row, int off) {
  return (ty == 0 ? a.x[0] : ty == 1 ? a.x[1] : a.x[2]) +
         row * (ty == 0 ? a.stride[0] : ty == 1 ? a.stride[1] : a.stride[2]) + off;
}
// A lane's two vectors of a head to where they belong; at: the slot's place in
// the pools, -1 for none.
template <int D>
DS_DEV void put_head(const RopeKArgs& a, int ty, int64_t row, int h, int64_t at, const uint4& u,
                     const uint4& v, int e0, int e1) {
  uint16_t* o = ty == 0 ? a.out[0] : ty == 1 ? a.out[1] : nullptr;
  if (o) {
    o += row * (ty == 0 ? a.out_stride[0] : a.out_stride[1]) + (int64_t)h * D;
    *reinterpret_cast<uint4*>(o + e0) = u;
    *reinterpret_cast<uint4*>(o + e1) = v;
  }
  if (ty > 0 && at >= 0) {
    o = (ty == 1 ? a.cache.pool[0] : a.cache.pool[1]) + at + (int64_t)h * a.cache.head_stride;
    *reinterpret_cast<uint4*>(o + e0) = u;
    *reinterpret_cast<uint4*>(o + e1) = v;
  }
}
// Cosine and sine at a position of a frequency, times the magnitude.  position *
// frequency wraps modulo one turn in 64 bits; its upper half, read as a signed
// number, is the angle in units of pi / 2^31.
DS_DEV float2 turn_of(const RopeKArgs& a, int pos, unsigned long long frequency) {
  const unsigned long long t = (unsigned long long)pos * frequency;
  float sn, c;
  sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &sn, &c);
  return make_float2(c * a.magnitude, sn * a.magnitude * a.sin_sign);
}
// The last blocks have a thread per sequence, which checks its offsets and
// length even when no row is mapped to it, and writes the new length.
DS_DEV void check_sequences(const RopeKArgs& a) {
  const int b = (blockIdx.x - a.row_blocks) * 32 * kRopeWarps + threadIdx.x;
  if (b >= a.batch || blockIdx.y > 0) return;
  int n0, n, from;
  bool usable = rope_rows_of(a, b, n0, n, from);
  if (!usable) flag(a.status, DS_DEV_BAD_LENGTH);
  bool all_found = true;
#pragma unroll 4
  for (int i = 0; (a.batch - 1) >> i > 0; ++i)
    all_found &= sure(way_to(a.row_offsets, a.batch, b, i), n0, n0 + n);
  if (usable && n > 0 && !all_found) {
    // left out (rows whose slots have neither a page nor a position or weight to be
    // noted go nowhere and count all the same)
    flag(a.status, DS_DEV_BAD_LENGTH);
    const int64_t page = a.cache.page_size;
    usable = a.cache.page_table != nullptr && a.slot_heads == 0;
    for (int64_t t = from; usable && t < (int64_t)from + n; t = (t / page + 1) * page)
      usable = slot_page(a.cache, b, (int)t) < 0;
    if (usable) flag(a.status, DS_DEV_BAD_PAGE);
  }
  if (a.new_lens) a.new_lens[b] = usable ? from + n : from;
}

template <int D, bool BF, bool HALVES>
__global__ void __launch_bounds__(32 * kRopeWarps, 7) rope_append(const RopeKArgs a) {
  constexpr int LPH = D / 16;             // lanes of a head
  constexpr int HPW = 32 / LPH;           // heads of a warp at a time
  __shared__ __align__(16) float2 s_cs[kRopeWarps][D / 2];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= a.row_blocks) {
    check_sequences(a);
    return;
  }
  const int64_t row64 = (int64_t)blockIdx.x * kRopeWarps + warp;
  if (row64 >= a.n_rows) return;
  const int row = (int)row64;
  const int groups = (a.heads + HPW - 1) / HPW;
  const int g0 = blockIdx.y * a.per, g1 = min(groups, g0 + a.per);
  if (g0 >= g1) return;
  const int l = lane % LPH, sub = lane / LPH;
  const bool turned = 16 * l < a.rotary;
  // the lane's two vectors of a head
  const int e0 = !turned || !HALVES ? 16 * l : 8 * l;
  const int e1 = !turned || !HALVES ? 16 * l + 8 : 8 * l + a.rotary / 2;
  uint4 u[kRopeBatch], v[kRopeBatch];
  auto load = [&](int gb) {
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int hh = (gb + k) * HPW + sub;
      if (gb + k >= g1 || hh >= a.heads) continue;
      int h;
      const int ty = head_of(a, hh, h);
      // plain loads: with q_out = q the same bytes are written below
      const uint16_t* p = head_row(a, ty, row, h * D);
      u[k] = *reinterpret_cast<const uint4*>(p + e0);
      v[k] = *reinterpret_cast<const uint4*>(p + e1);
    }
  };
  const int pos = a.positions[row];
  load(g0);                               // beside what the position asks for
  if (pos < 0) {
    if (lane == 0) flag(a.status, DS_DEV_BAD_LENGTH);
    return;
  }
  int64_t at = -1;                        // the slot's place in the pools
  if (a.write) {
    int b = guess_owner(a.row_offsets, a.batch, row), n0, n, from;
    bool use = rope_rows_of(a, b, n0, n, from);
    const Owner way = way_to(a.row_offsets, a.batch, b, lane);
    if (!__all_sync(0xffffffffu, row >= n0 && row < n0 + n && sure(way, n0, n0 + n))) {
      const Owner o = row_owner(a.row_offsets, a.batch, row);
      b = o.b;
      use = rope_rows_of(a, b, n0, n, from) && row >= n0 && row < n0 + n && sure(o, n0, n0 + n);
    }
    if (!use) return;
    const int slot = from + (row - n0);
    const int pg = slot_page(a.cache, b, slot);
    if (pg >= 0) at = slot_at(a.cache, pg, slot);
    else if (lane == 0) flag(a.status, DS_DEV_BAD_PAGE);
    if (blockIdx.y == 0)
      for (int h = lane; h < a.slot_heads; h += 32) {
        const int64_t i = ((int64_t)b * a.slot_heads + h) * a.slot_stride + slot;
        if (a.slot_positions) a.slot_positions[i] = pos;
        if (a.slot_weights) a.slot_weights[i] = 0.f;
      }
  }
  float2* const cs = s_cs[warp];
  for (int j = lane; j < a.rotary / 2; j += 32) cs[j] = turn_of(a, pos, a.turn[j]);
  __syncwarp();
  float4 rot[4];                          // of this lane's pairs, for all heads
#pragma unroll
  for (int i = 0; i < 4; ++i)
    rot[i] = turned ? *reinterpret_cast<const float4*>(&cs[8 * l + 2 * i])
                    : make_float4(1.f, 0.f, 1.f, 0.f);
  for (int gb = g0; gb < g1; gb += kRopeBatch) {
    if (gb > g0) load(gb);
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int hh = (gb + k) * HPW + sub;
      if (gb + k >= g1 || hh >= a.heads) continue;
      int h;
      const int ty = head_of(a, hh, h);
      if (turned && ty < 2) turn<BF, HALVES>(u[k], v[k], rot);
      put_head<D>(a, ty, row, h, at, u[k], v[k], e0, e1);
    }
  }
}

// The same for rows of few heads: a warp takes R rows and their heads one behind
// the other, so that a short last group of heads and what a row costs by itself
// are shared; most of that is the table of frequencies, which lies in constant
// memory, one address a cycle, and is read once for all rows here.  A lane looks
// up a row; cosines and sines are kept by row, in an order in which eight lanes
// read 128 bytes.  262,144 rows of 8 + 1 heads of 64: 178 us row by row, 125 by
// fours, 104 by eights (floor 89); 16,384 rows 12.4, 10.6, 12.0; of 4,096 rows one
// at a time is faster (4.7, 5.5, 7.2).  Rows of 12 + 2 heads of 64: 48,000 39 and 34
// (of 128 66 and 63), but 17,000 of 12 + 4 13.3 and 13.9, 48,000 of 20 + 4 50 and
// 51.5 (of 16 + 4 of 128 81 and 83).  70,000 rows of 8 + 4 + 4 heads of 128 into a
// cache 95 by fours, 100 by eights; 66,000 of 8 + 1 of 64 35 and 32.  By eights the first heads'
// loads go out before the rows' places are known (730,000 rows of 2 + 1 heads into
// a cache 176 us instead of 183); by fours that took longer (16,384 rows of 4 + 1
// heads of 128 into 16 sequences 16.4 instead of 15.4).  What the search sees on its
// way is kept for the check of its sequence: 720,000 rows of 2 + 1 heads into 16
// sequences 161 us instead of 159, 20,000 of 1 + 1 into as many 12.4 instead of 12.1.
template <int D, bool BF, bool HALVES, int R>
__global__ void __launch_bounds__(32 * kRopeWarps, 6) rope_few_heads(const RopeKArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  constexpr bool kEarly = R == 8;
  __shared__ __align__(16) float2 s_cs[kRopeWarps][R][D / 2];
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= a.row_blocks) {
    check_sequences(a);
    return;
  }
  const int64_t row0 = ((int64_t)blockIdx.x * kRopeWarps + warp) * R;
  if (row0 >= a.n_rows) return;
  const int rows = (int)min((int64_t)R, a.n_rows - row0);
  const int l = lane % LPH, sub = lane / LPH;
  const bool turned = 16 * l < a.rotary;
  const int e0 = !turned || !HALVES ? 16 * l : 8 * l;
  const int e1 = !turned || !HALVES ? 16 * l + 8 : 8 * l + a.rotary / 2;
  const int items = rows * a.heads;
  uint4 u[kRopeBatch], v[kRopeBatch];
  int r[kRopeBatch], hh[kRopeBatch];
  auto load = [&](int g0) {
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int e = min(g0 + k * HPW + sub, items - 1);
      r[k] = (int)(e * a.heads_magic >> 32);
      hh[k] = g0 + k * HPW + sub < items ? e - r[k] * a.heads : -1;
      if (hh[k] < 0) continue;
      int h;
      const int ty = head_of(a, hh[k], h);
      const uint16_t* p = head_row(a, ty, row0 + r[k], h * D);
      u[k] = *reinterpret_cast<const uint4*>(p + e0);
      v[k] = *reinterpret_cast<const uint4*>(p + e1);
    }
  };
  // ---- lane r: row r's position and place
  int pos = 0;
  int64_t at = -1;
  bool use = false;
  if (lane < rows) pos = a.positions[row0 + lane];
  if (kEarly) load(0);                    // beside what the positions ask for
  if (lane < rows) {
    const int row = (int)row0 + lane;
    use = pos >= 0;
    if (!use) flag(a.status, DS_DEV_BAD_LENGTH);
    if (use && a.write) {
      const Owner o = row_owner(a.row_offsets, a.batch, row);
      int n0, n, from;
      use = rope_rows_of(a, o.b, n0, n, from) && row >= n0 && row < n0 + n && sure(o, n0, n0 + n);
      if (use) {
        const int slot = from + (row - n0), pg = slot_page(a.cache, o.b, slot);
        if (pg >= 0) at = slot_at(a.cache, pg, slot);
        else flag(a.status, DS_DEV_BAD_PAGE);
        for (int h = 0; h < a.slot_heads; ++h) {
          const int64_t i = ((int64_t)o.b * a.slot_heads + h) * a.slot_stride + slot;
          if (a.slot_positions) a.slot_positions[i] = pos;
          if (a.slot_weights) a.slot_weights[i] = 0.f;
        }
      }
    }
  }
  const uint32_t used = __ballot_sync(0xffffffffu, use);
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {      // (a lane's frequency is read once for all rows)
    const int j = lane + 32 * k, to = (j % 8 / 2 * LPH + j / 8) * 2 + j % 2;
    const unsigned long long f = a.turn[j];
#pragma unroll 2
    for (int r = 0; r < rows; ++r)
      s_cs[warp][r][to] = turn_of(a, __shfl_sync(0xffffffffu, pos, r), f);
  }
  __syncwarp();
  for (int g0 = 0; g0 < items; g0 += HPW * kRopeBatch) {
    if (g0 > 0 || !kEarly) load(g0);
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int64_t to = __shfl_sync(0xffffffffu, at, r[k]);
      if (hh[k] < 0 || !(used >> r[k] & 1)) continue;
      int h;
      const int ty = head_of(a, hh[k], h);
      if (turned && ty < 2) {
        float4 rot[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          rot[i] = *reinterpret_cast<const float4*>(&s_cs[warp][r[k]][(i * LPH + l) * 2]);
        turn<BF, HALVES>(u[k], v[k], rot);
      }
      put_head<D>(a, ty, row0 + r[k], h, to, u[k], v[k], e0, e1);
    }
  }
}

cudaError_t launch_rope_append(const ds_rope_args& g, cudaStream_t stream) {
  RopeKArgs a = {};
  const bool cache = g.k_cache != nullptr;
  a.x[0] = static_cast<const uint16_t*>(g.q);
  a.x[1] = static_cast<const uint16_t*>(g.k);
  a.x[2] = static_cast<const uint16_t*>(g.v);
  a.stride[0] = g.q_row_stride;
  a.stride[1] = g.k_row_stride;
  a.stride[2] = g.v_row_stride;
  a.out[0] = static_cast<uint16_t*>(g.q_out);
  a.out[1] = static_cast<uint16_t*>(g.k_out);
  a.out_stride[0] = g.q_out_row_stride;
  a.out_stride[1] = g.k_out_row_stride;
  a.positions = g.positions;
  a.n_rows = g.n_rows;
  a.hq = g.num_q_heads;
  a.hkv = g.num_kv_heads;
  a.heads = a.hq + a.hkv * (cache ? 2 : 1);
  a.rotary = g.rotary_dim ? g.rotary_dim : g.head_dim;
  a.write = cache;
  if (cache) {
    a.cache = draft_cache(g);
    a.from_lens = g.from_lens;
    a.row_offsets = g.row_offsets;
    a.batch = g.batch;
    a.slot_positions = g.slot_positions;
    a.slot_weights = g.slot_weights;
    a.slot_heads = g.slot_positions || g.slot_weights ? g.slot_heads : 0;
    a.slot_stride = g.slot_stride;
    a.new_lens = g.new_lens;
  }
  a.status = static_cast<uint32_t*>(g.workspace);
  a.magnitude = g.magnitude;
  a.sin_sign = g.inverse ? -1.f : 1.f;
  // a double's 53 bits leave each frequency (at most a radian in use) off by
  // less than 2^-52 of a turn, and the angle, at positions below 2^31, by
  // less than 2^-21 of one; at 2^17 by less than 2^-35
  // (base^(-2j/r) as a product of two powers: sixteen calls of pow, not 64)
  constexpr double kTurns = 1.0 / 6.283185307179586;   // of a radian
  double lo[8], hi[8];
  if (!g.inv_freq)
    for (int k = 0; k < 8; ++k) {
      lo[k] = std::pow((double)g.rope_base, -2.0 * k / a.rotary);
      hi[k] = std::pow((double)g.rope_base, -16.0 * k / a.rotary) * kTurns;
    }
  for (int j = 0; j < a.rotary / 2; ++j) {
    const double turns = g.inv_freq ? g.inv_freq[j] * kTurns : lo[j & 7] * hi[j >> 3];
    const double frac = turns - std::floor(turns);   // whole turns drop out
    a.turn[j] = frac < 1.0 ? (unsigned long long)(frac * 18446744073709551616.0) : 0ull;
  }
  a.heads_magic = ((1ull << 32) + a.heads - 1) / a.heads;
  const int hpw = 32 / (g.head_dim / 16), groups = (a.heads + hpw - 1) / hpw;
  const int slices = (int)std::max<int64_t>(
      1, std::min<int64_t>(groups, 152 * 24 / std::max(1, g.n_rows)));
  a.per = (groups + slices - 1) / slices;
  const int few_heads = g.n_rows < kMoreRows ? kFewHeads : g.head_dim == 64 ? 20 : 16;
  const bool few = a.heads <= few_heads && g.n_rows >= kManyRows;
  const int most = a.heads * g.head_dim >= 1536 ? 2 * kMostRows : kMostRows;
  const int64_t each = !few ? 1 : g.n_rows >= most ? 8 : 4;   // rows of a warp
  const int64_t rows = kRopeWarps * each;                     // of a block
  a.row_blocks = (int)((g.n_rows + rows - 1) / rows);
  const dim3 grid((unsigned)(a.row_blocks + (a.batch + 32 * kRopeWarps - 1) / (32 * kRopeWarps)),
                  few ? 1u : (unsigned)((groups + a.per - 1) / a.per));
  const dim3 block(32 * kRopeWarps);
  const bool bf = g.dtype == DS_KV_BF16, halves = g.layout == DS_ROPE_HALF;
  auto go = [&](void (*k)(const RopeKArgs), dim3 blocks) {
    return launch_dependent(k, blocks, block, 0, stream, a);
  };
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (each == 8)
      return bf ? (halves ? go(rope_few_heads<D, true, true, 8>, grid)
                          : go(rope_few_heads<D, true, false, 8>, grid))
                : (halves ? go(rope_few_heads<D, false, true, 8>, grid)
                          : go(rope_few_heads<D, false, false, 8>, grid));
    if (each == 4)
      return bf ? (halves ? go(rope_few_heads<D, true, true, 4>, grid)
                          : go(rope_few_heads<D, true, false, 4>, grid))
                : (halves ? go(rope_few_heads<D, false, true, 4>, grid)
                          : go(rope_few_heads<D, false, false, 4>, grid));
    return bf ? (halves ? go(rope_append<D, true, true>, grid)
                        : go(rope_append<D, true, false>, grid))
              : (halves ? go(rope_append<D, false, true>, grid)
                        : go(rope_append<D, false, false>, grid));
  };
  return g.head_dim == 128 ? pick(std::integral_constant<int, 128>())
                           : pick(std::integral_constant<int, 64>());
}

}  // namespace ds
