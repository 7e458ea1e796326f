// Where a slot of the draft's cache lies (include/ds.h, "The draft's cache"),
// shared by the kernels that write, read and move its rows.  These kernels start
// before the one in front of them has ended (and wait for it), so what that one
// may write (lengths, tables, sums) is read with ordinary loads, not as data that
// stays the same while they run.
#pragma once

#include <stdint.h>

#include "dev_common.cuh"

namespace ds {

struct DraftCache {
  uint16_t* pool[2];              // K, V
  const int32_t* page_table;      // NULL: compact, sequence b is page b
  int32_t num_kv_heads, page_size, page_shift, num_pages, max_pages;
  int64_t slots;                  // of a sequence
  int64_t page_stride, slot_stride, head_stride;   // elements
};

template <typename Args>
DraftCache draft_cache(const Args& g) {
  DraftCache c;
  c.pool[0] = static_cast<uint16_t*>(const_cast<void*>((const void*)g.k_cache));
  c.pool[1] = static_cast<uint16_t*>(const_cast<void*>((const void*)g.v_cache));
  c.page_table = g.page_table;
  c.num_kv_heads = g.num_kv_heads;
  c.page_size = g.page_size;
  c.page_shift = g.page_table ? __builtin_ctz((unsigned)g.page_size) : 0;
  c.num_pages = g.num_pages;
  c.max_pages = g.max_pages;
  c.slots = g.page_table ? (int64_t)g.max_pages * g.page_size : g.page_size;
  c.page_stride = (int64_t)g.page_size * g.num_kv_heads * g.head_dim;
  const bool hnd = g.kv_layout == DS_KV_HND;
  c.slot_stride = (int64_t)g.head_dim * (hnd ? 1 : g.num_kv_heads);
  c.head_stride = (int64_t)g.head_dim * (hnd ? g.page_size : 1);
  return c;
}

// Page of a slot of sequence b (0 <= slot < slots); -1 when its id is none.
DS_DEV int slot_page(const DraftCache& c, int b, int slot) {
  if (!c.page_table) return b;
  const int pg = c.page_table[(int64_t)b * c.max_pages + (slot >> c.page_shift)];
  return (uint32_t)pg < (uint32_t)c.num_pages ? pg : -1;
}
// Elements from the pool's start to head 0 of the slot, in page pg.
DS_DEV int64_t slot_at(const DraftCache& c, int pg, int slot) {
  const int off = c.page_table ? slot & (c.page_size - 1) : slot;
  return (int64_t)pg * c.page_stride + (int64_t)off * c.slot_stride;
}

// A length a sequence can have, else 0 and a status bit (told once, by the
// caller that reports).
DS_DEV int checked_len(int n, int64_t slots, uint32_t* status, bool report) {
  if (n >= 0 && n <= slots) return n;
  if (report) flag(status, DS_DEV_BAD_LENGTH);
  return 0;
}

}  // namespace ds
