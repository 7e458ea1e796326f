// The launches of the draft cache's entry points over the runtime of two
// devices of two_devices.cpp: the shared memory they ask for is allowed on the
// device at hand, and their grids have sizes that a grid can have, from one
// sequence to 65,536.
#define main two_devices_main
#include "two_devices.cpp"
#undef main

static ds_status rope(int rows, int batch, int hq, int hkv, int d, bool paged) {
  ds_rope_args a;
  ds_rope_args_default(&a);
  a.q = at<void>(4096); a.k = at<void>(4096); a.v = at<void>(4096);
  a.q_out = at<void>(8192);
  a.q_row_stride = a.k_row_stride = a.v_row_stride = a.q_out_row_stride = 1 << 24;
  a.positions = at<int32_t>(64); a.n_rows = rows; a.num_q_heads = hq; a.num_kv_heads = hkv;
  a.head_dim = d; a.rope_base = 1e4f; a.k_cache = at<void>(4096); a.v_cache = at<void>(4096);
  a.page_table = paged ? at<int32_t>(64) : nullptr; a.from_lens = at<int32_t>(64);
  a.row_offsets = at<int32_t>(64); a.batch = batch; a.page_size = 16; a.num_pages = 65536;
  a.max_pages = 64; a.new_lens = at<int32_t>(128); a.workspace = at<void>(65536);
  a.workspace_bytes = 256;
  return ds_rope_append(&a, nullptr);
}

static ds_status decode(int batch, int hq, int hkv, int d, int page, bool paged, int slot_heads,
                        int max_pages) {
  ds_decode_args a;
  ds_decode_args_default(&a);
  a.q = at<void>(4096); a.q_row_stride = (int64_t)hq * d; a.k_cache = at<void>(4096);
  a.v_cache = at<void>(4096); a.page_table = paged ? at<int32_t>(64) : nullptr;
  a.lens = at<int32_t>(64); a.batch = batch; a.num_q_heads = hq; a.num_kv_heads = hkv;
  a.head_dim = d; a.page_size = page; a.num_pages = 65536; a.max_pages = max_pages;
  a.out = at<void>(4096); a.num_sms = 152;
  if (slot_heads) {
    a.weights_out = at<float>(64); a.slot_heads = slot_heads; a.slot_stride = (int64_t)1 << 30;
  }
  a.workspace = at<void>(65536); a.workspace_bytes = (size_t)1 << 60;
  return ds_decode_attn(&a, nullptr);
}

static ds_status evict(int batch, int hkv, int slot_heads, int d, int page, bool paged,
                       int max_pages, int budget) {
  ds_evict_args a;
  ds_evict_args_default(&a);
  a.k_cache = at<void>(4096); a.v_cache = at<void>(4096);
  a.page_table = paged ? at<int32_t>(64) : nullptr; a.lens = at<int32_t>(64); a.batch = batch;
  a.num_kv_heads = hkv; a.head_dim = d; a.page_size = page; a.num_pages = 65536;
  a.max_pages = max_pages; a.slot_heads = slot_heads; a.slot_stride = (int64_t)1 << 30;
  a.weights = at<float>(64); a.positions = at<int32_t>(64); a.next_positions = at<int32_t>(64);
  a.new_lens = at<int32_t>(128); a.budget = budget; a.workspace = at<void>(65536);
  a.workspace_bytes = (size_t)1 << 60;
  return ds_cache_evict(&a, nullptr);
}

int main() {
  int bad = 0, calls = 0;
  auto check = [&](const char* what, int x, ds_status st) {
    ++calls;
    if (st == DS_OK) return;
    ++bad;
    std::printf("device %d: %s %d: %s\n", g_device, what, x, ds_last_error());
  };
  for (int turn = 0; turn < 3; ++turn) {
    g_device = turn & 1;
    if (turn == 2) g_allowed.clear();          // a context torn down and made again
    for (int d : {64, 128})
      for (int batch : {1, 2, 33, 4097, 65536})
        for (int hkv : {1, 8, 40}) {
          const bool small = batch > 1638;     // (batch * heads at most 65,536)
          for (int rows : {0, 1, 31, 65536, 0x7fffffff})
            check("rope rows", rows, rope(rows, batch, 4 * hkv, hkv, d, batch & 1));
          for (int group : {1, 4, 16})
            for (int w : {0, 1, hkv})
              for (int pages : {1, 64, 1 << 26})
                check("decode batch", batch,
                      decode(batch, group * hkv, hkv, d, 16, pages > 1, w, pages));
          for (int w : {1, hkv})
            for (int pages : {1, 64, 1000, 1 << 26})
              for (int budget : {1, 100, 1 << 29})
                if (!small || w == 1)
                  check("evict batch", batch,
                        evict(batch, hkv, w, d, 16, pages > 1, pages, budget));
        }
  }
  std::printf("%d calls, %d launches above 48 KB, %d refused\n", calls, g_large, bad);
  return bad || g_large < 100;
}
