// What a kernel may use of shared memory belongs to the kernel in its context,
// not to a launch: two threads' calls share it.  So a call of the draft cache's
// entry points must never take away what another one, between its permission
// and its launch, relies on.  Over the runtime of two_devices.cpp, which keeps
// account of the permissions: none shrinks, whatever the order of the sizes.
#define main two_devices_main
#include "two_devices.cpp"
#undef main

static ds_status evict(int batch, int hkv, int capacity) {
  ds_evict_args a;
  ds_evict_args_default(&a);
  a.k_cache = at<void>(4096); a.v_cache = at<void>(4096); a.lens = at<int32_t>(64);
  a.batch = batch; a.num_kv_heads = hkv; a.head_dim = 128; a.page_size = capacity;
  a.num_pages = batch; a.slot_heads = hkv; a.slot_stride = capacity; a.weights = at<float>(64);
  a.positions = at<int32_t>(64); a.next_positions = at<int32_t>(64); a.new_lens = at<int32_t>(128);
  a.budget = capacity / 2 + 1; a.workspace = at<void>(65536);
  a.workspace_bytes = (size_t)1 << 60;
  return ds_cache_evict(&a, nullptr);
}

static ds_status decode(int hq, int d, int capacity) {
  ds_decode_args a;
  ds_decode_args_default(&a);
  a.q = at<void>(4096); a.q_row_stride = (int64_t)hq * d; a.k_cache = at<void>(4096);
  a.v_cache = at<void>(4096); a.lens = at<int32_t>(64); a.batch = 2; a.num_q_heads = hq;
  a.num_kv_heads = 1; a.head_dim = d; a.page_size = capacity; a.num_pages = 2;
  a.out = at<void>(4096); a.num_sms = 152; a.workspace = at<void>(65536);
  a.workspace_bytes = (size_t)1 << 60;
  return ds_decode_attn(&a, nullptr);
}

int main() {
  int bad = 0;
  auto held = g_allowed;
  auto check = [&](const char* what, int capacity, ds_status st) {
    if (st != DS_OK) {
      ++bad;
      std::printf("%s of %d slots: %s\n", what, capacity, ds_last_error());
    }
    for (auto& [kernel, bytes] : held)
      if (g_allowed[kernel] < bytes) {
        ++bad;
        std::printf("%s of %d slots: a kernel that could have %d bytes is left with %d\n", what,
                    capacity, bytes, g_allowed[kernel]);
      }
    held = g_allowed;
  };
  for (int batch : {1, 2, 40})
    for (int hkv : {1, 8})
      for (int capacity : {1000000, 300000, 140000, 70001, 18432, 9001, 4096, 2049, 100, 2, 500000})
        check("eviction", capacity, evict(batch, hkv, capacity));
  for (int hq : {4, 16})
    for (int d : {128, 64})
      for (int capacity : {100000, 10}) check("attention", capacity, decode(hq, d, capacity));
  std::printf("%d launches above 48 KB, %d faults\n", g_large, bad);
  return bad || g_large < 20;
}
