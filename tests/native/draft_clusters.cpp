// Evictions of long segments on devices that can place clusters of 16 blocks and
// on such that cannot, over a runtime that only keeps account: every launch is
// one that its device can take.
#include <cuda_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <map>
#include <set>

#include "ds.h"

static int g_device = 0, g_last = 0, g_asked = 0, g_launches = 0;
static std::set<const void*> g_large_allowed;
static bool fits(int device) { return device % 3 == 0; }   // of the others every second fails

extern "C" {
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeNonPortableClusterSizeAllowed && value) g_large_allowed.insert(f);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* cfg) {
  ++g_asked;
  *n = 0;
  if (cfg->numAttrs < 1 || cfg->attrs[0].val.clusterDim.x != 16 || !g_large_allowed.count(f))
    return cudaErrorInvalidValue;
  if (g_device % 3 == 2) return cudaErrorInvalidClusterSize;
  *n = fits(g_device) ? 7 : 0;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* f, void**) {
  int cluster = 1;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension)
      cluster = (int)cfg->attrs[i].val.clusterDim.x;
  if (cfg->gridDim.x % cluster || cluster > 16) return cudaErrorInvalidConfiguration;
  if (cluster > 8 && (!fits(g_device) || !g_large_allowed.count(f)))
    return cudaErrorInvalidClusterSize;
  if (cluster > g_last) g_last = cluster;
  ++g_launches;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
}

template <typename T>
static T* at(uintptr_t x) {
  return reinterpret_cast<T*>(x);
}

static ds_status evict(int batch, int capacity) {
  ds_evict_args a;
  ds_evict_args_default(&a);
  a.k_cache = at<void>(4096); a.v_cache = at<void>(4096); a.lens = at<int32_t>(64);
  a.batch = batch; a.num_kv_heads = 2; a.head_dim = 64; a.page_size = capacity;
  a.num_pages = batch; a.slot_heads = 1; a.slot_stride = capacity; a.weights = at<float>(64);
  a.positions = at<int32_t>(64); a.next_positions = at<int32_t>(64); a.new_lens = at<int32_t>(128);
  a.budget = capacity / 2 + 1; a.workspace = at<void>(65536);
  a.workspace_bytes = (size_t)1 << 60;
  return ds_cache_evict(&a, nullptr);
}

int main() {
  int bad = 0;
  for (g_device = 0; g_device < 70; ++g_device)            // (more than are remembered)
    for (int again = 0; again < 2; ++again)
      for (int batch : {1, 16, 17})
        for (int capacity : {100, 70000, 1000000}) {
          g_last = 0;
          const ds_status st = evict(batch, capacity);
          const bool large = capacity > 65536 && batch <= 16;
          const int most = !large ? 8 : fits(g_device) ? 16 : 8;
          if (st == DS_OK && g_last <= most && (!large || g_last == most)) continue;
          ++bad;
          std::printf("device %d, %d segments of %d: clusters of %d, status %d: %s\n", g_device,
                      batch, capacity, g_last, st, ds_last_error());
        }
  std::printf("%d launches, asked %d times, %d faults\n", g_launches, g_asked, bad);
  return bad || g_asked < 64;
}
