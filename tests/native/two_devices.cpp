// A CUDA runtime of two devices, as far as the library's launches see it, and
// the library's own entry points over it: a launch is refused unless its
// kernel may use as much dynamic shared memory on the current device, and its
// grid has sizes that a grid can have.  Nothing runs; the pointers are never
// read.  With the argument "batches": calls of batches up to 200,000.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <utility>

#include "ds.h"

static int g_device = 0, g_large = 0;
static std::map<std::pair<int, const void*>, int> g_allowed;

static CUresult fake_encode(...) { return CUDA_SUCCESS; }

extern "C" {
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) g_allowed[{g_device, f}] = value;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* f, void**) {
  const dim3 g = cfg->gridDim;
  if (g.x < 1 || g.x > 0x7fffffffu || g.y < 1 || g.y > 65535 || g.z < 1 || g.z > 65535)
    return cudaErrorInvalidConfiguration;
  if (cfg->dynamicSmemBytes > 48 * 1024) {
    ++g_large;
    auto it = g_allowed.find({g_device, f});
    if (it == g_allowed.end() || (size_t)it->second < cfg->dynamicSmemBytes)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}

template <typename T>
static T* at(uintptr_t x) {
  return reinterpret_cast<T*>(x);
}

static ds_status kv4(int nodes, int d, int batch = 1, bool scores = false) {
  ds_kv4_attn_args a;
  ds_kv4_attn_args_default(&a);
  a.q = at<void>(4096); a.k_cache = at<void>(8192); a.v_cache = at<void>(12288);
  a.page_table = at<int32_t>(64); a.ctx_lens = at<int32_t>(64);
  a.tree_offsets = at<int32_t>(64); a.parents = at<int32_t>(64);
  a.batch = batch; a.n_nodes = nodes; a.num_q_heads = 8; a.num_kv_heads = 2; a.head_dim = d;
  if (scores) {
    a.chunk_scores = at<float>(16384); a.chunk_size = 64; a.max_chunks = 9;
  }
  a.page_size = 16; a.num_pages = 9; a.max_pages = 9; a.num_sms = 152;
  a.out = at<void>(16384); a.workspace = at<void>(65536); a.workspace_bytes = (size_t)1 << 40;
  return ds_kv4_verify_attn(&a, nullptr);
}

static ds_status bf16(int d) {
  ds_verify_args a;
  ds_verify_args_default(&a);
  a.q = at<void>(4096); a.k_cache = at<void>(8192); a.v_cache = at<void>(12288);
  a.page_table = at<int32_t>(64); a.ctx_lens = at<int32_t>(64);
  a.tree_offsets = at<int32_t>(64); a.parents = at<int32_t>(64);
  a.batch = 1; a.n_nodes = 9; a.num_q_heads = 8; a.num_kv_heads = 2; a.head_dim = d;
  a.page_size = 16; a.num_pages = 9; a.max_pages = 9; a.num_sms = 152; a.chunk_size = 64;
  a.max_chunks = 9; a.chunk_scores = at<float>(16384);
  a.out = at<void>(16384); a.workspace = at<void>(65536); a.workspace_bytes = (size_t)1 << 40;
  return ds_verify_attn(&a, nullptr);
}

static ds_status reject(int vocab) {
  ds_accept_args a;
  ds_accept_args_default(&a);
  a.mode = DS_ACCEPT_REJECT;
  a.target_logits = at<float>(4096); a.draft_logits = at<float>(8192);
  a.draft_tokens = at<int32_t>(64); a.parents = at<int32_t>(64);
  a.tree_offsets = at<int32_t>(64); a.uniforms = at<float>(64);
  a.batch = 1; a.n_nodes = 4; a.vocab = vocab;
  a.out_path = at<int32_t>(64); a.out_n_accepted = at<int32_t>(64); a.out_bonus = at<int32_t>(64);
  a.workspace = at<void>(65536); a.workspace_bytes = (size_t)1 << 30;
  return ds_accept(&a, nullptr);
}

static int batches() {
  int bad = 0;
  for (int batch : {1, 33, 65535, 65536, 200000})
    for (int nodes : {1, 4, 9})
      for (bool scores : {false, true}) {
        if (kv4(nodes * batch, 64, batch, scores) == DS_OK) continue;
        ++bad;
        std::printf("batch %d, %d nodes each, salience %d: %s\n", batch, nodes, scores,
                    ds_last_error());
      }
  return bad;
}

int main(int argc, char** argv) {
  if (argc > 1 && !std::strcmp(argv[1], "batches")) return batches() != 0;
  int bad = 0;
  for (int turn = 0; turn < 4; ++turn) {
    g_device = turn & 1;
    if (turn == 3) g_allowed.clear();          // a context torn down and made again
    auto check = [&](const char* what, int x, ds_status st) {
      if (st == DS_OK) return;
      ++bad;
      std::printf("device %d, turn %d: %s %d: %s\n", g_device, turn, what, x, ds_last_error());
    };
    for (int d : {64, 128}) {
      for (int nodes : {1, 4, 20}) check("kv4 nodes", nodes * 1000 + d, kv4(nodes, d));
      check("verify head_dim", d, bf16(d));
    }
    for (int v : {1000, 32000, 128256, 151936}) check("reject vocab", v, reject(v));
  }
  std::printf("%d launches above 48 KB, %d refused\n", g_large, bad);
  return bad || g_large < 4 * 8;
}
