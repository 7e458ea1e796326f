// Kernel arguments of the 4-bit attention split passes.
#pragma once

#include "kv4.cuh"
#include "verify_common.cuh"

namespace ds {

struct Kv4KArgs {
  VerifyKArgs v;                  // k, v and the strides are not used
  const uint8_t* k4;
  const uint8_t* v4;
  float out_mult;                 // 2^v_exp
};

// The whole call for trees (kv4_tc.cu).
cudaError_t launch_kv4_tc(const Kv4KArgs& k, int head_dim, const VerifyLayout& L,
                          cudaStream_t stream);

// The whole call for few query rows per sequence and kv head (kv4_few.cu);
// `rows` is the number to plan for, any number is handled.
cudaError_t launch_kv4_few(const Kv4KArgs& k, int head_dim, int rows, const VerifyLayout& L,
                           cudaStream_t stream);

}  // namespace ds
