// Norm of queries and keys per head with the rotation by position (launch
// interface).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fc {

inline constexpr int kQkMaxDim = 128;

struct QkRopeArgs {
  int N, hq, hk, D, R;      // R rotated pairs
  int64_t qs, ks;           // row strides of q and k (elements)
  float eps;
  bool bf16, interleaved;
  const void *q, *k;
  const float *gamma_q, *gamma_k, *pos, *freq;
  // forward
  void *q_out, *k_out;
  // VJP
  const void *g_q, *g_k;
  void *q_grad, *k_grad;
  float* pos_grad;
  float* part;              // [2][blocks][D] when a gamma gradient is wanted
};

// Blocks of the VJP (each sums the gamma gradients of its nodes).
int qk_rope_vjp_blocks(const QkRopeArgs& a);
void launch_qk_rope_fwd(const QkRopeArgs& a, hipStream_t st);
// gamma gradients [D], each when non-null (then part is set)
void launch_qk_rope_vjp(const QkRopeArgs& a, float* gamma_q_grad, float* gamma_k_grad, hipStream_t st);

}  // namespace fc
