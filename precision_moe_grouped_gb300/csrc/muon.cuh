// muon.cuh -- what the orthogonalised step's two paths share (muon.cu: any size, on
// the tensor cores; muon_small.cu: a short side of up to 64).
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

// The momentum's and the update's ingredients, elementwise.
struct Momentum {
  const void* grad;
  float* m;
  const float* grad_scale;
  float mu, rest;                     // mu, 1 - mu
  int32_t bf16, nesterov;
};

__device__ __forceinline__ float grad_at(const Momentum& a, int64_t i, float gs) {
  return gs * (a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.grad)[i])
                      : static_cast<const float*>(a.grad)[i]);
}
__device__ __forceinline__ float update_of(const Momentum& a, float m, float g) {
  return a.nesterov ? fmaf(a.mu, m, a.rest * g) : m;
}

// Sum over the block in a fixed order; every thread gets it.
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* warp_sums) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += warp_sums[i];
  __syncthreads();
  return s;
}

// The tensors with a short side of up to kMuonSmall, all steps (muon_small.cu).
constexpr int kMuonSmall = 64;
bool muon_is_small(const moe_muon_tensor& t);
size_t muon_small_ws(const moe_muon_tensor* t, int32_t count);
int32_t muon_small_step(const moe_muon_tensor* t, int32_t count, const moe_muon_options* o, uint8_t* ws,
                        cudaStream_t st);

// An update's size, and the scalars of p <- decay p - step X.
float muon_decay(const moe_muon_options* o);
double muon_step(const moe_muon_options* o, const moe_muon_tensor& t);
bool muon_empty(const moe_muon_tensor& t);
constexpr int kMuonPartSteps = 3;   // steps between two Gram matrices

}  // namespace moe
