// diff.cuh -- the last step of differential attention, shared by its decode and
// prefill: the difference of the two maps' outputs and its norm.
#pragma once

#include <cuda_bf16.h>

#include "device.cuh"

namespace tvl {
namespace {

constexpr int kDV = 128;                 // a pair's value: two V heads side by side

struct DiffTail {
  const float* lam;                      // [pairs], or a row of them a token
  long long lam_stride;                  // 0, or pairs
  const __nv_bfloat16* weight;           // [kDV], or null: no norm
  float eps, out_scale;
};

// Factor of a row's d with sum of squares ss (its mean is taken over kDV).
__device__ __forceinline__ float diff_factor(const DiffTail& t, float ss) {
  if (t.weight == nullptr) return t.out_scale;
  const float ms = fmaf(ss, 1.0f / kDV, t.eps);
  return ms == 0.f ? 0.f : t.out_scale / sqrtf(ms);     // a row of zeros stays one
}

}  // namespace
}  // namespace tvl
