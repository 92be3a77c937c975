// One AdamW update in fp32 (decoupled weight decay, bias corrections folded
// into step_size and inv_sqrt_bc2 by the host).
#pragma once

#include <cuda_runtime.h>

namespace qlora {

struct AdamwHyper {
  float beta1, beta2, eps;
  float decay;              // 1 - lr * weight_decay
  float step_size;          // lr / (1 - beta1^t)
  float inv_sqrt_bc2;       // 1 / sqrt(1 - beta2^t)
  float one;                // 1, which the compiler does not know (the 8-bit states' sums)
};

// m, v become the new states, root = sqrt(v); returns the new parameter.
template <typename H>
__device__ __forceinline__ float adamw_update(float p, float g, float& m, float& v, float& root, const H& a) {
  m = fmaf(a.beta1, m, (1.0f - a.beta1) * g);
  v = fmaf(a.beta2, v, (1.0f - a.beta2) * g * g);
  root = sqrtf(v);
  p = p * a.decay;
  const float denom = root * a.inv_sqrt_bc2 + a.eps;
  return p - a.step_size * (m / denom);
}

}  // namespace qlora
