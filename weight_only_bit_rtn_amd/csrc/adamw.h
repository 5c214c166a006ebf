// adamw.h -- internal launchers of the AdamW step (not exported).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lowbit {

constexpr int kAdamBlock = 256;  // values that share a maximum

struct AdamTensor {
  void* param;
  const void* grad;
  int64_t n;
};
struct AdamState {
  void *m, *v;
  float *m_max, *v_max, *master;
};
struct AdamOptions {
  double lr, beta1, beta2, eps, decay;
  int64_t step;
  const float* lr_at;
  const int32_t* step_at;
  const float* grad_scale_at;
};

// Parameter and gradient types: ElemType's fp16 and bf16, and fp32.
constexpr int kAdamF32 = 3;
// bits: 32, 8, or 8 | kAdamRandom, whose codes are rounded up or down by a number of step and place.
constexpr int kAdamRandom = 256;

hipError_t launch_adamw(const AdamTensor* tensors, int64_t count, int param_type, int grad_type,
                        int bits, const AdamState& state, const AdamOptions& options,
                        hipStream_t stream);
hipError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_max,
                                const float* v_max, int64_t blocks, float* m_out, float* v_out,
                                hipStream_t stream);

}  // namespace lowbit
