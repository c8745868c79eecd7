// Host-side interface between the C ABI layer and the layer norm launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rwkv7 {

// One validated call; D and G at least 1, G divides D. M is at least 1 in the forward.
struct NormCall {
  const void* x;
  const float* weight;  // may be null (1)
  const float* bias;    // forward; may be null (0)
  void* y;              // forward
  float* mean;          // [M, G]: written (may be null) or read
  float* rstd;
  const void* dy;  // backward
  void* dx;
  float* dweight;  // backward; may be null
  float* dbias;
  int64_t M, D, G;
  float eps;
  bool x_f32, y_f32;  // element types of x and dx, and of y and dy (else bfloat16)
  hipStream_t stream;
};
hipError_t launch_layernorm_forward(const NormCall& c);
hipError_t launch_layernorm_backward(const NormCall& c);

}  // namespace rwkv7
