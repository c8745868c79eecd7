// Host-side interface between the C ABI layer and the gated linear recurrence's launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rwkv7 {

// One validated call; B and D at least 1, T at least 0.
struct GscanCall {
  const void* x;
  const float* log_w;
  const float* s_in;    // may be null (zeros)
  const int32_t* lens;  // may be null
  void* y;              // forward and step
  float* s_out;         // may be null; may be s_in
  const void* dy;       // backward
  const float* ds_out;  // may be null (zeros)
  void* dx;
  float* dlog_w;
  float* ds_in;  // may be null; may be ds_out
  int64_t B, T, D;
  bool f32;  // element type of x, y, dy, dx (else bfloat16)
  int input; // RWKV7_INPUT_*
  hipStream_t stream;
};
hipError_t launch_gscan_prefill(const GscanCall& c);
hipError_t launch_gscan_step(const GscanCall& c);
hipError_t launch_gscan_backward(const GscanCall& c);
// How often a workgroup of the backward looks for the others' maps before it leaves its tile to a second kernel (results
// are the same).
void set_gscan_polls(int polls);

}  // namespace rwkv7
