// Host-side interface between the C ABI layer and the gated linear unit's launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rwkv7 {

// One validated call; M, D and F at least 1.
struct GluCall {
  const void* x;       // [M, D]
  const void* w_gate;  // [D, F]
  const void* w_up;
  void* h;             // forward: [M, F]
  void* gate;          // [M, F]: written (both may be null) or read by the backward
  void* up;
  const void* dh;  // backward
  void* dx;        // may be null
  void* dw_gate;   // may be null, both or neither
  void* dw_up;
  int64_t M, D, F;
  bool f32;  // element type of everything (else bfloat16)
  int act;   // RWKV7_ACT_*
  hipStream_t stream;
};
hipError_t launch_glu_forward(const GluCall& c);
hipError_t launch_glu_backward(const GluCall& c);
// p <- zeros, n elements of 4 (f32) or 2 bytes.
hipError_t launch_glu_zero(void* p, int64_t n, bool f32, hipStream_t stream);

}  // namespace rwkv7
