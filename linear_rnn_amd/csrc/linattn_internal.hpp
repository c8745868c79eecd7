// Host-side interface between the C ABI layer and the linear attention launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rwkv7 {

// One validated call with work to do (B, H, T at least 1).
struct LinattnCall {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const float* s_in;    // may be null (zeros)
  const int32_t* lens;  // may be null (every sequence has T tokens)
  void* y;
  float* s_out;  // may be null
  int64_t B, T, H;
  bool f32;            // element type of r, k, v, y (else bfloat16)
  int32_t per_token;   // log_w is [B, T, H] (else [H])
  hipStream_t stream;
};
hipError_t launch_linattn(const LinattnCall& c);
hipError_t launch_linattn_step(const LinattnCall& c);

}  // namespace rwkv7
