// C ABI of the linear attention with a decay for each head: argument validation and dispatch.
// Every check runs before the first HIP call.
#include <stdint.h>

#include "api_checks.hpp"
#include "linattn_internal.hpp"
#include "rwkv7_wkv.h"
#include "wkv7_internal.hpp"

namespace {

using rwkv7::LinattnCall;
using rwkv7::Range;
using rwkv7::range_of;

// Sizes of a call's tensors in bytes.
struct Sizes {
  int64_t tokens, log_w, state, lens;
};

int check_sizes(int64_t B, int64_t T, int64_t H, int64_t N, int dtype, int decay, Sizes* out) {
  if (dtype != RWKV7_DTYPE_F32 && dtype != RWKV7_DTYPE_BF16) return RWKV7_ERR_DTYPE;
  if (decay != RWKV7_DECAY_HEAD && decay != RWKV7_DECAY_TOKEN) return RWKV7_ERR_DECAY;
  if (B < 0 || T < 0 || H < 0) return RWKV7_ERR_SHAPE;
  if (N != RWKV7_HEAD_SIZE) return RWKV7_ERR_HEAD_SIZE;
  // a workgroup for each head (and segment) within the grid's limit of 2^32 threads, and 32-bit
  // offsets inside 32 tokens
  int64_t units = 0, tok_heads = 0;
  if (H > (int64_t(1) << 18) || __builtin_mul_overflow(B, H, &units) || units > (int64_t(1) << 23))
    return RWKV7_ERR_SHAPE;
  if (__builtin_mul_overflow(units, T, &tok_heads) || tok_heads > (int64_t(1) << 50)) return RWKV7_ERR_SHAPE;
  out->tokens = tok_heads * 64 * (dtype == RWKV7_DTYPE_BF16 ? 2 : 4);
  out->log_w = (decay == RWKV7_DECAY_TOKEN ? tok_heads : H) * 4;
  out->state = units * 64 * 64 * 4;
  out->lens = B * 4;
  return RWKV7_OK;
}

int run_linattn(const void* r, const float* log_w, const void* k, const void* v, const float* state_in,
                const int32_t* lens, void* y, float* state_out, int64_t B, int64_t T, int64_t H, int64_t N, int dtype,
                int decay, bool step, void* stream) {
  Sizes z;
  const int st = check_sizes(B, T, H, N, dtype, decay, &z);
  if (st != RWKV7_OK) return st;
  if (step && T != 1) return RWKV7_ERR_SHAPE;
  if (z.tokens > 0 && (!r || !log_w || !k || !v || !y)) return RWKV7_ERR_NULL;
  for (const void* q : {r, (const void*)log_w, k, v, (const void*)state_in, (const void*)lens, (const void*)y,
                        (const void*)state_out})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[6] = {range_of(r, z.tokens),       range_of(log_w, z.log_w), range_of(k, z.tokens),
                       range_of(v, z.tokens),       range_of(lens, z.lens),   range_of(state_in, z.state)};
  const Range out[2] = {range_of(y, z.tokens), range_of(state_out, z.state)};
  if (rwkv7::outputs_overlap(out, 2, in, 6, &in[5])) return RWKV7_ERR_ALIAS;
  if (B * H == 0) return RWKV7_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (T == 0) {
    if (state_out && state_out != state_in) e = rwkv7::launch_state_copy(state_in, state_out, B * H, s);
    return e == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP;
  }
  const LinattnCall c{r, log_w, k, v, state_in, lens, y, state_out, B, T, H, dtype == RWKV7_DTYPE_F32,
                      decay == RWKV7_DECAY_TOKEN, s};
  e = step ? rwkv7::launch_linattn_step(c) : rwkv7::launch_linattn(c);
  return e == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP;
}

}  // namespace

extern "C" {

int rwkv7_linattn_prefill(const void* r, const float* log_w, const void* k, const void* v, const float* state_in,
                          const int32_t* lens, void* y, float* state_out, int64_t B, int64_t T, int64_t H, int64_t N,
                          int dtype, int decay, void* stream) {
  return run_linattn(r, log_w, k, v, state_in, lens, y, state_out, B, T, H, N, dtype, decay, false, stream);
}

int rwkv7_linattn_step(const void* r, const float* log_w, const void* k, const void* v, const float* state_in, void* y,
                       float* state_out, int64_t B, int64_t T, int64_t H, int64_t N, int dtype, int decay,
                       void* stream) {
  return run_linattn(r, log_w, k, v, state_in, nullptr, y, state_out, B, T, H, N, dtype, decay, true, stream);
}

}  // extern "C"
