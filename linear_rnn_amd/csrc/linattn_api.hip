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
  // four workgroups of 256 threads for each head within the grid's limit of 2^32 threads, and 32-bit offsets inside
  // 32 tokens
  int64_t units = 0, tok_heads = 0;
  if (H > (int64_t(1) << 18) || __builtin_mul_overflow(B, H, &units) || units > (int64_t(1) << 21))
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
  LinattnCall c{};
  c.r = r, c.log_w = log_w, c.k = k, c.v = v, c.s_in = state_in, c.lens = lens, c.y = y, c.s_out = state_out;
  c.B = B, c.T = T, c.H = H, c.f32 = dtype == RWKV7_DTYPE_F32, c.per_token = decay == RWKV7_DECAY_TOKEN, c.stream = s;
  return rwkv7::status_of([&] { return step ? rwkv7::launch_linattn_step(c) : rwkv7::launch_linattn(c); });
}

int run_backward(const LinattnCall& c, int64_t N, int dtype, int decay) {
  Sizes z;
  const int st = check_sizes(c.B, c.T, c.H, N, dtype, decay, &z);
  if (st != RWKV7_OK) return st;
  if (z.tokens > 0 && (!c.r || !c.log_w || !c.k || !c.v || !c.dy || !c.dr || !c.dlog_w || !c.dk || !c.dv))
    return RWKV7_ERR_NULL;
  for (const void* q : {c.r, (const void*)c.log_w, c.k, c.v, (const void*)c.s_in, (const void*)c.lens, c.dy,
                        (const void*)c.ds_out, (const void*)c.dr, (const void*)c.dlog_w, (const void*)c.dk,
                        (const void*)c.dv, (const void*)c.ds_in})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[8] = {range_of(c.r, z.tokens),   range_of(c.log_w, z.log_w), range_of(c.k, z.tokens),
                       range_of(c.v, z.tokens),   range_of(c.lens, z.lens),   range_of(c.s_in, z.state),
                       range_of(c.dy, z.tokens),  range_of(c.ds_out, z.state)};
  const Range out[5] = {range_of(c.dr, z.tokens), range_of(c.dlog_w, z.log_w), range_of(c.dk, z.tokens),
                        range_of(c.dv, z.tokens), range_of(c.ds_in, z.state)};
  if (rwkv7::outputs_overlap(out, 5, in, 8, &in[7])) return RWKV7_ERR_ALIAS;
  if (c.H == 0) return RWKV7_OK;
  hipError_t e = hipSuccess;
  if (c.B == 0 || c.T == 0) {  // no tokens: the state's gradient passes through, a decay's own is 0
    if (c.B > 0 && c.ds_in && c.ds_in != c.ds_out) e = rwkv7::launch_state_copy(c.ds_out, c.ds_in, c.B * c.H, c.stream);
    if (e == hipSuccess && !c.per_token && c.dlog_w) e = rwkv7::launch_linattn_zero(c.dlog_w, c.H, c.stream);
    return e == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP;
  }
  return rwkv7::status_of([&] { return rwkv7::launch_linattn_backward(c); });
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

int rwkv7_linattn_backward(const void* r, const float* log_w, const void* k, const void* v, const float* state_in,
                           const int32_t* lens, const void* dy, const float* dstate_out, void* dr, float* dlog_w, void* dk,
                           void* dv, float* dstate_in, int64_t B, int64_t T, int64_t H, int64_t N, int dtype, int decay,
                           void* stream) {
  LinattnCall c{};
  c.r = r, c.log_w = log_w, c.k = k, c.v = v, c.s_in = state_in, c.lens = lens, c.dy = dy, c.ds_out = dstate_out;
  c.dr = dr, c.dlog_w = dlog_w, c.dk = dk, c.dv = dv, c.ds_in = dstate_in;
  c.B = B, c.T = T, c.H = H, c.f32 = dtype == RWKV7_DTYPE_F32, c.per_token = decay == RWKV7_DECAY_TOKEN;
  c.stream = static_cast<hipStream_t>(stream);
  return run_backward(c, N, dtype, decay);
}

}  // extern "C"
