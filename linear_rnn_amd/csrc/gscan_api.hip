// C ABI of the gated linear recurrence: argument validation and dispatch.
// Every check runs before the first HIP call.
#include <stdint.h>

#include "api_checks.hpp"
#include "gscan_internal.hpp"
#include "rwkv7_wkv.h"

namespace {

using rwkv7::GscanCall;
using rwkv7::Range;
using rwkv7::range_of;

struct Sizes {
  int64_t x, log_w, states, lens;  // bytes
  bool empty;                      // no sequences or no channels
};

int check_sizes(int64_t B, int64_t T, int64_t D, int dtype, int input, Sizes* out) {
  if (dtype != RWKV7_DTYPE_F32 && dtype != RWKV7_DTYPE_BF16) return RWKV7_ERR_DTYPE;
  if (input != RWKV7_INPUT_PLAIN && input != RWKV7_INPUT_MIX && input != RWKV7_INPUT_NORM) return RWKV7_ERR_MODE;
  // a tile's offsets and the numbers of workgroups (64 channels and at least 32 tokens of a sequence) are 32-bit
  if (B < 0 || T < 0 || D < 0 || D > (int64_t(1) << 20)) return RWKV7_ERR_SHAPE;
  int64_t heads = 0, elems = 0;
  if (__builtin_mul_overflow(B, D > 0 ? D : 1, &heads) || heads > (int64_t(1) << 27)) return RWKV7_ERR_SHAPE;
  if (__builtin_mul_overflow(heads > 0 ? heads : 1, T, &elems) || elems > (int64_t(1) << 50)) return RWKV7_ERR_SHAPE;
  if (B > 0 && T > (int64_t(1) << 35) / (B * ((D + 63) / 64 > 0 ? (D + 63) / 64 : 1))) return RWKV7_ERR_SHAPE;
  out->empty = B == 0 || D == 0;
  if (out->empty) heads = elems = 0;
  out->x = elems * (dtype == RWKV7_DTYPE_BF16 ? 2 : 4);
  out->log_w = elems * 4;
  out->states = heads * 4;
  out->lens = B * 4;
  return RWKV7_OK;
}

GscanCall call_of(const void* x, const float* log_w, const float* state_in, const int32_t* lens, int64_t B, int64_t T,
                  int64_t D, int dtype, int input, void* stream) {
  GscanCall c{};
  c.x = x, c.log_w = log_w, c.s_in = state_in, c.lens = lens, c.B = B, c.T = T, c.D = D;
  c.f32 = dtype == RWKV7_DTYPE_F32, c.input = input, c.stream = static_cast<hipStream_t>(stream);
  return c;
}

int forward(const void* x, const float* log_w, const float* state_in, const int32_t* lens, void* y, float* state_out,
            int64_t B, int64_t T, int64_t D, int dtype, int input, void* stream, bool step) {
  Sizes z;
  const int st = check_sizes(B, T, D, dtype, input, &z);
  if (st != RWKV7_OK) return st;
  if (step && T != 1) return RWKV7_ERR_SHAPE;
  if (z.x > 0 && (!x || !log_w || !y)) return RWKV7_ERR_NULL;
  for (const void* q : {x, (const void*)log_w, (const void*)state_in, (const void*)lens, (const void*)y, (const void*)state_out})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[4] = {range_of(x, z.x), range_of(log_w, z.log_w), range_of(lens, z.lens), range_of(state_in, z.states)};
  const Range out[2] = {range_of(y, z.x), range_of(state_out, z.states)};
  if (rwkv7::outputs_overlap(out, 2, in, 4, &in[3])) return RWKV7_ERR_ALIAS;
  if (z.empty || (T == 0 && !state_out)) return RWKV7_OK;
  GscanCall c = call_of(x, log_w, state_in, lens, B, T, D, dtype, input, stream);
  c.y = y, c.s_out = state_out;
  return rwkv7::status_of([&] { return step ? rwkv7::launch_gscan_step(c) : rwkv7::launch_gscan_prefill(c); });
}

}  // namespace

extern "C" {

int rwkv7_gscan_prefill(const void* x, const float* log_w, const float* state_in, const int32_t* lens, void* y,
                        float* state_out, int64_t B, int64_t T, int64_t D, int dtype, int input, void* stream) {
  return forward(x, log_w, state_in, lens, y, state_out, B, T, D, dtype, input, stream, false);
}

int rwkv7_gscan_step(const void* x, const float* log_w, const float* state_in, void* y, float* state_out, int64_t B,
                     int64_t T, int64_t D, int dtype, int input, void* stream) {
  return forward(x, log_w, state_in, nullptr, y, state_out, B, T, D, dtype, input, stream, true);
}

int rwkv7_gscan_backward(const void* x, const float* log_w, const float* state_in, const int32_t* lens, const void* dy,
                         const float* dstate_out, void* dx, float* dlog_w, float* dstate_in, int64_t B, int64_t T,
                         int64_t D, int dtype, int input, void* stream) {
  Sizes z;
  const int st = check_sizes(B, T, D, dtype, input, &z);
  if (st != RWKV7_OK) return st;
  if (z.x > 0 && (!x || !log_w || !dy || !dx || !dlog_w)) return RWKV7_ERR_NULL;
  for (const void* q : {x, (const void*)log_w, (const void*)state_in, (const void*)lens, dy, (const void*)dstate_out,
                        (const void*)dx, (const void*)dlog_w, (const void*)dstate_in})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[6] = {range_of(x, z.x),  range_of(log_w, z.log_w), range_of(state_in, z.states), range_of(lens, z.lens),
                       range_of(dy, z.x), range_of(dstate_out, z.states)};
  const Range out[3] = {range_of(dx, z.x), range_of(dlog_w, z.log_w), range_of(dstate_in, z.states)};
  if (rwkv7::outputs_overlap(out, 3, in, 6, &in[5])) return RWKV7_ERR_ALIAS;
  if (z.empty || (T == 0 && !dstate_in)) return RWKV7_OK;
  GscanCall c = call_of(x, log_w, state_in, lens, B, T, D, dtype, input, stream);
  c.dy = dy, c.ds_out = dstate_out, c.dx = dx, c.dlog_w = dlog_w, c.ds_in = dstate_in;
  return rwkv7::status_of([&] { return rwkv7::launch_gscan_backward(c); });
}

}  // extern "C"
