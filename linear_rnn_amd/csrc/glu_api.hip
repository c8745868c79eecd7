// C ABI of the gated linear unit: argument validation and dispatch.
// Every check runs before the first HIP call.
#include <stdint.h>

#include "api_checks.hpp"
#include "glu_internal.hpp"
#include "rwkv7_wkv.h"

namespace {

using rwkv7::GluCall;
using rwkv7::Range;
using rwkv7::range_of;

struct Sizes {
  int64_t x, w, h;  // bytes
};

int check_sizes(int64_t M, int64_t D, int64_t F, int dtype, int act, Sizes* out) {
  if (dtype != RWKV7_DTYPE_F32 && dtype != RWKV7_DTYPE_BF16) return RWKV7_ERR_DTYPE;
  if (act != RWKV7_ACT_SIGMOID && act != RWKV7_ACT_SILU && act != RWKV7_ACT_GELU && act != RWKV7_ACT_RELU2)
    return RWKV7_ERR_MODE;
  // row numbers and the offsets inside a tile are 32-bit, and the tiles and threads of 8 elements fit a grid
  constexpr int64_t kMost = int64_t(1) << 20, kElems = int64_t(1) << 34;
  if (M < 0 || M > (int64_t(1) << 28) || D < 1 || D > kMost || F < 0 || F > kMost) return RWKV7_ERR_SHAPE;
  if (((M + 255) / 256) * ((F + 127) / 128) > (int64_t(1) << 22) || ((M + 255) / 256) * ((D + 127) / 128) > (int64_t(1) << 22) ||
      ((D + 255) / 256) * ((F + 127) / 128) > (int64_t(1) << 22))
    return RWKV7_ERR_SHAPE;
  if (M * D > kElems || M * F > kElems || D * F > kElems) return RWKV7_ERR_SHAPE;
  const int64_t e = dtype == RWKV7_DTYPE_BF16 ? 2 : 4;
  out->x = M * D * e, out->w = D * F * e, out->h = M * F * e;
  return RWKV7_OK;
}

}  // namespace

extern "C" {

int rwkv7_glu_forward(const void* x, const void* w_gate, const void* w_up, void* h, void* gate, void* up, int64_t M,
                      int64_t D, int64_t F, int dtype, int act, void* stream) {
  Sizes z;
  const int st = check_sizes(M, D, F, dtype, act, &z);
  if (st != RWKV7_OK) return st;
  if (z.h > 0 && (!x || !w_gate || !w_up || !h || (gate == nullptr) != (up == nullptr))) return RWKV7_ERR_NULL;
  for (const void* q : {x, w_gate, w_up, (const void*)h, (const void*)gate, (const void*)up})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[3] = {range_of(x, z.x), range_of(w_gate, z.w), range_of(w_up, z.w)};
  const Range out[3] = {range_of(h, z.h), range_of(gate, z.h), range_of(up, z.h)};
  if (rwkv7::outputs_overlap(out, 3, in, 3, nullptr)) return RWKV7_ERR_ALIAS;
  if (z.h == 0) return RWKV7_OK;
  GluCall c{};
  c.x = x, c.w_gate = w_gate, c.w_up = w_up, c.h = h, c.gate = gate, c.up = up, c.M = M, c.D = D, c.F = F;
  c.f32 = dtype == RWKV7_DTYPE_F32, c.act = act, c.stream = static_cast<hipStream_t>(stream);
  return rwkv7::status_of([&] { return rwkv7::launch_glu_forward(c); });
}

int rwkv7_glu_backward(const void* x, const void* w_gate, const void* w_up, const void* gate, const void* up,
                       const void* dh, void* dx, void* dw_gate, void* dw_up, int64_t M, int64_t D, int64_t F, int dtype,
                       int act, void* stream) {
  Sizes z;
  const int st = check_sizes(M, D, F, dtype, act, &z);
  if (st != RWKV7_OK) return st;
  if ((dw_gate == nullptr) != (dw_up == nullptr)) return RWKV7_ERR_NULL;
  if (z.h > 0 && (!x || !w_gate || !w_up || !gate || !up || !dh)) return RWKV7_ERR_NULL;
  for (const void* q : {x, w_gate, w_up, gate, up, dh, (const void*)dx, (const void*)dw_gate, (const void*)dw_up})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[6] = {range_of(x, z.x),    range_of(w_gate, z.w), range_of(w_up, z.w),
                       range_of(gate, z.h), range_of(up, z.h),     range_of(dh, z.h)};
  const Range out[3] = {range_of(dx, z.x), range_of(dw_gate, z.w), range_of(dw_up, z.w)};
  if (rwkv7::outputs_overlap(out, 3, in, 6, nullptr)) return RWKV7_ERR_ALIAS;
  const bool f32 = dtype == RWKV7_DTYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (z.h == 0) {  // no rows or no columns: sums of nothing
    return rwkv7::status_of([&] {
      hipError_t e = hipSuccess;
      if (dx && M > 0) e = rwkv7::launch_glu_zero(dx, M * D, f32, s);
      if (e == hipSuccess && dw_gate && F > 0) e = rwkv7::launch_glu_zero(dw_gate, D * F, f32, s);
      if (e == hipSuccess && dw_up && F > 0) e = rwkv7::launch_glu_zero(dw_up, D * F, f32, s);
      return e;
    });
  }
  GluCall c{};
  c.x = x, c.w_gate = w_gate, c.w_up = w_up, c.gate = const_cast<void*>(gate), c.up = const_cast<void*>(up), c.dh = dh;
  c.dx = dx, c.dw_gate = dw_gate, c.dw_up = dw_up, c.M = M, c.D = D, c.F = F, c.f32 = f32, c.act = act, c.stream = s;
  return rwkv7::status_of([&] { return rwkv7::launch_glu_backward(c); });
}

}  // extern "C"
