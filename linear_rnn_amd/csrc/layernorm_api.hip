// C ABI of the layer norm over groups of channels: argument validation and dispatch.
// Every check runs before the first HIP call.
#include <stdint.h>

#include "api_checks.hpp"
#include "layernorm_internal.hpp"
#include "rwkv7_wkv.h"

namespace {

using rwkv7::NormCall;
using rwkv7::Range;
using rwkv7::range_of;

struct Sizes {
  int64_t x, y, stats, channels;  // bytes
};

int check_sizes(int64_t M, int64_t D, int64_t G, int x_dtype, int y_dtype, Sizes* out) {
  for (int t : {x_dtype, y_dtype})
    if (t != RWKV7_DTYPE_F32 && t != RWKV7_DTYPE_BF16) return RWKV7_ERR_DTYPE;
  int64_t elems = 0;
  // channel numbers are 32-bit, and workgroups over groups and channels fit the grid
  if (M < 0 || D < 0 || G < 1 || D > (int64_t(1) << 24) || D % G != 0) return RWKV7_ERR_SHAPE;
  if (__builtin_mul_overflow(M, D > 0 ? D : 1, &elems) || elems > (int64_t(1) << 50)) return RWKV7_ERR_SHAPE;
  if (D == 0) elems = 0;
  out->x = elems * (x_dtype == RWKV7_DTYPE_BF16 ? 2 : 4);
  out->y = elems * (y_dtype == RWKV7_DTYPE_BF16 ? 2 : 4);
  out->stats = D == 0 ? 0 : M * G * 4;
  out->channels = D * 4;
  return RWKV7_OK;
}

}  // namespace

extern "C" {

int rwkv7_layernorm_forward(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                            int64_t M, int64_t D, int64_t G, float eps, int x_dtype, int y_dtype, void* stream) {
  Sizes z;
  const int st = check_sizes(M, D, G, x_dtype, y_dtype, &z);
  if (st != RWKV7_OK) return st;
  if (!(eps >= 0.f && eps < __builtin_inff())) return RWKV7_ERR_SHAPE;
  if (z.x > 0 && (!x || !y)) return RWKV7_ERR_NULL;
  for (const void* q : {x, (const void*)weight, (const void*)bias, (const void*)y, (const void*)mean, (const void*)rstd})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[3] = {range_of(x, z.x), range_of(weight, z.channels), range_of(bias, z.channels)};
  const Range out[3] = {range_of(y, z.y), range_of(mean, z.stats), range_of(rstd, z.stats)};
  if (rwkv7::outputs_overlap(out, 3, in, 3, nullptr)) return RWKV7_ERR_ALIAS;
  if (z.x == 0) return RWKV7_OK;
  NormCall c{};
  c.x = x, c.weight = weight, c.bias = bias, c.y = y, c.mean = mean, c.rstd = rstd, c.M = M, c.D = D, c.G = G, c.eps = eps;
  c.x_f32 = x_dtype == RWKV7_DTYPE_F32, c.y_f32 = y_dtype == RWKV7_DTYPE_F32;
  c.stream = static_cast<hipStream_t>(stream);
  return rwkv7::status_of([&] { return rwkv7::launch_layernorm_forward(c); });
}

int rwkv7_layernorm_backward(const void* x, const float* weight, const float* mean, const float* rstd, const void* dy,
                             void* dx, float* dweight, float* dbias, int64_t M, int64_t D, int64_t G, int x_dtype,
                             int y_dtype, void* stream) {
  Sizes z;
  const int st = check_sizes(M, D, G, x_dtype, y_dtype, &z);
  if (st != RWKV7_OK) return st;
  if (z.x > 0 && (!x || !mean || !rstd || !dy || !dx)) return RWKV7_ERR_NULL;
  for (const void* q : {x, (const void*)weight, (const void*)mean, (const void*)rstd, dy, (const void*)dx,
                        (const void*)dweight, (const void*)dbias})
    if (rwkv7::misaligned(q)) return RWKV7_ERR_ALIGN;
  const Range in[5] = {range_of(x, z.x), range_of(weight, z.channels), range_of(mean, z.stats), range_of(rstd, z.stats),
                       range_of(dy, z.y)};
  const Range out[3] = {range_of(dx, z.x), range_of(dweight, z.channels), range_of(dbias, z.channels)};
  if (rwkv7::outputs_overlap(out, 3, in, 5, nullptr)) return RWKV7_ERR_ALIAS;
  if (D == 0) return RWKV7_OK;
  NormCall c{};
  c.x = x, c.weight = weight, c.mean = const_cast<float*>(mean), c.rstd = const_cast<float*>(rstd), c.dy = dy, c.dx = dx;
  c.dweight = dweight, c.dbias = dbias, c.M = M, c.D = D, c.G = G;
  c.x_f32 = x_dtype == RWKV7_DTYPE_F32, c.y_f32 = y_dtype == RWKV7_DTYPE_F32;
  c.stream = static_cast<hipStream_t>(stream);
  return rwkv7::status_of([&] { return rwkv7::launch_layernorm_backward(c); });
}

}  // extern "C"
