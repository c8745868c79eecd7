// Gated linear recurrence: a decay for each token and channel.
//
// Per sequence b and channel d, with w_t = exp(log_w_t) in [0, 1]:
//   h_t = w_t h_{t-1} + s(w_t) x_t,   y_t = h_t,   s = 1, 1 - w or sqrt(1 - w^2).
// Gradients, with g_t = dL/dh_t (dy_t and what comes back from the next token):
//   g_t = dy_t + w_{t+1} g_{t+1},  dx_t = s g_t,  dlog_w_t = (w_t h_{t-1} + s'(log w_t) x_t) g_t.
// A run of tokens is an affine map of the state, h -> P h + L, and maps compose: (P2 P1, P2 L1 + L2). A workgroup
// takes 64 channels; a thread K tokens in a row of VEC channels, first as a map, then, when the maps before its own
// have been composed (lane exchanges in a wave, LDS between waves), token by token from its state. So every
// element is read once and h is the recurrence's own: no quotient of cumulative decays, which would overflow.
// The state, the maps and all sums are float32; a bfloat16 output is rounded once.
//
// Memory bounds all of it (8 bytes an element of a bfloat16 prompt, 14 of the gradients, and some ten operations).
#include "gscan_internal.hpp"
#include "operators_lock.hpp"
#include "rwkv7_wkv.h"
#include "wkv7_device.hpp"
#include "wkv7_internal.hpp"

namespace rwkv7 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kSlab = 64;      // channels of a workgroup
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTok = 8;        // tokens in a row of a thread
template <int VEC>
constexpr int kLanes = kSlab / VEC;  // threads side by side over the channels
template <int VEC>
constexpr int kTile = kThreads / kLanes<VEC> * kTok;  // tokens of a workgroup at a time
template <bool F32>
constexpr uint32_t kEsz = F32 ? 4 : 2;

struct ScanParams {
  const void* x;
  const float* log_w;
  const float* s_in;
  const int32_t* lens;
  void* y;
  float* s_out;
  const void* dy;
  void* dx;
  float* dlog_w;
  const float* ds_out;
  float* ds_in;
  // Maps of runs of tokens, [run][B][D] each. Forward: run 0 is the initial state (P = 0), run s + 1 segment s.
  // Backward: run s is tile s; `l` first holds its L, then the state before it, `r` first what it adds to the
  // gradient of the state, then the gradient that comes back to its last token.
  float *p, *l, *r;
  int64_t T, BD;
  int64_t seg_tokens;  // a multiple of the tile
  uint32_t B, D, slabs, segs;
  uint32_t first;  // number of the launch's first workgroup
};

// An access behind `bytes` reads zeros or writes nothing. That leaves out the tokens behind a sequence's end: a log w
// and an x of 0 are the map that changes nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset behind the end of every tile

// VEC values as loaded.
template <bool F32, int VEC>
struct Raw {
  uint32_t u[VEC == 1 ? 1 : F32 ? 4 : 2];
};
template <bool F32, int VEC>
__device__ __forceinline__ Raw<F32, VEC> load(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  Raw<F32, VEC> o;
  if constexpr (VEC == 4 && F32) {
    const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
    o.u[0] = x[0], o.u[1] = x[1], o.u[2] = x[2], o.u[3] = x[3];
  } else if constexpr (VEC == 4) {
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0));
    o.u[0] = x[0], o.u[1] = x[1];
  } else if constexpr (F32) {
    o.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
  } else {
    o.u[0] = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0);
  }
  return o;
}
template <bool F32, int VEC>
__device__ __forceinline__ float value(const Raw<F32, VEC>& r, int v) {
  if constexpr (F32) return __uint_as_float(r.u[v]);
  else if constexpr (VEC == 1) return bf16_lo(r.u[0]);
  else return v & 1 ? bf16_hi(r.u[v >> 1]) : bf16_lo(r.u[v >> 1]);
}
__device__ __forceinline__ uint32_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }  // nearest even
template <bool F32, int VEC>
__device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, uint32_t off, const float (&o)[VEC]) {
  if constexpr (VEC == 4 && F32) {
    __builtin_amdgcn_raw_buffer_store_b128(
        u32x4{__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])}, b, off, 0, 0);
  } else if constexpr (VEC == 4) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_bits(o[0]) | bf16_bits(o[1]) << 16, bf16_bits(o[2]) | bf16_bits(o[3]) << 16},
                                          b, off, 0, 0);
  } else if constexpr (F32) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), b, off, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_bits(o[0]), b, off, 0, 0);
  }
}

__device__ __forceinline__ float decay(float log_w) { return __builtin_amdgcn_exp2f(log_w * 1.44269504f); }
// 1 - exp(-z) for z >= 0, where w = exp(-z). 1 - w loses the digits of a decay close to 1, so up to 0.35 it is the
// alternating series, whose ninth term is below 2^-25 of the first there.
__device__ __forceinline__ float one_minus(float z, float w) {
  float p = fmaf(z, -1.f / 8, 1.f);
  p = fmaf(z * (-1.f / 7), p, 1.f);
  p = fmaf(z * (-1.f / 6), p, 1.f);
  p = fmaf(z * (-1.f / 5), p, 1.f);
  p = fmaf(z * (-1.f / 4), p, 1.f);
  p = fmaf(z * (-1.f / 3), p, 1.f);
  p = fmaf(z * (-1.f / 2), p, 1.f);
  return z < 0.35f ? z * p : 1.f - w;
}
template <int KIND>
__device__ __forceinline__ float scale(float log_w, float w) {
  if constexpr (KIND == RWKV7_INPUT_PLAIN) return 1.f;
  else if constexpr (KIND == RWKV7_INPUT_MIX) return one_minus(-log_w, w);
  else return __builtin_amdgcn_sqrtf(one_minus(-2.f * log_w, w * w));
}
// The derivative of s to log w; that of sqrt(1 - w^2) at w = 1, where it has none, counts as 0.
template <int KIND>
__device__ __forceinline__ float slope(float w, float s) {
  if constexpr (KIND == RWKV7_INPUT_PLAIN) return 0.f;
  else if constexpr (KIND == RWKV7_INPUT_MIX) return -w;
  else return s > 0.f ? -w * w * __builtin_amdgcn_rcpf(s) : s * 0.f;
}

// Values of the even and the odd row of 16 lanes of a pair, and of the lower and the upper half, in all their lanes.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two rows_of_pair(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)s[0]), __builtin_bit_cast(float, (uint32_t)s[1])};
}
__device__ __forceinline__ Two halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)s[0]), __builtin_bit_cast(float, (uint32_t)s[1])};
}

// The maps of the other waves: [turn][wave][channel].
struct Shared {
  float p[2][kWaves][kSlab], l[2][kWaves][kSlab];
};

// From each thread's map (P, L): the map of the threads before it (REV: behind it) in the wave, in (P, L), and the
// wave's own to LDS.
template <int VEC, bool REV>
__device__ __forceinline__ void maps_of_wave(float (&P)[VEC], float (&L)[VEC], float (*sp)[kSlab], float (*sl)[kSlab]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if constexpr (VEC == 1) {
    sp[wave][lane] = P[0];
    sl[wave][lane] = L[0];
    P[0] = 1.f;
    L[0] = 0.f;
  } else {
    const bool second = ((lane >> 4) & 1) == (REV ? 0 : 1), upper = (lane >> 5) == (REV ? 0 : 1);
    float tp[VEC], tl[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const Two p = rows_of_pair(P[v]), l = rows_of_pair(L[v]);
      const float p1 = REV ? p.b : p.a, p2 = REV ? p.a : p.b, l1 = REV ? l.b : l.a, l2 = REV ? l.a : l.b;
      const Two hp = halves(p1 * p2), hl = halves(fmaf(p2, l1, l2));
      const float hp1 = REV ? hp.b : hp.a, hp2 = REV ? hp.a : hp.b, hl1 = REV ? hl.b : hl.a, hl2 = REV ? hl.a : hl.b;
      tp[v] = hp1 * hp2;
      tl[v] = fmaf(hp2, hl1, hl2);
      const float ep = second ? p1 : 1.f, el = second ? l1 : 0.f;
      P[v] = upper ? ep * hp1 : ep;
      L[v] = upper ? fmaf(ep, hl1, el) : el;
    }
    if (lane < 16) {
      *reinterpret_cast<float4*>(&sp[wave][lane * 4]) = make_float4(tp[0], tp[1], tp[2], tp[3]);
      *reinterpret_cast<float4*>(&sl[wave][lane * 4]) = make_float4(tl[0], tl[1], tl[2], tl[3]);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void get(const float* at, float (&o)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 f = *reinterpret_cast<const float4*>(at);
    o[0] = f.x, o[1] = f.y, o[2] = f.z, o[3] = f.w;
  } else {
    o[0] = *at;
  }
}
template <int VEC>
__device__ __forceinline__ void put(float* at, const float (&o)[VEC]) {
  if constexpr (VEC == 4) *reinterpret_cast<float4*>(at) = make_float4(o[0], o[1], o[2], o[3]);
  else *at = o[0];
}
// After a barrier: `in` is the state before this thread's tokens (REV: the gradient behind them), from that before
// the tile, `carry`, which becomes the one behind the tile; `all` is multiplied by the tile's P.
template <int VEC, bool REV>
__device__ __forceinline__ void enter(const float (&P)[VEC], const float (&L)[VEC], const float (*sp)[kSlab],
                                      const float (*sl)[kSlab], float (&carry)[VEC], float (&in)[VEC], float (&all)[VEC]) {
  const int wave = threadIdx.x >> 6, c = threadIdx.x % kLanes<VEC> * VEC;
  float wp[VEC], wl[VEC];
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int w = REV ? kWaves - 1 - i : i;
    get<VEC>(&sp[w][c], wp);
    get<VEC>(&sl[w][c], wl);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (w == wave) in[v] = fmaf(P[v], carry[v], L[v]);
      carry[v] = fmaf(wp[v], carry[v], wl[v]);
      all[v] *= wp[v];
    }
  }
}

__device__ __forceinline__ int64_t length(const ScanParams& p, uint32_t b) {
  if (!p.lens) return p.T;
  const int64_t n = p.lens[b];
  return n < 0 ? 0 : n < p.T ? n : p.T;
}

// A prompt, segment by segment: each workgroup walks the tiles of one segment of one sequence, the next tile's loads
// in flight while one is summed. MAPS: only the segment's map (for the workgroups of the segments behind it).
template <bool F32, int VEC, int KIND, bool MAPS>
__global__ __launch_bounds__(kThreads) void gscan_kernel(ScanParams p) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC>;
  __shared__ Shared sh;
  const uint32_t id = p.first + blockIdx.x;
  const uint32_t slab = id % p.slabs, seg = id / p.slabs % p.segs, b = id / p.slabs / p.segs;
  const uint32_t c = slab * kSlab + threadIdx.x % kLanes<VEC> * VEC, group = threadIdx.x / kLanes<VEC>;
  const bool on = c < p.D;
  const int64_t t0 = (int64_t)seg * p.seg_tokens;
  const int64_t end = p.T - t0 < p.seg_tokens ? p.T - t0 : p.seg_tokens;  // of the segment, from t0
  int64_t live = length(p, b) - t0;                                      // its tokens that count
  live = live < 0 ? 0 : live < end ? live : end;
  const uint32_t at = group * kTok * p.D + c;
  const uint32_t xoff = on ? at * esz : kNowhere, woff = on ? at * 4 : kNowhere;
  const int64_t base = ((int64_t)b * p.T + t0) * p.D;
  const int64_t bd = (int64_t)b * p.D + c;

  float carry[VEC], all[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) carry[v] = 0.f, all[v] = 1.f;
  if constexpr (MAPS) {
    if (seg == 0 && on && group == 0) {  // run 0: the initial state, which may be overwritten while others start from it
      float s[VEC] = {}, none[VEC] = {};
      if (p.s_in) get<VEC>(p.s_in + bd, s);
      put<VEC>(p.p + bd, none);
      put<VEC>(p.l + bd, s);
    }
  } else if (on) {
    if (p.segs == 1) {
      if (p.s_in) get<VEC>(p.s_in + bd, carry);
    } else {
#pragma unroll 8
      for (uint32_t s = 0; s <= seg; ++s) {
        float mp[VEC], ml[VEC];
        get<VEC>(p.p + s * p.BD + bd, mp);
        get<VEC>(p.l + s * p.BD + bd, ml);
#pragma unroll
        for (int v = 0; v < VEC; ++v) carry[v] = fmaf(mp[v], carry[v], ml[v]);
      }
    }
  }

  Raw<F32, VEC> rx[kTok];
  Raw<true, VEC> rw[kTok];
  auto fetch = [&](int64_t m) {
    const int64_t n = live - m < 0 ? 0 : live - m < tile ? live - m : tile;
    const auto bx = buffer(static_cast<const char*>(p.x) + (base + m * p.D) * esz, (uint32_t)n * p.D * esz);
    const auto bw = buffer(p.log_w + base + m * p.D, (uint32_t)n * p.D * 4);
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      rw[k] = load<true, VEC>(bw, woff + k * p.D * 4);
      rx[k] = load<F32, VEC>(bx, xoff + k * p.D * esz);
    }
  };
  fetch(0);
  int turn = 0;
  for (int64_t m = 0; m < live; m += tile) {
    float w[kTok][VEC], a[kTok][VEC], P[VEC], L[VEC], in[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) P[v] = 1.f, L[v] = 0.f;
#pragma unroll
    for (int k = 0; k < kTok; ++k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float lw = value<true, VEC>(rw[k], v);
        w[k][v] = decay(lw);
        a[k][v] = scale<KIND>(lw, w[k][v]) * value<F32, VEC>(rx[k], v);
      }
    fetch(m + tile);
#pragma unroll
    for (int k = 0; k < kTok; ++k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        L[v] = fmaf(w[k][v], L[v], a[k][v]);
        P[v] *= w[k][v];
      }
    maps_of_wave<VEC, false>(P, L, sh.p[turn], sh.l[turn]);
    lds_barrier();
    enter<VEC, false>(P, L, sh.p[turn], sh.l[turn], carry, in, all);
    turn ^= 1;
    if constexpr (!MAPS) {
      const int64_t n = live - m < tile ? live - m : tile;
      const auto by = buffer(static_cast<char*>(p.y) + (base + m * p.D) * esz, (uint32_t)n * p.D * esz);
#pragma unroll
      for (int k = 0; k < kTok; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) in[v] = fmaf(w[k][v], in[v], a[k][v]);
        store<F32, VEC>(by, xoff + k * p.D * esz, in);
      }
    }
  }
  if constexpr (MAPS) {
    if (on && group == 0) {
      put<VEC>(p.p + (seg + 1) * p.BD + bd, all);
      put<VEC>(p.l + (seg + 1) * p.BD + bd, carry);
    }
  } else {
    if (p.s_out && on && group == 0 && seg == p.segs - 1) put<VEC>(p.s_out + bd, carry);
    const float none[VEC] = {};
    for (int64_t m = live; m < end; m += tile) {  // behind the sequence's end
      const int64_t n = end - m < tile ? end - m : tile;
      const auto by = buffer(static_cast<char*>(p.y) + (base + m * p.D) * esz, (uint32_t)n * p.D * esz);
#pragma unroll
      for (int k = 0; k < kTok; ++k) store<F32, VEC>(by, xoff + k * p.D * esz, none);
    }
  }
}

// Gradients: a workgroup a tile, which it holds in registers. MAPS: the tile's maps, of the state forward and of its
// gradient backward (they share P). Else, from the state before the tile and the gradient behind it, the gradients.
template <bool F32, int VEC, int KIND, bool MAPS>
__global__ __launch_bounds__(kThreads) void gscan_grad_kernel(ScanParams p) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC>;
  __shared__ Shared sh[2];
  const uint32_t id = p.first + blockIdx.x;
  const uint32_t slab = id % p.slabs, seg = id / p.slabs % p.segs, b = id / p.slabs / p.segs;
  const uint32_t c = slab * kSlab + threadIdx.x % kLanes<VEC> * VEC, group = threadIdx.x / kLanes<VEC>;
  const bool on = c < p.D;
  const int64_t t0 = (int64_t)seg * tile;
  const uint32_t end = (uint32_t)(p.T - t0 < tile ? p.T - t0 : tile);
  const int64_t here = length(p, b) - t0;
  const uint32_t live = here < 0 ? 0 : here < end ? (uint32_t)here : end;
  const uint32_t at = group * kTok * p.D + c;
  const uint32_t xoff = on ? at * esz : kNowhere, woff = on ? at * 4 : kNowhere;
  const int64_t base = ((int64_t)b * p.T + t0) * p.D;
  const int64_t run = seg * p.BD + (int64_t)b * p.D + c;

  const auto bx = buffer(static_cast<const char*>(p.x) + base * esz, live * p.D * esz);
  const auto bg = buffer(static_cast<const char*>(p.dy) + base * esz, live * p.D * esz);
  const auto bw = buffer(p.log_w + base, live * p.D * 4);
  Raw<F32, VEC> rx[kTok], rg[kTok];
  Raw<true, VEC> rw[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    rw[k] = load<true, VEC>(bw, woff + k * p.D * 4);
    rx[k] = load<F32, VEC>(bx, xoff + k * p.D * esz);
    rg[k] = load<F32, VEC>(bg, xoff + k * p.D * esz);
  }
  float state[VEC] = {}, grad[VEC] = {}, all[VEC] = {};
  if (!MAPS && on) {
    get<VEC>(p.l + run, state);
    get<VEC>(p.r + run, grad);
  }
  float w[kTok][VEC], s[kTok][VEC], P[VEC], L[VEC], Q[VEC], R[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) P[v] = all[v] = 1.f, L[v] = R[v] = 0.f;
#pragma unroll
  for (int k = 0; k < kTok; ++k)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float lw = value<true, VEC>(rw[k], v);
      w[k][v] = decay(lw);
      s[k][v] = scale<KIND>(lw, w[k][v]);
      L[v] = fmaf(w[k][v], L[v], s[k][v] * value<F32, VEC>(rx[k], v));
      P[v] *= w[k][v];
    }
#pragma unroll
  for (int k = kTok - 1; k >= 0; --k)
#pragma unroll
    for (int v = 0; v < VEC; ++v) R[v] = w[k][v] * (value<F32, VEC>(rg[k], v) + R[v]);
#pragma unroll
  for (int v = 0; v < VEC; ++v) Q[v] = P[v];
  maps_of_wave<VEC, false>(P, L, sh[0].p[0], sh[0].l[0]);
  maps_of_wave<VEC, true>(Q, R, sh[1].p[0], sh[1].l[0]);
  lds_barrier();
  float h[VEC], g[VEC], unused[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) unused[v] = 1.f;
  enter<VEC, false>(P, L, sh[0].p[0], sh[0].l[0], state, h, all);
  enter<VEC, true>(Q, R, sh[1].p[0], sh[1].l[0], grad, g, unused);
  if constexpr (MAPS) {
    if (on && group == 0) {
      put<VEC>(p.p + run, all);
      put<VEC>(p.l + run, state);
      put<VEC>(p.r + run, grad);
    }
  } else {
    float before[kTok][VEC];
#pragma unroll
    for (int k = 0; k < kTok; ++k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        before[k][v] = h[v];
        h[v] = fmaf(w[k][v], h[v], s[k][v] * value<F32, VEC>(rx[k], v));
      }
    // zeros behind the sequence's end
    const auto bdx = buffer(static_cast<char*>(p.dx) + base * esz, end * p.D * esz);
    const auto bdw = buffer(p.dlog_w + base, end * p.D * 4);
#pragma unroll
    for (int k = kTok - 1; k >= 0; --k) {
      float dx[VEC], dw[VEC];
      const bool counts = group * kTok + k < live;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float q = value<F32, VEC>(rg[k], v) + g[v];
        dx[v] = counts ? s[k][v] * q : 0.f;
        dw[v] = counts ? fmaf(w[k][v], before[k][v], slope<KIND>(w[k][v], s[k][v]) * value<F32, VEC>(rx[k], v)) * q : 0.f;
        g[v] = w[k][v] * q;
      }
      store<F32, VEC>(bdx, xoff + k * p.D * esz, dx);
      store<true, VEC>(bdw, woff + k * p.D * 4, dw);
    }
  }
}

// The maps of a sequence's tiles, composed from both ends: the state before each tile to `l`, the gradient behind it
// to `r`, the initial state's gradient. 64 channels a workgroup, a wave a sixteenth of the tiles.
__global__ __launch_bounds__(1024) void gscan_join_kernel(ScanParams p) {
  __shared__ float sp[16][64], sl[16][64], sr[16][64];
  const uint32_t id = p.first + blockIdx.x;
  const uint32_t b = id / p.slabs, c = id % p.slabs * kSlab + (threadIdx.x & 63), wave = threadIdx.x >> 6;
  const bool on = c < p.D;
  const int64_t bd = (int64_t)b * p.D + (on ? c : 0);
  const uint32_t each = (p.segs + 15) / 16, s0 = wave * each < p.segs ? wave * each : p.segs;
  const uint32_t s1 = s0 + each < p.segs ? s0 + each : p.segs;
  float P = 1.f, L = 0.f, R = 0.f, Q = 1.f;
#pragma unroll 4
  for (uint32_t s = s0; s < s1; ++s) {
    const float m = p.p[s * p.BD + bd];
    L = fmaf(m, L, p.l[s * p.BD + bd]);
    R = fmaf(Q, p.r[s * p.BD + bd], R);  // the maps in front are applied last
    Q *= m;
    P *= m;
  }
  float h = p.s_in ? p.s_in[bd] : 0.f, g = p.ds_out ? p.ds_out[bd] : 0.f;
  sp[wave][threadIdx.x & 63] = P;
  sl[wave][threadIdx.x & 63] = L;
  sr[wave][threadIdx.x & 63] = R;
  __syncthreads();
  for (uint32_t i = 0; i < wave; ++i) h = fmaf(sp[i][threadIdx.x & 63], h, sl[i][threadIdx.x & 63]);
  for (uint32_t i = 15; i > wave; --i) g = fmaf(sp[i][threadIdx.x & 63], g, sr[i][threadIdx.x & 63]);
  if (!on) return;
#pragma unroll 4
  for (uint32_t s = s0; s < s1; ++s) {
    const float m = p.p[s * p.BD + bd], l = p.l[s * p.BD + bd];
    p.l[s * p.BD + bd] = h;
    h = fmaf(m, h, l);
  }
#pragma unroll 4
  for (uint32_t s = s1; s > s0; --s) {
    const float m = p.p[(s - 1) * p.BD + bd], r = p.r[(s - 1) * p.BD + bd];
    p.r[(s - 1) * p.BD + bd] = g;
    g = fmaf(m, g, r);
  }
  if (wave == 0 && p.ds_in) p.ds_in[bd] = g;
}

// One token: VEC channels of a sequence a thread.
template <bool F32, int VEC, int KIND>
__global__ __launch_bounds__(kThreads) void gscan_step_kernel(ScanParams p) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC;
  if (i >= p.BD) return;
  float s[VEC] = {}, lw[VEC];
  if (p.s_in) get<VEC>(p.s_in + i, s);
  get<VEC>(p.log_w + i, lw);
  const char* x = static_cast<const char*>(p.x) + i * kEsz<F32>;
  char* y = static_cast<char*>(p.y) + i * kEsz<F32>;
  Raw<F32, VEC> rx;
  if constexpr (VEC == 4 && F32) {
    const uint4 u = *reinterpret_cast<const uint4*>(x);
    rx.u[0] = u.x, rx.u[1] = u.y, rx.u[2] = u.z, rx.u[3] = u.w;
  } else if constexpr (VEC == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(x);
    rx.u[0] = u.x, rx.u[1] = u.y;
  } else if constexpr (F32) {
    rx.u[0] = *reinterpret_cast<const uint32_t*>(x);
  } else {
    rx.u[0] = *reinterpret_cast<const uint16_t*>(x);
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float w = decay(lw[v]);
    s[v] = fmaf(w, s[v], scale<KIND>(lw[v], w) * value<F32, VEC>(rx, v));
  }
  if (p.s_out) put<VEC>(p.s_out + i, s);
  if constexpr (VEC == 4 && F32) {
    *reinterpret_cast<float4*>(y) = make_float4(s[0], s[1], s[2], s[3]);
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(y) = make_uint2(bf16_bits(s[0]) | bf16_bits(s[1]) << 16, bf16_bits(s[2]) | bf16_bits(s[3]) << 16);
  } else if constexpr (F32) {
    *reinterpret_cast<float*>(y) = s[0];
  } else {
    *reinterpret_cast<uint16_t*>(y) = (uint16_t)bf16_bits(s[0]);
  }
}

// In launches of at most 2^22 workgroups: a grid's threads are counted in 32 bits.
hipError_t start(const void* fn, uint64_t blocks, int threads, ScanParams p, hipStream_t stream) {
  for (uint64_t first = 0; first < blocks; first += 1u << 22) {
    const uint64_t n = blocks - first < (1u << 22) ? blocks - first : (1u << 22);
    p.first = (uint32_t)first;
    void* args[] = {&p};
    const hipError_t e = hipLaunchKernel(fn, dim3((uint32_t)n), dim3(threads), args, 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

ScanParams params(const GscanCall& c) {
  ScanParams p{};
  p.x = c.x, p.log_w = c.log_w, p.s_in = c.s_in, p.lens = c.lens, p.y = c.y, p.s_out = c.s_out;
  p.dy = c.dy, p.dx = c.dx, p.dlog_w = c.dlog_w, p.ds_out = c.ds_out, p.ds_in = c.ds_in;
  p.T = c.T, p.BD = c.B * c.D, p.B = (uint32_t)c.B, p.D = (uint32_t)c.D;
  p.slabs = (p.D + kSlab - 1) / kSlab;
  return p;
}

template <bool F32, int VEC, int KIND>
struct Kernels {
  static constexpr int tile = kTile<VEC>;
  static hipError_t prefill(const GscanCall& c) {
    ScanParams p = params(c);
    const int64_t tiles = (c.T + tile - 1) / tile, units = c.B * p.slabs;
    // Segments: a workgroup for each unit leaves compute units idle where there are fewer than 256 of them.
    int64_t segs = units >= 256 ? 1 : (512 + units - 1) / units;
    const int64_t most = tiles / 2;
    segs = segs < most ? segs : most;
    segs = segs < 1 ? 1 : segs;
    p.seg_tokens = (tiles + segs - 1) / segs * tile;
    p.segs = (uint32_t)(tiles == 0 ? 1 : (c.T + p.seg_tokens - 1) / p.seg_tokens);
    const void* fn = reinterpret_cast<const void*>(&gscan_kernel<F32, VEC, KIND, false>);
    if (p.segs == 1) return start(fn, (uint64_t)units, kThreads, p, c.stream);
    std::lock_guard<std::mutex> lock(operators_mutex());
    void* ws = nullptr;
    const uint32_t nsegs = p.segs;
    hipError_t e = device_workspace(c.stream, (size_t)2 * nsegs * p.BD * 4, &ws, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    p.p = static_cast<float*>(ws), p.l = p.p + nsegs * p.BD;
    p.segs = nsegs - 1;  // nothing starts behind the last
    e = start(reinterpret_cast<const void*>(&gscan_kernel<F32, VEC, KIND, true>), (uint64_t)units * p.segs, kThreads, p,
              c.stream);
    if (e != hipSuccess) return e;
    p.segs = nsegs;
    return start(fn, (uint64_t)units * p.segs, kThreads, p, c.stream);
  }
  static hipError_t step(const GscanCall& c) {
    const ScanParams p = params(c);
    const int64_t threads = (p.BD + VEC - 1) / VEC;
    return start(reinterpret_cast<const void*>(&gscan_step_kernel<F32, VEC, KIND>), (uint64_t)(threads + kThreads - 1) / kThreads,
                 kThreads, p, c.stream);
  }
  static hipError_t backward(const GscanCall& c) {
    ScanParams p = params(c);
    p.segs = (uint32_t)((c.T + tile - 1) / tile);
    const uint64_t units = (uint64_t)p.B * p.slabs;
    const void* join = reinterpret_cast<const void*>(&gscan_join_kernel);
    if (p.segs == 0) return start(join, units, 1024, p, c.stream);
    std::lock_guard<std::mutex> lock(operators_mutex());
    void* ws = nullptr;
    hipError_t e = device_workspace(c.stream, (size_t)3 * p.segs * p.BD * 4, &ws, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    p.p = static_cast<float*>(ws), p.l = p.p + p.segs * p.BD, p.r = p.l + p.segs * p.BD;
    e = start(reinterpret_cast<const void*>(&gscan_grad_kernel<F32, VEC, KIND, true>), units * p.segs, kThreads, p, c.stream);
    if (e == hipSuccess) e = start(join, units, 1024, p, c.stream);
    if (e == hipSuccess)
      e = start(reinterpret_cast<const void*>(&gscan_grad_kernel<F32, VEC, KIND, false>), units * p.segs, kThreads, p, c.stream);
    return e;
  }
};

enum class Op { kPrefill, kStep, kBackward };
template <bool F32, int VEC, int KIND>
hipError_t run(const GscanCall& c, Op op) {
  using K = Kernels<F32, VEC, KIND>;
  return op == Op::kPrefill ? K::prefill(c) : op == Op::kStep ? K::step(c) : K::backward(c);
}
template <bool F32, int VEC>
hipError_t by_kind(const GscanCall& c, Op op) {
  if (c.input == RWKV7_INPUT_PLAIN) return run<F32, VEC, RWKV7_INPUT_PLAIN>(c, op);
  if (c.input == RWKV7_INPUT_MIX) return run<F32, VEC, RWKV7_INPUT_MIX>(c, op);
  return run<F32, VEC, RWKV7_INPUT_NORM>(c, op);
}
// Four channels a thread where every row starts on four of them, else one.
hipError_t dispatch(const GscanCall& c, Op op) {
  const bool four = (op == Op::kStep ? c.B * c.D : c.D) % 4 == 0;
  if (c.f32) return four ? by_kind<true, 4>(c, op) : by_kind<true, 1>(c, op);
  return four ? by_kind<false, 4>(c, op) : by_kind<false, 1>(c, op);
}

}  // namespace

hipError_t launch_gscan_prefill(const GscanCall& c) { return dispatch(c, Op::kPrefill); }
hipError_t launch_gscan_step(const GscanCall& c) { return dispatch(c, Op::kStep); }
hipError_t launch_gscan_backward(const GscanCall& c) { return dispatch(c, Op::kBackward); }

}  // namespace rwkv7
