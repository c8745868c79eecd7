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
// Memory bounds all of it (8 bytes an element of a bfloat16 prompt, 14 of the gradients, and some ten operations), at
// the rate of a large copy (4.9 to 5.5 TB/s): B=8 T=4096 D=4096 bfloat16 205 us (5.25 TB/s), B=1 T=32767 D=1024 float32 88 us
// (4.6, with 4 us for emptying words), gradients of B=8 T=4096 D=1024 bfloat16 107 us (4.4, the words they pass on
// not counted), float32 137 us (4.9). A step of B=512 D=4096 takes 5.3 us (6.3 TB/s, from the last-level cache).
#include "gscan_internal.hpp"
#include "launch_chunks.hpp"
#include "operators_lock.hpp"
#include "rwkv7_wkv.h"
#include "wkv7_device.hpp"
#include "wkv7_internal.hpp"

#include <atomic>

namespace rwkv7 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kSlab = 64;      // channels of a workgroup
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTok = 8;        // tokens in a row of a thread
template <int VEC>
constexpr int kLanes = kSlab / VEC;  // threads side by side over the channels
template <int VEC, int W = kWaves>
constexpr int kTile = W * kWave / kLanes<VEC> * kTok;  // tokens of a workgroup of W waves at a time
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
  // Gradients in two passes: the maps of tiles, [tile][B][D] each; `l` first holds a tile's L, then the state before it,
  // `r` first what it adds to the gradient of the state, then the gradient that comes back to its last token.
  float *p, *l, *r;
  // Words that workgroups pass to each other: maps of tiles, [tile][channel of all slabs], P and L (`there`) or P and R
  // (`back`) in one; the states before every kGroup tiles (`there` again, behind the tiles); numbers of workgroups.
  uint64_t *there, *back;
  float *first_state, *last_grad;  // copies of s_in and ds_out (zeros where null), [unit][64]: those may be overwritten
  uint32_t* ticket;  // number of workgroups that have started
  uint32_t* left;    // tiles left to the second kernel: how many, which
  uint32_t tiles, units;
  uint64_t words;  // to be emptied
  int polls;
  int64_t T, BD;
  uint32_t B, D, slabs;
  uint32_t first;  // number of the launch's first workgroup
};

// An access behind `bytes` reads zeros or writes nothing. That leaves out the tokens behind a sequence's end: a log w
// and an x of 0 are the map that changes nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // an offset behind the end of every tile

// The channels of a thread's place c (a multiple of VEC) among all slabs': where D is no multiple of four the last place has
// the last four channels, some of them the place's before it too (of the same workgroup), and both compute and write the
// same. A place from D on has none. So rows of nearly any width are loaded in fours (B=1 T=20000 D=333 bfloat16 23 us,
// by single channels 36; B=8 T=4096 D=1023 71 us, D=1025, by single channels, 123).
template <int VEC>
__device__ __forceinline__ uint32_t channel(uint32_t c, uint32_t D) {
  return VEC == 4 && c < D && c + 4 > D ? D - 4 : c;
}
// That of a place of a single channel.
template <int VEC>
__device__ __forceinline__ uint32_t channel_at(uint32_t c, uint32_t D) {
  return VEC == 4 ? channel<4>(c & ~3u, D) + (c & 3) : c;
}
// Not where a slab has one to three channels: its places would share some with another workgroup, which may have
// overwritten their states.
__host__ __device__ constexpr bool in_fours(uint32_t D) { return D % kSlab == 0 || D % kSlab >= 4; }

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
// 1 - exp(-z) for z >= 0, where w = exp(-z). 1 - w loses the digits of a decay close to 1, so up to 0.36 it is z times a
// polynomial of degree 4: the interpolation of (1 - exp(-z)) / z at that interval's Chebyshev nodes, 2^-25 off.
__device__ __forceinline__ float one_minus(float z, float w) {
  float p = fmaf(z, 0.0071817646f, -0.041313525f);
  p = fmaf(z, p, 0.1666218f);
  p = fmaf(z, p, -0.499998f);
  p = fmaf(z, p, 1.f);
  return z < 0.36f ? z * p : 1.f - w;
}
template <int KIND>
__device__ __forceinline__ float scale(float log_w, float w) {
  if constexpr (KIND == RWKV7_INPUT_PLAIN) return 1.f;
  else if constexpr (KIND == RWKV7_INPUT_MIX) return one_minus(-log_w, w);
  else return __builtin_amdgcn_sqrtf(one_minus(-2.f * log_w, w * w));
}
// dh/dlog w = w h + s' x, with h the state before. The derivative s' of sqrt(1 - w^2) at w = 1, where it has none, counts
// as 0.
template <int KIND>
__device__ __forceinline__ float through(float w, float s, float h, float x) {
  if constexpr (KIND == RWKV7_INPUT_PLAIN) return w * h;
  else if constexpr (KIND == RWKV7_INPUT_MIX) return w * (h - x);
  else return w * fmaf(s > 0.f ? -w * __builtin_amdgcn_rcpf(s) : 0.f, x, h);
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
template <int W = kWaves>
struct Shared {
  float p[2][W][kSlab], l[2][W][kSlab];
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
// In LDS or in a workspace, where four channels begin on 16 bytes.
template <int VEC>
__device__ __forceinline__ void get(const float* at, float (&o)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 f = *reinterpret_cast<const float4*>(at);
    o[0] = f.x, o[1] = f.y, o[2] = f.z, o[3] = f.w;
  } else {
    o[0] = *at;
  }
}
// In a [B, D] tensor, where they may begin on any channel.
template <int VEC>
__device__ __forceinline__ void get_any(const float* at, float (&o)[VEC]) {
  if constexpr (VEC == 4) {
    const f32x4_any f = *reinterpret_cast<const f32x4_any*>(at);
    o[0] = f[0], o[1] = f[1], o[2] = f[2], o[3] = f[3];
  } else {
    o[0] = *at;
  }
}
template <int VEC>
__device__ __forceinline__ void put_any(float* at, const float (&o)[VEC]) {
  if constexpr (VEC == 4) *reinterpret_cast<f32x4_any*>(at) = f32x4_any{o[0], o[1], o[2], o[3]};
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

// A prompt, a workgroup for each unit (64 channels of a sequence): it walks the tiles, the next tile's loads in flight
// while one is summed.
template <bool F32, int VEC, int KIND>
__global__ __launch_bounds__(kThreads) void gscan_walk_kernel(ScanParams p) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC>;
  __shared__ Shared<> sh;
  const uint32_t unit = p.first + blockIdx.x, slab = unit % p.slabs, b = unit / p.slabs;
  const uint32_t c = channel<VEC>(slab * kSlab + threadIdx.x % kLanes<VEC> * VEC, p.D), group = threadIdx.x / kLanes<VEC>;
  const bool on = c < p.D;
  const int64_t live = length(p, b);
  const uint32_t at = group * kTok * p.D + c;
  const uint32_t xoff = on ? at * esz : kNowhere, woff = on ? at * 4 : kNowhere;
  const int64_t base = (int64_t)b * p.T * p.D;
  const int64_t bd = (int64_t)b * p.D + c;

  float carry[VEC] = {};
  if (on && p.s_in) get_any<VEC>(p.s_in + bd, carry);
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
    float w[kTok][VEC], a[kTok][VEC], P[VEC], L[VEC], in[VEC], unused[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) P[v] = unused[v] = 1.f, L[v] = 0.f;
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
    enter<VEC, false>(P, L, sh.p[turn], sh.l[turn], carry, in, unused);
    turn ^= 1;
    const int64_t n = live - m < tile ? live - m : tile;
    const auto by = buffer(static_cast<char*>(p.y) + (base + m * p.D) * esz, (uint32_t)n * p.D * esz);
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) in[v] = fmaf(w[k][v], in[v], a[k][v]);
      store<F32, VEC>(by, xoff + k * p.D * esz, in);
    }
  }
  if (p.s_out && on && group == 0) put_any<VEC>(p.s_out + bd, carry);
  const float none[VEC] = {};
  for (int64_t m = live; m < p.T; m += tile) {  // behind the sequence's end
    const int64_t n = p.T - m < tile ? p.T - m : tile;
    const auto by = buffer(static_cast<char*>(p.y) + (base + m * p.D) * esz, (uint32_t)n * p.D * esz);
#pragma unroll
    for (int k = 0; k < kTok; ++k) store<F32, VEC>(by, xoff + k * p.D * esz, none);
  }
}

// One more token in a thread's map of the state (P, L) and that of what comes back to the gradient (P, R).
template <bool F32, int VEC, int KIND>
__device__ __forceinline__ void add_token(const Raw<F32, VEC>& rx, const Raw<F32, VEC>& rg, const Raw<true, VEC>& rw,
                                          float (&w)[VEC], float (&s)[VEC], float (&P)[VEC], float (&L)[VEC], float (&R)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float lw = value<true, VEC>(rw, v);
    w[v] = decay(lw);
    s[v] = scale<KIND>(lw, w[v]);
    L[v] = fmaf(w[v], L[v], s[v] * value<F32, VEC>(rx, v));
    P[v] *= w[v];
    R[v] = fmaf(P[v], value<F32, VEC>(rg, v), R[v]);
  }
}

template <int N>
__device__ __forceinline__ void forget(uint32_t (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(u[i]));
}

// A thread's tokens' gradients from the state before them (h) and the gradient behind them (g): that of the states
// from the last token, then the rest from the first; zeros behind the sequence's end.
template <bool F32, int VEC, int KIND>
__device__ __forceinline__ void write_grads(const ScanParams& p, int64_t base, uint32_t end, uint32_t live, uint32_t group,
                                            uint32_t xoff, uint32_t woff, Raw<F32, VEC> (&rx)[kTok],
                                            Raw<F32, VEC> (&rg)[kTok], const float (&w)[kTok][VEC],
                                            const float (&s)[kTok][VEC], float (&h)[VEC], float (&g)[VEC]) {
  constexpr uint32_t esz = kEsz<F32>;
  // What is quickly formed again is not kept in registers since the loads: offsets, widened values, s x.
  asm volatile("" : "+v"(xoff), "+v"(woff));
#pragma unroll
  for (int k = 0; k < kTok; ++k) forget(rx[k].u), forget(rg[k].u);
  float q[kTok][VEC];
#pragma unroll
  for (int k = kTok - 1; k >= 0; --k)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      q[k][v] = value<F32, VEC>(rg[k], v) + g[v];
      g[v] = w[k][v] * q[k][v];
    }
  auto bdx = buffer(static_cast<char*>(p.dx) + base * esz, live * p.D * esz);
  auto bdw = buffer(p.dlog_w + base, live * p.D * 4);
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    float dx[VEC], dw[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float x = value<F32, VEC>(rx[k], v);
      dx[v] = s[k][v] * q[k][v];
      dw[v] = through<KIND>(w[k][v], s[k][v], h[v], x) * q[k][v];
      h[v] = fmaf(w[k][v], h[v], s[k][v] * x);
    }
    store<F32, VEC>(bdx, xoff + k * p.D * esz, dx);
    store<true, VEC>(bdw, woff + k * p.D * 4, dw);
  }
  if (live < end) {
    const float none[VEC] = {};
    bdx = buffer(static_cast<char*>(p.dx) + base * esz, end * p.D * esz);
    bdw = buffer(p.dlog_w + base, end * p.D * 4);
#pragma unroll 1
    for (int k = 0; k < kTok; ++k) {
      if (group * kTok + k < live) continue;
      store<F32, VEC>(bdx, xoff + k * p.D * esz, none);
      store<true, VEC>(bdw, woff + k * p.D * 4, none);
    }
  }
}

// Gradients: a workgroup a tile, which it holds in registers. MAPS: the tile's maps, of the state forward and of its
// gradient backward (they share P). Else, from the state before the tile and the gradient behind it, the gradients.
template <bool F32, int VEC, int KIND, bool MAPS>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(F32 ? 2 : 3))) void gscan_grad_kernel(ScanParams p) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC>;
  __shared__ Shared<> sh[2];
  const uint32_t id = p.first + blockIdx.x;
  const uint32_t slab = id % p.slabs, seg = id / p.slabs % p.tiles, b = id / p.slabs / p.tiles;
  const uint32_t c = channel<VEC>(slab * kSlab + threadIdx.x % kLanes<VEC> * VEC, p.D), group = threadIdx.x / kLanes<VEC>;
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
  __builtin_amdgcn_sched_barrier(0);  // all loads before the first that is waited for
  float state[VEC] = {}, grad[VEC] = {}, all[VEC] = {};
  if (!MAPS && on) {
    get_any<VEC>(p.l + run, state);
    get_any<VEC>(p.r + run, grad);
  }
  float w[kTok][VEC], s[kTok][VEC], P[VEC], L[VEC], Q[VEC], R[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) P[v] = all[v] = 1.f, L[v] = R[v] = 0.f;
#pragma unroll
  for (int k = 0; k < kTok; ++k) add_token<F32, VEC, KIND>(rx[k], rg[k], rw[k], w[k], s[k], P, L, R);
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
      put_any<VEC>(p.p + run, all);
      put_any<VEC>(p.l + run, state);
      put_any<VEC>(p.r + run, grad);
    }
  } else {
    write_grads<F32, VEC, KIND>(p, base, end, live, group, xoff, woff, rx, rg, w, s, h, g);
  }
}

// ---- one pass over the data where the tiles of a sequence are spread over workgroups: each passes its tile's map on
// to the others of its sequence, in words of memory that hold both numbers of a map, so that a word is valid or empty.

constexpr uint64_t kEmpty = ~uint64_t(0);  // a NaN that no published word has as its P
// Tiles whose maps are composed at once: with 16 B=8 T=8192 D=4096 takes 399 us and with 32 404, B=1 T=200000 D=256, a
// chain of more links, 90 and 88 (8: 397 and 120).
constexpr uint32_t kGroup = 32;
// Waves of a tile of a prompt: with 4, tiles of 128 tokens, B=8 T=4096 D=1024 takes 71 us, with 8 55.
constexpr int kChainWaves = 8;

__device__ __forceinline__ void publish(uint64_t* at, float p, float l) {
  const uint32_t bits = p == p ? __float_as_uint(p) : 0x7fc00000u;
  __hip_atomic_store(at, (uint64_t)__float_as_uint(l) << 32 | bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Before each call: empties the words and copies the states that the call may overwrite.
__global__ __launch_bounds__(256) void gscan_empty_kernel(ScanParams p) {
  const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x, n = (uint64_t)gridDim.x * 256;
  if (i == 0) *p.ticket = 0, *p.left = 0;
  for (uint64_t w = 2 * i; w < p.words; w += 2 * n)
    *reinterpret_cast<ulonglong2*>(p.there + w) = make_ulonglong2(kEmpty, kEmpty);
  for (uint64_t w = i; w < (uint64_t)p.units * kSlab; w += n) {
    const uint32_t unit = w / kSlab, at_c = unit % p.slabs * kSlab + w % kSlab;
    const uint32_t c = in_fours(p.D) ? channel_at<4>(at_c, p.D) : at_c;
    const int64_t at = (int64_t)(unit / p.slabs) * p.D + c;
    if (p.first_state) p.first_state[w] = p.s_in && c < p.D ? p.s_in[at] : 0.f;
    if (p.last_grad) p.last_grad[w] = p.ds_out && c < p.D ? p.ds_out[at] : 0.f;
  }
}

// Workgroups take their numbers as they start, so that one waits only for others that have started too.
__device__ __forceinline__ uint32_t take_ticket(const ScanParams& p, uint32_t* shared) {
  if (threadIdx.x == 0) *shared = atomicAdd(p.ticket, 1u);
  __syncthreads();
  return *shared;
}

// After a barrier: the map of the wave's tokens before this thread's (REV: behind them) becomes the tile's. ROLLED: the
// waves' maps are read from LDS one by one; at once they would take the registers of a third of the workgroups of the
// bfloat16 gradients (213 registers and 161; B=8 T=4096 D=1024 114 and 107 us, B=4 D=4096 230 and 213), while the other kernels gain nothing by fewer.
template <int VEC, bool REV, int W, bool ROLLED>
__device__ __forceinline__ void compose(float (&P)[VEC], float (&L)[VEC], const float (*sp)[kSlab], const float (*sl)[kSlab]) {
  constexpr int kTurns = ROLLED ? 1 : W;
  const int wave = threadIdx.x >> 6, c = threadIdx.x % kLanes<VEC> * VEC;
  float wp[VEC], wl[VEC], ap[VEC], al[VEC], ep[VEC], el[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) ap[v] = 1.f, al[v] = 0.f, ep[v] = P[v], el[v] = L[v];
#pragma unroll kTurns
  for (int i = 0; i < W; ++i) {
    const int w = REV ? W - 1 - i : i;
    get<VEC>(&sp[w][c], wp);
    get<VEC>(&sl[w][c], wl);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (w == wave) P[v] = ep[v] * ap[v], L[v] = fmaf(ep[v], al[v], el[v]);
      al[v] = fmaf(wp[v], al[v], wl[v]);
      ap[v] *= wp[v];
    }
  }
}

// After a barrier: the map of the whole tile of channel `lane`, from the waves' maps.
template <bool REV, int W>
__device__ __forceinline__ void whole_map(const float (*sp)[kSlab], const float (*sl)[kSlab], float& p, float& l) {
  const int lane = threadIdx.x & 63;
  p = 1.f, l = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int w = REV ? W - 1 - i : i;
    l = fmaf(sp[w][lane], l, sl[w][lane]);
    p *= sp[w][lane];
  }
}
// After a barrier: what the waves' maps make of `v`, the values of the channels from c on at their beginning.
template <int VEC, bool REV, int W, bool ROLLED>
__device__ __forceinline__ void pass(const float (*sp)[kSlab], const float (*sl)[kSlab], int c, float (&v)[VEC]) {
  constexpr int kTurns = ROLLED ? 1 : W;
  float p[VEC], l[VEC];
#pragma unroll kTurns
  for (int i = 0; i < W; ++i) {
    get<VEC>(&sp[REV ? W - 1 - i : i][c], p);
    get<VEC>(&sl[REV ? W - 1 - i : i][c], l);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf(p[e], v[e], l[e]);
  }
}

// A prompt: a workgroup a tile, all sequences' first tiles before their second ones. The state before a tile comes
// from the state before its kGroup tiles, which the last of those before them published, and the maps of those of its
// kGroup that are before it: the same composition whenever they come. All of them are workgroups that started earlier, and a
// tile's map waits for nobody.
template <bool F32, int VEC, int KIND, int W>
__global__ __launch_bounds__(W * kWave) void gscan_chain_kernel(ScanParams p) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC, W>;
  constexpr uint32_t kEach = kGroup / W;  // tiles whose maps a wave reads, a channel a lane
  __shared__ Shared<W> sh;
  __shared__ uint32_t number;
  const uint32_t id = take_ticket(p, &number), unit = id % p.units, k = id / p.units;
  if (k >= p.tiles) return;  // only where two calls share a workspace against the rules
  const uint32_t slab = unit % p.slabs, b = unit / p.slabs;
  const uint32_t lc = threadIdx.x % kLanes<VEC> * VEC, c = channel<VEC>(slab * kSlab + lc, p.D), group = threadIdx.x / kLanes<VEC>;
  const bool on = c < p.D;
  const int64_t t0 = (int64_t)k * tile;
  const uint32_t end = (uint32_t)(p.T - t0 < tile ? p.T - t0 : tile);
  const int64_t here = length(p, b) - t0;
  const uint32_t live = here < 0 ? 0 : here < end ? (uint32_t)here : end;
  const uint32_t at = group * kTok * p.D + c;
  const uint32_t xoff = on ? at * esz : kNowhere, woff = on ? at * 4 : kNowhere;
  const int64_t base = ((int64_t)b * p.T + t0) * p.D;
  const uint64_t row = (uint64_t)p.units * kSlab, word = (uint64_t)unit * kSlab;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const auto bx = buffer(static_cast<const char*>(p.x) + base * esz, live * p.D * esz);
  const auto bw = buffer(p.log_w + base, live * p.D * 4);
  Raw<F32, VEC> rx[kTok];
  Raw<true, VEC> rw[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    rw[i] = load<true, VEC>(bw, woff + i * p.D * 4);
    rx[i] = load<F32, VEC>(bx, xoff + i * p.D * esz);
  }
  __builtin_amdgcn_sched_barrier(0);  // all loads before the first that is waited for
  float w[kTok][VEC], a[kTok][VEC], P[VEC], L[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) P[v] = 1.f, L[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float lw = value<true, VEC>(rw[i], v);
      w[i][v] = decay(lw);
      a[i][v] = scale<KIND>(lw, w[i][v]) * value<F32, VEC>(rx[i], v);
      L[v] = fmaf(w[i][v], L[v], a[i][v]);
      P[v] *= w[i][v];
    }
  maps_of_wave<VEC, false>(P, L, sh.p[0], sh.l[0]);
  lds_barrier();
  if (wave == 0) {
    float q, l;
    whole_map<false, W>(sh.p[0], sh.l[0], q, l);
    publish(p.there + k * row + word + lane, q, l);
  }
  compose<VEC, false, W, false>(P, L, sh.p[0], sh.l[0]);

  // the state before this tile's kGroup tiles in wave 0's map, as a constant
  const uint32_t before = k / kGroup * kGroup;
  // (all looked for at once, without a branch between them: this tile's own in the place of those it does not need)
  const uint64_t* const own = p.there + k * row + word + lane;
  auto from = [&](uint32_t i) {
    if (i == kEach) return wave == 0 && before > 0 ? p.there + (p.tiles + before / kGroup - 1) * row + word + lane : own;
    const uint32_t j = before + wave * kEach + i;
    return j < k ? p.there + j * row + word + lane : own;
  };
  // Some seconds at most: what two calls that share a workspace against the rules may wait for never comes (an empty
  // word is a NaN, and so are the results).
  uint64_t m[kEach + 1];
#pragma unroll 1
  for (uint32_t polls = 0; polls < 1u << 21; ++polls) {
#pragma unroll
    for (uint32_t i = 0; i <= kEach; ++i) m[i] = peek(from(i));
    uint32_t missing = 0;
#pragma unroll
    for (uint32_t i = 0; i <= kEach; ++i) missing = missing | ((uint32_t)(from(i) != own) & (uint32_t)(m[i] == kEmpty));
    if (missing == 0) break;
    __builtin_amdgcn_s_sleep(1);
  }
  float mp = 1.f, ml = 0.f;
  if (wave == 0) mp = 0.f, ml = before > 0 ? __uint_as_float((uint32_t)(m[kEach] >> 32)) : p.first_state[word + lane];
#pragma unroll
  for (uint32_t i = 0; i < kEach; ++i) {
    const bool counts = before + wave * kEach + i < k;
    const float q = counts ? __uint_as_float((uint32_t)m[i]) : 1.f;
    ml = fmaf(q, ml, counts ? __uint_as_float((uint32_t)(m[i] >> 32)) : 0.f);
    mp *= q;
  }
  sh.p[1][wave][lane] = mp;
  sh.l[1][wave][lane] = ml;
  lds_barrier();
  const bool ends = k + 1 == p.tiles;
  const uint32_t lane_c = channel_at<VEC>(slab * kSlab + lane, p.D);
  if (wave == 0 && (ends || k % kGroup == kGroup - 1)) {  // the state behind this tile
    float q, l, next[1] = {0.f};
    pass<1, false, W, false>(sh.p[1], sh.l[1], lane, next);
    whole_map<false, W>(sh.p[0], sh.l[0], q, l);
    next[0] = fmaf(q, next[0], l);
    if (!ends) publish(p.there + (p.tiles + k / kGroup) * row + word + lane, 0.f, next[0]);
    else if (p.s_out && lane_c < p.D) p.s_out[(int64_t)b * p.D + lane_c] = next[0];
  }
  float state[VEC] = {};
  pass<VEC, false, W, false>(sh.p[1], sh.l[1], lc, state);
  auto by = buffer(static_cast<char*>(p.y) + base * esz, live * p.D * esz);
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = fmaf(P[v], state[v], L[v]);
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = fmaf(w[i][v], h[v], a[i][v]);
    store<F32, VEC>(by, xoff + i * p.D * esz, h);
  }
  if (live < end) {  // zeros behind the sequence's end
    const float none[VEC] = {};
    by = buffer(static_cast<char*>(p.y) + base * esz, end * p.D * esz);
#pragma unroll 1
    for (int i = 0; i < kTok; ++i)
      if (group * kTok + i >= live) store<F32, VEC>(by, xoff + i * p.D * esz, none);
  }
}

// Gradients in one pass, for at most kAcross<VEC> tiles a sequence: a workgroup a tile, a sequence's (of 64 channels) tiles
// in a row. Every tile needs the maps of those before it and, for the gradient, of those behind it, whose workgroups
// start later. So a workgroup looks for them `polls` times, some 100 us, and where one is not there (other work holds
// the compute units) leaves its tile to a second kernel, before which all maps are: no wait depends on another
// workgroup, and the results are the same.
template <int VEC>
constexpr uint32_t kAcross = VEC == 4 ? 160 : 64;
template <bool F32, int VEC, int KIND>
__device__ __forceinline__ void across(const ScanParams& p, uint32_t id, bool again) {
  constexpr uint32_t esz = kEsz<F32>;
  constexpr int tile = kTile<VEC>;
  constexpr uint32_t kAtOnce = 8;  // maps that a wave looks for at once
  __shared__ Shared<> sh[2];
  __shared__ float4 parked[VEC][kThreads];
  const uint32_t unit = id / p.tiles, k = id % p.tiles;
  const uint32_t slab = unit % p.slabs, b = unit / p.slabs;
  const uint32_t lc = threadIdx.x % kLanes<VEC> * VEC, c = channel<VEC>(slab * kSlab + lc, p.D), group = threadIdx.x / kLanes<VEC>;
  const bool on = c < p.D;
  const uint32_t at = group * kTok * p.D + c;
  const uint32_t xoff = on ? at * esz : kNowhere, woff = on ? at * 4 : kNowhere;
  const int64_t len = length(p, b);
  const uint64_t row = (uint64_t)p.units * kSlab, word = (uint64_t)unit * kSlab;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t each = (p.tiles + kWaves - 1) / kWaves;  // tiles whose maps a wave reads, in a row, a channel a lane

  const int64_t t0 = (int64_t)k * tile, base = ((int64_t)b * p.T + t0) * p.D;
  const uint32_t end = (uint32_t)(p.T - t0 < tile ? p.T - t0 : tile);
  const uint32_t live = len - t0 < 0 ? 0 : len - t0 < end ? (uint32_t)(len - t0) : end;
  const auto bx = buffer(static_cast<const char*>(p.x) + base * esz, live * p.D * esz);
  const auto bg = buffer(static_cast<const char*>(p.dy) + base * esz, live * p.D * esz);
  const auto bw = buffer(p.log_w + base, live * p.D * 4);
  Raw<F32, VEC> rx[kTok], rg[kTok];
  Raw<true, VEC> rw[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    rw[i] = load<true, VEC>(bw, woff + i * p.D * 4);
    rx[i] = load<F32, VEC>(bx, xoff + i * p.D * esz);
    rg[i] = load<F32, VEC>(bg, xoff + i * p.D * esz);
  }
  __builtin_amdgcn_sched_barrier(0);  // all loads before the first that is waited for
  float w[kTok][VEC], s[kTok][VEC], P[VEC], L[VEC], Q[VEC], R[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) P[v] = 1.f, L[v] = R[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i) add_token<F32, VEC, KIND>(rx[i], rg[i], rw[i], w[i], s[i], P, L, R);
#pragma unroll
  for (int v = 0; v < VEC; ++v) Q[v] = P[v];
  maps_of_wave<VEC, false>(P, L, sh[0].p[0], sh[0].l[0]);
  maps_of_wave<VEC, true>(Q, R, sh[0].p[1], sh[0].l[1]);
  lds_barrier();
  // what this thread's tokens need of the tile's other threads, out of the registers while others' maps are looked for
#pragma unroll
  for (int v = 0; v < VEC; ++v) parked[v][threadIdx.x] = make_float4(P[v], L[v], Q[v], R[v]);
  float fp = 1.f, fl = 0.f, gp = 1.f, gl = 0.f;
  if (p.tiles > 1) {
    if (wave < 2 && !again) {
      float q, l;
      if (wave == 0) whole_map<false, kWaves>(sh[0].p[0], sh[0].l[0], q, l);
      else whole_map<true, kWaves>(sh[0].p[1], sh[0].l[1], q, l);
      publish((wave == 0 ? p.there : p.back) + k * row + word + lane, q, l);
    }
    uint32_t missing = 0;
    int polls = p.polls;  // for all of them together
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < each && missing == 0; i0 += kAtOnce) {
      // all looked for at once, without a branch between them: this tile's own in the place of those it does not need
      uint64_t m[kAtOnce];
      auto tile_of = [&](uint32_t i) { return wave * each + i0 + i; };
      auto other = [&](uint32_t i) { return (uint32_t)(i0 + i < each) & (uint32_t)(tile_of(i) < p.tiles) & (uint32_t)(tile_of(i) != k); };
      auto from = [&](uint32_t i) {
        const uint32_t o = other(i) ? tile_of(i) : k;
        return (o < k ? p.there : p.back) + o * row + word + lane;
      };
#pragma unroll 1
      for (;; --polls) {
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) m[i] = peek(from(i));
        missing = 0;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) missing = missing | (other(i) & (uint32_t)(m[i] == kEmpty));
        if (missing == 0 || polls <= 0) break;
        __builtin_amdgcn_s_sleep(4);
      }
#pragma unroll
      for (uint32_t i = 0; i < kAtOnce; ++i) {
        const float q = __uint_as_float((uint32_t)m[i]), l = __uint_as_float((uint32_t)(m[i] >> 32));
        const bool in_front = other(i) & (uint32_t)(tile_of(i) < k), behind = other(i) & (uint32_t)(tile_of(i) > k);
        fl = fmaf(in_front ? q : 1.f, fl, in_front ? l : 0.f);
        fp *= in_front ? q : 1.f;
        gl = fmaf(gp, behind ? l : 0.f, gl);  // what comes back passes the tiles in front last
        gp *= behind ? q : 1.f;
      }
    }
    if (!again && __syncthreads_or((int)missing)) {
      if (threadIdx.x == 0) {
        const uint32_t n = atomicAdd(p.left, 1u);
        if (n < p.units * p.tiles) p.left[1 + n] = id;  // (always, but for calls that share a workspace against the rules)
      }
      return;
    }
  }

  sh[1].p[0][wave][lane] = fp;
  sh[1].l[0][wave][lane] = fl;
  sh[1].p[1][wave][lane] = gp;
  sh[1].l[1][wave][lane] = gl;
  float state[VEC] = {}, grad[VEC] = {}, h[VEC], g[VEC], end_grad = 0.f;
  const uint32_t lane_c = channel_at<VEC>(slab * kSlab + lane, p.D);
  const int64_t of_b = (int64_t)b * p.D;
  if (p.tiles > 1) {
    get<VEC>(p.first_state + word + lc, state);
    get<VEC>(p.last_grad + word + lc, grad);
    end_grad = p.last_grad[word + lane];
  } else {
    if (on && p.s_in) get_any<VEC>(p.s_in + of_b + c, state);
    if (on && p.ds_out) get_any<VEC>(p.ds_out + of_b + c, grad);
    if (lane_c < p.D && p.ds_out) end_grad = p.ds_out[of_b + lane_c];
  }
  __syncthreads();  // ds_out has been read, before ds_in, which it may be, is written
  if (k == 0 && wave == 0 && p.ds_in && lane_c < p.D) {
    float q, l, d[1] = {end_grad};
    pass<1, true, kWaves, !F32>(sh[1].p[1], sh[1].l[1], lane, d);
    whole_map<true, kWaves>(sh[0].p[1], sh[0].l[1], q, l);
    p.ds_in[of_b + lane_c] = fmaf(q, d[0], l);
  }
  pass<VEC, false, kWaves, !F32>(sh[1].p[0], sh[1].l[0], lc, state);
  pass<VEC, true, kWaves, !F32>(sh[1].p[1], sh[1].l[1], lc, grad);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float4 f = parked[v][threadIdx.x];
    P[v] = f.x, L[v] = f.y, Q[v] = f.z, R[v] = f.w;
  }
  compose<VEC, false, kWaves, !F32>(P, L, sh[0].p[0], sh[0].l[0]);
  compose<VEC, true, kWaves, !F32>(Q, R, sh[0].p[1], sh[0].l[1]);
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = fmaf(P[v], state[v], L[v]), g[v] = fmaf(Q[v], grad[v], R[v]);
  write_grads<F32, VEC, KIND>(p, base, end, live, group, xoff, woff, rx, rg, w, s, h, g);
}

template <bool F32, int VEC, int KIND>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void gscan_across_kernel(ScanParams p) {
  across<F32, VEC, KIND>(p, p.first + blockIdx.x, false);
}
template <bool F32, int VEC, int KIND>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void gscan_left_kernel(ScanParams p) {
  const uint32_t all = p.units * p.tiles, listed = *p.left, n = listed < all ? listed : all;
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint32_t id = p.left[1 + i];
    if (id < all) across<F32, VEC, KIND>(p, id, true);
    __syncthreads();  // LDS is written again
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
  const uint32_t each = (p.tiles + 15) / 16, s0 = wave * each < p.tiles ? wave * each : p.tiles;
  const uint32_t s1 = s0 + each < p.tiles ? s0 + each : p.tiles;
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
  if (p.s_in) get<VEC>(p.s_in + i, s);  // here four channels begin on 16 bytes
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
  if (p.s_out) put_any<VEC>(p.s_out + i, s);
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

hipError_t start(const void* fn, uint64_t blocks, int threads, ScanParams p, hipStream_t stream) {
  return static_cast<hipError_t>(in_chunks(blocks, threads, [&](uint32_t first, uint32_t n) {
    p.first = first;
    void* args[] = {&p};
    return static_cast<int>(hipLaunchKernel(fn, dim3(n), dim3(threads), args, 0, stream));
  }));
}

ScanParams params(const GscanCall& c) {
  ScanParams p{};
  p.x = c.x, p.log_w = c.log_w, p.s_in = c.s_in, p.lens = c.lens, p.y = c.y, p.s_out = c.s_out;
  p.dy = c.dy, p.dx = c.dx, p.dlog_w = c.dlog_w, p.ds_out = c.ds_out, p.ds_in = c.ds_in;
  p.T = c.T, p.BD = c.B * c.D, p.B = (uint32_t)c.B, p.D = (uint32_t)c.D;
  p.slabs = (p.D + kSlab - 1) / kSlab;
  p.units = p.B * p.slabs;
  return p;
}

// Polls of a workgroup for the others' maps before it leaves its tile to the second kernel.
std::atomic<int> g_polls{64};

// The words that workgroups pass on, in the workspace: `rows` of them for each unit's 64 channels, a second array of as
// many for the gradient, copies of the states, and the number of workgroups. The caller holds the operators' lock.
hipError_t words(ScanParams& p, const GscanCall& c, uint64_t rows, bool back) {
  const uint64_t row = (uint64_t)p.units * kSlab, n = rows * row * (back ? 2 : 1);
  void* ws = nullptr;
  const size_t list = back ? ((size_t)p.units * p.tiles + 1) * 4 : 4;
  const hipError_t e = device_workspace(c.stream, n * 8 + 2 * row * 4 + 4 + list, &ws, kWorkspaceOperators);
  if (e != hipSuccess) return e;
  p.there = static_cast<uint64_t*>(ws), p.back = back ? p.there + rows * row : nullptr, p.words = n;
  p.first_state = reinterpret_cast<float*>(p.there + n), p.last_grad = back ? p.first_state + row : nullptr;
  p.ticket = reinterpret_cast<uint32_t*>(p.first_state + 2 * row), p.left = p.ticket + 1;
  p.polls = g_polls.load(std::memory_order_relaxed);
  const uint64_t blocks = (n / 4 + 255) / 256;
  return start(reinterpret_cast<const void*>(&gscan_empty_kernel), blocks < 1024 ? (blocks ? blocks : 1) : 1024, 256, p, c.stream);
}

template <bool F32, int VEC, int KIND>
struct Kernels {
  static constexpr int tile = kTile<VEC>;
  // Whether a prompt of so many units is walked, in `tiles`, or passes maps on, in `chain_tiles`.
  // In fours walking takes 2 us a tile (128 tokens) or, from 192 units on, the memory's time; passing maps on 3 us for
  // emptying their words and then the memory's time, at some 5 TB/s with any number of units: B=8 T=4096 D=1024 (128 units)
  // 72 and 54 us, B=1 T=8192 D=768 (12) 134 and 19, B=16 T=2048 D=768 (192) 41 and 44, B=1 T=256 D=768 7.2 and 9.4, B=8
  // T=4096 D=4096 (512) 219 and 205.
  // By single channels a tile has 32 tokens and takes 0.6 us to walk, one after the other, 1.0 to 1.2 where the inputs come from
  // memory and not from the last-level cache; a tile of 64 that passes its maps on takes 0.014 us of the device's time,
  // after 6 us. From memory, MIX, bfloat16: D=65 with 16 units T=512 14 and 8 us, 64 units T=2048 67 and 37, 128 units T=512
  // 20 and 23, T=4096 138 and 112, 192 units T=4096 148 and 162, 512 units T=1024 54 and 112; float32 D=1025 B=8 (136)
  // T=1024 44 and 46, T=4096 167 and 135, from the cache T=2048 44 and 70.
  static bool walks(uint32_t units, uint32_t tiles, uint32_t chain_tiles) {
    if (VEC == 4) return tiles <= 3 || (units >= 192 && tiles <= 16);
    return 80 * ((int64_t)tiles - 7) <= (int64_t)units * chain_tiles;
  }
  static hipError_t prefill(const GscanCall& c) {
    ScanParams p = params(c);
    const uint32_t tiles = (uint32_t)((c.T + tile - 1) / tile);
    const uint32_t chain_tiles = (uint32_t)((c.T + kTile<VEC, kChainWaves> - 1) / kTile<VEC, kChainWaves>);
    if (walks(p.units, tiles, chain_tiles))
      return start(reinterpret_cast<const void*>(&gscan_walk_kernel<F32, VEC, KIND>), p.units, kThreads, p, c.stream);
    p.tiles = chain_tiles;
    std::lock_guard<std::mutex> lock(operators_mutex());
    const hipError_t e = words(p, c, (uint64_t)p.tiles + (p.tiles + kGroup - 1) / kGroup, false);
    if (e != hipSuccess) return e;
    return start(reinterpret_cast<const void*>(&gscan_chain_kernel<F32, VEC, KIND, kChainWaves>), (uint64_t)p.units * p.tiles,
                 kChainWaves * kWave, p, c.stream);
  }
  static hipError_t step(const GscanCall& c) {
    const ScanParams p = params(c);
    const int64_t threads = (p.BD + VEC - 1) / VEC;
    return start(reinterpret_cast<const void*>(&gscan_step_kernel<F32, VEC, KIND>), (uint64_t)(threads + kThreads - 1) / kThreads,
                 kThreads, p, c.stream);
  }
  static hipError_t backward(const GscanCall& c) {
    ScanParams p = params(c);
    p.tiles = (uint32_t)((c.T + tile - 1) / tile);
    const uint64_t blocks = (uint64_t)p.units * p.tiles;
    const void* join = reinterpret_cast<const void*>(&gscan_join_kernel);
    const void* one_pass = reinterpret_cast<const void*>(&gscan_across_kernel<F32, VEC, KIND>);
    if (p.tiles == 0) return start(join, p.units, 1024, p, c.stream);
    if (p.tiles == 1) return start(one_pass, blocks, kThreads, p, c.stream);
    std::lock_guard<std::mutex> lock(operators_mutex());
    hipError_t e = hipSuccess;
    // In one pass or two, bfloat16: B=8 T=4096 D=1024 (32 tiles) 107 and 146 us, B=4 T=8192 D=2048 (64) 224 and 290, B=4 T=16384
    // D=1024 (128) 283 and 306, T=20480 (160) 340 and 371, T=32768 (256) 623 and 588; B=1 D=1024 T=16384 63 and 69, T=20480 93
    // and 86, T=24576 118 and 101; float32 B=4 D=1024 (96) 244 and 325, (160) 455 and 529, (192) 664 and 627: every tile
    // reads all others' maps. (Words are of 64 channels and would outgrow the data of one to three; of 8 B=512 T=4096 takes
    // 184 and 158.) Single channels, with tiles of 32 tokens: B=8 T=1024 D=1025 (32) 38 and 52, B=4 T=2048 (64) 45 and 52,
    // float32 50 and 64; a few units of a few tiles 9.6 and 8.6; D=65 B=128 T=2048 125 and 101, the most that the rule loses there.
    if (p.tiles <= kAcross<VEC> && p.D >= 16) {
      e = words(p, c, p.tiles, true);
      if (e == hipSuccess) e = start(one_pass, blocks, kThreads, p, c.stream);
      if (e == hipSuccess)
        e = start(reinterpret_cast<const void*>(&gscan_left_kernel<F32, VEC, KIND>), blocks < 256 ? blocks : 256, kThreads, p, c.stream);
      return e;
    }
    void* ws = nullptr;
    e = device_workspace(c.stream, (size_t)3 * p.tiles * p.BD * 4, &ws, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    p.p = static_cast<float*>(ws), p.l = p.p + p.tiles * p.BD, p.r = p.l + p.tiles * p.BD;
    e = start(reinterpret_cast<const void*>(&gscan_grad_kernel<F32, VEC, KIND, true>), blocks, kThreads, p, c.stream);
    if (e == hipSuccess) e = start(join, p.units, 1024, p, c.stream);
    if (e == hipSuccess)
      e = start(reinterpret_cast<const void*>(&gscan_grad_kernel<F32, VEC, KIND, false>), blocks, kThreads, p, c.stream);
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
// Four channels a thread, or one: also in a step whose states are no multiple of four (no two threads may have the same
// channel there, as it may be updated in place).
hipError_t dispatch(const GscanCall& c, Op op) {
  const bool four = op == Op::kStep ? c.B * c.D % 4 == 0 : in_fours((uint32_t)c.D);
  if (c.f32) return four ? by_kind<true, 4>(c, op) : by_kind<true, 1>(c, op);
  return four ? by_kind<false, 4>(c, op) : by_kind<false, 1>(c, op);
}

}  // namespace

void set_gscan_polls(int polls) { g_polls.store(polls, std::memory_order_relaxed); }

hipError_t launch_gscan_prefill(const GscanCall& c) { return dispatch(c, Op::kPrefill); }
hipError_t launch_gscan_step(const GscanCall& c) { return dispatch(c, Op::kStep); }
hipError_t launch_gscan_backward(const GscanCall& c) { return dispatch(c, Op::kBackward); }

}  // namespace rwkv7
