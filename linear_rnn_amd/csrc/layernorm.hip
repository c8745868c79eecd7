// Layer norm over groups of channels, forward and backward with the reduction of the weight's and the
// bias's gradients.
//
// x is [M, D] with D = G n: every row has G groups of n consecutive channels with a mean and a variance
// each (G = 1: layer norm; G = heads, n = 64: ln_x). For one group, xh = (x - mean) rstd:
//   y  = xh w + b,                 mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   dx = rstd (g - sum g / n - xh sum(g xh) / n),     g = dy w
//   dw = sum over rows of dy xh,   db = sum over rows of dy
// Everything is read once and written once, so memory bounds all of it. A group lives in the registers of
// L threads (NV vectors of VEC channels each), so that the variance is the two-pass one, and a thread
// keeps its channels for all the rows it takes: weights are read once, and the sums over rows of dw and
// db stay in registers until the end. A workgroup covers S groups of R rows at a time; the sums of its R
// rows meet in LDS, those of the workgroups in a second kernel, always in the same order.
// All statistics and sums are float32; bfloat16 outputs are rounded once.
// [32768, 768] float32 to bfloat16 27.8 us (5.4 TB/s); gradients of [16384, 4096] bfloat16 78 us (5.2), of [8191, 1024]
// float32 in 16 groups 23.3 us (4.3).
#include "lane_sums.hpp"
#include "layernorm_internal.hpp"
#include "operators_lock.hpp"
#include "wkv7_device.hpp"
#include "wkv7_internal.hpp"

namespace rwkv7 {
namespace {

struct NormParams {
  const void* x;
  const float* weight;  // may be null (1)
  const float* bias;    // may be null (0)
  void* y;              // forward
  float* mean;          // [M, G]: written by the forward (may be null), read by the backward
  float* rstd;
  const void* dy;   // backward
  void* dx;
  float* partial;   // [2][nb][D]: sums of dy xh and of dy over a workgroup's rows; null: not asked for
  int64_t M;
  int32_t D, G, n;
  int32_t S, R;     // groups and rows of a workgroup
  int32_t slabs;    // workgroups side by side over a row's groups
  int32_t nb;       // workgroups over the rows
  float eps;
};

// VEC channels as loaded, and as float32.
template <bool F32, int VEC>
struct Raw;
template <>
struct Raw<true, 8> {
  float4 a, b;
};
template <>
struct Raw<false, 8> {
  uint4 a;
};
template <>
struct Raw<true, 1> {
  float a;
};
template <>
struct Raw<false, 1> {
  uint16_t a;
};
template <bool F32, int VEC>
__device__ __forceinline__ Raw<F32, VEC> load_raw(const void* base, int64_t at) {
  if constexpr (VEC == 8 && F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    return {p[0], p[1]};
  } else if constexpr (VEC == 8) {
    return {*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at)};
  } else if constexpr (F32) {
    return {static_cast<const float*>(base)[at]};
  } else {
    return {static_cast<const uint16_t*>(base)[at]};
  }
}
template <bool F32, int VEC>
__device__ __forceinline__ void widen(const Raw<F32, VEC>& r, float (&o)[VEC]) {
  if constexpr (VEC == 8 && F32) {
    o[0] = r.a.x, o[1] = r.a.y, o[2] = r.a.z, o[3] = r.a.w, o[4] = r.b.x, o[5] = r.b.y, o[6] = r.b.z, o[7] = r.b.w;
  } else if constexpr (VEC == 8) {
    o[0] = bf16_lo(r.a.x), o[1] = bf16_hi(r.a.x), o[2] = bf16_lo(r.a.y), o[3] = bf16_hi(r.a.y);
    o[4] = bf16_lo(r.a.z), o[5] = bf16_hi(r.a.z), o[6] = bf16_lo(r.a.w), o[7] = bf16_hi(r.a.w);
  } else if constexpr (F32) {
    o[0] = r.a;
  } else {
    o[0] = __uint_as_float((uint32_t)r.a << 16);
  }
}
template <bool F32, int VEC>
__device__ __forceinline__ void load_vec(const void* base, int64_t at, float (&o)[VEC]) {
  widen<F32, VEC>(load_raw<F32, VEC>(base, at), o);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {  // round to nearest even
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
}
template <bool F32, int VEC>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&o)[VEC]) {
  if constexpr (VEC == 8 && F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(o[0], o[1], o[2], o[3]);
    p[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]), bf16_pair(o[4], o[5]), bf16_pair(o[6], o[7]));
  } else if constexpr (F32) {
    static_cast<float*>(base)[at] = o[0];
  } else {
    static_cast<uint16_t*>(base)[at] = __builtin_bit_cast(uint16_t, (__bf16)o[0]);
  }
}

// Sums over the L threads of a group, the same bits in each of them. L over 64: through LDS with a barrier, so
// every thread of the workgroup calls it; consecutive calls take the halves of `red` (two floats for each wave and
// half) in turn, so that one barrier is enough.
template <int L>
__device__ __forceinline__ float wave_sum(float x) {  // butterflies of the vector unit, no LDS
  static_assert(L >= 8, "");
  if constexpr (L >= 16) x = x + dpp_f32<0x128>(x);  // row_ror:8
  x = x + dpp_f32<0x141>(x);                         // row_half_mirror
  x = x + dpp_f32<0x4E>(x);                          // quad_perm [2,3,0,1]
  x = x + dpp_f32<0xB1>(x);                          // quad_perm [1,0,3,2]
  if constexpr (L >= 32) x = pair_rows_sum(x);
  if constexpr (L >= 64) x = halves_sum(x);
  return x;
}
template <int L>
__device__ __forceinline__ void group_sum2(float& a, float& b, float2 (*red)[16], int& turn) {
  a = wave_sum<L>(a);
  b = wave_sum<L>(b);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[turn][wave] = make_float2(a, b);
    lds_barrier();
    const int w0 = wave / W * W;
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) a += red[turn][w0 + w].x, b += red[turn][w0 + w].y;
    turn ^= 1;
  }
}
template <int L>
__device__ __forceinline__ float group_sum(float a, float2 (*red)[16], int& turn) {
  float b = 0.f;
  group_sum2<L>(a, b, red, turn);
  return a;
}

// Threads of a workgroup whose threads hold NV vectors each. Groups of eight waves go two to a workgroup where the
// registers allow it: half as many rows of partial sums.
template <int L, int NV>
constexpr int kBlock = L > 256 ? (NV == 1 ? 1024 : L) : 256;

// A thread's place: its group of the row, its first row, its channels.
template <int L>
struct Place {
  int lane, group, chunk;
  int64_t row, stride;
  bool on;
  __device__ __forceinline__ explicit Place(const NormParams& p) {
    const int slot = threadIdx.x / L;
    lane = threadIdx.x % L;
    chunk = blockIdx.x / p.slabs;
    const int s = slot % p.S, r = slot / p.S;
    group = (blockIdx.x % p.slabs) * p.S + s;
    on = r < p.R && group < p.G;
    if (!on) group = 0;
    row = (int64_t)chunk * p.R + r;
    stride = (int64_t)p.nb * p.R;
  }
};

template <bool XF, bool YF, int VEC, int L, int NV>
__global__ __launch_bounds__((kBlock<L, NV>)) void layernorm_forward_kernel(NormParams p) {
  __shared__ float2 red[2][16];
  int turn = 0;
  const Place<L> at(p);
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * L + at.lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[v][i] = 1.f, b[v][i] = 0.f;
    if (c < p.n) {
      if (p.weight) load_vec<true, VEC>(p.weight, (int64_t)at.group * p.n + c, w[v]);
      if (p.bias) load_vec<true, VEC>(p.bias, (int64_t)at.group * p.n + c, b[v]);
    }
  }
  const float inv = 1.f / (float)p.n;
  // The next row's loads are in flight while this one is summed. A thread without a row or channels of its own
  // loads what the first has, and its values count as 0.
  Raw<XF, VEC> x0[NV];
  auto load = [&](int64_t m) {
    const int64_t base = (at.on && m < p.M ? m : 0) * p.D + (int64_t)at.group * p.n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      x0[v] = load_raw<XF, VEC>(p.x, base + (c < p.n ? c : 0));
    }
  };
  load(at.row);
  // every thread of the workgroup takes the same number of turns (the sums may hold barriers)
  for (int64_t m0 = (int64_t)at.chunk * p.R; m0 < p.M; m0 += at.stride) {
    const int64_t m = at.row + (m0 - (int64_t)at.chunk * p.R);
    const bool on = at.on && m < p.M;
    float x[NV][VEC], sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      widen<XF, VEC>(x0[v], x[v]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += c < p.n ? x[v][i] : 0.f;
    }
    load(m + at.stride);
    const float mean = group_sum<L>(sum, red, turn) * inv;
    float sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        x[v][i] -= mean;
        sq += c < p.n ? x[v][i] * x[v][i] : 0.f;
      }
    }
    const float rstd = 1.f / sqrtf(group_sum<L>(sq, red, turn) * inv + p.eps);
    if (!on) continue;
    if (at.lane == 0) {
      if (p.mean) p.mean[m * p.G + at.group] = mean;
      if (p.rstd) p.rstd[m * p.G + at.group] = rstd;
    }
    const int64_t base = m * p.D + (int64_t)at.group * p.n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      if (c < p.n) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[v][i] = x[v][i] * rstd * w[v][i] + b[v][i];
        store_vec<YF, VEC>(p.y, base + c, x[v]);
      }
    }
  }
}

template <bool XF, bool YF, int VEC, int L, int NV>
__global__ __launch_bounds__((kBlock<L, NV>)) void layernorm_backward_kernel(NormParams p) {
  constexpr int kThreads = kBlock<L, NV>;
  __shared__ float2 red[2][16];
  __shared__ float rows[NV * VEC][kThreads];
  int turn = 0;
  const Place<L> at(p);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * L + at.lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[v][i] = 1.f, dw[v][i] = 0.f, db[v][i] = 0.f;
    if (c < p.n && p.weight) load_vec<true, VEC>(p.weight, (int64_t)at.group * p.n + c, w[v]);
  }
  const float inv = 1.f / (float)p.n;
  Raw<XF, VEC> x0[NV];  // the next row, as in the forward
  Raw<YF, VEC> g0[NV];
  float mean0, rstd0;
  auto load = [&](int64_t m) {
    m = at.on && m < p.M ? m : 0;
    const int64_t base = m * p.D + (int64_t)at.group * p.n;
    mean0 = p.mean[m * p.G + at.group], rstd0 = p.rstd[m * p.G + at.group];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      x0[v] = load_raw<XF, VEC>(p.x, base + (c < p.n ? c : 0));
      g0[v] = load_raw<YF, VEC>(p.dy, base + (c < p.n ? c : 0));
    }
  };
  load(at.row);
  for (int64_t m0 = (int64_t)at.chunk * p.R; m0 < p.M; m0 += at.stride) {
    const int64_t m = at.row + (m0 - (int64_t)at.chunk * p.R);
    const bool on = at.on && m < p.M;
    const float mean = mean0, rstd = rstd0;
    float x[NV][VEC], g[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      widen<XF, VEC>(x0[v], x[v]);
      widen<YF, VEC>(g0[v], g[v]);
      const bool counts = on && c < p.n;
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[v][i] = counts ? (x[v][i] - mean) * rstd : 0.f, g[v][i] = counts ? g[v][i] : 0.f;
    }
    load(m + at.stride);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[v][i] = fmaf(g[v][i], x[v][i], dw[v][i]);
        db[v][i] += g[v][i];
        g[v][i] *= w[v][i];
        s1 += g[v][i];
        s2 = fmaf(g[v][i], x[v][i], s2);
      }
    group_sum2<L>(s1, s2, red, turn);
    s1 *= inv;
    s2 *= inv;
    if (!on) continue;
    const int64_t base = m * p.D + (int64_t)at.group * p.n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      if (c < p.n) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[v][i] = rstd * (g[v][i] - s1 - x[v][i] * s2);
        store_vec<XF, VEC>(p.dx, base + c, g[v]);
      }
    }
  }
  if (!p.partial) return;
  // the workgroup's rows r = 0 .. R - 1 in this order, then its row of the partial sums
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) rows[v * VEC + i][threadIdx.x] = which ? db[v][i] : dw[v][i];
    __syncthreads();
    if (!at.on || threadIdx.x >= p.S * L) continue;
    float* out = p.partial + ((int64_t)which * p.nb + at.chunk) * p.D + (int64_t)at.group * p.n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + at.lane) * VEC;
      if (c >= p.n) continue;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float s = rows[v * VEC + i][threadIdx.x];
        for (int r = 1; r < p.R; ++r) s += rows[v * VEC + i][threadIdx.x + r * p.S * L];
        out[c + i] = s;
      }
    }
  }
}

// Groups too long for registers: a workgroup reads its group once for each pass (from the caches mostly).
template <bool XF, bool YF>
__global__ __launch_bounds__(1024) void layernorm_forward_long_kernel(NormParams p) {
  __shared__ float2 red[2][16];
  int turn = 0;
  const float inv = 1.f / (float)p.n;
  const int64_t units = p.M * p.G;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t base = u * p.n, wb = u % p.G * p.n;
    float sum = 0.f, v[1];
    for (int c = threadIdx.x; c < p.n; c += 1024) load_vec<XF, 1>(p.x, base + c, v), sum += v[0];
    const float mean = group_sum<1024>(sum, red, turn) * inv;
    float sq = 0.f;
    for (int c = threadIdx.x; c < p.n; c += 1024) load_vec<XF, 1>(p.x, base + c, v), sq += (v[0] - mean) * (v[0] - mean);
    const float rstd = 1.f / sqrtf(group_sum<1024>(sq, red, turn) * inv + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[u] = mean;
      if (p.rstd) p.rstd[u] = rstd;
    }
    for (int c = threadIdx.x; c < p.n; c += 1024) {
      load_vec<XF, 1>(p.x, base + c, v);
      const float w = p.weight ? p.weight[wb + c] : 1.f, b = p.bias ? p.bias[wb + c] : 0.f;
      const float o[1] = {(v[0] - mean) * rstd * w + b};
      store_vec<YF, 1>(p.y, base + c, o);
    }
  }
}
template <bool XF, bool YF>
__global__ __launch_bounds__(1024) void layernorm_backward_long_kernel(NormParams p) {
  __shared__ float2 red[2][16];
  int turn = 0;
  const float inv = 1.f / (float)p.n;
  const int64_t units = p.M * p.G;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t base = u * p.n, wb = u % p.G * p.n;
    const float mean = p.mean[u], rstd = p.rstd[u];
    float s1 = 0.f, s2 = 0.f, x[1], d[1];
    for (int c = threadIdx.x; c < p.n; c += 1024) {
      load_vec<XF, 1>(p.x, base + c, x);
      load_vec<YF, 1>(p.dy, base + c, d);
      const float g = d[0] * (p.weight ? p.weight[wb + c] : 1.f);
      s1 += g;
      s2 = fmaf(g, (x[0] - mean) * rstd, s2);
    }
    group_sum2<1024>(s1, s2, red, turn);
    s1 *= inv;
    s2 *= inv;
    for (int c = threadIdx.x; c < p.n; c += 1024) {
      load_vec<XF, 1>(p.x, base + c, x);
      load_vec<YF, 1>(p.dy, base + c, d);
      const float g = d[0] * (p.weight ? p.weight[wb + c] : 1.f);
      const float o[1] = {rstd * (g - s1 - (x[0] - mean) * rstd * s2)};
      store_vec<XF, 1>(p.dx, base + c, o);
    }
  }
}
// Their sums over rows: a thread a channel, rows chunk, chunk + nb, ...
template <bool XF, bool YF>
__global__ __launch_bounds__(256) void layernorm_columns_kernel(NormParams p) {
  const int64_t c = (int64_t)(blockIdx.x / p.nb) * 256 + threadIdx.x;
  const int chunk = blockIdx.x % p.nb;
  if (c >= p.D) return;
  const int group = (int)(c / p.n);
  float dw = 0.f, db = 0.f, x[1], d[1];
  for (int64_t m = chunk; m < p.M; m += p.nb) {
    load_vec<XF, 1>(p.x, m * p.D + c, x);
    load_vec<YF, 1>(p.dy, m * p.D + c, d);
    const float xh = (x[0] - p.mean[m * p.G + group]) * p.rstd[m * p.G + group];
    dw = fmaf(d[0], xh, dw);
    db += d[0];
  }
  p.partial[(int64_t)chunk * p.D + c] = dw;
  p.partial[((int64_t)p.nb + chunk) * p.D + c] = db;
}

// dweight and dbias from the partial rows: 64 channels a workgroup, 16 of its threads a channel.
__global__ __launch_bounds__(1024) void layernorm_join_kernel(const float* partial, float* dweight, float* dbias, int32_t nb,
                                                              int32_t D) {
  __shared__ float part[16][64];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int k = threadIdx.x >> 6;
  float s = 0.f;
  if (c < D) {
    const float* src = partial + (int64_t)blockIdx.y * nb * D + c;
#pragma unroll 16
    for (int i = k; i < nb; i += 16) s += src[(int64_t)i * D];
  }
  part[k][threadIdx.x & 63] = s;
  __syncthreads();
  if (k == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][threadIdx.x];
    out[c] = s;
  }
}

struct Config {
  const void* fn;
  int L, threads;
};
template <bool BWD, bool XF, bool YF, int VEC, int L, int NV>
Config config() {
  if constexpr (BWD) return {reinterpret_cast<const void*>(&layernorm_backward_kernel<XF, YF, VEC, L, NV>), L, kBlock<L, NV>};
  else return {reinterpret_cast<const void*>(&layernorm_forward_kernel<XF, YF, VEC, L, NV>), L, kBlock<L, NV>};
}
// The threads of a group: as few as hold it in 16 registers each, or 8 where two rows share a workgroup (so that a wave takes several short
// groups and a row of weights is spread over few threads), in vectors of 8 channels where every group
// starts on 16 bytes. 1024 threads have 128 registers each, which the gradients of a long group pass by a little:
// M=4096 n=16384 bfloat16 still 135 us, 234 by the long kernels, but channel by channel n=16380 403 against 234.
template <bool BWD, bool XF, bool YF>
Config pick(int n) {
  if (n % 8 == 0) {
    if (n <= 64) return config<BWD, XF, YF, 8, 8, 1>();
    if (n <= 128) return config<BWD, XF, YF, 8, 16, 1>();
    if (n <= 256) return config<BWD, XF, YF, 8, 32, 1>();
    if (n <= 512) return config<BWD, XF, YF, 8, 64, 1>();
    if (n <= 1024) return config<BWD, XF, YF, 8, 64, 2>();
    if (n <= 2048) return config<BWD, XF, YF, 8, 128, 2>();
    if (n <= 4096) return config<BWD, XF, YF, 8, 512, 1>();
    if (n <= 8192) return config<BWD, XF, YF, 8, 1024, 1>();
    if (n <= 16384) return config<BWD, XF, YF, 8, 1024, 2>();
  } else {
    if (n <= 16) return config<BWD, XF, YF, 1, 16, 1>();
    if (n <= 64) return config<BWD, XF, YF, 1, 16, 4>();
    if (n <= 256) return config<BWD, XF, YF, 1, 64, 4>();
    if (n <= 1024) return config<BWD, XF, YF, 1, 64, 16>();
    if (n <= 2048) return config<BWD, XF, YF, 1, 128, 16>();
    if (n <= 4096) return config<BWD, XF, YF, 1, 256, 16>();
    if (n <= 8192) return config<BWD, XF, YF, 1, 512, 16>();
    if constexpr (!BWD)
      if (n <= 16384) return config<BWD, XF, YF, 1, 1024, 16>();
  }
  return {nullptr, 0, 0};
}

hipError_t start(const void* fn, int64_t blocks, int threads, NormParams& p, hipStream_t stream) {
  void* args[] = {&p};
  return hipLaunchKernel(fn, dim3((uint32_t)blocks), dim3(threads), args, 0, stream);
}

NormParams params(const NormCall& c) {
  NormParams p{};
  p.x = c.x, p.weight = c.weight, p.bias = c.bias, p.y = c.y, p.mean = c.mean, p.rstd = c.rstd, p.dy = c.dy, p.dx = c.dx;
  p.M = c.M, p.D = (int32_t)c.D, p.G = (int32_t)c.G, p.n = (int32_t)(c.D / c.G), p.eps = c.eps;
  return p;
}
// Workgroups: of `most` threads together, no more than there are rows for.
void spread(NormParams& p, const Config& f, int64_t most) {
  const int slots = f.threads / f.L;
  p.S = p.G < slots ? p.G : slots;
  p.R = slots / p.S;
  p.slabs = (p.G + p.S - 1) / p.S;
  int64_t nb = most / f.threads / p.slabs;
  const int64_t rows = (p.M + p.R - 1) / p.R;
  if (nb > rows) nb = rows;
  p.nb = (int32_t)(nb < 1 ? 1 : nb);
}

template <bool XF, bool YF>
hipError_t forward(const NormCall& c) {
  NormParams p = params(c);
  const Config f = pick<false, XF, YF>(p.n);
  if (!f.fn) {
    const int64_t units = p.M * p.G;
    return start(reinterpret_cast<const void*>(&layernorm_forward_long_kernel<XF, YF>), units < 2048 ? units : 2048, 1024,
                 p, c.stream);
  }
  spread(p, f, 1 << 19);
  return start(f.fn, (int64_t)p.nb * p.slabs, f.threads, p, c.stream);
}

template <bool XF, bool YF>
hipError_t backward(const NormCall& c) {
  NormParams p = params(c);
  const bool sums = c.dweight || c.dbias;
  const Config f = pick<true, XF, YF>(p.n);
  if (f.fn) {
    // each workgroup adds a row of partial sums: M=16384 D=4096 bfloat16 97 us with four times as many, 79 so
    // (M=32768 D=768 41 us with twice as many, 35 so)
    spread(p, f, f.threads > 256 ? 1 << 18 : 1 << 17);
  } else {
    int64_t nb = (int64_t(1) << 23) / p.D;  // partial sums of at most 64 MiB, as those of shorter groups
    nb = nb < 1 ? 1 : nb < 64 ? nb : 64;
    p.nb = (int32_t)(p.M < nb ? p.M : nb);
  }
  std::unique_lock<std::mutex> lock(operators_mutex(), std::defer_lock);
  if (sums) {
    lock.lock();
    void* ws = nullptr;
    const hipError_t e = device_workspace(c.stream, (size_t)2 * p.nb * p.D * 4, &ws, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    p.partial = static_cast<float*>(ws);
  }
  hipError_t e;
  if (f.fn) {
    e = start(f.fn, (int64_t)p.nb * p.slabs, f.threads, p, c.stream);
  } else {
    const int64_t units = p.M * p.G;
    e = start(reinterpret_cast<const void*>(&layernorm_backward_long_kernel<XF, YF>), units < 2048 ? units : 2048, 1024, p,
              c.stream);
    if (e == hipSuccess && sums)
      e = start(reinterpret_cast<const void*>(&layernorm_columns_kernel<XF, YF>), ((int64_t)p.D + 255) / 256 * p.nb, 256, p,
                c.stream);
  }
  if (e != hipSuccess || !sums) return e;
  const float* partial = p.partial;
  float *dweight = c.dweight, *dbias = c.dbias;
  void* args[] = {&partial, &dweight, &dbias, &p.nb, &p.D};
  return hipLaunchKernel(reinterpret_cast<const void*>(&layernorm_join_kernel), dim3((uint32_t)((p.D + 63) / 64), 2),
                         dim3(1024), args, 0, c.stream);
}

__global__ __launch_bounds__(256) void layernorm_zero_kernel(float* a, float* b, int32_t D) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  if (a) a[c] = 0.f;
  if (b) b[c] = 0.f;
}

}  // namespace

hipError_t launch_layernorm_forward(const NormCall& c) {
  if (c.x_f32) return c.y_f32 ? forward<true, true>(c) : forward<true, false>(c);
  return c.y_f32 ? forward<false, true>(c) : forward<false, false>(c);
}

hipError_t launch_layernorm_backward(const NormCall& c) {
  if (c.M == 0) {  // no rows: the sums over them are 0
    float *a = c.dweight, *b = c.dbias;
    int32_t D = (int32_t)c.D;
    if (!a && !b) return hipSuccess;
    void* args[] = {&a, &b, &D};
    return hipLaunchKernel(reinterpret_cast<const void*>(&layernorm_zero_kernel), dim3((uint32_t)((D + 255) / 256)),
                           dim3(256), args, 0, c.stream);
  }
  if (c.x_f32) return c.y_f32 ? backward<true, true>(c) : backward<true, false>(c);
  return c.y_f32 ? backward<false, true>(c) : backward<false, false>(c);
}

}  // namespace rwkv7
