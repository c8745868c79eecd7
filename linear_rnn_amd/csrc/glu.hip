// Gated linear unit, forward and backward.
//
//   g = x Wg, u = x Wu ([M, D] times [D, F]),  h = act(g) u
//   dg = dh u act'(g),  du = dh act(g),  dx = dg Wg^T + du Wu^T,  dWg = x^T dg,  dWu = x^T du
//
// The forward is one kernel: a tile of the output takes the same columns of both weights, so g and u meet in
// registers and only h (and on demand g and u) leave. The backward forms dg and du once and then its three products.
//
// Numbers. Sums are float32. A bfloat16 call's operands are its inputs, exact; dg and du are rounded to bfloat16
// where they enter the products (2^-8 of each at most, half a step, as a bfloat16 program that keeps them in memory
// rounds them). A float32 call's operands are sums of three bfloat16 pieces, of whose nine products the six whose
// orders add to at most 2 are kept, the smallest first: errors of about 2^-24, at 1/6 of the bfloat16 rate, which is
// more than the float32 matrix instructions' 1/16.
#include "glu_internal.hpp"
#include "once_per_device.hpp"
#include "operators_lock.hpp"
#include "rwkv7_wkv.h"
#include "wkv7_internal.hpp"

#include "glu_gemm.hpp"

namespace rwkv7 {
namespace {

using namespace glu;

// ---- operands in the form that the products take: bfloat16 pieces in planes of padded rows

// [rows][cols] in the caller's type to NP planes [rows][ld] of pieces, zeros behind the columns. Eight columns a thread.
struct StageParams {
  const void* src;
  uint16_t* dst;
  int64_t rows, cols, ld;
};
template <bool F32>
__device__ __forceinline__ void load8(const void* src, int64_t at, int64_t left, bool wide, float (&v)[8]) {
  if (wide) {
    if constexpr (F32) {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
      const float4 a = f[0], b = f[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + at);
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i < left) {
        if constexpr (F32) v[i] = static_cast<const float*>(src)[at + i];
        else v[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(src)[at + i] << 16);
      }
    }
  }
}
template <int NP>
__device__ __forceinline__ void store_pieces(uint16_t* dst, int64_t at, int64_t plane, const float (&v)[8]) {
  linattn::Op<NP> o;
#pragma unroll
  for (int i = 0; i < 8; i += 2) linattn::put2(o, i, v[i], v[i + 1]);
#pragma unroll
  for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(dst + p * plane + at) = o.p[p];
}
template <bool F32>
__global__ __launch_bounds__(256) void glu_stage_kernel(StageParams p) {
  const int64_t per_row = p.ld / 8, plane = p.rows * p.ld;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.rows * per_row; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row, c = i % per_row * 8;
    float v[8];
    load8<F32>(p.src, row * p.cols + c, p.cols - c, p.cols % 8 == 0, v);
    store_pieces<F32 ? 3 : 1>(p.dst, row * p.ld + c, plane, v);
  }
}

// dg and du, in pieces.
struct GradParams {
  const void *gate, *up, *dh;
  uint16_t *dg, *du;  // planes [M][ld]
  int64_t M, F, ld;
  int act;
};
__device__ __forceinline__ void act_and_slope(float g, int act, float& a, float& s) {
  if (act == RWKV7_ACT_GELU) {
    const float c = 0.5f * (1.f + erff(g * 0.70710678f));
    a = g * c;
    s = fmaf(g * 0.39894228f, __builtin_amdgcn_exp2f(g * g * -0.72134752f), c);
  } else if (act == RWKV7_ACT_RELU2) {
    const float r = g > 0.f ? g : 0.f;
    a = r * r;
    s = 2.f * r;
  } else {
    const float e = sigmoid(g), f = sigmoid(-g);
    if (act == RWKV7_ACT_SILU) {
      a = g * e;
      s = e * fmaf(g, f, 1.f);
    } else {
      a = e;
      s = e * f;
    }
  }
}
template <bool F32>
__global__ __launch_bounds__(256) void glu_grad_kernel(GradParams p) {
  const int64_t per_row = p.ld / 8, plane = p.M * p.ld;
  const bool wide = p.F % 8 == 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M * per_row; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row, c = i % per_row * 8, at = row * p.F + c;
    float g[8], u[8], d[8], dg[8], du[8];
    load8<F32>(p.gate, at, p.F - c, wide, g);
    load8<F32>(p.up, at, p.F - c, wide, u);
    load8<F32>(p.dh, at, p.F - c, wide, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, s;
      act_and_slope(g[e], p.act, a, s);
      dg[e] = d[e] * u[e] * s;
      du[e] = d[e] * a;
    }
    store_pieces<F32 ? 3 : 1>(p.dg, row * p.ld + c, plane, dg);
    store_pieces<F32 ? 3 : 1>(p.du, row * p.ld + c, plane, du);
  }
}

// The sums of the parts, in their order.
struct JoinParams {
  const float* partial;  // [splits][products][n]
  void* out[2];
  int64_t n;
  int32_t splits, products;
  bool f32;
};
__global__ __launch_bounds__(256) void glu_join_kernel(JoinParams p) {
  const int which = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.n; i += (int64_t)gridDim.x * 256) {
    float s = 0.f;
    for (int k = 0; k < p.splits; ++k) s += p.partial[((int64_t)k * p.products + which) * p.n + i];
    if (p.f32) static_cast<float*>(p.out[which])[i] = s;
    else static_cast<uint16_t*>(p.out[which])[i] = __builtin_bit_cast(uint16_t, (__bf16)s);
  }
}
template <typename T>
__global__ __launch_bounds__(256) void glu_zero_kernel(T* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = T(0);
}

template <class P>
hipError_t start(const void* fn, dim3 blocks, int threads, int lds, const P& params, hipStream_t stream) {
  P p = params;
  void* args[] = {&p};
  return hipLaunchKernel(fn, blocks, dim3(threads), args, lds, stream);
}
uint32_t blocks_for(int64_t threads) {
  const int64_t n = (threads + 255) / 256;
  return (uint32_t)(n < 1 ? 1 : n < 16384 ? n : 16384);
}

// More than 64 KB of LDS has to be asked for on every device.
template <bool AC, bool BC, int WM, int WN, int TM, int TN, int EPI>
hipError_t gemm(GemmParams p, hipStream_t stream) {
  constexpr int BM = WM * TM * 16, BN = WN * TN * 16, lds = 2 * (BM + BN) * kBK * 2;
  const void* fn = reinterpret_cast<const void*>(&glu_gemm_kernel<AC, BC, WM, WN, TM, TN, EPI>);
  static std::atomic<uint64_t> granted{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  e = static_cast<hipError_t>(once_per_device(granted, dev, [&] {
    return static_cast<int>(hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  }));
  if (e != hipSuccess) return e;
  const int per_tile = EPI == kGlu ? BN / 2 : BN;
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = (p.N + per_tile - 1) / per_tile * (EPI == kProduct && p.out2 ? 2 : 1);
  return start(fn, dim3((uint32_t)p.tiles_m * p.tiles_n * p.splits), 64 * WM * WN, lds, p, stream);
}

// ---- the workspace of a call, in parts
struct Parts {
  size_t bytes = 0;
  size_t add(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};
int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

// A matrix as an operand: the caller's own where it is bfloat16 with rows of whole 16 bytes, else a copy.
struct Matrix {
  const void* src;
  int64_t rows, cols;
  bool f32;
  size_t at = 0;
  bool copied() const { return f32 || cols % 8 != 0; }
  int64_t ld() const { return padded(cols); }
  void place(Parts& parts) {
    if (copied()) at = parts.add((size_t)rows * ld() * 2 * (f32 ? 3 : 1));
  }
  const uint16_t* piece(char* ws, int i) const {
    return copied() ? reinterpret_cast<const uint16_t*>(ws + at) + i * rows * ld() : static_cast<const uint16_t*>(src);
  }
  hipError_t stage(char* ws, hipStream_t stream) const {
    if (!copied()) return hipSuccess;
    const StageParams p{src, reinterpret_cast<uint16_t*>(ws + at), rows, cols, ld()};
    const void* fn = f32 ? reinterpret_cast<const void*>(&glu_stage_kernel<true>)
                         : reinterpret_cast<const void*>(&glu_stage_kernel<false>);
    return start(fn, dim3(blocks_for(rows * ld() / 8)), 256, 0, p, stream);
  }
};

// The pairs of pieces of two operands, the smallest products first.
constexpr int kPairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
int pairs(bool f32) { return f32 ? 6 : 1; }
int first_of(bool f32, int s) { return f32 ? kPairs[s][0] : 0; }
int second_of(bool f32, int s) { return f32 ? kPairs[s][1] : 0; }

hipError_t forward(const GluCall& c) {
  Matrix x{c.x, c.M, c.D, c.f32}, wg{c.w_gate, c.D, c.F, c.f32}, wu{c.w_up, c.D, c.F, c.f32};
  Parts parts;
  for (Matrix* m : {&x, &wg, &wu}) m->place(parts);
  std::unique_lock<std::mutex> lock(operators_mutex(), std::defer_lock);
  char* ws = nullptr;
  if (parts.bytes) {
    lock.lock();
    void* p = nullptr;
    const hipError_t e = device_workspace(c.stream, parts.bytes, &p, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    ws = static_cast<char*>(p);
    for (Matrix* m : {&x, &wg, &wu}) {
      const hipError_t e2 = m->stage(ws, c.stream);
      if (e2 != hipSuccess) return e2;
    }
  }
  GemmParams p{};
  p.nseg = pairs(c.f32);
  for (int s = 0; s < p.nseg; ++s) {
    p.a[s] = x.piece(ws, first_of(c.f32, s));
    p.b[s] = wg.piece(ws, second_of(c.f32, s));
    p.b2[s] = wu.piece(ws, second_of(c.f32, s));
  }
  p.lda = x.ld(), p.ldb = wg.ld(), p.M = (int32_t)c.M, p.N = (int32_t)c.F, p.K = (int32_t)c.D, p.splits = 1;
  p.out = c.h, p.gate = c.gate, p.up = c.up, p.f32 = c.f32, p.act = c.act;
  return gemm<false, true, 2, 4, 8, 4, kGlu>(p, c.stream);
}

hipError_t backward(const GluCall& c) {
  const bool dx = c.dx != nullptr, dw = c.dw_gate != nullptr;
  if (!dx && !dw) return hipSuccess;
  Matrix x{c.x, c.M, c.D, c.f32}, wg{c.w_gate, c.D, c.F, c.f32}, wu{c.w_up, c.D, c.F, c.f32};
  const int np = c.f32 ? 3 : 1;
  const int64_t ldf = padded(c.F);
  Parts parts;
  if (dw) x.place(parts);
  if (dx) wg.place(parts), wu.place(parts);
  const size_t dg_at = parts.add((size_t)np * c.M * ldf * 2), du_at = parts.add((size_t)np * c.M * ldf * 2);
  // parts of the weights' gradients, where their tiles are too few for the compute units
  const int64_t wtiles = (c.D + 255) / 256 * ((c.F + 255) / 256) * 2, steps = (c.M + kBK - 1) / kBK * pairs(c.f32);
  int64_t splits = 256 / wtiles;
  splits = splits < steps / 8 ? splits : steps / 8;
  splits = splits < 1 ? 1 : splits;
  const size_t partial_at = dw && splits > 1 ? parts.add((size_t)splits * 2 * c.D * c.F * 4) : 0;

  std::lock_guard<std::mutex> lock(operators_mutex());
  void* space = nullptr;
  hipError_t e = device_workspace(c.stream, parts.bytes, &space, kWorkspaceOperators);
  if (e != hipSuccess) return e;
  char* ws = static_cast<char*>(space);
  if (dw && (e = x.stage(ws, c.stream)) != hipSuccess) return e;
  if (dx && ((e = wg.stage(ws, c.stream)) != hipSuccess || (e = wu.stage(ws, c.stream)) != hipSuccess)) return e;
  uint16_t *dg = reinterpret_cast<uint16_t*>(ws + dg_at), *du = reinterpret_cast<uint16_t*>(ws + du_at);
  const int64_t plane = c.M * ldf;
  const GradParams gp{c.gate, c.up, c.dh, dg, du, c.M, c.F, ldf, c.act};
  e = start(c.f32 ? reinterpret_cast<const void*>(&glu_grad_kernel<true>) : reinterpret_cast<const void*>(&glu_grad_kernel<false>),
            dim3(blocks_for(plane / 8)), 256, 0, gp, c.stream);
  if (e != hipSuccess) return e;
  if (dx) {
    GemmParams p{};
    for (int s = 0; s < pairs(c.f32); ++s) {
      const int i = first_of(c.f32, s), j = second_of(c.f32, s);
      p.a[2 * s] = dg + i * plane, p.b[2 * s] = wg.piece(ws, j);
      p.a[2 * s + 1] = du + i * plane, p.b[2 * s + 1] = wu.piece(ws, j);
    }
    p.nseg = 2 * pairs(c.f32);
    p.lda = ldf, p.ldb = ldf, p.M = (int32_t)c.M, p.N = (int32_t)c.D, p.K = (int32_t)ldf, p.splits = 1;
    p.out = c.dx, p.f32 = c.f32;
    e = gemm<false, false, 2, 4, 8, 4, kProduct>(p, c.stream);
    if (e != hipSuccess) return e;
  }
  if (dw) {
    GemmParams p{};
    p.nseg = pairs(c.f32);
    for (int s = 0; s < p.nseg; ++s) {
      const int i = first_of(c.f32, s), j = second_of(c.f32, s);
      p.a[s] = x.piece(ws, i), p.b[s] = dg + j * plane, p.b2[s] = du + j * plane;
    }
    p.lda = x.ld(), p.ldb = ldf, p.M = (int32_t)c.D, p.N = (int32_t)c.F, p.K = (int32_t)c.M, p.splits = (int32_t)splits;
    p.out = c.dw_gate, p.out2 = c.dw_up, p.f32 = c.f32;
    p.partial = reinterpret_cast<float*>(ws + partial_at);
    e = gemm<true, true, 2, 4, 8, 4, kProduct>(p, c.stream);
    if (e != hipSuccess || splits == 1) return e;
    const JoinParams jp{p.partial, {c.dw_gate, c.dw_up}, c.D * c.F, (int32_t)splits, 2, c.f32};
    e = start(reinterpret_cast<const void*>(&glu_join_kernel), dim3(blocks_for(c.D * c.F), 2), 256, 0, jp, c.stream);
  }
  return e;
}

}  // namespace

hipError_t launch_glu_forward(const GluCall& c) { return forward(c); }
hipError_t launch_glu_backward(const GluCall& c) { return backward(c); }

hipError_t launch_glu_zero(void* p, int64_t n, bool f32, hipStream_t stream) {
  void* args[] = {&p, &n};
  const void* fn = f32 ? reinterpret_cast<const void*>(&glu_zero_kernel<uint32_t>)
                       : reinterpret_cast<const void*>(&glu_zero_kernel<uint16_t>);
  return hipLaunchKernel(fn, dim3(blocks_for(n)), dim3(256), args, 0, stream);
}

}  // namespace rwkv7
