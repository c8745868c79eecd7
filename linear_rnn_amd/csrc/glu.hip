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
// rounds them). A large float32 call's operands, and those of the gradients, are sums of three bfloat16 pieces, of whose
// nine products the six whose orders add to at most 2 are kept, the smallest first: errors of about 2^-24, at 1/6 of
// the bfloat16 rate, which is more than the float32 matrix instructions' 1/16. Other float32 forwards take these
// (glu_f32.hpp), without pieces, workspace and sums in parts.
#include "glu_internal.hpp"
#include "launch_chunks.hpp"
#include "once_per_device.hpp"
#include "operators_lock.hpp"
#include "rwkv7_wkv.h"
#include "wkv7_internal.hpp"

#include "glu_f32.hpp"
#include "glu_few.hpp"
#include "glu_gemm.hpp"
#include "glu_rules.hpp"

namespace rwkv7 {
namespace {

using namespace glu;

// ---- operands in the form that the products take: bfloat16 pieces in planes of padded rows

// A matrix [rows][cols] in the caller's type, to planes [rows][ld] of pieces, zeros behind the columns.
struct StageJob {
  const void* src;
  uint16_t* dst;
  int64_t rows, cols, ld;
};
// dg and du from g, u and dh, to planes [rows][ld] of pieces.
struct GradJob {
  const void *gate, *up, *dh;
  uint16_t *dg, *du;
  int64_t rows, cols, ld;
  int act;
};
// What a call prepares, in one launch: workgroups first[i] .. first[i + 1] - 1 do job i (the gradients are the last).
struct StageParams {
  StageJob job[3];
  GradJob grad;
  uint32_t first[5];
  uint32_t begin;  // number of the launch's first workgroup
};
// Rows need not begin on 16 bytes here.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32>
__device__ __forceinline__ void load8(const void* src, int64_t at, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (F32) {
      const f32x4_any* f = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(src) + at);
      const f32x4_any a = f[0], b = f[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
      const u32x4_any u = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(src) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
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
__device__ __forceinline__ void act_and_slope(float g, int act, float& a, float& s) {
  if (act == RWKV7_ACT_GELU) {
    const float c = 0.5f * erfcf(g * -0.70710678f);
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
// Eight columns a thread.
template <bool F32>
__device__ __forceinline__ void stage(const StageJob& j, int64_t i) {
  const int64_t per_row = j.ld / 8, row = i / per_row, c = i % per_row * 8;
  if (row >= j.rows) return;
  float v[8];
  load8<F32>(j.src, row * j.cols + c, j.cols - c, v);
  store_pieces<F32 ? 3 : 1>(j.dst, row * j.ld + c, j.rows * j.ld, v);
}
template <bool F32>
__device__ __forceinline__ void stage(const GradJob& j, int64_t i) {
  const int64_t per_row = j.ld / 8, row = i / per_row, c = i % per_row * 8, at = row * j.cols + c;
  if (row >= j.rows) return;
  float g[8], u[8], d[8], dg[8], du[8];
  load8<F32>(j.gate, at, j.cols - c, g);
  load8<F32>(j.up, at, j.cols - c, u);
  load8<F32>(j.dh, at, j.cols - c, d);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, s;
    act_and_slope(g[e], j.act, a, s);
    dg[e] = d[e] * u[e] * s;
    du[e] = d[e] * a;
  }
  store_pieces<F32 ? 3 : 1>(j.dg, row * j.ld + c, j.rows * j.ld, dg);
  store_pieces<F32 ? 3 : 1>(j.du, row * j.ld + c, j.rows * j.ld, du);
}
template <bool F32>
__global__ __launch_bounds__(256) void glu_stage_kernel(StageParams p) {
  const uint32_t block = p.begin + blockIdx.x;
  if (block >= p.first[3]) stage<F32>(p.grad, (int64_t)(block - p.first[3]) * 256 + threadIdx.x);
  else if (block >= p.first[2]) stage<F32>(p.job[2], (int64_t)(block - p.first[2]) * 256 + threadIdx.x);
  else if (block >= p.first[1]) stage<F32>(p.job[1], (int64_t)(block - p.first[1]) * 256 + threadIdx.x);
  else stage<F32>(p.job[0], (int64_t)block * 256 + threadIdx.x);
}

// The sums of the parts of a product, in their order: [splits][products][rows * cols] to one or two outputs, or, of
// g and u, to h (and g and u themselves). Workgroups first .. of the grid's.
struct JoinJob {
  const float* partial;
  void *out, *out2;  // the products; with `h` they may be null
  void* h;
  int64_t n;
  int32_t splits, products;
  bool f32;
  int act;
};
struct JoinParams {
  JoinJob job[2];
  uint32_t second;  // first workgroup of the second job
};
// Four elements a thread.
__device__ __forceinline__ void join(const JoinJob& j, int64_t i) {
  i *= 4;
  if (i >= j.n) return;
  const int n = j.n - i < 4 ? (int)(j.n - i) : 4;
  f32x4 a = linattn::zero4(), b = linattn::zero4();
  const float* at = j.partial + i;
  auto add = [&](f32x4& to, const float* from) {
    if (n == 4) {
      const f32x4_any x = *reinterpret_cast<const f32x4_any*>(from);
#pragma unroll
      for (int e = 0; e < 4; ++e) to[e] += x[e];
    } else {
      for (int e = 0; e < n; ++e) to[e] += from[e];
    }
  };
#pragma unroll 4
  for (int s = 0; s < j.splits; ++s) {
    add(a, at);
    if (j.products == 2) add(b, at + j.n);
    at += j.products * j.n;
  }
  if (j.h) {
    f32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = activation(a[e], j.act) * b[e];
    store4(j.h, j.f32, i, n, h);
  }
  if (j.out) store4(j.out, j.f32, i, n, a);
  if (j.out2) store4(j.out2, j.f32, i, n, b);
}
__global__ __launch_bounds__(256) void glu_join_kernel(JoinParams p) {
  if (blockIdx.x < p.second) join(p.job[0], (int64_t)blockIdx.x * 256 + threadIdx.x);
  else join(p.job[1], (int64_t)(blockIdx.x - p.second) * 256 + threadIdx.x);
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
uint32_t blocks_for(int64_t threads) { return (uint32_t)((threads + 255) / 256); }

// ---- tiles (which, and how many workgroups share a sum: glu_rules.hpp)

int compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      n <= 0)
    n = 256;
  return n;
}

// More than 64 KB of LDS has to be asked for on every device.
template <int LDS>
hipError_t grant(const void* fn, std::atomic<uint64_t>& granted) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  return static_cast<hipError_t>(once_per_device(granted, dev, [&] {
    return static_cast<int>(hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, LDS));
  }));
}
template <int BM, int BN>
uint32_t set_tiles(GemmParams& p) {
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = (p.N + BN - 1) / BN * (p.two ? 2 : 1);
  return (uint32_t)p.tiles_m * p.tiles_n * p.splits;
}
template <int WM, int WN, int TM, int TN, int NB>
hipError_t forward_product(GemmParams p, hipStream_t stream) {
  constexpr int BM = WM * TM * 16, BN = WN * TN * 16, lds = NB * (BM + BN) * kBK * 2;
  const void* fn = reinterpret_cast<const void*>(&glu_forward_kernel<WM, WN, TM, TN, NB>);
  static std::atomic<uint64_t> granted{0};
  const hipError_t e = grant<lds>(fn, granted);
  if (e != hipSuccess) return e;
  const uint32_t blocks = set_tiles<BM, BN / 2>(p);
  return start(fn, dim3(blocks), 64 * WM * WN, lds, p, stream);
}
template <int WM, int WN, int TM, int TN, int NB>
hipError_t grad_products(GradProducts p, bool x, bool w, hipStream_t stream) {
  constexpr int BM = WM * TM * 16, BN = WN * TN * 16, lds = NB * (BM + BN) * kBK * 2;
  const void* fn = reinterpret_cast<const void*>(&glu_backward_kernel<WM, WN, TM, TN, NB>);
  static std::atomic<uint64_t> granted{0};
  const hipError_t e = grant<lds>(fn, granted);
  if (e != hipSuccess) return e;
  const uint32_t nx = x ? set_tiles<BM, BN>(p.x) : 0, nw = w ? set_tiles<BM, BN>(p.w) : 0;
  p.first = p.w_first ? nw : nx;
  const uint32_t blocks = nx + nw;
  return start(fn, dim3(blocks), 64 * WM * WN, lds, p, stream);
}
hipError_t forward_products(const GemmParams& p, Shape s, hipStream_t stream) {
  if (s == kLarge) return forward_product<2, 4, 8, 4, 2>(p, stream);
  if (s == kHalf) return forward_product<2, 4, 4, 4, 3>(p, stream);
  return forward_product<1, 4, 4, 4, 2>(p, stream);
}
hipError_t backward_products(const GradProducts& p, bool x, bool w, Shape s, hipStream_t stream) {
  if (s == kLarge) return grad_products<2, 4, 8, 4, 2>(p, x, w, stream);
  if (s == kHalf) return grad_products<2, 4, 4, 4, 3>(p, x, w, stream);
  return grad_products<2, 2, 4, 4, 2>(p, x, w, stream);
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
int64_t whole(int64_t n, int64_t of) { return (n + of - 1) / of * of; }
// Elements between rows of a copy: whole 128-byte lines, where that adds little.
int64_t padded(int64_t cols) { return whole(cols, cols >= 256 ? 64 : 8); }

// A matrix as an operand: the caller's own where it is bfloat16 with rows of whole 16 bytes, else a copy.
struct Matrix {
  const void* src;
  int64_t rows, cols;
  bool f32;
  size_t at = 0;
  bool copied() const { return f32 || cols % 8 != 0; }
  int64_t ld() const { return copied() ? padded(cols) : cols; }
  void place(Parts& parts) {
    if (copied()) at = parts.add((size_t)rows * ld() * 2 * (f32 ? 3 : 1));
  }
  const uint16_t* piece(char* ws, int i) const {
    return copied() ? reinterpret_cast<const uint16_t*>(ws + at) + i * rows * ld() : static_cast<const uint16_t*>(src);
  }
};

// The launch that prepares a call's operands.
struct Stage {
  StageParams p{};
  int jobs = 0;
  uint32_t blocks = 0;
  void add(const Matrix& m, char* ws) {
    if (!m.copied()) return;
    p.job[jobs] = StageJob{m.src, reinterpret_cast<uint16_t*>(ws + m.at), m.rows, m.cols, m.ld()};
    p.first[jobs++] = blocks;
    blocks += blocks_for(m.rows * m.ld() / 8);
  }
  hipError_t launch(const GradJob* grad, bool f32, hipStream_t stream) {
    // a job that is not there has no workgroups: the one before it ends where the next begins
    for (int i = jobs; i < 5; ++i) p.first[i] = blocks;
    if (grad) {
      p.grad = *grad;
      blocks += blocks_for(grad->rows * grad->ld / 8);
    }
    const void* fn = f32 ? reinterpret_cast<const void*>(&glu_stage_kernel<true>)
                         : reinterpret_cast<const void*>(&glu_stage_kernel<false>);
    return static_cast<hipError_t>(in_chunks(blocks, 256, [&](uint32_t first, uint32_t n) {
      p.begin = first;
      return static_cast<int>(start(fn, dim3(n), 256, 0, p, stream));
    }));
  }
};

// The pairs of pieces of two operands, the smallest products first.
constexpr int kPairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
int first_of(bool f32, int s) { return f32 ? kPairs[s][0] : 0; }
int second_of(bool f32, int s) { return f32 ? kPairs[s][1] : 0; }

template <bool F32, int C>
hipError_t forward_few(const GluCall& c) {
  const FewParams p{c.x, c.w_gate, c.w_up, c.h, c.gate, c.up, (int32_t)c.M, (int32_t)c.D, (int32_t)c.F, c.act};
  const void* fn = c.M <= 16 ? reinterpret_cast<const void*>(&glu_few_kernel<F32, C, 1>)
                             : reinterpret_cast<const void*>(&glu_few_kernel<F32, C, 2>);
  return start(fn, dim3((uint32_t)((c.F + 16 * C - 1) / (16 * C)), (uint32_t)((c.M + 31) / 32)), 64 * kFewWaves, 0, p, c.stream);
}
hipError_t forward_few(const GluCall& c) {
  if (!c.f32) return forward_few<false, 4>(c);
  return few_columns(Sizes{c.M, c.D, c.F, c.f32}, compute_units()) == 32 ? forward_few<true, 2>(c) : forward_few<true, 4>(c);
}

template <int TM>
hipError_t forward_f32(const GluCall& c) {
  F32Params p{static_cast<const float*>(c.x), static_cast<const float*>(c.w_gate), static_cast<const float*>(c.w_up),
              static_cast<float*>(c.h), static_cast<float*>(c.gate), static_cast<float*>(c.up), (int32_t)c.M, (int32_t)c.D,
              (int32_t)c.F, 0, 0, c.act};
  p.tiles_m = (int32_t)((c.M + 16 * TM - 1) / (16 * TM)), p.tiles_n = (int32_t)((c.F + kCols32 - 1) / kCols32);
  return start(reinterpret_cast<const void*>(&glu_forward32_kernel<TM>), dim3((uint32_t)p.tiles_m * p.tiles_n), 64 * kWaves32, 0, p,
               c.stream);
}
constexpr hipError_t (*kForwardF32[kMostTM32])(const GluCall&) = {&forward_f32<1>, &forward_f32<2>, &forward_f32<3>,
                                                                  &forward_f32<4>, &forward_f32<5>};
// Rows that are in the workspace at once: what lives there for each of them (copies of x, dg and du) is at most 4 GiB, or 128
// rows. Gradients of larger calls add up the weights' from one slab of rows to the next, in float32: 131072 x 4096 x 10944 bfloat16
// in two slabs 39.7 ms, at once 39.0; float32 32768 x 64 x 10944 4.5 and 5.0.
constexpr size_t kSlabBytes = size_t(1) << 32;
int64_t slab_rows(int64_t M, size_t row_bytes) {
  const int64_t fit = row_bytes ? (int64_t)(kSlabBytes / row_bytes / 128 * 128) : M, most = fit > 128 ? fit : 128;
  if (M <= most) return M;
  const int64_t slabs = (M + most - 1) / most;
  return whole((M + slabs - 1) / slabs, 128);
}
// Row `row` of a caller's matrix (null stays null).
const void* at_row(const void* p, int64_t row, int64_t cols, bool f32) {
  return p ? static_cast<const char*>(p) + row * cols * (f32 ? 4 : 2) : nullptr;
}
void* at_row(void* p, int64_t row, int64_t cols, bool f32) {
  return const_cast<void*>(at_row(static_cast<const void*>(p), row, cols, f32));
}

hipError_t forward(const GluCall& c) {
  const ForwardPlan how = plan_forward(Sizes{c.M, c.D, c.F, c.f32}, compute_units());
  if (how.way == kFew) return forward_few(c);
  if (how.way == kInstructions) return kForwardF32[how.tm - 1](c);
  Matrix x{c.x, c.M, c.D, c.f32}, wg{c.w_gate, c.D, c.F, c.f32}, wu{c.w_up, c.D, c.F, c.f32};
  const int splits = how.tiles.splits[0];
  const int64_t rows = slab_rows(c.M, x.copied() ? x.ld() * 2 * (c.f32 ? 3 : 1) : 0);
  x.rows = rows;
  Parts parts;
  for (Matrix* m : {&x, &wg, &wu}) m->place(parts);
  const size_t partial_at = splits > 1 ? parts.add((size_t)splits * 2 * rows * c.F * 4) : 0;
  std::unique_lock<std::mutex> lock(operators_mutex(), std::defer_lock);
  char* ws = nullptr;
  if (parts.bytes) {
    lock.lock();
    void* space = nullptr;
    const hipError_t e = device_workspace(c.stream, parts.bytes, &space, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    ws = static_cast<char*>(space);
  }
  for (int64_t first = 0; first < c.M; first += rows) {
    const int64_t here = c.M - first < rows ? c.M - first : rows;
    x.src = at_row(c.x, first, c.D, c.f32), x.rows = here;
    Stage stage;
    stage.add(x, ws);
    if (first == 0) stage.add(wg, ws), stage.add(wu, ws);
    hipError_t e = stage.launch(nullptr, c.f32, c.stream);
    if (e != hipSuccess) return e;
    GemmParams p{};
    p.nseg = pairs(c.f32);
    for (int s = 0; s < p.nseg; ++s) {
      p.a[s] = x.piece(ws, first_of(c.f32, s));
      p.b[s] = wg.piece(ws, second_of(c.f32, s));
      p.b2[s] = wu.piece(ws, second_of(c.f32, s));
    }
    p.lda = x.ld(), p.ldb = wg.ld(), p.M = (int32_t)here, p.N = (int32_t)c.F, p.K = (int32_t)c.D, p.splits = splits;
    p.out = at_row(c.h, first, c.F, c.f32), p.gate = at_row(c.gate, first, c.F, c.f32), p.up = at_row(c.up, first, c.F, c.f32);
    p.f32 = c.f32, p.act = c.act;
    p.partial = reinterpret_cast<float*>(ws + partial_at);
    e = forward_products(p, how.tiles.shape, c.stream);
    if (e != hipSuccess) return e;
    if (splits == 1) continue;
    JoinParams j{};
    j.job[0] = JoinJob{p.partial, p.gate, p.up, p.out, here * c.F, splits, 2, c.f32, c.act};
    j.second = blocks_for((j.job[0].n + 3) / 4);
    e = start(reinterpret_cast<const void*>(&glu_join_kernel), dim3(j.second), 256, 0, j, c.stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t backward(const GluCall& c) {
  const bool dx = c.dx != nullptr, dw = c.dw_gate != nullptr;
  if (!dx && !dw) return hipSuccess;
  Matrix x{c.x, c.M, c.D, c.f32}, wg{c.w_gate, c.D, c.F, c.f32}, wu{c.w_up, c.D, c.F, c.f32};
  const int np = c.f32 ? 3 : 1;
  const int64_t ldf = padded(c.F);
  const int64_t sum_f = whole(c.F, 8);  // with zeros in the copies' columns behind F
  const int64_t rows = slab_rows(c.M, (size_t)np * 2 * (2 * ldf + (dw && x.copied() ? x.ld() : 0)));
  const bool slabs = rows < c.M;
  Product job[2] = {{rows, c.D, 1, steps_of(sum_f, 2 * pairs(c.f32))}, {c.D, c.F, 2, steps_of(rows, pairs(c.f32))}};
  if (!dx) job[0] = Product{0, 0, 0, 0};
  if (!dw) job[1] = Product{0, 0, 0, 0};
  const Plan how = plan(kGradShapes, job, compute_units());
  const int sx = how.splits[0], sw = how.splits[1];
  Parts parts;
  x.rows = rows;
  if (dw) x.place(parts);
  if (dx) wg.place(parts), wu.place(parts);
  const size_t dg_at = parts.add((size_t)np * rows * ldf * 2), du_at = parts.add((size_t)np * rows * ldf * 2);
  const size_t px_at = dx && sx > 1 ? parts.add((size_t)sx * rows * c.D * 4) : 0;
  // with slabs the weights' gradients are parts too, behind their sum over the slabs before
  const bool join_w = dw && (sw > 1 || slabs);
  const int64_t weights = c.D * c.F;
  const size_t pw_at = join_w ? parts.add((size_t)(sw + slabs) * 2 * weights * 4) : 0;

  std::lock_guard<std::mutex> lock(operators_mutex());
  void* space = nullptr;
  hipError_t e = device_workspace(c.stream, parts.bytes, &space, kWorkspaceOperators);
  if (e != hipSuccess) return e;
  char* ws = static_cast<char*>(space);
  uint16_t *dg = reinterpret_cast<uint16_t*>(ws + dg_at), *du = reinterpret_cast<uint16_t*>(ws + du_at);
  float* const sum_w = reinterpret_cast<float*>(ws + pw_at);
  float* const parts_w = sum_w + (slabs ? 2 * weights : 0);
  for (int64_t first = 0; first < c.M; first += rows) {
    const int64_t here = c.M - first < rows ? c.M - first : rows, plane = here * ldf;
    const bool last = first + here == c.M;
    x.src = at_row(c.x, first, c.D, c.f32), x.rows = here;
    Stage stage;
    if (dw) stage.add(x, ws);
    if (dx && first == 0) stage.add(wg, ws), stage.add(wu, ws);
    const GradJob grad{at_row(c.gate, first, c.F, c.f32), at_row(c.up, first, c.F, c.f32), at_row(c.dh, first, c.F, c.f32),
                       dg, du, here, c.F, ldf, c.act};
    e = stage.launch(&grad, c.f32, c.stream);
    if (e != hipSuccess) return e;

    GradProducts p{};
    p.w_first = (job[1].steps + sw - 1) / sw > (job[0].steps + sx - 1) / sx;
    JoinParams j{};
    int joins = 0;
    uint32_t blocks = 0;
    if (dx) {
      GemmParams& o = p.x;
      for (int s = 0; s < pairs(c.f32); ++s) {
        const int f = first_of(c.f32, s), t = second_of(c.f32, s);
        o.a[2 * s] = dg + f * plane, o.b[2 * s] = wg.piece(ws, t);
        o.a[2 * s + 1] = du + f * plane, o.b[2 * s + 1] = wu.piece(ws, t);
      }
      o.nseg = 2 * pairs(c.f32);
      o.lda = ldf, o.ldb = wg.ld(), o.M = (int32_t)here, o.N = (int32_t)c.D, o.K = (int32_t)sum_f, o.splits = sx;
      o.out = at_row(c.dx, first, c.D, c.f32), o.f32 = c.f32, o.partial = reinterpret_cast<float*>(ws + px_at);
      if (sx > 1) {
        j.job[joins++] = JoinJob{o.partial, o.out, nullptr, nullptr, here * c.D, sx, 1, c.f32, 0};
        blocks += blocks_for((here * c.D + 3) / 4);
      }
    }
    j.second = blocks;
    if (dw) {
      GemmParams& o = p.w;
      o.nseg = pairs(c.f32);
      for (int s = 0; s < o.nseg; ++s) {
        const int f = first_of(c.f32, s), t = second_of(c.f32, s);
        o.a[s] = x.piece(ws, f), o.b[s] = dg + t * plane, o.b2[s] = du + t * plane;
      }
      o.lda = x.ld(), o.ldb = ldf, o.M = (int32_t)c.D, o.N = (int32_t)c.F, o.K = (int32_t)here, o.splits = sw;
      o.out = c.dw_gate, o.out2 = c.dw_up, o.two = true, o.f32 = c.f32, o.partial = parts_w;
      const bool more = first > 0;  // there is a sum already
      if (join_w && sw == 1 && !more) {
        o.out = sum_w, o.out2 = sum_w + weights, o.f32 = true;  // the product is the sum
      } else if (join_w) {
        if (sw == 1) o.out = parts_w, o.out2 = parts_w + weights, o.f32 = true;
        j.job[joins++] = JoinJob{more ? sum_w : parts_w, last ? c.dw_gate : sum_w, last ? c.dw_up : sum_w + weights, nullptr,
                                 weights, sw + more, 2, c.f32 || !last, 0};
        blocks += blocks_for((weights + 3) / 4);
        if (joins == 1) j.second = blocks;  // the only job
      }
    }
    e = backward_products(p, dx, dw, how.shape, c.stream);
    if (e == hipSuccess && joins > 0) e = start(reinterpret_cast<const void*>(&glu_join_kernel), dim3(blocks), 256, 0, j, c.stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_glu_forward(const GluCall& c) { return forward(c); }
hipError_t launch_glu_backward(const GluCall& c) { return backward(c); }

hipError_t launch_glu_zero(void* p, int64_t n, bool f32, hipStream_t stream) {
  void* args[] = {&p, &n};
  const void* fn = f32 ? reinterpret_cast<const void*>(&glu_zero_kernel<uint32_t>)
                       : reinterpret_cast<const void*>(&glu_zero_kernel<uint16_t>);
  const uint32_t blocks = n < (int64_t(1) << 22) ? blocks_for(n) : 1 << 14;
  return hipLaunchKernel(fn, dim3(blocks), dim3(256), args, 0, stream);
}

}  // namespace rwkv7
