// The gated linear unit of float32 operands as they are, by the float32 matrix instructions.
//
// These bound it: 154 TFLOP/s at most, where products of bfloat16 pieces reach 220, but there are no pieces to be made and
// no parts to be added, and rows begin anywhere. A workgroup takes 16 TM rows and 64 columns of both weights, so TM fits
// the tiles to the compute units; a wave 16 columns of both, for half of the k: the two waves of a SIMD fill each other's
// gaps. 32 k at a time go through registers, one step ahead, to LDS, k contiguous, rows 144 bytes apart so that 8 lanes'
// 16 bytes meet every bank once. A float32 instruction takes 4 of k, in any order that both operands keep: instruction j
// of 16 k takes k = 4 q + j from the lanes' quarter q, so that a lane's 16 bytes are its operands of four instructions.
// Loads of 4 bytes take the compute unit some 14 cycles each; between the products they cost nothing (all before the
// first: 1.56 us a step of 80 rows, so 1.35; the instructions alone take 1.07). 4096 x 4096 x 4096: 141 TFLOP/s.
#pragma once

#include "glu_gemm.hpp"

namespace rwkv7 {
namespace glu {

constexpr int kRow32 = kStep32 + 4;
constexpr int kWaves32 = 8;

struct F32Params {
  const float* x;  // [M, D]
  const float* w_gate;
  const float* w_up;
  float* h;
  float* gate;  // may be null
  float* up;
  int32_t M, D, F, tiles_m, tiles_n, act;
};

template <int TM>
__global__ __launch_bounds__(64 * kWaves32) __attribute__((amdgpu_waves_per_eu(4))) void glu_forward32_kernel(F32Params p) {
  constexpr int BM = 16 * TM, kRows = 2 * kCols32 + BM;
  constexpr int kSum = 2 * kCols32 + 4;  // floats between rows of the sums
  constexpr int kFloats = 2 * kRows * kRow32 > BM * kSum ? 2 * kRows * kRow32 : BM * kSum;
  __shared__ __attribute__((aligned(16))) float lds[kFloats];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, li = lane & 15, part = wave >> 2, own = (wave & 3) * 16;  // its half of k, its first column
  const uint32_t id = xcd_swizzle(blockIdx.x, (uint32_t)p.tiles_m * p.tiles_n);
  const int64_t m0 = (int64_t)(id % p.tiles_m) * BM;
  const int n0 = (int)(id / p.tiles_m) * kCols32;
  const int rows = p.M - m0 < BM ? (int)(p.M - m0) : BM;

  // Weights: a thread four k of a column, of each; x: one k of TM rows.
  const int wn = lane, wk = wave * 4, xk = threadIdx.x % kStep32, xm = threadIdx.x / kStep32;
  const auto bx = linattn::buffer(p.x + m0 * p.D, (uint32_t)rows * p.D * 4);
  float rw[2][4], rx[TM];
  constexpr int kLoads = 8 + TM;
  struct Step {
    __amdgpu_buffer_rsrc_t gate, up;
    int k0, left;
  };
  auto step_at = [&](int k0) {
    const int left = p.D - k0 < kStep32 ? p.D - k0 : kStep32;
    const uint32_t bytes = left > 0 ? (uint32_t)left * p.F * 4 : 0;
    const int64_t at = left > 0 ? (int64_t)k0 * p.F : 0;
    return Step{linattn::buffer(p.w_gate + at, bytes), linattn::buffer(p.w_up + at, bytes), k0, left};
  };
  auto load = [&](const Step& s, int i) {
    if (i < 8) {
      const uint32_t off = ((uint32_t)(wk + i / 2) * p.F + n0 + wn) * 4;
      rw[i % 2][i / 2] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(i % 2 ? s.up : s.gate, off, 0, 0));
    } else {
      const uint32_t off = ((uint32_t)(xm + 16 * (i - 8)) * p.D + s.k0 + xk) * 4;
      rx[i - 8] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bx, xk < s.left ? off : kNowhere, 0, 0));
    }
  };
  auto load_all = [&](int k0) {
    const Step s = step_at(k0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(s, i);
  };
  auto store = [&](float* to) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<f32x4*>(to + (i * kCols32 + wn) * kRow32 + wk) = f32x4{rw[i][0], rw[i][1], rw[i][2], rw[i][3]};
#pragma unroll
    for (int i = 0; i < TM; ++i) to[(2 * kCols32 + xm + 16 * i) * kRow32 + xk] = rx[i];
  };
  f32x4 acc[2][TM];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[i][t] = linattn::zero4();

  // A step's operands are in registers before its products begin. While these run the next step's are read, the
  // second next goes from registers to LDS and the third next begins to come from memory.
  struct Operands {
    f32x4 w[2], x[TM];
  } first, second;
  constexpr int kBuf = kRows * kRow32;
  auto read = [&](Operands& o, const float* buf) {
    const float* const from = buf + li * kRow32 + 16 * part + 4 * q;
#pragma unroll
    for (int i = 0; i < 2; ++i) o.w[i] = *reinterpret_cast<const f32x4*>(from + (i * kCols32 + own) * kRow32);
#pragma unroll
    for (int t = 0; t < TM; ++t) o.x[t] = *reinterpret_cast<const f32x4*>(from + (2 * kCols32 + 16 * t) * kRow32);
  };
  auto step = [&](const Operands& now, Operands& next, int k0, float* here, const float* there) {
    read(next, there);
    const Step s = step_at(k0 + 3 * kStep32);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j == 1) store(here);
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const int slot = (j - 1) * TM + t;  // of 3 TM
#pragma unroll
        for (int i = slot < 0 ? 0 : slot * kLoads / (3 * TM); i < (slot < 0 ? 0 : (slot + 1) * kLoads / (3 * TM)); ++i) load(s, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.w[i][j], now.x[t][j], acc[i][t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
  };
  load_all(0);
  store(lds);
  load_all(kStep32);
  lds_barrier();
  read(first, lds);
  store(lds + kBuf);
  load_all(2 * kStep32);
  lds_barrier();
  for (int k0 = 0; k0 < p.D; k0 += 2 * kStep32) {  // (behind the last step: zeros)
    step(first, second, k0, lds, lds + kBuf);
    if (k0 + kStep32 < p.D) step(second, first, k0 + kStep32, lds + kBuf, lds);
  }

  // The two halves' sums meet in LDS, and leave it in whole rows. A lane has columns 4 q .. 4 q + 3 of row li.
  float* const mine = lds + li * kSum + own + 4 * q;
#pragma unroll
  for (int turn = 1; turn >= 0; --turn) {
    if (part == turn) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          f32x4* const at = reinterpret_cast<f32x4*>(mine + 16 * t * kSum + i * kCols32);
          if (turn == 1) *at = acc[i][t];
          else *at = *at + acc[i][t];
        }
    }
    lds_barrier();
  }
  const int n = n0 + lane;
  if (n >= p.F) return;
  for (int m = wave; m < rows; m += kWaves32) {
    const float g = lds[m * kSum + lane], u = lds[m * kSum + kCols32 + lane];
    const int64_t at = (m0 + m) * p.F + n;
    p.h[at] = activation(g, p.act) * u;
    if (p.gate) p.gate[at] = g, p.up[at] = u;
  }
}

}  // namespace glu
}  // namespace rwkv7
