// The gated linear unit of a few rows (a decode step): the weights are read once, which is all that counts.
//
// A workgroup takes 64 columns of both weights, its waves the blocks of k in turn. Weights go from memory to registers
// and from there to the matrix cores, the rows of x as the other operand (up to 16 a tile): a lane reads 4 columns of
// the rows of k that are its part of an operand, so column c of its 4 is an operand whose 16 rows are the columns
// 4 li + c. No LDS until the waves' sums meet there.
#pragma once

#include "glu_gemm.hpp"

namespace rwkv7 {
namespace glu {

constexpr int kFewWaves = 8;
constexpr int kFewCols = 64;  // of a workgroup

struct FewParams {
  const void* x;  // [M, D]
  const void* w_gate;
  const void* w_up;
  void* h;
  void* gate;  // may be null
  void* up;
  int32_t M, D, F;
  int act;
};

// acc[weights][c] += columns 4 li + c (rows of the result) times rows m of x (its columns), over k0 .. k0 + kBlock - 1.
template <bool F32, int MT>
struct FewBlock;
template <int MT>
struct FewBlock<false, MT> {
  static constexpr int kBlock = 32;
  uint2 w[2][8];  // rows k0 + 8 q + j
  bf16x8 x[MT];
  __device__ __forceinline__ void load(const FewParams& p, int k0, int col, int lane) {
    const int q = lane >> 4, li = lane & 15;
    const int64_t at = (int64_t)k0 * p.F;
    const uint32_t bytes = (uint32_t)(p.D - k0 < kBlock ? p.D - k0 : kBlock) * (uint32_t)p.F * 2;
    const auto bg = linattn::buffer(static_cast<const uint16_t*>(p.w_gate) + at, bytes);
    const auto bu = linattn::buffer(static_cast<const uint16_t*>(p.w_up) + at, bytes);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t off = ((uint32_t)(8 * q + j) * p.F + col + 4 * li) * 2;
      w[0][j] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(bg, off, 0, 0));
      w[1][j] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(bu, off, 0, 0));
    }
    const int k = k0 + 8 * q;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = 16 * t + li;
      u32x4 v = {0, 0, 0, 0};
      if (m < p.M && k < p.D) v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + (int64_t)m * p.D + k);
      x[t] = __builtin_bit_cast(bf16x8, v);
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[2][4][MT]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = c < 2 ? w[i][2 * j].x : w[i][2 * j].y, hi = c < 2 ? w[i][2 * j + 1].x : w[i][2 * j + 1].y;
          a[j] = __builtin_amdgcn_perm(hi, lo, c & 1 ? 0x07060302u : 0x05040100u);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
          acc[i][c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), x[t], acc[i][c][t], 0, 0, 0);
      }
  }
};
template <int MT>
struct FewBlock<true, MT> {
  static constexpr int kBlock = 16;
  f32x4 w[2][4];  // rows k0 + 4 q + j
  f32x4 x[MT];
  __device__ __forceinline__ void load(const FewParams& p, int k0, int col, int lane) {
    const int q = lane >> 4, li = lane & 15;
    const int64_t at = (int64_t)k0 * p.F;
    const uint32_t bytes = (uint32_t)(p.D - k0 < kBlock ? p.D - k0 : kBlock) * (uint32_t)p.F * 4;
    const auto bg = linattn::buffer(static_cast<const float*>(p.w_gate) + at, bytes);
    const auto bu = linattn::buffer(static_cast<const float*>(p.w_up) + at, bytes);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t off = ((uint32_t)(4 * q + j) * p.F + col + 4 * li) * 4;
      w[0][j] = __builtin_bit_cast(f32x4, linattn::load16(bg, off));
      w[1][j] = __builtin_bit_cast(f32x4, linattn::load16(bu, off));
    }
    const int k = k0 + 4 * q;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = 16 * t + li;
      x[t] = linattn::zero4();
      if (m < p.M && k < p.D) x[t] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.x) + (int64_t)m * p.D + k);
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[2][4][MT]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[i][c][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i][j][c], x[t][j], acc[i][c][t], 0, 0, 0);
  }
};

// A lane's element i of acc[..][c]: column 4 (4 q + i) + c, row m = li of x.
template <bool F32, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void glu_few_kernel(FewParams p) {
  constexpr int kRow = kFewCols + 4;  // floats, so that lanes of different rows meet different banks
  __shared__ float sums[kFewWaves][16][kRow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = blockIdx.x * kFewCols;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;  // its rows
  {
    constexpr int esz = F32 ? 4 : 2;
    p.x = static_cast<const char*>(p.x) + m0 * p.D * esz;
    p.h = static_cast<char*>(p.h) + m0 * p.F * esz;
    if (p.gate) p.gate = static_cast<char*>(p.gate) + m0 * p.F * esz, p.up = static_cast<char*>(p.up) + m0 * p.F * esz;
    p.M = p.M - (int)m0 < 16 * MT ? p.M - (int)m0 : 16 * MT;
  }
  f32x4 acc[2][4][MT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][c][t] = linattn::zero4();
  using Block = FewBlock<F32, MT>;
  constexpr int kStride = kFewWaves * Block::kBlock;
  Block now, next;
  int k = wave * Block::kBlock;
  if (k < p.D) now.load(p, k, col, lane);
  for (; k < p.D; k += 2 * kStride) {
    const bool more = k + kStride < p.D;
    if (more) next.load(p, k + kStride, col, lane);
    now.multiply(acc);
    if (!more) break;
    if (k + 2 * kStride < p.D) now.load(p, k + 2 * kStride, col, lane);
    next.multiply(acc);
  }

  const int q = lane >> 4, li = lane & 15;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (16 * t >= p.M) break;
    // up to two (row, column) pairs a thread: threads 0 .. 63 the columns of a row
    constexpr int kEach = 16 * kFewCols / (64 * kFewWaves);
    float v[2][kEach];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x4 o = {acc[i][0][t][r], acc[i][1][t][r], acc[i][2][t][r], acc[i][3][t][r]};
        *reinterpret_cast<f32x4*>(&sums[wave][li][4 * (4 * q + r)]) = o;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int m = (threadIdx.x >> 6) + e * kFewWaves, n = threadIdx.x & 63;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += sums[w][m][n];
        v[i][e] = s;
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int m = 16 * t + (threadIdx.x >> 6) + e * kFewWaves, n = col + (threadIdx.x & 63);
      if (m >= p.M || n >= p.F) continue;
      const int64_t at = (int64_t)m * p.F + n;
      const float h = activation(v[0][e], p.act) * v[1][e];
      if constexpr (F32) {
        static_cast<float*>(p.h)[at] = h;
        if (p.gate) static_cast<float*>(p.gate)[at] = v[0][e], static_cast<float*>(p.up)[at] = v[1][e];
      } else {
        static_cast<uint16_t*>(p.h)[at] = __builtin_bit_cast(uint16_t, (__bf16)h);
        if (p.gate) {
          static_cast<uint16_t*>(p.gate)[at] = __builtin_bit_cast(uint16_t, (__bf16)v[0][e]);
          static_cast<uint16_t*>(p.up)[at] = __builtin_bit_cast(uint16_t, (__bf16)v[1][e]);
        }
      }
    }
  }
}

}  // namespace glu
}  // namespace rwkv7
