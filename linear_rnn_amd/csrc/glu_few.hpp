// The gated linear unit of a few rows (a decode step): the weights are read once, which is all that counts.
//
// A workgroup takes 16 C columns of both weights, its waves the blocks of k in turn. Weights go from memory to registers
// and from there to the matrix cores, the rows of x as the other operand (up to 16 a tile): a lane reads C columns of
// the rows of k that are its part of an operand, so column c of its C is an operand whose 16 rows are the columns
// C li + c. No LDS until the waves' sums meet there.
#pragma once

#include "glu_gemm.hpp"

namespace rwkv7 {
namespace glu {

constexpr int kFewWaves = 8;

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

// C columns of a row as loaded.
template <int BYTES>
struct Words {
  uint32_t u[BYTES / 4];
};
template <int BYTES>
__device__ __forceinline__ Words<BYTES> load_words(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  if constexpr (BYTES == 16) return __builtin_bit_cast(Words<16>, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
  else if constexpr (BYTES == 8) return __builtin_bit_cast(Words<8>, __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0));
  else return __builtin_bit_cast(Words<4>, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}

// acc[weights][c] += columns C li + c (rows of the result) times rows m of x (its columns), over k0 .. k0 + kBlock - 1.
template <bool F32, int C, int MT>
struct FewBlock;
template <int C, int MT>
struct FewBlock<false, C, MT> {
  static constexpr int kBlock = 32;
  Words<2 * C> w[2][8];  // rows k0 + 8 q + j
  bf16x8 x[MT];
  __device__ __forceinline__ void load(const FewParams& p, int k0, int col, int lane) {
    const int q = lane >> 4, li = lane & 15;
    const int64_t at = (int64_t)k0 * p.F;
    const uint32_t bytes = (uint32_t)(p.D - k0 < kBlock ? p.D - k0 : kBlock) * (uint32_t)p.F * 2;
    const auto bg = linattn::buffer(static_cast<const uint16_t*>(p.w_gate) + at, bytes);
    const auto bu = linattn::buffer(static_cast<const uint16_t*>(p.w_up) + at, bytes);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t off = ((uint32_t)(8 * q + j) * p.F + col + C * li) * 2;
      w[0][j] = load_words<2 * C>(bg, off);
      w[1][j] = load_words<2 * C>(bu, off);
    }
    const int k = k0 + 8 * q;
    const auto bx = linattn::buffer(p.x, (uint32_t)p.M * p.D * 2);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bx, ((uint32_t)(16 * t + li) * p.D + k) * 2, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = k + 2 * i < p.D ? v[i] : 0;  // not the next row's
      x[t] = __builtin_bit_cast(bf16x8, v);
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[2][C][MT]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[i][2 * j].u[c >> 1], hi = w[i][2 * j + 1].u[c >> 1];
          a[j] = __builtin_amdgcn_perm(hi, lo, c & 1 ? 0x07060302u : 0x05040100u);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
          acc[i][c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), x[t], acc[i][c][t], 0, 0, 0);
      }
  }
};
template <int C, int MT>
struct FewBlock<true, C, MT> {
  static constexpr int kBlock = 16;
  Words<4 * C> w[2][4];  // rows k0 + 4 q + j
  f32x4 x[MT];
  __device__ __forceinline__ void load(const FewParams& p, int k0, int col, int lane) {
    const int q = lane >> 4, li = lane & 15;
    const int64_t at = (int64_t)k0 * p.F;
    const uint32_t bytes = (uint32_t)(p.D - k0 < kBlock ? p.D - k0 : kBlock) * (uint32_t)p.F * 4;
    const auto bg = linattn::buffer(static_cast<const float*>(p.w_gate) + at, bytes);
    const auto bu = linattn::buffer(static_cast<const float*>(p.w_up) + at, bytes);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t off = ((uint32_t)(4 * q + j) * p.F + col + C * li) * 4;
      w[0][j] = load_words<4 * C>(bg, off);
      w[1][j] = load_words<4 * C>(bu, off);
    }
    const int k = k0 + 4 * q;
    const auto bx = linattn::buffer(p.x, (uint32_t)p.M * p.D * 4);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      x[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bx, ((uint32_t)(16 * t + li) * p.D + k) * 4, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) x[t][i] = k + i < p.D ? x[t][i] : 0.f;  // not the next row's
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[2][C][MT]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[i][c][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i][j].u[c]), x[t][j], acc[i][c][t], 0, 0, 0);
  }
};

// A lane's element i of acc[..][c]: column C (4 q + i) + c, row m = li of x.
template <bool F32, int C, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void glu_few_kernel(FewParams p) {
  constexpr int kCols = 16 * C, kRow = kCols + 4;  // floats, so that lanes of different rows meet different banks
  __shared__ float sums[kFewWaves][16][kRow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = blockIdx.x * kCols;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;  // its rows
  {
    constexpr int esz = F32 ? 4 : 2;
    p.x = static_cast<const char*>(p.x) + m0 * p.D * esz;
    p.h = static_cast<char*>(p.h) + m0 * p.F * esz;
    if (p.gate) p.gate = static_cast<char*>(p.gate) + m0 * p.F * esz, p.up = static_cast<char*>(p.up) + m0 * p.F * esz;
    p.M = p.M - (int)m0 < 16 * MT ? p.M - (int)m0 : 16 * MT;
  }
  f32x4 acc[2][C][MT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][c][t] = linattn::zero4();
  using Block = FewBlock<F32, C, MT>;
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
    // (row, column) pairs, threads side by side the columns of a row
    constexpr int kEach = 16 * kCols / (64 * kFewWaves), kRows = 16 / kEach;
    const int mine = threadIdx.x / kCols, n0 = threadIdx.x % kCols;
    float v[2][kEach];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) sums[wave][li][C * (4 * q + r) + c] = acc[i][c][t][r];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += sums[w][mine + e * kRows][n0];
        v[i][e] = s;
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int m = 16 * t + mine + e * kRows, n = col + n0;
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
