// Tiled matrix products on the matrix cores for the gated linear unit: bfloat16 operands, float32 sums.
//
//   out[m][n] = sum over segments s and k of a_s[m][k] b_s[n][k]
//
// An operand is stored with k contiguous ([m][k] or [n][k]: "rows") or with m or n contiguous ([k][m] or [k][n]:
// "columns"). Segments are pairs of operands of the same sizes, added up one after the other: the pieces of float32
// operands, or the two products of an input's gradient.
//
// A workgroup takes BM x BN of the output, a wave TM x TN tiles of 16 x 16, 64 of k at a time. Both operands' next
// 64 of k come to LDS by direct loads (no registers) while the present ones are multiplied. LDS holds
//  - rows: [row][64 k], 128 bytes a row, the 16-byte pieces of a row exchanged by row & 7, so that 16 lanes reading one
//    piece of 16 rows meet every bank as often;
//  - columns: blocks [64 k][128 columns], 256 bytes a row, runs of 16 columns exchanged by the bits of k that the
//    lanes of a turned read differ in.
// The exchange is in which piece of memory a lane loads; what lies behind an operand's end loads as zeros.
// The product is formed turned (rows of a D tile are n, columns m), so that a lane has four consecutive n of one m.
#pragma once

#include "linattn_ops.hpp"

namespace rwkv7 {
namespace glu {

using linattn::bf16x4;
using linattn::bf16x8;
using linattn::f32x4;
using linattn::u32x4;

constexpr int kBK = 64;
constexpr int kMaxSegs = 12;
constexpr uint32_t kNowhere = 0x80000000u;

struct GemmParams {
  const uint16_t* a[kMaxSegs];
  const uint16_t* b[kMaxSegs];
  const uint16_t* b2[kMaxSegs];  // the second of two products with the same a
  int64_t lda, ldb;              // elements, multiples of 8
  int32_t M, N, K;               // N: of one product
  int32_t nseg;
  int32_t tiles_m, tiles_n;      // tiles_n: of all products
  int32_t splits;                // workgroups that share the sum over segments and k
  void* out;                     // [M, N]
  void* out2;                    // of the second product
  bool two;                      // kProduct: there is a second one
  void* gate;                    // pre-activations, may be null
  void* up;
  float* partial;                // [splits][products][M][N] with splits > 1, in place of the outputs
  bool f32;                      // element type of the outputs
  int act;
};

enum Epilogue {
  kGlu,      // b and b2 side by side in a tile: out = act(a b) (a b2)
  kProduct,  // out = a b, and out2 = a b2 in tiles of their own where there is a b2
};

// One operand's part in a step: where a lane loads from, and what to LDS. R: rows or columns of the tile.
template <bool COLS, int R, int NW>
struct Loader {
  static constexpr int kLoads = R * kBK * 2 / (1024 * NW);  // of a wave: 1 KiB each
  uint32_t off[kLoads];
  int piece8;  // first k of the lane's piece (rows)
  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if constexpr (COLS) {
        const int unit = i * NW + wave, block = unit / 16, k = unit % 16 * 4 + (lane >> 4);
        const int key = (k & 3) | (k >> 3 & 1) << 2;
        off[i] = (uint32_t)((k * ld + block * 128 + (((lane & 15) ^ key << 1) * 8)) * 2);
      } else {
        const int row = (i * NW + wave) * 8 + (lane >> 3);
        piece8 = ((lane & 7) ^ (row & 7)) * 8;
        off[i] = (uint32_t)((row * ld + piece8) * 2);
      }
    }
  }
  // The tile's step k0 .. k0 + 63 of an operand; `first`: its first row or column, `n` how many the operand has.
  __device__ __forceinline__ void fetch(const uint16_t* p, int64_t ld, int64_t first, int64_t n, int k0, int K, uint32_t to,
                                        int wave) const {
    if constexpr (COLS) {
      const int64_t left = (K - k0 < kBK ? K - k0 : kBK) * ld - first;
      const u32x4 d = linattn::descriptor(p + (int64_t)k0 * ld + first, (uint32_t)(left * 2));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) linattn::to_lds16(d, off[i], to + (i * NW + wave) * 1024);
    } else {
      const int64_t rows = n - first < R ? n - first : R;
      const u32x4 d = linattn::descriptor(p + first * ld + k0, (uint32_t)((rows * ld - k0) * 2));
      const bool inside = piece8 < K - k0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) linattn::to_lds16(d, inside ? off[i] : kNowhere, to + (i * NW + wave) * 1024);
    }
  }
};
// Operand of 16 rows or columns from `first` on, k = 32 h + 8 q .. + 7.
template <bool COLS>
__device__ __forceinline__ bf16x8 fragment(const char* lds, int first, int h, int lane) {
  const int q = lane >> 4;
  if constexpr (COLS) {
    const int r = lane >> 2 & 3, key = r | (q & 1) << 2;
    const char* at = lds + (first >> 7) * (kBK * 256) + (32 * h + 8 * q + r) * 256 + (((first >> 4 & 7) ^ key) * 32) + (lane & 3) * 8;
    return linattn::join(linattn::turned4(at), linattn::turned4(at + 4 * 256));
  } else {
    return *reinterpret_cast<const bf16x8*>(lds + (first + (lane & 15)) * 128 + (((4 * h + q) ^ (lane & 7)) * 16));
  }
}

// ---- activations
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}
__device__ __forceinline__ float activation(float g, int act) {
  if (act == RWKV7_ACT_SILU) return g * sigmoid(g);
  if (act == RWKV7_ACT_GELU) return 0.5f * g * (1.f + erff(g * 0.70710678f));
  if (act == RWKV7_ACT_RELU2) return g > 0.f ? g * g : 0.f;
  return sigmoid(g);
}

// Four consecutive n of row m.
__device__ __forceinline__ void store4(void* out, bool f32, int64_t ld, int64_t m, int n, int N, f32x4 x) {
  const int64_t at = m * ld + n;
  if (n + 3 < N && (ld & 3) == 0) {
    if (f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      const bf16x4 o = __builtin_convertvector(x, bf16x4);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = __builtin_bit_cast(uint2, o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) {
        if (f32) static_cast<float*>(out)[at + i] = x[i];
        else static_cast<uint16_t*>(out)[at + i] = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
      }
  }
}

template <bool ACOLS, bool BCOLS, int WM, int WN, int TM, int TN, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void glu_gemm_kernel(GemmParams p) {
  constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  constexpr int kProducts = EPI == kGlu ? 2 : 1;  // in one tile
  constexpr int BNp = BN / kProducts;
  constexpr int kA = BM * kBK * 2, kB = BNp * kBK * 2, kBuf = kA + kProducts * kB;
  extern __shared__ char lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // Neighbouring tiles on one die: eight rows of tiles at a time.
  const uint32_t tiles = p.tiles_m * p.tiles_n;
  const uint32_t id = xcd_swizzle(blockIdx.x, tiles * p.splits);
  const uint32_t split = id / tiles, t = id % tiles;
  const uint32_t group = t / (8 * p.tiles_n), in = t % (8 * p.tiles_n);
  const uint32_t high = p.tiles_m - group * 8 < 8 ? p.tiles_m - group * 8 : 8;
  const uint32_t tm0 = group * 8 + in % high;
  uint32_t tn0 = in / high;
  const bool second = EPI == kProduct && p.two && tn0 >= (uint32_t)p.tiles_n / 2;
  if (second) tn0 -= p.tiles_n / 2;
  const int64_t m0 = (int64_t)tm0 * BM;
  const int n0 = tn0 * BNp;

  const int ksteps = (p.K + kBK - 1) / kBK, total = ksteps * p.nseg;
  const int s0 = (int)((int64_t)total * split / p.splits), s1 = (int)((int64_t)total * (split + 1) / p.splits);

  Loader<ACOLS, BM, NW> la;
  Loader<BCOLS, BNp, NW> lb;
  la.init(p.lda, wave, lane);
  lb.init(p.ldb, wave, lane);
  int seg = s0 / ksteps, kt = s0 % ksteps;  // of the step to be fetched
  auto fetch = [&](int buf) {
    const uint32_t to = lds0 + buf * kBuf;
    const int k0 = kt * kBK;
    const uint16_t* b = second ? p.b2[seg] : p.b[seg];
    la.fetch(p.a[seg], p.lda, m0, p.M, k0, p.K, to, wave);
    lb.fetch(b, p.ldb, n0, p.N, k0, p.K, to + kA, wave);
    if constexpr (EPI == kGlu) lb.fetch(p.b2[seg], p.ldb, n0, p.N, k0, p.K, to + kA + kB, wave);
    if (++kt == ksteps) kt = 0, ++seg;
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = linattn::zero4();

  if (s0 < s1) fetch(0);
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + 1 < s1) fetch(buf ^ 1);
    const char* at = lds + buf * kBuf;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 a[TM], b[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int col = EPI == kGlu ? wn * (TN / 2 * 16) + (j % (TN / 2)) * 16 : wn * (TN * 16) + j * 16;
        b[j] = fragment<BCOLS>(at + kA + (EPI == kGlu && j >= TN / 2 ? kB : 0), col, h, lane);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) a[i] = fragment<ACOLS>(at, wm * (TM * 16) + i * 16, h, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    }
    buf ^= 1;
  }

  const int q = lane >> 4, li = lane & 15;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + wm * (TM * 16) + i * 16 + li;
    if (m >= p.M) continue;
    if (EPI == kGlu && p.splits > 1) {
      float* out = p.partial + (int64_t)split * 2 * p.M * p.N;
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) {
        const int n = n0 + wn * (TN / 2 * 16) + j * 16 + 4 * q;
        store4(out, true, p.N, m, n, p.N, acc[i][j]);
        store4(out + (int64_t)p.M * p.N, true, p.N, m, n, p.N, acc[i][j + TN / 2]);
      }
    } else if constexpr (EPI == kGlu) {
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) {
        const int n = n0 + wn * (TN / 2 * 16) + j * 16 + 4 * q;
        const f32x4 g = acc[i][j], u = acc[i][j + TN / 2];
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = activation(g[e], p.act) * u[e];
        store4(p.out, p.f32, p.N, m, n, p.N, h);
        if (p.gate) {
          store4(p.gate, p.f32, p.N, m, n, p.N, g);
          store4(p.up, p.f32, p.N, m, n, p.N, u);
        }
      }
    } else {
      void* out = second ? p.out2 : p.out;
      bool f32 = p.f32;
      if (p.splits > 1) {
        const int64_t number = split * (p.two ? 2 : 1) + (second ? 1 : 0);
        out = p.partial + number * p.M * p.N;
        f32 = true;
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) store4(out, f32, p.N, m, n0 + wn * (TN * 16) + j * 16 + 4 * q, p.N, acc[i][j]);
    }
  }
}

}  // namespace glu
}  // namespace rwkv7
