// Tiled matrix products on the matrix cores for the gated linear unit: bfloat16 operands, float32 sums.
//
//   out[m][n] = sum over segments s and k of a_s[m][k] b_s[n][k]
//
// An operand is stored with k contiguous ([m][k] or [n][k]: "rows") or with m or n contiguous ([k][m] or [k][n]:
// "columns"). Segments are pairs of operands of the same sizes, added up one after the other: the pieces of float32
// operands, or the two products of an input's gradient.
//
// A workgroup takes BM x BN of the output, a wave TM x TN tiles of 16 x 16, 64 of k at a time. Both operands' next
// NB - 1 steps come to LDS by direct loads (no registers) while the present one is multiplied. LDS holds
//  - rows: [row][64 k], 128 bytes a row, the 16-byte pieces of a row exchanged by row & 7, so that 16 lanes reading one
//    piece of 16 rows meet every bank as often;
//  - columns: blocks [64 k][128 columns], 256 bytes a row, runs of 16 columns exchanged by the bits of k that the
//    lanes of a turned read differ in.
// The exchange is in which piece of memory a lane loads; what lies behind an operand's end loads as zeros.
// The product is formed turned (rows of a D tile are n, columns m), so that a lane has four consecutive n of one m.
#pragma once

#include "glu_rules.hpp"
#include "linattn_ops.hpp"

namespace rwkv7 {
namespace glu {

using linattn::bf16x4;
using linattn::bf16x8;
using linattn::f32x4;
using linattn::u32x4;

// Four floats that need not begin on 16 bytes.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

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
  __device__ __forceinline__ static u32x4 source(const uint16_t* p, int64_t ld, int64_t first, int64_t n, int k0, int K) {
    if constexpr (COLS) {
      const int64_t left = (K - k0 < kBK ? K - k0 : kBK) * ld - first;
      return linattn::descriptor(p + (int64_t)k0 * ld + first, (uint32_t)(left * 2));
    } else {
      const int64_t rows = n - first < R ? n - first : R;
      return linattn::descriptor(p + first * ld + k0, (uint32_t)((rows * ld - k0) * 2));
    }
  }
  __device__ __forceinline__ void load(int i, u32x4 from, int k0, int K, uint32_t to, int wave) const {
    const uint32_t o = COLS || piece8 < K - k0 ? off[i] : kNowhere;
    linattn::to_lds16(from, o, to + (i * NW + wave) * 1024);
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
  if (act == RWKV7_ACT_GELU) return 0.5f * g * erfcf(g * -0.70710678f);  // 1 + erf would cancel below 0
  if (act == RWKV7_ACT_RELU2) return g > 0.f ? g * g : 0.f;
  return sigmoid(g);
}

// The first `count` of four elements from `at` on, which may begin anywhere.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ void store4(void* out, bool f32, int64_t at, int count, f32x4 x) {
  if (count >= 4) {
    if (f32) {
      *reinterpret_cast<f32x4_any*>(static_cast<float*>(out) + at) = x;
    } else {
      const bf16x4 o = __builtin_convertvector(x, bf16x4);
      *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(out) + at) = __builtin_bit_cast(u32x2_any, o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) {
        if (f32) static_cast<float*>(out)[at + i] = x[i];
        else static_cast<uint16_t*>(out)[at + i] = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
      }
  }
}

// Workgroup `block` of a product's tiles_m tiles_n splits.
template <bool ACOLS, bool BCOLS, int WM, int WN, int TM, int TN, int NB, int EPI>
__device__ __forceinline__ void tile_product(const GemmParams& p, uint32_t block) {
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
  const uint32_t id = xcd_swizzle(block, tiles * p.splits);
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
  int seg = s0 / ksteps, kt = s0 % ksteps;  // of the step to be loaded
  constexpr int kLoadsA = Loader<ACOLS, BM, NW>::kLoads, kLoadsB = Loader<BCOLS, BNp, NW>::kLoads;
  constexpr int kLoads = kLoadsA + kProducts * kLoadsB;
  struct Step {
    u32x4 a, b, b2;
    int k0;
    uint32_t to;
  };
  // Steps behind the last load zeros, which nobody reads.
  auto step_to = [&](int buf, bool any) {
    Step x;
    x.k0 = kt * kBK;
    x.to = lds0 + buf * kBuf;
    x.a = la.source(p.a[seg], p.lda, m0, p.M, x.k0, p.K);
    x.b = lb.source(second ? p.b2[seg] : p.b[seg], p.ldb, n0, p.N, x.k0, p.K);
    if constexpr (EPI == kGlu) x.b2 = lb.source(p.b2[seg], p.ldb, n0, p.N, x.k0, p.K);
    if (!any) x.a[2] = x.b[2] = x.b2[2] = 0;
    if (++kt == ksteps) {
      kt = 0;
      if (seg + 1 < p.nseg) ++seg;
    }
    return x;
  };
  auto load = [&](const Step& x, int i) {
    if (i < kLoadsA) la.load(i, x.a, x.k0, p.K, x.to, wave);
    else if (i < kLoadsA + kLoadsB) lb.load(i - kLoadsA, x.b, x.k0, p.K, x.to + kA, wave);
    else lb.load(i - kLoadsA - kLoadsB, x.b2, x.k0, p.K, x.to + kA + kB, wave);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = linattn::zero4();

  // Fragments of a half step are in registers before its products begin: those of the second half are read from LDS
  // between the first half's products, those of the next step's first half between the second's, and so are the loads
  // into this step's buffer begun. The barrier stands between the halves: everything of this step has been read then,
  // and the next step's loads, begun NB - 1 steps ago, are in. All 8 waves read at once otherwise, and multiply at once:
  // the matrix cores were idle 47% of the cycles.
  struct Half {
    bf16x8 a[TM], b[TN];
  } first, last;
  auto read_a = [&](Half& f, int buf, int h, int i) {
    f.a[i] = fragment<ACOLS>(lds + buf * kBuf, wm * (TM * 16) + i * 16, h, lane);
  };
  auto read_b = [&](Half& f, int buf, int h, int j) {
    const int col = EPI == kGlu ? wn * (TN / 2 * 16) + (j % (TN / 2)) * 16 : wn * (TN * 16) + j * 16;
    f.b[j] = fragment<BCOLS>(lds + buf * kBuf + kA + (EPI == kGlu && j >= TN / 2 ? kB : 0), col, h, lane);
  };
  // The products of row i of the wave's tiles, behind what is read for row i of the next half. Two workgroups of the
  // small shape share a compute unit and fill each other's gaps: they read all first (4% faster there, 4 to 8% slower
  // with a workgroup of 8 waves).
  constexpr bool kInRows = NW >= 8;
  auto row = [&](const Half& f, Half& next, int buf, int h, int i) {
    if (kInRows || i == 0) {
#pragma unroll
      for (int j = kInRows ? i * TN / TM : 0; j < (kInRows ? (i + 1) * TN / TM : TN); ++j) read_b(next, buf, h, j);
#pragma unroll
      for (int k = i; k < (kInRows ? i + 1 : TM); ++k) read_a(next, buf, h, k);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
    if (kInRows || i == TM - 1) __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const Step x = step_to(n, s0 + n < s1);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(x, i);
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NB - 1) * kLoads) : "memory");
#pragma unroll
  for (int j = 0; j < TN; ++j) read_b(first, 0, 0, j);
#pragma unroll
  for (int i = 0; i < TM; ++i) read_a(first, 0, 0, i);
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int i = 0; i < TM; ++i) row(first, last, buf, 1, i);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NB - 2) * kLoads) : "memory");
    const Step x = step_to(buf, s + NB < s1);
    buf = buf + 1 == NB ? 0 : buf + 1;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int l = kInRows || i == 0 ? i * kLoads / TM : kLoads; l < (kInRows ? (i + 1) * kLoads / TM : kLoads); ++l) load(x, l);
      row(last, first, buf, 0, i);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // before the workgroup's LDS is another's

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
        store4(out, true, m * p.N + n, p.N - n, acc[i][j]);
        store4(out + (int64_t)p.M * p.N, true, m * p.N + n, p.N - n, acc[i][j + TN / 2]);
      }
    } else if constexpr (EPI == kGlu) {
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) {
        const int n = n0 + wn * (TN / 2 * 16) + j * 16 + 4 * q;
        const f32x4 g = acc[i][j], u = acc[i][j + TN / 2];
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = activation(g[e], p.act) * u[e];
        store4(p.out, p.f32, m * p.N + n, p.N - n, h);
        if (p.gate) {
          store4(p.gate, p.f32, m * p.N + n, p.N - n, g);
          store4(p.up, p.f32, m * p.N + n, p.N - n, u);
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
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + wn * (TN * 16) + j * 16 + 4 * q;
        store4(out, f32, m * p.N + n, p.N - n, acc[i][j]);
      }
    }
  }
}

template <int WM, int WN, int TM, int TN, int NB>
__global__ __launch_bounds__(64 * WM * WN) void glu_forward_kernel(GemmParams p) {
  tile_product<false, true, WM, WN, TM, TN, NB, kGlu>(p, blockIdx.x);
}
// The products of the backward side by side: the input's gradient (operands in rows) and the weights' (in columns), the
// one with the longer sums first, so that the last workgroups to start are the short ones. `first`: its workgroups.
struct GradProducts {
  GemmParams x, w;
  uint32_t first;
  bool w_first;
};
template <int WM, int WN, int TM, int TN, int NB>
__global__ __launch_bounds__(64 * WM * WN) void glu_backward_kernel(GradProducts p) {
  const bool early = blockIdx.x < p.first;
  const uint32_t block = early ? blockIdx.x : blockIdx.x - p.first;
  if (early != p.w_first) tile_product<false, false, WM, WN, TM, TN, NB, kProduct>(p.x, block);
  else tile_product<true, true, WM, WN, TM, TN, NB, kProduct>(p.w, block);
}

}  // namespace glu
}  // namespace rwkv7
