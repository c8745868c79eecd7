// Chunk algebra of the linear attention with a decay for each head, shared by the prompt
// kernels and the backward.
//
// Recurrence per (batch, head), state S [value i, key j] in float32, w_t = exp(log_w_t) a scalar:
//   S_t = w_t S_{t-1} + v_t k_t^T,   y_t = S_t r_t.
// A wave works on 32 tokens (two tiles of 16) at a time. With c_t the inclusive sum of log w from
// the first of them, D_ij = exp(c_i - c_j) for i >= j (else 0), S_0 the state before them:
//   y_i = sum_j D_ij (r_i . k_j) v_j + exp(c_i) S_0 r_i
//   S_32 = exp(c_31) S_0 + sum_j exp(c_31 - c_j) v_j k_j^T
// The scalar decay needs no solve (unlike the WKV-7 chunk form), so everything is 16x16x32 bf16
// MFMA products and row or column scales.
//
// Numbers. The operands are bfloat16 pieces (round to nearest) whose sum is the value: a bfloat16
// input is one piece, exact; a float32 input and every scaled intermediate are two or three
// (16 or 24 significant bits, float32's exponent range). Products keep the pairs of pieces whose
// orders add to at most 2, which leaves errors of about 2^-24, so a float32 result (the state, the
// decay's gradient, everything of a float32 call) is as good as float32 arithmetic; where the
// result is rounded to bfloat16 (2^-8) two pieces (2^-16) do. Three bf16 products cost less than
// one of the float32 matrix instructions (1/16 of the bf16 rate). Sums of log w are float64, so a
// reset (log w = -inf, held as -1e4: every exponential of a sum with it is 0) does not take digits
// from the tokens behind it.
//
// Layouts (wave64; l = lane, li = l % 16, q = l / 16; e = 0..1, i = 0..3):
//   operand A[row = li][slot 8q + 4e + i], B[slot 8q + 4e + i][col = li]; D[row = 4q + i][col = li].
// A sum over slots may number them freely, as long as both operands do it alike. So:
//  - channel number 32h + 8q + 4e + i is slot (q, e, i) of depth step h: a lane's natural 16 bytes of
//    a token's row are an operand (token = li), and row 4q + i of a D tile t = 2h + e stands for the
//    same channel: the tiles of a product over tokens are, two by two, operands of a product over
//    channels, and a token's 8 channels of tiles 2h, 2h + 1 are one 16-byte store;
//  - token 16J + 4q + i is slot (q, e = J, i): the two token tiles of a D column are an operand of
//    a product over the 32 tokens.
// The only layout change left is to turn a token-row operand into a channel-row one: bfloat16 rows
// are read from LDS turned, and so are float32 rows in the gradients' kernel, which keeps their pieces
// there; in the prompt and state kernels float32 rows go by registers, and through products with a
// 0/1 matrix (exact).
#pragma once

#include "lane_sums.hpp"
#include "wkv7_device.hpp"

namespace rwkv7 {
namespace linattn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kSub = 32;              // tokens a wave takes at a time
constexpr int kWaves = 4;             // waves of a workgroup
constexpr int kBlk = kSub * kWaves;   // tokens a workgroup takes at a time

template <int NP>
struct Op {
  bf16x8 p[NP];
};

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// acc += A B over 32 slots; the smallest products first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Op<NA>& a, const Op<NB>& b, f32x4 acc) {
#pragma unroll
  for (int s = NA + NB - 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (s <= 2 && j >= 0 && j < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], acc, 0, 0, 0);
    }
  return acc;
}

// a b + c with one rounding.
__device__ __forceinline__ f32x4 fma4(f32x4 a, float b, f32x4 c) {
  f32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = fmaf(a[i], b, c[i]);
  return o;
}

// Elements i, i + 1 of an operand from two float32 values, in NP pieces; the remainders are exact in float32.
// (A remainder as one two-term dot product with (-1, 0), v_dot2c_f32_bf16, saves two of five instructions and
// measured far slower: the prompt of B=4 T=16384 H=64 1160 us against 700.)
template <int NP>
__device__ __forceinline__ void put2(Op<NP>& o, int i, float x0, float x1) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const bf16x2 h = __builtin_convertvector(f32x2{x0, x1}, bf16x2);
    o.p[p][i] = h[0];
    o.p[p][i + 1] = h[1];
    if (p + 1 < NP) {
      const uint32_t b = __builtin_bit_cast(uint32_t, h);
      x0 -= __uint_as_float(b << 16);
      x1 -= __uint_as_float(b & 0xffff0000u);
    }
  }
}
// An operand from two D tiles (slots e = 0 and e = 1).
template <int NP>
__device__ __forceinline__ Op<NP> pack(f32x4 d0, f32x4 d1) {
  Op<NP> o;
  put2(o, 0, d0[0], d0[1]);
  put2(o, 2, d0[2], d0[3]);
  put2(o, 4, d1[0], d1[1]);
  put2(o, 6, d1[2], d1[3]);
  return o;
}

// ---- global memory, by buffer descriptors: an access behind `bytes` reads zeros or writes nothing,
// which is how tokens behind a sequence's end are left out.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t b, uint32_t off, u32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(x, b, off, 0, 0);
}

// The same descriptor as four scalar words, for the direct loads to LDS: 16 (or 4) bytes a lane, lane l's to
// `lds` + 16 l (4 l), zeros from behind the end. vmcnt counts them and the caller waits for them. A memory instruction
// may read a scalar register five wait states after the vector unit (a readfirstlane, as the descriptor's) wrote it and
// M0 one after it was set. The compiler keeps no such distances into assembly, so the idle states are in here.
__device__ __forceinline__ u32x4 descriptor(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00027000u};
}
__device__ __forceinline__ void to_lds16(u32x4 b, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(b), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory");
}
// Without temporal hint, for what no later kernel of the call reads.
__device__ __forceinline__ void to_lds16_last(u32x4 b, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" ::"v"(off), "s"(b), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory");
}
__device__ __forceinline__ void to_lds4(u32x4 b, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(b), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory");
}

// Rows of 64 bfloat16 in LDS. Where 16-byte piece `piece` of row `row` is: exchanged within the row so that reads of one
// piece of 16 rows, and turned reads of four pieces of 8 rows, meet as many banks as there are.
constexpr int kRow = kN * 2;  // bytes
__device__ __forceinline__ int row_key(int row) { return (row >> 1 & 1) | (row >> 2 & 2) | (row & 4); }
__device__ __forceinline__ int swizzled(int row, int piece) { return row * kRow + 16 * (piece ^ row_key(row)); }
// Turned: of each 16 lanes, lanes 4r .. 4r + 3 give the places of 16 consecutive elements of a row r, lane c gets
// element c of the four rows.
__device__ __forceinline__ bf16x4 turned4(const char* at) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(
      bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// One tensor's 32 tokens of one head, as loaded: [token tile][depth step].
template <bool F32>
struct Raw {
  u32x4 x[2][2][F32 ? 2 : 1];
};
// Pieces of an input element.
template <bool F32>
constexpr int kIn = F32 ? 3 : 1;
template <bool F32>
constexpr uint32_t kEsz = F32 ? 4 : 2;

template <bool F32>
__device__ __forceinline__ void load_raw(Raw<F32>& o, __amdgpu_buffer_rsrc_t b, uint32_t row_bytes, int lane) {
  const uint32_t off = (lane & 15) * row_bytes + (lane >> 4) * 8 * kEsz<F32>;
#pragma unroll
  for (int J = 0; J < 2; ++J)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < (F32 ? 2 : 1); ++m)
        o.x[J][h][m] = load16(b, off + J * 16 * row_bytes + h * 32 * kEsz<F32> + 16 * m);
}
// The operand of a lane's eight channels as loaded.
template <bool F32>
__device__ __forceinline__ Op<kIn<F32>> pieces(const u32x4 (&x)[F32 ? 2 : 1]) {
  Op<kIn<F32>> o;
  if constexpr (F32) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      put2(o, 4 * m, __uint_as_float(x[m][0]), __uint_as_float(x[m][1]));
      put2(o, 4 * m + 2, __uint_as_float(x[m][2]), __uint_as_float(x[m][3]));
    }
  } else {
    o.p[0] = __builtin_bit_cast(bf16x8, x[0]);
  }
  return o;
}
template <bool F32>
__device__ __forceinline__ Op<kIn<F32>> natural(const Raw<F32>& r, int J, int h) {
  return pieces<F32>(r.x[J][h]);
}
// Two D tiles (channels of a token column) as eight consecutive channels of a [token][channel] tensor.
template <bool F32>
__device__ __forceinline__ void store_pair(__amdgpu_buffer_rsrc_t b, uint32_t off, f32x4 d0, f32x4 d1) {
  if constexpr (F32) {
    store16(b, off, __builtin_bit_cast(u32x4, d0));
    store16(b, off + 16, __builtin_bit_cast(u32x4, d1));
  } else {
    store16(b, off, __builtin_bit_cast(u32x4, pack<1>(d0, d1).p[0]));
  }
}

// The 0/1 matrices E_e: B[slot (q, e', i)][col li] = 1 where channel 8q + 4e' + i is that of row li of
// a D tile (2h + e).
struct Turn {
  Op<1> e[2];
};
__device__ __forceinline__ Turn make_turn(int lane) {
  Turn t;
  const int li = lane & 15, q = lane >> 4;
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int s = 0; s < 8; ++s) t.e[e].p[0][s] = (__bf16)((q == (li >> 2) && s == 4 * e + (li & 3)) ? 1.f : 0.f);
  return t;
}
// Tile t of a tensor, turned: D rows are the 16 tokens of tile J, columns the tile's channels. The
// sum of an input's pieces, so exactly the input's values.
template <int NP>
__device__ __forceinline__ f32x4 turned(const Op<NP>& x, const Turn& E, int t) {
  return mma(x, E.e[t & 1], zero4());
}
// The same as an operand over the 32 tokens (row or column li = channel of tile t): its pieces are
// the input's pieces, turned one by one.
template <int NP>
__device__ __forceinline__ Op<NP> turned_op(const Op<NP>& x0, const Op<NP>& x1, const Turn& E, int t) {
  Op<NP> o;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const Op<1> a0{{x0.p[p]}}, a1{{x1.p[p]}};
    o.p[p] = pack<1>(turned(a0, E, t), turned(a1, E, t)).p[0];
  }
  return o;
}

// ---- decays of a wave's 32 tokens
struct Decay {
  float col[2];      // exp(c) of token 16I + li
  float row[2][4];   // exp(c_31 - c) of token 16J + 4q + i: what is left of it at the end
  f32x4 d00, d01, d11;  // D with the tokens j as rows: tile (J, I) has rows j = 16J + 4q + i, columns i = 16I + li
  float all;         // exp(c_31)
};

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double readlane_f64(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float exp_diff(double a, double b) { return __builtin_amdgcn_exp2f((float)(a - b)); }

// Inclusive sums of log2 w over the wave's 32 tokens; lane l (and l + 32) holds token l % 32.
__device__ __forceinline__ double log_sums(float log_w, int lane) {
  // -inf and what is as good as it; a NaN stays one
  double x = (double)(log_w < -1e4f ? -1e4f : log_w) * 1.4426950408889634;
  x += dpp_f64<0x111>(x);  // row_shr:1, 2, 4, 8 (zeros come in): inclusive sums of 16 lanes
  x += dpp_f64<0x112>(x);
  x += dpp_f64<0x114>(x);
  x += dpp_f64<0x118>(x);
  const double first = readlane_f64(x, 15);
  return (lane & 16) ? x + first : x;
}
// `sums`: 32 doubles of LDS that are this wave's own.
__device__ __forceinline__ Decay make_decay(float log_w, double* sums, int lane) {
  const int li = lane & 15, q = lane >> 4;
  const double c = log_sums(log_w, lane);
  if (lane < kSub) sums[lane] = c;
  __builtin_amdgcn_wave_barrier();
  const double end = readlane_f64(c, 31);
  Decay d;
  double cc[2], cr[2][4];
#pragma unroll
  for (int J = 0; J < 2; ++J) {
    cc[J] = sums[16 * J + li];
#pragma unroll
    for (int i = 0; i < 4; ++i) cr[J][i] = sums[16 * J + 4 * q + i];
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int J = 0; J < 2; ++J) {
    d.col[J] = exp_diff(cc[J], 0.0);
#pragma unroll
    for (int i = 0; i < 4; ++i) d.row[J][i] = exp_diff(end, cr[J][i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // in the tiles on the diagonal also where D is 0 (masked_j() leaves that out)
    d.d00[i] = exp_diff(cc[0], cr[0][i]);
    d.d01[i] = exp_diff(cc[1], cr[0][i]);
    d.d11[i] = exp_diff(cc[1], cr[1][i]);
  }
  d.all = exp_diff(end, 0.0);
  return d;
}
// p D in a tile on the diagonal, 0 for the pairs that D leaves out (whatever p and the factor are there):
// rows j <= columns i, or rows i >= columns j.
__device__ __forceinline__ f32x4 masked_j(f32x4 p, f32x4 d, int lane) {
  f32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (4 * (lane >> 4) + i <= (lane & 15)) ? p[i] * d[i] : 0.f;
  return o;
}
__device__ __forceinline__ f32x4 masked_i(f32x4 p, f32x4 d, int lane) {
  f32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (4 * (lane >> 4) + i >= (lane & 15)) ? p[i] * d[i] : 0.f;
  return o;
}

// ---- state tiles. A state is [value][key] in memory; tile (t, u) of the wave's layout is D with rows the keys of
// tile t and columns the values of tile u: a lane's four elements are four consecutive keys of one value row.
// Between waves a state is 16 tiles [4t + u][lane].
__device__ __forceinline__ int channel(int t, int rho) { return 32 * (t >> 1) + 8 * (rho >> 2) + 4 * (t & 1) + (rho & 3); }
__device__ __forceinline__ uint32_t state_offset(int t, int u, int lane) {  // in elements
  return channel(u, lane & 15) * kN + channel(t, 4 * (lane >> 4));
}

// Where a call's tokens are: head h of sequence b, `len` valid tokens of T.
struct Seq {
  int64_t T;
  int32_t H;
  const int32_t* lens;  // may be null
};
__device__ __forceinline__ int64_t seq_len(const Seq& s, int64_t b) {
  if (!s.lens) return s.T;
  const int64_t n = s.lens[b];
  return n < 0 ? 0 : n < s.T ? n : s.T;
}
// `n` tokens (at most `most`) of a [B, T, H, 64] tensor from token t0 on, head h first: where they start, and the
// bytes to the end of the last one's 64 channels.
struct Span {
  const char* base;
  uint32_t bytes;
};
template <uint32_t ESZ>
__device__ __forceinline__ Span token_span(const void* base, const Seq& s, int64_t b, int32_t h, int64_t t0, int64_t n,
                                           int most) {
  const int64_t left = n <= 0 ? 0 : n < most ? n : most;
  return Span{static_cast<const char*>(base) + ((b * s.T + t0) * s.H + h) * (int64_t)(kN * ESZ),
              left ? ((uint32_t)(left - 1) * s.H * kN + kN) * ESZ : 0};
}
template <uint32_t ESZ>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_buffer(const void* base, const Seq& s, int64_t b, int32_t h,
                                                               int64_t t0, int64_t n, int most) {
  const Span x = token_span<ESZ>(base, s, b, h, t0, n, most);
  return buffer(x.base, x.bytes);
}
// Tile tu = 4t + u of state number `index` of an array of states in the caller's layout.
__device__ __forceinline__ f32x4* state_tile(float* states, int64_t index, int tu, int lane) {
  return reinterpret_cast<f32x4*>(states + index * (kN * kN) + state_offset(tu >> 2, tu & 3, lane));
}
__device__ __forceinline__ const f32x4* state_tile(const float* states, int64_t index, int tu, int lane) {
  return reinterpret_cast<const f32x4*>(states + index * (kN * kN) + state_offset(tu >> 2, tu & 3, lane));
}
// log w of the tokens t0 + lane % 32: 0 (decay 1) behind the sequence's end for a decay of each token, by a
// descriptor that ends with the sequence; a head's one decay is the same load with a stride of 0, so that there is
// no branch around the load. log_w_here() takes out the tokens behind the end in both.
__device__ __forceinline__ Span log_w_span(const float* log_w, bool per_token, const Seq& s, int64_t b, int32_t h,
                                           int64_t t0, int64_t len) {
  const int64_t left = len - t0 <= 0 ? 0 : len - t0 < kSub ? len - t0 : kSub;
  return Span{reinterpret_cast<const char*>(log_w + (per_token ? (b * s.T + t0) * s.H + h : h)),
              !left ? 0 : per_token ? ((uint32_t)(left - 1) * s.H + 1) * 4 : 4};
}
__device__ __forceinline__ float load_log_w(const float* log_w, bool per_token, const Seq& s, int64_t b, int32_t h,
                                            int64_t t0, int64_t len, int lane) {
  const Span x = log_w_span(log_w, per_token, s, b, h, t0, len);
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer(x.base, x.bytes),
                                                                        (lane & 31) * (per_token ? s.H * 4 : 0), 0, 0));
}
__device__ __forceinline__ float log_w_here(float loaded, int64_t t0, int64_t len, int lane) {
  return t0 + (lane & 31) < len ? loaded : 0.f;
}

}  // namespace linattn
}  // namespace rwkv7
