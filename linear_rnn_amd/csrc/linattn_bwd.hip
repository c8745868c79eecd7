// Gradients of the linear attention with a decay for each head (number formats and operand layouts in
// linattn_ops.hpp).
//
// With G_t = dL/dS_t from the tokens behind t; for a block, S_0 the state before it, G the gradient behind it, c the sum of
// log w from its start, D_ij = exp(c_i - c_j) for i >= j, P_ij = D_ij dy_i . v_j:
//   dr_i = sum_{j<=i} P_ij k_j + exp(c_i) S_0^T dy_i
//   dk_j = sum_{i>=j} P_ij r_i + exp(c_end - c_j) G^T v_j
//   dv_j = sum_{i>=j} D_ij (r_i . k_j) dy_i + exp(c_end - c_j) G k_j
// With S_0 and G of every block at hand (linattn_state.hip), the blocks are independent. A workgroup takes the blocks of
// a segment one after the other, each of its waves 16 tokens (a tile): dr of its tokens i from the tiles J before,
// dk and dv of its tokens j from the tiles I behind, and each from the block's border through S_0 and G. That is
// quadratic within a block, but neither S nor G has to be carried through it, and what all waves need of them, their
// bfloat16 pieces, is formed once.
//
// Decays. With c now the sum since a tile's start, the factor between token j of tile J and i of a later tile I is
// left_j (J's end to the tiles between) in_i: left_j = exp(c_end - c_j), in_i = exp(c_i), all at most 1. A wave's own
// factor is common to all of its tokens' sums, so it is applied once, to the accumulators, and only the tile on the
// diagonal needs a factor for each pair.
//
// dlog_w_t, t in tile w: the pairs of the tile that cross t, the sums over i >= t of r_i . dr_i from before the tile, over
// j < t of k_j . dk_j to behind it, and the paths over the whole tile: <S_0, G> with the block's decay, what S_0 gives
// to later tiles, what earlier tiles give to G, and the pairs of earlier with later tiles. All of them are sums of what
// crosses t, so nothing cancels.
//
// bfloat16: blocks of 128 tokens, eight waves; rows come to LDS by direct loads a block ahead, and with two buffers and
// the pieces of one state the LDS is full, so that dk and dv are done with G, then dr with S in the same place.
// float32: the rows are kept as three bfloat16 pieces each, so blocks of 64 tokens, four waves, one buffer.
//
// B=8 T=4096 H=12 bfloat16 145 us (520 MB, but the same without waiting for memory): vector instructions issue for 42% of
// it, matrix products for 20%, with two waves on a SIMD; a wave's chain from block to block instead (the states carried, no borders in memory) took 432. B=3 T=515
// H=16 float32 29 us, carried 156.
#include "linattn_internal.hpp"
#include "linattn_ops.hpp"
#include "operators_lock.hpp"
#include "wkv7_internal.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

constexpr int kPiece = kN * kRow;  // of one piece of a state
// Sizes and the LDS of one element type.
template <bool F32>
struct Cfg {
  static constexpr int kTiles = F32 ? 4 : 8;      // 16-token tiles of a block, one a wave
  static constexpr int kTokens = 16 * kTiles;
  static constexpr int kRows = kTokens * kRow;    // one piece of one tensor's rows of a block
  static constexpr int kIn = 0;                   // bfloat16: [parity][r, k, v, dy] kRows; float32: [r, k, v, dy][piece]
  static constexpr int kPieces = (F32 ? 12 : 8) * kRows;  // [piece][64 values] rows of 64 keys
  static constexpr int kSums = kPieces + 3 * kPiece;      // [kTokens] double: c
  static constexpr int kLeft = kSums + kTokens * 8;       // [kTokens] float
  static constexpr int kInto = kLeft + kTokens * 4;       // [kTokens] float
  static constexpr int kPerTile = kInto + kTokens * 4;    // [4][kTiles] float: exp(c_end), and the three sums below
  static constexpr int kPairs = kPerTile + 4 * kTiles * 4;     // [J][I] float: sums over the pairs of two tiles
  static constexpr int kLogW = kPairs + kTiles * kTiles * 4;   // bfloat16: [parity][kTokens] float
  static constexpr int kLds = kLogW + (F32 ? 0 : 2 * kTokens * 4);
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};

struct GradParams {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const void* dy;
  // the state before a block: of its piece (or the caller's), decayed since, and the piece's sum up to the block
  const float* states;
  const float* marks;
  const float* mark_decay;
  const float* grads;  // the gradient behind a block, alike
  const float* grad_marks;
  const float* grad_mark_decay;
  int64_t state_stride, grad_stride;  // states of a sequence
  void* dr;
  float* dlog_w;  // per token, or [units][nseg] sums
  void* dk;
  void* dv;
  Seq seq;
  int64_t first;  // number of the first head; states, gradients and marks begin with it
  int32_t per_token;
  int32_t nseg;
  int64_t seg_blocks;
};

// swizzled() for a state's pieces, whose rows follow each other as channel() numbers them.
__device__ __forceinline__ int in_pieces(int row, int piece) {
  return row * kRow + 16 * (piece ^ ((row >> 1 & 1) | (row >> 3 & 2) | (row >> 1 & 4)));
}

// Sums over a row of 16 lanes up to each lane, and from each lane on.
__device__ __forceinline__ float sums_to(float x) {
  x += dpp_f32<0x111>(x);
  x += dpp_f32<0x112>(x);
  x += dpp_f32<0x114>(x);
  x += dpp_f32<0x118>(x);
  return x;
}
__device__ __forceinline__ float sums_from(float x) {
  x += dpp_f32<0x101>(x);
  x += dpp_f32<0x102>(x);
  x += dpp_f32<0x104>(x);
  x += dpp_f32<0x108>(x);
  return x;
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b, float c) {
  return fmaf(a[3], b[3], fmaf(a[2], b[2], fmaf(a[1], b[1], fmaf(a[0], b[0], c))));
}
// Times the lane that many places up or down the row of 16, 1 behind its ends.
template <int CTRL>
__device__ __forceinline__ float times_dpp(float x) {
  return x * __uint_as_float(__builtin_amdgcn_update_dpp(0x3f800000, (int)__float_as_uint(x), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float readlane_f32(float x, int l) {
  return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(x), l));
}
__device__ __forceinline__ float wave_sum(float x) { return rows_sum(row16_sum(x)); }

// Element 4e + i of an operand, as float32.
template <int NP>
__device__ __forceinline__ float value(const Op<NP>& o, int e, int i) {
  float x = (float)o.p[NP - 1][4 * e + i];
#pragma unroll
  for (int n = NP - 2; n >= 0; --n) x += (float)o.p[n][4 * e + i];
  return x;
}

// Eight floats of a state: row `row`, columns from `col`; zeros where there is no state.
struct Eight {
  f32x4 x[2];
};
__device__ __forceinline__ Eight load_eight(const float* states, int64_t index, bool there, int row, int col) {
  const __amdgpu_buffer_rsrc_t b = buffer(states + index * (kN * kN), there ? kN * kN * 4 : 0);
  const uint32_t off = (row * kN + col) * 4;
  return Eight{{__builtin_bit_cast(f32x4, load16(b, off)), __builtin_bit_cast(f32x4, load16(b, off + 16))}};
}

template <int M>
struct Border {
  Eight piece[M], mark[M];  // the piece's state or gradient, and what the piece adds to it
  float decay;              // since the piece's border
};

template <bool F32>
__global__ __launch_bounds__(64 * Cfg<F32>::kTiles, F32 ? 1 : 2) void linattn_grad_kernel(GradParams p) {
  using C = Cfg<F32>;
  constexpr int kTiles = C::kTiles, kTokens = C::kTokens, kRows = C::kRows, kPieces = C::kPieces;
  constexpr int NI = kIn<F32>, NO = F32 ? 3 : 2;
  extern __shared__ char lds[];
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  // The wave's tile. Tile w has w tiles before it (one product of pairs each) and 7 - w behind it (two), and the waves
  // i and i + 4 share a SIMD: tiles w and 7 - w together have the same work on every one. (float32: tile w is wave w's.)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave < 4 ? wave : 11 - wave;
  const int64_t unit = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
  const int64_t b = (p.first + unit) / p.seq.H;
  const int32_t h = (p.first + unit) % p.seq.H;
  const int64_t T = p.seq.T, len = seq_len(p.seq, b);
  constexpr int kRowBytes = kN * kEsz<F32>;  // a token's, in memory
  const uint32_t row_bytes = p.seq.H * kRowBytes;
  const int64_t nblk = (T + kTokens - 1) / kTokens;
  const int64_t blk0 = seg * p.seg_blocks;
  const int64_t blk1 = blk0 + p.seg_blocks < nblk ? blk0 + p.seg_blocks : nblk;
  const int64_t live = (len + kTokens - 1) / kTokens < blk1 ? (len + kTokens - 1) / kTokens : blk1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  auto f32s = [&](int at) { return reinterpret_cast<float*>(lds + at); };

  // ---- loads
  const uint32_t src0 = (lane >> 3) * row_bytes + 16 * ((lane & 7) ^ row_key(lane >> 3));
  const uint32_t src1 = ((lane >> 3) + 8) * row_bytes + 16 * ((lane & 7) ^ row_key(8 + (lane >> 3)));
  // A block: the row of its first token in every tensor (and element of log w); of its tokens, how many count and how many the
  // tensors hold; where the wave's 16 rows start, and the bytes to the end of the last of them that counts.
  struct Block {
    int64_t row;
    int live, rows, parity;
    int64_t start;
    uint32_t bytes;
  };
  const uint32_t own = 16 * w * p.seq.H;  // the wave's first row, from the block's
  auto rows_bytes = [&](int n) {
    n -= 16 * w;
    n = n < 16 ? n : 16;
    return n > 0 ? (uint32_t)(n - 1) * row_bytes + kRowBytes : 0;
  };
  auto tokens = [&](int64_t n) { return n < 0 ? 0 : n < kTokens ? (int)n : kTokens; };
  auto block = [&](int64_t blk) {
    const int64_t t = blk * kTokens;
    Block x{(b * T + t) * p.seq.H + h, tokens(len - t), tokens(T - t), (int)(blk & 1), 0, 0};
    x.start = (x.row + own) * (int64_t)kRowBytes;
    x.bytes = rows_bytes(x.live);
    return x;
  };
  auto stage = [&](const void* x, int number, const Block& at) {
    const u32x4 d = descriptor(static_cast<const char*>(x) + at.start, at.bytes);
    const uint32_t to = lds0 + C::kIn + (at.parity * 4 + number) * kRows + w * 16 * kRow;
    to_lds16_last(d, src0, to);
    to_lds16_last(d, src1, to + 8 * kRow);
  };
  // log w of `most` tokens from the block's token `first` on, as log_w_span() has it
  auto log_w_at = [&](const Block& at, int first, int most) {
    int n = at.live - first;
    n = n < most ? n : most;
    return Span{reinterpret_cast<const char*>(p.log_w + (p.per_token ? at.row + (uint32_t)first * p.seq.H : h)),
                n <= 0 ? 0 : p.per_token ? ((uint32_t)(n - 1) * p.seq.H + 1) * 4 : 4};
  };
  auto stage_w = [&](const Block& at) {
    if (wave < 4 && lane < kSub) {
      const Span s = log_w_at(at, wave * kSub, kSub);
      to_lds4(descriptor(s.base, s.bytes), lane * (p.per_token ? p.seq.H * 4 : 0),
              lds0 + C::kLogW + at.parity * kTokens * 4 + wave * kSub * 4);
    }
  };
  // float32: the wave's rows from memory to LDS by way of registers, in pieces
  struct Rows {
    u32x4 x[4][2][F32 ? 2 : 1];
  };
  auto load_rows = [&](const Block& at) {
    Rows o;
    const void* src[4] = {p.r, p.k, p.v, p.dy};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const __amdgpu_buffer_rsrc_t from = buffer(static_cast<const char*>(src[x]) + at.start, at.bytes);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int m = 0; m < (F32 ? 2 : 1); ++m)
          o.x[x][hh][m] = load16(from, li * row_bytes + 32 * q + 128 * hh + 16 * m);
    }
    return o;
  };
  // Eighths of a state, of 8 value rows each: the wave's
  constexpr int kEighths = 8 / kTiles;
  const int own_col = 8 * (lane & 7);
  auto own_row = [&](int m) { return 8 * (wave + m * kTiles) + (lane >> 3); };
  auto load_border = [&](const float* states, const float* marks, const float* decays, int64_t stride, int unmarked,
                         int64_t blk) {
    Border<kEighths> x;
    const bool there = blk < live && states, marked = there && marks && blk % kPieceBlocks != unmarked;
    const int64_t at = unit * nblk + (marked ? blk : 0);
#pragma unroll
    for (int m = 0; m < kEighths; ++m) {
      x.piece[m] = load_eight(states, there ? unit * stride + (stride > 1 ? blk / kPieceBlocks : 0) : 0, there, own_row(m), own_col);
      x.mark[m] = load_eight(marks, marked ? at : 0, marked, own_row(m), own_col);
    }
    x.decay = marked ? decays[at] : 1.f;
    return x;
  };
  auto load_grad = [&](int64_t blk) {
    return load_border(p.grads, p.grad_marks, p.grad_mark_decay, p.grad_stride, kPieceBlocks - 1, blk);
  };
  auto state_of = [&](const Border<kEighths>& x, float (&o)[kEighths][8]) {
#pragma unroll
    for (int m = 0; m < kEighths; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[m][i] = fmaf(x.piece[m].x[i >> 2][i & 3], x.decay, x.mark[m].x[i >> 2][i & 3]);
  };
  auto put_pieces = [&](const float (&x)[kEighths][8]) {
#pragma unroll
    for (int m = 0; m < kEighths; ++m) {
      Op<3> o;
#pragma unroll
      for (int i = 0; i < 8; i += 2) put2(o, i, x[m][i], x[m][i + 1]);
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *reinterpret_cast<bf16x8*>(lds + kPieces + n * kPiece + in_pieces(own_row(m), lane & 7)) = o.p[n];
    }
  };
  // ---- operands. Piece 4m + x of a row is 64 m bytes, by exclusive or, from piece x, in both numberings, so a lane's
  // place in a tile is one of two and everything else in an address a constant or the tile's.
  const int nat0 = swizzled(li, q), turn0 = swizzled(4 * q + (li >> 2), li & 3);
  const int pnat0 = in_pieces(8 * (li >> 2) + (li & 3), q), pturn0 = in_pieces(8 * q + (li >> 2), li & 3);
  // rows row0 + li as they are (row0 a multiple of 16)
  auto nat = [&](int from, int row0, int hh) {
    Op<NI> o;
#pragma unroll
    for (int n = 0; n < NI; ++n)
      o.p[n] = *reinterpret_cast<const bf16x8*>(lds + (from + row0 * kRow) + (nat0 ^ 64 * hh) + n * kRows);
    return o;
  };
  auto turn4 = [&](int at) { return turned4(lds + at); };
  // an operand over the tokens of tiles I0, I1 of a tensor, rows its channels of tile t
  auto turned_tokens = [&](int from, int I0, int I1, int t) {
    const int in_tile = (turn0 ^ 64 * (t >> 1)) + 8 * (t & 1);
    Op<NI> o;
#pragma unroll
    for (int n = 0; n < NI; ++n)
      o.p[n] = join(turn4(from + I0 * 16 * kRow + in_tile + n * kRows), turn4(from + I1 * 16 * kRow + in_tile + n * kRows));
    return o;
  };
  // the pieces' operand over values 32 hv .., rows the keys of tile t
  auto turned_values = [&](int t, int hv) {
    Op<3> o;
    const int at = kPieces + (pturn0 ^ 64 * (t >> 1)) + 8 * (t & 1) + 32 * hv * kRow;
#pragma unroll
    for (int n = 0; n < 3; ++n) o.p[n] = join(turn4(at + n * kPiece), turn4(at + n * kPiece + 4 * kRow));
    return o;
  };

  float head_sum = 0.f;
  Border<kEighths> grad;
  Block now = block(blk0);
  if (blk0 < live) {
    if constexpr (!F32) stage(p.r, 0, now), stage(p.k, 1, now), stage(p.v, 2, now), stage(p.dy, 3, now), stage_w(now);
    grad = load_grad(blk0);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  for (int64_t blk = blk0; blk < live; ++blk) {
    const Block next = block(blk + 1);
    const int rows_r = C::kIn + (F32 ? 0 : now.parity * 4 * kRows), rows_k = rows_r + NI * kRows,
              rows_v = rows_k + NI * kRows, rows_d = rows_v + NI * kRows;
    float lw;
    if constexpr (F32) {
      const Rows x = load_rows(now);
      const Span s = log_w_at(now, 16 * w, 16);
      lw = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer(s.base, s.bytes),
                                                                          li * (p.per_token ? p.seq.H * 4 : 0), 0, 0));
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const Op<NI> o = pieces<F32>(x.x[n][hh]);
#pragma unroll
          for (int m = 0; m < NI; ++m)
            *reinterpret_cast<bf16x8*>(lds + C::kIn + (n * NI + m) * kRows + 16 * w * kRow + (nat0 ^ 64 * hh)) = o.p[m];
        }
    } else {
      lw = f32s(C::kLogW + now.parity * kTokens * 4)[16 * w + li];
    }
    float g8[kEighths][8];
    state_of(grad, g8);
    // the next block's rows, a tensor at a time through the block: all at once they fill the queue of loads and hold the
    // waves up where they are asked for
    if constexpr (!F32) stage_w(next), stage(p.r, 0, next);
    put_pieces(g8);
    const Border<kEighths> state = load_border(p.states, p.marks, p.mark_decay, p.state_stride, 0, blk);
    // decays of the tile's tokens, in all four rows of lanes
    float left, into;
    double c;
    {
      c = 16 * w + li < now.live ? (double)(lw < -1e4f ? -1e4f : lw) * 1.4426950408889634 : 0.0;
      c += dpp_f64<0x111>(c);
      c += dpp_f64<0x112>(c);
      c += dpp_f64<0x114>(c);
      c += dpp_f64<0x118>(c);
      const double end = readlane_f64(c, 15);
      left = exp_diff(end, c), into = exp_diff(c, 0.0);
      if (lane < 16) {
        reinterpret_cast<double*>(lds + C::kSums)[16 * w + li] = c;
        f32s(C::kLeft)[16 * w + li] = left;
        f32s(C::kInto)[16 * w + li] = into;
      }
      if (lane == 0) f32s(C::kPerTile)[w] = exp_diff(end, 0.0);
    }
    Op<NI> R[2], K[2], V[2], D[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      R[hh] = nat(rows_r, 16 * w, hh), K[hh] = nat(rows_k, 16 * w, hh), V[hh] = nat(rows_v, 16 * w, hh),
      D[hh] = nat(rows_d, 16 * w, hh);
    lds_barrier();

    // decays of the tiles before and behind, of the block: products over the lanes that hold the tiles'
    float before, behind, all;
    {
      const float e = li < kTiles ? f32s(C::kPerTile)[li] : 1.f;
      float to = times_dpp<0x111>(e), from = times_dpp<0x101>(e);
      to = times_dpp<0x112>(to), from = times_dpp<0x102>(from);
      if constexpr (kTiles == 8) to = times_dpp<0x114>(to), from = times_dpp<0x104>(from);
      before = w > 0 ? readlane_f32(to, w - 1) : 1.f;
      behind = readlane_f32(from, w + 1);
      all = readlane_f32(to, kTiles - 1);
    }
    int place = lane;  // in here, so that the masks made of it are not kept in scalar registers, of which there are too few
    asm volatile("" : "+v"(place));
    f32x4 dj, di;  // factors of the tile on the diagonal: rows j, rows i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double r = reinterpret_cast<const double*>(lds + C::kSums)[16 * w + 4 * q + i];
      dj[i] = exp_diff(c, r), di[i] = exp_diff(r, c);
    }
    if constexpr (!F32) stage(p.k, 1, next);
    // The pairs with the tiles behind (for dk, dv) and before (for dr). Their part of k_j . dk_j and r_i . dr_i is summed
    // here, in float32: the products with the pairs' pieces are only as good as dk and dr need them.
    float kdk = 0.f, rdr = 0.f;
    f32x4 ak[4], av[4], ar[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) ak[t] = av[t] = ar[t] = zero4();
    float between = 1.f;
#pragma clang loop unroll(disable)
    for (int I = w + 1; I < kTiles; I += 2) {
      const int I1 = I + 1 < kTiles ? I + 1 : I;
      f32x4 pq[2], pa[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int X = e ? I1 : I;
        f32x4 x = zero4(), a = zero4();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) x = mma(nat(rows_d, 16 * X, hh), V[hh], x), a = mma(nat(rows_r, 16 * X, hh), K[hh], a);
        const bool on = e == 0 || I1 > I;
        const f32x4 f = *reinterpret_cast<const f32x4*>(f32s(C::kInto) + 16 * X + 4 * q) * (on ? between : 0.f);
        pq[e] = x * f, pa[e] = a * f;
        if (on) {
          const float mine = dot4(a, pq[e], 0.f) * left;
          kdk += mine;
          const float s = wave_sum(mine);
          if (lane == 0) f32s(C::kPairs)[w * kTiles + X] = s;
          between *= f32s(C::kPerTile)[X];
        }
      }
      const Op<NO> Pq = pack<NO>(pq[0], pq[1]), Pa = pack<NO>(pa[0], pa[1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ak[t] = mma(turned_tokens(rows_r, I, I1, t), Pq, ak[t]);
        av[t] = mma(turned_tokens(rows_d, I, I1, t), Pa, av[t]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!F32) stage(p.v, 2, next);
    between = 1.f;
#pragma clang loop unroll(disable)
    for (int J = w - 1; J >= 0; J -= 2) {
      const int J1 = J > 0 ? J - 1 : J;
      f32x4 pp[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int X = e ? J1 : J;
        const bool on = e == 0 || J1 < J;
        f32x4 x = mma(nat(rows_v, 16 * X, 0), D[0], zero4());
        x = mma(nat(rows_v, 16 * X, 1), D[1], x);
        const f32x4 a = mma(nat(rows_k, 16 * X, 1), R[1], mma(nat(rows_k, 16 * X, 0), R[0], zero4()));
        pp[e] = x * (*reinterpret_cast<const f32x4*>(f32s(C::kLeft) + 16 * X + 4 * q) * (on ? between : 0.f));
        if (on) {
          rdr = dot4(a, pp[e], rdr);
          between *= f32s(C::kPerTile)[X];
        }
      }
      const Op<NO> P = pack<NO>(pp[0], pp[1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) ar[t] = mma(turned_tokens(rows_k, J, J1, t), P, ar[t]);
    }
    __builtin_amdgcn_sched_barrier(0);  // phases whose registers would not fit together
    if constexpr (!F32) stage(p.dy, 3, next);
    rdr *= into;
    float cross = 0.f;
    {  // dk and dv: the gradient behind the block, the factor of the tokens, the tile's own pairs
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int rows = (32 * (u >> 1) + 4 * (u & 1)) * kRow;  // value channel(u, li)
        f32x4 o = zero4();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          Op<NO> G;
#pragma unroll
          for (int n = 0; n < NO; ++n)
            G.p[n] = *reinterpret_cast<const bf16x8*>(lds + kPieces + (pnat0 ^ 64 * hh) + rows + n * kPiece);
          o = mma(G, K[hh], o);
        }
        av[u] = fma4(o, behind, av[u]) * left;
      }
      __builtin_amdgcn_sched_barrier(0);
      float kg = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4 o = mma(turned_values(t, 0), V[0], zero4());
        o = mma(turned_values(t, 1), V[1], o) * (behind * left);
        ak[t] = fma4(ak[t], left, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float k = value(K[t >> 1], t & 1, i);
          kg = fmaf(o[i], k, kg);
        }
      }
      kdk = rows_sum(kdk + kg);
      kg = wave_sum(kg);
      if (lane == 0) f32s(C::kPerTile)[2 * kTiles + w] = kg;
      __builtin_amdgcn_sched_barrier(0);
      f32x4 x = mma(D[1], V[1], mma(D[0], V[0], zero4())), a = mma(R[1], K[1], mma(R[0], K[0], zero4()));
      x = masked_i(x, di, place);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float to = sums_to(dpp_f32<0x111>(a[i] * x[i]));  // columns j before t of the row i
        cross += 4 * (place >> 4) + i >= (place & 15) ? to : 0.f;
      }
      cross = rows_sum(cross);
      const Op<NO> Pq = pack<NO>(x, zero4()), Pa = pack<NO>(masked_i(a, di, place), zero4());
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ak[t] = mma(turned_tokens(rows_r, w, w, t), Pq, ak[t]);
        av[t] = mma(turned_tokens(rows_d, w, w, t), Pa, av[t]);
      }
      const __amdgpu_buffer_rsrc_t kb = buffer(static_cast<char*>(p.dk) + now.start, rows_bytes(now.rows));
      const __amdgpu_buffer_rsrc_t vb = buffer(static_cast<char*>(p.dv) + now.start, rows_bytes(now.rows));
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        store_pair<F32>(kb, li * row_bytes + (32 * hh + 8 * q) * kEsz<F32>, ak[2 * hh], ak[2 * hh + 1]);
        store_pair<F32>(vb, li * row_bytes + (32 * hh + 8 * q) * kEsz<F32>, av[2 * hh], av[2 * hh + 1]);
      }
    }
    grad = load_grad(blk + 1);
    lds_barrier();
    {
      float s8[kEighths][8], x = 0.f;
      state_of(state, s8);
      put_pieces(s8);
#pragma unroll
      for (int m = 0; m < kEighths; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) x = fmaf(s8[m][i], g8[m][i], x);
      x = wave_sum(x);
      if (lane == 0) f32s(C::kPerTile)[kTiles + wave] = x;
    }
    lds_barrier();
    {  // dr, alike with the state before the block
      float rs = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4 o = mma(turned_values(t, 0), D[0], zero4());
        o = mma(turned_values(t, 1), D[1], o) * (before * into);
        ar[t] = fma4(ar[t], into, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float r = value(R[t >> 1], t & 1, i);
          rs = fmaf(o[i], r, rs);
        }
      }
      rdr = rows_sum(rdr + rs);
      rs = wave_sum(rs);
      if (lane == 0) f32s(C::kPerTile)[3 * kTiles + w] = rs;
      const f32x4 x = masked_j(mma(V[1], D[1], mma(V[0], D[0], zero4())), dj, place);
      const Op<NO> P = pack<NO>(x, zero4());
#pragma unroll
      for (int t = 0; t < 4; ++t) ar[t] = mma(turned_tokens(rows_k, w, w, t), P, ar[t]);
      const __amdgpu_buffer_rsrc_t rb = buffer(static_cast<char*>(p.dr) + now.start, rows_bytes(now.rows));
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        store_pair<F32>(rb, li * row_bytes + (32 * hh + 8 * q) * kEsz<F32>, ar[2 * hh], ar[2 * hh + 1]);
    }
    lds_barrier();
    {  // dlog_w: lane kTiles J + I the pairs of two tiles, lanes 0 .. kTiles - 1 the borders
      const int J = place / kTiles, I = place % kTiles;
      float x = J < w && I > w ? f32s(C::kPairs)[place] : 0.f;
      if (place < kTiles)
        x += all * f32s(C::kPerTile)[kTiles + place] + (place < w ? f32s(C::kPerTile)[2 * kTiles + place] : 0.f) +
             (place > w ? f32s(C::kPerTile)[3 * kTiles + place] : 0.f);
      float dlw = cross + sums_from(rdr) + sums_to(dpp_f32<0x111>(kdk)) + wave_sum(x);
      if (16 * w + li >= now.live) dlw = 0.f;
      if (p.per_token) {
        if (lane < 16 && 16 * w + li < now.rows) p.dlog_w[now.row + own + (uint32_t)li * p.seq.H] = dlw;
      } else {
        head_sum += dlw;
      }
    }
    // the next block's rows are there: behind them are at least six stores
    asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    now = next;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to this workgroup's LDS when it ends
  for (int64_t blk = live > blk0 ? live : blk0; blk < blk1; ++blk) {  // behind the sequence's end: no gradients
    const Block at = block(blk);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t off = li * row_bytes + (32 * hh + 8 * q) * kEsz<F32>;
      void* const out[3] = {p.dr, p.dk, p.dv};
#pragma unroll
      for (int x = 0; x < 3; ++x)
        store_pair<F32>(buffer(static_cast<char*>(out[x]) + at.start, rows_bytes(at.rows)), off, zero4(), zero4());
    }
    if (p.per_token && lane < 16 && 16 * w + lane < at.rows) p.dlog_w[at.row + own + (uint32_t)lane * p.seq.H] = 0.f;
  }
  if (!p.per_token) {
    const float s = row16_sum(head_sum);
    if (lane == 0) f32s(C::kPerTile)[w] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float x = 0.f;
      for (int i = 0; i < kTiles; ++i) x += f32s(C::kPerTile)[i];
      p.dlog_w[unit * p.nseg + seg] = x;
    }
  }
}

// dlog_w[h] from the sums of its sequences and segments, in order.
__global__ __launch_bounds__(64) void linattn_head_sum_kernel(const float* parts, float* dlog_w, int64_t B, int32_t H,
                                                              int32_t nseg) {
  const int32_t h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < B * nseg; i += 64) s += parts[(i / nseg * H + h) * nseg + i % nseg];
#pragma unroll
  for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
  if (threadIdx.x == 0) dlog_w[h] = (float)s;
}

__global__ __launch_bounds__(256) void linattn_zero_kernel(float* x, int64_t n) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i < n) x[i] = 0.f;
}

// Workspace of a call for what its heads have between their blocks, or one head's where that is more: the heads are taken
// in slabs that fit. Smaller slabs cost time, since less is under way at once: B=4 T=16384 H=64 bfloat16 (1.3 GB) 2.11 ms in one
// slab, 2.14 in two of this size, 2.37 at 512 MiB, 2.47 at 256; B=8 T=4096 H=32 (420 MB) 0.54, 0.54, 0.54, 0.56.
constexpr size_t kSlabBytes = size_t(1) << 30;

template <bool F32>
hipError_t launch(const LinattnCall& c) {
  constexpr int64_t kTokens = Cfg<F32>::kTokens, kStateFloats = kLinattnStateBytes / 4;
  const int64_t units = c.B * c.H, nblk = (c.T + kTokens - 1) / kTokens,
                pieces = (nblk + kPieceBlocks - 1) / kPieceBlocks, cus = linattn_cus();
  const bool border = nblk > 1;            // blocks whose state is not the caller's
  const bool states = border || c.ds_in;  // one block: its state is the caller's, and so is its gradient; a copy where
                                          // dstate_in is written over it
  // bytes of a head: its pieces' states and gradients, the marks, and their decays
  const size_t head = (size_t)(border ? pieces + 2 * nblk : 0) * kLinattnStateBytes +
                      (size_t)(states ? pieces : 0) * kLinattnStateBytes + (size_t)(pieces + nblk) * 8;
  const int64_t fit = kSlabBytes / head > 0 ? (int64_t)(kSlabBytes / head) : 1;
  const int64_t slabs = (units + fit - 1) / fit, slab = (units + slabs - 1) / slabs;

  // Segments: as many workgroups as fill the compute units in whole rounds best, each with its first loads to wait for.
  // B=8 T=4096 H=12 bfloat16 210 us in 8 segments of 4 blocks, 371 in one, 247 in 32; B=4 T=4096 H=64 540 in one, 557 in 8.
  int64_t nseg = 1;
  double best = 0;
  for (int64_t n = 1; n <= nblk && (n == 1 || slab * n <= 4 * cus); ++n) {
    const int64_t length = (nblk + n - 1) / n, rounds = (slab * n + cus - 1) / cus;
    const double us = rounds * (length * (F32 ? 10.0 : 5.0) + 3.0);
    if (n == 1 || us < best) best = us, nseg = n;
  }
  const int64_t seg_blocks = (nblk + nseg - 1) / nseg;
  nseg = (nblk + seg_blocks - 1) / seg_blocks;

  size_t need = 0;
  auto room = [&](size_t bytes) {
    const size_t at = need;
    need += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t o_states = room(border ? slab * pieces * kLinattnStateBytes : 0), o_decay = room(slab * pieces * 4);
  const size_t o_marks = room(border ? slab * nblk * kLinattnStateBytes : 0), o_mdecay = room(slab * nblk * 4);
  const size_t o_grads = room(states ? slab * pieces * kLinattnStateBytes : 0), o_gdecay = room(slab * pieces * 4);
  const size_t o_gmarks = room(border ? slab * nblk * kLinattnStateBytes : 0), o_gmdecay = room(slab * nblk * 4);
  const size_t o_parts = room(c.per_token ? 0 : units * nseg * 4);
  std::lock_guard<std::mutex> lock(operators_mutex());
  void* ws = nullptr;
  hipError_t e = device_workspace(c.stream, need, &ws, kWorkspaceOperators);
  if (e != hipSuccess) return e;
  char* base = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const void* fn = reinterpret_cast<const void*>(&linattn_grad_kernel<F32>);
  static std::atomic<uint64_t> granted{0};
  e = allow_lds(granted, fn, Cfg<F32>::kLds);
  if (e != hipSuccess) return e;

  LinattnPieces f{}, g{};
  f.pieces = g.pieces = f.stride = g.stride = pieces;
  f.every = g.every = 1;
  f.states = at(o_states), f.decay = at(o_decay), f.marks = border ? at(o_marks) : nullptr, f.mark_decay = at(o_mdecay);
  g.states = at(o_grads), g.decay = at(o_gdecay), g.marks = border ? at(o_gmarks) : nullptr, g.mark_decay = at(o_gmdecay);
  g.end_stride = 1;
  GradParams p{};
  p.r = c.r, p.log_w = c.log_w, p.k = c.k, p.v = c.v, p.dy = c.dy;
  // the state before a block: of its piece (or the caller's), decayed since, and the piece's sum up to the block
  p.marks = f.marks, p.mark_decay = f.mark_decay;
  p.grad_marks = g.marks, p.grad_mark_decay = g.mark_decay;
  p.state_stride = p.grad_stride = border ? pieces : 1;
  p.dr = c.dr, p.dk = c.dk, p.dv = c.dv;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  p.nseg = (int32_t)nseg, p.seg_blocks = seg_blocks;
  for (int64_t first = 0; first < units; first += slab) {
    const int64_t some = units - first < slab ? units - first : slab;
    auto of = [&](auto* x) { return x ? x + first * kStateFloats : x; };  // the caller's states from the first head on
    f.first = g.first = p.first = first;
    f.units = g.units = some;
    f.start = of(c.s_in), g.start = of(c.ds_out), g.end = of(c.ds_in);
    p.states = border ? f.states : f.start;
    p.grads = states ? g.states : g.start;
    p.dlog_w = c.per_token ? c.dlog_w : at(o_parts) + first * nseg;
    if (states) {
      e = launch_linattn_states(c, kTokens, border ? &f : nullptr, &g);
      if (e != hipSuccess) return e;
    }
    void* args[] = {&p};
    e = hipLaunchKernel(fn, dim3((uint32_t)(some * nseg)), dim3(64 * Cfg<F32>::kTiles), args, Cfg<F32>::kLds, c.stream);
    if (e != hipSuccess) return e;
  }
  if (c.per_token) return hipSuccess;
  const float* parts = at(o_parts);
  float* dlog_w = c.dlog_w;
  int64_t B = c.B;
  int32_t H = (int32_t)c.H, n = (int32_t)nseg;
  void* hargs[] = {&parts, &dlog_w, &B, &H, &n};
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_head_sum_kernel), dim3((uint32_t)H), dim3(64), hargs, 0, c.stream);
}

}  // namespace

hipError_t launch_linattn_zero(float* dlog_w, int64_t H, hipStream_t stream) {
  void* args[] = {&dlog_w, &H};
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_zero_kernel), dim3((uint32_t)((H + 255) / 256)), dim3(256),
                         args, 0, stream);
}

hipError_t launch_linattn_backward(const LinattnCall& c) { return c.f32 ? launch<true>(c) : launch<false>(c); }

}  // namespace rwkv7
