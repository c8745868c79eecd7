// What pieces of a sequence add to the state (or to its gradient), and the states at their starts: how the
// linear attention spreads one sequence over the device, and where its backward gets the states from.
//
// The state after a piece is (the piece's decay) (the state before) + (what the piece adds), so the pieces
// are independent until a short scan over their sums. A workgroup takes a piece of four blocks, each of its waves
// one block (128 tokens, or 64), 32 at a time from the last to the first: a token's factor is then the decay to
// the block's end, known when the token is met, and the sum stays in the matrix products' accumulators. The
// gradient G = dL/dS of the reverse pass has the same form with (r, dy) in place of (k, v), a token's factor being
// the decay from the block's start.
#include "linattn_internal.hpp"
#include "linattn_ops.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

struct Side {
  const void* k;  // the key rows: k, or r backwards
  const void* v;  // the value rows: v, or dy backwards
  float* total;   // [units][pieces]: what each piece adds
  float* decay;   // [units][pieces]
  float* marks;   // may be null; [units][blocks]: the sum from the piece's start before each block but the piece's first
                  // (backwards: from its end behind each block but its last)
  float* mark_decay;  // [units][blocks]: the decay since then
  const float* start;  // the state before the first piece (backwards: the gradient behind the last), may be null
  float* end;          // may be null: that behind the last (before the first)
  int32_t rev;
  int32_t every;
};
struct StateParams {
  Side side[2];
  const float* log_w;
  Seq seq;
  int32_t per_token;
  int32_t block;  // tokens
  int64_t pieces;
};

template <bool F32>
__global__ __launch_bounds__(256, 2) void linattn_state_kernel(StateParams p) {
  const Side x = p.side[blockIdx.y];
  const bool rev = x.rev;
  constexpr int NI = kIn<F32>;
  __shared__ f32x4 sum[kWaves][16][64];
  __shared__ double sums[kWaves][kSub];
  __shared__ float all[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
  const int64_t b = unit / p.seq.H;
  const int32_t h = unit % p.seq.H;
  const int64_t len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kN * kEsz<F32>;
  const int64_t nblk = (p.seq.T + p.block - 1) / p.block;
  const int64_t blk = piece * kPieceBlocks + wave;
  const Turn E = make_turn(lane);
  f32x4 S[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) S[t][u] = zero4();
  float decay = 1.f;
  const int64_t left = len - blk * p.block;
  const int subs = left <= 0 ? 0 : left >= p.block ? p.block / kSub : (int)((left + kSub - 1) / kSub);
#pragma clang loop unroll(disable)
  for (int n = 0; n < subs; ++n) {
    const int64_t t0 = blk * p.block + (rev ? n : subs - 1 - n) * kSub;
    Raw<F32> rk, rv;
    load_raw<F32>(rv, token_buffer<kEsz<F32>>(x.v, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    load_raw<F32>(rk, token_buffer<kEsz<F32>>(x.k, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    const Decay d = make_decay(log_w_here(load_log_w(p.log_w, p.per_token, p.seq, b, h, t0, len, lane), t0, len, lane), sums[wave], lane);
    float f[2][4];
#pragma unroll
    for (int J = 0; J < 2; ++J)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[J][i] = (rev ? d.inrow[J][i] : d.row[J][i]) * decay;
    Op<3> Vs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f32x4 a0 = turned(natural<F32>(rv, 0, u >> 1), E, u), a1 = turned(natural<F32>(rv, 1, u >> 1), E, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) a0[i] *= f[0][i], a1[i] *= f[1][i];
      Vs[u] = pack<3>(a0, a1);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const Op<NI> Kt = turned_op(natural<F32>(rk, 0, t >> 1), natural<F32>(rk, 1, t >> 1), E, t);
#pragma unroll
      for (int u = 0; u < 4; ++u) S[t][u] = mma(Kt, Vs[u], S[t][u]);
    }
    decay *= d.all;
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) sum[wave][4 * t + u][lane] = S[t][u];
  if (lane == 0) all[wave] = decay;
  __syncthreads();
  // the four blocks one after the other: a quarter of the tiles each
  f32x4 s[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) s[m] = zero4();
  float since = 1.f;
#pragma unroll
  for (int n = 0; n < kWaves; ++n) {
    const int w = rev ? kWaves - 1 - n : n;
    const int64_t at = unit * nblk + piece * kPieceBlocks + w;
    if (x.marks && n > 0 && piece * kPieceBlocks + w < nblk) {
#pragma unroll
      for (int m = 0; m < 4; ++m) *state_tile(x.marks, at, 4 * wave + m, lane) = s[m];
      if (threadIdx.x == 0) x.mark_decay[at] = since;
    }
    const float a = all[w];
    since *= a;
#pragma unroll
    for (int m = 0; m < 4; ++m) s[m] = fma4(s[m], a, sum[w][4 * wave + m][lane]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) *state_tile(x.total, unit * p.pieces + piece, 4 * wave + m, lane) = s[m];
  if (threadIdx.x == 0) x.decay[unit * p.pieces + piece] = since;
}

// total[piece / every] <- the state before every every-th piece (backwards: the gradient behind each piece, in place).
// A thread four elements of one head's state, which lie one after the other; eight loads at a time.
__global__ __launch_bounds__(256) void linattn_join_kernel(StateParams p) {
  constexpr int kAhead = 8, kFours = kN * kN / 4;
  const Side x = p.side[blockIdx.y];
  const int64_t unit = blockIdx.x / 4;
  const int e = (blockIdx.x % 4) * 256 + threadIdx.x;
  const f32x4* start = reinterpret_cast<const f32x4*>(x.start);
  f32x4* total = reinterpret_cast<f32x4*>(x.total);
  f32x4 s = start ? start[unit * kFours + e] : zero4();
  for (int64_t n0 = 0; n0 < p.pieces; n0 += kAhead) {
    f32x4 add[kAhead];
    float a[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t n = n0 + i < p.pieces ? n0 + i : p.pieces - 1, at = unit * p.pieces + (x.rev ? p.pieces - 1 - n : n);
      add[i] = total[at * kFours + e];
      a[i] = x.decay[at];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t n = n0 + i;
      if (n < p.pieces) {
        if (n % x.every == 0) total[(unit * p.pieces + (x.rev ? p.pieces - 1 - n : n / x.every)) * kFours + e] = s;
        s = fma4(s, a[i], add[i]);
      }
    }
  }
  if (x.end) reinterpret_cast<f32x4*>(x.end)[unit * kFours + e] = s;
}

}  // namespace

hipError_t launch_linattn_states(const LinattnCall& c, int64_t block, const LinattnPieces* forward, const LinattnPieces* backward) {
  StateParams p{};
  int sides = 0;
  if (forward)
    p.side[sides++] = Side{c.k, c.v, forward->states, forward->decay, forward->marks, forward->mark_decay, c.s_in, nullptr, 0,
                           forward->every};
  if (backward)
    p.side[sides++] = Side{c.r, c.dy, backward->states, backward->decay, backward->marks, backward->mark_decay, c.ds_out,
                           backward->end, 1, backward->every};
  p.log_w = c.log_w;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  p.block = (int32_t)block;
  p.pieces = linattn_pieces(c.T, block);
  const int64_t units = c.B * c.H;
  const void* fn = c.f32 ? reinterpret_cast<const void*>(&linattn_state_kernel<true>)
                         : reinterpret_cast<const void*>(&linattn_state_kernel<false>);
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(fn, dim3((uint32_t)(units * p.pieces), sides), dim3(256), args, 0, c.stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_join_kernel), dim3((uint32_t)(units * 4), sides), dim3(256),
                         args, 0, c.stream);
}

}  // namespace rwkv7
