// What pieces of a sequence add to the state (or to its gradient), and the states at their starts: how the
// linear attention spreads one sequence over the device, and where its backward gets the states from.
//
// The state after a piece is (the piece's decay) (the state before) + (what the piece adds), so the pieces
// are independent until a short scan over their sums. A workgroup takes a piece of four blocks, each of its waves
// one block (128 tokens, or 64), 32 at a time from the last to the first: a token's factor is then the decay to
// the block's end, known when the token is met, and the sum stays in the matrix products' accumulators. The
// gradient G = dL/dS of the reverse pass has the same form with (r, dy) in place of (k, v), a token's factor being
// the decay from the block's start.
//
// Memory bounds it. bfloat16 rows come to LDS whole, by direct loads that each wave keeps 32 tokens ahead of itself in the
// place where its sum goes at the end, and leave it turned: B=8 T=4096 H=12 with both directions and the states of
// every block (300 MB) 64 us; 74 with loads to registers in operand order and turns by matrix products. They are
// loaded to stay in the caches, since the kernel that follows reads them again (with a hint against that it takes 4 us
// longer at B=1 T=8191 H=32). float32 rows, three pieces each, still go by registers.
#include "linattn_internal.hpp"
#include "linattn_ops.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

struct Side {
  const void* k;  // the key rows: k, or r backwards
  const void* v;  // the value rows: v, or dy backwards
  float* total;   // [units][stride]: what each piece adds
  float* decay;   // [units][stride]
  float* marks;   // may be null; [units][blocks]: the sum from the piece's start before each block but the piece's first
                  // (backwards: from its end behind each block but its last)
  float* mark_decay;  // [units][blocks]: the decay since then
  const float* start;  // the state before the first piece (backwards: the gradient behind the last), may be null
  float* end;          // may be null: that behind the last (before the first), `end_stride` states from one to the next
  int64_t end_stride;
  int32_t rev;
  int32_t every;
};
struct StateParams {
  Side side[2];
  const float* log_w;
  Seq seq;
  int32_t per_token;
  int32_t block;  // tokens
  int64_t first;  // number of the first head; the arrays of a side begin with it
  int64_t pieces, stride;
};

// Factors of a lane's tokens 16J + 4q + i of the 32, from their log w: what is left of them behind the 32 tokens (backwards:
// the decay from before them); `all`: the decay of the 32.
struct Left {
  f32x4 f[2];
  float all;
};
__device__ __forceinline__ Left make_left(float log_w, bool rev, double* sums, int lane) {
  const double c = log_sums(log_w, lane);
  if (lane < kSub) sums[lane] = c;
  __builtin_amdgcn_wave_barrier();
  const double end = readlane_f64(c, 31);
  Left o;
#pragma unroll
  for (int J = 0; J < 2; ++J)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = sums[16 * J + 4 * (lane >> 4) + i];
      o.f[J][i] = exp_diff(rev ? x : end, rev ? 0.0 : x);
    }
  __builtin_amdgcn_wave_barrier();
  o.all = exp_diff(end, 0.0);
  return o;
}

template <bool F32>
__global__ __launch_bounds__(256, 2) void linattn_state_kernel(StateParams p) {
  const Side x = p.side[blockIdx.y];
  const bool rev = x.rev;
  constexpr int NI = kIn<F32>;
  // What a wave's block adds, at the end; before that the wave's own quarter takes the rows of the tokens: two buffers of
  // 32 rows of k and v.
  __shared__ f32x4 sum[kWaves][16][64];
  constexpr int kBuffer = 2 * kSub * kRow;
  static_assert(2 * kBuffer <= sizeof(sum[0]), "a wave's rows");
  __shared__ float log_ws[kWaves][2][kSub];
  __shared__ double sums[kWaves][kSub];
  __shared__ float all[kWaves];
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
  const int64_t b = (p.first + unit) / p.seq.H;
  const int32_t h = (p.first + unit) % p.seq.H;
  const int64_t len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kN * kEsz<F32>;
  const int64_t nblk = (p.seq.T + p.block - 1) / p.block;
  const int64_t blk = piece * kPieceBlocks + wave;
  f32x4 S[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) S[t][u] = zero4();
  float decay = 1.f;
  const int64_t left = len - blk * p.block;
  const int subs = left <= 0 ? 0 : left >= p.block ? p.block / kSub : (int)((left + kSub - 1) / kSub);
  auto first = [&](int n) { return blk * p.block + (rev ? n : subs - 1 - n) * kSub; };
  if constexpr (F32) {
    const Turn E = make_turn(lane);
#pragma clang loop unroll(disable)
    for (int n = 0; n < subs; ++n) {
      const int64_t t0 = first(n);
      Raw<F32> rk, rv;
      load_raw<F32>(rv, token_buffer<kEsz<F32>>(x.v, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
      load_raw<F32>(rk, token_buffer<kEsz<F32>>(x.k, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
      const Left d = make_left(log_w_here(load_log_w(p.log_w, p.per_token, p.seq, b, h, t0, len, lane), t0, len, lane), rev,
                               sums[wave], lane);
      Op<3> Vs[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        Vs[u] = pack<3>(turned(natural<F32>(rv, 0, u >> 1), E, u) * (d.f[0] * decay),
                        turned(natural<F32>(rv, 1, u >> 1), E, u) * (d.f[1] * decay));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Op<NI> Kt = turned_op(natural<F32>(rk, 0, t >> 1), natural<F32>(rk, 1, t >> 1), E, t);
#pragma unroll
        for (int u = 0; u < 4; ++u) S[t][u] = mma(Kt, Vs[u], S[t][u]);
      }
      decay *= d.all;
    }
  } else {
    char* const rows = reinterpret_cast<char*>(sum[wave]);
    const uint32_t rows_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)rows;
    const uint32_t log_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)log_ws[wave][0];
    const uint32_t src0 = (lane >> 3) * row_bytes + 16 * ((lane & 7) ^ row_key(lane >> 3));
    const uint32_t src1 = ((lane >> 3) + 8) * row_bytes + 16 * ((lane & 7) ^ row_key(8 + (lane >> 3)));
    auto stage = [&](int n) {  // nine loads
      const int64_t t0 = first(n);
      const uint32_t to = rows_at + (n & 1) * kBuffer;
      const void* const from[2] = {x.v, x.k};
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const Span s = token_span<2>(from[m], p.seq, b, h, t0, len - t0, kSub);
        const u32x4 d = descriptor(s.base, s.bytes);
#pragma unroll
        for (int J = 0; J < 2; ++J) {
          to_lds16(d, src0 + J * 16 * row_bytes, to + (m * kSub + 16 * J) * kRow);
          to_lds16(d, src1 + J * 16 * row_bytes, to + (m * kSub + 16 * J + 8) * kRow);
        }
      }
      const Span s = log_w_span(p.log_w, p.per_token, p.seq, b, h, t0, len);
      if (lane < kSub)
        to_lds4(descriptor(s.base, s.bytes), lane * (p.per_token ? p.seq.H * 4 : 0), log_at + (n & 1) * kSub * 4);
    };
    const int turn0 = swizzled(4 * q + (li >> 2), li & 3);
    if (subs > 0) stage(0);
#pragma clang loop unroll(disable)
    for (int n = 0; n < subs; ++n) {
      // the next tokens' rows go to the other buffer, which has been read; then this one's are there
      if (n + 1 < subs) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        stage(n + 1);
        asm volatile("s_waitcnt vmcnt(9)" ::: "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      const char* const at = rows + (n & 1) * kBuffer;
      auto tile = [&](int m, int t) {
        const char* const a = at + m * kSub * kRow + (turn0 ^ 64 * (t >> 1)) + 8 * (t & 1);
        return Op<NI>{{join(turned4(a), turned4(a + 16 * kRow))}};
      };
      const Left d = make_left(log_w_here(log_ws[wave][n & 1][lane & 31], first(n), len, lane), rev, sums[wave], lane);
      const f32x4 f0 = d.f[0] * decay, f1 = d.f[1] * decay;
      Op<3> Vs[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const Op<NI> v = tile(0, u);
        f32x4 a0, a1;
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] = (float)v.p[0][i], a1[i] = (float)v.p[0][4 + i];
        Vs[u] = pack<3>(a0 * f0, a1 * f1);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Op<NI> Kt = tile(1, t);
#pragma unroll
        for (int u = 0; u < 4; ++u) S[t][u] = mma(Kt, Vs[u], S[t][u]);
      }
      decay *= d.all;
    }
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
  for (int m = 0; m < 4; ++m) *state_tile(x.total, unit * p.stride + piece, 4 * wave + m, lane) = s[m];
  if (threadIdx.x == 0) x.decay[unit * p.stride + piece] = since;
}

// total[piece / every] <- the state before every every-th piece (backwards: the gradient behind each piece, in place).
// A thread four elements of one head's state, which lie one after the other; 16 loads at a time.
__global__ __launch_bounds__(256) void linattn_join_kernel(StateParams p) {
  constexpr int kAhead = 16, kFours = kN * kN / 4;
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
      const int64_t n = n0 + i < p.pieces ? n0 + i : p.pieces - 1, at = unit * p.stride + (x.rev ? p.pieces - 1 - n : n);
      add[i] = total[at * kFours + e];
      a[i] = x.decay[at];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t n = n0 + i;
      if (n < p.pieces) {
        if (n % x.every == 0) total[(unit * p.stride + (x.rev ? p.pieces - 1 - n : n / x.every)) * kFours + e] = s;
        s = fma4(s, a[i], add[i]);
      }
    }
  }
  if (x.end) reinterpret_cast<f32x4*>(x.end)[unit * x.end_stride * kFours + e] = s;
}

}  // namespace

hipError_t launch_linattn_states(const LinattnCall& c, int64_t block, const LinattnPieces* forward, const LinattnPieces* backward) {
  StateParams p{};
  int sides = 0;
  if (forward)
    p.side[sides++] = Side{c.k, c.v, forward->states, forward->decay, forward->marks, forward->mark_decay, forward->start, forward->end,
                           forward->end_stride, 0, forward->every};
  if (backward)
    p.side[sides++] = Side{c.r, c.dy, backward->states, backward->decay, backward->marks, backward->mark_decay, backward->start,
                           backward->end, backward->end_stride, 1, backward->every};
  p.log_w = c.log_w;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  p.block = (int32_t)block;
  const LinattnPieces& any = forward ? *forward : *backward;
  p.first = any.first, p.pieces = any.pieces, p.stride = any.stride;
  const int64_t units = any.units;
  const void* fn = c.f32 ? reinterpret_cast<const void*>(&linattn_state_kernel<true>)
                         : reinterpret_cast<const void*>(&linattn_state_kernel<false>);
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(fn, dim3((uint32_t)(units * p.pieces), sides), dim3(256), args, 0, c.stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_join_kernel), dim3((uint32_t)(units * 4), sides), dim3(256),
                         args, 0, c.stream);
}

}  // namespace rwkv7
