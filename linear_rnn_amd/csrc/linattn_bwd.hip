// Gradients of the linear attention with a decay for each head. The chunk algebra, number formats and
// layouts are those of linattn_ops.hpp.
//
// With G_t = dL/dS_t from the tokens behind t, for the 32 tokens of a wave (S_0 the state before them, G_32 the
// gradient behind them, A_ij = r_i . k_j, P_ij = D_ij dy_i . v_j):
//   dr_i = sum_{j<=i} P_ij k_j + exp(c_i) S_0^T dy_i
//   dk_j = sum_{i>=j} P_ij r_i + exp(c_31 - c_j) G_32^T v_j
//   dv_j = sum_{i>=j} D_ij A_ij dy_i + exp(c_31 - c_j) G_32 k_j
//   G_0  = exp(c_31) G_32 + sum_i exp(c_i) dy_i r_i^T
// A token's log decay scales every path that crosses it, from tokens j before it to tokens i from it on:
//   dlog_w_t = sum_{j<t<=i} A_ij P_ij + sum_{i>=t} r_i . exp(c_i) S_0^T dy_i
//            + sum_{j<t} k_j . exp(c_31 - c_j) G_32^T v_j + exp(c_31) <S_0, G_32>
// each of them a sum of prefix and suffix sums, so that nothing cancels but what cancels in the value itself.
//
// Kernels: the states before the blocks of 128 tokens (linattn_state.hip: the sums of pieces, a scan), then a
// workgroup for each head and segment walks its blocks from the last to the first with G carried in LDS; its
// four waves take 32 tokens each and exchange what they add to S (forwards) and to G (backwards).
#include "linattn_internal.hpp"
#include "linattn_ops.hpp"
#include "wkv7_internal.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

struct GradParams {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const void* dy;
  const float* s_in;       // the caller's state (pieces == 1), may be null
  const float* ds_out;     // the caller's (nseg == 1), may be null
  const float* states;     // [units][pieces] states before the pieces (pieces > 1)
  const float* marks;      // [units][blocks]
  const float* mark_decay; // [units][blocks]
  const float* grads;      // [units][pieces] gradients behind the pieces (nseg > 1)
  void* dr;
  float* dlog_w;  // per token, or [units][nseg] sums
  void* dk;
  void* dv;
  float* ds_in;  // may be null
  Seq seq;
  int32_t per_token;
  int32_t nseg;
  int64_t pieces, seg_pieces;  // of a sequence, of a segment
};

// Sums over 32 lanes' values from each on (lane l and l + 32 alike), and of those before each.
__device__ __forceinline__ float sum_from(float x, int lane) {
  x += dpp_f32<0x101>(x);  // row_shl:1, 2, 4, 8 (zeros come in)
  x += dpp_f32<0x102>(x);
  x += dpp_f32<0x104>(x);
  x += dpp_f32<0x108>(x);
  const float second = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16));
  return (lane & 16) ? x : x + second;
}
__device__ __forceinline__ float row_sums_to(float x) {  // of a row's 16 lanes up to each
  x += dpp_f32<0x111>(x);  // row_shr
  x += dpp_f32<0x112>(x);
  x += dpp_f32<0x114>(x);
  x += dpp_f32<0x118>(x);
  return x;
}
__device__ __forceinline__ float sum_before(float x, int lane) {
  const float first = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, row_sums_to(x)), 15));
  const float s = row_sums_to(dpp_f32<0x111>(x));
  return (lane & 16) ? s + first : s;
}
template <bool F32>
__global__ __launch_bounds__(256, 1) void linattn_grad_kernel(GradParams p) {
  constexpr int NI = kIn<F32>, NO = F32 ? 3 : 2;
  extern __shared__ f32x4 shared[];
  f32x4(*addS)[16][64] = reinterpret_cast<f32x4(*)[16][64]>(shared);              // of waves 0 .. 2
  f32x4(*addG)[16][64] = reinterpret_cast<f32x4(*)[16][64]>(shared + 3 * 1024);   // of waves 0 .. 3
  f32x4(*carry)[64] = reinterpret_cast<f32x4(*)[64]>(shared + 7 * 1024);          // G behind the block
  double(*sums)[kSub] = reinterpret_cast<double(*)[kSub]>(shared + 8 * 1024);     // [kWaves]
  float* all = reinterpret_cast<float*>(shared + 8 * 1024 + kWaves * kSub / 2);
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int64_t unit = id / p.nseg;
  const int32_t seg = id % p.nseg;
  const int64_t b = unit / p.seq.H;
  const int32_t h = unit % p.seq.H;
  const int64_t T = p.seq.T, len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kN * kEsz<F32>;
  const int64_t nblk = (T + kBlk - 1) / kBlk;
  const int64_t blk0 = seg * p.seg_pieces * kPieceBlocks;
  int64_t blk1 = blk0 + p.seg_pieces * kPieceBlocks;
  if (blk1 > nblk) blk1 = nblk;
  const int last_piece = (int)((blk1 - 1) / kPieceBlocks);
  const uint32_t off = li * row_bytes + q * 8 * kEsz<F32>;
  auto at = [&](const void* x, int64_t t0, int64_t n) { return token_buffer<kEsz<F32>>(x, p.seq, b, h, t0, n, kSub); };

#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int tu = 4 * wave + m;
    f32x4 g = zero4();
    if (p.nseg > 1)
      g = *state_tile(p.grads, unit * p.pieces + last_piece, tu, lane);
    else if (p.ds_out)
      g = *reinterpret_cast<const f32x4*>(p.ds_out + unit * kN * kN + state_offset(tu >> 2, tu & 3, lane));
    carry[tu][lane] = g;
  }
  const Turn E = make_turn(lane);
  float head_sum = 0.f;  // one decay per head: its gradient's terms of this lane's tokens
  for (int64_t blk = blk1 - 1; blk >= blk0; --blk) {
    const int64_t t0 = blk * kBlk + wave * kSub;
    if (blk * kBlk >= len) {  // behind the sequence's end: no gradients
#pragma unroll
      for (int J = 0; J < 2; ++J)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t o = off + J * 16 * row_bytes + hh * 32 * kEsz<F32>;
          store_pair<F32>(at(p.dr, t0, T - t0), o, zero4(), zero4());
          store_pair<F32>(at(p.dk, t0, T - t0), o, zero4(), zero4());
          store_pair<F32>(at(p.dv, t0, T - t0), o, zero4(), zero4());
        }
      if (p.per_token && lane < kSub && t0 + lane < T) p.dlog_w[(b * T + t0 + lane) * p.seq.H + h] = 0.f;
      continue;
    }
    Raw<F32> rr, rk, rv, rd;
    load_raw<F32>(rr, at(p.r, t0, len - t0), row_bytes, lane);
    load_raw<F32>(rd, at(p.dy, t0, len - t0), row_bytes, lane);
    load_raw<F32>(rk, at(p.k, t0, len - t0), row_bytes, lane);
    load_raw<F32>(rv, at(p.v, t0, len - t0), row_bytes, lane);
    const Decay d = make_decay(log_w_here(load_log_w(p.log_w, p.per_token, p.seq, b, h, t0, len, lane), t0, len, lane), sums[wave], lane);

    auto turn = [&](const Raw<F32>& x, int t) { return turned_op(natural<F32>(x, 0, t >> 1), natural<F32>(x, 1, t >> 1), E, t); };
    // What the 32 tokens add to S and to G, for the other waves (wave 0's G for the next carry). A phase ends where
    // its registers do: the compiler is kept from mixing the phases, whose operands together would not fit.
    if (wave < kWaves - 1) {
      Op<NI> Kt[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) Kt[t] = turn(rk, t);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 a0 = turned(natural<F32>(rv, 0, u >> 1), E, u), a1 = turned(natural<F32>(rv, 1, u >> 1), E, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] *= d.row[0][i], a1[i] *= d.row[1][i];
        const Op<3> Vs = pack<3>(a0, a1);
#pragma unroll
        for (int t = 0; t < 4; ++t) addS[wave][4 * t + u][lane] = mma(Kt[t], Vs, zero4());
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    {
      Op<NI> Rt[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) Rt[t] = turn(rr, t);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 a0 = turned(natural<F32>(rd, 0, u >> 1), E, u), a1 = turned(natural<F32>(rd, 1, u >> 1), E, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] *= d.inrow[0][i], a1[i] *= d.inrow[1][i];
        const Op<3> Ds = pack<3>(a0, a1);
#pragma unroll
        for (int t = 0; t < 4; ++t) addG[wave][4 * t + u][lane] = mma(Rt[t], Ds, zero4());
      }
    }
    if (lane == 0) all[wave] = d.all;
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);

    // the gradient behind the wave's tokens, tile (t, u)
    auto grad_tile = [&](int tu) {
      f32x4 g = carry[tu][lane];
      for (int w = kWaves - 1; w > wave; --w) g = fma4(g, all[w], addG[w][tu][lane]);
      return g;
    };
    float cross[2] = {0.f, 0.f};  // this lane's rows of the pairs that cross token 16J + li
    float kdk[2] = {0.f, 0.f}, rdr[2] = {0.f, 0.f}, dot = 0.f;
    {  // dv and dk
      Op<NO> Pi[2], Ai[2];  // P and D A with rows i
      {
        f32x4 q00 = zero4(), q10 = zero4(), q11 = zero4(), a00 = zero4(), a10 = zero4(), a11 = zero4();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const Op<NI> D0 = natural<F32>(rd, 0, hh), D1 = natural<F32>(rd, 1, hh);
          const Op<NI> V0 = natural<F32>(rv, 0, hh), V1 = natural<F32>(rv, 1, hh);
          q00 = mma(D0, V0, q00), q10 = mma(D1, V0, q10), q11 = mma(D1, V1, q11);
          const Op<NI> R0 = natural<F32>(rr, 0, hh), R1 = natural<F32>(rr, 1, hh);
          const Op<NI> K0 = natural<F32>(rk, 0, hh), K1 = natural<F32>(rk, 1, hh);
          a00 = mma(R0, K0, a00), a10 = mma(R1, K0, a10), a11 = mma(R1, K1, a11);
        }
        q00 = masked_i(q00, d.t00, lane), q10 = q10 * d.t10, q11 = masked_i(q11, d.t11, lane);
        Pi[0] = pack<NO>(q00, q10);
        Pi[1] = pack<NO>(zero4(), q11);
        Ai[0] = pack<NO>(masked_i(a00, d.t00, lane), a10 * d.t10);
        Ai[1] = pack<NO>(zero4(), masked_i(a11, d.t11, lane));
        // pairs i >= t > j: what each row has in the columns before t, from the rows from t on
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w00 = a00[i] * q00[i], w10 = a10[i] * q10[i], w11 = a11[i] * q11[i];
          const float before00 = row_sums_to(dpp_f32<0x111>(w00)), before10 = row_sums_to(dpp_f32<0x111>(w10));
          const float before11 = row_sums_to(dpp_f32<0x111>(w11)) + row16_sum(w10);
          const bool from = 4 * q + i >= li;
          cross[0] += (from ? before00 : 0.f) + before10;
          cross[1] += from ? before11 : 0.f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      f32x4 dk[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t) dk[t][0] = dk[t][1] = zero4();
#pragma unroll
      for (int hv = 0; hv < 2; ++hv) {  // half of the values at a time
        f32x4 dv[2][2];
        Op<3> Go[2][2];  // [value tile 2hv + e][key half]: rows are values
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int u = 2 * hv + e;
#pragma unroll
          for (int m = 0; m < 2; ++m) Go[e][m] = pack<3>(grad_tile(8 * m + u), grad_tile(8 * m + 4 + u));
          const Op<NI> Dt = turn(rd, u);
#pragma unroll
          for (int J = 0; J < 2; ++J) {
            f32x4 o = mma(Go[e][0], natural<F32>(rk, J, 0), zero4());
            o = mma(Go[e][1], natural<F32>(rk, J, 1), o);
            dv[e][J] = mma(Dt, Ai[J], o * d.out[J]);
          }
        }
#pragma unroll
        for (int J = 0; J < 2; ++J)
          store_pair<F32>(at(p.dv, t0, T - t0), off + J * 16 * row_bytes + hv * 32 * kEsz<F32>, dv[0][J], dv[1][J]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const Op<3> Gt = turned_op(Go[0][t >> 1], Go[1][t >> 1], E, t);
#pragma unroll
          for (int J = 0; J < 2; ++J) dk[t][J] = mma(Gt, natural<F32>(rv, J, hv), dk[t][J]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int J = 0; J < 2; ++J) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = 2 * hh + e;
            dk[t][J] = dk[t][J] * d.out[J];
#pragma unroll
            for (int i = 0; i < 4; ++i) kdk[J] = fmaf(dk[t][J][i], element<F32>(rk, J, hh, e, i), kdk[J]);
            dk[t][J] = mma(turn(rr, t), Pi[J], dk[t][J]);
          }
          store_pair<F32>(at(p.dk, t0, T - t0), off + J * 16 * row_bytes + hh * 32 * kEsz<F32>, dk[2 * hh][J],
                          dk[2 * hh + 1][J]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    {  // dr
      const int64_t piece = blk / kPieceBlocks;
      const bool marked = blk % kPieceBlocks != 0;
      const float mark_decay = marked ? p.mark_decay[unit * nblk + blk] : 1.f;
      f32x4 dr[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t) dr[t][0] = dr[t][1] = zero4();
#pragma unroll
      for (int hv = 0; hv < 2; ++hv) {
        Op<3> So[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int u = 2 * hv + e;
          f32x4 s[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int tu = 4 * t + u;
            s[t] = zero4();
            if (p.pieces > 1)
              s[t] = *state_tile(p.states, unit * p.pieces + piece, tu, lane);
            else if (p.s_in)
              s[t] = *reinterpret_cast<const f32x4*>(p.s_in + unit * kN * kN + state_offset(t, u, lane));
            if (marked) s[t] = fma4(s[t], mark_decay, *state_tile(p.marks, unit * nblk + blk, tu, lane));
            for (int w = 0; w < wave; ++w) s[t] = fma4(s[t], all[w], addS[w][tu][lane]);
            const f32x4 g = grad_tile(tu);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot = fmaf(s[t][i], g[i], dot);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) So[e][m] = pack<3>(s[2 * m], s[2 * m + 1]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const Op<3> St = turned_op(So[0][t >> 1], So[1][t >> 1], E, t);
#pragma unroll
          for (int J = 0; J < 2; ++J) dr[t][J] = mma(St, natural<F32>(rd, J, hv), dr[t][J]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      Op<NO> Pj[2];  // P with rows j
      {
        f32x4 p00 = zero4(), p01 = zero4(), p11 = zero4();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const Op<NI> D0 = natural<F32>(rd, 0, hh), D1 = natural<F32>(rd, 1, hh);
          const Op<NI> V0 = natural<F32>(rv, 0, hh), V1 = natural<F32>(rv, 1, hh);
          p00 = mma(V0, D0, p00), p01 = mma(V0, D1, p01), p11 = mma(V1, D1, p11);
        }
        Pj[0] = pack<NO>(masked_j(p00, d.d00, lane), zero4());
        Pj[1] = pack<NO>(p01 * d.d01, masked_j(p11, d.d11, lane));
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int J = 0; J < 2; ++J) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = 2 * hh + e;
            dr[t][J] = dr[t][J] * d.col[J];
#pragma unroll
            for (int i = 0; i < 4; ++i) rdr[J] = fmaf(dr[t][J][i], element<F32>(rr, J, hh, e, i), rdr[J]);
            dr[t][J] = mma(turn(rk, t), Pj[J], dr[t][J]);
          }
          store_pair<F32>(at(p.dr, t0, T - t0), off + J * 16 * row_bytes + hh * 32 * kEsz<F32>, dr[2 * hh][J],
                          dr[2 * hh + 1][J]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    // dlog_w: lane l has token l % 32
#pragma unroll
    for (int J = 0; J < 2; ++J) cross[J] = rows_sum(cross[J]), rdr[J] = rows_sum(rdr[J]), kdk[J] = rows_sum(kdk[J]);
    const bool second = lane & 16;
    const float pairs = second ? cross[1] : cross[0];
    const float here = second ? rdr[1] : rdr[0], before = second ? kdk[1] : kdk[0];
    dot = rows_sum(row16_sum(dot));
    const int64_t t = t0 + (lane & 31);
    float dlw = pairs + sum_from(here, lane) + sum_before(before, lane) + dot * d.all;
    if (t >= len) dlw = 0.f;
    if (p.per_token) {
      if (lane < kSub && t < T) p.dlog_w[(b * T + t) * p.seq.H + h] = dlw;
    } else {
      head_sum += dlw;
    }
    __syncthreads();  // every wave has read what was added and the carried gradient
#pragma unroll
    for (int m = 0; m < 4; ++m) {  // the gradient behind the next block, before this one
      const int tu = 4 * wave + m;
      f32x4 g = carry[tu][lane];
#pragma unroll
      for (int w = kWaves - 1; w >= 0; --w) g = fma4(g, all[w], addG[w][tu][lane]);
      carry[tu][lane] = g;
    }
    __syncthreads();
  }
  if (p.ds_in && seg == 0) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int tu = 4 * wave + m;
      *reinterpret_cast<f32x4*>(p.ds_in + unit * kN * kN + state_offset(tu >> 2, tu & 3, lane)) = carry[tu][lane];
    }
  }
  if (!p.per_token) {  // both halves of the wave hold the same 32 tokens
    float s = row16_sum(head_sum);
    s += __shfl_xor(s, 16, 64);
    if (lane == 0) all[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.dlog_w[unit * p.nseg + seg] = (all[0] + all[1]) + (all[2] + all[3]);
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

constexpr int kGradLds = 8 * 16384 + kWaves * kSub * 8 + 64;

}  // namespace

hipError_t launch_linattn_zero(float* dlog_w, int64_t H, hipStream_t stream) {
  void* args[] = {&dlog_w, &H};
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_zero_kernel), dim3((uint32_t)((H + 255) / 256)), dim3(256),
                         args, 0, stream);
}

hipError_t launch_linattn_head_sum(const float* parts, float* dlog_w, int64_t B, int64_t H, int64_t n, hipStream_t stream) {
  int32_t heads = (int32_t)H, nseg = (int32_t)n;
  void* args[] = {&parts, &dlog_w, &B, &heads, &nseg};
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_head_sum_kernel), dim3((uint32_t)H), dim3(64), args, 0, stream);
}

hipError_t launch_linattn_backward(const LinattnCall& c) {
  if (!c.f32) return launch_linattn_backward16(c);
  const int64_t units = c.B * c.H, nblk = linattn_blocks(c.T), pieces = linattn_pieces(c.T), cus = linattn_cus();
  // Segments: a workgroup for each compute unit, of whole pieces.
  int64_t nseg = cus / units > 0 ? cus / units : 1;
  if (nseg > pieces) nseg = pieces;
  const int64_t seg_pieces = (pieces + nseg - 1) / nseg;
  nseg = (pieces + seg_pieces - 1) / seg_pieces;

  const bool marks = nblk > 1, states = marks;
  size_t need = 0;
  auto room = [&](size_t bytes) {
    const size_t at = need;
    need += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t o_states = room(states ? units * pieces * kLinattnStateBytes : 0), o_decay = room(units * pieces * 4), o_gdecay = room(units * pieces * 4);
  const size_t o_marks = room(marks ? units * nblk * kLinattnStateBytes : 0), o_mdecay = room(marks ? units * nblk * 4 : 0);
  const size_t o_grads = room(nseg > 1 ? units * pieces * kLinattnStateBytes : 0);
  const size_t o_parts = room(c.per_token ? 0 : units * nseg * 4);
  void* ws = nullptr;
  hipError_t e = device_workspace(c.stream, need, &ws, kWorkspaceOperators);
  if (e != hipSuccess) return e;
  char* base = static_cast<char*>(ws);

  LinattnPieces f{}, g{};
  f.every = g.every = 1;
  f.states = reinterpret_cast<float*>(base + o_states), f.decay = reinterpret_cast<float*>(base + o_decay);
  f.marks = reinterpret_cast<float*>(base + o_marks), f.mark_decay = reinterpret_cast<float*>(base + o_mdecay);
  g.states = reinterpret_cast<float*>(base + o_grads), g.decay = reinterpret_cast<float*>(base + o_gdecay);
  if (states) {
    e = launch_linattn_states(c, &f, nseg > 1 ? &g : nullptr);
    if (e != hipSuccess) return e;
  }
  GradParams p{};
  p.r = c.r, p.log_w = c.log_w, p.k = c.k, p.v = c.v, p.dy = c.dy, p.s_in = c.s_in, p.ds_out = c.ds_out;
  p.states = reinterpret_cast<const float*>(base + o_states);
  p.marks = reinterpret_cast<const float*>(base + o_marks);
  p.mark_decay = reinterpret_cast<const float*>(base + o_mdecay);
  p.grads = reinterpret_cast<const float*>(base + o_grads);
  float* parts = reinterpret_cast<float*>(base + o_parts);
  p.dr = c.dr, p.dlog_w = c.per_token ? c.dlog_w : parts, p.dk = c.dk, p.dv = c.dv, p.ds_in = c.ds_in;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  p.nseg = (int32_t)nseg, p.pieces = pieces, p.seg_pieces = seg_pieces;
  const void* fn = c.f32 ? reinterpret_cast<const void*>(&linattn_grad_kernel<true>)
                         : reinterpret_cast<const void*>(&linattn_grad_kernel<false>);
  static const hipError_t a0 = hipFuncSetAttribute(reinterpret_cast<const void*>(&linattn_grad_kernel<true>),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, kGradLds);
  static const hipError_t a1 = hipFuncSetAttribute(reinterpret_cast<const void*>(&linattn_grad_kernel<false>),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, kGradLds);
  if (a0 != hipSuccess) return a0;
  if (a1 != hipSuccess) return a1;
  void* args[] = {&p};
  e = hipLaunchKernel(fn, dim3((uint32_t)(units * nseg)), dim3(64 * kWaves), args, kGradLds, c.stream);
  if (e != hipSuccess || c.per_token) return e;
  return launch_linattn_head_sum(parts, c.dlog_w, c.B, c.H, nseg, c.stream);
}

}  // namespace rwkv7
