// Linear attention with a decay for each head: whole prompts and single tokens.
// The chunk algebra and its number formats are in linattn_ops.hpp.
#include <atomic>

#include "linattn_internal.hpp"
#include "linattn_ops.hpp"
#include "once_per_device.hpp"
#include "operators_lock.hpp"
#include "wkv7_internal.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

struct OutParams {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const float* states;  // [units][stride] states, the first nseg those before the segments (nseg > 1)
  const float* s_in;    // the caller's state (nseg == 1), may be null
  void* y;
  float* s_out;  // may be null
  Seq seq;
  int32_t per_token;
  int32_t nseg;        // segments of a sequence
  int64_t seg_blocks;  // blocks of kBlk tokens in a segment
  int64_t stride;
};

// ---- float32. A workgroup carries 32 of the state's 64 value rows (two tiles) over one segment of one head, 128 tokens
// at a time: each wave takes 32 of them and leaves what they add to the state in LDS. Then each wave takes a quarter of
// the state's tiles through the four waves' tokens (the carried part stays in its registers) and leaves the states
// before each wave's tokens for the others. The two workgroups of a head follow each other on the same die, so
// r and k come from memory once. What the pieces of three operands take in registers leaves no room for loads ahead;
// two workgroups on a compute unit cover for each other. Issue bounds it: 6 to 7 us a block for a workgroup alone, 10 for two side
// by side; B=8 T=2048 H=32 170 us (3.1 TB/s), 236 with one on a compute unit and loads ahead.
constexpr int kVt = 2;  // value tiles of a workgroup

struct Inputs {
  Raw<true> r, k;
  u32x4 v[2][2];  // [token tile], the workgroup's 32 values
  float log_w;
};

__global__ __launch_bounds__(256, 2) void linattn_out32_kernel(OutParams p) {
  constexpr bool F32 = true;
  constexpr int NI = 3, NO = 3;
  __shared__ f32x4 added[kWaves][4 * kVt][64];
  __shared__ double sums[kWaves][kSub];
  __shared__ float all[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int half = id & 1;
  const uint32_t unit = (id >> 1) / p.nseg, seg = (id >> 1) % p.nseg;
  const int64_t b = unit / p.seq.H;
  const int32_t h = unit % p.seq.H;
  const int64_t T = p.seq.T, len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kN * kEsz<F32>;
  const int64_t blk0 = seg * p.seg_blocks;
  const int64_t nblk = (T + kBlk - 1) / kBlk;
  const int64_t blk1 = blk0 + p.seg_blocks < nblk ? blk0 + p.seg_blocks : nblk;
  // blocks with tokens in them; behind those the sequence has ended
  const int64_t live = (len + kBlk - 1) / kBlk < blk1 ? (len + kBlk - 1) / kBlk : blk1;
  const uint32_t off = (lane & 15) * row_bytes + ((lane >> 4) * 8 + half * 32) * kEsz<F32>;  // of v and y

  Inputs x;
  auto load = [&](int64_t blk) {
    const int64_t t0 = blk * kBlk + wave * kSub;
    const __amdgpu_buffer_rsrc_t vb = token_buffer<kEsz<F32>>(p.v, p.seq, b, h, t0, len - t0, kSub);
    load_raw<F32>(x.k, token_buffer<kEsz<F32>>(p.k, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
#pragma unroll
    for (int J = 0; J < 2; ++J)
#pragma unroll
      for (int m = 0; m < 2; ++m) x.v[J][m] = load16(vb, off + J * 16 * row_bytes + 16 * m);
    load_raw<F32>(x.r, token_buffer<kEsz<F32>>(p.r, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    x.log_w = load_log_w(p.log_w, p.per_token, p.seq, b, h, t0, len, lane);
  };
  f32x4 carry[kVt];  // tiles (wave, 0), (wave, 1) of the half
#pragma unroll
  for (int m = 0; m < kVt; ++m) {
    carry[m] = zero4();
    if (p.nseg > 1)
      carry[m] = *state_tile(p.states, (int64_t)unit * p.stride + seg, 4 * wave + kVt * half + m, lane);
    else if (p.s_in)
      carry[m] = *reinterpret_cast<const f32x4*>(p.s_in + (int64_t)unit * kN * kN + state_offset(wave, kVt * half + m, lane));
  }
  const Turn E = make_turn(lane);
  for (int64_t blk = blk0; blk < live; ++blk) {
    load(blk);
    const int64_t t0 = blk * kBlk + wave * kSub;
    const Decay d = make_decay(log_w_here(x.log_w, t0, len, lane), sums[wave], lane);
    // what the 32 tokens add to the state: tiles (t, u) of sum_j k_j (left_j v_j)^T
    Op<NI> Vt[kVt];
    {
      Op<3> Vs[kVt];
#pragma unroll
      for (int m = 0; m < kVt; ++m) {
        const Op<NI> v0 = pieces<F32>(x.v[0]), v1 = pieces<F32>(x.v[1]);
        f32x4 a0 = turned(v0, E, m), a1 = turned(v1, E, m);
        Vt[m] = turned_op(v0, v1, E, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] *= d.row[0][i], a1[i] *= d.row[1][i];
        Vs[m] = pack<3>(a0, a1);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Op<NI> Kt = turned_op(natural<F32>(x.k, 0, t >> 1), natural<F32>(x.k, 1, t >> 1), E, t);
#pragma unroll
        for (int m = 0; m < kVt; ++m) added[wave][kVt * t + m][lane] = mma(Kt, Vs[m], zero4());
      }
    }
    if (lane == 0) all[wave] = d.all;
    lds_barrier();
    // the states before each wave's tokens: this wave's two tiles of them, in the place of what the wave adds
    f32x4 add[kWaves][kVt];
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int m = 0; m < kVt; ++m) add[w][m] = added[w][kVt * wave + m][lane];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float a = all[w];
#pragma unroll
      for (int m = 0; m < kVt; ++m) {
        added[w][kVt * wave + m][lane] = carry[m];
        carry[m] = fma4(carry[m], a, add[w][m]);
      }
    }
    // the pairs inside the 32 tokens, as operands over the tokens j: column i
    Op<NO> P[2];
    {
      f32x4 a00 = zero4(), a01 = zero4(), a11 = zero4();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const Op<NI> K0 = natural<F32>(x.k, 0, hh), K1 = natural<F32>(x.k, 1, hh);
        const Op<NI> R0 = natural<F32>(x.r, 0, hh), R1 = natural<F32>(x.r, 1, hh);
        a00 = mma(K0, R0, a00);
        a01 = mma(K0, R1, a01);
        a11 = mma(K1, R1, a11);
      }
      P[0] = pack<NO>(masked_j(a00, d.d00, lane), zero4());
      P[1] = pack<NO>(a01 * d.d01, masked_j(a11, d.d11, lane));
    }
    lds_barrier();
    f32x4 y[2][kVt];
#pragma unroll
    for (int m = 0; m < kVt; ++m) {
      const Op<NO> S0 = pack<NO>(added[wave][m][lane], added[wave][kVt + m][lane]);
      const Op<NO> S1 = pack<NO>(added[wave][2 * kVt + m][lane], added[wave][3 * kVt + m][lane]);
#pragma unroll
      for (int I = 0; I < 2; ++I) {
        f32x4 o = mma(S0, natural<F32>(x.r, I, 0), zero4());
        o = mma(S1, natural<F32>(x.r, I, 1), o);
        y[I][m] = mma(Vt[m], P[I], o * d.col[I]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const __amdgpu_buffer_rsrc_t yb = token_buffer<kEsz<F32>>(p.y, p.seq, b, h, t0, T - t0, kSub);
#pragma unroll
    for (int I = 0; I < 2; ++I) store_pair<F32>(yb, off + I * 16 * row_bytes, y[I][0], y[I][1]);
  }
  for (int64_t blk = live > blk0 ? live : blk0; blk < blk1; ++blk) {  // behind the sequence's end: zeros
    const int64_t t0 = blk * kBlk + wave * kSub;
    const __amdgpu_buffer_rsrc_t yb = token_buffer<kEsz<F32>>(p.y, p.seq, b, h, t0, T - t0, kSub);
#pragma unroll
    for (int I = 0; I < 2; ++I) store_pair<F32>(yb, off + I * 16 * row_bytes, zero4(), zero4());
  }
  if (p.s_out && blk1 == nblk) {
#pragma unroll
    for (int m = 0; m < kVt; ++m)
      *reinterpret_cast<f32x4*>(p.s_out + (int64_t)unit * kN * kN + state_offset(wave, kVt * half + m, lane)) = carry[m];
  }
}

// ---- bfloat16. Eight waves of one workgroup take a whole head: 128 tokens at a time, in quarters of 32, two waves
// (32 value rows each) to a quarter. Memory bounds this kernel, and what it reaches hangs on whole 128-byte rows, each
// asked for once: a stream of this layout (three tensors read, one written, a workgroup a head) measured 4.9 TB/s
// in whole rows without temporal hint and consecutive workgroups on consecutive dies, 4.3 with an L2-friendly
// numbering, and 3.2 where two workgroups a head loaded 64-byte pieces in operand order. So the rows go to LDS by
// direct loads, a block ahead (into the same place, as soon as every wave has taken its operands into registers),
// their 16-byte pieces exchanged within a row so that the operand reads of 16 rows fall into different banks.
//
// B=4 T=16384 H=64 513 to 518 us (4.2 TB/s); the loads and stores alone take 482, the arithmetic alone 436.
//
// What is common to the two waves of a quarter, the decay factors of its tokens, one of them leaves in LDS during
// the block before (once, if the head has one decay and the tokens are all there).
constexpr int kTile = kSub * kRow;        // bytes of a quarter's rows of one tensor
constexpr int kExchange = 0;              // [quarter][half][8 tiles][64 lanes] 16 bytes
constexpr int kStage = 64 << 10;          // [quarter][r, k, v] kTile
constexpr int kStageW = kStage + 12 * kTile;       // [block % 4][quarter][32] float
constexpr int kFactors = kStageW + 16 * kSub * 4;  // [quarter] Factors
struct Factors {
  f32x4 d[3][64];     // D tiles (0, 0), (0, 1), (1, 1) in the layout of Decay::d00
  float left[kSub];   // exp(c_31 - c)
  float in[kSub];     // exp(c)
  float all, unused[3];
};
constexpr int kOutLds = kFactors + 4 * sizeof(Factors);
static_assert(kOutLds <= 160 * 1024, "LDS of a compute unit");

__global__ __launch_bounds__(512, 2) void linattn_out16_kernel(OutParams p) {
  extern __shared__ char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 2, quarter = wave & 3;
  const uint32_t unit = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
  const int64_t b = unit / p.seq.H;
  const int32_t h = unit % p.seq.H;
  const int64_t T = p.seq.T, len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kRow;
  const int64_t blk0 = seg * p.seg_blocks;
  const int64_t nblk = (T + kBlk - 1) / kBlk;
  const int64_t blk1 = blk0 + p.seg_blocks < nblk ? blk0 + p.seg_blocks : nblk;
  const int64_t live = (len + kBlk - 1) / kBlk < blk1 ? (len + kBlk - 1) / kBlk : blk1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  // Rows to LDS: an instruction takes 8 rows. The two waves of a quarter take 16 rows each.
  const int row = 16 * half + (lane >> 3);
  const uint32_t src0 = row * row_bytes + 16 * ((lane & 7) ^ row_key(row));
  const uint32_t src1 = (row + 8) * row_bytes + 16 * ((lane & 7) ^ row_key(row + 8));
  const int64_t first = blk0 * kBlk + quarter * kSub, start = ((b * T + first) * p.seq.H + h) * kRow;
  const char *next_r = static_cast<const char*>(p.r) + start, *next_k = static_cast<const char*>(p.k) + start,
             *next_v = static_cast<const char*>(p.v) + start;
  int64_t left = len - first;  // tokens from the next staged one on
  const uint32_t to0 = lds0 + kStage + quarter * 3 * kTile + 16 * half * kRow;
  auto stage = [&](const char*& x, int number) {
    const u32x4 d = descriptor(x, left <= 0 ? 0 : (uint32_t)((left < kSub ? left : kSub) - 1) * row_bytes + kRow);
    to_lds16_last(d, src0, to0 + number * kTile);
    to_lds16_last(d, src1, to0 + number * kTile + 8 * kRow);
    x += (int64_t)kBlk * row_bytes;
  };
  auto stage_w = [&](int64_t blk) {
    if (half == 1 && lane < kSub) {
      const Span span = log_w_span(p.log_w, p.per_token, p.seq, b, h, blk * kBlk + quarter * kSub, len);
      to_lds4(descriptor(span.base, span.bytes), lane * (p.per_token ? p.seq.H * 4 : 0),
              lds0 + kStageW + ((blk & 3) * 4 + quarter) * kSub * 4);
    }
  };
  const int rows_r = kStage + quarter * 3 * kTile, rows_k = rows_r + kTile, rows_v = rows_k + kTile;
  const int li = lane & 15, q = lane >> 4;
  const int nat0 = swizzled(li, q), turn0 = swizzled(4 * q + (li >> 2), li & 3);
  // operand of the rows 16J + li, channels 32hh + 8q ..
  auto staged = [&](int from, int J, int hh) {
    return Op<1>{{*reinterpret_cast<const bf16x8*>(lds + from + 16 * J * kRow + (nat0 ^ 64 * hh))}};
  };
  // operand over the 32 tokens, rows the channels of tile t
  auto staged_turned = [&](int from, int t) {
    const char* const at = lds + from + (turn0 ^ 64 * (t >> 1)) + 8 * (t & 1);
    return Op<1>{{join(turned4(at), turned4(at + 16 * kRow))}};
  };

  f32x4 carry[kVt];  // tiles (quarter, 0), (quarter, 1) of the half
#pragma unroll
  for (int m = 0; m < kVt; ++m) {
    carry[m] = zero4();
    if (p.nseg > 1)
      carry[m] = *state_tile(p.states, (int64_t)unit * p.stride + seg, 4 * quarter + kVt * half + m, lane);
    else if (p.s_in)
      carry[m] = *reinterpret_cast<const f32x4*>(p.s_in + (int64_t)unit * kN * kN + state_offset(quarter, kVt * half + m, lane));
  }
  f32x4(*exch)[2][8][64] = reinterpret_cast<f32x4(*)[2][8][64]>(lds + kExchange);
  Factors* factors = reinterpret_cast<Factors*>(lds + kFactors);
  // The factors of a block's quarter, by its second wave, which has its exchange slot to itself then.
  auto fill = [&](int64_t blk) {
    const float lw = reinterpret_cast<const float*>(lds + kStageW)[((blk & 3) * 4 + quarter) * kSub + (lane & 31)];
    const Decay d = make_decay(log_w_here(lw, blk * kBlk + quarter * kSub, len, lane),
                               reinterpret_cast<double*>(exch[quarter][1]), lane);
    Factors& f = factors[quarter];
    f.d[0][lane] = d.d00, f.d[1][lane] = d.d01, f.d[2][lane] = d.d11;
    if ((lane & 15) == 0)
#pragma unroll
      for (int J = 0; J < 2; ++J)
        *reinterpret_cast<f32x4*>(f.left + 16 * J + (lane >> 2)) = f32x4{d.row[J][0], d.row[J][1], d.row[J][2], d.row[J][3]};
    if (lane < 16) f.in[lane] = d.col[0], f.in[16 + lane] = d.col[1];
    if (lane == 0) f.all = d.all;
  };
  if (blk0 < live) {
    stage_w(blk0), stage_w(blk0 + 1), stage_w(blk0 + 2);
    stage(next_k, 1), stage(next_v, 2), stage(next_r, 0);
    left -= kBlk;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (half == 1) fill(blk0);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  for (int64_t blk = blk0; blk < live; ++blk) {
    const int64_t t0 = blk * kBlk + quarter * kSub;
    const Factors& f = factors[quarter];
    Op<1> R[2][2];
    f32x4 y[2][kVt];
    float in[2];
    {
      Op<1> K[2][2];
#pragma unroll
      for (int J = 0; J < 2; ++J)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) K[J][hh] = staged(rows_k, J, hh), R[J][hh] = staged(rows_r, J, hh);
      Op<1> Kt[4], Vt[kVt];
#pragma unroll
      for (int x = 0; x < 4; ++x) Kt[x] = staged_turned(rows_k, x);
#pragma unroll
      for (int m = 0; m < kVt; ++m) Vt[m] = staged_turned(rows_v, kVt * half + m);
      lds_barrier();  // both waves of every quarter have their operands
      // the next block's rows, a tensor at a time: all at once they fill the queue of loads and hold the waves up
      stage_w(blk + 3);
      stage(next_k, 1);
      const f32x4 left0 = *reinterpret_cast<const f32x4*>(f.left + 4 * q);
      const f32x4 left1 = *reinterpret_cast<const f32x4*>(f.left + 16 + 4 * q);
      in[0] = f.in[li], in[1] = f.in[16 + li];
      // what the 32 tokens add to the state: tiles (t, m) of sum_j k_j (left_j v_j)^T
      Op<3> Vs[kVt];
#pragma unroll
      for (int m = 0; m < kVt; ++m) {
        f32x4 a0, a1;
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] = (float)Vt[m].p[0][i], a1[i] = (float)Vt[m].p[0][4 + i];
        Vs[m] = pack<3>(a0 * left0, a1 * left1);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int m = 0; m < kVt; ++m) exch[quarter][half][kVt * x + m][lane] = mma(Kt[x], Vs[m], zero4());
      stage(next_v, 2);
      // the pairs inside the 32 tokens
      f32x4 a00 = zero4(), a01 = zero4(), a11 = zero4();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        a00 = mma(K[0][hh], R[0][hh], a00);
        a01 = mma(K[0][hh], R[1][hh], a01);
        a11 = mma(K[1][hh], R[1][hh], a11);
      }
      const Op<2> P0 = pack<2>(masked_j(a00, f.d[0][lane], lane), zero4());
      const Op<2> P1 = pack<2>(a01 * f.d[1][lane], masked_j(a11, f.d[2][lane], lane));
#pragma unroll
      for (int m = 0; m < kVt; ++m) y[0][m] = mma(Vt[m], P0, zero4()), y[1][m] = mma(Vt[m], P1, zero4());
    }
    stage(next_r, 0);
    left -= kBlk;
    lds_barrier();
    // The states before each quarter's tokens: this wave takes its two tiles through them, and leaves each as two
    // bfloat16 pieces where it found what the quarter adds (nobody else reads that).
    f32x4 add[4][kVt];
    float all[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      all[w] = factors[w].all;
#pragma unroll
      for (int m = 0; m < kVt; ++m) add[w][m] = exch[w][half][kVt * quarter + m][lane];
    }
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int m = 0; m < kVt; ++m) {
        const Op<2> o = pack<2>(carry[m], zero4());
#pragma unroll
        for (int n = 0; n < 2; ++n)
          reinterpret_cast<bf16x4*>(exch[w][half][kVt * quarter + m])[64 * n + lane] =
              __builtin_shufflevector(o.p[n], o.p[n], 0, 1, 2, 3);
        carry[m] = fma4(carry[m], all[w], add[w][m]);
      }
    lds_barrier();
#pragma unroll
    for (int m = 0; m < kVt; ++m) {
      Op<2> S[2];
#pragma unroll
      for (int kh = 0; kh < 2; ++kh)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const bf16x4 e0 = reinterpret_cast<const bf16x4*>(exch[quarter][half][kVt * (2 * kh) + m])[64 * n + lane];
          const bf16x4 e1 = reinterpret_cast<const bf16x4*>(exch[quarter][half][kVt * (2 * kh + 1) + m])[64 * n + lane];
          S[kh].p[n] = __builtin_shufflevector(e0, e1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
#pragma unroll
      for (int I = 0; I < 2; ++I) y[I][m] = fma4(mma(S[1], R[I][1], mma(S[0], R[I][0], zero4())), in[I], y[I][m]);
    }
    const __amdgpu_buffer_rsrc_t yb = token_buffer<2>(p.y, p.seq, b, h, t0, T - t0, kSub);
#pragma unroll
    for (int I = 0; I < 2; ++I)
      store_pair<false>(yb, (16 * I + li) * row_bytes + 64 * half + 16 * q, y[I][0], y[I][1]);
    if (half == 1 && blk + 1 < live && (p.per_token || t0 + kBlk + kSub > len)) fill(blk + 1);
    // the next block's rows are there (and log w of three blocks): behind them are two stores
    asm volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to this workgroup's LDS when it ends
  for (int64_t blk = live > blk0 ? live : blk0; blk < blk1; ++blk) {  // behind the sequence's end: zeros
    const int64_t t0 = blk * kBlk + quarter * kSub;
    const __amdgpu_buffer_rsrc_t yb = token_buffer<2>(p.y, p.seq, b, h, t0, T - t0, kSub);
#pragma unroll
    for (int I = 0; I < 2; ++I) store_pair<false>(yb, (16 * I + li) * row_bytes + 64 * half + 16 * q, zero4(), zero4());
  }
  if (p.s_out && blk1 == nblk) {
#pragma unroll
    for (int m = 0; m < kVt; ++m)
      *reinterpret_cast<f32x4*>(p.s_out + (int64_t)unit * kN * kN + state_offset(quarter, kVt * half + m, lane)) = carry[m];
  }
}

// Pieces of a segment of a sequence. A workgroup a head and segment, alone on a compute unit, takes 3.5 us for a block of 128
// tokens; float32: two workgroups, two to a compute unit, 7 us alone and 10 side by side. So a call of few heads, or of a few
// more than a round of the compute units takes, ends sooner in segments: each in its own workgroup, from the state that the
// pieces before it add up to. Those cost another pass over k and v and two more launches: about 12 us, and the segments but
// the last at 4 TB/s. B=1 T=16384 H=32 bfloat16 113 us in segments of 4 pieces, 133 of one, 162 of 8, 474 in one segment
// (float32 H=64: 420 in segments of 8, 458 of one, 527 of 16, 831 in one); B=4 T=2048 H=64 71 in one segment, 104 in two
// (float32 165 and 214).
int64_t segment_pieces(int64_t units, int64_t blocks, int64_t pieces, bool f32) {
  const int64_t cus = linattn_cus(), slots = f32 ? 2 : 1;  // workgroups of a head and segment, and of a compute unit
  int64_t best_every = pieces;
  double best = 0;
  for (int64_t every = pieces; every >= 1; every = every > 1 ? (every + 1) / 2 : 0) {
    const int64_t nseg = (pieces + every - 1) / every, groups = units * nseg * slots;
    const int64_t rounds = (groups + slots * cus - 1) / (slots * cus);
    const double length = (double)(every * kPieceBlocks < blocks ? every * kPieceBlocks : blocks);
    double us = rounds * (length * (!f32 ? 3.5 : groups <= cus ? 7.0 : 10.0) + 2.0);
    if (nseg > 1) us += 12.0 + (double)units * (nseg - 1) * length * kBlk * (f32 ? 512 : 256) / 4e6;
    if (every == pieces || us < best) best = us, best_every = every;
  }
  return best_every;
}

template <bool F32>
hipError_t launch_out(const LinattnCall& c) {
  const int64_t units = c.B * c.H, blocks = linattn_blocks(c.T, kBlk);
  OutParams p{};
  p.r = c.r, p.log_w = c.log_w, p.k = c.k, p.v = c.v, p.s_in = c.s_in, p.y = c.y, p.s_out = c.s_out;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  const int64_t pieces = linattn_pieces(c.T, kBlk), every = segment_pieces(units, blocks, pieces, F32);
  p.nseg = (int32_t)((pieces + every - 1) / every);
  p.seg_blocks = p.nseg > 1 ? every * kPieceBlocks : blocks;
  std::unique_lock<std::mutex> lock(operators_mutex(), std::defer_lock);
  if (p.nseg > 1) {
    lock.lock();
    // what the last segment adds nobody asks for here
    LinattnPieces q{};
    q.units = units, q.pieces = (p.nseg - 1) * every, q.every = (int32_t)every;
    q.start = c.s_in;
    p.stride = q.stride = q.end_stride = q.pieces + 1;
    const size_t states = (size_t)units * q.stride * kLinattnStateBytes;
    void* ws = nullptr;
    hipError_t e = device_workspace(c.stream, states + units * q.stride * 4, &ws, kWorkspaceOperators);
    if (e != hipSuccess) return e;
    q.states = static_cast<float*>(ws);
    q.end = q.states + (p.nseg - 1) * (kLinattnStateBytes / 4);
    q.decay = reinterpret_cast<float*>(static_cast<char*>(ws) + states);
    e = launch_linattn_states(c, kBlk, &q, nullptr);
    if (e != hipSuccess) return e;
    p.states = static_cast<const float*>(ws);
  }
  void* args[] = {&p};
  if constexpr (!F32) {
    static std::atomic<uint64_t> granted{0};
    const void* fn = reinterpret_cast<const void*>(&linattn_out16_kernel);
    const hipError_t a = allow_lds(granted, fn, kOutLds);
    if (a != hipSuccess) return a;
    return hipLaunchKernel(fn, dim3((uint32_t)(units * p.nseg)), dim3(512), args, kOutLds, c.stream);
  } else {
    return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_out32_kernel), dim3((uint32_t)(units * p.nseg * 2)),
                           dim3(64 * kWaves), args, 0, c.stream);
  }
}

// ---- single tokens. S is read and written once (32 KiB of a head's 32.5): 16 lanes hold a value
// row's 64 keys, a wave 16 rows, one workgroup a head. Row sums by the DPP butterfly. B=512 H=32 96 us (5.6 TB/s).
struct StepParams {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const float* s_in;  // may be null
  void* y;
  float* s_out;  // may be null
  int32_t H;
  int32_t per_token;
};

__device__ __forceinline__ float4 widen4(const void* base, int64_t at, bool f32) {
  if (f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

template <bool F32>
__global__ __launch_bounds__(256) void linattn_step_kernel(StepParams p) {
  const int lane = threadIdx.x & 63, c = lane & 15, ri = lane >> 4;
  const int64_t unit = blockIdx.x;
  const int row0 = 16 * (threadIdx.x >> 6);
  const int64_t sbase = unit * kN * kN;
  f32x4 S[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    S[m] = p.s_in ? *reinterpret_cast<const f32x4*>(p.s_in + sbase + (row0 + 4 * m + ri) * kN + 4 * c) : zero4();
  }
  const float4 r4 = widen4(p.r, unit * kN + 4 * c, F32), k4 = widen4(p.k, unit * kN + 4 * c, F32);
  const float lw = p.log_w[p.per_token ? unit : unit % p.H];
  const float w = expf(lw);
  float vm[4], yo = 0.f;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int64_t at = unit * kN + row0 + 4 * m + ri;
    vm[m] = F32 ? static_cast<const float*>(p.v)[at] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.v)[at] << 16);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    S[m][0] = fmaf(S[m][0], w, vm[m] * k4.x);
    S[m][1] = fmaf(S[m][1], w, vm[m] * k4.y);
    S[m][2] = fmaf(S[m][2], w, vm[m] * k4.z);
    S[m][3] = fmaf(S[m][3], w, vm[m] * k4.w);
    const float y = row16_sum(fmaf(S[m][3], r4.w, fmaf(S[m][2], r4.z, fmaf(S[m][1], r4.y, S[m][0] * r4.x))));
    yo = c == m ? y : yo;
    if (p.s_out) *reinterpret_cast<f32x4*>(p.s_out + sbase + (row0 + 4 * m + ri) * kN + 4 * c) = S[m];
  }
  if (c < 4) {
    const int64_t at = unit * kN + row0 + 4 * c + ri;
    if (F32)
      static_cast<float*>(p.y)[at] = yo;
    else
      static_cast<uint16_t*>(p.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)yo);
  }
}

}  // namespace

int64_t linattn_cus() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  cus = cached[dev].load(std::memory_order_relaxed);
  if (cus == 0 && hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && cus > 0)
    cached[dev].store(cus, std::memory_order_relaxed);
  return cus > 0 ? cus : 256;
}

hipError_t allow_lds(std::atomic<uint64_t>& granted, const void* fn, int bytes) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  return static_cast<hipError_t>(once_per_device(granted, dev, [&] {
    return static_cast<int>(hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
  }));
}

hipError_t launch_linattn(const LinattnCall& c) { return c.f32 ? launch_out<true>(c) : launch_out<false>(c); }

hipError_t launch_linattn_step(const LinattnCall& c) {
  StepParams p{c.r, c.log_w, c.k, c.v, c.s_in, c.y, c.s_out, (int32_t)c.H, c.per_token};
  void* args[] = {&p};
  const void* fn = c.f32 ? reinterpret_cast<const void*>(&linattn_step_kernel<true>)
                         : reinterpret_cast<const void*>(&linattn_step_kernel<false>);
  return hipLaunchKernel(fn, dim3((uint32_t)(c.B * c.H)), dim3(256), args, 0, c.stream);
}

}  // namespace rwkv7
