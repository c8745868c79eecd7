// Linear attention with a decay for each head: whole prompts and single tokens.
// The chunk algebra and its number formats are in linattn_ops.hpp.
#include "linattn_ops.hpp"
#include "rwkv7_wkv.h"
#include "linattn_internal.hpp"

namespace rwkv7 {
namespace {

using namespace linattn;

struct OutParams {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const float* first;  // [units][nseg] starts in the wave layout (nseg > 1), or the caller's state, or null
  void* y;
  float* s_out;        // may be null
  Seq seq;
  int32_t per_token;
  int32_t nseg;        // segments of a sequence
  int64_t seg_blocks;  // blocks of kBlk tokens in a segment
  int32_t pieces;      // state pieces in a segment: its start is that of piece seg * pieces
  int64_t piece_stride;  // pieces of a sequence in `first`
};

// One workgroup carries one segment of one head from its start state, kBlk = 128 tokens at a time:
// each wave takes 32 of them, forms what they add to the state, leaves it in LDS, and takes the
// state before its own tokens from the carried state and what the waves before it added.
template <bool F32>
__global__ __launch_bounds__(256) void linattn_out_kernel(OutParams p) {
  constexpr int NI = kIn<F32>, NO = F32 ? 3 : 2;
  __shared__ f32x4 added[kWaves - 1][16][64];
  __shared__ f32x4 carry[16][64];
  __shared__ double sums[kWaves][kSub];
  __shared__ float all[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t unit = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
  const int64_t b = unit / p.seq.H;
  const int32_t h = unit % p.seq.H;
  const int64_t T = p.seq.T, len = seq_len(p.seq, b);
  const uint32_t row_bytes = p.seq.H * kN * kEsz<F32>;
  const int64_t blk0 = seg * p.seg_blocks;
  const int64_t nblk = (T + kBlk - 1) / kBlk;
  const int64_t blk1 = blk0 + p.seg_blocks < nblk ? blk0 + p.seg_blocks : nblk;

#pragma unroll
  for (int m = 0; m < 4; ++m) {  // the start state: tiles 4m .. of the wave m
    const int tu = 4 * wave + m;
    f32x4 s = zero4();
    if (p.nseg > 1)
      s = reinterpret_cast<const f32x4*>(p.first)[((unit * p.piece_stride + (int64_t)seg * p.pieces) * 16 + tu) * 64 + lane];
    else if (p.first)
      s = *reinterpret_cast<const f32x4*>(p.first + (int64_t)unit * kN * kN + state_offset(tu >> 2, tu & 3, lane));
    carry[tu][lane] = s;
  }
  const Turn E = make_turn(lane);
  for (int64_t blk = blk0; blk < blk1; ++blk) {
    const int64_t t0 = blk * kBlk + wave * kSub;
    const __amdgpu_buffer_rsrc_t yb = token_buffer<kEsz<F32>>(p.y, p.seq, b, h, t0, T - t0, kSub);
    const uint32_t yoff = (lane & 15) * row_bytes + (lane >> 4) * 8 * kEsz<F32>;
    if (blk * kBlk >= len) {  // nothing but tokens behind the sequence's end: zeros
#pragma unroll
      for (int I = 0; I < 2; ++I)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          store_pair<F32>(yb, yoff + I * 16 * row_bytes + hh * 32 * kEsz<F32>, zero4(), zero4());
      continue;
    }
    Raw<F32> rr, rk, rv;
    load_raw<F32>(rk, token_buffer<kEsz<F32>>(p.k, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    load_raw<F32>(rv, token_buffer<kEsz<F32>>(p.v, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    load_raw<F32>(rr, token_buffer<kEsz<F32>>(p.r, p.seq, b, h, t0, len - t0, kSub), row_bytes, lane);
    const Decay d = make_decay(load_log_w(p.log_w, p.per_token, p.seq, b, h, t0, len, lane), sums[wave], lane);
    Op<NI> K[2][2], R[2][2];
#pragma unroll
    for (int J = 0; J < 2; ++J)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) K[J][hh] = natural<F32>(rk, J, hh), R[J][hh] = natural<F32>(rr, J, hh);
    // what the 32 tokens add to the state: tiles (t, u) of sum_j k_j (left_j v_j)^T
    Op<NI> Vt[4];
    f32x4 S[4][4];
    {
      Op<3> Vs[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const Op<NI> v0 = natural<F32>(rv, 0, u >> 1), v1 = natural<F32>(rv, 1, u >> 1);
        f32x4 a0 = turned(v0, E, u), a1 = turned(v1, E, u);
        if constexpr (F32)
          Vt[u] = turned_op(v0, v1, E, u);
        else
          Vt[u] = pack<NI>(a0, a1);
#pragma unroll
        for (int i = 0; i < 4; ++i) a0[i] *= d.row[0][i], a1[i] *= d.row[1][i];
        Vs[u] = pack<3>(a0, a1);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Op<NI> Kt = turned_op(K[0][t >> 1], K[1][t >> 1], E, t);
#pragma unroll
        for (int u = 0; u < 4; ++u) S[t][u] = mma(Kt, Vs[u], zero4());
      }
    }
    // the pairs inside the 32 tokens, as operands over the tokens j: column i
    Op<NO> P[2];
    {
      f32x4 a00 = zero4(), a01 = zero4(), a11 = zero4();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        a00 = mma(K[0][hh], R[0][hh], a00);
        a01 = mma(K[0][hh], R[1][hh], a01);
        a11 = mma(K[1][hh], R[1][hh], a11);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) a01[i] *= d.d01[i];
      P[0] = pack<NO>(masked_j(a00, d.d00, lane), zero4());
      P[1] = pack<NO>(a01, masked_j(a11, d.d11, lane));
    }
    if (wave < kWaves - 1) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) added[wave][4 * t + u][lane] = S[t][u];
    }
    if (lane == 0) all[wave] = d.all;
    __syncthreads();
    f32x4 next[4][4];
    const __amdgpu_buffer_rsrc_t* ybp = &yb;
#pragma unroll
    for (int uu = 0; uu < 2; ++uu) {  // value tiles 2uu, 2uu + 1: eight values of a token at a time
      f32x4 y[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int u = 2 * uu + e;
        f32x4 s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s[t] = carry[4 * t + u][lane];
          for (int w = 0; w < wave; ++w) s[t] = s[t] * all[w] + added[w][4 * t + u][lane];
          next[t][u] = s[t] * d.all + S[t][u];
        }
        const Op<NO> S0 = pack<NO>(s[0], s[1]), S1 = pack<NO>(s[2], s[3]);
#pragma unroll
        for (int I = 0; I < 2; ++I) {
          f32x4 o = mma(S0, R[I][0], zero4());
          o = mma(S1, R[I][1], o);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] *= d.col[I];
          y[I][e] = mma(Vt[u], P[I], o);
        }
      }
#pragma unroll
      for (int I = 0; I < 2; ++I)
        store_pair<F32>(*ybp, yoff + I * 16 * row_bytes + uu * 32 * kEsz<F32>, y[I][0], y[I][1]);
    }
    __syncthreads();  // every wave has read what was added and the carried state
    if (wave == kWaves - 1) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) carry[4 * t + u][lane] = next[t][u];
    }
  }
  __syncthreads();
  if (p.s_out && blk1 == nblk) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int tu = 4 * wave + m;
      *reinterpret_cast<f32x4*>(p.s_out + (int64_t)unit * kN * kN + state_offset(tu >> 2, tu & 3, lane)) = carry[tu][lane];
    }
  }
}

template <bool F32>
hipError_t launch_out(const LinattnCall& c) {
  OutParams p{};
  p.r = c.r, p.log_w = c.log_w, p.k = c.k, p.v = c.v, p.first = c.s_in, p.y = c.y, p.s_out = c.s_out;
  p.seq = Seq{c.T, (int32_t)c.H, c.lens};
  p.per_token = c.per_token;
  p.nseg = 1;
  p.seg_blocks = (c.T + kBlk - 1) / kBlk;
  void* args[] = {&p};
  return hipLaunchKernel(reinterpret_cast<const void*>(&linattn_out_kernel<F32>), dim3((uint32_t)(c.B * c.H)),
                         dim3(64 * kWaves), args, 0, c.stream);
}

// ---- single tokens. S is read and written once (32 KiB of a head's 32.5): 16 lanes hold a value
// row's 64 keys, a wave 16 rows, one workgroup a head. Row sums by the DPP butterfly.
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

template <bool F32, bool NT>
__global__ __launch_bounds__(256) void linattn_step_kernel(StepParams p) {
  const int lane = threadIdx.x & 63, c = lane & 15, ri = lane >> 4;
  const int64_t unit = blockIdx.x;
  const int row0 = 16 * (threadIdx.x >> 6);
  const int64_t sbase = unit * kN * kN;
  f32x4 S[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const f32x4* s = reinterpret_cast<const f32x4*>(p.s_in + sbase + (row0 + 4 * m + ri) * kN + 4 * c);
    S[m] = !p.s_in ? zero4() : NT ? __builtin_nontemporal_load(s) : *s;
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
    if (p.s_out) {
      f32x4* s = reinterpret_cast<f32x4*>(p.s_out + sbase + (row0 + 4 * m + ri) * kN + 4 * c);
      if (NT)
        __builtin_nontemporal_store(S[m], s);
      else
        *s = S[m];
    }
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

hipError_t launch_linattn(const LinattnCall& c) { return c.f32 ? launch_out<true>(c) : launch_out<false>(c); }

hipError_t launch_linattn_step(const LinattnCall& c) {
  StepParams p{c.r, c.log_w, c.k, c.v, c.s_in, c.y, c.s_out, (int32_t)c.H, c.per_token};
  void* args[] = {&p};
  const void* fn = c.f32 ? reinterpret_cast<const void*>(&linattn_step_kernel<true, false>)
                         : reinterpret_cast<const void*>(&linattn_step_kernel<false, false>);
  return hipLaunchKernel(fn, dim3((uint32_t)(c.B * c.H)), dim3(256), args, 0, c.stream);
}

}  // namespace rwkv7
