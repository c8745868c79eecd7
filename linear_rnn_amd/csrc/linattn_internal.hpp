// Host-side interface between the C ABI layer and the linear attention launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace rwkv7 {

// One validated call with work to do (B, H, T at least 1).
struct LinattnCall {
  const void* r;
  const float* log_w;
  const void* k;
  const void* v;
  const float* s_in;    // may be null (zeros)
  const int32_t* lens;  // may be null (every sequence has T tokens)
  void* y;              // forward
  float* s_out;         // forward; may be null
  int64_t B, T, H;
  bool f32;           // element type of r, k, v, y, dy, dr, dk, dv (else bfloat16)
  int32_t per_token;  // log_w is [B, T, H] (else [H])
  hipStream_t stream;
  // backward
  const void* dy;
  const float* ds_out;  // may be null (zeros)
  void* dr;
  float* dlog_w;  // in log_w's layout
  void* dk;
  void* dv;
  float* ds_in;  // may be null
};
hipError_t launch_linattn(const LinattnCall& c);
hipError_t launch_linattn_step(const LinattnCall& c);
hipError_t launch_linattn_backward(const LinattnCall& c);
hipError_t launch_linattn_zero(float* dlog_w, int64_t H, hipStream_t stream);

constexpr int64_t kLinattnStateBytes = 64 * 64 * 4;  // one state

// Every sequence in pieces of kPieceBlocks blocks, and the device memory for the states at their starts.
constexpr int64_t kPieceBlocks = 4;
inline int64_t linattn_blocks(int64_t T, int64_t block) { return (T + block - 1) / block; }
inline int64_t linattn_pieces(int64_t T, int64_t block) { return (linattn_blocks(T, block) + kPieceBlocks - 1) / kPieceBlocks; }
struct LinattnPieces {
  int64_t first, units;  // the heads (b H + h) of this launch; every array but the call's tensors begins with the first of them
  int64_t pieces;     // of a sequence, from its start on (backward: all of them)
  int32_t every;      // keep the state before every every-th piece
  float* states;      // [units][stride] states, stride at least pieces; the kept ones come first in a sequence's
  int64_t stride;
  float* decay;       // [units][stride]
  float* marks;       // may be null; [units][blocks] states
  float* mark_decay;  // [units][blocks]
  const float* start; // may be null (zeros); the state before the first piece (backward: the gradient behind the last), [units]
  float* end;         // may be null; the state behind the last piece (backward: the gradient before the first), [units] with
  int64_t end_stride; // that many states from one to the next
};
// Forward (from k, v): states <- the state before each every-th piece, and, if asked for, marks <- the sum of each
// piece before each of its blocks but the first. Backward (from r, dy; every is 1): the gradient behind each piece,
// and the sums behind each block but the last. Either may be null. `block`: tokens of a block, a multiple of 32.
hipError_t launch_linattn_states(const LinattnCall& c, int64_t block, const LinattnPieces* forward, const LinattnPieces* backward);
// Compute units of the current device (256 if it cannot be asked).
int64_t linattn_cus();
// Grants kernel `fn` `bytes` of LDS at launch on the current device; `granted` is the kernel's own.
hipError_t allow_lds(std::atomic<uint64_t>& granted, const void* fn, int bytes);

}  // namespace rwkv7
