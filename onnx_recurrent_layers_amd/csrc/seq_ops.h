// seq_ops.h -- arguments and launchers of the state space operators (short
// causal convolution, selective scan) and of layer normalization, between
// their C ABI (seq_api.cpp) and their kernels.  Internal.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "rnn.h"

namespace rnnhip {

// A row tensor: its first element and the elements from one row to the next.
struct Rows {
  char* p;
  int64_t rs;
};

// Which rows a batch row's steps are: rows t*B + b (layout 0) or b*S + t.
struct SeqGeom {
  int32_t S, B, layout, reverse;
  const int32_t* lens;   // NULL: every row takes S steps
};

struct ConvArgs {
  SeqGeom geo;
  int32_t C, K, silu;
  Rows X, Y, dY, dX;
  const char *W, *bias, *init, *dfin;
  char *fin, *dinit;
  float* part;        // backward: partial weight gradients, [parts][(K+1)*C]
  int32_t tile;       // steps a thread walks
  int32_t ntb, ncb;   // workgroups along time and along channels
  int32_t tx;         // threads of a workgroup along channels
};

struct ScanArgs {
  SeqGeom geo;
  int32_t C, N, G, softplus;
  int32_t cpg, cbg;          // channels of a group, workgroups along them
  int32_t chunk, nchunk;     // steps of a chunk of the time axis, chunks
  int32_t vec_state;         // state rows may be moved 16 bytes at a time
  int32_t have_z;
  Rows X, delta, Bm, Cm, Z, Y;
  const float *A, *D, *dbias, *init;
  float* fin;
  // scratch, f32; NP = N padded to four lanes' shares, [c][NP] channel-major
  float* loc;     // [B][nchunk][C][NP]: a chunk's end state from a zero (first chunk: the initial) state
  float* sum;     // [B][nchunk][C]: a chunk's sum of step sizes
  float* first;   // [B][C][NP]: the initial state, kept apart for an update in place
  // backward
  Rows dY, dX, ddelta, dB, dC, dZ;
  const float* dfin;
  float* dinit;
  float *dA, *dD, *ddbias;
  float* ckpt;    // [B][nseg][C][NP]: the chunk-local state before each segment
  float* cum;     // [B][nseg][C]: the sum of step sizes from the chunk's start to the segment's
  float* gloc;    // [B][nchunk][C][NP]: a chunk's gradient at its start, from a zero one at its end
  float* pbc;     // [G*cbg][B][S][2][NP]: dB and dC of a workgroup's channels
  float* pA;      // [B*nchunk][C][NP]
  float* pD;      // [B*nchunk][2][C]: dD, ddelta_bias
  int32_t nseg;   // segments of a row (chunks begin on segment borders)
  int32_t np;
};

struct NormArgs {
  int64_t rows;
  int32_t size;
  float eps;
  Rows X, Y, dY, dX;
  const char *scale, *shift;
  float *mean, *inv;
  float* part;        // backward: [parts][2][size]
  int32_t parts;
  int32_t vec;        // 16-byte accesses
};

// Column sums of part[P][cols] in a fixed order, f32.  Column j of a block of
// (K+1)*C columns [k][c] goes to out[c*K + k] (k < K) or out2[c].
struct ColSumArgs {
  const float* part;
  int32_t P;
  int64_t cols;
  float *out, *out2;
  int32_t C, K;
};

constexpr int kScanMaxState = 128;

// States a lane holds (four lanes share a channel), from the state size.
inline int scan_lane_states(int64_t N) {
  int ns = 1;
  while (4 * ns < N) ns *= 2;
  return ns;
}
// Steps of a segment of the backward pass: what a lane's registers hold of
// states and decays (64 of each where a segment may be as short as four).
inline int scan_segment(int ns) { return ns <= 4 ? 16 : ns == 8 ? 8 : 4; }
// Steps of a tile of B and C in shared memory.
constexpr int scan_tile(int ns) { return ns <= 8 ? 32 : 16; }

hipError_t launch_conv(const ConvArgs& a, int dtype, int vec, hipStream_t s);
hipError_t launch_conv_backward(const ConvArgs& a, int dtype, int vec, hipStream_t s);
hipError_t launch_scan_local(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_colsum(const ColSumArgs& a, hipStream_t s);

// From api.cpp: the thread's error message, "who: text".
int set_error_of(int code, const char* who, const char* text);

}  // namespace rnnhip
