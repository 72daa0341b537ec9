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
  int32_t vec_state;         // states may be moved 16 bytes at a time (tokens)
  int32_t vec_rows;          // groups and rows of channels are whole aligned packs of four
  int32_t have_z;
  int32_t balance;           // rows in an order of their lengths (one chunk, at most 256 rows)
  Rows X, delta, Bm, Cm, Z, Y;
  const float *A, *D, *dbias, *init;
  float* fin;
  // scratch, f32; NP = N padded to nw waves' shares
  int32_t nw, np;            // waves of a workgroup, NP
  float* loc;     // [B][nchunk][NP][C]: a chunk's end state from a zero (first chunk: the initial) state
  float* sum;     // [B][nchunk][C]: a chunk's sum of step sizes
  float* first;   // [B][NP][C]: the initial state, kept apart for an update in place
  char* sink;     // [C] of the tensor type: what is stored for no step (any workgroup, never read)
  // backward
  Rows dY, dX, ddelta, dB, dC, dZ;
  const float* dfin;
  float* dinit;
  float *dA, *dD, *ddbias;
  float* ckpt;    // [B][nseg][NP][C]: the chunk-local state before each segment
  float* cum;     // [B][nseg][C]: the sum of step sizes from the chunk's start to the segment's
  float* gloc;    // [B][nchunk][NP][C]: a chunk's gradient at its start, from a zero one at its end
  float* pbc;     // [G*cbg][B][S][nw][dB: NP/nw, dC: NP/nw] of a workgroup's channels
  float* pA;      // [B*nchunk][NP][C]
  float* pD;      // [B*nchunk][2][C]: dD, ddelta_bias
  int32_t nseg;   // segments of a row (chunks begin on segment borders)
  int64_t sums0;  // first workgroup of a launch of the sums
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

// The threads of a row, and the shares of `v` values that each holds in
// registers (0: rows too long for that).  The least threads that hold the row.
// Many rows: a wave of up to 3 shares a lane (forward 4), since rows then need no
// meeting of waves and fewer lanes idle (16 bits, forward and backward: 65536
// rows of 1280 67 and 103 us, with a workgroup a row 104 and 179; 8192 of 1536
// 11.1 and 20.7, 13.3 and 25.5; 8192 of 2048 13.7 forward, 15.4; but backward,
// its registers full, 16384 of 2048 49, 46.8).  With few rows compute units
// would idle so (64 rows of 1024 f32: 8.9 us, 8.4).
struct NormRow {
  int threads, shares;
};
inline NormRow norm_row(int64_t size, int v, int64_t rows, bool backward) {
  const int64_t n = (size + v - 1) / v;
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  if (n <= 192 && rows >= 1024) return {64, 3};
  if (n <= 256 && rows >= 4096 && !backward) return {64, 4};
  if (n <= 256) return {256, 1};
  if (n <= 512) return {256, 2};
  if (n <= 1024) return {256, 4};
  if (v < 8 && n <= 2048) return {256, 8};
  return {256, 0};
}

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

// Steps of a tile of the scan: every wave of a workgroup prepares some.
constexpr int kScanTile = 16;
// Steps up to which the kernel for tokens takes a sequence.
constexpr int kScanTokens = 4;
// Waves of a workgroup and the states that each takes (a power of two): the
// split with the least padding.  The backward pass takes up to 16 states on
// eight waves, two each, since its registers hold 16 steps of them.
inline void scan_split(int64_t N, bool backward, int* nw, int* np) {
  static const struct { int upto, nw, ns; } split[] = {{8, 4, 2}, {16, 4, 4}, {24, 6, 4}, {32, 8, 4}, {64, 8, 8}, {128, 8, 16}};
  int i = 0;
  while (split[i].upto < N) ++i;
  *nw = split[i].nw;
  *np = split[i].nw * split[i].ns;
  if (backward && split[i].upto == 16) *nw = 8;
}
// Steps of a segment of the backward pass, from a wave's states: at most 64
// states and as many decays a lane.  (Its 256 registers hold them with all else
// up to 16 states in all, and nearly so at 32 and 64; see scan_grad_kernel.h.)
constexpr int scan_segment(int ns) { return ns <= 4 ? 16 : ns <= 8 ? 8 : 4; }

hipError_t launch_conv(const ConvArgs& a, int dtype, int vec, hipStream_t s);
hipError_t launch_conv_backward(const ConvArgs& a, int dtype, int vec, hipStream_t s);
hipError_t launch_scan_tokens(const ScanArgs& a, int dtype, hipStream_t s);
// (one definition a type: k_scan_f32.hip, k_scan_f16.hip, k_scan_bf16.hip)
hipError_t launch_scan_local_f32(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_local_f16(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_local_bf16(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_f32(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_f16(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bf16(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_backward_f32(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_backward_f16(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_backward_bf16(const ScanArgs& a, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_colsum(const ColSumArgs& a, hipStream_t s);

// From api.cpp: the thread's error message, "who: text".
int set_error_of(int code, const char* who, const char* text);

}  // namespace rnnhip
