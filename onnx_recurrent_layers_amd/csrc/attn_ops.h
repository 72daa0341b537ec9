// attn_ops.h -- arguments and launchers of linear attention and of the norms and
// rotations of its queries and keys, between their C ABI (attn_api.cpp) and
// their kernels.  Internal.
#pragma once

#include "seq_ops.h"

namespace rnnhip {

// A row tensor of heads: head h's elements begin (h / per) * size after the
// row's first.
struct HeadRows {
  char* p;
  int64_t rs;
  int32_t per;
};

// One walk of linear attention's recurrence over the steps of each row and head,
//   S_u = e^(g_u) S_(u-1) + in_scale * b_u v_u^T,   out_u = out_scale * a_u^T S_u.
// The operator itself has a, b, v = Q, K, V.  Its gradients are the same walk
// with the roles changed: dQ has dY, V, K; from the last step to the first,
// where the decay between two steps is that of the later one, dK has V, dY, Q
// and dV has K, Q, dY (what grows there is the state's gradient, scale and all).
struct AttnArgs {
  SeqGeom geo;
  int32_t back;            // from a row's last step to its first
  int32_t H, K, V;         // heads, size of a and b, size of v and out
  HeadRows a, b, v, out;
  int32_t out_f32;         // out holds f32 (a part of a sum over heads), else the tensor type
  float in_scale, out_scale;
  Rows G;                  // f32, the steps' log decays of each head (NULL: none)
  const float* decay;      // [H], added to every step's (NULL: none)
  // A state's element (k, v) is at k * sk + v * sv of its head's K * V.
  int32_t sk, sv;
  const float* init;       // [B][H] (NULL: zeros)
  // The time axis in pieces, walked side by side, each of so many steps: the
  // states that they begin with (before: those that they leave from zero ones),
  // [B][H][pieces], and their decays.  (One piece: from init, and none of these.)
  // `sub`: a walk begins from init and what the parts before its piece leave, `sub`
  // parts a piece, [B][H][pieces][sub].
  int32_t piece, pieces, sub;
  float *starts, *totals;
  float* fin;              // [B][H], or NULL; `back`: times the first step's decay
  // for the decays' gradient
  HeadRows dot;            // rows that each step's output, less its own v, is multiplied with
  float* dots;             // [slices][B][H][S], or NULL
  const float* other;      // [B][H] states that the last one is multiplied with (NULL: none)
  const float* others;     // of several pieces: [B][H][pieces], those of the pieces' ends
  float* ends;             // [slices][B][H][pieces], or NULL
};

// Up to three walks in one launch, walk k's workgroups from first[k] on.
struct AttnWalks {
  AttnArgs w[3];
  int32_t first[4];
};

// The states that pieces begin with, in their place: from those that they leave
// from a zero one.
struct AttnJoinArgs {
  int32_t pieces, back;
  int64_t heads, size;   // B * H, K * V
  float* starts;
  const float *totals, *init;
};

// The decays' gradient from what the walks left: dG_t is the sum over the steps
// i >= t of its piece of (rows_i - cols_i), and the product at the piece's end.
struct AttnDecayArgs {
  SeqGeom geo;
  int32_t H, slices, piece, pieces;
  const float *rows, *cols, *ends;   // ends: [slices][B][H][pieces]
  Rows G;
  const float* decay;
  Rows dG;
  float* part;                       // [B][pieces][H] sums over a piece's steps, or NULL
};

// out[i][row][g * K + k] = the sum over a group's heads of part[i][row][h][k], for
// n tensors, one or two.
struct HeadSumArgs {
  const float* part[2];
  int64_t rows;
  int32_t n, H, per, K;
  Rows out[2];
};

// Norms and rotations of a row's heads, queries [0] and keys [1].
struct RotaryArgs {
  int64_t rows;
  int32_t heads[2], size;
  int32_t rotary, half, table, interleaved;   // elements rotated, pairs, positions of the table
  float eps;
  Rows x[2], out[2], dy[2];   // out: the outputs, backward the gradients of x
  const char* scale[2];
  const float *cos, *sin;
  const int32_t* positions;
  float* part;                // backward: [workgroups][2][size], or NULL
  int32_t vec, units, lph;    // 16-byte accesses; pieces of a head, lanes that share them
  int32_t splits, take;       // waves of a row, heads that each takes
};

constexpr int kRotaryMaxSize = 512;
constexpr int64_t kRotaryBlocks = 512;   // workgroups of a launch at most
constexpr int kAttnMaxSize = 256;   // of a head's keys and values
constexpr int kAttnCols = 64;       // columns of v and out that a workgroup takes
constexpr int kAttnParts = 8;      // parts before a piece that a walk joins by itself
constexpr int kAttnSteps = 4, kAttnManySteps = 8;   // steps up to which a sequence is taken one by one, few or many

hipError_t launch_attn_steps(const AttnArgs& a, int dtype, hipStream_t s);
// (one definition a type: k_attn_f32.hip, k_attn_f16.hip, k_attn_bf16.hip)
hipError_t launch_attn_chunks_f32(const AttnArgs& a, bool local, hipStream_t s);
hipError_t launch_attn_walks_f32(const AttnArgs* w, int n, int K, hipStream_t s);   // (n up to 3, K the most of any)
hipError_t launch_attn_chunks_f16(const AttnArgs& a, bool local, hipStream_t s);
hipError_t launch_attn_walks_f16(const AttnArgs* w, int n, int K, hipStream_t s);   // (n up to 3, K the most of any)
hipError_t launch_attn_chunks_bf16(const AttnArgs& a, bool local, hipStream_t s);
hipError_t launch_attn_walks_bf16(const AttnArgs* w, int n, int K, hipStream_t s);   // (n up to 3, K the most of any)
hipError_t launch_attn_join(const AttnJoinArgs& a, hipStream_t s);
hipError_t launch_attn_decay(const AttnDecayArgs& a, hipStream_t s);
hipError_t launch_head_sum(const HeadSumArgs& a, int dtype, hipStream_t s);
hipError_t launch_rotary(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s);
hipError_t launch_rotary_backward(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s);

}  // namespace rnnhip
