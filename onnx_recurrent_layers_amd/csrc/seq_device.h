// seq_device.h -- device helpers of the state space operators and layer
// normalization: element types, rows and steps, the functions of the formulas,
// sums across lanes.  Internal.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "seq_ops.h"

namespace rnnhip {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

template <typename T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Pack { T v[V]; };

// Launch one kernel that takes its arguments as one struct; the launch's own
// status (not an error some earlier call left behind).
template <typename Args>
inline hipError_t go(void (*kernel)(Args), int64_t blocks, int threads, const Args& a, hipStream_t s) {
  if (blocks <= 0) return hipSuccess;
  void* p[] = {const_cast<Args*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(unsigned(blocks)), dim3(unsigned(threads)), p, 0, s);
}

__device__ __forceinline__ int geo_len(const SeqGeom& g, int b) {
  int L = g.lens ? g.lens[b] : g.S;
  L = L < 0 ? 0 : (L > g.S ? g.S : L);
  return __builtin_amdgcn_readfirstlane(L);
}

// Rows of batch row b in the order of its steps: step s < L is row
// base + s * step; past the row's length time runs on as stored (dead_row).
struct StepRows {
  int64_t base, step;
};
__device__ __forceinline__ StepRows step_rows(const SeqGeom& g, int b, int L) {
  StepRows r;
  r.step = g.layout ? 1 : g.B;
  r.base = g.layout ? int64_t(b) * g.S : b;
  if (g.reverse) {
    r.base += int64_t(L - 1) * r.step;
    r.step = -r.step;
  }
  return r;
}
__device__ __forceinline__ int64_t dead_row(const SeqGeom& g, int b, int t) {
  return g.layout ? int64_t(b) * g.S + t : int64_t(t) * g.B + b;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// sigmoid(x) = 1 / (1 + e^-x), from the hardware's 2^x and reciprocal.
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// softplus(x) = max(x, 0) + log1p(e^-|x|), to a few units in the last place (and
// |x|/2 of them from the rounding of 2^x's argument) also where it is small:
// log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, and artanh(s) = s + s t q(t)
// with t = s^2 and q of the third degree, fitted over t <= 1/9 for the least
// largest error (4.6e-9 of the sum; the odd series itself would take six terms
// for as much).  NaN passes.
__device__ __forceinline__ float softplus(float x) {
  const float e = __builtin_amdgcn_exp2f((x < 0.f ? x : -x) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float t = s * s;
  float q = __builtin_fmaf(t, 0.1401223093f, 0.1399957091f);
  q = __builtin_fmaf(q, t, 0.2001084983f);
  q = __builtin_fmaf(q, t, 0.3333320618f);
  const float w = __builtin_fmaf(q * t, s, s);
  return __builtin_fmaf(2.f, w, x > 0.f ? x : 0.f);
}

// The value that lane P of each group of four lanes holds.
template <int P>
__device__ __forceinline__ float quad_of(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), P * 0x55, 0xf, 0xf, true));
}
// lane ^ 1, lane ^ 2 within the group of four
__device__ __forceinline__ float quad_x1(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));
}
__device__ __forceinline__ float quad_x2(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, true));
}
// Four sums over a group of four lanes at once: lane q gets that of a[q].
// Each exchange halves what is left, so three exchanges do for four sums.
__device__ __forceinline__ float quad_sum4(float a0, float a1, float a2, float a3, bool q1, bool q2) {
  const float r0 = (q1 ? a1 : a0) + quad_x1(q1 ? a0 : a1);
  const float r1 = (q1 ? a3 : a2) + quad_x1(q1 ? a2 : a3);
  return (q2 ? r1 : r0) + quad_x2(q2 ? r0 : r1);
}

}  // namespace rnnhip
