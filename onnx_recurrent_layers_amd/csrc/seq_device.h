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

template <typename T>
struct Elem;
template <>
struct Elem<float> { static constexpr int vec = 4; };
template <>
struct Elem<f16_t> { static constexpr int vec = 8; };
template <>
struct Elem<bf16_t> { static constexpr int vec = 8; };

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

// softplus(x) = max(x, 0) + log1p(e^-|x|), to about two units in the last
// place also where it is small (x far below 0, the usual place of a step
// size): e^-|x| from 2^x with the rounding of the argument made good, log1p(e)
// = 2 artanh(s), s = e / (2 + e) <= 1/3, by its odd series up to s^13 (the
// next term is below 2^-26 of the sum).  NaN passes.
__device__ __forceinline__ float softplus(float x) {
  float ax = x < 0.f ? -x : x;
  ax = ax > 120.f ? 120.f : ax;   // e^-120 is 0 in f32
  const float hi = ax * -kLog2e;
  const float lo = __builtin_fmaf(ax, -kLog2e, -hi) - ax * 1.925963033500512e-8f;   // log2(e) - f32(log2(e))
  float e = __builtin_amdgcn_exp2f(hi);
  e = __builtin_fmaf(e, lo * kLn2, e);
  const float d = 2.f + e;
  float s = e * __builtin_amdgcn_rcpf(d);
  s = __builtin_fmaf(__builtin_fmaf(-s, d, e), 0.5f, s);   // one correction of the quotient (1/d is within 1/3 and 1/2)
  const float t = s * s;
  float p = __builtin_fmaf(t, 1.f / 13.f, 1.f / 11.f);
  p = __builtin_fmaf(p, t, 1.f / 9.f);
  p = __builtin_fmaf(p, t, 1.f / 7.f);
  p = __builtin_fmaf(p, t, 1.f / 5.f);
  p = __builtin_fmaf(p, t, 1.f / 3.f);
  p = __builtin_fmaf(p * t, s, s);
  return (x > 0.f ? x : 0.f) + 2.f * p;
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
__device__ __forceinline__ float quad_sum(float v) {
  v += quad_x1(v);
  return v + quad_x2(v);
}
// Four sums over a group of four lanes at once: lane q gets that of a[q].
// Each exchange halves what is left, so three exchanges do for four sums.
__device__ __forceinline__ float quad_sum4(float a0, float a1, float a2, float a3, bool q1, bool q2) {
  const float r0 = (q1 ? a1 : a0) + quad_x1(q1 ? a0 : a1);
  const float r1 = (q1 ? a3 : a2) + quad_x1(q1 ? a2 : a3);
  return (q2 ? r1 : r0) + quad_x2(q2 ? r0 : r1);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace rnnhip
