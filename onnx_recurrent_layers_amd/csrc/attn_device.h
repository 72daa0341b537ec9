// attn_device.h -- what linear attention's kernels share: a walk's steps and
// their rows, decays, states.  Internal.
#pragma once

#include "attn_ops.h"
#include "seq_device.h"

namespace rnnhip {

// A step's log decay: never above zero (a decay above one counts as one); what
// is below any that f32 tells from zero, infinity too, is one that it does not.
__device__ __forceinline__ float attn_log_decay(float g) {
  g = g > 0.f ? 0.f : g;
  return g < -1000.f ? -1000.f : g;   // (NaN passes)
}

// Steps lo to hi of batch row b, which has L, and head h, in a walk's order.
template <typename T>
struct AttnSteps {
  const AttnArgs& a;
  int h, L, lo, hi;
  StepRows r;
  float fixed;
  __device__ __forceinline__ AttnSteps(const AttnArgs& a, int b, int h, int L, int lo, int hi)
      : a(a), h(h), L(L), lo(lo), hi(hi), r(step_rows(a.geo, b, L)), fixed(a.decay ? a.decay[h] : 0.f) {}
  __device__ __forceinline__ int step(int u) const { return a.back ? hi - 1 - u : lo + u; }
  __device__ __forceinline__ int64_t row(int u) const { return r.base + step(u) * r.step; }
  __device__ __forceinline__ float raw_decay(int s) const {
    return reinterpret_cast<const float*>(a.G.p)[(r.base + s * r.step) * a.G.rs + h];
  }
  __device__ __forceinline__ float log_decay_at(int s) const { return attn_log_decay((a.G.p ? raw_decay(s) : 0.f) + fixed); }
  // From the step before in the walk's order: the later one's of the two, and
  // none before the last step of all.
  __device__ __forceinline__ float log_decay(int u) const {
    const int s = step(u) + (a.back ? 1 : 0);
    return s < L ? log_decay_at(s) : 0.f;
  }
  __device__ __forceinline__ float first_decay() const { return log_decay_at(0); }
  __device__ __forceinline__ float get(const HeadRows& t, int size, int64_t row, int c) const {
    return float(reinterpret_cast<const T*>(t.p)[row * t.rs + (h / t.per) * int64_t(size) + c]);
  }
  __device__ __forceinline__ void put(int64_t row, int c, float v) const {
    if (!a.out.p) return;
    const int64_t at = row * a.out.rs + (h / a.out.per) * int64_t(a.V) + c;
    if (a.out_f32) reinterpret_cast<float*>(a.out.p)[at] = v;
    else reinterpret_cast<T*>(a.out.p)[at] = T(v);
  }
};

// Four columns of a row of a head's state, zero where there is none.
template <bool VEC>
__device__ __forceinline__ void attn_get_state(const AttnArgs& a, const float* p, int64_t st, int k, int c, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.f;
  if (!p || k >= a.K || c >= a.V) return;
  if constexpr (VEC) {
    const float4 x = *reinterpret_cast<const float4*>(p + st + int64_t(k) * a.V + c);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < a.V) v[j] = p[st + int64_t(k) * a.sk + int64_t(c + j) * a.sv];
  }
}
template <bool VEC>
__device__ __forceinline__ void attn_put_state(const AttnArgs& a, float* p, int64_t st, int k, int c, const float (&v)[4], float by) {
  if (!p || k >= a.K || c >= a.V) return;
  if constexpr (VEC) {
    *reinterpret_cast<float4*>(p + st + int64_t(k) * a.V + c) = float4{v[0] * by, v[1] * by, v[2] * by, v[3] * by};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < a.V) p[st + int64_t(k) * a.sk + int64_t(c + j) * a.sv] = v[j] * by;
  }
}

}  // namespace rnnhip
