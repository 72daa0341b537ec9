// k_scan_tokens.hip -- the selective scan over a few steps: single tokens with
// the state carried, bound by the state's read and write.
//
// Four lanes share a channel, NS states each in 16-byte pieces (state
// 4 (4 k + q) + j is piece k of lane q), so that a wave reads and writes whole
// lines of 16 channels' states at once; B and C come straight from their rows.
// Lane q of a channel prepares step 4k+q and shares it with the group through
// the DPP crossbar.  One launch, no scratch, no shared memory.  (64 rows by 2048
// channels by 16 states, one step: 8.2 us for 17.9 MB, of which the states' read
// and write are 16.8; the arithmetic is a small part.  A first version with
// states read an element a time took 12.1.  Up to kScanTokens = 4 steps, one
// for each lane of a group.)
#include "seq_device.h"

namespace rnnhip {
namespace {

// The place of a lane's state i among N: pieces of V.
template <int NS>
__device__ __forceinline__ int state_of(int q, int i) {
  constexpr int V = NS < 4 ? NS : 4;
  return ((i / V) * 4 + q) * V + i % V;
}

template <int NS>
__device__ __forceinline__ void get_state(const ScanArgs& a, const float* t, int64_t chan, int q, float (&v)[NS]) {
  constexpr int V = NS < 4 ? NS : 4;
  const float* p = t + chan * a.N;
  if (!t) {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = 0.f;
  } else if (a.vec_state) {
#pragma unroll
    for (int i = 0; i < NS; i += V) {
      const Pack<float, V> k = *reinterpret_cast<const Pack<float, V>*>(p + state_of<NS>(q, i));
#pragma unroll
      for (int j = 0; j < V; ++j) v[i + j] = k.v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = state_of<NS>(q, i) < a.N ? p[state_of<NS>(q, i)] : 0.f;
  }
}

template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_tokens_kernel(ScanArgs a) {
  constexpr int V = NS < 4 ? NS : 4;
  const int nb = a.G * a.cbg;
  const int cb = int(blockIdx.x) % nb, b = int(blockIdx.x) / nb;
  const int g = cb / a.cbg, in = (cb % a.cbg) * 64 + (int(threadIdx.x) >> 2), q = int(threadIdx.x) & 3;
  const bool ok = in < a.cpg, q1 = q & 1, q2 = q & 2;
  const int c = g * a.cpg + (ok ? in : a.cpg - 1);
  const int L = geo_len(a.geo, b);
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t cs = int64_t(b) * a.C + c;
  float h[NS], A[NS];
  get_state<NS>(a, a.init, cs, q, h);
  get_state<NS>(a, a.A, c, q, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
  const float bias = a.dbias ? a.dbias[c] : 0.f;
  const float skip = a.D ? a.D[c] : 0.f;
  for (int s = 0; s < L; s += 4) {
    const bool live = s + q < L;
    const int64_t row = r.base + (live ? s + q : L - 1) * r.step;
    float x = float((reinterpret_cast<const T*>(a.X.p) + c)[row * a.X.rs]);
    float d = float((reinterpret_cast<const T*>(a.delta.p) + c)[row * a.delta.rs]) + bias;
    float z = 0.f;
    if (a.have_z) z = float((reinterpret_cast<const T*>(a.Z.p) + c)[row * a.Z.rs]);
    if (a.softplus) d = softplus(d);
    const float u = d * x;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](int j, float dj, float uj) {
      const int64_t at = r.base + (s + j) * r.step;
      const T* Bp = reinterpret_cast<const T*>(a.Bm.p) + at * a.Bm.rs + int64_t(g) * a.N;
      const T* Cp = reinterpret_cast<const T*>(a.Cm.p) + at * a.Cm.rs + int64_t(g) * a.N;
      float v = 0.f, Bv[NS], Cv[NS];
      if (a.vec_state) {
#pragma unroll
        for (int i = 0; i < NS; i += V) {
          const Pack<T, V> kb = *reinterpret_cast<const Pack<T, V>*>(Bp + state_of<NS>(q, i));
          const Pack<T, V> kc = *reinterpret_cast<const Pack<T, V>*>(Cp + state_of<NS>(q, i));
#pragma unroll
          for (int j = 0; j < V; ++j) {
            Bv[i + j] = float(kb.v[j]);
            Cv[i + j] = float(kc.v[j]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int n = state_of<NS>(q, i);
          Bv[i] = n < a.N ? float(Bp[n]) : 0.f;
          Cv[i] = n < a.N ? float(Cp[n]) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(dj * A[i]), h[i], uj * Bv[i]);
        v = __builtin_fmaf(h[i], Cv[i], v);
      }
      return v;
    };
    acc[0] = step(0, quad_of<0>(d), quad_of<0>(u));
    if (s + 1 < L) acc[1] = step(1, quad_of<1>(d), quad_of<1>(u));
    if (s + 2 < L) acc[2] = step(2, quad_of<2>(d), quad_of<2>(u));
    if (s + 3 < L) acc[3] = step(3, quad_of<3>(d), quad_of<3>(u));
    float y = __builtin_fmaf(skip, x, quad_sum4(acc[0], acc[1], acc[2], acc[3], q1, q2));
    if (a.have_z) y *= z * logistic(z);
    if (live && ok && a.Y.p) (reinterpret_cast<T*>(a.Y.p) + c)[row * a.Y.rs] = T(y);
  }
  if (!ok) return;
  if (a.Y.p)
    for (int s = L + q; s < a.geo.S; s += 4) (reinterpret_cast<T*>(a.Y.p) + c)[dead_row(a.geo, b, s) * a.Y.rs] = T(0.f);
  if (a.fin) {
    float* p = a.fin + cs * a.N;
    if (a.vec_state) {
#pragma unroll
      for (int i = 0; i < NS; i += V) {
        Pack<float, V> k;
#pragma unroll
        for (int j = 0; j < V; ++j) k.v[j] = h[i + j];
        *reinterpret_cast<Pack<float, V>*>(p + state_of<NS>(q, i)) = k;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (state_of<NS>(q, i) < a.N) p[state_of<NS>(q, i)] = h[i];
    }
  }
}

template <typename T>
hipError_t tokens_t(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.G * a.cbg;
  const int ns = (a.N + 3) / 4;
  if (ns <= 1) return go(scan_tokens_kernel<T, 1>, blocks, 256, a, s);
  if (ns <= 2) return go(scan_tokens_kernel<T, 2>, blocks, 256, a, s);
  if (ns <= 4) return go(scan_tokens_kernel<T, 4>, blocks, 256, a, s);
  if (ns <= 8) return go(scan_tokens_kernel<T, 8>, blocks, 256, a, s);
  if (ns <= 16) return go(scan_tokens_kernel<T, 16>, blocks, 256, a, s);
  return go(scan_tokens_kernel<T, 32>, blocks, 256, a, s);
}

}  // namespace

hipError_t launch_scan_tokens(const ScanArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return tokens_t<float>(a, s);
    case RNN_DTYPE_F16: return tokens_t<f16_t>(a, s);
    default: return tokens_t<bf16_t>(a, s);
  }
}

}  // namespace rnnhip
