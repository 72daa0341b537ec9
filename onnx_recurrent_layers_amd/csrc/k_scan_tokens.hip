// k_scan_tokens.hip -- the selective scan over a few steps: single tokens with
// the state carried, bound by the state's read and write.
//
// Four lanes share a channel, NS states each in 16-byte pieces (state
// 4 (4 k + q) + j is piece k of lane q), so that a wave reads and writes whole
// lines of 16 channels' states at once; B and C come straight from their rows.
// Lane q of a channel prepares step 4k+q and shares it with the group through
// the DPP crossbar.  One launch, no scratch, no shared memory.  (64 rows by 2048
// channels by 16 states, one step: 6.3 us for 17.9 MB, of which the states' read
// and write are 16.8; 512 rows 28 us with the call, 4.8 TB/s.  With loads that
// waited for those before them, behind branches on alignment and absent
// tensors, 8.2 and 42; with states read an element a time 12.1.  Up to
// kScanTokens = 4 steps, one for each lane of a group.)
#include "seq_device.h"

namespace rnnhip {
namespace {

// The place of a lane's state i among N: pieces of V.
template <int NS>
__device__ __forceinline__ int state_of(int q, int i) {
  constexpr int V = NS < 4 ? NS : 4;
  return ((i / V) * 4 + q) * V + i % V;
}

// A lane's NS elements of a row of N, as loaded.  VEC: whole aligned pieces,
// N = 4 NS; else one by one, those past N from the last one's place (dropped by
// `value`), so that no load waits behind a branch.
template <typename T, int NS, bool VEC>
struct Mine {
  static constexpr int V = NS < 4 ? NS : 4;
  Pack<T, V> k[NS / V];
  __device__ __forceinline__ void load(const T* p, int N, int q) {
#pragma unroll
    for (int i = 0; i < NS / V; ++i) {
      if constexpr (VEC) {
        k[i] = *reinterpret_cast<const Pack<T, V>*>(p + state_of<NS>(q, i * V));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) k[i].v[j] = p[min(state_of<NS>(q, i * V + j), N - 1)];
      }
    }
  }
  __device__ __forceinline__ float value(int i, int N, int q) const {
    const float v = float(k[i / V].v[i % V]);
    return VEC || state_of<NS>(q, i) < N ? v : 0.f;
  }
};

// Everything that the first step takes is asked for before anything is waited
// for: absent tensors give way to a place that is there.
template <typename T, int NS, bool VEC>
__global__ __launch_bounds__(256) void scan_tokens_kernel(ScanArgs a) {
  constexpr int V = NS < 4 ? NS : 4;
  const int nb = a.G * a.cbg;
  const int cb = int(blockIdx.x) % nb, b = int(blockIdx.x) / nb;
  const int g = cb / a.cbg, in = (cb % a.cbg) * 64 + (int(threadIdx.x) >> 2), q = int(threadIdx.x) & 3;
  const bool ok = in < a.cpg, q1 = q & 1, q2 = q & 2;
  const int c = g * a.cpg + (ok ? in : a.cpg - 1);
  const int64_t cs = int64_t(b) * a.C + c;
  Mine<float, NS, VEC> h0, A0;
  h0.load(a.init ? a.init + cs * a.N : a.A + int64_t(c) * a.N, a.N, q);
  A0.load(a.A + int64_t(c) * a.N, a.N, q);
  const float bias0 = (a.dbias ? a.dbias : a.A)[c], skip0 = (a.D ? a.D : a.A)[c];
  const int L = geo_len(a.geo, b);
  const StepRows r = step_rows(a.geo, b, L);
  float h[NS];
  if (L > 0) {   // (uniform)
    // lane q prepares step q
    const bool live = q < L;
    const int64_t row = r.base + min(q, L - 1) * r.step;
    const T x0 = (reinterpret_cast<const T*>(a.X.p) + c)[row * a.X.rs];
    const T d0 = (reinterpret_cast<const T*>(a.delta.p) + c)[row * a.delta.rs];
    const Rows& Zr = a.have_z ? a.Z : a.X;
    const T z0 = (reinterpret_cast<const T*>(Zr.p) + c)[row * Zr.rs];
    Mine<T, NS, VEC> B, C;
    auto weights = [&](int j) {
      const int64_t at = r.base + j * r.step;
      B.load(reinterpret_cast<const T*>(a.Bm.p) + at * a.Bm.rs + int64_t(g) * a.N, a.N, q);
      C.load(reinterpret_cast<const T*>(a.Cm.p) + at * a.Cm.rs + int64_t(g) * a.N, a.N, q);
    };
    weights(0);
    __builtin_amdgcn_sched_barrier(0);
    float A[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      A[i] = A0.value(i, a.N, q) * kLog2e;
      h[i] = a.init ? h0.value(i, a.N, q) : 0.f;
    }
    const float x = float(x0), u0 = float(d0) + (a.dbias ? bias0 : 0.f);
    const float d = a.softplus ? softplus(u0) : u0;
    const float u = d * x;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](float dj, float uj) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float next = __builtin_fmaf(__builtin_amdgcn_exp2f(dj * A[i]), h[i], uj * B.value(i, a.N, q));
        h[i] = VEC || state_of<NS>(q, i) < a.N ? next : 0.f;   // (0 times an infinite step is not 0)
        v = __builtin_fmaf(h[i], C.value(i, a.N, q), v);
      }
      return v;
    };
    acc[0] = step(quad_of<0>(d), quad_of<0>(u));
    if (L > 1) {
      weights(1);
      acc[1] = step(quad_of<1>(d), quad_of<1>(u));
    }
    if (L > 2) {
      weights(2);
      acc[2] = step(quad_of<2>(d), quad_of<2>(u));
    }
    if (L > 3) {
      weights(3);
      acc[3] = step(quad_of<3>(d), quad_of<3>(u));
    }
    float y = __builtin_fmaf(a.D ? skip0 : 0.f, x, quad_sum4(acc[0], acc[1], acc[2], acc[3], q1, q2));
    if (a.have_z) {
      const float z = float(z0);
      y *= z * logistic(z);
    }
    if (live && ok && a.Y.p) (reinterpret_cast<T*>(a.Y.p) + c)[row * a.Y.rs] = T(y);
  } else {
    float none = 0.f;
    asm volatile("" : "+v"(none));   // (else the choice is made for both ways at once, before the loads above)
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = a.init ? h0.value(i, a.N, q) : none;
  }
  if (!ok) return;
  // (at most kScanTokens = 4 steps: one a lane of the group)
  if (a.Y.p && q >= L && q < a.geo.S) (reinterpret_cast<T*>(a.Y.p) + c)[dead_row(a.geo, b, q) * a.Y.rs] = T(0.f);
  if (a.fin) {
    float* p = a.fin + cs * a.N;
#pragma unroll
    for (int i = 0; i < NS; i += V) {
      if constexpr (VEC) {
        Pack<float, V> k;
#pragma unroll
        for (int j = 0; j < V; ++j) k.v[j] = h[i + j];
        *reinterpret_cast<Pack<float, V>*>(p + state_of<NS>(q, i)) = k;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (state_of<NS>(q, i + j) < a.N) p[state_of<NS>(q, i + j)] = h[i + j];
      }
    }
  }
}

template <typename T, int NS>
hipError_t tokens_n(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.G * a.cbg;
  return a.vec_state ? go(scan_tokens_kernel<T, NS, true>, blocks, 256, a, s) : go(scan_tokens_kernel<T, NS, false>, blocks, 256, a, s);
}

template <typename T>
hipError_t tokens_t(const ScanArgs& a, hipStream_t s) {
  const int ns = (a.N + 3) / 4;
  if (ns <= 1) return tokens_n<T, 1>(a, s);
  if (ns <= 2) return tokens_n<T, 2>(a, s);
  if (ns <= 4) return tokens_n<T, 4>(a, s);
  if (ns <= 8) return tokens_n<T, 8>(a, s);
  if (ns <= 16) return tokens_n<T, 16>(a, s);
  return tokens_n<T, 32>(a, s);
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
