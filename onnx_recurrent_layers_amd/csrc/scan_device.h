// scan_device.h -- what the selective scan's forward and backward kernels
// share: a workgroup's place, the lanes' shares of A and of states, tiles of B
// and C, the join of chunks.  Internal.
#pragma once

#include "seq_device.h"

namespace rnnhip {

template <int J>
struct IntC { static constexpr int value = J; };

// Workgroup i: channel block, then chunk, then batch row.  A lane past its
// group's channels works on the last one and stores nothing.
struct ScanPlace {
  int b, ch, g, cb, c;   // batch row, chunk, group, channel block of all groups, channel
  bool ok;
};
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a, int nchunk) {
  ScanPlace p;
  const int nb = a.G * a.cbg;
  const int blk = int(blockIdx.x);
  p.cb = blk % nb;
  const int rest = blk / nb;
  p.ch = rest % nchunk;
  p.b = rest / nchunk;
  p.g = p.cb / a.cbg;
  const int in = (p.cb % a.cbg) * 64 + (int(threadIdx.x) >> 2);
  p.ok = in < a.cpg;
  p.c = p.g * a.cpg + (p.ok ? in : a.cpg - 1);
  return p;
}

// NS floats that lie together and 4*NS bytes (at most 16) aligned.
template <int NS>
__device__ __forceinline__ void scan_get(const float* p, float (&v)[NS]) {
  constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
  for (int i = 0; i < NS; i += V) {
    const Pack<float, V> k = *reinterpret_cast<const Pack<float, V>*>(p + i);
#pragma unroll
    for (int j = 0; j < V; ++j) v[i + j] = k.v[j];
  }
}
template <int NS>
__device__ __forceinline__ void scan_put(float* p, const float (&v)[NS]) {
  constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
  for (int i = 0; i < NS; i += V) {
    Pack<float, V> k;
#pragma unroll
    for (int j = 0; j < V; ++j) k.v[j] = v[i + j];
    *reinterpret_cast<Pack<float, V>*>(p + i) = k;
  }
}

// Lane q's states [q*NS, q*NS + NS) of one channel of a caller's tensor
// [..][N]; states past N are 0 and stay 0.
template <int NS>
__device__ __forceinline__ void scan_load_state(const ScanArgs& a, const float* t, int64_t chan, int q, float (&v)[NS]) {
  if (!t) {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = 0.f;
  } else if (a.vec_state) {
    scan_get<NS>(t + chan * a.N + q * NS, v);
  } else {
    const float* p = t + chan * a.N;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = q * NS + i < a.N ? p[q * NS + i] : 0.f;
  }
}
template <int NS>
__device__ __forceinline__ void scan_store_state(const ScanArgs& a, float* t, int64_t chan, int q, const float (&v)[NS]) {
  if (a.vec_state) {
    scan_put<NS>(t + chan * a.N + q * NS, v);
  } else {
    float* p = t + chan * a.N;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (q * NS + i < a.N) p[q * NS + i] = v[i];
  }
}
// A of one channel, times log2(e): exp(d A) = 2^(d * this).
template <int NS>
__device__ __forceinline__ void scan_load_A(const ScanArgs& a, int c, int q, float (&A)[NS]) {
  scan_load_state<NS>(a, a.A, c, q, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
}

// A row of a tile in shared memory: state n's place, so that the four lanes'
// shares are read 16 bytes at a time from neighbouring places.
template <int NS>
__device__ __forceinline__ int tile_place(int n) {
  constexpr int V = NS < 4 ? NS : 4;
  const int q = n / NS, i = n % NS;
  return ((i / V) * 4 + q) * V + i % V;
}
template <int NS>
__device__ __forceinline__ void tile_get(const float* row, int q, float (&v)[NS]) {
  constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
  for (int i = 0; i < NS; i += V) {
    const Pack<float, V> k = *reinterpret_cast<const Pack<float, V>*>(row + ((i / V) * 4 + q) * V);
#pragma unroll
    for (int j = 0; j < V; ++j) v[i + j] = k.v[j];
  }
}

// A tile of TT steps of B (and C, COUNT = 2) on its way from memory to shared
// memory through the 256 threads' registers.  Steps past `send` and states
// past N are 0; nothing past them is read.
template <typename T, int NS, int TT, int COUNT>
struct BCTile {
  static constexpr int NP = 4 * NS, E = (TT * NP + 255) / 256;
  T v[COUNT][E];
  __device__ __forceinline__ void fetch(const ScanArgs& a, const StepRows& r, int g, int s, int send, int tid) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int e = tid + k * 256;
      const int st = s + e / NP, n = e % NP;
      const bool in = e < TT * NP && st < send && n < a.N;
      const int64_t row = r.base + st * r.step;
      v[0][k] = T(0.f);
      if (in) v[0][k] = reinterpret_cast<const T*>(a.Bm.p)[row * a.Bm.rs + int64_t(g) * a.N + n];
      if constexpr (COUNT > 1) {
        v[1][k] = T(0.f);
        if (in) v[1][k] = reinterpret_cast<const T*>(a.Cm.p)[row * a.Cm.rs + int64_t(g) * a.N + n];
      }
    }
  }
  __device__ __forceinline__ void put(float (*B)[NP], float (*C)[NP], int tid) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int e = tid + k * 256;
      if (E * 256 == TT * NP || e < TT * NP) {
        B[e / NP][tile_place<NS>(e % NP)] = float(v[0][k]);
        if constexpr (COUNT > 1) C[e / NP][tile_place<NS>(e % NP)] = float(v[1][k]);
      }
    }
  }
};

// The state at the start of chunk ch > 0 (live), from the end states of the
// chunks before it: h = decay_j h + loc_j, decay_j = 2^(A sum_j).
template <int NS>
__device__ __forceinline__ void scan_join(const ScanArgs& a, int b, int ch, int c, int q, const float (&A)[NS], float (&h)[NS]) {
  const int64_t at = int64_t(b) * a.nchunk * a.C + c;
  scan_get<NS>(a.loc + at * a.np + q * NS, h);
#pragma unroll 4
  for (int j = 1; j < ch; ++j) {
    float l[NS];
    const int64_t aj = at + int64_t(j) * a.C;
    scan_get<NS>(a.loc + aj * a.np + q * NS, l);
    const float sum = a.sum[aj];
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(A[i] * sum), h[i], l[i]);
  }
}

}  // namespace rnnhip
