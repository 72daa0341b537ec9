// k_rotary.hip -- norms of queries and keys for each head with the position
// rotation in the same pass, and its gradient.
//
// With n = x / sqrt(mean(x^2) + eps) * scale over a head's elements and (c, s)
// the cosine and sine of a row's position, a rotated pair (n1, n2) goes to
//   (n1 c - n2 s, n2 c + n1 s).
// Backward, with g the gradient turned back, (d1 c + d2 s, d2 c - d1 s), and
// xh = x / sqrt(..):  dscale = sum g xh,  dx = (g scale - xh mean(g scale xh)) / sqrt(..).
// Both are bound by memory: every element is read once and written once.
//
// A lane takes V pairs of a head (16 bytes of each of a pair's halves where
// sizes and alignment allow, else V = 1), LPH lanes a head, a wave 64 / LPH heads
// of a row at a time: what a lane loads of the table of cosines and sines, and of
// scale, then serves all heads that it takes of the row, which keeps the table
// (as many bytes a head as the head itself) out of the way.
#include "attn_ops.h"
#include "seq_device.h"

namespace rnnhip {
namespace {

// Where a lane's pairs lie in a head: two runs of V elements; for interleaved
// pairs one run of 2 V.
struct Place {
  int o1, o2;
  bool ok1, ok2, turned;
};
template <int V, bool IL>
__device__ __forceinline__ Place rotary_place(const RotaryArgs& a, int u) {
  Place p;
  const int turned = a.half / V;
  p.turned = u < turned;
  p.o1 = p.turned ? (IL ? u * 2 * V : u * V) : a.rotary + (u - turned) * 2 * V;
  p.o2 = p.turned && !IL ? a.half + u * V : p.o1 + V;
  p.ok1 = p.o1 < a.size;
  p.ok2 = p.ok1 && p.o2 < a.size;
  return p;
}

// The pairs (x, y) of a place.
template <typename T, int V, bool IL>
__device__ __forceinline__ void rotary_get(const T* h, const Place& p, float (&x)[V], float (&y)[V]) {
  float r[2 * V];
  Pack<T, V> k1 = {}, k2 = {};
  if (p.ok1) k1 = *reinterpret_cast<const Pack<T, V>*>(h + p.o1);
  if (p.ok2) k2 = *reinterpret_cast<const Pack<T, V>*>(h + p.o2);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r[i] = float(k1.v[i]);
    r[V + i] = float(k2.v[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = IL ? r[2 * i] : r[i];
    y[i] = IL ? r[2 * i + 1] : r[V + i];
  }
}
template <typename T, int V, bool IL>
__device__ __forceinline__ void rotary_put(T* h, const Place& p, const float (&x)[V], const float (&y)[V]) {
  Pack<T, V> k1, k2;
  T r[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r[IL ? 2 * i : i] = T(x[i]);
    r[IL ? 2 * i + 1 : V + i] = T(y[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    k1.v[i] = r[i];
    k2.v[i] = r[V + i];
  }
  if (p.ok1) *reinterpret_cast<Pack<T, V>*>(h + p.o1) = k1;
  if (p.ok2) *reinterpret_cast<Pack<T, V>*>(h + p.o2) = k2;
}

// The cosines and sines of a place at a position: 1 and 0 where there is no
// rotation, no numbers past the table.
template <int V>
__device__ __forceinline__ void rotary_angles(const RotaryArgs& a, int pos, int u, const Place& p, float (&c)[V], float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.f, s[i] = 0.f;
  if (!p.turned) return;
  if (pos >= a.table) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = s[i] = __builtin_nanf("");
    return;
  }
  const int64_t at = int64_t(pos) * a.half + u * V;
  const Pack<float, V> kc = *reinterpret_cast<const Pack<float, V>*>(a.cos + at);
  const Pack<float, V> ks = *reinterpret_cast<const Pack<float, V>*>(a.sin + at);
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = kc.v[i], s[i] = ks.v[i];
}

// A sum over the lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lph) {
  for (int m = 1; m < lph; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// M: units of V pairs that a lane takes of each head.
template <typename T, int V, bool IL, int M, bool BACK>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int u0 = lane & (a.lph - 1), per = 64 / a.lph, slot = lane / a.lph;
  const float each = 1.f / float(a.size);
  Place p[M];
  float scale[2][M][2][V];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    p[m] = rotary_place<V, IL>(a, u0 + m * a.lph);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (a.scale[k]) rotary_get<T, V, IL>(reinterpret_cast<const T*>(a.scale[k]), p[m], scale[k][m][0], scale[k][m][1]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) scale[k][m][0][i] = scale[k][m][1][i] = 1.f;
    }
  }
  float ds[2][M][2][V] = {};   // (BACK) the scales' gradients
  const int64_t all = a.rows * a.splits, step = int64_t(gridDim.x) * 4;
  for (int64_t id = int64_t(blockIdx.x) * 4 + w; id < all; id += step) {
    const int64_t row = id / a.splits;
    const int h0 = int(id - row * a.splits) * a.take;
    const int pos = a.positions ? __builtin_amdgcn_readfirstlane(a.positions[row]) : 0;
    const bool is = pos >= 0;   // (a row of a negative position is none)
    float c[M][V], s[M][V];
    if (is)
#pragma unroll
      for (int m = 0; m < M; ++m) rotary_angles<V>(a, pos, u0 + m * a.lph, p[m], c[m], s[m]);
    auto heads = [&](auto KEY) {
      constexpr int k = decltype(KEY)::value;
      const Rows &X = a.x[k], &O = a.out[k];
      if (!X.p || (!BACK && !O.p)) return;
      const int lo = max(h0, k ? a.heads[0] : 0) - (k ? a.heads[0] : 0), hi = min(h0 + a.take - (k ? a.heads[0] : 0), a.heads[k]);
      for (int hb = lo; hb < hi; hb += per) {
        const int h = hb + slot;
        const bool in = h < hi;
        const T* x = reinterpret_cast<const T*>(X.p) + row * X.rs + int64_t(in ? h : hb) * a.size;
        T* o = reinterpret_cast<T*>(O.p) + row * O.rs + int64_t(in ? h : hb) * a.size;
        float x1[M][V], x2[M][V], g1[M][V], g2[M][V];
        if (!is) {
          if (in && O.p)
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
              for (int i = 0; i < V; ++i) x1[m][i] = 0.f;
              rotary_put<T, V, IL>(o, p[m], x1[m], x1[m]);
            }
          continue;
        }
        float sum = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) rotary_get<T, V, IL>(x, p[m], x1[m], x2[m]);
        if constexpr (BACK) {
          const T* d = reinterpret_cast<const T*>(a.dy[k].p) + row * a.dy[k].rs + int64_t(in ? h : hb) * a.size;
#pragma unroll
          for (int m = 0; m < M; ++m) rotary_get<T, V, IL>(d, p[m], g1[m], g2[m]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < V; ++i) sum = __builtin_fmaf(x1[m][i], x1[m][i], __builtin_fmaf(x2[m][i], x2[m][i], sum));
        const float inv = 1.f / __builtin_sqrtf(__builtin_fmaf(head_sum(sum, a.lph), each, a.eps));
        if constexpr (!BACK) {
#pragma unroll
          for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float n1 = x1[m][i] * inv * scale[k][m][0][i], n2 = x2[m][i] * inv * scale[k][m][1][i];
              x1[m][i] = p[m].turned ? __builtin_fmaf(n1, c[m][i], -n2 * s[m][i]) : n1;
              x2[m][i] = p[m].turned ? __builtin_fmaf(n2, c[m][i], n1 * s[m][i]) : n2;
            }
            if (in) rotary_put<T, V, IL>(o, p[m], x1[m], x2[m]);
          }
        } else {
          sum = 0.f;
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float d1 = g1[m][i], d2 = g2[m][i];
              g1[m][i] = p[m].turned ? __builtin_fmaf(d1, c[m][i], d2 * s[m][i]) : d1;
              g2[m][i] = p[m].turned ? __builtin_fmaf(d2, c[m][i], -d1 * s[m][i]) : d2;
              x1[m][i] *= inv;
              x2[m][i] *= inv;
              if (in) {
                ds[k][m][0][i] = __builtin_fmaf(g1[m][i], x1[m][i], ds[k][m][0][i]);
                ds[k][m][1][i] = __builtin_fmaf(g2[m][i], x2[m][i], ds[k][m][1][i]);
              }
              g1[m][i] *= scale[k][m][0][i];
              g2[m][i] *= scale[k][m][1][i];
              sum = __builtin_fmaf(g1[m][i], x1[m][i], __builtin_fmaf(g2[m][i], x2[m][i], sum));
            }
          const float mean = head_sum(sum, a.lph) * each;
          if (in && O.p)
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
              for (int i = 0; i < V; ++i) {
                g1[m][i] = inv * __builtin_fmaf(-x1[m][i], mean, g1[m][i]);
                g2[m][i] = inv * __builtin_fmaf(-x2[m][i], mean, g2[m][i]);
              }
              rotary_put<T, V, IL>(o, p[m], g1[m], g2[m]);
            }
        }
      }
    };
    heads(std::integral_constant<int, 0>{});
    heads(std::integral_constant<int, 1>{});
  }
  if constexpr (BACK) {
    if (!a.part) return;
    // the heads of a wave, then the waves
    __shared__ float red[3][2][64 * M * 2 * V];
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.size;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float v = ds[k][m][j][i];
            for (int q = a.lph; q < 64; q <<= 1) v += __shfl_xor(v, q, 64);
            ds[k][m][j][i] = v;
            if (w && slot == 0) red[w - 1][k][((m * 2 + j) * V + i) * 64 + lane] = v;
          }
    __syncthreads();
    if (w || slot) return;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int at = ((m * 2 + j) * V + i) * 64 + lane, n = 2 * i + j;
            const float v = ((ds[k][m][j][i] + red[0][k][at]) + red[1][k][at]) + red[2][k][at];
            if (IL ? (n < V ? p[m].ok1 : p[m].ok2) : (j ? p[m].ok2 : p[m].ok1))
              part[k * a.size + (IL ? p[m].o1 + n : (j ? p[m].o2 : p[m].o1) + i)] = v;
          }
  }
}

template <typename T, int V, bool BACK>
hipError_t rotary_shape(const RotaryArgs& a, int64_t blocks, hipStream_t s) {
  if constexpr (V == 1) {
    if (a.units > 64) return a.interleaved ? go(rotary_kernel<T, 1, true, 4, BACK>, blocks, 256, a, s) : go(rotary_kernel<T, 1, false, 4, BACK>, blocks, 256, a, s);
  }
  return a.interleaved ? go(rotary_kernel<T, V, true, 1, BACK>, blocks, 256, a, s) : go(rotary_kernel<T, V, false, 1, BACK>, blocks, 256, a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? rotary_shape<float, 4, false>(a, blocks, s) : rotary_shape<float, 1, false>(a, blocks, s);
    case RNN_DTYPE_F16: return a.vec ? rotary_shape<f16_t, 8, false>(a, blocks, s) : rotary_shape<f16_t, 1, false>(a, blocks, s);
    default: return a.vec ? rotary_shape<bf16_t, 8, false>(a, blocks, s) : rotary_shape<bf16_t, 1, false>(a, blocks, s);
  }
}

hipError_t launch_rotary_backward(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? rotary_shape<float, 4, true>(a, blocks, s) : rotary_shape<float, 1, true>(a, blocks, s);
    case RNN_DTYPE_F16: return a.vec ? rotary_shape<f16_t, 8, true>(a, blocks, s) : rotary_shape<f16_t, 1, true>(a, blocks, s);
    default: return a.vec ? rotary_shape<bf16_t, 8, true>(a, blocks, s) : rotary_shape<bf16_t, 1, true>(a, blocks, s);
  }
}

}  // namespace rnnhip
