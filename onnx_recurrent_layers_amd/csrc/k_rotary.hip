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
//
// The grid is at most 512 workgroups, two a CU, that go on over the rows: scales
// are read and the scales' gradients summed once a workgroup, and more of them
// cost more than they hide (8192 rows of 32 heads of 128, f16, the same inputs again
// and again: forward 31.7 us with 512, 33.1 with 768, 34.9 with 1024, 40.1 with one
// for every four rows; gradient 50.3, 53.2, 62.1, - ; with 256 46.2 and 60.7).  Heads
// that lie on all lanes with every element turned take a kernel without conditions in
// the lanes (ALL; else the same call 35.8 and 72.5).  Over inputs that change the
// forward call takes 32.2 and the gradient's, bf16, 52.9: its kernel 48.5, the scales'
// sums, a launch of their own, the rest.  A copy of the same bytes (134 and 203 MB)
// takes 27 and 43.  Not kept: loads of the next heads under way while a wave
// takes these (33.2), and of the next row (32.1 to 46, the registers of 151).
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
template <int V, bool IL, bool ALL>
__device__ __forceinline__ Place rotary_place(const RotaryArgs& a, int u) {
  Place p;
  if constexpr (ALL) {
    p.turned = p.ok1 = p.ok2 = true;
    p.o1 = IL ? u * 2 * V : u * V;
    p.o2 = IL ? p.o1 + V : a.half + p.o1;
    return p;
  }
  const int turned = a.half / V;
  p.turned = u < turned;
  p.o1 = p.turned ? (IL ? u * 2 * V : u * V) : a.rotary + (u - turned) * 2 * V;
  p.o2 = p.turned && !IL ? a.half + u * V : p.o1 + V;
  p.ok1 = p.o1 < a.size;
  p.ok2 = p.ok1 && p.o2 < a.size;
  return p;
}

// A place's elements as they lie, and as pairs (x, y), zero where there are none.
template <typename T, int V>
struct Pairs {
  Pack<T, V> a, b;
};
template <typename T, int V>
__device__ __forceinline__ Pairs<T, V> rotary_load(const T* h, const Place& p) {
  Pairs<T, V> k = {};
  if (p.ok1) k.a = *reinterpret_cast<const Pack<T, V>*>(h + p.o1);
  if (p.ok2) k.b = *reinterpret_cast<const Pack<T, V>*>(h + p.o2);
  return k;
}
template <typename T, int V, bool IL>
__device__ __forceinline__ void rotary_pairs(const Pairs<T, V>& k, float (&x)[V], float (&y)[V]) {
  float r[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r[i] = float(k.a.v[i]);
    r[V + i] = float(k.b.v[i]);
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
// rotation, no numbers past the table.  (ALL: of the table's last position then,
// see rotary_past.)
template <int V, bool ALL>
__device__ __forceinline__ void rotary_angles(const RotaryArgs& a, int pos, int u, const Place& p, float (&c)[V], float (&s)[V]) {
  if constexpr (ALL) {
    pos = max(min(pos, a.table - 1), 0);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 1.f, s[i] = 0.f;
    if (!p.turned || pos < 0) return;
    if (pos >= a.table) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = s[i] = __builtin_nanf("");
      return;
    }
  }
  const int64_t at = int64_t(pos) * a.half + u * V;
  const Pack<float, V> kc = *reinterpret_cast<const Pack<float, V>*>(a.cos + at);
  const Pack<float, V> ks = *reinterpret_cast<const Pack<float, V>*>(a.sin + at);
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = kc.v[i], s[i] = ks.v[i];
}

// (ALL) What a position past the table makes of a head's factor: no number.
template <bool ALL>
__device__ __forceinline__ float rotary_past(const RotaryArgs& a, int pos, float inv) {
  return ALL && pos >= a.table ? __builtin_nanf("") : inv;
}

// A sum over the lanes of a head, a power of two of neighbours.
template <int CTRL>
__device__ __forceinline__ float lanes_swap(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float head_sum(float v, int lph) {
  const float one = v + lanes_swap<0xb1>(v);   // lane ^ 1
  v = lph > 1 ? one : v;
  const float two = v + lanes_swap<0x4e>(v);   // lane ^ 2
  v = lph > 2 ? two : v;
  const float four = v + lanes_swap<0x141>(v);   // the other half of eight lanes
  v = lph > 4 ? four : v;
  const float eight = v + lanes_swap<0x140>(v);   // the other half of sixteen
  v = lph > 8 ? eight : v;
  if (lph > 16) {
    v += __shfl_xor(v, 16, 64);
    if (lph > 32) v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// A lane's places and their scales of queries and keys.  M: units of V pairs that
// it takes of each head.
template <typename T, int V, bool IL, int M, bool ALL>
__device__ __forceinline__ void rotary_scales(const RotaryArgs& a, int u0, Place (&p)[M], float (&scale)[2][M][2][V]) {
#pragma unroll
  for (int m = 0; m < M; ++m) {
    p[m] = rotary_place<V, IL, ALL>(a, u0 + m * a.lph);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (a.scale[k]) rotary_pairs<T, V, IL>(rotary_load<T, V>(reinterpret_cast<const T*>(a.scale[k]), p[m]), scale[k][m][0], scale[k][m][1]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) scale[k][m][0][i] = scale[k][m][1][i] = 1.f;
    }
  }
}

// A wave's share of a row: its heads of the queries and of the keys.
struct Share {
  int64_t row;
  int lo[2], hi[2];
};
__device__ __forceinline__ Share share_at(const RotaryArgs& a, int64_t id) {
  Share t;
  t.row = id / a.splits;
  const int h0 = int(id - t.row * a.splits) * a.take;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int first = k ? a.heads[0] : 0;
    t.lo[k] = max(h0 - first, 0);
    t.hi[k] = a.x[k].p ? min(h0 + a.take - first, a.heads[k]) : 0;
  }
  return t;
}

// Zeros for the outputs of a row that is none.
template <typename T, int V, bool IL, int M>
__device__ __forceinline__ void rotary_none(T* o, const Place (&p)[M]) {
  const float z[V] = {};
#pragma unroll
  for (int m = 0; m < M; ++m) rotary_put<T, V, IL>(o, p[m], z, z);
}

template <typename T, int V, bool IL, int M, bool ALL>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int u0 = lane & (a.lph - 1), per = 64 / a.lph, slot = lane / a.lph;
  const float each = 1.f / float(a.size);
  Place p[M];
  float scale[2][M][2][V];
  rotary_scales<T, V, IL, M, ALL>(a, u0, p, scale);
  const int64_t all = a.rows * a.splits, step = int64_t(gridDim.x) * 4;
  int64_t id = int64_t(blockIdx.x) * 4 + w;
  if (id >= all) return;
  Share t = share_at(a, id);
  int asked = a.positions ? a.positions[t.row] : 0;
  for (; id < all; id += step) {
    const int pos = __builtin_amdgcn_readfirstlane(asked);
    const Share next = share_at(a, id + step);
    if (a.positions && id + step < all) asked = a.positions[next.row];
    float c[M][V], s[M][V];
#pragma unroll
    for (int m = 0; m < M; ++m) rotary_angles<V, ALL>(a, pos, u0 + m * a.lph, p[m], c[m], s[m]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int lo = t.lo[k]; lo < t.hi[k]; lo += per) {
        const bool in = lo + slot < t.hi[k];
        const int64_t h = min(lo + slot, t.hi[k] - 1);   // (past the last head: that one again, for nothing)
        const T* from = reinterpret_cast<const T*>(a.x[k].p) + t.row * a.x[k].rs + h * a.size;
        T* o = reinterpret_cast<T*>(a.out[k].p) + t.row * a.out[k].rs + h * a.size;
        if (pos < 0) {
          if (in) rotary_none<T, V, IL>(o, p);
          continue;
        }
        float x1[M][V], x2[M][V], sum = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) rotary_pairs<T, V, IL>(rotary_load<T, V>(from, p[m]), x1[m], x2[m]);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < V; ++i) sum = __builtin_fmaf(x1[m][i], x1[m][i], __builtin_fmaf(x2[m][i], x2[m][i], sum));
        const float inv = rotary_past<ALL>(a, pos, 1.f / __builtin_sqrtf(__builtin_fmaf(head_sum(sum, a.lph), each, a.eps)));
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
      }
    t = next;
  }
}

template <typename T, int V, bool IL, int M, bool ALL>
__global__ __launch_bounds__(256) void rotary_back_kernel(RotaryArgs a) {
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int u0 = lane & (a.lph - 1), per = 64 / a.lph, slot = lane / a.lph;
  const float each = 1.f / float(a.size);
  Place p[M];
  float scale[2][M][2][V];
  rotary_scales<T, V, IL, M, ALL>(a, u0, p, scale);
  float ds[2][M][2][V] = {};   // the scales' gradients
  const int64_t all = a.rows * a.splits, step = int64_t(gridDim.x) * 4;
  for (int64_t id = int64_t(blockIdx.x) * 4 + w; id < all; id += step) {
    const Share t = share_at(a, id);
    const int pos = a.positions ? __builtin_amdgcn_readfirstlane(a.positions[t.row]) : 0;
    float c[M][V], s[M][V];
#pragma unroll
    for (int m = 0; m < M; ++m) rotary_angles<V, ALL>(a, pos, u0 + m * a.lph, p[m], c[m], s[m]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int lo = t.lo[k]; lo < t.hi[k]; lo += per) {
        const bool in = lo + slot < t.hi[k];
        const int64_t h = min(lo + slot, t.hi[k] - 1);   // (past the last head: that one again, for nothing)
        const T* from = reinterpret_cast<const T*>(a.x[k].p) + t.row * a.x[k].rs + h * a.size;
        const T* grad = reinterpret_cast<const T*>(a.dy[k].p) + t.row * a.dy[k].rs + h * a.size;
        T* o = reinterpret_cast<T*>(a.out[k].p) + t.row * a.out[k].rs + h * a.size;
        if (pos < 0) {
          if (in && a.out[k].p) rotary_none<T, V, IL>(o, p);
          continue;
        }
        Pairs<T, V> x[M], d[M];
#pragma unroll
        for (int m = 0; m < M; ++m) x[m] = rotary_load<T, V>(from, p[m]), d[m] = rotary_load<T, V>(grad, p[m]);
        float x1[M][V], x2[M][V], g1[M][V], g2[M][V], sum = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          rotary_pairs<T, V, IL>(x[m], x1[m], x2[m]);
#pragma unroll
          for (int i = 0; i < V; ++i) sum = __builtin_fmaf(x1[m][i], x1[m][i], __builtin_fmaf(x2[m][i], x2[m][i], sum));
        }
        const float inv = rotary_past<ALL>(a, pos, 1.f / __builtin_sqrtf(__builtin_fmaf(head_sum(sum, a.lph), each, a.eps)));
        sum = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          rotary_pairs<T, V, IL>(d[m], g1[m], g2[m]);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float d1 = in ? g1[m][i] : 0.f, d2 = in ? g2[m][i] : 0.f;
            g1[m][i] = p[m].turned ? __builtin_fmaf(d1, c[m][i], d2 * s[m][i]) : d1;
            g2[m][i] = p[m].turned ? __builtin_fmaf(d2, c[m][i], -d1 * s[m][i]) : d2;
            x1[m][i] = in ? x1[m][i] * inv : 0.f;
            x2[m][i] = in ? x2[m][i] * inv : 0.f;
            ds[k][m][0][i] = __builtin_fmaf(g1[m][i], x1[m][i], ds[k][m][0][i]);
            ds[k][m][1][i] = __builtin_fmaf(g2[m][i], x2[m][i], ds[k][m][1][i]);
            g1[m][i] *= scale[k][m][0][i];
            g2[m][i] *= scale[k][m][1][i];
            sum = __builtin_fmaf(g1[m][i], x1[m][i], __builtin_fmaf(g2[m][i], x2[m][i], sum));
          }
        }
        const float mean = head_sum(sum, a.lph) * each;
        if (in && a.out[k].p)
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

// Whole heads on all lanes, every element turned, need no conditions in the lanes.
template <int V>
bool rotary_all(const RotaryArgs& a) {
  return V > 1 && a.rotary == a.size && a.units == a.lph && a.table > 0;
}

template <typename T, int V>
hipError_t rotary_shape(const RotaryArgs& a, int64_t blocks, hipStream_t s) {
  if constexpr (V == 1) {
    if (a.units > 64) return a.interleaved ? go(rotary_kernel<T, 1, true, 4, false>, blocks, 256, a, s) : go(rotary_kernel<T, 1, false, 4, false>, blocks, 256, a, s);
  } else if (rotary_all<V>(a)) {
    return a.interleaved ? go(rotary_kernel<T, V, true, 1, true>, blocks, 256, a, s) : go(rotary_kernel<T, V, false, 1, true>, blocks, 256, a, s);
  }
  return a.interleaved ? go(rotary_kernel<T, V, true, 1, false>, blocks, 256, a, s) : go(rotary_kernel<T, V, false, 1, false>, blocks, 256, a, s);
}

template <typename T, int V>
hipError_t rotary_back_shape(const RotaryArgs& a, int64_t blocks, hipStream_t s) {
  if constexpr (V == 1) {
    if (a.units > 64) return a.interleaved ? go(rotary_back_kernel<T, 1, true, 4, false>, blocks, 256, a, s) : go(rotary_back_kernel<T, 1, false, 4, false>, blocks, 256, a, s);
  } else if (rotary_all<V>(a)) {
    return a.interleaved ? go(rotary_back_kernel<T, V, true, 1, true>, blocks, 256, a, s) : go(rotary_back_kernel<T, V, false, 1, true>, blocks, 256, a, s);
  }
  return a.interleaved ? go(rotary_back_kernel<T, V, true, 1, false>, blocks, 256, a, s) : go(rotary_back_kernel<T, V, false, 1, false>, blocks, 256, a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? rotary_shape<float, 4>(a, blocks, s) : rotary_shape<float, 1>(a, blocks, s);
    case RNN_DTYPE_F16: return a.vec ? rotary_shape<f16_t, 8>(a, blocks, s) : rotary_shape<f16_t, 1>(a, blocks, s);
    default: return a.vec ? rotary_shape<bf16_t, 8>(a, blocks, s) : rotary_shape<bf16_t, 1>(a, blocks, s);
  }
}

hipError_t launch_rotary_backward(const RotaryArgs& a, int dtype, int64_t blocks, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? rotary_back_shape<float, 4>(a, blocks, s) : rotary_back_shape<float, 1>(a, blocks, s);
    case RNN_DTYPE_F16: return a.vec ? rotary_back_shape<f16_t, 8>(a, blocks, s) : rotary_back_shape<f16_t, 1>(a, blocks, s);
    default: return a.vec ? rotary_back_shape<bf16_t, 8>(a, blocks, s) : rotary_back_shape<bf16_t, 1>(a, blocks, s);
  }
}

}  // namespace rnnhip
