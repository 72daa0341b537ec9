// k_norm.hip -- layer normalization and its gradient, and the column sums in
// which the gradients of weights end.
//
// Forward: a row is read once into registers; the mean, then the squares of
// what is left of it (the variance of a row far from zero keeps its digits
// so), then the outputs.  Backward: with xh = (x - Mean) InvStdDev, g = dY Scale,
//   dX = InvStdDev (g - mean(g) - xh mean(g xh)),  dScale = sum dY xh,  dB = sum dY;
// a workgroup walks several rows and keeps its columns' dScale and dB in
// registers, so that the partial sums written are few against the rows read.
// Both are bound by memory.
//
// A row is taken by W threads (a part of a wave, or a workgroup), V
// neighbouring values a time (16 bytes where rows and stride allow), M times;
// rows too long for registers are read again for each use.  Rows that are not
// whole 16-byte pieces go one value an access (8192 rows of 1290, 16 bits: 23 us,
// of 1288 11), and above 2048 of them count as too long.  (8192 rows of 2048, 16
// bits, the whole call: forward 12.8 us for 67 MB, 5.2 TB/s, a copy of 32 MiB
// taking 10.1; gradient 27.6 for 101 MB, of which the sums of 512 partials are
// 4.6, and 1024 partials took as long.  2048 rows of 8192, gradient: f32 76 us
// for 201 MB, 16 bits 40 for 101, with 66 and 32 registers spilled.  64 rows of
// 1024, f32: 3.2 us the kernel.)
#include "seq_device.h"

namespace rnnhip {
namespace {

// Sums of N values over the W threads of a row; all threads get them.  Calls
// one after another take two places in turn: whoever writes a place again has
// passed the barrier of the call between, after which all had read it.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[16]) {
  constexpr int M = W < 64 ? W : 64;
#pragma unroll
  for (int m = M / 2; m >= 1; m >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], m, 64);
  if constexpr (W > 64) {
    const int w = int(threadIdx.x) >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) lds[n][w] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < W / 64; ++k) t += lds[n][k];
      v[n] = t;
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void get(const T* p, float (&v)[V]) {
  const Pack<T, V> k = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = float(k.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const float (&v)[V]) {
  Pack<T, V> k;
#pragma unroll
  for (int i = 0; i < V; ++i) k.v[i] = T(v[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = k;
}

// M = 0: the row is read three times.
template <typename T, int W, int V, int M>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  __shared__ float lds[2][1][16];
  const int64_t row = int64_t(blockIdx.x) * (256 / W) + int(threadIdx.x) / W;
  const int t = int(threadIdx.x) % W;
  const bool in = row < a.rows;   // (uniform where a row takes the whole workgroup)
  const int64_t at = in ? row : a.rows - 1;
  const T* X = reinterpret_cast<const T*>(a.X.p) + at * a.X.rs;
  T* Y = reinterpret_cast<T*>(a.Y.p) + at * a.Y.rs;
  const T* scale = reinterpret_cast<const T*>(a.scale);
  const T* shift = reinterpret_cast<const T*>(a.shift);
  const float per = 1.f / float(a.size);
  constexpr int R = M > 0 ? M : 1;
  float x[R][V];
  float v[1] = {0.f};
  if constexpr (M > 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int c = (m * W + t) * V;
      if (c < a.size) get<T, V>(X + c, x[m]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) x[m][i] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[0] += x[m][i];
    }
  } else {
    for (int c = t * V; c < a.size; c += W * V) {
      get<T, V>(X + c, x[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) v[0] += x[0][i];
    }
  }
  row_sums<W, 1>(v, lds[0]);
  const float mean = v[0] * per;
  v[0] = 0.f;
  if constexpr (M > 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const bool is = (m * W + t) * V < a.size;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[m][i] -= mean;
        v[0] = __builtin_fmaf(is ? x[m][i] : 0.f, x[m][i], v[0]);
      }
    }
  } else {
    for (int c = t * V; c < a.size; c += W * V) {
      get<T, V>(X + c, x[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) v[0] = __builtin_fmaf(x[0][i] - mean, x[0][i] - mean, v[0]);
    }
  }
  row_sums<W, 1>(v, lds[1]);
  const float inv = 1.f / __builtin_sqrtf(__builtin_fmaf(v[0], per, a.eps));
  if (!in) return;
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.inv) a.inv[row] = inv;
  }
  if (!a.Y.p) return;
  auto out = [&](int c, const float (&d)[V]) {
    float s[V], h[V], y[V];
    get<T, V>(scale + c, s);
    if (shift) get<T, V>(shift + c, h);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __builtin_fmaf(d[i] * inv, s[i], shift ? h[i] : 0.f);
    put<T, V>(Y + c, y);
  };
  if constexpr (M > 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int c = (m * W + t) * V;
      if (c < a.size) out(c, x[m]);
    }
  } else {
    for (int c = t * V; c < a.size; c += W * V) {
      get<T, V>(X + c, x[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) x[0][i] -= mean;
      out(c, x[0]);
    }
  }
}

// Workgroup i takes rows i*RB + r, i + parts ... : row slots (256 / W rows a
// time) in steps of the grid.  M = 0: long rows; dX here, dScale and dB by
// norm_columns_kernel.
template <typename T, int W, int V, int M>
__global__ __launch_bounds__(256, 2) void norm_backward_kernel(NormArgs a) {
  __shared__ float lds[2][2][16];
  constexpr int RB = 256 / W;
  constexpr int R = M > 0 ? M : 1;
  const int t = int(threadIdx.x) % W, slot = int(threadIdx.x) / W;
  const T* scale = reinterpret_cast<const T*>(a.scale);
  const float per = 1.f / float(a.size);
  float ds[R][V] = {}, db[R][V] = {}, sc[R][V] = {};
  if constexpr (M > 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int c = (m * W + t) * V;
      if (c < a.size) get<T, V>(scale + c, sc[m]);
    }
  }
  // the next rows' values are under way while these are summed
  const int64_t by = int64_t(gridDim.x) * RB;
  Pack<T, V> px[R], pg[R];
  float pm = 0.f, pi = 0.f;
  auto fetch = [&](int64_t row) {
    const int64_t at = row < a.rows ? row : a.rows - 1;
    const T* X = reinterpret_cast<const T*>(a.X.p) + at * a.X.rs;
    const T* G = reinterpret_cast<const T*>(a.dY.p) + at * a.dY.rs;
#pragma unroll
    for (int m = 0; m < R; ++m) {
      const int c = min((m * W + t) * V, a.size - V);
      px[m] = *reinterpret_cast<const Pack<T, V>*>(X + c);
      pg[m] = *reinterpret_cast<const Pack<T, V>*>(G + c);
    }
    pm = a.mean[at];
    pi = a.inv[at];
  };
  if (M > 0 && int64_t(blockIdx.x) * RB < a.rows) fetch(int64_t(blockIdx.x) * RB + slot);
  int place = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * RB; r0 < a.rows; r0 += by, place ^= 1) {
    const int64_t row = r0 + slot;
    const bool in = row < a.rows;
    const int64_t at = in ? row : a.rows - 1;
    T* D = reinterpret_cast<T*>(a.dX.p) + at * a.dX.rs;
    float v[2] = {0.f, 0.f};
    if constexpr (M > 0) {
      float xh[M][V], g[M][V];
      const float mean = pm, inv = pi;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const bool is = in && (m * W + t) * V < a.size;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xh[m][i] = is ? (float(px[m].v[i]) - mean) * inv : 0.f;
          const float dy = is ? float(pg[m].v[i]) : 0.f;
          ds[m][i] = __builtin_fmaf(dy, xh[m][i], ds[m][i]);
          db[m][i] += dy;
          g[m][i] = dy * sc[m][i];
          v[0] += g[m][i];
          v[1] = __builtin_fmaf(g[m][i], xh[m][i], v[1]);
        }
      }
      if (r0 + by < a.rows) fetch(row + by);   // uniform
      if (a.dX.p) {
        row_sums<W, 2>(v, lds[place]);
        const float m0 = v[0] * per, m1 = v[1] * per;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int c = (m * W + t) * V;
          if (in && c < a.size) {
            float d[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = inv * (g[m][i] - __builtin_fmaf(xh[m][i], m1, m0));
            put<T, V>(D + c, d);
          }
        }
      }
    } else if (a.dX.p) {
      const T* X = reinterpret_cast<const T*>(a.X.p) + at * a.X.rs;
      const T* G = reinterpret_cast<const T*>(a.dY.p) + at * a.dY.rs;
      const float mean = a.mean[at], inv = a.inv[at];
      for (int c = t * V; c < a.size; c += W * V) {
        float x[V], g[V], s[V];
        get<T, V>(X + c, x);
        get<T, V>(G + c, g);
        get<T, V>(scale + c, s);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float gs = g[i] * s[i];
          v[0] += gs;
          v[1] = __builtin_fmaf(gs, (x[i] - mean) * inv, v[1]);
        }
      }
      row_sums<W, 2>(v, lds[place]);
      const float m0 = v[0] * per, m1 = v[1] * per;
      for (int c = t * V; c < a.size; c += W * V) {
        float x[V], g[V], s[V];
        get<T, V>(X + c, x);
        get<T, V>(G + c, g);
        get<T, V>(scale + c, s);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = inv * (g[i] * s[i] - __builtin_fmaf((x[i] - mean) * inv, m1, m0));
        put<T, V>(D + c, x);
      }
    }
  }
  if (M == 0 || !a.part) return;
  // the row slots' partials, then one of the workgroup
  __shared__ float sum[RB > 1 ? (RB - 1) * W * V : 1];
  float* part = a.part + int64_t(blockIdx.x) * 2 * a.size;
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float (&v)[V] = w ? db[m] : ds[m];
      if constexpr (RB > 1) {
        __syncthreads();
        if (slot > 0)
#pragma unroll
          for (int i = 0; i < V; ++i) sum[((slot - 1) * W + t) * V + i] = v[i];
        __syncthreads();
        if (slot == 0)
          for (int k = 0; k < RB - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += sum[(k * W + t) * V + i];
      }
      const int c = (m * W + t) * V;
      if (slot == 0 && c < a.size)
#pragma unroll
        for (int i = 0; i < V; ++i) part[int64_t(w) * a.size + c + i] = v[i];
    }
}

// Long rows: dScale and dB of 64 columns over a share of the rows.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs a) {
  __shared__ float red[2][3][64];
  const int ncb = (a.size + 63) / 64;
  const int cb = int(blockIdx.x) % ncb, pt = int(blockIdx.x) / ncb;
  const int l = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const int c = cb * 64 + l;
  float ds = 0.f, db = 0.f;
  if (c < a.size) {
    for (int64_t row = int64_t(pt) * 4 + w; row < a.rows; row += int64_t(a.parts) * 4) {
      const float dy = float((reinterpret_cast<const T*>(a.dY.p) + row * a.dY.rs)[c]);
      const float x = float((reinterpret_cast<const T*>(a.X.p) + row * a.X.rs)[c]);
      ds = __builtin_fmaf(dy, (x - a.mean[row]) * a.inv[row], ds);
      db += dy;
    }
  }
  if (w) {
    red[0][w - 1][l] = ds;
    red[1][w - 1][l] = db;
  }
  __syncthreads();
  if (w || c >= a.size) return;
  float* part = a.part + int64_t(pt) * 2 * a.size;
  part[c] = ((ds + red[0][0][l]) + red[0][1][l]) + red[0][2][l];
  part[a.size + c] = ((db + red[1][0][l]) + red[1][1][l]) + red[1][2][l];
}

// 64 columns a workgroup, 16 threads a column.
__global__ __launch_bounds__(1024) void colsum_kernel(ColSumArgs a) {
  __shared__ float red[16][64];
  const int l = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const int64_t col = int64_t(blockIdx.x) * 64 + l;
  float v = 0.f;
  if (col < a.cols) {
    const float* p = a.part + col;
#pragma unroll 8
    for (int k = w; k < a.P; k += 16) v += p[int64_t(k) * a.cols];
  }
  red[w][l] = v;
  __syncthreads();
  if (w || col >= a.cols) return;
  v = red[0][l];
#pragma unroll
  for (int k = 1; k < 16; ++k) v += red[k][l];
  const int64_t k = col / a.C, c = col - k * a.C;
  if (k < a.K) {
    if (a.out) a.out[c * a.K + k] = v;
  } else if (a.out2) {
    a.out2[c] = v;
  }
}

template <typename T, int V, template <typename, int, int, int> class F>
hipError_t norm_shape(const NormArgs& a, hipStream_t s) {
  const NormRow r = norm_row(a.size, V, a.rows, F<T, 64, V, 1>::back);
  switch (r.threads * 16 + r.shares) {
    case 16 * 16 + 1: return F<T, 16, V, 1>::run(a, s);
    case 32 * 16 + 1: return F<T, 32, V, 1>::run(a, s);
    case 64 * 16 + 1: return F<T, 64, V, 1>::run(a, s);
    case 64 * 16 + 2: return F<T, 64, V, 2>::run(a, s);
    case 64 * 16 + 3: return F<T, 64, V, 3>::run(a, s);
    case 64 * 16 + 4:
      if constexpr (!F<T, 64, V, 1>::back) return F<T, 64, V, 4>::run(a, s);
      return hipErrorInvalidValue;
    case 256 * 16 + 1: return F<T, 256, V, 1>::run(a, s);
    case 256 * 16 + 2: return F<T, 256, V, 2>::run(a, s);
    case 256 * 16 + 4: return F<T, 256, V, 4>::run(a, s);
    case 256 * 16 + 8:
      if constexpr (V < 8) return F<T, 256, V, 8>::run(a, s);
      return hipErrorInvalidValue;
    default: return F<T, 256, V, 0>::run(a, s);
  }
}

template <typename T, int W, int V, int M>
struct Forward {
  static constexpr bool back = false;
  static hipError_t run(const NormArgs& a, hipStream_t s) {
    return go(norm_kernel<T, W, V, M>, (a.rows + 256 / W - 1) / (256 / W), 256, a, s);
  }
};
template <typename T, int W, int V, int M>
struct Backward {
  static constexpr bool back = true;
  static hipError_t run(const NormArgs& a, hipStream_t s) {
    if (M > 0 || a.dX.p) {
      const int64_t blocks = (a.rows + 256 / W - 1) / (256 / W);
      // (with partials wanted, every part is written, by a workgroup of no rows too)
      const int64_t grid = M == 0 ? blocks : a.part || blocks > a.parts ? a.parts : blocks;
      if (hipError_t e = go(norm_backward_kernel<T, W, V, M>, grid, 256, a, s); e != hipSuccess) return e;
    }
    if (M == 0 && a.part) return go(norm_columns_kernel<T>, int64_t((a.size + 63) / 64) * a.parts, 256, a, s);
    return hipSuccess;
  }
};

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? norm_shape<float, 4, Forward>(a, s) : norm_shape<float, 1, Forward>(a, s);
    case RNN_DTYPE_F16: return a.vec ? norm_shape<f16_t, 8, Forward>(a, s) : norm_shape<f16_t, 1, Forward>(a, s);
    default: return a.vec ? norm_shape<bf16_t, 8, Forward>(a, s) : norm_shape<bf16_t, 1, Forward>(a, s);
  }
}

hipError_t launch_norm_backward(const NormArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return a.vec ? norm_shape<float, 4, Backward>(a, s) : norm_shape<float, 1, Backward>(a, s);
    case RNN_DTYPE_F16: return a.vec ? norm_shape<f16_t, 8, Backward>(a, s) : norm_shape<f16_t, 1, Backward>(a, s);
    default: return a.vec ? norm_shape<bf16_t, 8, Backward>(a, s) : norm_shape<bf16_t, 1, Backward>(a, s);
  }
}

hipError_t launch_colsum(const ColSumArgs& a, hipStream_t s) { return go(colsum_kernel, (a.cols + 63) / 64, 1024, a, s); }

}  // namespace rnnhip
