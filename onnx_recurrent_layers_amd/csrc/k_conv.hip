// k_conv.hip -- the short causal convolution, one filter a channel, and its
// gradient.
//
// y_s = act(b + sum_k w_k x_{s-K+1+k}): 2K + about 6 operations for each
// element read once and written once, so memory is what the forward pass cannot
// do without.  A thread walks `tile` steps of V neighbouring channels (16 bytes
// of a row forward, 4 channels backward) with the last K inputs in registers:
// each element is read once but for the K-1 steps before a tile, which the cache
// holds (the tile before has just read them).  Eight steps' loads are in flight
// at once; but before them the K-1 inputs before the tile and the bias, and
// after the stores the final state's inputs, are loads behind branches, each
// waited for, and with walks of eight steps these trips are what bounds it.
// Kernel times, 4 taps, 16 bits, under a trace (the whole call in brackets): 8
// rows of up to 1024 steps by 2048 channels, 55 MB, 16.5 us (15.7), 3.4 TB/s,
// where layer normalization moves 67 MB in 14 to 15.6 (12.8); all steps there,
// 67 MB, (17.0); the gradient, 100 MB, 30.4, at 34 vector instructions an element
// with the vector units busy for 55 of 100 clocks, and 4.8 for the sums of 128
// partials (32.6 both); 64 single tokens 5.2 (6.6): trips to memory one after
// another, not their 2 MB.
#include <type_traits>

#include "seq_device.h"

namespace rnnhip {
namespace {

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
  const Pack<T, V> k = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = float(k.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
  Pack<T, V> k;
#pragma unroll
  for (int i = 0; i < V; ++i) k.v[i] = T(x[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = k;
}

// The taps of channels c .. c+V-1: V*K elements in a row, as K packs of V.
template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, float (&w)[K][V]) {
  const T* W = reinterpret_cast<const T*>(a.W) + int64_t(c) * K;
  float flat[K][V];
#pragma unroll
  for (int j = 0; j < K; ++j) load_v<T, V>(W + j * V, flat[j]);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = flat[(i * K + j) / V][(i * K + j) % V];
}

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs a) {
  const int cb = int(blockIdx.x) % a.ncb;
  const int rest = int(blockIdx.x) / a.ncb;
  const int b = rest / a.ntb;
  const int ty = int(threadIdx.x) / a.tx, tx = int(threadIdx.x) % a.tx;
  const int tile = (rest % a.ntb) * (256 / a.tx) + ty;
  const int c = (cb * a.tx + tx) * V;
  const int s0 = tile * a.tile;
  if (c >= a.C || (s0 >= a.geo.S && tile > 0)) return;
  const int L = geo_len(a.geo, b);
  const int s1 = min(s0 + a.tile, a.geo.S), send = min(s1, L);
  const StepRows r = step_rows(a.geo, b, L);
  const T* X = reinterpret_cast<const T*>(a.X.p) + c;
  const T* init = a.init ? reinterpret_cast<const T*>(a.init) + int64_t(b) * (K - 1) * a.C + c : nullptr;
  const int64_t xd = r.step * a.X.rs;

  // the inputs before step s: entry i is x_{s-K+1+i}
  auto before = [&](int s, float (&x)[V]) {
    if (s >= 0) {
      load_v<T, V>(X + (r.base + s * r.step) * a.X.rs, x);
    } else if (init) {
      load_v<T, V>(init + int64_t(s + K - 1) * a.C, x);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.f;
    }
  };

  if (a.Y.p && s0 < send) {
    T* Y = reinterpret_cast<T*>(a.Y.p) + c;
    const int64_t yd = r.step * a.Y.rs;
    float w[K][V], bias[V];
    load_taps<T, V, K>(a, c, w);
    if (a.bias) load_v<T, V>(reinterpret_cast<const T*>(a.bias) + c, bias);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = 0.f;
    float win[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) before(s0 - K + 1 + j, win[j]);
    const T* xp = X + (r.base + s0 * r.step) * a.X.rs;
    T* yp = Y + (r.base + s0 * r.step) * a.Y.rs;
    for (int s = s0; s < send; s += 8, xp += 8 * xd, yp += 8 * yd) {
      Pack<T, V> in[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) in[u] = *reinterpret_cast<const Pack<T, V>*>(xp + min(u, send - 1 - s) * xd);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s + u < send) {
          float x[V], y[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            x[i] = float(in[u].v[i]);
            float p = bias[i];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) p = __builtin_fmaf(w[j][i], win[j][i], p);
            p = __builtin_fmaf(w[K - 1][i], x[i], p);
            y[i] = a.silu ? p * logistic(p) : p;
          }
          store_v<T, V>(yp + u * yd, y);
#pragma unroll
          for (int j = 0; j + 1 < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
          for (int i = 0; i < V; ++i) win[K - 2][i] = x[i];
        }
      }
    }
  }
  if (a.Y.p) {
    float zero[V] = {};
    for (int s = max(s0, send); s < s1; ++s)
      store_v<T, V>(reinterpret_cast<T*>(a.Y.p) + c + dead_row(a.geo, b, s) * a.Y.rs, zero);
  }
  // the last K-1 inputs; this thread alone reads and writes the row's states,
  // all reads (those above too) before the first write: an update in place
  if (a.fin && tile == 0) {
    float f[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) before(L - K + 1 + j, f[j]);
    T* fin = reinterpret_cast<T*>(a.fin) + int64_t(b) * (K - 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_v<T, V>(fin + int64_t(j) * a.C, f[j]);
  }
}

// The gradient.  With dp_s = dY_s act'(p_s) (p computed again from X):
//   dx_e = sum_k w_k dp_{e+K-1-k} (+ d_final of the same input)
//   dw_k = sum dp_s x_{s-K+1+k},  db = sum dp_s
// Step s computes dp_s, adds its share of dw and db (tile's own steps only),
// and emits dx of the input K-1 steps back, whose K terms are then known; a
// tile walks K-1 steps past its end for the last of them.  Inputs before the
// row's first step (s < 0) are the initial state's.  A workgroup is 64 channel
// threads by four tiles; the four tiles' dw and db are added in shared memory
// and written as one partial, in a fixed order everywhere.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void conv_backward_kernel(ConvArgs a) {
  __shared__ float red[3][64 * V];
  const int cb = int(blockIdx.x) % a.ncb;
  const int rest = int(blockIdx.x) / a.ncb;
  const int b = rest / a.ntb;
  const int ty = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6), tx = int(threadIdx.x) & 63;   // (a wave's tile)
  const int tile = (rest % a.ntb) * 4 + ty;
  const int c = (cb * 64 + tx) * V;
  const int s0 = tile * a.tile;
  const int S = a.geo.S;
  const int L = geo_len(a.geo, b);
  const int s1 = min(s0 + a.tile, S), send = min(s1, L);
  const StepRows r = step_rows(a.geo, b, L);
  float dw[K][V] = {}, db[V] = {};

  if (c < a.C && (s0 < S || tile == 0)) {
    const T* X = reinterpret_cast<const T*>(a.X.p) + c;
    const T* dY = reinterpret_cast<const T*>(a.dY.p) + c;
    const int64_t sb = int64_t(b) * (K - 1) * a.C + c;
    const T* init = a.init ? reinterpret_cast<const T*>(a.init) + sb : nullptr;
    const T* dfin = a.dfin ? reinterpret_cast<const T*>(a.dfin) + sb : nullptr;
    float w[K][V], bias[V];
    load_taps<T, V, K>(a, c, w);
    if (a.bias) load_v<T, V>(reinterpret_cast<const T*>(a.bias) + c, bias);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = 0.f;
    float win[K - 1][V];   // x_{s-K+1} .. x_{s-1}
    float dp[K][V] = {};   // dp_{s-K+1} .. dp_s: those of steps before the tile are not needed (0 stands for them)
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int s = s0 - K + 1 + j;
      if (s >= 0 && s < L) load_v<T, V>(X + (r.base + s * r.step) * a.X.rs, win[j]);
      else if (s < 0 && init) load_v<T, V>(init + int64_t(s + K - 1) * a.C, win[j]);
      else
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = 0.f;
    }
    // inputs whose gradient this tile emits: [e0, e1); the first tile emits
    // the initial state's too
    const int e0 = tile == 0 ? -(K - 1) : s0;
    const int e1 = s0 >= L && tile > 0 ? s0 : max(send, tile == 0 ? 0 : s0);
    const T* xp = X + (r.base + s0 * r.step) * a.X.rs;
    const T* gp = dY + (r.base + s0 * r.step) * a.dY.rs;
    const int64_t xd = r.step * a.X.rs, gd = r.step * a.dY.rs;
    // four steps' rows, and the next four's under way; past the row's end its
    // last step's (not used)
    Pack<T, V> nin[4], ngin[4];
    auto fetch = [&](int s) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = min(u, L - 1 - s);
        nin[u] = *reinterpret_cast<const Pack<T, V>*>(xp + at * xd);
        ngin[u] = *reinterpret_cast<const Pack<T, V>*>(gp + at * gd);
      }
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) nin[u] = ngin[u] = Pack<T, V>{};
    if (s0 < L) fetch(s0);
    for (int s = s0; s - K + 1 < e1; s += 4) {
      Pack<T, V> in[4], gin[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        in[u] = nin[u];
        gin[u] = ngin[u];
      }
      xp += 4 * xd;
      gp += 4 * gd;
      if (s + 4 < L && s + 4 - K + 1 < e1) fetch(s + 4);
      // WHOLE: steps of this tile, and inputs that are its own and not the final
      // state's, which leaves four steps without a question asked (8 x 1024 x
      // 2048, the whole call: 32.6 us, with the questions 35.1)
      auto four = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int st = s + u;
          const bool live = WHOLE || st < L;
          const bool mine = WHOLE || st < send;
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) dp[j][i] = dp[j + 1][i];
            float x = 0.f, d = 0.f;
            if (live) {
              x = float(in[u].v[i]);
              d = float(gin[u].v[i]);
              if (a.silu) {
                float p = bias[i];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) p = __builtin_fmaf(w[j][i], win[j][i], p);
                p = __builtin_fmaf(w[K - 1][i], x, p);
                const float sg = logistic(p);
                d *= sg * __builtin_fmaf(p, 1.f - sg, 1.f);
              }
            }
            dp[K - 1][i] = d;
            if (mine) {
#pragma unroll
              for (int j = 0; j < K - 1; ++j) dw[j][i] = __builtin_fmaf(d, win[j][i], dw[j][i]);
              dw[K - 1][i] = __builtin_fmaf(d, x, dw[K - 1][i]);
              db[i] += d;
            }
#pragma unroll
            for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
            win[K - 2][i] = x;
          }
          const int e = st - K + 1;
          if (WHOLE || (e >= e0 && e < e1)) {
            float dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float v = 0.f;
#pragma unroll
              for (int j = 0; j < K; ++j) v = __builtin_fmaf(w[K - 1 - j][i], dp[j][i], v);
              dx[i] = v;
            }
            const int f = e - (L - K + 1);   // its place in the final state
            if (!WHOLE && dfin && f >= 0) {
              float t[V];
              load_v<T, V>(dfin + int64_t(f) * a.C, t);
#pragma unroll
              for (int i = 0; i < V; ++i) dx[i] += t[i];
            }
            if (WHOLE || e >= 0) {
              if (a.dX.p) store_v<T, V>(reinterpret_cast<T*>(a.dX.p) + c + (r.base + e * r.step) * a.dX.rs, dx);
            } else if (a.dinit) {
              store_v<T, V>(reinterpret_cast<T*>(a.dinit) + sb + int64_t(e + K - 1) * a.C, dx);
            }
          }
        }
      };
      if (s - K + 1 >= max(e0, 0) && s + 3 < send && s + 3 < L - K + 1) four(std::true_type{});
      else four(std::false_type{});
    }
    if (a.dX.p) {
      float zero[V] = {};
      for (int s = max(s0, send); s < s1; ++s)
        store_v<T, V>(reinterpret_cast<T*>(a.dX.p) + c + dead_row(a.geo, b, s) * a.dX.rs, zero);
    }
  }
  if (!a.part) return;
  float* part = a.part + int64_t(rest) * (K + 1) * a.C;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = j < K ? dw[j < K ? j : 0][i] : db[i];
    if (ty > 0)
#pragma unroll
      for (int i = 0; i < V; ++i) red[ty - 1][i * 64 + tx] = v[i];
    __syncthreads();
    if (ty == 0 && c < a.C) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = ((v[i] + red[0][i * 64 + tx]) + red[1][i * 64 + tx]) + red[2][i * 64 + tx];
        part[int64_t(j) * a.C + c + i] = v[i];
      }
    }
    __syncthreads();
  }
}

template <typename T, int V>
hipError_t conv_k(const ConvArgs& a, int64_t blocks, hipStream_t s) {
  switch (a.K) {
    case 2: return go(conv_kernel<T, V, 2>, blocks, 256, a, s);
    case 3: return go(conv_kernel<T, V, 3>, blocks, 256, a, s);
    case 4: return go(conv_kernel<T, V, 4>, blocks, 256, a, s);
    case 5: return go(conv_kernel<T, V, 5>, blocks, 256, a, s);
    case 6: return go(conv_kernel<T, V, 6>, blocks, 256, a, s);
    case 7: return go(conv_kernel<T, V, 7>, blocks, 256, a, s);
    case 8: return go(conv_kernel<T, V, 8>, blocks, 256, a, s);
    default: return hipErrorInvalidValue;
  }
}
template <typename T, int V>
hipError_t conv_backward_k(const ConvArgs& a, int64_t blocks, hipStream_t s) {
  switch (a.K) {
    case 2: return go(conv_backward_kernel<T, V, 2>, blocks, 256, a, s);
    case 3: return go(conv_backward_kernel<T, V, 3>, blocks, 256, a, s);
    case 4: return go(conv_backward_kernel<T, V, 4>, blocks, 256, a, s);
    case 5: return go(conv_backward_kernel<T, V, 5>, blocks, 256, a, s);
    case 6: return go(conv_backward_kernel<T, V, 6>, blocks, 256, a, s);
    case 7: return go(conv_backward_kernel<T, V, 7>, blocks, 256, a, s);
    case 8: return go(conv_backward_kernel<T, V, 8>, blocks, 256, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, int dtype, int vec, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.ntb * a.ncb;
  switch (dtype) {
    case RNN_DTYPE_F32: return vec > 1 ? conv_k<float, 4>(a, blocks, s) : conv_k<float, 1>(a, blocks, s);
    case RNN_DTYPE_F16: return vec > 1 ? conv_k<f16_t, 8>(a, blocks, s) : conv_k<f16_t, 1>(a, blocks, s);
    default: return vec > 1 ? conv_k<bf16_t, 8>(a, blocks, s) : conv_k<bf16_t, 1>(a, blocks, s);
  }
}

hipError_t launch_conv_backward(const ConvArgs& a, int dtype, int vec, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.ntb * a.ncb;
  switch (dtype) {
    case RNN_DTYPE_F32: return vec > 1 ? conv_backward_k<float, 4>(a, blocks, s) : conv_backward_k<float, 1>(a, blocks, s);
    case RNN_DTYPE_F16: return vec > 1 ? conv_backward_k<f16_t, 4>(a, blocks, s) : conv_backward_k<f16_t, 1>(a, blocks, s);
    default: return vec > 1 ? conv_backward_k<bf16_t, 4>(a, blocks, s) : conv_backward_k<bf16_t, 1>(a, blocks, s);
  }
}

}  // namespace rnnhip
