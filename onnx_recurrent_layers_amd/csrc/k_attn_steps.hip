// k_attn_steps.hip -- linear attention step after step, and what finishes its
// gradient: the decays' sums and the sums over the heads of a group.
//
//   S_u = e^(g_u) S_(u-1) + in_scale * b_u v_u^T,   out_u = out_scale * a_u^T S_u
//
// A workgroup takes 64 columns of a head's state, 16 lanes of four columns (256
// bytes of a state's row) by 16 shares of the rows, and holds them in registers.
// Everything that the first step needs is asked for at once.  A token is bound by
// the state, which is read and written once: one of 64 rows, 16 heads of 128 x 128,
// bf16, takes 30.0 us for 136 MB, 4.5 TB/s, where a copy takes 28.5; one of one row,
// 8 heads of 64 x 64, 4.8 of latency.
#include "attn_device.h"

namespace rnnhip {
namespace {

// KI: rows of the state that a thread holds; DOT: what the decays' gradient
// needs, too; VEC: states in aligned pieces of four columns.
template <typename T, int KI, bool DOT, bool VEC>
__global__ __launch_bounds__(256) void attn_steps_kernel(AttnArgs a) {
  __shared__ float sa[2][256], sb[2][256], sv[2][kAttnCols], red[2][DOT ? 2 : 1][4][kAttnCols];
  const int t = int(threadIdx.x), l = t & 15, kg = t >> 4, w = t >> 6;
  const int slices = (a.V + kAttnCols - 1) / kAttnCols;
  const int slice = int(blockIdx.x) % slices, bh = int(blockIdx.x) / slices;
  const int b = bh / a.H, h = bh - b * a.H;
  const int c0 = slice * kAttnCols, c = c0 + 4 * l;
  const int L = geo_len(a.geo, b);
  const AttnSteps<T> r(a, b, h, L, 0, L);
  const int64_t st = int64_t(bh) * a.K * a.V;

  float ra = 0.f, rb = 0.f, rv = 0.f, rg = 0.f;
  auto fetch = [&](int u) {
    const int64_t row = r.row(u);
    if (t < a.K) {
      ra = r.get(a.a, a.K, row, t);
      rb = r.get(a.b, a.K, row, t);
    }
    if (t < kAttnCols) rv = c0 + t < a.V ? r.get(a.v, a.V, row, c0 + t) : 0.f;
    rg = r.log_decay(u);
  };
  if (L > 0) fetch(0);
  float S[KI][4];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int k = kg + 16 * i;
    attn_get_state<VEC>(a, a.init, st, k, c, S[i]);
  }
  float first = 1.f;
  for (int u = 0; u < L; ++u) {
    const int p = u & 1;
    if (t < a.K) {
      sa[p][t] = ra;
      sb[p][t] = rb * a.in_scale;
    }
    if (t < kAttnCols) sv[p][t] = rv;
    const float dec = __builtin_amdgcn_exp2f(rg * kLog2e);
    if (u + 1 < L) fetch(u + 1);
    __syncthreads();
    float y[4] = {}, off[4] = {};
    const float4 v = *reinterpret_cast<const float4*>(&sv[p][4 * l]);
    const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int k = kg + 16 * i;
      if (k >= a.K) break;
      const float qa = sa[p][k], kb = sb[p][k];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] *= dec;
        if (DOT) off[j] = __builtin_fmaf(qa, S[i][j], off[j]);
        S[i][j] = __builtin_fmaf(kb, vv[j], S[i][j]);
        y[j] = __builtin_fmaf(qa, S[i][j], y[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int m = 16; m < 64; m *= 2) {
        y[j] += __shfl_xor(y[j], m, 64);
        if (DOT) off[j] += __shfl_xor(off[j], m, 64);
      }
      if ((t & 63) < 16) {
        red[p][0][w][4 * l + j] = y[j];
        if (DOT) red[p][DOT ? 1 : 0][w][4 * l + j] = off[j];
      }
    }
    __syncthreads();
    if (t < kAttnCols) {
      auto sum = [&](int n) { return a.out_scale * (((red[p][n][0][t] + red[p][n][1][t]) + red[p][n][2][t]) + red[p][n][3][t]); };
      const int64_t row = r.row(u);
      if (c0 + t < a.V) r.put(row, c0 + t, sum(0));
      if constexpr (DOT) {
        float d = c0 + t < a.V ? sum(1) * r.get(a.dot, a.V, row, c0 + t) : 0.f;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) d += __shfl_xor(d, m, 64);
        if (t == 0) a.dots[((int64_t(slice) * a.geo.B + b) * a.H + h) * a.geo.S + r.step(u)] = d;
      }
    }
  }
  if (a.back && L > 0) first = __builtin_amdgcn_exp2f(r.first_decay() * kLog2e);
#pragma unroll
  for (int i = 0; i < KI; ++i) attn_put_state<VEC>(a, a.fin, st, kg + 16 * i, c, S[i], first);
  if (DOT && a.ends) {
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      float o[4];
      attn_get_state<VEC>(a, a.other, st, kg + 16 * i, c, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) d = __builtin_fmaf(S[i][j], o[j], d);
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) d += __shfl_xor(d, m, 64);
    __syncthreads();
    if ((t & 63) == 0) red[0][0][0][w] = d;
    __syncthreads();
    if (t == 0)
      a.ends[int64_t(slice) * a.geo.B * a.H + bh] = ((red[0][0][0][0] + red[0][0][0][1]) + red[0][0][0][2]) + red[0][0][0][3];
  }
  // steps that the row does not take
  if (a.out.p)
    for (int s = L + w; s < a.geo.S; s += 4)
      if (c0 + (t & 63) < a.V) r.put(dead_row(a.geo, b, s), c0 + (t & 63), 0.f);
}

// An element of a head's states a thread, through the pieces in the walk's order.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoinArgs a) {
  const int64_t per = (a.size + 255) / 256, bh = int64_t(blockIdx.x) / per, i = (int64_t(blockIdx.x) - bh * per) * 256 + threadIdx.x;
  if (i >= a.size) return;
  float* p = a.starts + bh * a.pieces * a.size + i;
  float v = a.init ? a.init[bh * a.size + i] : 0.f;
  for (int k = 0; k < a.pieces; ++k) {
    const int at = a.back ? a.pieces - 1 - k : k;
    const float local = k + 1 < a.pieces ? p[at * a.size] : 0.f;
    p[at * a.size] = v;
    if (k + 1 < a.pieces) v = __builtin_fmaf(v, a.totals[bh * a.pieces + at], local);
  }
}

// A piece's steps of a head, 256 at a time from the last: the sum of what is left
// of each step's pairs with earlier steps less those with later ones, whose
// whole is at hand again at each piece's end.  64-bit sums, since the two
// nearly cancel.
__global__ __launch_bounds__(256) void attn_decay_kernel(AttnDecayArgs a) {
  __shared__ double part[4];
  const int t = int(threadIdx.x), w = t >> 6;
  const int64_t head = int64_t(a.geo.B) * a.H, bh = int64_t(blockIdx.x) / a.pieces;
  const int piece = int(int64_t(blockIdx.x) - bh * a.pieces), b = int(bh / a.H), h = int(bh - int64_t(b) * a.H);
  const int L = geo_len(a.geo, b);
  const int64_t lo64 = int64_t(piece) * a.piece;
  const int lo = int(min(lo64, int64_t(a.geo.S))), end = int(min(lo64 + a.piece, int64_t(a.geo.S))), hi = min(end, L);
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t n = head * a.geo.S, at = bh * a.geo.S;
  double after = 0., total = 0.;   // the gradient just after the block's steps; a thread's part of its sum
  if (a.ends && hi > lo)
    for (int k = 0; k < a.slices; ++k) after += a.ends[(k * head + bh) * a.pieces + piece];
  for (int s1 = hi; s1 > lo; s1 -= 256) {
    const int s = s1 - 1 - t;   // thread 0: the last step
    double x = 0.;
    if (s >= lo)
      for (int k = 0; k < a.slices; ++k) x += double(a.rows[k * n + at + s]) - double(a.cols[k * n + at + s]);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_up(x, m, 64);
      if ((t & 63) >= m) x += o;
    }
    __syncthreads();
    if ((t & 63) == 63) part[w] = x;
    __syncthreads();
    double before = after;
    for (int k = 0; k < 4; ++k) {
      if (k < w) before += part[k];
      after += part[k];
    }
    if (s >= lo) {
      const int64_t row = r.base + s * r.step;
      float g = a.G.p ? reinterpret_cast<const float*>(a.G.p)[row * a.G.rs + h] : 0.f;
      if (a.decay) g += a.decay[h];
      const double d = g > 0.f ? 0. : before + x;   // (a decay above one counts as one)
      if (a.dG.p) reinterpret_cast<float*>(a.dG.p)[row * a.dG.rs + h] = float(d);
      total += d;
    }
  }
  if (a.dG.p)
    for (int s = max(lo, L) + t; s < end; s += 256) reinterpret_cast<float*>(a.dG.p)[dead_row(a.geo, b, s) * a.dG.rs + h] = 0.f;
  if (!a.part) return;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) total += __shfl_xor(total, m, 64);
  __syncthreads();
  if ((t & 63) == 0) part[w] = total;
  __syncthreads();
  if (t == 0) a.part[(int64_t(b) * a.pieces + piece) * a.H + h] = float(((part[0] + part[1]) + part[2]) + part[3]);
}

template <typename T>
__global__ __launch_bounds__(256) void head_sum_kernel(HeadSumArgs a) {
  const int groups = a.H / a.per;
  const int64_t cols = int64_t(groups) * a.K;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.n * a.rows * cols; i += int64_t(gridDim.x) * 256) {
    const bool second = i >= a.rows * cols;
    const int64_t row = i / cols - (second ? a.rows : 0), c = i % cols, g = c / a.K, k = c - g * a.K;
    const float* p = (second ? a.part[1] : a.part[0]) + (row * a.H + g * a.per) * a.K + k;
    const Rows& out = second ? a.out[1] : a.out[0];
    float v = 0.f;
    for (int j = 0; j < a.per; ++j) v += p[int64_t(j) * a.K];
    reinterpret_cast<T*>(out.p)[row * out.rs + c] = T(v);
  }
}

template <typename T, bool DOT, bool VEC>
hipError_t steps_of(const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.H * ((a.V + kAttnCols - 1) / kAttnCols);
  if (a.K <= 64) return go(attn_steps_kernel<T, 4, DOT, VEC>, blocks, 256, a, s);
  if (a.K <= 128) return go(attn_steps_kernel<T, 8, DOT, VEC>, blocks, 256, a, s);
  return go(attn_steps_kernel<T, 16, DOT, VEC>, blocks, 256, a, s);
}

template <typename T>
hipError_t steps(const AttnArgs& a, hipStream_t s) {
  const auto whole = [](const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = a.sv == 1 && a.V % 4 == 0 && whole(a.init) && whole(a.fin);
  if (a.dots) return steps_of<T, true, false>(a, s);
  return vec ? steps_of<T, false, true>(a, s) : steps_of<T, false, false>(a, s);
}

}  // namespace

hipError_t launch_attn_steps(const AttnArgs& a, int dtype, hipStream_t s) {
  return dtype == RNN_DTYPE_F32 ? steps<float>(a, s) : dtype == RNN_DTYPE_F16 ? steps<f16_t>(a, s) : steps<bf16_t>(a, s);
}

hipError_t launch_attn_join(const AttnJoinArgs& a, hipStream_t s) {
  return go(attn_join_kernel, a.heads * ((a.size + 255) / 256), 256, a, s);
}

hipError_t launch_attn_decay(const AttnDecayArgs& a, hipStream_t s) {
  return go(attn_decay_kernel, int64_t(a.geo.B) * a.H * a.pieces, 256, a, s);
}

hipError_t launch_head_sum(const HeadSumArgs& a, int dtype, hipStream_t s) {
  const int64_t all = (a.n * a.rows * (a.H / a.per) * a.K + 255) / 256, blocks = all < 1 << 20 ? all : 1 << 20;
  return dtype == RNN_DTYPE_F32   ? go(head_sum_kernel<float>, blocks, 256, a, s)
         : dtype == RNN_DTYPE_F16 ? go(head_sum_kernel<f16_t>, blocks, 256, a, s)
                                  : go(head_sum_kernel<bf16_t>, blocks, 256, a, s);
}

}  // namespace rnnhip
