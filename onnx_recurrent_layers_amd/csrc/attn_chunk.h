// attn_chunk.h -- linear attention over chunks of the time axis on the matrix
// cores (instantiated for one element type by k_attn_f32.hip, k_attn_f16.hip and
// k_attn_bf16.hip).
//
// With c_i the sum of the log decays of a chunk's steps up to i, and S0 the state
// before the chunk,
//   out_i = out_scale ( e^(c_i) a_i^T S0 + sum_{j <= i} e^(c_i - c_j) (a_i . b_j) in_scale v_j )
//   S     = e^(c_end) S0 + sum_j b_j (e^(c_end - c_j) in_scale v_j)^T
// which is four products: scores of the chunk's steps by each other, the scores by
// v, a by the state, and b by v.  Every exponent is a difference that the
// definition has, and at most zero: nothing overflows, whatever the decays.  The
// sums c are taken in 64 bits and kept as two floats, so that a difference keeps
// its digits next to a step that forgets everything.
//
// A workgroup takes 64 columns of v and out, 16 a wave, all rows of the state for
// them, in registers as the products leave them: a product's result has four
// neighbouring rows a lane, which is an operand of the next product when the rows
// of a 32-deep step are taken as 4 g + (0..3) and 16 + 4 g + (0..3) by lane group
// g.  Scores go by shared memory, each wave computing those of 16 steps.  b and v
// by steps (the second product and the fourth) are read from shared memory by the
// transposing reads.
//
// Values of 32 bits (scores, state, decayed v) enter a product of 16-bit operands
// in parts: bf16 two for the scores and the state (2^-16 of each), three (2^-24)
// for what is summed into the state or into the decays' gradient; f16 two (2^-22),
// scaled by a power of two to the largest of the wave's, since f16 has neither
// the state's range nor the scores'.  f32 uses the f32 matrix cores.
//
// A masked score is a zero, but a zero times a later step's infinity or NaN is
// not; and an infinite value has no parts.  A wave whose chunk has an output that
// is not finite goes back to the steps one by one.
#pragma once

#include "attn_device.h"

namespace rnnhip {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

// Operands of a 32-deep product, 8 values a lane: Coarse parts of a score or a
// state, Fine ones of what is summed on.
template <typename T>
struct Mma;

template <>
struct Mma<bf16_t> {
  static constexpr int Coarse = 2, Fine = 3, Vec = 8, Pad = 8;
  static constexpr bool Scaled = false;
  typedef bf16x8 Op;
  typedef bf16x4 Half;
  static __device__ __forceinline__ f32x4 mul(Op a, Op b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ Half column(const bf16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4*)(p));
  }
};
template <>
struct Mma<f16_t> {
  static constexpr int Coarse = 2, Fine = 2, Vec = 8, Pad = 8;
  static constexpr bool Scaled = true;
  typedef f16x8 Op;
  typedef f16x4 Half;
  static __device__ __forceinline__ f32x4 mul(Op a, Op b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ Half column(const f16_t* p) {
    return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p)));
  }
};
struct f32x8 {
  f32x4 lo, hi;
  __device__ __forceinline__ float operator[](int i) const { return i < 4 ? lo[i] : hi[i - 4]; }
};
template <>
struct Mma<float> {
  static constexpr int Coarse = 1, Fine = 1, Vec = 4, Pad = 4;
  static constexpr bool Scaled = false;
  typedef f32x8 Op;
  static __device__ __forceinline__ f32x4 mul(const Op& a, const Op& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// Eight neighbouring values, or two runs of four.
template <typename T>
__device__ __forceinline__ typename Mma<T>::Op op_run(const T* p) {
  if constexpr (sizeof(T) == 4) return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
  else return *reinterpret_cast<const typename Mma<T>::Op*>(p);
}
template <typename T>
__device__ __forceinline__ typename Mma<T>::Op op_runs(const T* p, const T* q) {
  if constexpr (sizeof(T) == 4) {
    return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(q)};
  } else {
    typedef typename Mma<T>::Half H;
    return __builtin_shufflevector(*reinterpret_cast<const H*>(p), *reinterpret_cast<const H*>(q), 0, 1, 2, 3, 4, 5, 6, 7);
  }
}
// Eight steps, first to first + 7, of the lane's column among 16 from c0 on.
// (16 bits: a transposing read takes four rows of 16 columns for 16 lanes, each
// lane naming four columns of a row.)
template <typename T>
__device__ __forceinline__ typename Mma<T>::Op op_column(const T* base, int stride, int first, int c0, int q) {
  if constexpr (sizeof(T) == 4) {
    const float* p = base + first * stride + c0 + q;
    return {f32x4{p[0], p[stride], p[2 * stride], p[3 * stride]}, f32x4{p[4 * stride], p[5 * stride], p[6 * stride], p[7 * stride]}};
  } else {
    const T* p = base + (first + (q >> 2)) * stride + c0 + 4 * (q & 3);
    return __builtin_shufflevector(Mma<T>::column(p), Mma<T>::column(p + 4 * stride), 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// N parts of eight values of 32 bits.
template <typename T, int N>
struct Parts {
  typename Mma<T>::Op p[N];
};
template <typename T, int N>
__device__ __forceinline__ Parts<T, N> op_parts(const float (&x)[8]) {
  Parts<T, N> r;
  if constexpr (sizeof(T) == 4) {
    r.p[0] = {f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}};
  } else {
    float left[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) left[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r.p[n][i] = T(left[i]);
        if (n + 1 < N) left[i] -= float(T(left[i]));
      }
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ f32x4 mul_parts(const Parts<T, N>& a, const typename Mma<T>::Op& b, f32x4 c) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) c = Mma<T>::mul(a.p[n], b, c);
  return c;
}
template <typename T, int N>
__device__ __forceinline__ f32x4 mul_parts(const typename Mma<T>::Op& a, const Parts<T, N>& b, f32x4 c) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) c = Mma<T>::mul(a, b.p[n], c);
  return c;
}

// The power of two that takes the largest magnitude of a wave's values, m, to
// 2^13 to 2^14, and its inverse (1 for a zero, and for what is not finite).
struct Scale {
  float by, back;
};
__device__ __forceinline__ Scale wave_scale(float m) {
  auto of = [&](auto CTRL) {
    const float o = __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, m), decltype(CTRL)::value, 0xf, 0xf, true));
    m = m > o ? m : o;
  };
  of(std::integral_constant<int, 0xb1>{});    // lane ^ 1
  of(std::integral_constant<int, 0x4e>{});    // lane ^ 2
  of(std::integral_constant<int, 0x141>{});   // the other half of eight lanes
  of(std::integral_constant<int, 0x140>{});   // the other half of sixteen
  int e = 0;
#pragma unroll
  for (int l = 0; l < 64; l += 16) e = max(e, __builtin_amdgcn_readlane(__builtin_bit_cast(int, m), l));
  e >>= 23;
  e = e == 0 || e >= 255 ? 140 : max(e, 14);
  return {__builtin_bit_cast(float, (267 - e) << 23), __builtin_bit_cast(float, (e - 13) << 23)};
}

__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

// The value, unknown to the compiler from here on: conditions on it are made where
// they are used.  (Kept from the kernel's start to its end, masks of 64 lanes for
// each row of a state fill the scalar registers.)
__device__ __forceinline__ int afresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

enum { kAttnLocal, kAttnWalk, kAttnDots };

// KT: 32-wide pieces of a and b.  MODE: the state that a piece of the time axis
// leaves from a zero one; the outputs; these with what the decays' gradient
// needs.  VEC: rows in aligned 16-byte pieces.
template <typename T, int KT, int MODE, bool VEC>
__global__ __launch_bounds__(256, 2) void attn_chunk_kernel(AttnArgs a) {
  typedef Mma<T> M;
  typedef typename M::Op Op;
  constexpr bool WALK = MODE != kAttnLocal, DOTS = MODE == kAttnDots;
  constexpr int TC = sizeof(T) == 4 && KT == 8 ? 32 : 64, IT = TC / 16, ST = TC / 32;   // steps of a chunk, in 16s and 32s
  constexpr int KP = 32 * KT + M::Pad, VP = kAttnCols + M::Pad, PP = TC + M::Pad;
  constexpr int NP = DOTS ? M::Fine : M::Coarse, NU = M::Fine;
  constexpr int CK = 32 * KT / M::Vec, CV = kAttnCols / M::Vec;                          // 16-byte pieces of a row
  constexpr int NK = TC * CK / 256, NV = TC * CV / 256;                                  // of a thread
  __shared__ alignas(16) T sa[WALK ? TC : 1][KP];
  __shared__ alignas(16) T sb[TC][KP];
  __shared__ alignas(16) T sv[TC][VP];
  __shared__ alignas(16) T sp[WALK ? NP : 1][WALK ? TC : 1][PP];
  __shared__ alignas(16) float shi[TC], slo[TC], ssince[TC], sleft[TC], slog[TC], sdiag[TC], sback[IT], red[4][TC];
  const int t = int(threadIdx.x), lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), q = lane & 15, g = lane >> 4;
  const int slices = (a.V + kAttnCols - 1) / kAttnCols, pieces = WALK ? a.pieces : a.pieces - 1;
  const int slice = int(blockIdx.x) % slices, bp = int(blockIdx.x) / slices, bh = bp / pieces;
  const int piece = bp - bh * pieces + (!WALK && a.back ? 1 : 0);
  const int b = bh / a.H, h = bh - b * a.H;
  const int L = geo_len(a.geo, b);
  const int64_t lo64 = int64_t(piece) * a.piece;
  const int lo = int(min(lo64, int64_t(a.geo.S))), end = int(min(lo64 + a.piece, int64_t(a.geo.S))), hi = min(end, L), n = max(hi - lo, 0);
  const AttnSteps<T> r(a, b, h, L, lo, hi);
  const int c0 = slice * kAttnCols, cw = c0 + 16 * w;   // columns of the workgroup, of the wave
  const int64_t KV = int64_t(a.K) * a.V;
  const float scale = a.in_scale * a.out_scale;

  // a chunk's rows, in registers until the one before is done with.  A thread's
  // rows of a tensor are RK (RV) apart; past the last one it repeats that, and
  // what it got is made zero on the way to shared memory.
  typedef Pack<T, M::Vec> Piece;
  constexpr int RK = 256 / CK, RV = 256 / CV;
  const int tk = t / CK, ck = t % CK * M::Vec, tv = t / CV, cv = t % CV * M::Vec;
  const int64_t way = a.back ? -r.r.step : r.r.step, top = n > 0 ? r.row(0) : 0;
  struct Walker {   // a thread's pieces of one tensor, a chunk's first row first
    const T *p, *last;
    int64_t rs;
  };
  auto walker = [&](const HeadRows& x, int size, int row, int c) {
    const int64_t rs = way * x.rs;
    const T* p = reinterpret_cast<const T*>(x.p) + top * x.rs + (h / x.per) * int64_t(size) + (c < size ? c : 0);
    return Walker{p + row * rs, p + max(n - 1, 0) * rs, rs};
  };
  Walker wa = WALK ? walker(a.a, a.K, tk, ck) : Walker{}, wb = walker(a.b, a.K, tk, ck), wv = walker(a.v, a.V, tv, c0 + cv);
  Piece ra[WALK ? NK : 1], rb[NK], rv[NV];
  auto load = [&](const Walker& x, int u, int i, int by, int size, int c) {
    const T* at = u + i * by < n ? x.p + i * by * x.rs : x.last;
    Piece p = {};
    if constexpr (VEC) {
      p = *reinterpret_cast<const Piece*>(at);
    } else {
#pragma unroll
      for (int k = 0; k < M::Vec; ++k)
        if (c + k < size) p.v[k] = at[k];
    }
    return p;
  };
  float rg = 0.f;
  auto fetch = [&](int u0) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      if constexpr (WALK) ra[i] = load(wa, u0 + tk, i, RK, a.K, ck);
      rb[i] = load(wb, u0 + tk, i, RK, a.K, ck);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) rv[i] = load(wv, u0 + tv, i, RV, a.V, c0 + cv);
    rg = lane < TC && u0 + lane < n ? r.log_decay(u0 + lane) : 0.f;
    wa.p += TC * wa.rs;
    wb.p += TC * wb.rs;
    wv.p += TC * wv.rs;
  };
  auto keep = [&](Piece& p, bool is) {
    if (!is) p = Piece{};
  };
  // lane i: the sums of log decays (to base 2) up to step i
  double csum = 0., ctotal = 0.;
  float clog = 0.f;
  auto sums = [&] {
    clog = rg * kLog2e;
    csum = double(rg) * 1.4426950408889634;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_up(csum, m, 64);
      if (lane >= m) csum += o;
    }
    ctotal = __shfl(csum, 63, 64);
  };

  // rows 16 k + 4 g + (0..3) of the state, column cw + q
  f32x4 S[2 * KT];
  const bool col = cw + q < a.V;
  const float* start = !WALK ? nullptr : a.pieces > 1 ? a.starts + (int64_t(bh) * a.pieces + piece) * KV : a.init ? a.init + bh * KV : nullptr;
  auto state_at = [&](int k, int i) { return int64_t(16 * k + 4 * g + i) * a.sk + int64_t(cw + q) * a.sv; };
  // rows that there are among 4 g + (0..3) on (none without a column): for k, i those below
  auto rows_of = [&] { return afresh(col ? a.K - 4 * g : 0); };
  if (n > 0) fetch(0);
#pragma unroll
  for (int k = 0; k < 2 * KT; ++k) S[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (start) {   // (past the last row or column: some other, made zero)
    const float* at = start + int64_t(col ? cw + q : 0) * a.sv;
    const int rows = rows_of();
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[k][i] = at[min(16 * k + 4 * g + i, a.K - 1) * a.sk];
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[k][i] = 16 * k + i < rows ? S[k][i] : 0.f;
  }
  if constexpr (WALK) {   // scores above the diagonal that a product reads
    for (int i = t; i < NP * TC * PP; i += 256) sp[0][0][i] = T(0.f);
  }
  sums();
  double all = 0.;   // of the piece
  // this lane's first element of a chunk's outputs, and of the rows that they are multiplied with
  const int64_t ors = way * a.out.rs, drs = way * a.dot.rs;
  int64_t po = 0, pd = 0;
  if constexpr (WALK) po = top * a.out.rs + (h / a.out.per) * int64_t(a.V) + cw + 4 * g + q * ors;
  if constexpr (DOTS) pd = top * a.dot.rs + (h / a.dot.per) * int64_t(a.V) + cw + 4 * g + q * drs;

  // The steps of the chunk one by one, from shared memory.
  auto one_by_one = [&](int u0, int steps) {
    for (int u = 0; u < steps; ++u) {
      const float dec = __builtin_amdgcn_exp2f(slog[u]);
      const float v = float(sv[u][16 * w + q]);
      float off = 0.f, y = 0.f;
      const int rows = afresh(a.K - 4 * g);
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 16 * k + 4 * g + i;
          if (16 * k + i < rows) {
            const float kb = float(sb[u][d]) * a.in_scale;
            S[k][i] *= dec;
            if constexpr (WALK) off = __builtin_fmaf(float(sa[u][d]), S[k][i], off);
            S[k][i] = __builtin_fmaf(kb, v, S[k][i]);
            if constexpr (WALK) y = __builtin_fmaf(float(sa[u][d]), S[k][i], y);
          }
        }
      if constexpr (WALK) {
        y += __shfl_xor(y, 16, 64);
        y += __shfl_xor(y, 32, 64);
        const int64_t row = r.row(u0 + u);
        if (g == 0 && col) r.put(row, cw + q, y * a.out_scale);
        if constexpr (DOTS) {
          off += __shfl_xor(off, 16, 64);
          off += __shfl_xor(off, 32, 64);
          off = col ? off * a.out_scale * r.get(a.dot, a.V, row, cw + q) : 0.f;
#pragma unroll
          for (int m = 1; m < 16; m *= 2) off += __shfl_xor(off, m, 64);
          if (lane == 0) red[w][u] = off;
        }
      }
    }
  };
  auto put_dots = [&](int u0) {
    if (t < TC && u0 + t < n)
      a.dots[((int64_t(slice) * a.geo.B + b) * a.H + h) * a.geo.S + r.step(u0 + t)] = ((red[0][t] + red[1][t]) + red[2][t]) + red[3][t];
  };

  for (int u0 = 0; u0 < n; u0 += TC) {
    __syncthreads();   // all are done with the chunk before
    if (u0 + TC > n || a.K < 32 * KT || c0 + kAttnCols > a.V) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        if constexpr (WALK) keep(ra[i], u0 + tk + i * RK < n && ck < a.K);
        keep(rb[i], u0 + tk + i * RK < n && ck < a.K);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) keep(rv[i], u0 + tv + i * RV < n && c0 + cv < a.V);
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      if constexpr (WALK) *reinterpret_cast<Piece*>(&sa[tk + i * RK][ck]) = ra[i];
      *reinterpret_cast<Piece*>(&sb[tk + i * RK][ck]) = rb[i];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) *reinterpret_cast<Piece*>(&sv[tv + i * RV][cv]) = rv[i];
    if (t < TC) {
      shi[t] = float(csum);
      slo[t] = float(csum - double(float(csum)));
      ssince[t] = __builtin_amdgcn_exp2f(float(csum)) * a.out_scale;
      sleft[t] = __builtin_amdgcn_exp2f(float(ctotal - csum)) * a.in_scale;
      slog[t] = clog;
    }
    const float total = __builtin_amdgcn_exp2f(float(ctotal));
    all += ctotal;
    if (DOTS && u0 > 0) put_dots(u0 - TC);
    __syncthreads();
    const int steps = min(n - u0, TC);
    if (u0 + TC < n) fetch(u0 + TC);

    bool fine = true;
    if constexpr (WALK) {
      // the scores of steps 16 w to 16 w + 15 (this lane's: 16 w + q) by those up to them
      if (w < IT) {
        Op fa[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) fa[k] = op_run<T>(&sa[16 * w + q][32 * k + 8 * g]);
        const int i = 16 * w + q;
        const float hi_i = shi[i], lo_i = slo[i];
        float p[IT][4], most = 0.f;
#pragma unroll
        for (int j = 0; j < IT; ++j) {
          if (j > w) break;
          f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KT; ++k) c = M::mul(op_run<T>(&sb[16 * j + q][32 * k + 8 * g]), fa[k], c);
          const f32x4 hj = *reinterpret_cast<const f32x4*>(&shi[16 * j + 4 * g]), lj = *reinterpret_cast<const f32x4*>(&slo[16 * j + 4 * g]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = 16 * j + 4 * g + k;
            const float x = c[k] * scale * __builtin_amdgcn_exp2f((hi_i - hj[k]) + (lo_i - lj[k]));
            if (DOTS && at == i) sdiag[i] = c[k] * scale;
            p[j][k] = (DOTS ? at < i : at <= i) ? x : 0.f;
            if (M::Scaled) most = fmaxf(most, __builtin_fabsf(p[j][k]));
          }
        }
        Scale sc{1.f, 1.f};
        if constexpr (M::Scaled) {
          sc = wave_scale(most);
          if (lane == 0) sback[w] = sc.back;
        }
#pragma unroll
        for (int j = 0; j < IT; ++j) {
          if (j > w) break;
          float left[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) left[k] = p[j][k] * sc.by;
#pragma unroll
          for (int m = 0; m < NP; ++m) {
            Pack<T, 4> x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x.v[k] = T(left[k]);
              left[k] -= float(x.v[k]);
            }
            *reinterpret_cast<Pack<T, 4>*>(&sp[m][i][16 * j + 4 * g]) = x;
          }
        }
      }
      __syncthreads();
    }
    // v by steps: this lane's column, eight steps of each 32
    Op fv[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) fv[s] = op_column<T>(&sv[0][0], VP, 32 * s + 8 * g, 16 * w, q);

    if constexpr (WALK) {
      // outputs of step 16 i + q, columns cw + 4 g + (0..3): the state's part, then the chunk's
      f32x4 y[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i) y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      Scale ss{1.f, 1.f};
      if constexpr (M::Scaled) {
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) most = fmaxf(most, __builtin_fabsf(S[k][i]));
        ss = wave_scale(most);
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = S[2 * k + i / 4][i % 4] * ss.by;
        const Parts<T, NP> fs = op_parts<T, NP>(x);
#pragma unroll
        for (int i = 0; i < IT; ++i)
          y[i] = mul_parts<T, NP>(fs, op_runs<T>(&sa[16 * i + q][32 * k + 4 * g], &sa[16 * i + q][32 * k + 16 + 4 * g]), y[i]);
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const float by = ssince[16 * i + q] * ss.back;
        y[i] *= by;
        f32x4 c = M::Scaled ? f32x4{0.f, 0.f, 0.f, 0.f} : y[i];
#pragma unroll
        for (int s = 0; s < ST; ++s) {
          if (16 * i + 15 < 32 * s) break;
          Parts<T, NP> fp;
#pragma unroll
          for (int m = 0; m < NP; ++m) fp.p[m] = op_run<T>(&sp[m][16 * i + q][32 * s + 8 * g]);
          c = mul_parts<T, NP>(fv[s], fp, c);
        }
        if constexpr (M::Scaled) {
          const float back = sback[i];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][k] = __builtin_fmaf(c[k], back, y[i][k]);
        } else {
          y[i] = c;
        }
      }
      float dots[IT];
      if constexpr (DOTS) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int u = 16 * i + q, c = cw + 4 * g;
          float d[4] = {};
          if (u < steps) {
            const T* at = reinterpret_cast<const T*>(a.dot.p) + pd + i * 16 * drs;
            if (VEC && c < a.V) {
              const Pack<T, 4> x = *reinterpret_cast<const Pack<T, 4>*>(at);
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] = float(x.v[k]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < a.V) d[k] = float(at[k]);
            }
          }
          const Pack<T, 4> own = *reinterpret_cast<const Pack<T, 4>*>(&sv[u][16 * w + 4 * g]);
          const float by = sdiag[u];
          dots[i] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (c + k < a.V) dots[i] = __builtin_fmaf(y[i][k], d[k], dots[i]);
            y[i][k] = __builtin_fmaf(by, float(own.v[k]), y[i][k]);
          }
        }
      }
      float zero = 0.f;   // (not so once anything is not finite)
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) zero = __builtin_fmaf(y[i][k], 0.f, zero);
      fine = __builtin_amdgcn_ballot_w64(zero != 0.f) == 0;
      if (fine) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int u = 16 * i + q, c = cw + 4 * g;
          if (a.out.p && u < steps && c < a.V) {
            const int64_t at = po + i * 16 * ors;
            if (a.out_f32) {
              float* o = reinterpret_cast<float*>(a.out.p) + at;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < a.V) o[k] = y[i][k];
            } else if (VEC) {
              Pack<T, 4> x;
#pragma unroll
              for (int k = 0; k < 4; ++k) x.v[k] = T(y[i][k]);
              *reinterpret_cast<Pack<T, 4>*>(reinterpret_cast<T*>(a.out.p) + at) = x;
            } else {
              T* o = reinterpret_cast<T*>(a.out.p) + at;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < a.V) o[k] = T(y[i][k]);
            }
          }
          if constexpr (DOTS) {
            dots[i] += __shfl_xor(dots[i], 16, 64);
            dots[i] += __shfl_xor(dots[i], 32, 64);
            if (g == 0) red[w][u] = dots[i];
          }
        }
      } else {
        one_by_one(u0, steps);
      }
    }
    if (fine) {
      // the state after the chunk
      float x[ST][8];
      float most = 0.f;
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const f32x4 l0 = *reinterpret_cast<const f32x4*>(&sleft[32 * s + 8 * g]), l1 = *reinterpret_cast<const f32x4*>(&sleft[32 * s + 8 * g + 4]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[s][i] = float(fv[s][i]) * (i < 4 ? l0[i] : l1[i - 4]);
          if (M::Scaled) most = fmaxf(most, __builtin_fabsf(x[s][i]));
        }
      }
      Scale sc{1.f, 1.f};
      if constexpr (M::Scaled) {
        sc = wave_scale(most);
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[s][i] *= sc.by;
      }
      Parts<T, NU> fx[ST];
#pragma unroll
      for (int s = 0; s < ST; ++s) fx[s] = op_parts<T, NU>(x[s]);
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k) {
        f32x4 c = M::Scaled ? f32x4{0.f, 0.f, 0.f, 0.f} : S[k] * total;
#pragma unroll
        for (int s = 0; s < ST; ++s) c = mul_parts<T, NU>(op_column<T>(&sb[0][0], KP, 32 * s + 8 * g, 16 * k, q), fx[s], c);
        if constexpr (M::Scaled) {
#pragma unroll
          for (int i = 0; i < 4; ++i) S[k][i] = __builtin_fmaf(S[k][i], total, c[i] * sc.back);
        } else {
          S[k] = c;
        }
      }
    }
    if (u0 + TC < n) sums();
    po += TC * ors;
    pd += TC * drs;
  }
  if constexpr (!WALK) {
    // (what the products make of values that are not finite, the steps decide)
    bool fine = true;
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) fine = fine && finite(S[k][i]);
    if (__builtin_amdgcn_ballot_w64(!fine) != 0) {
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k) S[k] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int u = 0; u < n; ++u) {
        const int64_t row = r.row(u);
        const float dec = __builtin_amdgcn_exp2f(r.log_decay(u) * kLog2e), v = col ? r.get(a.v, a.V, row, cw + q) : 0.f;
        const int rows = afresh(a.K - 4 * g);
#pragma unroll
        for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * k + i < rows) S[k][i] = __builtin_fmaf(r.get(a.b, a.K, row, 16 * k + 4 * g + i) * a.in_scale, v, S[k][i] * dec);
      }
    }
    float* to = a.starts + (int64_t(bh) * a.pieces + piece) * KV;
    const int rows = rows_of();
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * k + i < rows) to[state_at(k, i)] = S[k][i];
    if (t == 0 && slice == 0) a.totals[int64_t(bh) * a.pieces + piece] = __builtin_amdgcn_exp2f(float(all));
    return;
  }
  if (a.fin && (a.back ? piece == 0 : lo < L ? hi == L : piece == 0 && L == 0)) {
    const float by = a.back && L > 0 ? __builtin_amdgcn_exp2f(r.first_decay() * kLog2e) : 1.f;
    float* to = a.fin + bh * KV;
    const int rows = rows_of();
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * k + i < rows) to[state_at(k, i)] = S[k][i] * by;
  }
  if constexpr (DOTS) {
    __syncthreads();
    if (n > 0) put_dots((n - 1) / TC * TC);
    if (a.ends) {   // the state after the piece by the gradient of the one before the next
      float d = 0.f;
      const float* other = a.others ? a.others + (int64_t(bh) * a.pieces + piece) * KV : a.other ? a.other + bh * KV : nullptr;
      const int rows = other ? rows_of() : 0;
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * k + i < rows) d = __builtin_fmaf(S[k][i], other[state_at(k, i)], d);
#pragma unroll
      for (int m = 1; m < 64; m *= 2) d += __shfl_xor(d, m, 64);
      __syncthreads();
      if (lane == 0) red[w][0] = d;
      __syncthreads();
      const float by = hi > 0 && hi < L ? __builtin_amdgcn_exp2f(r.log_decay_at(hi) * kLog2e) : 1.f;
      if (t == 0)
        a.ends[(int64_t(slice) * a.geo.B * a.H + bh) * a.pieces + piece] = by * (((red[0][0] + red[1][0]) + red[2][0]) + red[3][0]);
    }
  }
  // steps that the row does not take
  if (a.out.p)
    for (int s = max(lo, L) + w; s < end; s += 4)
      if (c0 + lane < a.V) r.put(dead_row(a.geo, b, s), c0 + lane, 0.f);
}

template <typename T, int MODE, bool VEC>
hipError_t attn_chunks_of(const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.H * ((a.V + kAttnCols - 1) / kAttnCols) * (MODE == kAttnLocal ? a.pieces - 1 : a.pieces);
  if (a.K <= 32) return go(attn_chunk_kernel<T, 1, MODE, VEC>, blocks, 256, a, s);
  if (a.K <= 64) return go(attn_chunk_kernel<T, 2, MODE, VEC>, blocks, 256, a, s);
  if (a.K <= 128) return go(attn_chunk_kernel<T, 4, MODE, VEC>, blocks, 256, a, s);
  return go(attn_chunk_kernel<T, 8, MODE, VEC>, blocks, 256, a, s);
}

template <typename T>
hipError_t attn_chunks(const AttnArgs& a, bool local, hipStream_t s) {
  const auto whole = [](const HeadRows& x, int size) {
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.rs * sizeof(T) % 16 == 0 && size * sizeof(T) % 16 == 0;
  };
  // (outputs of 32 bits are stored one by one)
  const bool vec = whole(a.b, a.K) && whole(a.v, a.V) && (local || whole(a.a, a.K)) && (!a.dots || whole(a.dot, a.V)) &&
                   (local || !a.out.p || a.out_f32 || whole(a.out, a.V));
  if (local) return vec ? attn_chunks_of<T, kAttnLocal, true>(a, s) : attn_chunks_of<T, kAttnLocal, false>(a, s);
  if (a.dots) return vec ? attn_chunks_of<T, kAttnDots, true>(a, s) : attn_chunks_of<T, kAttnDots, false>(a, s);
  return vec ? attn_chunks_of<T, kAttnWalk, true>(a, s) : attn_chunks_of<T, kAttnWalk, false>(a, s);
}

}  // namespace
}  // namespace rnnhip
