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
// A workgroup takes 64 columns of v and out.  Four of its waves hold all rows of
// the state for 16 of them each, in registers as the products leave them: a
// product's result has four neighbouring rows a lane, which is an operand of the
// next product when the rows of a 32-deep step are taken as 4 g + (0..3) and 16 +
// 4 g + (0..3) by lane group g.  The other four bring the next chunk's rows to
// shared memory, with those of two chunks more on their way in registers, and make
// its scores, while the first four walk this one: two barriers a chunk, one where
// the rows are there and one where the scores are.  b and v by steps (the second
// product and the fourth) are read from shared memory by the transposing reads.
//
// The state is in f32 and never leaves the registers inside a piece of the time
// axis.  No unit is busy for the whole of a chunk's time (64 steps, heads of 128 x
// 128, bf16: 3.1 us, 8 x 1024 steps of 16 heads 51 us): shared memory 42 clocks of
// 100, vector instructions, most of them the splitting of 32-bit values below, 40,
// the matrix units 26.  In the rest the waves, one of each role a SIMD, wait for what
// they read and for each other at the barriers.  All eight waves doing both with one
// chunk of rows ahead took 97 us.
//
// Values of 32 bits (scores, state, decayed v) enter a product of 16-bit operands
// in parts: bf16 two for the scores and the state (2^-16 of each), three (2^-24)
// for what is summed into the state or into the decays' gradient; f16 two (2^-22),
// scaled by a power of two, since f16 has neither the state's range nor the
// scores': each step's scores to their largest, each column of the state and of the
// decayed v to its own (one scale for a block of steps or for sixteen columns took
// the digits of those beside a large one), and what the first part leaves once more
// by itself, so that the smaller values of a column keep theirs, too: 2^-22 of
// each value down to 2^-28 of the largest, and 2^-50 of that below.  f32 uses the
// f32 matrix cores.
//
// A masked score is a zero, but a zero times a later step's infinity or NaN is
// not; and an infinite value has no parts.  A wave whose chunk has an output that
// is not finite goes back to the steps one by one.
#pragma once

#include <type_traits>

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
// state, Fine ones of what is summed on.  Values between rows in shared memory, 16
// bits (clocks that a wave's read takes the memory, measured): b's and the scores'
// rows, read 16 bytes a lane, a multiple of 32 and 16 (4; with 8: 8; 32), a's,
// read in runs of 8 bytes, and 4 (4; with 8: 8, with 16: 16), v's, and b's too, by
// the transposing reads, and 8 or 16 (4; none: 16).
template <typename T>
struct Mma;

template <>
struct Mma<bf16_t> {
  static constexpr int Coarse = 2, Fine = 3, Vec = 8, PadA = 4, PadB = 16, PadV = 8;
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
  static constexpr int Coarse = 2, Fine = 2, Vec = 8, PadA = 4, PadB = 16, PadV = 8;
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
  static constexpr int Coarse = 1, Fine = 1, Vec = 4, PadA = 4, PadB = 4, PadV = 4;
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

// Two values as 16 bits each, and what that leaves of them.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
constexpr float kLeft = 8192.f;   // f16: what is left of 2^14, 4 at most, fills the type's range, too
__device__ __forceinline__ uint32_t take_pair(f32x2& x, bf16_t) {
  const uint32_t k = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  x[0] -= __builtin_bit_cast(float, k << 16);
  x[1] -= __builtin_bit_cast(float, k & 0xffff0000u);
  return k;
}
__device__ __forceinline__ uint32_t take_pair(f32x2& x, f16_t) {
  const f16x2 k = __builtin_convertvector(x, f16x2);
  x[0] = __builtin_fmaf(float(k[0]), -1.f, x[0]) * kLeft;
  x[1] = __builtin_fmaf(float(k[1]), -1.f, x[1]) * kLeft;
  return __builtin_bit_cast(uint32_t, k);
}

// N parts of eight values of 32 bits (f16: the second times kLeft, which its
// products are summed with apart).
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
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 k[N];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x2 left = {x[2 * i], x[2 * i + 1]};
#pragma unroll
      for (int n = 0; n < N; ++n) k[n][i] = take_pair(left, T());
    }
#pragma unroll
    for (int n = 0; n < N; ++n) r.p[n] = __builtin_bit_cast(typename Mma<T>::Op, k[n]);
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ f32x4 mul_parts(const typename Mma<T>::Op& a, const Parts<T, N>& b, f32x4 c) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) c = Mma<T>::mul(a, b.p[n], c);
  return c;
}
// The sum of products by first parts and that by second ones.
__device__ __forceinline__ f32x4 with_left(f32x4 c, const f32x4& left) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(left[i], 1.f / kLeft, c[i]);
  return c;
}

// The power of two that takes the largest magnitude, m, of the values of the four
// lanes that share a place among sixteen to 2^13 to 2^14, and its inverse (1 for a
// zero, and for what is not finite).
struct Scale {
  float by, back;
};
__device__ __forceinline__ Scale lane_scale(float m) {
  auto of = [&](auto p) {
    const float x = __builtin_bit_cast(float, uint32_t(p[0])), y = __builtin_bit_cast(float, uint32_t(p[1]));
    m = x > y ? x : y;
  };
  of(__builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, m), false, false));
  of(__builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, m), false, false));
  int e = __builtin_bit_cast(int, m) >> 23;
  e = e == 0 || e >= 255 ? 140 : max(e, 14);
  return {__builtin_bit_cast(float, (267 - e) << 23), __builtin_bit_cast(float, (e - 13) << 23)};
}

// A sum over the lanes up to each one, without shared memory.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_before(double x) {
  const uint64_t k = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(k)), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(k >> 32)), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double lanes_up_to(double x) {
  x += lanes_before<0x111, 0xf>(x);   // by 1, 2, 4, 8 within sixteen
  x += lanes_before<0x112, 0xf>(x);
  x += lanes_before<0x114, 0xf>(x);
  x += lanes_before<0x118, 0xf>(x);
  x += lanes_before<0x142, 0xa>(x);   // the last of the sixteen before
  x += lanes_before<0x143, 0xc>(x);   // and of the half before
  return x;
}

__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

// The value, unknown to the compiler from here on: conditions on it are made where
// they are used.  (Kept from the kernel's start to its end, masks of 64 lanes for
// each row of a state fill the scalar registers.)
__device__ __forceinline__ int afresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Reads of shared memory above stay above: they are under way while the products
// below are made.  (Left to itself the compiler asks for an operand right before
// its use, and every product waits for one.)
__device__ __forceinline__ void asked() { __builtin_amdgcn_sched_barrier(0); }

// The instructions up to the next such mark in the order of N times one product and
// V vector instructions (a product takes the matrix unit four times as long as
// its issue: the vector instructions between cost nothing).
template <int N, int V>
__device__ __forceinline__ void between_products() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
  }
}

enum { kAttnLocal, kAttnWalk, kAttnDots, kAttnSome };

// KT: 32-wide pieces of a and b.  MODE: the state that a piece of the time axis
// leaves from a zero one; the outputs; these with what the decays' gradient
// needs; these, of walks that have some of it.  VEC: rows in aligned 16-byte
// pieces.
template <typename T, int KT, int MODE, bool VEC>
__device__ __forceinline__ void attn_walk(const AttnArgs& a, int id, int blocks) {
  typedef Mma<T> M;
  typedef typename M::Op Op;
  constexpr bool WALK = MODE != kAttnLocal, DOTS = MODE >= kAttnDots;
  const bool dots = MODE == kAttnDots || (MODE == kAttnSome && a.dots);
  constexpr int TC = KT * int(sizeof(T)) >= 16 ? 32 : 64, IT = TC / 16, ST = TC / 32;    // steps of a chunk, in 16s and 32s
  constexpr int COLS = kAttnCols;                                                        // of a workgroup
  constexpr int KA = 32 * KT + M::PadA, KB = 32 * KT + M::PadB, VP = COLS + M::PadV, PP = 32 + M::PadB, PB = ST == 2 ? 6 : 2;
  constexpr int NP = DOTS ? M::Fine : M::Coarse, NU = M::Fine;
  constexpr int CK = 32 * KT / M::Vec, CV = COLS / M::Vec;                               // 16-byte pieces of a row
  constexpr int RK = 256 / CK, RV = 256 / CV;                                            // rows that the threads take at once
  constexpr int NK = (TC + RK - 1) / RK, NV = (TC + RV - 1) / RV;                        // pieces of a thread
  constexpr int AHEAD = sizeof(T) == 4 && KT >= 4 ? 1 : 2;   // (wide rows of f32 fill the registers)
  // two chunks' rows, sums and scores
  __shared__ alignas(16) T sa[2][WALK ? TC : 1][KA];
  __shared__ alignas(16) T sb[2][TC][KB];
  __shared__ alignas(16) T sv[2][TC][VP];
  // scores, 16 steps by 32: those of the first 32 steps for all, those of the next for the last 32
  __shared__ alignas(16) T sp[2][WALK ? NP : 1][WALK ? PB : 1][16][PP];
  __shared__ alignas(16) float shi[2][TC], slo[2][TC], ssince[2][TC], sleft[2][TC], slog[2][TC], sdiag[2][TC], stotal[2], red[4][TC];
  __shared__ float sback[2][WALK && M::Scaled ? PB : 1][16];   // what the scores of a block's steps were scaled by, back
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int t = int(threadIdx.x) & 255, lane = t & 63, q = lane & 15, g = lane >> 4;
  const int sub = a.sub ? a.sub : 1, parts = a.pieces * sub;   // (of a head; what is walked for its state)
  const int slices = (a.V + COLS - 1) / COLS, pieces = WALK ? a.pieces : parts - sub;
  // a die's workgroups (they go to eight in turn) are neighbours: a head's slices share its a and b there
  const int per_die = blocks / 8, rest = blocks % 8, die = id % 8;
  const int block = die * per_die + min(die, rest) + id / 8;
  const int slice = block % slices, bp = block / slices, bh = bp / pieces;
  const int piece = bp - bh * pieces + (!WALK && a.back ? sub : 0);
  const int b = bh / a.H, h = bh - b * a.H;
  const int L = geo_len(a.geo, b);
  const int size = WALK ? a.piece : a.piece / sub;
  const int64_t lo64 = int64_t(piece) * size;
  const int lo = int(min(lo64, int64_t(a.geo.S))), end = int(min(lo64 + size, int64_t(a.geo.S))), hi = min(end, L), n = max(hi - lo, 0);
  const AttnSteps<T> r(a, b, h, L, lo, hi);
  const int c0 = slice * COLS;
  const int64_t KV = int64_t(a.K) * a.V;
  const int64_t way = a.back ? -r.r.step : r.r.step, top = n > 0 ? r.row(0) : 0;
  const bool down = way < 0;   // (the rows of later steps lie below: in one of a reverse layer and a walk back)
  // the place of step u of a chunk among its rows from the lowest
  auto place = [&](int u) { return down ? TC - 1 - u : u; };
  const int chunks = (n + TC - 1) / TC;

  if (w >= 4) {
    // ---- rows into shared memory, and the scores
    __builtin_amdgcn_s_setprio(1);   // (they are few instructions that all waves wait for)
    // The rows of AHEAD chunks, in registers until their place is free (with one
    // chunk's the loads come late).  A thread's rows of a tensor are RK (RV) apart;
    // past the last one it repeats that, and what it got is made zero on the way to
    // shared memory.  VEC: a chunk's lowest row is
    // at a uniform address, a thread's own at an offset of 32 bits.
    typedef Pack<T, M::Vec> Piece;
    const int tk = t / CK, ck = t % CK * M::Vec, tv = t / CV, cv = t % CV * M::Vec;
    struct Walker {
      const T* p;     // of the head, the chunk's lowest row (VEC), or its first
      int64_t rs;     // elements from a step to the next
    };
    auto walker = [&](const HeadRows& x, int size) {
      const int64_t rs = way * x.rs;
      const T* p = reinterpret_cast<const T*>(x.p) + top * x.rs + (h / x.per) * int64_t(size);
      return Walker{p + (VEC && down ? (TC - 1) * rs : 0), rs};
    };
    Walker wa = WALK ? walker(a.a, a.K) : Walker{}, wb = walker(a.b, a.K), wv = walker(a.v, a.V);
    struct Rows {
      Piece a[WALK ? NK : 1], b[NK], v[NV];
    } x[AHEAD];
    auto load = [&](const Walker& from, int u, int left, int size, int c) {
      u = min(u, left);
      Piece p = {};
      if constexpr (VEC) {
        const uint32_t stride = uint32_t(down ? -from.rs : from.rs) * sizeof(T);
        p = *reinterpret_cast<const Piece*>(reinterpret_cast<const char*>(from.p) + (uint32_t(place(u)) * stride + uint32_t(c < size ? c : 0) * uint32_t(sizeof(T))));
      } else if (size >= M::Vec) {   // (past the row's last whole piece: the one that ends it, moved down later)
        __builtin_memcpy(&p, from.p + u * from.rs + min(c, size - M::Vec), sizeof(p));
      } else {   // (heads of a few elements, all in the first piece: one by one, in few registers)
        typedef std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t> Bits;
        unsigned __int128 x = 0;
        const Bits* row = reinterpret_cast<const Bits*>(from.p + u * from.rs);
#pragma unroll 1
        for (int k = size - 1; k >= c; --k) x = x << (8 * int(sizeof(T))) | row[k];
        p = __builtin_bit_cast(Piece, x);
      }
      return p;
    };
    // b and v of the steps from u0 on, and a
    auto fetch_bv = [&](int u0, Rows& x) {
      const int left = min(n - 1 - u0, TC - 1);   // (threads past a chunk's pieces repeat the last, too)
#pragma unroll
      for (int i = 0; i < NK; ++i) x.b[i] = load(wb, tk + i * RK, left, a.K, ck);
#pragma unroll
      for (int i = 0; i < NV; ++i) x.v[i] = load(wv, tv + i * RV, left, a.V, c0 + cv);
      wb.p += TC * wb.rs;
      wv.p += TC * wv.rs;
    };
    auto fetch_a = [&](int u0, Rows& x) {
      if constexpr (WALK) {
        const int left = min(n - 1 - u0, TC - 1);
#pragma unroll
        for (int i = 0; i < NK; ++i) x.a[i] = load(wa, tk + i * RK, left, a.K, ck);
        wa.p += TC * wa.rs;
      }
    };
    // a row's last elements to the piece's begin, and zeros after them
    auto settle = [&](Piece& p, int size, int c) {
      if (size < M::Vec || size % M::Vec == 0 || c + M::Vec <= size) return;
      p = __builtin_bit_cast(Piece, __builtin_bit_cast(unsigned __int128, p) >> ((M::Vec - size % M::Vec) * 8 * int(sizeof(T))));
    };
    auto keep = [&](Piece& p, bool is) {
      if (!is) p = Piece{};
    };
    // The last wave, lane i: the sums of log decays (to base 2) up to step i of the
    // chunk to come, asked for a chunk earlier.
    const bool sums_here = w == 7;
    double all = 0.;   // of the piece
    float rg = 0.f, clog = 0.f, chi = 0.f, clo = 0.f, csince = 0.f, cleft = 0.f, ctotal = 0.f;
    auto later = [&](int u) { return r.step(u) + (a.back ? 1 : 0); };   // (AttnSteps::log_decay)
    auto ask = [&](int u0) {
      if (a.G.p) rg = r.raw_decay(min(later(min(u0 + lane, n - 1)), L - 1));
    };
    auto sums = [&](int u0) {
      const bool is = lane < TC && u0 + lane < n && later(u0 + lane) < L;
      const float x = is ? attn_log_decay(rg + r.fixed) : 0.f;
      clog = x * kLog2e;
      const double sum = lanes_up_to(double(x) * 1.4426950408889634);
      const uint64_t k = __builtin_bit_cast(uint64_t, sum);
      const double whole = __builtin_bit_cast(double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(k >> 32), 63))) << 32 | uint32_t(__builtin_amdgcn_readlane(int(uint32_t(k)), 63)));
      chi = float(sum);
      clo = float(sum - double(chi));
      csince = __builtin_amdgcn_exp2f(chi) * a.out_scale;
      cleft = __builtin_amdgcn_exp2f(float(whole - sum)) * a.in_scale;
      ctotal = __builtin_amdgcn_exp2f(float(whole));
      all += whole;
    };
    // (a's rows of 16 bits begin at eight bytes)
    auto put_a = [&](T* to, const Piece& p) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<Piece*>(to) = p;
      } else {
        *reinterpret_cast<Pack<T, 4>*>(to) = Pack<T, 4>{{p.v[0], p.v[1], p.v[2], p.v[3]}};
        *reinterpret_cast<Pack<T, 4>*>(to + 4) = Pack<T, 4>{{p.v[4], p.v[5], p.v[6], p.v[7]}};
      }
    };
    // what was fetched, of the steps from u0 on, and b and v of AHEAD chunks later asked for
    auto put_rows = [&](int u0, int at, Rows& x) {
      if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          if constexpr (WALK) settle(x.a[i], a.K, ck);
          settle(x.b[i], a.K, ck);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) settle(x.v[i], a.V, c0 + cv);
      }
      if (u0 + TC > n || a.K < 32 * KT || c0 + COLS > a.V) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          if constexpr (WALK) keep(x.a[i], u0 + tk + i * RK < n && ck < a.K);
          keep(x.b[i], u0 + tk + i * RK < n && ck < a.K);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) keep(x.v[i], u0 + tv + i * RV < n && c0 + cv < a.V);
      }
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        if (TC % RK && tk + i * RK >= TC) break;   // (more threads than pieces)
        if constexpr (WALK) put_a(&sa[at][tk + i * RK][ck], x.a[i]);
        *reinterpret_cast<Piece*>(&sb[at][tk + i * RK][ck]) = x.b[i];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (TC % RV && tv + i * RV >= TC) break;
        *reinterpret_cast<Piece*>(&sv[at][tv + i * RV][cv]) = x.v[i];
      }
      if (sums_here && lane < TC) {
        shi[at][lane] = chi;
        slo[at][lane] = clo;
        ssince[at][lane] = csince;
        sleft[at][lane] = cleft;
        slog[at][lane] = clog;
        stotal[at] = ctotal;
      }
      if (u0 + AHEAD * TC < n) fetch_bv(u0 + AHEAD * TC, x);
    };
    // when the scores are made: the rest of those loads, and the next chunk's sums
    // (loads are spread over a chunk's time: they come no faster than the memory has
    // them)
    auto prepare = [&](int u0, Rows& x) {
      if (u0 < n && sums_here) {
        sums(u0);
        ask(u0 + TC);
      }
      if (u0 + (AHEAD - 1) * TC < n) fetch_a(u0 + (AHEAD - 1) * TC, x);
    };
    // The scores of a block: of steps 16 it + q (a lane's) by those of one half of
    // the chunk, zero past step 16 it + q.
    const float scale = a.in_scale * a.out_scale;
    auto scores = [&](int at, int it, int half) {
      const int i = 16 * it + q, j0 = 32 * half, block = it + (half ? 2 : 0);
      constexpr int KG = KT * int(sizeof(T)) > 16 ? 16 / int(sizeof(T)) : KT;   // (more fill the registers)
      f32x4 hj[2], lj[2], c[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        hj[j] = *reinterpret_cast<const f32x4*>(&shi[at][j0 + 16 * j + 4 * g]);
        lj[j] = *reinterpret_cast<const f32x4*>(&slo[at][j0 + 16 * j + 4 * g]);
      }
      const float hi_i = shi[at][i], lo_i = slo[at][i];
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += KG) {
        Op fa[KG], fb[2][KG];
#pragma unroll
        for (int k = 0; k < KG; ++k) fa[k] = op_runs<T>(&sa[at][i][32 * (k0 + k) + 8 * g], &sa[at][i][32 * (k0 + k) + 8 * g + 4]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < KG; ++k) fb[j][k] = op_run<T>(&sb[at][j0 + 16 * j + q][32 * (k0 + k) + 8 * g]);
        asked();
#pragma unroll
        for (int k = 0; k < KG; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) c[j] = M::mul(fb[j][k], fa[k], c[j]);
        asked();
      }
      float p[2][4], most = 0.f, own = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j0 + 16 * j > 16 * it) {   // (past the diagonal)
#pragma unroll
          for (int k = 0; k < 4; ++k) p[j][k] = 0.f;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) p[j][k] = c[j][k] * (scale * __builtin_amdgcn_exp2f((hi_i - hj[j][k]) + (lo_i - lj[j][k])));
          if (j0 + 16 * j == 16 * it)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int to = q - (4 * g + k);   // steps from one to the other
              if (DOTS) own = to == 0 ? c[j][k] * scale : own;
              p[j][k] = to >= (DOTS ? 1 : 0) ? p[j][k] : 0.f;
            }
          if constexpr (M::Scaled)
#pragma unroll
            for (int k = 0; k < 4; ++k) most = fmaxf(most, __builtin_fabsf(p[j][k]));
        }
      }
      Scale sc{1.f, 1.f};
      if constexpr (M::Scaled) {
        sc = lane_scale(most);
        if (g == 0) sback[at][block][q] = sc.back;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        T* to = &sp[at][0][block][q][16 * j + 4 * g];
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<f32x4*>(to) = f32x4{p[j][0], p[j][1], p[j][2], p[j][3]};
        } else {
          f32x2 left[2] = {{p[j][0] * sc.by, p[j][1] * sc.by}, {p[j][2] * sc.by, p[j][3] * sc.by}};
#pragma unroll
          for (int m = 0; m < NP; ++m) {
            uint2 x;
            x.x = take_pair(left[0], T());
            x.y = take_pair(left[1], T());
            *reinterpret_cast<uint2*>(to + m * (PB * 16 * PP)) = x;
          }
        }
      }
      // (a step's own score: where its sixteen is among the block's, of four lanes the one that has it)
      if (DOTS && it / 2 == half && (q >> 2) == g) sdiag[at][i] = own;
    };
    // A wave's blocks (steps, half): 3 0 and 0 0; 1 0; 2 0 and 2 1; 3 1.
    auto all_scores = [&](int at) {
      const int x = w - 4;
      if constexpr (ST == 1) {
        if (x < 2) scores(at, x, 0);
      } else {
        scores(at, x == 0 ? 3 : x, x == 3 ? 1 : 0);
        if ((x & 1) == 0) scores(at, x, x / 2);
      }
    };
    auto put_dots = [&](int u0) {
      if (!dots || t >= TC || u0 + t >= n) return;
      a.dots[((int64_t(slice) * a.geo.B + b) * a.H + h) * a.geo.S + r.step(u0 + t)] = ((red[0][t] + red[1][t]) + red[2][t]) + red[3][t];
    };

    if (n > 0) {
      if (sums_here) ask(0);
      fetch_bv(0, x[0]);
      fetch_a(0, x[0]);
      if (AHEAD == 2 && n > TC) {
        fetch_bv(TC, x[AHEAD - 1]);
        fetch_a(TC, x[AHEAD - 1]);
      }
      if (sums_here) {
        sums(0);
        ask(TC);
      }
      put_rows(0, 0, x[0]);
    }
    __syncthreads();
    if (WALK && n > 0) all_scores(0);
    prepare(TC, x[0]);
    if constexpr (WALK) __syncthreads();
    auto next = [&](int u0, auto AT) {   // the chunk from u0 on, while the one before is walked
      constexpr int at = decltype(AT)::value;
      if (DOTS && u0 > TC) put_dots(u0 - 2 * TC);
      if (u0 < n) put_rows(u0, at, x[at % AHEAD]);
      if constexpr (WALK) {
        __syncthreads();
        if (u0 < n) all_scores(at);
      }
      prepare(u0 + TC, x[at % AHEAD]);
      __syncthreads();
    };
    for (int c = 0; c < chunks; c += 2) {
      next((c + 1) * TC, std::integral_constant<int, 1>{});
      if (c + 1 < chunks) next((c + 2) * TC, std::integral_constant<int, 0>{});
    }
    if (DOTS && chunks > 0) put_dots((chunks - 1) * TC);
    if (!WALK && sums_here && lane == 0 && slice == 0) a.totals[int64_t(bh) * parts + piece] = __builtin_amdgcn_exp2f(float(all));
    if constexpr (DOTS)
      if (a.ends) {
        __syncthreads();
        __syncthreads();
      }
    return;
  }

  // ---- the state and the outputs: rows 16 k + 4 g + (0..3), column c0 + 16 w + q
  f32x4 S[2 * KT];
  const int cw = 16 * w, column = c0 + cw + q;
  auto state_at = [&](int k, int i) { return int64_t(16 * k + 4 * g + i) * a.sk + int64_t(column) * a.sv; };
  // rows that there are among 4 g + (0..3) on (none without a column): for k, i those below
  auto rows_of = [&] { return afresh(column < a.V ? a.K - 4 * g : 0); };
  {
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k) S[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int rows = rows_of();
    auto add = [&](const float* start, float total) {   // (past the last row or column: some other, made zero)
      const float* from = start + int64_t(min(column, a.V - 1)) * a.sv;
      f32x4 x[2 * KT];
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = from[min(16 * k + 4 * g + i, a.K - 1) * a.sk];
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[k][i] = 16 * k + i < rows ? __builtin_fmaf(S[k][i], total, x[k][i]) : 0.f;
    };
    if constexpr (WALK) {
      if (a.pieces > 1 && a.sub == 0) {
        add(a.starts + (int64_t(bh) * parts + piece) * KV, 1.f);
      } else {
        if (a.init) add(a.init + bh * KV, 1.f);
        const int before = (a.back ? a.pieces - 1 - piece : piece) * a.sub;
        for (int k = 0; k < before; ++k) {
          const int64_t at = int64_t(bh) * parts + (a.back ? parts - 1 - k : k);
          add(a.starts + at * KV, a.totals[at]);
        }
      }
    }
  }
  // a chunk's outputs, and the rows that they are multiplied with
  const int64_t ors = way * a.out.rs, drs = way * a.dot.rs;
  const int oes = a.out_f32 ? 4 : int(sizeof(T));
  char* po = a.out.p ? a.out.p + (top * a.out.rs + (h / a.out.per) * int64_t(a.V) + (VEC && down ? (TC - 1) * ors : 0)) * oes : nullptr;
  const T* pd = dots ? reinterpret_cast<const T*>(a.dot.p) + top * a.dot.rs + (h / a.dot.per) * int64_t(a.V) + (VEC && down ? (TC - 1) * drs : 0) : nullptr;

  // The steps of the chunk one by one, from shared memory.
  auto one_by_one = [&](int u0, int steps, int at) {
    for (int u = 0; u < steps; ++u) {
      const float dec = __builtin_amdgcn_exp2f(slog[at][u]);
      const int64_t row = r.row(u0 + u);
      const float v = float(sv[at][u][cw + q]);
      float off = 0.f, y = 0.f;
      const int rows = afresh(a.K - 4 * g);
#pragma unroll
      for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 16 * k + 4 * g + i;
          if (16 * k + i < rows) {
            S[k][i] *= dec;
            if constexpr (WALK) off = __builtin_fmaf(float(sa[at][u][d]), S[k][i], off);
            S[k][i] = __builtin_fmaf(float(sb[at][u][d]) * a.in_scale, v, S[k][i]);
            if constexpr (WALK) y = __builtin_fmaf(float(sa[at][u][d]), S[k][i], y);
          }
        }
      y += __shfl_xor(y, 16, 64);
      y += __shfl_xor(y, 32, 64);
      if (g == 0 && column < a.V) r.put(row, column, y * a.out_scale);
      if constexpr (DOTS) {
        off += __shfl_xor(off, 16, 64);
        off += __shfl_xor(off, 32, 64);
        float dot = dots && column < a.V ? off * a.out_scale * r.get(a.dot, a.V, row, column) : 0.f;
#pragma unroll
        for (int m = 1; m < 16; m *= 2) dot += __shfl_xor(dot, m, 64);
        if (lane == 0) red[w][u] = dot;
      }
    }
  };

  __syncthreads();
  if constexpr (WALK) __syncthreads();
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int u0 = chunk * TC, at = chunk & 1, steps = min(n - u0, TC);
    // the rows that the outputs are multiplied with, on their way until then
    Pack<T, 4> dx[DOTS && VEC ? IT : 1];
    if (DOTS && VEC && dots) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = c0 + cw + 4 * g;   // (past the last step: that one again)
        const uint32_t off = uint32_t(place(min(16 * i + q, steps - 1))) * uint32_t(down ? -drs : drs) + uint32_t(c < a.V ? c : 0);
        dx[i] = *reinterpret_cast<const Pack<T, 4>*>(reinterpret_cast<const char*>(pd) + off * uint32_t(sizeof(T)));
      }
    }
    // v by steps: this lane's column, eight steps of each 32
    Op fv[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) fv[s] = op_column<T>(&sv[at][0][0], VP, 32 * s + 8 * g, cw, q);

    // outputs of step 16 i + q, columns c0 + cw + 4 g + (0..3): the state's part, then the chunk's
    f32x4 y[IT];
    bool fine = true;
    if constexpr (WALK) {
#pragma unroll
      for (int i = 0; i < IT; ++i) y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      f32x4 z[M::Scaled ? IT : 1];   // of second parts
#pragma unroll
      for (int i = 0; i < (M::Scaled ? IT : 1); ++i) z[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      Scale ss{1.f, 1.f};   // of this lane's column
      float back[4];        // of the outputs' columns
      if constexpr (M::Scaled) {
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) most = fmaxf(most, __builtin_fabsf(S[k][i]));
        ss = lane_scale(most);
#pragma unroll
        for (int i = 0; i < 4; ++i) back[i] = __shfl(ss.back, 4 * g + i, 16);
      }
      Op fa[2][IT];
      auto read_a = [&](int k) {
#pragma unroll
        for (int i = 0; i < IT; ++i) fa[k & 1][i] = op_runs<T>(&sa[at][16 * i + q][32 * k + 4 * g], &sa[at][16 * i + q][32 * k + 16 + 4 * g]);
      };
      constexpr int BL = ST == 2 ? 6 : 2;   // blocks of scores: i = 0 1 2 2 3 3, s = 0 0 0 1 0 1
      Parts<T, NP> fp[3];
      float since[IT];
      auto read_p = [&](int m) {
        const int i = m < 2 ? m : (m - 2) / 2 + 2, s = m < 2 ? 0 : m & 1;
#pragma unroll
        for (int x = 0; x < NP; ++x) fp[m % 3].p[x] = op_run<T>(&sp[at][x][s ? i + 2 : i][q][8 * g]);
      };
      auto state_parts = [&](int k) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = S[2 * k + i / 4][i % 4] * ss.by;
        return op_parts<T, NP>(x);
      };
      read_a(0);
      Parts<T, NP> fs = state_parts(0);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        if (k + 1 < KT) {
          read_a(k + 1);
        } else {
          read_p(0);
          read_p(1);
#pragma unroll
          for (int i = 0; i < IT; ++i) since[i] = ssince[at][16 * i + q];
        }
        asked();
#pragma unroll
        for (int m = NP - 1; m >= 0; --m)
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            f32x4& to = M::Scaled && m == 1 ? z[M::Scaled ? i : 0] : y[i];
            to = M::mul(fs.p[m], fa[k & 1][i], to);
          }
        if (k + 1 < KT) fs = state_parts(k + 1);
        if constexpr (sizeof(T) == 2) between_products<NP * IT, 3>();
        asked();
      }
#pragma unroll
      for (int m = 0; m < BL; ++m) {
        const int i = m < 2 ? m : (m - 2) / 2 + 2, s = m < 2 ? 0 : m & 1;
        if (m + 2 < BL) read_p(m + 2);
        asked();
        if constexpr (M::Scaled) {
          const f32x4 left = M::mul(fv[s], fp[m % 3].p[1], f32x4{0.f, 0.f, 0.f, 0.f});
          const f32x4 c = with_left(M::mul(fv[s], fp[m % 3].p[0], f32x4{0.f, 0.f, 0.f, 0.f}), left);
          const float by = sback[at][s ? i + 2 : i][q];
          if (s == 0) y[i] = with_left(y[i], z[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][k] = __builtin_fmaf(c[k], by, s == 0 ? y[i][k] * (since[i] * back[k]) : y[i][k]);
        } else {
          if (s == 0) y[i] *= since[i];
          y[i] = mul_parts<T, NP>(fv[s], fp[m % 3], y[i]);
        }
      }
      __syncthreads();   // (the next chunk's rows are there)
      if constexpr (DOTS) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int u = 16 * i + q, c = c0 + cw + 4 * g;
          const float by = sdiag[at][u];
          float d[4] = {};
          if (dots && u < steps) {
            if (VEC) {
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] = float(dx[i].v[k]);
            } else if (c + 4 <= a.V) {
              T x[4];
              __builtin_memcpy(x, pd + u * drs + c, sizeof(x));
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] = float(x[k]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < a.V) d[k] = float(pd[u * drs + c + k]);
            }
          }
          const Pack<T, 4> own = *reinterpret_cast<const Pack<T, 4>*>(&sv[at][u][cw + 4 * g]);
          float dot = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (c + k < a.V) dot = __builtin_fmaf(y[i][k], d[k], dot);
            y[i][k] = __builtin_fmaf(by, float(own.v[k]), y[i][k]);
          }
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (g == 0) red[w][u] = dot;
        }
      }
      float zero = 0.f;   // (not so once anything is not finite)
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) zero = __builtin_fmaf(y[i][k], 0.f, zero);
      fine = __builtin_amdgcn_ballot_w64(zero != 0.f) == 0;
    }
    if (__builtin_expect(fine, 1)) {
      // the state after the chunk; the outputs on their way between
      const float total = stotal[at];
      f32x4 left[2 * ST];
#pragma unroll
      for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) left[2 * s + i] = *reinterpret_cast<const f32x4*>(&sleft[at][32 * s + 8 * g + 4 * i]);
      constexpr int J = KT >= 4 && sizeof(T) == 2 ? 4 : 2;   // sixteens of rows multiplied at once
      Op fb[2][J][ST];   // theirs, while those before are multiplied
      auto read_b = [&](int k) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int s = 0; s < ST; ++s) fb[k & 1][j][s] = op_column<T>(&sb[at][0][0], KB, 32 * s + 8 * g, 16 * (J * k + j), q);
      };
      read_b(0);
      asked();
      if constexpr (WALK) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int u = 16 * i + q, c = c0 + cw + 4 * g;
          if (po && u < steps && c < a.V) {
            if constexpr (VEC) {   // (whole pieces of four columns)
              char* to = po + (uint32_t(place(u)) * uint32_t(down ? -ors : ors) + uint32_t(c)) * uint32_t(oes);
              if (a.out_f32) {
                *reinterpret_cast<f32x4*>(to) = y[i];
              } else {
                Pack<T, 4> x;
#pragma unroll
                for (int k = 0; k < 4; ++k) x.v[k] = T(y[i][k]);
                *reinterpret_cast<Pack<T, 4>*>(to) = x;
              }
            } else if (c + 4 <= a.V) {
              char* to = po + (u * ors + c) * oes;
              if (a.out_f32) {
                __builtin_memcpy(to, &y[i], 16);
              } else {
                T x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = T(y[i][k]);
                __builtin_memcpy(to, x, sizeof(x));
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < a.V) {
                  char* to = po + (u * ors + c + k) * oes;
                  if (a.out_f32) *reinterpret_cast<float*>(to) = y[i][k];
                  else *reinterpret_cast<T*>(to) = T(y[i][k]);
                }
            }
          }
        }
      }
      Scale sc{1.f, 1.f};
      auto value = [&](int s, int i) { return float(fv[s][i]) * left[2 * s + i / 4][i % 4]; };
      if constexpr (M::Scaled) {
        float most = 0.f;
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) most = fmaxf(most, __builtin_fabsf(value(s, i)));
        sc = lane_scale(most);
      }
      auto value_parts = [&](int s) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = value(s, i) * sc.by;
        return op_parts<T, NU>(x);
      };
      Parts<T, NU> fx[ST];
      fx[0] = value_parts(0);
#pragma unroll
      for (int k = 0; k < 2 * KT / J; ++k) {
        if (k + 1 < 2 * KT / J) read_b(k + 1);
        asked();
        f32x4 c[J], z[M::Scaled ? J : 1];   // (second parts' apart)
#pragma unroll
        for (int j = 0; j < J; ++j) c[j] = M::Scaled ? f32x4{0.f, 0.f, 0.f, 0.f} : S[J * k + j] * total;
#pragma unroll
        for (int j = 0; j < (M::Scaled ? J : 1); ++j) z[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < ST; ++s) {
#pragma unroll
          for (int m = NU - 1; m >= 0; --m)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              f32x4& to = M::Scaled && m == 1 ? z[M::Scaled ? j : 0] : c[j];
              to = M::mul(fb[k & 1][j][s], fx[s].p[m], to);
            }
          if (ST == 2 && s == 0 && k == 0) {
            fx[ST - 1] = value_parts(ST - 1);
            if constexpr (sizeof(T) == 2) between_products<NU * J, 4>();
            asked();
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if constexpr (M::Scaled) {
            c[j] = with_left(c[j], z[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) S[J * k + j][i] = __builtin_fmaf(S[J * k + j][i], total, c[j][i] * sc.back);
          } else {
            S[J * k + j] = c[j];
          }
        }
      }
    } else {
      one_by_one(u0, steps, at);
    }
    if (po) po += TC * ors * oes;
    if (dots) pd += TC * drs;
    __syncthreads();   // (the next chunk's scores are there, this one's rows are done with)
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
        const float dec = __builtin_amdgcn_exp2f(r.log_decay(u) * kLog2e), v = column < a.V ? r.get(a.v, a.V, row, column) : 0.f;
        const int rows = afresh(a.K - 4 * g);
#pragma unroll
        for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * k + i < rows) S[k][i] = __builtin_fmaf(r.get(a.b, a.K, row, 16 * k + 4 * g + i) * a.in_scale, v, S[k][i] * dec);
      }
    }
    float* to = a.starts + (int64_t(bh) * parts + piece) * KV;
    const int rows = rows_of();
#pragma unroll
    for (int k = 0; k < 2 * KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * k + i < rows) to[state_at(k, i)] = S[k][i];
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
  if constexpr (DOTS)
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
      __syncthreads();   // (the last chunk's sums are read)
      if (lane == 0) red[w][0] = d;
      __syncthreads();
      const float by = hi > 0 && hi < L ? __builtin_amdgcn_exp2f(r.log_decay_at(hi) * kLog2e) : 1.f;
      if (t == 0)
        a.ends[(int64_t(slice) * a.geo.B * a.H + bh) * a.pieces + piece] = by * (((red[0][0] + red[1][0]) + red[2][0]) + red[3][0]);
    }
  // steps that the row does not take
  if (a.out.p)
    for (int s = max(lo, L) + w; s < end; s += 4)
      if (c0 + lane < a.V) r.put(dead_row(a.geo, b, s), c0 + lane, 0.f);
}

template <typename T, int KT, int MODE, bool VEC>
__global__ __launch_bounds__(512, 2) void attn_chunk_kernel(AttnArgs a) {
  attn_walk<T, KT, MODE, VEC>(a, int(blockIdx.x), int(gridDim.x));
}

// Walks that do not fill the chip by themselves, side by side.
template <typename T, int KT, bool VEC>
__global__ __launch_bounds__(512, 2) void attn_walks_kernel(AttnWalks) {
  // (read where they lie: a copy of which one is chosen by index goes by memory)
  const AttnWalks& s = *(const AttnWalks*)__builtin_amdgcn_kernarg_segment_ptr();
  const int id = int(blockIdx.x), k = (id >= s.first[1]) + (id >= s.first[2]);
  attn_walk<T, KT, kAttnSome, VEC>(s.w[k], id - s.first[k], s.first[k + 1] - s.first[k]);
}

template <typename T, int MODE, bool VEC>
hipError_t attn_chunks_of(const AttnArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.H * ((a.V + kAttnCols - 1) / kAttnCols) * (MODE == kAttnLocal ? (a.pieces - 1) * (a.sub ? a.sub : 1) : a.pieces);
  if (a.K <= 32) return go(attn_chunk_kernel<T, 1, MODE, VEC>, blocks, 512, a, s);
  if (a.K <= 64) return go(attn_chunk_kernel<T, 2, MODE, VEC>, blocks, 512, a, s);
  if (a.K <= 128) return go(attn_chunk_kernel<T, 4, MODE, VEC>, blocks, 512, a, s);
  return go(attn_chunk_kernel<T, 8, MODE, VEC>, blocks, 512, a, s);
}

// Rows in whole aligned pieces, a chunk's within 2^31 bytes (2^25 a step).
template <typename T>
bool attn_whole(const AttnArgs& a, bool local) {
  const auto whole = [&](const HeadRows& x, int size, size_t es) {
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.rs * es % 16 == 0 && size * sizeof(T) % 16 == 0 &&
           x.rs * es <= (size_t(1) << 25) / (a.geo.layout ? 1 : a.geo.B);
  };
  return whole(a.b, a.K, sizeof(T)) && whole(a.v, a.V, sizeof(T)) && (local || whole(a.a, a.K, sizeof(T))) &&
         (!a.dots || whole(a.dot, a.V, sizeof(T))) && (local || !a.out.p || whole(a.out, a.V, a.out_f32 ? 4 : sizeof(T)));
}

template <typename T>
hipError_t attn_chunks(const AttnArgs& a, bool local, hipStream_t s) {
  const bool vec = attn_whole<T>(a, local);
  if (local) return vec ? attn_chunks_of<T, kAttnLocal, true>(a, s) : attn_chunks_of<T, kAttnLocal, false>(a, s);
  if (a.dots) return vec ? attn_chunks_of<T, kAttnDots, true>(a, s) : attn_chunks_of<T, kAttnDots, false>(a, s);
  return vec ? attn_chunks_of<T, kAttnWalk, true>(a, s) : attn_chunks_of<T, kAttnWalk, false>(a, s);
}

template <typename T, bool VEC>
hipError_t attn_walks_of(const AttnWalks& w, int K, hipStream_t s) {
  const int64_t blocks = w.first[3];
  if (K <= 32) return go(attn_walks_kernel<T, 1, VEC>, blocks, 512, w, s);
  if (K <= 64) return go(attn_walks_kernel<T, 2, VEC>, blocks, 512, w, s);
  if (K <= 128) return go(attn_walks_kernel<T, 4, VEC>, blocks, 512, w, s);
  return go(attn_walks_kernel<T, 8, VEC>, blocks, 512, w, s);
}

template <typename T>
hipError_t attn_walks(const AttnArgs* w, int n, int K, hipStream_t s) {
  AttnWalks all{};
  bool vec = true;
  for (int k = 0; k < n; ++k) {
    const AttnArgs& a = all.w[k] = w[k];
    all.first[k + 1] = all.first[k] + a.geo.B * a.H * ((a.V + kAttnCols - 1) / kAttnCols) * a.pieces;
    vec = vec && attn_whole<T>(a, false);
  }
  for (int k = n; k < 3; ++k) all.first[k + 1] = all.first[k];
  return vec ? attn_walks_of<T, true>(all, K, s) : attn_walks_of<T, false>(all, K, s);
}

}  // namespace
}  // namespace rnnhip
