// scan_device.h -- what the selective scan's kernels share: a workgroup's
// place, a lane's share of states, B and C in the lanes of a wave, the join of
// chunks.  Internal.
//
// A workgroup takes 64 channels of one batch row and group, a lane a channel,
// and its NW waves NS states each: state w*NS + i of wave w.  B and C are then
// the same for a whole wave; the lanes of a row of 16 hold them and share them
// as operands through the DPP crossbar (BCTile).
#pragma once

#include "seq_device.h"

namespace rnnhip {

template <int J>
struct IntC { static constexpr int value = J; };
// f(0), f(1), ... f(K-1), each with its number known to the compiler
template <int K, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < K) {
    f(IntC<I>{});
    each<K, I + 1>(f);
  }
}

// The work of workgroup `blockIdx.x` as a number in the order channel block,
// chunk, batch row: its own number, or (`fold`) every second round of 256, one
// a compute unit, in falling order.  (Giving a die's workgroups neighbouring
// channel blocks instead made no difference, 191.5 and 191.3 us: a block's 64
// channels are whole cache lines that no other reads.)
__device__ __forceinline__ int scan_order(bool fold) {
  const int blk = int(blockIdx.x), base = blk / 256 * 256, n = min(256, int(gridDim.x) - base);
  return fold && (base & 256) ? base + (n - 1 - (blk - base)) : blk;
}

// The batch row of rank `rank` by falling length (ties by number).  Uniform; up
// to 256 rows, at least as many threads.
__device__ __forceinline__ int scan_row_of_rank(const ScanArgs& a, int rank) {
  __shared__ int lens[256];
  __shared__ int found;
  const int B = a.geo.B, tid = int(threadIdx.x);
  int len = -1;
  if (tid < B) {
    len = a.geo.lens[tid];
    len = len < 0 ? 0 : (len > a.geo.S ? a.geo.S : len);
    lens[tid] = len;
  }
  __syncthreads();
  if (tid < B) {
    int before = 0;
    for (int j = 0; j < B; ++j) before += lens[j] > len || (lens[j] == len && j < tid);
    if (before == rank) found = tid;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(found);
}

// A workgroup's work.  A lane past its group's channels takes the last one's
// states and weights, with inputs that are some other channel's or zero: what it
// computes is stored nowhere.
struct ScanPlace {
  int b, ch, g, cb;   // batch row, chunk, group, channel block of all groups
  unsigned c;         // channel
  bool ok;
};
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a, int nchunk, int lane) {
  ScanPlace p;
  const int nb = a.G * a.cbg;
  const int i = scan_order(a.balance);
  p.cb = i % nb;
  const int rest = i / nb;
  p.ch = rest % nchunk;
  p.b = rest / nchunk;
  // Rows of unequal length: by falling length, and with every second round
  // turned a compute unit that got a long row gets a short one next.  (16 rows
  // of all lengths up to 1024 by 2048 channels: 125.6 us, as stored 147.6.)
  if (a.balance) p.b = scan_row_of_rank(a, p.b);
  p.g = p.cb / a.cbg;
  const int in = (p.cb % a.cbg) * 64 + lane;
  p.ok = in < a.cpg;
  p.c = p.g * a.cpg + (p.ok ? in : a.cpg - 1);
  return p;
}

// States [n0, n0 + NS) of one channel of a caller's tensor [..][N]; states past
// N are 0 and stay 0.
template <int NS>
__device__ __forceinline__ void scan_load_state(const ScanArgs& a, const float* t, int64_t chan, int n0, float (&v)[NS]) {
  const float* p = t + chan * a.N;
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = t && n0 + i < a.N ? p[n0 + i] : 0.f;
}
template <int NS>
__device__ __forceinline__ void scan_store_state(const ScanArgs& a, float* t, int64_t chan, int n0, const float (&v)[NS]) {
  float* p = t + chan * a.N;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (n0 + i < a.N) p[n0 + i] = v[i];
}
// States in scratch: [..][NP][C], so that a wave's lanes lie together.
template <int NS>
__device__ __forceinline__ void scan_get(const ScanArgs& a, const float* t, int64_t at, int n0, int c, float (&v)[NS]) {
  const float* p = t + (at * a.np + n0) * a.C + c;
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = p[int64_t(i) * a.C];
}
template <int NS>
__device__ __forceinline__ void scan_put(const ScanArgs& a, float* t, int64_t at, int n0, int c, const float (&v)[NS]) {
  float* p = t + (at * a.np + n0) * a.C + c;
#pragma unroll
  for (int i = 0; i < NS; ++i) p[int64_t(i) * a.C] = v[i];
}
// A of one channel, times log2(e): exp(d A) = 2^(d * this).
template <int NS>
__device__ __forceinline__ void scan_load_A(const ScanArgs& a, int c, int n0, float (&A)[NS]) {
  scan_load_state<NS>(a, a.A, c, n0, A);
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] *= kLog2e;
}

// A thread's part of a tile of ROWS steps by 64 channels: V neighbouring
// channels of one step, so that a tile's rows take few and wide accesses
// (measured with a lane an element: 20 loads of 2 bytes and 4 such stores a
// wave and tile cost as much time as all its arithmetic).  Threads past the
// tile repeat its tasks from the first on: same values to the same places.
template <int NW, int ROWS>
struct Task {
  static constexpr int PER = ROWS / NW;
  static constexpr int V = PER >= 4 || NW == 6 ? 4 : PER >= 2 ? 2 : 1;
  static constexpr int COUNT = ROWS * 64 / V;
  int t, q;        // step within the tile, first of its channels within the 64
  int n;           // channels there (V but at a group's end)
  unsigned c;      // the first one's number (past the group: one of it)
  __device__ __forceinline__ Task(const ScanArgs& a, int cb, int g) {
    const int k = int(threadIdx.x) % COUNT;
    t = k / (64 / V);
    q = k % (64 / V) * V;
    const int in = (cb % a.cbg) * 64 + q;
    n = min(max(a.cpg - in, 0), V);
    c = g * a.cpg + (n > 0 ? in : 0);
  }
};

// V channels of one row on their way from memory, as loaded: VEC (groups and
// rows are whole aligned packs) one access, its words one after another; else
// one element a word, those that are not there from the first one's place.
// Nothing is put together before it is used, or a load would be waited for
// where it is issued; and the choice is the kernel's, not a branch in it: with
// both ways of loading in one loop the compiler cannot tell how many loads are
// in flight and waits for all (measured: twice the time).
template <typename T, int V, bool VEC>
struct Raw {
  static constexpr int WORDS = int(sizeof(T)) * V / 4 > 0 ? int(sizeof(T)) * V / 4 : 1;
  unsigned r[V];
  __device__ __forceinline__ void load(const T* row, int n) {
    if constexpr (VEC) {
      if constexpr (sizeof(T) * V >= 4) {
        const Pack<unsigned, WORDS> k = *reinterpret_cast<const Pack<unsigned, WORDS>*>(row);
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r[i] = k.v[i];
      } else {
        r[0] = *reinterpret_cast<const unsigned short*>(row);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(T) == 4) r[i] = *reinterpret_cast<const unsigned*>(row + (i < n ? i : 0));
        else r[i] = *reinterpret_cast<const unsigned short*>(row + (i < n ? i : 0));
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __builtin_bit_cast(float, r[i]);
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = float(__builtin_bit_cast(T, static_cast<unsigned short>(r[i / 2] >> (i % 2 * 16))));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = float(__builtin_bit_cast(T, static_cast<unsigned short>(r[i])));
    }
  }
};
template <bool VEC, typename T, int V>
__device__ __forceinline__ void row_put(T* row, int n, const float (&x)[V]) {
  if constexpr (VEC) {
    Pack<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.v[i] = T(x[i]);
    *reinterpret_cast<Pack<T, V>*>(row) = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) row[i] = T(x[i]);
  }
}

// A thread's way along a row tensor, tile after tile of STEPS steps (or back,
// BY < 0): its element of the tile where it stands.  An address goes on by one
// addition; in a tile that ends early, rows past the last one there give way
// to that.
template <typename T, int STEPS, int BY = STEPS>
struct Walk {
  T* p;
  int64_t one;   // elements from a step to the next
  // at step s (the tile's first) + t
  __device__ __forceinline__ Walk(const Rows& w, const StepRows& r, int64_t column, int s, int t) {
    one = r.step * w.rs;
    p = reinterpret_cast<T*>(w.p) + (r.base + (s + t) * r.step) * w.rs + column;
  }
  __device__ __forceinline__ T* next(int s, int t, int end) {
    T* q = p;
    if (s + STEPS > end) q += (min(s + t, end - 1) - (s + t)) * one;   // uniform
    p += one * BY;
    return q;
  }
};

// B and C of a tile of STEPS steps in shared memory, f32, [step][wave][B: NS,
// C: NS]; each thread brings E values of either, of one state.
template <typename T, int NW, int NS, int STEPS, int BY = STEPS>
struct BCWalk {
  static constexpr int NP = NW * NS, E = (STEPS * NP + NW * 64 - 1) / (NW * 64), EVERY = 64 / NS;   // steps between a thread's values
  struct Values { T b[E], c[E]; };
  int n, t;
  bool in;
  Walk<const T, STEPS, BY> b, c;
  static __device__ __forceinline__ int task() { return int(threadIdx.x) % (STEPS * NP); }
  __device__ __forceinline__ BCWalk(const ScanArgs& a, const StepRows& r, int g, int s)
      : n(task() % NP), t(task() / NP), in(n < a.N),
        b(a.Bm, r, int64_t(g) * a.N + (in ? n : 0), s, t), c(a.Cm, r, int64_t(g) * a.N + (in ? n : 0), s, t) {}
  // the tile's steps; for those past the last one there, `end` - 1, its values
  __device__ __forceinline__ void next(int s, int end, Values& v) {
    int64_t ob[E], oc[E];
    if (s + STEPS <= end) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        ob[k] = k * EVERY * b.one;
        oc[k] = k * EVERY * c.one;
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const int back = min(s + t + k * EVERY, end - 1) - (s + t);
        ob[k] = back * b.one;
        oc[k] = back * c.one;
      }
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      v.b[k] = b.p[ob[k]];
      v.c[k] = c.p[oc[k]];
    }
    b.p += b.one * BY;
    c.p += c.one * BY;
  }
  // the tile that begins at s; zero where there is no step or no state (times a
  // step size of zero, an infinite B or C would make a state NaN)
  __device__ __forceinline__ void put(const Values& v, int s, int end, float (*to)[2 * NP]) const {
    float* p = &to[t][n / NS * 2 * NS + n % NS];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const bool is = in && s + t + k * EVERY < end;
      p[k * EVERY * 2 * NP] = is ? float(v.b[k]) : 0.f;
      p[k * EVERY * 2 * NP + NS] = is ? float(v.c[k]) : 0.f;
    }
  }
};

// The same for one wave's NS states, one value a lane: register j holds values
// 16 j to 16 j + 15 of [step][B: NS, C: NS] in the lanes of each row of 16.  An
// operand then comes from its lane through the DPP crossbar (row_newbcast),
// which costs a product or a fused multiply-add nothing but the crossbar's own
// time; read from shared memory at each step, the values would take most of
// its bandwidth (the same 16 bytes to each of 64 lanes), and as scalars a wait
// for all scalar loads at each of a few steps (measured: 1.8 us a tile of 16
// steps, whatever the states).
template <int NW, int NS, int STEPS>
struct BCRegs {
  static constexpr int R = STEPS * 2 * NS / 16;
  static_assert(R * 16 == STEPS * 2 * NS && (NS & (NS - 1)) == 0 && NS <= 16, "whole registers");
  static __device__ __forceinline__ void get(const float (*from)[2 * NW * NS], int w, int lane, float (&v)[R]) {
    const int l = lane & 15;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int at = 16 * j + l;   // of [step][2 NS]
      v[j] = from[at / (2 * NS)][w * 2 * NS + at % (2 * NS)];
      asm volatile("" : "+v"(v[j]));   // made once, here: a DPP operand must not have just been written
    }
  }
};
// Value I of [step][B, C][NS] as a factor, and as one of fused multiply-adds
// acc += value x.  (The two waits stand for a value just written: the compiler
// looks after those of its own instructions only.  An accumulator is written
// before the last factor is read: `&`.)
template <int I, int R>
__device__ __forceinline__ float bc_mul(const float (&v)[R], float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v[I / 16]), 0x150 + I % 16, 0xf, 0xf, true)) * x;
}
#define RNN_DPP "row_mask:0xf bank_mask:0xf"
template <int I, int N, int R>
__device__ __forceinline__ void bc_dot(const float (&v)[R], float& acc, const float* x) {   // acc += sum_i value(I + i) x[i]
  static_assert(I / 16 == (I + N - 1) / 16, "one register");
  if constexpr (N == 1) {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 " RNN_DPP : "+&v"(acc) : "v"(v[I / 16]), "v"(x[0]), "n"(I % 16));
  } else if constexpr (N == 2) {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%4 " RNN_DPP "\n\tv_fmac_f32_dpp %0, %1, %3 row_newbcast:%5 " RNN_DPP
        : "+&v"(acc) : "v"(v[I / 16]), "v"(x[0]), "v"(x[1]), "n"(I % 16), "n"(I % 16 + 1));
  } else {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%6 " RNN_DPP "\n\tv_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 " RNN_DPP
        "\n\tv_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 " RNN_DPP "\n\tv_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 " RNN_DPP
        : "+&v"(acc)
        : "v"(v[I / 16]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "n"(I % 16), "n"(I % 16 + 1), "n"(I % 16 + 2), "n"(I % 16 + 3));
    if constexpr (N > 4) bc_dot<I + 4, N - 4>(v, acc, x + 4);
  }
}
template <int I, int N, int R>
__device__ __forceinline__ void bc_add(const float (&v)[R], float* acc, float x) {   // acc[i] += value(I + i) x
  static_assert(I / 16 == (I + N - 1) / 16, "one register");
  if constexpr (N == 1) {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 " RNN_DPP : "+&v"(acc[0]) : "v"(v[I / 16]), "v"(x), "n"(I % 16));
  } else if constexpr (N == 2) {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %2, %3 row_newbcast:%4 " RNN_DPP "\n\tv_fmac_f32_dpp %1, %2, %3 row_newbcast:%5 " RNN_DPP
        : "+&v"(acc[0]), "+&v"(acc[1]) : "v"(v[I / 16]), "v"(x), "n"(I % 16), "n"(I % 16 + 1));
  } else {
    asm("s_nop 1\n\tv_fmac_f32_dpp %0, %4, %5 row_newbcast:%6 " RNN_DPP "\n\tv_fmac_f32_dpp %1, %4, %5 row_newbcast:%7 " RNN_DPP
        "\n\tv_fmac_f32_dpp %2, %4, %5 row_newbcast:%8 " RNN_DPP "\n\tv_fmac_f32_dpp %3, %4, %5 row_newbcast:%9 " RNN_DPP
        : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3])
        : "v"(v[I / 16]), "v"(x), "n"(I % 16), "n"(I % 16 + 1), "n"(I % 16 + 2), "n"(I % 16 + 3));
    if constexpr (N > 4) bc_add<I + 4, N - 4>(v, acc + 4, x);
  }
}
#undef RNN_DPP

// 2^x h + l for a sum x of many steps' exponents, where 2^x may leave f32
// though the product does not (steps one by one would not have left it either):
// 2^x as two factors, the second 1 for |x| <= 120, and none but the first, which
// is neither zero nor infinite, for a zero or infinite h, which no finite number
// of steps changes.
__device__ __forceinline__ float scan_carry(float x, float h, float l) {
  const float x1 = __builtin_amdgcn_fmed3f(x, -120.f, 120.f);
  const float beyond = __builtin_amdgcn_exp2f(x - x1) * h;
  const bool keep = h == 0.f || __builtin_fabsf(h) == __builtin_huge_valf();
  return __builtin_fmaf(__builtin_amdgcn_exp2f(x1), keep ? h : beyond, l);
}
// Where the plain product does: no more than 2^120, and of an h that falls to
// nothing without being missed (to 2^-80 or less).  `up`: the largest x, `big`:
// the largest |h|.  Uniform.
__device__ __forceinline__ bool scan_carry_plain(float up, float big) { return !__any(up > 120.f || big >= 0x1p40f); }

// h, a state (or, going back, its gradient) at the end of one chunk, through
// `n` chunks more: h = decay h + local of each, decay = 2^(A sum).  `at(k)` is
// the k-th one's place in `local` and in `sum`.  (With scan_carry in the loop a
// long prompt took 2 us more.)
template <int NS, typename At>
__device__ __forceinline__ void scan_through(const ScanArgs& a, const float* local, int n, int c, int n0, const float (&A)[NS],
                                             float (&h)[NS], At at) {
  float first[NS], up = 0.f, big = 0.f;
#pragma unroll
  for (int i = 0; i < NS; ++i) first[i] = h[i];
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    float l[NS];
    scan_get<NS>(a, local, at(k), n0, c, l);
    const float sum = a.sum[at(k) * a.C + c];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float x = A[i] * sum;
      up = __builtin_fmaxf(up, x);
      big = __builtin_fmaxf(big, __builtin_fabsf(h[i]));
      h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(x), h[i], l[i]);
    }
  }
  if (scan_carry_plain(up, big)) return;
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = first[i];
  for (int k = 0; k < n; ++k) {
    float l[NS];
    scan_get<NS>(a, local, at(k), n0, c, l);
    const float sum = a.sum[at(k) * a.C + c];
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = scan_carry(A[i] * sum, h[i], l[i]);
  }
}

// The state at the start of chunk ch > 0 (live), from the end states of the
// chunks before it.
template <int NS>
__device__ __forceinline__ void scan_join(const ScanArgs& a, int b, int ch, int c, int n0, const float (&A)[NS], float (&h)[NS]) {
  const int64_t at = int64_t(b) * a.nchunk;
  scan_get<NS>(a, a.loc, at, n0, c, h);
  scan_through<NS>(a, a.loc, ch - 1, c, n0, A, h, [&](int k) { return at + 1 + k; });
}

}  // namespace rnnhip
