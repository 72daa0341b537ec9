// scan_grad_kernel.h -- the selective scan's gradient (instantiated for one
// element type by k_scan_f32.hip, k_scan_f16.hip and k_scan_bf16.hip).
//
// With gy = dY silu(z) (or dY), a_s = exp(d_s A), u_s = d_s x_s:
//   G_s  = C_s gy_s + a_{s+1} G_{s+1}           (after the last step: d_final)
//   q_s  = G_s a_s h_{s-1}                       = dL/d(d_s A)
//   dA   = sum q_s d_s;    dd_s = sum_n q_s A + x_s sum_n G_s B_s
//   dx_s = d_s sum_n G_s B_s + D gy_s;           dB_s = sum_c G_s u_s
//   dC_s = sum_c gy_s h_s;  dD = sum gy_s x_s;   dz_s = dY y_s silu'(z)
//   d_initial = a_0 G_0
// Nothing of the forward pass is kept.  Three launches:
//   1. along time: states, written before each segment of 16 steps (fewer with
//      many states), and each chunk's end state, sum of step sizes and gradient
//      at its start.  That gradient needs no walk back: sum_s (prod_{r<=s} a_r)
//      C_s gy_s runs forward with the product, at three operations and no
//      exponential.  The product falls to zero harmlessly; but where steps grow
//      the states it may leave f32 upwards, or come back from zero with steps of
//      both signs.  The sum is not finite then, or marked so, and whoever wants
//      it walks back after all.
//   2. each chunk, segment after segment from its end: the segment's states
//      and decays forward from the one written, kept in registers (at most 64
//      of each a lane), then the gradients backward.
//   3. sums of the workgroups' dB, dC, dA, dD, ddelta_bias, in a fixed order.
// Chunks start from zero states; a segment's true state is the written one
// plus decay(chunk start -> segment) times the chunk's true start, joined from
// the chunks before as in the forward pass, and the gradient at a chunk's end
// likewise from those after.
//
// Lanes are channels and waves share the states, as in the forward pass, for
// the same reasons and one more: dB and dC sum over channels, so 64 such sums
// at once are folded over a wave's 64 lanes (Fold), each exchange halving what
// is left: two to three instructions a value, where one sum after another
// would take twelve, and no meeting of waves.
//
// 8 rows of 512 steps by 1024 channels, 16 states, bf16: launch 1 40 us, launch
// 2 87, launch 3 4.8.  Launch 2 issues 27 vector instructions a (step, channel,
// state) where the forward pass issues 9 (by the counters, which show the vector
// units busy for 66 of 100 clocks), and its registers and 118 KB of shared memory
// leave a compute unit one workgroup: these bound it, not its 60 MB.  Four waves
// of four states instead of eight of two: 129 us the whole pass at best against
// 123.
//
// More states.  Launch 1 does not fit its 256 registers from 24 states on: 61 to
// 102 are spilled at 24, 22 to 40 at 32, 77 to 98 at 64 and 157 to 183 at 128;
// launch 2 spills 24 to 44 at 24 and 71 to 114 at 128, and 18 at 64 where there
// are places without a state.  And segments of 8
// steps at 64 states, of 4 at 128, are more states written ahead: for 8 x 1024 x
// 4096 the scratch is 0.2 GB at 16 states, 1.4 at 64 and 4.9 at 128, most of it
// written and read once.  (8 x 512 x 1024, the whole pass and launches 1 and 2: 24
// states 245 us, 98 and 142; 32 206, 80 and 132; 64 420, 183 and 233; 128 1445,
// 399 and 1037.)
#pragma once

#include <algorithm>

#include "scan_device.h"

namespace rnnhip {
namespace {

template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_into(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL,
                                                               0xf, BANKS, false));
}

// Sums of 64 values over a wave's 64 lanes, taken one after another: value I
// (in the order of push<I>) ends in the lane that is I with its six bits
// reversed.  Two values become one by an exchange of half their lanes: values
// that differ in bit l of I over lane bit 5 - l.  st[l] waits for its partner.
struct Fold {
  float st[6];
  bool b3, b2, b1, b0;   // lane bits
  __device__ __forceinline__ explicit Fold(int lane) : b3(lane & 8), b2(lane & 4), b1(lane & 2), b0(lane & 1) {}

  template <int L>
  __device__ __forceinline__ float join(float a, float b) const {
    if constexpr (L == 0) {
      const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
      return __builtin_bit_cast(float, unsigned(p[0])) + __builtin_bit_cast(float, unsigned(p[1]));
    } else if constexpr (L == 1) {
      const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
      return __builtin_bit_cast(float, unsigned(p[0])) + __builtin_bit_cast(float, unsigned(p[1]));
    } else {
      // lanes with the bit clear keep a and give b, the others the reverse
      const bool bit = L == 2 ? b3 : L == 3 ? b2 : L == 4 ? b1 : b0;
      const float keep = bit ? b : a, give = bit ? a : b;
      if constexpr (L == 2) return keep + dpp_into<0x128, 0xf>(0.f, give);   // row_ror:8
      if constexpr (L == 3)   // lane ^ 4: banks 0 and 2 from four lanes up, 1 and 3 from four down
        return keep + dpp_into<0x114, 0xa>(dpp_into<0x104, 0x5>(0.f, give), give);
      if constexpr (L == 4) return keep + quad_x2(give);
      if constexpr (L == 5) return keep + quad_x1(give);
    }
  }
  template <int I, int L = 0>
  __device__ __forceinline__ float push(float v) {   // of I % 64 == 63: the sums
    if constexpr (L == 6) return v;
    else if constexpr ((I >> L) & 1) return push<I, L + 1>(join<L>(st[L], v));
    else {
      st[L] = v;
      return 0.f;
    }
  }
};

__device__ __forceinline__ float gate_of(float z) { return z * logistic(z); }

// Launch 1.
template <typename T, int NW, int NS, bool VEC>
__global__ __launch_bounds__(NW * 64) void scan_ahead_kernel(ScanArgs a) {
  constexpr int TT = kScanTile, D = 2, TS = scan_segment(NS);
  typedef Task<NW, TT> Mine;
  constexpr int V = Mine::V;
  __shared__ float2 du[2][TT][64];   // step size and input
  __shared__ float dg[2][TT][64];    // gy
  __shared__ float sbc[2][TT][2 * NW * NS];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const ScanPlace p = scan_place(a, a.nchunk, lane);
  const int b = p.b, ch = p.ch, n0 = w * NS;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  if (s0 >= L) return;   // uniform
  const int send = int(min(int64_t(s0) + a.chunk, int64_t(L)));
  const StepRows r = step_rows(a.geo, b, L);
  const Mine k(a, p.cb, p.g);

  float h[NS], A[NS], Q[NS], G[NS];
  scan_load_A<NS>(a, p.c, n0, A);
  scan_load_state<NS>(a, ch == 0 ? a.init : nullptr, int64_t(b) * a.C + p.c, n0, h);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    Q[i] = 1.f;
    G[i] = 0.f;
  }
  float total = 0.f;
  const bool behind = ch > 0;   // a chunk before this one needs the gradient at its start
  const bool gz = behind && a.have_z;
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = a.dbias ? a.dbias[k.c + (VEC || i < k.n ? i : 0)] : 0.f;

  Walk<const T, TT> X(a.X, r, k.c, s0, k.t), De(a.delta, r, k.c, s0, k.t), Z(gz ? a.Z : a.X, r, k.c, s0, k.t),
      Dy(behind ? a.dY : a.X, r, k.c, s0, k.t);
  BCWalk<T, NW, NS, TT> BC(a, r, p.g, s0);
  Raw<T, V, VEC> nx[D], nd[D], nz[D], ng[D];
  typename BCWalk<T, NW, NS, TT>::Values nbc[D];
  auto fetch = [&](int s, auto SLOT) {
    constexpr int j = decltype(SLOT)::value;
    nx[j].load(X.next(s, k.t, send), k.n);
    nd[j].load(De.next(s, k.t, send), k.n);
    ng[j].load(Dy.next(s, k.t, send), k.n);
    nz[j].load(Z.next(s, k.t, send), k.n);
    BC.next(s, send, nbc[j]);
  };
  auto prepare = [&](int s, int buf, auto SLOT) {
    constexpr int j = decltype(SLOT)::value;
    float x[V], d[V];
    nx[j].values(x);
    nd[j].values(d);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] += bias[i];
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = softplus(d[i]);
    }
    const bool there = s + k.t < send;   // a step that is not changes no state
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i] = there ? d[i] : 0.f;
      du[buf][k.t][k.q + i] = make_float2(d[i], there ? d[i] * x[i] : 0.f);
    }
    if (behind) {
      float g[V], z[V];
      ng[j].values(g);
      nz[j].values(z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (gz) g[i] *= gate_of(z[i]);
        dg[buf][k.t][k.q + i] = there ? g[i] : 0.f;
      }
    }
    BC.put(nbc[j], s, send, sbc[buf]);
  };
  const int64_t seg0 = int64_t(b) * a.nseg;
  each<D>([&](auto J) { fetch(s0 + decltype(J)::value * TT, J); });
  prepare(s0, 0, IntC<0>{});
  fetch(s0 + D * TT, IntC<0>{});
  int buf = 0, s = s0;
  auto body = [&](auto SLOT) {
    constexpr int next = (decltype(SLOT)::value + 1) % D;
    __syncthreads();
    float bc[BCRegs<NW, NS, TT>::R];
    BCRegs<NW, NS, TT>::get(sbc[buf], w, lane, bc);
    prepare(s + TT, buf ^ 1, IntC<next>{});
    fetch(s + (D + 1) * TT, IntC<next>{});
    each<TT>([&](auto J) {
      constexpr int t = decltype(J)::value, at = t * 2 * NS;
      if (t % TS == 0 && s + t < send && p.ok) {   // a segment begins
        const int64_t seg = seg0 + (s + t) / TS;
        scan_put<NS>(a, a.ckpt, seg, n0, p.c, h);
        if (w == 0) a.cum[seg * a.C + p.c] = total;
      }
      const float2 f = du[buf][t][lane];
      total += f.x;
      float e[NS];
      each<NS>([&](auto I) {
        constexpr int i = decltype(I)::value;
        e[i] = __builtin_amdgcn_exp2f(f.x * A[i]);
        h[i] = __builtin_fmaf(e[i], h[i], bc_mul<at + i>(bc, f.y));
      });
      if (behind) {
        const float g = dg[buf][t][lane];
        each<NS>([&](auto I) {
          constexpr int i = decltype(I)::value;
          Q[i] *= e[i];
          G[i] = __builtin_fmaf(Q[i], bc_mul<at + NS + i>(bc, g), G[i]);
        });
      }
      __builtin_amdgcn_sched_barrier(0);   // (the decays of all steps ahead of it would not fit the registers)
    });
    buf ^= 1;
    s += TT;
  };
  // (tiles past the end change and store nothing; a way out between two bodies
  // would have the compiler move registers whose loads are in flight)
  while (s < send) each<D>(body);
  if (p.ok && a.nchunk > 1) {
    const int64_t at = int64_t(b) * a.nchunk + ch;
    scan_put<NS>(a, a.loc, at, n0, p.c, h);
    if (behind) scan_put<NS>(a, a.gloc, at, n0, p.c, G);
    if (w == 0) a.sum[at * a.C + p.c] = total;
  }
}

// Between the first two, where steps may be negative: the gradients at chunks'
// starts are marked as not to be used for channels that have such steps.
template <typename T>
__global__ __launch_bounds__(256) void scan_signs_kernel(ScanArgs a) {
  __shared__ int negative[64];
  const int lane = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const ScanPlace p = scan_place(a, a.nchunk, lane);
  const int L = geo_len(a.geo, p.b), s0 = p.ch * a.chunk;
  if (p.ch == 0 || s0 >= L) return;   // uniform
  const int send = int(min(int64_t(s0) + a.chunk, int64_t(L)));
  const StepRows r = step_rows(a.geo, p.b, L);
  const float bias = a.dbias ? a.dbias[p.c] : 0.f;
  if (w == 0) negative[lane] = 0;
  __syncthreads();
  bool below = false;
#pragma unroll 4
  for (int s = s0 + w; s < send; s += 4)
    below = below || float((reinterpret_cast<const T*>(a.delta.p) + p.c)[(r.base + s * r.step) * a.delta.rs]) + bias < 0.f;
  if (below) negative[lane] = 1;
  __syncthreads();
  if (!negative[lane] || !p.ok) return;
  float* to = a.gloc + (int64_t(p.b) * a.nchunk + p.ch) * a.np * a.C + p.c;
  for (int n = w; n < a.np; n += 4) to[int64_t(n) * a.C] = __builtin_nanf("");
}

// Launch 2.  PAD: there are states past N among a wave's, or lanes past a
// group's channels.  They are zero as their inputs are, and stay so while values
// are finite; but zero times an infinite one is not a number, and would enter
// the sums over states (dX, ddelta, dZ) and over lanes (dB, dC).  So they are put
// back to zero in the steps of a segment with such a value, or, where watching
// costs more than that, with states past N in all.  (8 rows of 512 steps by 1024
// channels, bf16, the whole pass, and what it took when they were left alone: 10
// states 128 us, 125; 1 state 122, 120.5; 40 states 450, 415; 16 states by 1000
// channels 129, 126; and 16 by 1024, which has none, 125.5, 125.)
template <typename T, int NW, int NS, bool VEC, bool PAD>
__global__ __launch_bounds__(NW * 64) void scan_back_kernel(ScanArgs a) {
  constexpr int TS = scan_segment(NS);
  typedef Task<NW, TS> Mine;
  constexpr int V = Mine::V;
  constexpr int FOLDS = (TS * 2 * NS + 63) / 64;
  __shared__ float4 in[TS][64];               // step size, input, gy of a step
  __shared__ float part[3][NW][TS][64];       // the waves' parts of y, sum G B, sum q A
  __shared__ float sbc[TS][2 * NW * NS];
  constexpr bool WATCH = PAD && NS == 2;      // whether states past N are watched for an input that is not finite
  __shared__ int marks[2];                    // WATCH: this segment and the next have one
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const ScanPlace p = scan_place(a, a.nchunk, lane);
  const int b = p.b, ch = p.ch, n0 = w * NS;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  const int s1 = int(min(int64_t(s0) + a.chunk, int64_t(a.geo.S)));
  const int send = min(s1, L);
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t cs = int64_t(b) * a.C + p.c;
  const Mine k(a, p.cb, p.g);

  float dA[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;
  float dD[V] = {}, dbias[V] = {};

  if (s0 < send) {
    float A[NS], G[NS], hs[NS];
    scan_load_A<NS>(a, p.c, n0, A);
    const bool joined = ch > 0;
    if (joined) scan_join<NS>(a, b, ch, p.c, n0, A, hs);
    // the gradient at the chunk's end, from the chunks after it
    scan_load_state<NS>(a, a.dfin, cs, n0, G);
    const int last_chunk = (L - 1) / a.chunk;
    scan_through<NS>(a, a.gloc, last_chunk - ch, p.c, n0, A, G, [&](int k) { return int64_t(b) * a.nchunk + last_chunk - k; });
    bool walk = false;
#pragma unroll
    for (int i = 0; i < NS; ++i) walk = walk || !(__builtin_fabsf(G[i]) < __builtin_huge_valf());
    if (__any(walk)) {
      scan_load_state<NS>(a, a.dfin, cs, n0, G);
      const float step_bias = a.dbias ? a.dbias[p.c] : 0.f;
      for (int t = L - 1; t >= send; --t) {
        const int64_t row = r.base + t * r.step;
        float d = float((reinterpret_cast<const T*>(a.delta.p) + p.c)[row * a.delta.rs]) + step_bias;
        if (a.softplus) d = softplus(d);
        float g = float((reinterpret_cast<const T*>(a.dY.p) + p.c)[row * a.dY.rs]);
        if (a.have_z) g *= gate_of(float((reinterpret_cast<const T*>(a.Z.p) + p.c)[row * a.Z.rs]));
        const T* C = reinterpret_cast<const T*>(a.Cm.p) + row * a.Cm.rs + int64_t(p.g) * a.N;
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (n0 + i < a.N) G[i] = __builtin_amdgcn_exp2f(d * A[i]) * __builtin_fmaf(float(C[n0 + i]), g, G[i]);
      }
    }
    float big = 0.f;   // the largest state at the chunk's start
    auto is = [&](int i) { return !PAD || (p.ok && n0 + i < a.N); };   // whether a lane's state is one
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      A[i] = is(i) ? A[i] : 0.f;
      G[i] = is(i) ? G[i] : 0.f;
      if (joined) hs[i] = is(i) ? hs[i] : 0.f;
      if (joined) big = __builtin_fmaxf(big, __builtin_fabsf(hs[i]));
    }
    float bias[V], skip[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned c = k.c + (VEC || i < k.n ? i : 0);
      bias[i] = a.dbias ? a.dbias[c] : 0.f;
      skip[i] = a.D ? a.D[c] : 0.f;
    }
    const int last = s0 + (send - 1 - s0) / TS * TS;
    Walk<const T, TS, -TS> X(a.X, r, k.c, last, k.t), De(a.delta, r, k.c, last, k.t), Z(a.Z, r, k.c, last, k.t), Dy(a.dY, r, k.c, last, k.t);
    Walk<T, TS, -TS> oX(a.dX, r, k.c, last, k.t), oD(a.ddelta, r, k.c, last, k.t), oZ(a.dZ, r, k.c, last, k.t);
    BCWalk<T, NW, NS, TS, -TS> BC(a, r, p.g, last);
    Raw<T, V, VEC> nx, nd, nz, ng;
    typename BCWalk<T, NW, NS, TS, -TS>::Values nbc;
    float nh[NS], ncum = 0.f;
    auto fetch = [&](int s) {   // the segment that begins at s
      nx.load(X.next(s, k.t, send), k.n);
      nd.load(De.next(s, k.t, send), k.n);
      ng.load(Dy.next(s, k.t, send), k.n);
      if (a.have_z) nz.load(Z.next(s, k.t, send), k.n);
      BC.next(s, send, nbc);
      const int64_t seg = int64_t(b) * a.nseg + s / TS;
      scan_get<NS>(a, a.ckpt, seg, n0, p.c, nh);
      if (joined) ncum = a.cum[seg * a.C + p.c];
    };
    Fold fold(lane);
    // where this lane's sum of a fold belongs: value (lane reversed) of the
    // fold's 64, in the order pushed: steps falling, then dB, then dC
    const int mine = int(__builtin_bitreverse32(unsigned(lane)) >> 26);
    float* pbc = a.pbc + (int64_t(p.cb) * a.geo.B + b) * a.geo.S * (2 * a.np) + w * 2 * NS;

    int mark = 0;
    if constexpr (WATCH) {
      if (threadIdx.x < 2) marks[threadIdx.x] = 0;
      __syncthreads();
    }
    fetch(last);
    for (int s = last; s >= s0; s -= TS) {
      float x[V], d[V], g[V], gy[V], z[V], raw[V], h0[NS];
      const bool there = s + k.t < send;   // a step that is not changes nothing
      nx.values(x);
      nd.values(raw);
      ng.values(g);
      if (a.have_z) nz.values(z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool is = there && i < k.n;
        x[i] = is ? x[i] : 0.f;
        d[i] = raw[i] = is ? raw[i] + bias[i] : 0.f;
        gy[i] = g[i] = is ? g[i] : 0.f;
        z[i] = a.have_z && is ? z[i] : 0.f;
      }
      if (a.softplus) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = softplus(raw[i]);
      }
      if (a.have_z) {
#pragma unroll
        for (int i = 0; i < V; ++i) gy[i] = g[i] * gate_of(z[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] = there ? d[i] : 0.f;
        in[k.t][k.q + i] = make_float4(d[i], d[i] * x[i], gy[i], 0.f);
      }
      if (WATCH && a.N < a.np) {
        float odd = 0.f;   // (NaN for an infinite step size, input or gy)
#pragma unroll
        for (int i = 0; i < V; ++i) odd = __builtin_fmaf(d[i] * x[i], 0.f, __builtin_fmaf(gy[i], 0.f, odd));
        if (__any(odd != odd)) marks[mark] = 1;
      }
      BC.put(nbc, s, send, sbc);
#pragma unroll
      for (int i = 0; i < NS; ++i) h0[i] = nh[i];
      if (joined) {
        float up = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) up = __builtin_fmaxf(up, A[i] * ncum);
        if (scan_carry_plain(up, big)) {
#pragma unroll
          for (int i = 0; i < NS; ++i) h0[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(A[i] * ncum), hs[i], h0[i]);
        } else {
#pragma unroll
          for (int i = 0; i < NS; ++i) h0[i] = scan_carry(A[i] * ncum, hs[i], h0[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) h0[i] = is(i) ? h0[i] : 0.f;
      if (s > s0) fetch(s - TS);
      __syncthreads();
      float bc[BCRegs<NW, NS, TS>::R];
      BCRegs<NW, NS, TS>::get(sbc, w, lane, bc);

      auto steps = [&](auto mask) {
        constexpr bool MASK = decltype(mask)::value;
        float h[TS][NS], e[TS][NS];
        each<TS>([&](auto TT) {
          constexpr int t = decltype(TT)::value, at = t * 2 * NS;
          const float4 f = in[t][lane];
          each<NS>([&](auto I) {
            constexpr int i = decltype(I)::value;
            const float decay = __builtin_amdgcn_exp2f(f.x * A[i]);
            const float next = __builtin_fmaf(decay, t ? h[t ? t - 1 : 0][i] : h0[i], bc_mul<at + i>(bc, f.y));
            e[t][i] = !MASK || is(i) ? decay : 0.f;
            h[t][i] = !MASK || is(i) ? next : 0.f;
          });
          if (a.dZ.p) {
            float v = 0.f;
            bc_dot<at + NS, NS>(bc, v, h[t]);
            part[0][w][t][lane] = v;
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        // Steps past the row's end (in the segment that is taken first) add q * 0 to
        // dA, which is not 0 where a state or gradient is infinite: with the row's
        // last step the sum begins anew.
        const int edge = s + TS > send ? send - 1 - s : -1;
        each<TS>([&](auto TT) {
          constexpr int t = TS - 1 - decltype(TT)::value, base = decltype(TT)::value * 2 * NS;
          const float4 f = in[t][lane];
          if (t == edge) {   // (uniform)
#pragma unroll
            for (int i = 0; i < NS; ++i) dA[i] = 0.f;
          }
          float sb = 0.f, sq = 0.f;
          auto out = [&](int fold_at, float v) {   // 64 sums are there
            const int at = fold_at * 64 + mine;
            const int st = s + TS - 1 - at / (2 * NS);
            if (at < TS * 2 * NS && st < send) pbc[int64_t(st) * (2 * a.np) + at % (2 * NS)] = v;
          };
          bc_add<t * 2 * NS + NS, NS>(bc, G, f.z);
          if constexpr (MASK) {
#pragma unroll
            for (int i = 0; i < NS; ++i) G[i] = is(i) ? G[i] : 0.f;
          }
          bc_dot<t * 2 * NS, NS>(bc, sb, G);
          each<NS>([&](auto I) {
            constexpr int i = decltype(I)::value;
            const float v = fold.template push<base + i>(G[i] * f.y);
            if constexpr ((base + i) % 64 == 63) out((base + i) / 64, v);
            G[i] *= e[t][i];
            const float qi = G[i] * (t ? h[t ? t - 1 : 0][i] : h0[i]);
            sq = __builtin_fmaf(qi, A[i], sq);
            dA[i] = __builtin_fmaf(qi, f.x, dA[i]);
          });
          each<NS>([&](auto I) {
            constexpr int i = decltype(I)::value;
            const float v = fold.template push<base + NS + i>(f.z * h[t][i]);
            if constexpr ((base + NS + i) % 64 == 63) out((base + NS + i) / 64, v);
          });
          if constexpr (t == 0 && (TS * 2 * NS) % 64 != 0) {   // the last fold's empty places
            each<FOLDS * 64 - TS * 2 * NS>([&](auto I) {
              constexpr int at = TS * 2 * NS + decltype(I)::value;
              const float v = fold.template push<at>(0.f);
              if constexpr (at % 64 == 63) out(at / 64, v);
            });
          }
          part[1][w][t][lane] = sb;
          part[2][w][t][lane] = sq;
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      if constexpr (PAD) {
        float odd = 0.f;
#pragma unroll
        for (float v : bc) odd = __builtin_fmaf(v, 0.f, odd);
        bool fix = a.N < a.np;
        if (WATCH && fix) {
          fix = __builtin_amdgcn_readfirstlane(marks[mark]);
          mark ^= 1;
          if (threadIdx.x == 0) marks[mark] = 0;
        }
        if (fix || __any(odd != odd)) steps(IntC<1>{});
        else steps(IntC<0>{});
      } else {
        steps(IntC<0>{});
      }
      __syncthreads();
      float y[V], sb[V], sq[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[i] = skip[i] * x[i];
        sb[i] = sq[i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const Pack<float, V> vb = *reinterpret_cast<const Pack<float, V>*>(&part[1][j][k.t][k.q]);
        const Pack<float, V> vq = *reinterpret_cast<const Pack<float, V>*>(&part[2][j][k.t][k.q]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sb[i] += vb.v[i];
          sq[i] += vq.v[i];
        }
        if (a.dZ.p) {
          const Pack<float, V> vy = *reinterpret_cast<const Pack<float, V>*>(&part[0][j][k.t][k.q]);
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] += vy.v[i];
        }
      }
      if (there && k.n > 0) {
        float dr[V], o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dr[i] = __builtin_fmaf(x[i], sb[i], sq[i] * kLn2);   // (A carries log2(e))
          if (a.softplus) dr[i] *= logistic(raw[i]);
          dbias[i] += dr[i];
          dD[i] = __builtin_fmaf(gy[i], x[i], dD[i]);
        }
        if (a.dX.p) {
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = __builtin_fmaf(d[i], sb[i], skip[i] * gy[i]);
          row_put<VEC, T, V>(oX.p, k.n, o);
        }
        if (a.ddelta.p) row_put<VEC, T, V>(oD.p, k.n, dr);
        if (a.dZ.p) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float sg = logistic(z[i]);
            o[i] = g[i] * y[i] * (sg * __builtin_fmaf(z[i], 1.f - sg, 1.f));
          }
          row_put<VEC, T, V>(oZ.p, k.n, o);
        }
      }
      oX.p -= oX.one * TS;
      oD.p -= oD.one * TS;
      oZ.p -= oZ.one * TS;
    }
    if (ch == 0 && a.dinit && p.ok) scan_store_state<NS>(a, a.dinit, cs, n0, G);
  } else if (ch == 0 && a.dinit && p.ok) {   // a row of no steps
    float G[NS];
    scan_load_state<NS>(a, a.dfin, cs, n0, G);
    scan_store_state<NS>(a, a.dinit, cs, n0, G);
  }

  const int64_t at = int64_t(b) * a.nchunk + ch;
  if (p.ok) {
    // rows past the length: zero
    for (int s = max(s0, send) + w; s < s1; s += NW) {
      const int64_t row = dead_row(a.geo, b, s);
      if (a.dX.p) (reinterpret_cast<T*>(a.dX.p) + p.c)[row * a.dX.rs] = T(0.f);
      if (a.ddelta.p) (reinterpret_cast<T*>(a.ddelta.p) + p.c)[row * a.ddelta.rs] = T(0.f);
      if (a.dZ.p) (reinterpret_cast<T*>(a.dZ.p) + p.c)[row * a.dZ.rs] = T(0.f);
    }
    if (a.dA) scan_put<NS>(a, a.pA, at, n0, p.c, dA);
  }
  if (a.dD || a.ddbias) {   // over the steps that the threads prepared
    __syncthreads();
    float (*sum)[64] = reinterpret_cast<float (*)[64]>(part);   // [2][TS]
    if (int(threadIdx.x) < Mine::COUNT) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum[k.t][k.q + i] = dD[i];
        sum[TS + k.t][k.q + i] = dbias[i];
      }
    }
    __syncthreads();
    if (w < 2 && p.ok) {
      float v = 0.f;
#pragma unroll
      for (int t = 0; t < TS; ++t) v += sum[w * TS + t][lane];
      a.pD[(at * 2 + w) * a.C + p.c] = v;
    }
  }
}

// Launch 3: workgroups [0, nbc) sum dB and dC over their group's channel
// blocks, one element of one row a thread; then 64 columns of dA, then of dD
// and ddelta_bias, a workgroup, four threads a column.
template <typename T>
__global__ __launch_bounds__(256) void scan_sums_kernel(ScanArgs a) {
  const int tid = int(threadIdx.x);
  const int64_t gn = int64_t(a.G) * a.N;
  const int64_t nbc = (a.dB.p || a.dC.p) ? (int64_t(a.geo.B) * a.geo.S * 2 * gn + 255) / 256 : 0;
  const int64_t block = a.sums0 + blockIdx.x;
  if (block < nbc) {
    const int64_t i = block * 256 + tid;
    if (i >= int64_t(a.geo.B) * a.geo.S * 2 * gn) return;
    const int64_t row = i / (2 * gn);
    const int in = int(i - row * 2 * gn);
    const int which = in >= gn, gi = which ? in - int(gn) : in;
    const int g = gi / a.N, n = gi - g * a.N;
    const int b = int(row / a.geo.S), s = int(row - int64_t(b) * a.geo.S);
    const Rows& out = which ? a.dC : a.dB;
    if (!out.p) return;
    int L = a.geo.lens ? a.geo.lens[b] : a.geo.S;
    L = L < 0 ? 0 : (L > a.geo.S ? a.geo.S : L);
    float v = 0.f;
    int t = s;
    if (s < L) {
      const int64_t per = int64_t(a.geo.B) * a.geo.S * 2 * a.np;
      const int ns = a.np / a.nw, w = n / ns;
      const float* p = a.pbc + int64_t(g) * a.cbg * per + row * 2 * a.np + w * 2 * ns + which * ns + (n - w * ns);
#pragma unroll 4
      for (int k = 0; k < a.cbg; ++k) v += p[k * per];
      if (a.geo.reverse) t = L - 1 - s;
    }
    reinterpret_cast<T*>(out.p)[dead_row(a.geo, b, t) * out.rs + gi] = T(v);
    return;
  }
  __shared__ float red[3][64];
  const int64_t ncA = a.dA ? (int64_t(a.C) * a.np + 63) / 64 : 0;
  const int64_t blk = block - nbc;
  const bool isA = blk < ncA;
  const int64_t cols = isA ? int64_t(a.C) * a.np : 2 * int64_t(a.C);
  const float* part = isA ? a.pA : a.pD;
  const int64_t col = (isA ? blk : blk - ncA) * 64 + (tid & 63);
  const int64_t P = int64_t(a.geo.B) * a.nchunk;
  const int w = tid >> 6;
  float v = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int64_t k = w; k < P; k += 4) v += part[k * cols + col];
  }
  if (w) red[w - 1][tid & 63] = v;
  __syncthreads();
  if (w || col >= cols) return;
  v = ((v + red[0][tid]) + red[1][tid]) + red[2][tid];
  if (isA) {
    const int n = int(col / a.C), c = int(col - int64_t(n) * a.C);
    if (n < a.N) a.dA[int64_t(c) * a.N + n] = v;
  } else if (col < a.C) {
    if (a.dD) a.dD[col] = v;
  } else if (a.ddbias) {
    a.ddbias[col - a.C] = v;
  }
}

template <typename T, int NW, int NS, bool VEC>
hipError_t back_of(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.nchunk * a.G * a.cbg;
  if (hipError_t e = go(scan_ahead_kernel<T, NW, NS, VEC>, blocks, NW * 64, a, s); e != hipSuccess) return e;
  if (!a.softplus && a.nchunk > 1)
    if (hipError_t e = go(scan_signs_kernel<T>, blocks, 256, a, s); e != hipSuccess) return e;
  return a.N < a.np || a.cpg % 64 ? go(scan_back_kernel<T, NW, NS, VEC, true>, blocks, NW * 64, a, s)
                                  : go(scan_back_kernel<T, NW, NS, VEC, false>, blocks, NW * 64, a, s);
}

template <typename T>
hipError_t scan_backward_of(const ScanArgs& a, hipStream_t s) {
  hipError_t e;
  switch (a.nw * 32 + a.np / a.nw) {   // the splits of scan_split
    case 4 * 32 + 2: e = a.vec_rows ? back_of<T, 4, 2, true>(a, s) : back_of<T, 4, 2, false>(a, s); break;
    case 8 * 32 + 2: e = a.vec_rows ? back_of<T, 8, 2, true>(a, s) : back_of<T, 8, 2, false>(a, s); break;
    case 6 * 32 + 4: e = a.vec_rows ? back_of<T, 6, 4, true>(a, s) : back_of<T, 6, 4, false>(a, s); break;
    case 8 * 32 + 4: e = a.vec_rows ? back_of<T, 8, 4, true>(a, s) : back_of<T, 8, 4, false>(a, s); break;
    case 8 * 32 + 8: e = a.vec_rows ? back_of<T, 8, 8, true>(a, s) : back_of<T, 8, 8, false>(a, s); break;
    case 8 * 32 + 16: e = a.vec_rows ? back_of<T, 8, 16, true>(a, s) : back_of<T, 8, 16, false>(a, s); break;
    default: return hipErrorInvalidValue;
  }
  if (e != hipSuccess) return e;
  int64_t blocks = 0;
  if (a.dB.p || a.dC.p) blocks += (int64_t(a.geo.B) * a.geo.S * 2 * a.G * a.N + 255) / 256;
  if (a.dA) blocks += (int64_t(a.C) * a.np + 63) / 64;
  if (a.dD || a.ddbias) blocks += (2 * int64_t(a.C) + 63) / 64;
  constexpr int64_t most = (int64_t(1) << 24) - 1;   // workgroups of a launch
  for (ScanArgs part = a; part.sums0 < blocks; part.sums0 += most)
    if (e = go(scan_sums_kernel<T>, std::min(blocks - part.sums0, most), 256, part, s); e != hipSuccess) return e;
  return hipSuccess;
}

}  // namespace
}  // namespace rnnhip
