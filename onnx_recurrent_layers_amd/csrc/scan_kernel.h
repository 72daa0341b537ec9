// scan_kernel.h -- the selective scan, forward, over prompts (instantiated for
// one element type by k_scan_f32.hip, k_scan_f16.hip and k_scan_bf16.hip).
//
//   h_s = exp(d_s A) h_{s-1} + d_s x_s B_s,   y_s = sum_n C_s h_s + D x_s
//
// For each step, channel and state: the product d*A, an exponential, the
// product with B and two fused multiply-adds; A is kept times log2(e), so the
// exponential is the hardware's 2^x.  With 16 states and more these
// instructions bound a layer, with fewer and for few steps memory does.
//
// Why a lane a channel and the states over the waves: the five instructions in
// a loop of registers take a SIMD 28.8 clocks for a wave's 64 (step, channel,
// state) with two waves on it or more, 32.5 with one, which is nearly alone in
// waiting for each result; a workgroup of 64 channels by 4 to 8 waves fills a
// chip of 1024 SIMDs with the fewest rows.  And a wave's lanes share B and C
// then, which cost it one register a 16 values instead of a read of shared
// memory an operand (BCRegs).  For 16 rows of 1024 steps by 2048 channels, 16
// states, bf16, rows of all lengths up to it: four lanes of a wave to a channel
// with B and C read from shared memory 186 us (154 with rows in order of
// length), B and C by scalar loads 148, this with an element a load 138, with
// packs of four channels a load 117 to 124 (rows of full length: 168, 1.7 times the
// bare loop's time, the rest being softplus, gate, sums of parts and barriers;
// counters show the vector units busy for 80 of 100 clocks).  Sixteen states
// on eight waves take 172 where four take 124, each wave doing the tile's fixed
// work for half as many states; only with one workgroup a compute unit or less
// do they win (8 rows 103 and 114).
//
// A tile is 16 steps.  Each thread prepares its part of it, 4 neighbouring
// channels of a step (Task: loads, softplus), and puts step size and input into
// shared memory; all waves run the tile's steps on their states and put their
// parts of y there; each thread then sums, gates and stores what it prepared.
// One barrier a tile: the next tile's preparation and the last tile's outputs
// come between barrier and steps, in the other halves of the buffers.
//
// Few rows: the time axis is cut into chunks.  A first launch gives each
// chunk's end state from a zero state and its sum of step sizes (the decay
// over a chunk is exp(A * sum)); the second joins them at its start.  That
// costs the recurrence twice, so it is done only where the chunks fill a chip
// that the rows alone leave empty (rule in seq_api.cpp).  (1 row of 4096 steps
// by 2048 channels, f16: 16 states 40 us of the first launch and 55 of the second
// under a trace, 87.4 together without; 64 states, bf16, 113 and 142, 254; 128
// states 665 and 258, 920.  At 64 and 128 the first launch does not fit its
// registers: 4 to 10 and 174 to 182 of them are spilled, in its loop.  Rows
// enough, 8 x 1024 x 2048: 64 states 254 us, 128 states 465.)
#pragma once

#include "scan_device.h"

namespace rnnhip {
namespace {

// LOCAL: the first of two launches (end states and sums of all chunks but
// each row's last); else the outputs.  PAD: there are states past N among a
// wave's, which are kept zero in a step's y: their B and C are zero, but times
// an infinite step or state that is not a number.  (8 x 1024 x 2048, bf16: 10
// states 122 us, 114.5 if they are left alone; 20 states 174.5 and 162.5.  Zeroed
// only in tiles with an infinite step, as whoever prepares them would mark it:
// 127 and 173.5.)
template <typename T, int NW, int NS, bool LOCAL, bool VEC, bool PAD>
__global__ __launch_bounds__(NW * 64) void scan_kernel(ScanArgs a) {
  constexpr int TT = kScanTile, D = 2;   // steps of a tile, tiles of rows in flight
  typedef Task<NW, TT> Mine;
  constexpr int V = Mine::V;
  __shared__ float2 du[2][TT][64];                                // step size and input
  __shared__ float part[LOCAL ? 1 : 2][NW][LOCAL ? 1 : TT][64];   // the waves' parts of y
  __shared__ float sbc[2][TT][2 * NW * NS];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const ScanPlace p = scan_place(a, LOCAL ? a.nchunk - 1 : a.nchunk, lane);
  const int b = p.b, ch = p.ch, n0 = w * NS;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  const int s1 = int(min(int64_t(s0) + a.chunk, int64_t(a.geo.S)));
  const int send = min(s1, L);
  if (LOCAL && s1 >= L) return;   // nothing follows this chunk (uniform)
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t cs = int64_t(b) * a.C + p.c;   // the channel among all rows' states
  const Mine k(a, p.cb, p.g);

  float h[NS], A[NS];
  scan_load_A<NS>(a, p.c, n0, A);
  if (ch == 0 && !LOCAL && a.init && s1 < L) {
    // the first launch's copy: the last chunk's workgroup may be writing the
    // final state over the initial one
    scan_get<NS>(a, a.first, b, n0, p.c, h);
  } else if (ch == 0) {
    scan_load_state<NS>(a, a.init, cs, n0, h);
    if (LOCAL && a.init && p.ok) scan_put<NS>(a, a.first, b, n0, p.c, h);
  } else if (LOCAL || s0 >= L) {
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = 0.f;
  } else {
    scan_join<NS>(a, b, ch, p.c, n0, A, h);
  }
  float total = 0.f;   // LOCAL: the sum of step sizes

  if (s0 < send) {
    const bool gate = !LOCAL && a.have_z;
    float bias[V], skip[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned c = k.c + (VEC || i < k.n ? i : 0);
      bias[i] = a.dbias ? a.dbias[c] : 0.f;
      skip[i] = !LOCAL && a.D ? a.D[c] : 0.f;
    }
    Walk<const T, TT> X(a.X, r, k.c, s0, k.t), De(a.delta, r, k.c, s0, k.t), Z(gate ? a.Z : a.X, r, k.c, s0, k.t);
    Walk<T, TT> Y(a.Y, r, k.c, s0 - TT, k.t);
    BCWalk<T, NW, NS, TT> BC(a, r, p.g, s0);
    // This thread's channels of a tile, D tiles in flight.  Rows past the last
    // one there repeat it: the number of loads and stores in flight is then the
    // same on every way through the loop, and a wait for the oldest waits for
    // no other.
    Raw<T, V, VEC> nx[D], nd[D], nz[D];
    typename BCWalk<T, NW, NS, TT>::Values nbc[D];
    auto fetch = [&](int s, auto SLOT) {
      constexpr int j = decltype(SLOT)::value;
      nx[j].load(X.next(s, k.t, send), k.n);
      nd[j].load(De.next(s, k.t, send), k.n);
      if constexpr (!LOCAL) nz[j].load(Z.next(s, k.t, send), k.n);
      BC.next(s, send, nbc[j]);
    };
    float px[V];     // the prepared tile's inputs and gates, for its outputs
    Raw<T, V, VEC> pz;
    auto prepare = [&](int s, int buf, auto SLOT) {
      constexpr int j = decltype(SLOT)::value;
      float d[V];
      nx[j].values(px);
      nd[j].values(d);
      if constexpr (!LOCAL) pz = nz[j];
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
        du[buf][k.t][k.q + i] = make_float2(d[i], there ? d[i] * px[i] : 0.f);
      }
      BC.put(nbc[j], s, send, sbc[buf]);
    };
    float ox[V] = {};
    Raw<T, V, VEC> oz = {};
    // the outputs of the tile that began at s (before the first: to scratch)
    auto finish = [&](int s, int buf) {
      if constexpr (!LOCAL) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = skip[i] * ox[i];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          const Pack<float, V> v = *reinterpret_cast<const Pack<float, V>*>(&part[buf][j][k.t][k.q]);
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] += v.v[i];
        }
        if (gate) {
          float z[V];
          oz.values(z);
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] *= z[i] * logistic(z[i]);
        }
        const bool there = s >= s0 && s + k.t < send && k.n > 0;
        row_put<VEC, T, V>(there ? Y.p : reinterpret_cast<T*>(a.sink) + k.c, k.n, y);
        Y.p += Y.one * TT;
      }
    };

    each<D>([&](auto J) { fetch(s0 + decltype(J)::value * TT, J); });
    prepare(s0, 0, IntC<0>{});
    fetch(s0 + D * TT, IntC<0>{});
    int buf = 0, s = s0;
    auto body = [&](auto SLOT) {
      constexpr int next = (decltype(SLOT)::value + 1) % D;
      __syncthreads();
      float bc[BCRegs<NW, NS, TT>::R];
      BCRegs<NW, NS, TT>::get(sbc[buf], w, lane, bc);
      float qx[V];
#pragma unroll
      for (int i = 0; i < V; ++i) qx[i] = px[i];
      const Raw<T, V, VEC> qz = pz;
      prepare(s + TT, buf ^ 1, IntC<next>{});
      finish(s - TT, buf ^ 1);
#pragma unroll
      for (int i = 0; i < V; ++i) ox[i] = qx[i];
      oz = qz;
      fetch(s + (D + 1) * TT, IntC<next>{});
      each<TT>([&](auto J) {
        constexpr int t = decltype(J)::value, at = t * 2 * NS;
        const float2 f = du[buf][t][lane];
        each<NS>([&](auto I) {
          constexpr int i = decltype(I)::value;
          const float next = __builtin_fmaf(__builtin_amdgcn_exp2f(f.x * A[i]), h[i], bc_mul<at + i>(bc, f.y));
          h[i] = PAD && n0 + i >= a.N ? 0.f : next;   // (uniform)
        });
        if constexpr (LOCAL) {
          total += f.x;
        } else {
          float y = 0.f;
          bc_dot<at + NS, NS>(bc, y, h);
          part[buf][w][t][lane] = y;
        }
      });
      buf ^= 1;
      s += TT;
    };
    // (tiles past the end change and store nothing; a way out between two bodies
    // would have the compiler move registers whose loads are in flight)
    while (s < send) each<D>(body);
    __syncthreads();
    finish(s - TT, buf ^ 1);
  }

  if constexpr (LOCAL) {
    if (p.ok) {
      const int64_t at = int64_t(b) * a.nchunk + ch;
      scan_put<NS>(a, a.loc, at, n0, p.c, h);
      if (w == 0) a.sum[at * a.C + p.c] = total;
    }
  } else {
    if (p.ok)
      for (int s = max(s0, send) + w; s < s1; s += NW)
        (reinterpret_cast<T*>(a.Y.p) + p.c)[dead_row(a.geo, b, s) * a.Y.rs] = T(0.f);
    // the row's last step is in this chunk (a row of no steps: the first)
    if (a.fin && p.ok && ch == (L > 0 ? (L - 1) / a.chunk : 0)) scan_store_state<NS>(a, a.fin, cs, n0, h);
  }
}

template <typename T, bool LOCAL, bool VEC, bool PAD>
hipError_t scan_split_of(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * (LOCAL ? a.nchunk - 1 : a.nchunk) * a.G * a.cbg;
  switch (a.nw * 32 + a.np / a.nw) {   // the splits of scan_split
    case 4 * 32 + 2: return go(scan_kernel<T, 4, 2, LOCAL, VEC, PAD>, blocks, 256, a, s);
    case 4 * 32 + 4: return go(scan_kernel<T, 4, 4, LOCAL, VEC, PAD>, blocks, 256, a, s);
    case 6 * 32 + 4: return go(scan_kernel<T, 6, 4, LOCAL, VEC, PAD>, blocks, 384, a, s);
    case 8 * 32 + 4: return go(scan_kernel<T, 8, 4, LOCAL, VEC, PAD>, blocks, 512, a, s);
    case 8 * 32 + 8: return go(scan_kernel<T, 8, 8, LOCAL, VEC, PAD>, blocks, 512, a, s);
    case 8 * 32 + 16: return go(scan_kernel<T, 8, 16, LOCAL, VEC, PAD>, blocks, 512, a, s);
    default: return hipErrorInvalidValue;
  }
}
template <typename T, bool LOCAL>
hipError_t scan_of(const ScanArgs& a, hipStream_t s) {
  if constexpr (!LOCAL) {
    if (a.N < a.np) return a.vec_rows ? scan_split_of<T, LOCAL, true, true>(a, s) : scan_split_of<T, LOCAL, false, true>(a, s);
  }
  return a.vec_rows ? scan_split_of<T, LOCAL, true, false>(a, s) : scan_split_of<T, LOCAL, false, false>(a, s);
}

}  // namespace
}  // namespace rnnhip
