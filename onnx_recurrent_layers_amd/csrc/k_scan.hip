// k_scan.hip -- the selective scan, forward: prompts and single tokens.
//
//   h_s = exp(d_s A) h_{s-1} + d_s x_s B_s,   y_s = sum_n C_s h_s + D x_s
//
// Four lanes share a channel, NS states each, so a wave carries 16 channels
// and a workgroup 64 of one batch row and group.  For each step and state:
// the product d*A, an exponential, the product with B and two fused
// multiply-adds; A is kept times log2(e), so the exponential is the
// hardware's 2^x.  Measured on a register-only loop of these five
// instructions the chip does 7.5e12 of them a second (20.8 clocks of a SIMD
// for 64), which bounds a layer of 16 states and more; with fewer, and for
// single tokens, memory bounds it.
//
// Why four lanes: lane q of a channel prepares step 4k+q (its loads, softplus
// and gate), and the group shares the results through the DPP crossbar, which
// is free as an operand of the products; y's sum over the lanes takes three
// exchanges for four steps (quad_sum4).  A wave so needs nothing from other
// waves but the tile of B and C in shared memory, f32, double-buffered, one
// barrier a tile of 16 or 32 steps; the next tile's rows are in flight
// meanwhile.
//
// Few rows: the time axis is cut into chunks.  A first launch gives each
// chunk's end state from a zero state and its sum of step sizes (the decay
// over a chunk is exp(A * sum)); the second joins them at its start.  That
// costs the recurrence twice, so it is done only where the chunks fill a chip
// that the rows alone leave empty (rule in seq_api.cpp).
#include "scan_device.h"

namespace rnnhip {
namespace {

// LOCAL: the first of two launches (end states and sums of all chunks but
// each row's last); else the outputs.
template <typename T, int NS, bool LOCAL>
__global__ __launch_bounds__(256) void scan_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, TT = scan_tile(NS), TG = TT / 4;
  __shared__ float sB[2][TT][NP];
  __shared__ float sC[LOCAL ? 1 : 2][LOCAL ? 1 : TT][NP];
  const ScanPlace p = scan_place(a, LOCAL ? a.nchunk - 1 : a.nchunk);
  const int b = p.b, ch = p.ch;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  const int s1 = int(min(int64_t(s0) + a.chunk, int64_t(a.geo.S)));
  const int send = min(s1, L);
  if (LOCAL && s1 >= L) return;   // nothing follows this chunk (uniform)
  const int tid = int(threadIdx.x), q = tid & 3;
  const bool q1 = q & 1, q2 = q & 2;
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t cs = int64_t(b) * a.C + p.c;   // the channel among all rows' states

  float h[NS], A[NS];
  scan_load_A<NS>(a, p.c, q, A);
  if (ch == 0 && !LOCAL && a.init && s1 < L) {
    // the first launch's copy: the last chunk's workgroup may be writing the
    // final state over the initial one
    scan_get<NS>(a.first + cs * NP + q * NS, h);
  } else if (ch == 0) {
    scan_load_state<NS>(a, a.init, cs, q, h);
    if (LOCAL && a.init && p.ok) scan_put<NS>(a.first + cs * NP + q * NS, h);
  } else if (LOCAL) {
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = 0.f;
  } else if (s0 < L) {
    scan_join<NS>(a, b, ch, p.c, q, A, h);
  }

  const float bias = a.dbias ? a.dbias[p.c] : 0.f;
  const float skip = !LOCAL && a.D ? a.D[p.c] : 0.f;
  float total = 0.f;   // LOCAL: this lane's share of the sum of step sizes

  if (s0 < send) {
    const int64_t dx = r.step * a.X.rs, dd = r.step * a.delta.rs, dz = r.step * a.Z.rs, dy = r.step * a.Y.rs;
    const T* X = reinterpret_cast<const T*>(a.X.p) + r.base * a.X.rs + p.c;
    const T* De = reinterpret_cast<const T*>(a.delta.p) + r.base * a.delta.rs + p.c;
    const T* Z = reinterpret_cast<const T*>(a.Z.p) + r.base * a.Z.rs + p.c;
    T* Y = reinterpret_cast<T*>(a.Y.p) + r.base * a.Y.rs + p.c;
    const bool gate = !LOCAL && a.have_z;
    BCTile<T, NS, TT, LOCAL ? 1 : 2> bc;
    T nx[TG], nd[TG], nz[TG];
    auto fetch = [&](int s) {
      bc.fetch(a, r, p.g, s, send, tid);
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const int64_t at = min(s + 4 * k + q, send - 1);
        nx[k] = X[at * dx];
        nd[k] = De[at * dd];
        if (gate) nz[k] = Z[at * dz];
      }
    };
    fetch(s0);
    int buf = 0;
    for (int s = s0; s < send; s += TT, buf ^= 1) {
      bc.put(sB[buf], LOCAL ? nullptr : sC[buf], tid);
      T cx[TG], cd[TG], cz[TG];
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        cx[k] = nx[k];
        cd[k] = nd[k];
        if (gate) cz[k] = nz[k];
      }
      __syncthreads();
      if (s + TT < send) fetch(s + TT);
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        if (s + 4 * k < send) {
          const bool live = s + 4 * k + q < send;
          const float x = live ? float(cx[k]) : 0.f;
          float d = float(cd[k]) + bias;
          if (a.softplus) d = softplus(d);
          d = live ? d : 0.f;
          const float u = d * x;
          if constexpr (LOCAL) total += d;
          float acc[4];
          auto step = [&](auto J) {
            constexpr int j = decltype(J)::value;
            const float dj = quad_of<j>(d), uj = quad_of<j>(u);
            float Bv[NS], Cv[NS];
            tile_get<NS>(sB[buf][4 * k + j], q, Bv);
            if constexpr (!LOCAL) tile_get<NS>(sC[buf][4 * k + j], q, Cv);
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              const float e = __builtin_amdgcn_exp2f(dj * A[i]);
              h[i] = __builtin_fmaf(e, h[i], uj * Bv[i]);
              if constexpr (!LOCAL) y = __builtin_fmaf(h[i], Cv[i], y);
            }
            acc[j] = y;
          };
          step(IntC<0>{});
          step(IntC<1>{});
          step(IntC<2>{});
          step(IntC<3>{});
          if constexpr (!LOCAL) {
            float y = quad_sum4(acc[0], acc[1], acc[2], acc[3], q1, q2);
            y = __builtin_fmaf(skip, x, y);
            if (gate) {
              const float z = float(cz[k]);
              y *= z * logistic(z);
            }
            if (live && p.ok && a.Y.p) Y[int64_t(s + 4 * k + q) * dy] = T(y);
          }
        }
      }
    }
  }

  if constexpr (LOCAL) {
    total = quad_sum(total);
    if (p.ok) {
      const int64_t at = (int64_t(b) * a.nchunk + ch) * a.C + p.c;
      scan_put<NS>(a.loc + at * NP + q * NS, h);
      if (q == 0) a.sum[at] = total;
    }
  } else {
    if (a.Y.p && p.ok)
      for (int s = max(s0, send) + q; s < s1; s += 4)
        (reinterpret_cast<T*>(a.Y.p) + p.c)[dead_row(a.geo, b, s) * a.Y.rs] = T(0.f);
    // the row's last step is in this chunk (a row of no steps: the first)
    if (a.fin && p.ok && ch == (L > 0 ? (L - 1) / a.chunk : 0)) scan_store_state<NS>(a, a.fin, cs, q, h);
  }
}

template <typename T, bool LOCAL>
hipError_t scan_n(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * (LOCAL ? a.nchunk - 1 : a.nchunk) * a.G * a.cbg;
  switch (a.np / 4) {
    case 1: return go(scan_kernel<T, 1, LOCAL>, blocks, 256, a, s);
    case 2: return go(scan_kernel<T, 2, LOCAL>, blocks, 256, a, s);
    case 4: return go(scan_kernel<T, 4, LOCAL>, blocks, 256, a, s);
    case 8: return go(scan_kernel<T, 8, LOCAL>, blocks, 256, a, s);
    case 16: return go(scan_kernel<T, 16, LOCAL>, blocks, 256, a, s);
    case 32: return go(scan_kernel<T, 32, LOCAL>, blocks, 256, a, s);
    default: return hipErrorInvalidValue;
  }
}

template <bool LOCAL>
hipError_t scan_t(const ScanArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return scan_n<float, LOCAL>(a, s);
    case RNN_DTYPE_F16: return scan_n<f16_t, LOCAL>(a, s);
    default: return scan_n<bf16_t, LOCAL>(a, s);
  }
}

}  // namespace

hipError_t launch_scan_local(const ScanArgs& a, int dtype, hipStream_t s) { return scan_t<true>(a, dtype, s); }
hipError_t launch_scan(const ScanArgs& a, int dtype, hipStream_t s) { return scan_t<false>(a, dtype, s); }

}  // namespace rnnhip
