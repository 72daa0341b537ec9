// k_scan_grad.hip -- the selective scan's gradient.
//
// With gy = dY silu(z) (or dY), a_s = exp(d_s A), u_s = d_s x_s:
//   G_s  = C_s gy_s + a_{s+1} G_{s+1}           (after the last step: d_final)
//   q_s  = G_s a_s h_{s-1}                       = dL/d(d_s A)
//   dA   = sum q_s d_s;    dd_s = sum_n q_s A + x_s sum_n G_s B_s
//   dx_s = d_s sum_n G_s B_s + D gy_s;           dB_s = sum_c G_s u_s
//   dC_s = sum_c gy_s h_s;  dD = sum gy_s x_s;   dz_s = dY y_s silu'(z)
//   d_initial = a_0 G_0
// Nothing of the forward pass is kept.  Three launches:
//   1. along time: states, written before each segment of `segment` steps, and
//      each chunk's end state, sum of step sizes and gradient at its start.
//      That gradient needs no walk back: sum_s (prod_{r<=s} a_r) C_s gy_s runs
//      forward with the product, at three operations and no exponential.
//   2. each chunk, segment after segment from its end: the segment's states
//      and decays forward from the one written, kept in registers (64 of each
//      a lane), then the gradients backward.
//   3. sums of the workgroups' dB, dC, dA, dD, ddelta_bias, in a fixed order.
// Chunks start from zero states; a segment's true state is the written one
// plus decay(chunk start -> segment) times the chunk's true start, joined from
// the chunks before as in the forward pass, and the gradient at a chunk's end
// likewise from those after.
//
// dB and dC sum over channels, which lie across lanes: sixteen such values
// are folded over the sixteen channels of a wave at once (fold16), each
// exchange halving what is left, about two instructions a value where one sum
// after another would take twelve; the four waves' parts meet in shared
// memory.
#include "scan_device.h"

namespace rnnhip {
namespace {

template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_into(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL,
                                                               0xf, BANKS, false));
}

// Sixteen sums over a wave's sixteen channels (lane / 4): lane l gets that of
// v[l >> 2] over the lanes of its l & 3.  Lane bit 5 chooses v's bit 3, bit 4
// bit 2 (swaps of half waves and of rows of 16), bits 3 and 2 v's bits 1 and 0
// (DPP moves within a row, each half of the row from another register).
__device__ __forceinline__ float fold16(const float (&v)[16], bool b3, bool b2) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v[j]), __builtin_bit_cast(unsigned, v[j + 8]),
                                                    false, false);
    r[j] = __builtin_bit_cast(float, unsigned(p[0])) + __builtin_bit_cast(float, unsigned(p[1]));
  }
  float t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, r[j]), __builtin_bit_cast(unsigned, r[j + 4]),
                                                    false, false);
    t[j] = __builtin_bit_cast(float, unsigned(p[0])) + __builtin_bit_cast(float, unsigned(p[1]));
  }
  float w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // lanes with bit 3 clear end with t[j]'s sum, the others with t[j+2]'s
    const float keep = b3 ? t[j + 2] : t[j], give = b3 ? t[j] : t[j + 2];
    w[j] = keep + dpp_into<0x128, 0xf>(0.f, give);   // row_ror:8
  }
  const float keep = b2 ? w[1] : w[0], give = b2 ? w[0] : w[1];
  // lane ^ 4: banks 0 and 2 take from four lanes up, banks 1 and 3 from four down
  const float m = dpp_into<0x114, 0xa>(dpp_into<0x104, 0x5>(0.f, give), give);   // row_shl:4, row_shr:4
  return keep + m;
}

template <typename T>
__device__ __forceinline__ float gate_of(float z) { return z * logistic(z); }

// Launch 1.
template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_ahead_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, TT = scan_tile(NS), TG = TT / 4, TS = NS <= 4 ? 16 : NS == 8 ? 8 : 4;
  __shared__ float sB[2][TT][NP];
  __shared__ float sC[2][TT][NP];
  const ScanPlace p = scan_place(a, a.nchunk);
  const int b = p.b, ch = p.ch;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  if (s0 >= L) return;   // uniform
  const int send = int(min(int64_t(s0) + a.chunk, int64_t(L)));
  const int tid = int(threadIdx.x), q = tid & 3;
  const StepRows r = step_rows(a.geo, b, L);

  float h[NS], A[NS], P[NS], G[NS];
  scan_load_A<NS>(a, p.c, q, A);
  scan_load_state<NS>(a, ch == 0 ? a.init : nullptr, int64_t(b) * a.C + p.c, q, h);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    P[i] = 1.f;
    G[i] = 0.f;
  }
  const float bias = a.dbias ? a.dbias[p.c] : 0.f;
  float total = 0.f;
  const bool behind = ch > 0;   // a chunk before this one needs the gradient at its start

  const int64_t dx = r.step * a.X.rs, dd = r.step * a.delta.rs, dz = r.step * a.Z.rs, dg = r.step * a.dY.rs;
  const T* X = reinterpret_cast<const T*>(a.X.p) + r.base * a.X.rs + p.c;
  const T* De = reinterpret_cast<const T*>(a.delta.p) + r.base * a.delta.rs + p.c;
  const T* Z = reinterpret_cast<const T*>(a.Z.p) + r.base * a.Z.rs + p.c;
  const T* Dy = reinterpret_cast<const T*>(a.dY.p) + r.base * a.dY.rs + p.c;
  BCTile<T, NS, TT, 2> bc;
  T nx[TG], nd[TG], nz[TG], ng[TG];
  auto fetch = [&](int s) {
    bc.fetch(a, r, p.g, s, send, tid);
#pragma unroll
    for (int k = 0; k < TG; ++k) {
      const int64_t at = min(s + 4 * k + q, send - 1);
      nx[k] = X[at * dx];
      nd[k] = De[at * dd];
      if (behind) {
        ng[k] = Dy[at * dg];
        if (a.have_z) nz[k] = Z[at * dz];
      }
    }
  };
  fetch(s0);
  int buf = 0;
  for (int s = s0; s < send; s += TT, buf ^= 1) {
    bc.put(sB[buf], sC[buf], tid);
    T cx[TG], cd[TG], cz[TG], cg[TG];
#pragma unroll
    for (int k = 0; k < TG; ++k) {
      cx[k] = nx[k];
      cd[k] = nd[k];
      if (behind) {
        cg[k] = ng[k];
        if (a.have_z) cz[k] = nz[k];
      }
    }
    __syncthreads();
    if (s + TT < send) fetch(s + TT);
#pragma unroll
    for (int k = 0; k < TG; ++k) {
      const int sg = s + 4 * k;
      if (sg < send) {
        if (4 * k % TS == 0 && p.ok) {   // a segment begins
          const int64_t at = (int64_t(b) * a.nseg + sg / TS) * a.C + p.c;
          scan_put<NS>(a.ckpt + at * NP + q * NS, h);
          if (q == 0) a.cum[at] = total;
        }
        const bool live = sg + q < send;
        const float x = live ? float(cx[k]) : 0.f;
        float d = float(cd[k]) + bias;
        if (a.softplus) d = softplus(d);
        d = live ? d : 0.f;
        const float u = d * x;
        total += quad_sum(d);
        float gy = 0.f;
        if (behind) {
          gy = live ? float(cg[k]) : 0.f;
          if (a.have_z) gy = live ? gy * gate_of<T>(float(cz[k])) : 0.f;
        }
        auto step = [&](auto J) {
          constexpr int j = decltype(J)::value;
          const float dj = quad_of<j>(d), uj = quad_of<j>(u), gj = quad_of<j>(gy);
          float Bv[NS], Cv[NS];
          tile_get<NS>(sB[buf][4 * k + j], q, Bv);
          if (behind) tile_get<NS>(sC[buf][4 * k + j], q, Cv);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float e = __builtin_amdgcn_exp2f(dj * A[i]);
            h[i] = __builtin_fmaf(e, h[i], uj * Bv[i]);
            if (behind) {
              P[i] *= e;
              G[i] = __builtin_fmaf(P[i], gj * Cv[i], G[i]);
            }
          }
        };
        step(IntC<0>{});
        step(IntC<1>{});
        step(IntC<2>{});
        step(IntC<3>{});
      }
    }
  }
  if (p.ok && a.nchunk > 1) {
    const int64_t at = (int64_t(b) * a.nchunk + ch) * a.C + p.c;
    scan_put<NS>(a.loc + at * NP + q * NS, h);
    if (behind) scan_put<NS>(a.gloc + at * NP + q * NS, G);
    if (q == 0) a.sum[at] = total;
  }
}

// Launch 2.
template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_back_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, TS = NS <= 4 ? 16 : NS == 8 ? 8 : 4, TG = TS / 4;
  constexpr int NV = TS * NS * 2 / 16;   // folds of sixteen a segment
  __shared__ float sB[2][TS][NP];
  __shared__ float sC[2][TS][NP];
  __shared__ float red[2][4][NV][64];
  const ScanPlace p = scan_place(a, a.nchunk);
  const int b = p.b, ch = p.ch;
  const int L = geo_len(a.geo, b);
  const int s0 = ch * a.chunk;
  const int s1 = int(min(int64_t(s0) + a.chunk, int64_t(a.geo.S)));
  const int send = min(s1, L);
  const int tid = int(threadIdx.x), q = tid & 3, lane = tid & 63, wave = tid >> 6;
  const bool q1 = q & 1, q2 = q & 2, b3 = lane & 8, b2 = lane & 4;
  const StepRows r = step_rows(a.geo, b, L);
  const int64_t cs = int64_t(b) * a.C + p.c;

  float dA[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;
  float dD = 0.f, dbias = 0.f;

  if (s0 < send) {
    float A[NS], G[NS], hs[NS];
    scan_load_A<NS>(a, p.c, q, A);
    const bool joined = ch > 0;
    if (joined) scan_join<NS>(a, b, ch, p.c, q, A, hs);
    // a lane past its group's channels adds nothing to dB and dC: all its
    // values are zero
    // the gradient at the chunk's end, from the chunks after it
    scan_load_state<NS>(a, a.dfin, cs, q, G);
    for (int j = (L - 1) / a.chunk; j > ch; --j) {
      const int64_t at = (int64_t(b) * a.nchunk + j) * a.C + p.c;
      float l[NS];
      scan_get<NS>(a.gloc + at * NP + q * NS, l);
      const float sum = a.sum[at];
#pragma unroll
      for (int i = 0; i < NS; ++i) G[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(A[i] * sum), G[i], l[i]);
    }
    if (!p.ok) {
#pragma unroll
      for (int i = 0; i < NS; ++i) A[i] = G[i] = hs[i] = 0.f;
    }
    const float bias = a.dbias ? a.dbias[p.c] : 0.f;
    const float skip = a.D ? a.D[p.c] : 0.f;
    const int64_t xd = r.step * a.X.rs, dd = r.step * a.delta.rs, zd = r.step * a.Z.rs, gd = r.step * a.dY.rs;
    const T* X = reinterpret_cast<const T*>(a.X.p) + r.base * a.X.rs + p.c;
    const T* De = reinterpret_cast<const T*>(a.delta.p) + r.base * a.delta.rs + p.c;
    const T* Z = reinterpret_cast<const T*>(a.Z.p) + r.base * a.Z.rs + p.c;
    const T* Dy = reinterpret_cast<const T*>(a.dY.p) + r.base * a.dY.rs + p.c;
    BCTile<T, NS, TS, 2> bc;
    T nx[TG], nd[TG], nz[TG], ng[TG];
    float nh[NS], ncum = 0.f;
    auto fetch = [&](int s) {
      bc.fetch(a, r, p.g, s, send, tid);
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const int64_t at = min(s + 4 * k + q, send - 1);
        nx[k] = X[at * xd];
        nd[k] = De[at * dd];
        ng[k] = Dy[at * gd];
        if (a.have_z) nz[k] = Z[at * zd];
      }
      const int64_t at = (int64_t(b) * a.nseg + s / TS) * a.C + p.c;
      scan_get<NS>(a.ckpt + at * NP + q * NS, nh);
      if (joined) ncum = a.cum[at];
    };
    // the four waves' dB and dC of a segment that began at s, to memory
    auto finish = [&](int s, int rb) {
      for (int e = tid; e < NV * 64; e += 256) {
        const int f = e >> 6, l = e & 63;
        const float v = ((red[rb][0][f][l] + red[rb][1][f][l]) + red[rb][2][f][l]) + red[rb][3][f][l];
        // fold f, lane l: value 16 f + (l >> 2) of [step][B, C][NS], lane share l & 3
        const int at = 16 * f + (l >> 2);
        const int st = s + at / (2 * NS), which = at / NS % 2, n = (l & 3) * NS + at % NS;
        if (st < send && n < a.N)
          a.pbc[(((int64_t(p.cb) * a.geo.B + b) * a.geo.S + st) * 2 + which) * NP + n] = v;
      }
    };
    const int last = s0 + (send - 1 - s0) / TS * TS;
    fetch(last);
    int buf = 0;
    for (int s = last; s >= s0; s -= TS, buf ^= 1) {
      bc.put(sB[buf], sC[buf], tid);
      float x[TG], d[TG], g[TG], gy[TG], z[TG], raw[TG], h0[NS];
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const bool live = p.ok && s + 4 * k + q < send;
        x[k] = live ? float(nx[k]) : 0.f;
        raw[k] = float(nd[k]) + bias;
        d[k] = live ? (a.softplus ? softplus(raw[k]) : raw[k]) : 0.f;
        g[k] = live ? float(ng[k]) : 0.f;
        z[k] = a.have_z && live ? float(nz[k]) : 0.f;
        gy[k] = a.have_z ? g[k] * gate_of<T>(z[k]) : g[k];
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        h0[i] = p.ok ? nh[i] : 0.f;
        if (joined) h0[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(A[i] * ncum), hs[i], h0[i]);
      }
      __syncthreads();
      if (s != last) finish(s + TS, buf ^ 1);
      if (s > s0) fetch(s - TS);

      float h[TS][NS], e[TS][NS];
      float y[TG];
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        float acc[4];
        auto step = [&](auto J) {
          constexpr int j = decltype(J)::value;
          const int t = 4 * k + j;
          const float dj = quad_of<j>(d[k]), uj = quad_of<j>(d[k] * x[k]);
          float Bv[NS], Cv[NS];
          tile_get<NS>(sB[buf][t], q, Bv);
          tile_get<NS>(sC[buf][t], q, Cv);
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            e[t][i] = __builtin_amdgcn_exp2f(dj * A[i]);
            h[t][i] = __builtin_fmaf(e[t][i], t ? h[t ? t - 1 : 0][i] : h0[i], uj * Bv[i]);
            v = __builtin_fmaf(h[t][i], Cv[i], v);
          }
          acc[j] = v;
        };
        step(IntC<0>{});
        step(IntC<1>{});
        step(IntC<2>{});
        step(IntC<3>{});
        y[k] = quad_sum4(acc[0], acc[1], acc[2], acc[3], q1, q2);
      }
      float v16[16];
#pragma unroll
      for (int k = TG - 1; k >= 0; --k) {
        float gb[4], qa[4];
        auto step = [&](auto J) {
          constexpr int j = decltype(J)::value;
          const int t = 4 * k + j;
          const float dj = quad_of<j>(d[k]), uj = quad_of<j>(d[k] * x[k]), gj = quad_of<j>(gy[k]);
          float Bv[NS], Cv[NS];
          tile_get<NS>(sB[buf][t], q, Bv);
          tile_get<NS>(sC[buf][t], q, Cv);
          float sb = 0.f, sq = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            G[i] = __builtin_fmaf(gj, Cv[i], G[i]);
            sb = __builtin_fmaf(G[i], Bv[i], sb);
            const int at = t * 2 * NS + i;   // place among the segment's [step][B, C][NS]
            v16[at % 16] = G[i] * uj;
            if constexpr (NS < 16) v16[(at + NS) % 16] = gj * h[t][i];   // (with more states dC's folds follow dB's)
            G[i] *= e[t][i];
            const float qi = G[i] * (t ? h[t ? t - 1 : 0][i] : h0[i]);
            sq = __builtin_fmaf(qi, A[i], sq);
            dA[i] = __builtin_fmaf(qi, dj, dA[i]);
            if constexpr (NS >= 16) {
              if (i % 16 == 15) red[buf][wave][at / 16][lane] = fold16(v16, b3, b2);
            }
          }
          if constexpr (NS >= 16) {
#pragma unroll
            for (int i0 = 0; i0 < NS; i0 += 16) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v16[i] = gj * h[t][i0 + i];
              red[buf][wave][(t * 2 * NS + NS + i0) / 16][lane] = fold16(v16, b3, b2);
            }
          } else if (t * 2 * NS % 16 == 0) {
            red[buf][wave][t * 2 * NS / 16][lane] = fold16(v16, b3, b2);
          }
          gb[j] = sb;
          qa[j] = sq;
        };
        step(IntC<3>{});
        step(IntC<2>{});
        step(IntC<1>{});
        step(IntC<0>{});
        const float sb = quad_sum4(gb[0], gb[1], gb[2], gb[3], q1, q2);
        const float sq = quad_sum4(qa[0], qa[1], qa[2], qa[3], q1, q2);
        const int st = s + 4 * k + q;
        if (st < send) {
          const int64_t row = r.base + st * r.step;
          float dr = __builtin_fmaf(x[k], sb, sq * kLn2);   // (A carries log2(e))
          if (a.softplus) dr *= logistic(raw[k]);
          dbias += dr;
          dD = __builtin_fmaf(gy[k], x[k], dD);
          if (p.ok) {
            if (a.dX.p) (reinterpret_cast<T*>(a.dX.p) + p.c)[row * a.dX.rs] = T(__builtin_fmaf(d[k], sb, skip * gy[k]));
            if (a.ddelta.p) (reinterpret_cast<T*>(a.ddelta.p) + p.c)[row * a.ddelta.rs] = T(dr);
            if (a.dZ.p) {
              const float sg = logistic(z[k]);
              (reinterpret_cast<T*>(a.dZ.p) + p.c)[row * a.dZ.rs] =
                  T(g[k] * __builtin_fmaf(skip, x[k], y[k]) * (sg * __builtin_fmaf(z[k], 1.f - sg, 1.f)));
            }
          }
        }
      }
    }
    __syncthreads();
    finish(s0, buf ^ 1);
    if (ch == 0 && a.dinit && p.ok) scan_store_state<NS>(a, a.dinit, cs, q, G);
  } else if (ch == 0 && a.dinit && p.ok) {   // a row of no steps
    float G[NS];
    scan_load_state<NS>(a, a.dfin, cs, q, G);
    scan_store_state<NS>(a, a.dinit, cs, q, G);
  }

  if (p.ok) {
    // rows past the length: zero
    for (int s = max(s0, send) + q; s < s1; s += 4) {
      const int64_t row = dead_row(a.geo, b, s);
      if (a.dX.p) (reinterpret_cast<T*>(a.dX.p) + p.c)[row * a.dX.rs] = T(0.f);
      if (a.ddelta.p) (reinterpret_cast<T*>(a.ddelta.p) + p.c)[row * a.ddelta.rs] = T(0.f);
      if (a.dZ.p) (reinterpret_cast<T*>(a.dZ.p) + p.c)[row * a.dZ.rs] = T(0.f);
    }
    const int64_t part = int64_t(b) * a.nchunk + ch;
    if (a.dA) scan_put<NS>(a.pA + (part * a.C + p.c) * NP + q * NS, dA);
    if (a.dD || a.ddbias) {
      dD = quad_sum(dD);
      dbias = quad_sum(dbias);
      if (q == 0) {
        a.pD[part * 2 * a.C + p.c] = dD;
        a.pD[(part * 2 + 1) * a.C + p.c] = dbias;
      }
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
  if (int64_t(blockIdx.x) < nbc) {
    const int64_t i = int64_t(blockIdx.x) * 256 + tid;
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
      const float* p = a.pbc + int64_t(g) * a.cbg * per + (row * 2 + which) * a.np + n;
#pragma unroll 4
      for (int k = 0; k < a.cbg; ++k) v += p[k * per];
      if (a.geo.reverse) t = L - 1 - s;
    }
    reinterpret_cast<T*>(out.p)[dead_row(a.geo, b, t) * out.rs + gi] = T(v);
    return;
  }
  __shared__ float red[3][64];
  const int64_t ncA = a.dA ? (int64_t(a.C) * a.np + 63) / 64 : 0;
  const int64_t blk = int64_t(blockIdx.x) - nbc;
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
    const int64_t c = col / a.np;
    const int n = int(col - c * a.np);
    if (n < a.N) a.dA[c * a.N + n] = v;
  } else if (col < a.C) {
    if (a.dD) a.dD[col] = v;
  } else if (a.ddbias) {
    a.ddbias[col - a.C] = v;
  }
}

template <typename T, int NS>
hipError_t back_ns(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.geo.B) * a.nchunk * a.G * a.cbg;
  if (hipError_t e = go(scan_ahead_kernel<T, NS>, blocks, 256, a, s); e != hipSuccess) return e;
  return go(scan_back_kernel<T, NS>, blocks, 256, a, s);
}

template <typename T>
hipError_t back_t(const ScanArgs& a, hipStream_t s) {
  hipError_t e;
  switch (a.np / 4) {
    case 1: e = back_ns<T, 1>(a, s); break;
    case 2: e = back_ns<T, 2>(a, s); break;
    case 4: e = back_ns<T, 4>(a, s); break;
    case 8: e = back_ns<T, 8>(a, s); break;
    case 16: e = back_ns<T, 16>(a, s); break;
    case 32: e = back_ns<T, 32>(a, s); break;
    default: return hipErrorInvalidValue;
  }
  if (e != hipSuccess) return e;
  int64_t blocks = 0;
  if (a.dB.p || a.dC.p) blocks += (int64_t(a.geo.B) * a.geo.S * 2 * a.G * a.N + 255) / 256;
  if (a.dA) blocks += (int64_t(a.C) * a.np + 63) / 64;
  if (a.dD || a.ddbias) blocks += (2 * int64_t(a.C) + 63) / 64;
  return go(scan_sums_kernel<T>, blocks, 256, a, s);
}

}  // namespace

hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RNN_DTYPE_F32: return back_t<float>(a, s);
    case RNN_DTYPE_F16: return back_t<f16_t>(a, s);
    default: return back_t<bf16_t>(a, s);
  }
}

}  // namespace rnnhip
