// attn_api.cpp -- the C ABI of linear attention and of the norms and rotations
// of its queries and keys: validation, scratch sizing, the launches of a call.
// Every check runs in 64-bit checked arithmetic before anything is enqueued;
// messages name operator and argument.
#include <cmath>
#include <cstdlib>
#include <new>

#include "attn_ops.h"
#include "seq_check.h"

using namespace rnnhip;

// The time axis of a call in pieces.
struct AttnPlan {
  int piece, pieces, sub;
};

struct rnn_attn {
  rnn_attn_desc d;
  int es;
  int per;                    // heads of a group
  int key_cols, value_cols;   // workgroups along a head's keys and values
  bool tokens;                // step after step
  AttnPlan f, b, bd;          // forward; the gradient without and with the decays'
  size_t forward_bytes, backward_bytes;
};

struct rnn_rotary {
  rnn_rotary_desc d;
  int es;
  int64_t parts;          // workgroups of the gradient
  size_t backward_bytes;
};

namespace {

const char kAttn[] = "linear attention", kRotary[] = "rotary norm";

// The pieces of a call whose walks have `blocks` workgroups a piece: as many as
// have 256 in all (one a CU; more take turns), of 128 steps at least, two chunks.
// (Time axes in one piece and in the rule's, forward, us: 1 x 512 steps, 16 heads of
// 128 x 128, bf16, 25 and 19; 1 x 2048 79 and 33; 4 x 1024 44 and 41; 5 x 1024 of 8
// heads 44 and 34; 8 x 1024, 256 workgroups, 48, and in two pieces 72.)  `most`:
// steps of a piece at most.
AttnPlan attn_plan(const rnn_attn_desc& d, bool tokens, int64_t blocks, int64_t most) {
  if (tokens) return {int(std::max<int64_t>(d.seq, 1)), 1, 0};
  const int64_t whole = ceil_div(d.seq, 64) * 64;
  int64_t piece = whole;
  if (blocks <= 128) piece = std::max<int64_t>(ceil_div(ceil_div(whole, 256 / std::max<int64_t>(blocks, 1)), 64) * 64, 128);
  piece = std::min(std::min(piece, most), whole);
  if (const char* e = std::getenv("RNN_ATTN_PIECE")) {
    const int64_t c = std::atoll(e);
    if (c > 0) piece = c >= whole ? whole : ceil_div(c, 64) * 64;
  }
  return {int(piece), int(ceil_div(d.seq, piece)), 0};
}

// Few pieces' walks join what the pieces before them leave by themselves, without a
// launch, and then these are walked for their states in parts that fill the chip,
// too.  (Two pieces of 1024 steps, 128 workgroups a piece, bf16: 63 us in two parts
// each, 73 joined by a launch; eight of 512, 32 workgroups, f16: 50.3, 51.0.)
int attn_sub(const AttnPlan& f, int64_t blocks) {
  const int64_t before = f.pieces - 1;
  if (before < 1 || before > kAttnParts) return 0;
  int sub = 1;
  while (2 * sub * before <= kAttnParts && 2 * sub * before * blocks <= 256 && f.piece % (128 * sub) == 0 && f.piece / (2 * sub) >= 128) sub *= 2;
  return sub;
}

// Whether a gradient's walks go side by side in one launch: those that do not fill
// the chip.  A rule on the sizes alone: an output is the same whichever others are
// asked for, but for the decays' gradient, which has its own pieces and its own way
// with a step's own part.  (5 x 80 steps, 4 heads of 24 x 30, f32: 22 us, one after another 51.)
bool attn_side_by_side(const rnn_attn& p, const AttnPlan& plan) {
  return !p.tokens && p.d.batch * p.d.heads * (2 * p.key_cols + p.value_cols) * plan.pieces <= 256;
}

// Whether the launches of walks of `cols` workgroups a head and piece fit: the walks
// themselves (256 threads a workgroup step after step, 512 over chunks) and, of more
// pieces than one, their join.
bool attn_fits(const rnn_attn& p, const AttnPlan& plan, int cols) {
  const int64_t heads = p.d.batch * p.d.heads;   // (at most 2^54)
  return heads * cols <= kMaxThreads / (p.tokens ? 256 : 512) / plan.pieces &&
         (plan.pieces == 1 || heads <= kMaxThreads / 256 / ceil_div(p.d.key * p.d.value, 256));
}

// The scratch regions of the two directions, in the order that they are taken.
struct AttnScratch {
  size_t starts, totals, back_starts, back_totals, rows, cols, ends, decay, part[2];
};
bool attn_scratch(const rnn_attn& p, bool backward, AttnScratch* at, size_t* total) {
  const rnn_attn_desc& d = p.d;
  const int64_t pieces = backward ? std::max(p.b.pieces, p.bd.pieces) : int64_t(p.f.pieces) * std::max(p.f.sub, 1);
  Regions r;
  *at = AttnScratch{};
  if (pieces > 1) {
    at->starts = r.take({d.batch, d.heads, pieces, d.key, d.value, 4});
    at->totals = r.take({d.batch, d.heads, pieces, 4});
  }
  if (backward) {
    if (pieces > 1) {
      at->back_starts = r.take({d.batch, d.heads, pieces, d.key, d.value, 4});
      at->back_totals = r.take({d.batch, d.heads, pieces, 4});
    }
    at->rows = r.take({p.key_cols, d.batch, d.heads, d.seq, 4});
    at->cols = r.take({p.key_cols, d.batch, d.heads, d.seq, 4});
    at->ends = r.take({p.key_cols, d.batch, d.heads, p.bd.pieces, 4});
    at->decay = r.take({d.batch, d.heads, p.bd.pieces, 4});
    const bool two = attn_side_by_side(p, p.b) || attn_side_by_side(p, p.bd);
    for (int k = 0; p.per > 1 && k < (two ? 2 : 1); ++k) at->part[k] = r.take({d.seq, d.batch, d.heads, d.key, 4});
  }
  *total = r.off;
  return r.ok;
}

HeadRows head_rows(const Rows& r, int per) { return HeadRows{r.p, r.rs, per}; }

// The operands both directions read.
struct AttnInputs {
  HeadRows Q, K, V;
  const float* init;
};
AttnInputs attn_inputs(const rnn_attn& p, const rnn_attn_operands& o, Tensors& t, AttnArgs& a) {
  const rnn_attn_desc& d = p.d;
  const int64_t rows = d.seq * d.batch, gk = d.groups * d.key, hv = d.heads * d.value;
  const bool any = rows > 0;
  AttnInputs in{};
  in.Q = head_rows(t.rows(o.Q, p.es, gk, rows, "Q", any), p.per);
  in.K = head_rows(t.rows(o.K, p.es, gk, rows, "K", any), p.per);
  in.V = head_rows(t.rows(o.V, p.es, hv, rows, "V", any), 1);
  a.G = t.rows(o.G, 4, d.heads, rows, "G", false);
  a.decay = reinterpret_cast<const float*>(t.tensor(o.decay, 4, "decay", false));
  a.geo = geometry(d.seq, d.batch, d.layout, d.direction, t.tensor(o.sequence_lens, 4, "sequence_lens", false));
  in.init = reinterpret_cast<const float*>(t.tensor(o.initial_state, 4, kInitial, false));
  a.H = int(d.heads);
  return in;
}

// One walk of all pieces.
hipError_t attn_walk(const rnn_attn& p, const AttnArgs& a, bool local, hipStream_t s) {
  if (p.tokens) return launch_attn_steps(a, p.d.dtype, s);
  return p.d.dtype == RNN_DTYPE_F32   ? launch_attn_chunks_f32(a, local, s)
         : p.d.dtype == RNN_DTYPE_F16 ? launch_attn_chunks_f16(a, local, s)
                                      : launch_attn_chunks_bf16(a, local, s);
}

// A few walks in one launch, as wide as any of the problem's: width decides the
// chunks, and so the bits of an output, whichever others go along.
hipError_t attn_walks(const rnn_attn& p, const AttnArgs* w, int n, hipStream_t s) {
  const int K = int(std::max(p.d.key, p.d.value));
  return p.d.dtype == RNN_DTYPE_F32   ? launch_attn_walks_f32(w, n, K, s)
         : p.d.dtype == RNN_DTYPE_F16 ? launch_attn_walks_f16(w, n, K, s)
                                      : launch_attn_walks_bf16(w, n, K, s);
}

int attn_launch(const char* what, hipError_t e) {
  return e == hipSuccess ? RNN_OK : fail(RNN_ERR_HIP, kAttn, "%s launch: %s", what, hipGetErrorString(e));
}

// The states that the pieces of a walk begin with, from `init`.
int attn_starts(const rnn_attn& p, const AttnArgs& a, hipStream_t s) {
  if (a.pieces == 1) return RNN_OK;
  AttnArgs w = a;
  w.K = int(p.d.key), w.V = int(p.d.value);
  w.sk = int(p.d.value), w.sv = 1;
  w.dots = w.ends = nullptr;
  if (int rc = attn_launch("pieces", attn_walk(p, w, true, s))) return rc;
  if (a.sub) return RNN_OK;
  const AttnJoinArgs j{a.pieces, a.back, p.d.batch * p.d.heads, p.d.key * p.d.value, a.starts, a.totals, a.init};
  return attn_launch("join", launch_attn_join(j, s));
}

}  // namespace

extern "C" int rnn_attn_create(const rnn_attn_desc* desc, rnn_attn** out) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (out) *out = nullptr;
  if (!desc) return fail(RNN_ERR_ARG, kAttn, "desc: NULL");
  if (!out) return fail(RNN_ERR_ARG, kAttn, "out: NULL");
  const rnn_attn_desc& d = *desc;
  if (int rc = check_seq(kAttn, d.dtype, d.direction, d.layout, d.seq, d.batch, d.heads, "heads")) return rc;
  if (!std::isfinite(d.scale)) return fail(RNN_ERR_ARG, kAttn, "scale: must be finite");
  if (d.groups < 1 || d.groups > d.heads || d.heads % d.groups)
    return fail(RNN_ERR_SHAPE, kAttn, "groups: must divide heads (%lld of %lld)", (long long)d.groups, (long long)d.heads);
  if (d.key < 1) return fail(RNN_ERR_SHAPE, kAttn, "key: must be at least 1 (%lld)", (long long)d.key);
  if (d.value < 1) return fail(RNN_ERR_SHAPE, kAttn, "value: must be at least 1 (%lld)", (long long)d.value);
  if (d.key > kAttnMaxSize) return fail(RNN_ERR_UNSUPPORTED, kAttn, "key: above %d", kAttnMaxSize);
  if (d.value > kAttnMaxSize) return fail(RNN_ERR_UNSUPPORTED, kAttn, "value: above %d", kAttnMaxSize);
  rnn_attn p{};
  p.d = d;
  p.es = elem_size(d.dtype);
  p.per = int(d.heads / d.groups);
  p.key_cols = int(ceil_div(d.key, kAttnCols));
  p.value_cols = int(ceil_div(d.value, kAttnCols));
  if (bytes_of({d.seq, d.batch, d.heads, d.key, p.es}) < 0) return fail(RNN_ERR_SHAPE, kAttn, "Q: size overflows");
  if (bytes_of({d.seq, d.batch, d.heads, d.value, p.es}) < 0) return fail(RNN_ERR_SHAPE, kAttn, "V: size overflows");
  if (bytes_of({d.batch, d.heads, d.key, d.value, 4}) < 0) return fail(RNN_ERR_SHAPE, kAttn, "initial_state: size overflows");
  const int64_t heads = d.batch * d.heads, blocks = heads * std::max(p.key_cols, p.value_cols);   // (below 2^57)
  // (Step after step or a chunk, us, bf16: 8 x 16 heads of 128 x 128, 4 steps 10.9
  // and 10.0, 8 steps 16.5 and 9.9; f32, 8 x 8 of 64 x 64, 7.6 and 10.3, 11.9 and 10.3;
  // bf16, 64 x 16 of 128 x 128, where the state's bytes count and a chunk's workgroups
  // take turns, 8 steps 48.8 and 60.6, 12 steps 62.4 and 61.4.)
  p.tokens = d.seq <= (blocks < 1024 ? kAttnSteps : kAttnManySteps);
  p.f = attn_plan(d, p.tokens, heads * p.value_cols, d.seq + 64);
  p.f.sub = attn_sub(p.f, heads * p.value_cols);
  p.b = attn_plan(d, p.tokens, heads * std::min(p.key_cols, p.value_cols), d.seq + 64);
  // (the decays' gradient is summed back from a piece's end, and what the sums lose
  // grows with it: 2 x 2048 steps, 8 heads of 128 x 128, bf16, dG off by 3.3e-7 of its
  // norm with pieces of 256, 8.1e-7 of 1024, 1.3e-6 of 2048; f32, d_decay 6.2e-7,
  // 1.3e-6, 3.1e-6)
  p.bd = attn_plan(d, p.tokens, heads * std::min(p.key_cols, p.value_cols), 1024);
  // (Few walks of not too many steps go side by side in one piece, one launch for
  // four: 1 x 512 steps, 16 heads of 128 x 128, bf16, 44 us and in pieces 74; 1 x 1024
  // 75 and 82; 5 x 1024 of 8 heads 79 and 143.  f32, 1 x 512, 8 heads of 64 x 64: 51
  // and 43.)
  if (!p.tokens && heads * (2 * p.key_cols + p.value_cols) <= 256 && d.seq <= (d.dtype == RNN_DTYPE_F32 ? 256 : 1024) &&
      !std::getenv("RNN_ATTN_PIECE"))
    p.b = p.bd = {int(ceil_div(d.seq, 64) * 64), 1, 0};
  if (!attn_fits(p, p.f, p.value_cols))   // (the gradient's launches are seen to by its call)
    return fail(RNN_ERR_UNSUPPORTED, kAttn, "batch x heads: too large for one launch");
  AttnScratch at;
  if (!attn_scratch(p, false, &at, &p.forward_bytes) || !attn_scratch(p, true, &at, &p.backward_bytes))
    return fail(RNN_ERR_SHAPE, kAttn, "scratch: size overflows");
  rnn_attn* q = new (std::nothrow) rnn_attn(p);
  if (!q) return fail(RNN_ERR_ARG, kAttn, "out of host memory");
  *out = q;
  return RNN_OK;
}

extern "C" void rnn_attn_destroy(rnn_attn* attn) { delete attn; }

extern "C" int rnn_attn_scratch_size(const rnn_attn* attn, size_t* forward_bytes, size_t* backward_bytes) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!attn) return fail(RNN_ERR_ARG, kAttn, "attn: NULL");
  if (forward_bytes) *forward_bytes = attn->forward_bytes;
  if (backward_bytes) *backward_bytes = attn->backward_bytes;
  return RNN_OK;
}

extern "C" int rnn_attn_encode(const rnn_attn* attn, const rnn_attn_operands* operands, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!attn) return fail(RNN_ERR_ARG, kAttn, "attn: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kAttn, "operands: NULL");
  const rnn_attn& p = *attn;
  const rnn_attn_desc& d = p.d;
  Tensors t(kAttn);
  AttnArgs a{};
  const AttnInputs in = attn_inputs(p, *operands, t, a);
  a.a = in.Q, a.b = in.K, a.v = in.V;
  a.init = in.init;
  a.out = head_rows(t.rows(operands->Y, p.es, d.heads * d.value, d.seq * d.batch, "Y", false, true), 1);
  a.fin = reinterpret_cast<float*>(t.tensor(operands->final_state, 4, kFinal, false, true));
  t.apart({{kInitial, kFinal}});
  if (t.status != RNN_OK) return t.status;
  if (d.batch == 0 || (!a.out.p && !a.fin)) return RNN_OK;
  a.K = int(d.key), a.V = int(d.value);
  a.sk = int(d.value), a.sv = 1;
  a.in_scale = 1.f, a.out_scale = d.scale;
  a.piece = p.f.piece, a.pieces = p.f.pieces;
  a.sub = a.init && a.init == a.fin ? 0 : p.f.sub;   // (the last piece's final state may be written before another walk begins)
  if (int rc = check_scratch(kAttn, scratch, p.forward_bytes)) return rc;
  AttnScratch at;
  size_t total;
  attn_scratch(p, false, &at, &total);
  a.starts = reinterpret_cast<float*>(static_cast<char*>(scratch) + at.starts);
  a.totals = reinterpret_cast<float*>(static_cast<char*>(scratch) + at.totals);
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (int rc = attn_starts(p, a, s)) return rc;
  return attn_launch("forward", attn_walk(p, a, false, s));
}

extern "C" int rnn_attn_encode_backward(const rnn_attn* attn, const rnn_attn_operands* operands,
                                        const rnn_attn_gradients* gradients, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!attn) return fail(RNN_ERR_ARG, kAttn, "attn: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kAttn, "operands: NULL");
  if (!gradients) return fail(RNN_ERR_ARG, kAttn, "gradients: NULL");
  const rnn_attn& p = *attn;
  const rnn_attn_desc& d = p.d;
  const rnn_attn_gradients& g = *gradients;
  const int64_t rows = d.seq * d.batch, gk = d.groups * d.key, hv = d.heads * d.value;
  Tensors t(kAttn);
  AttnArgs a{};
  const AttnInputs in = attn_inputs(p, *operands, t, a);
  const HeadRows dY = head_rows(t.rows(g.dY, p.es, hv, rows, "dY", rows > 0), 1);
  const float* dfin = reinterpret_cast<const float*>(t.tensor(g.d_final_state, 4, "d_final_state", false));
  const Rows dQ = t.rows(g.dQ, p.es, gk, rows, "dQ", false, true);
  const Rows dK = t.rows(g.dK, p.es, gk, rows, "dK", false, true);
  const Rows dV = t.rows(g.dV, p.es, hv, rows, "dV", false, true);
  const Rows dG = t.rows(g.dG, 4, d.heads, rows, "dG", false, true);
  float* ddecay = reinterpret_cast<float*>(t.tensor(g.d_decay, 4, "d_decay", false, true));
  float* dinit = reinterpret_cast<float*>(t.tensor(g.d_initial_state, 4, "d_initial_state", false, true));
  t.apart();
  if (t.status != RNN_OK) return t.status;
  const bool decays = dG.p || ddecay;
  if (!dQ.p && !dK.p && !dV.p && !decays && !dinit) return RNN_OK;
  const AttnPlan& plan = decays ? p.bd : p.b;
  if (!attn_fits(p, plan, std::max(p.key_cols, p.value_cols)))
    return fail(RNN_ERR_UNSUPPORTED, kAttn, "batch x heads: too large for one launch of the gradient");
  if (int rc = check_scratch(kAttn, scratch, p.backward_bytes)) return rc;
  AttnScratch at;
  size_t total;
  attn_scratch(p, true, &at, &total);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(static_cast<char*>(scratch) + off); };
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  auto sum_decay = [&](int parts) {
    const ColSumArgs cs{f(at.decay), parts, d.heads, ddecay, nullptr, int(d.heads), 1};
    return attn_launch("sums", launch_colsum(cs, s));
  };
  if (d.batch == 0) return ddecay ? sum_decay(0) : int(RNN_OK);   // (no walk, only a sum of nothing)
  a.piece = plan.piece, a.pieces = plan.pieces;
  // forward in time from the initial state, back from the final one's gradient
  AttnArgs fore = a, back = a;
  fore.in_scale = 1.f, fore.out_scale = d.scale;
  fore.init = in.init;
  fore.b = in.K, fore.v = in.V;
  fore.starts = f(at.starts), fore.totals = f(at.totals);
  back.back = 1;
  back.in_scale = d.scale, back.out_scale = 1.f;
  back.init = dfin;
  back.b = in.Q, back.v = dY;
  back.starts = f(at.back_starts), back.totals = f(at.back_totals);
  if (dQ.p || decays)
    if (int rc = attn_starts(p, fore, s)) return rc;
  if (dK.p || dV.p || dinit || decays)
    if (int rc = attn_starts(p, back, s)) return rc;

  // dQ and dK: of each head by itself, summed over a group's heads
  AttnArgs walks[3];
  HeadSumArgs sums{};
  sums.rows = rows, sums.H = int(d.heads), sums.per = p.per, sums.K = int(d.key);
  int n = 0;
  const bool side = attn_side_by_side(p, plan);
  auto sum = [&] {
    const HeadSumArgs now = sums;
    sums.n = 0;
    return now.n ? attn_launch("sum", launch_head_sum(now, d.dtype, s)) : RNN_OK;
  };
  auto add = [&](const char* name, const AttnArgs& w) -> int {
    walks[n++] = w;
    if (side) return RNN_OK;
    if (int rc = attn_launch(name, attn_walk(p, w, false, s))) return rc;
    return sum();
  };
  auto shared = [&](const char* name, AttnArgs w, const Rows& out, const HeadRows& dot, float* dots) -> int {
    w.K = int(d.value), w.V = int(d.key);
    w.sk = 1, w.sv = int(d.value);
    w.out = head_rows(out, 1);
    w.dot = dot;
    w.dots = decays ? dots : nullptr;
    if (p.per > 1 && out.p) {
      sums.part[sums.n] = f(at.part[sums.n]);
      w.out = HeadRows{reinterpret_cast<char*>(f(at.part[sums.n])), d.heads * d.key, 1};
      w.out_f32 = 1;
      sums.out[sums.n++] = out;
    }
    return add(name, w);
  };
  const bool ends = decays && (dfin || a.pieces > 1);
  if (dQ.p || decays) {
    AttnArgs w = fore;
    w.a = dY, w.b = in.V, w.v = in.K;
    if (ends) {
      w.other = dfin;
      w.others = a.pieces > 1 ? back.starts : nullptr;
      w.ends = f(at.ends);
    }
    if (int rc = shared("dQ", w, dQ, in.Q, f(at.rows))) return rc;
  }
  if (dK.p || decays) {
    AttnArgs w = back;
    w.a = in.V, w.b = dY, w.v = in.Q;
    if (int rc = shared("dK", w, dK, in.K, f(at.cols))) return rc;
  }
  if (dV.p || dinit) {
    AttnArgs w = back;
    w.a = in.K, w.b = in.Q, w.v = dY;
    w.K = int(d.key), w.V = int(d.value);
    w.sk = int(d.value), w.sv = 1;
    w.out = head_rows(dV, 1);
    w.fin = dinit;
    if (int rc = add("dV", w)) return rc;
  }
  if (side) {
    if (int rc = attn_launch("gradient", attn_walks(p, walks, n, s))) return rc;
    if (int rc = sum()) return rc;
  }
  if (!decays) return RNN_OK;
  const AttnDecayArgs da{a.geo, a.H, p.key_cols, a.piece, a.pieces, f(at.rows), f(at.cols), ends ? f(at.ends) : nullptr, a.G, a.decay, dG,
                         ddecay ? f(at.decay) : nullptr};
  if (int rc = attn_launch("decay", launch_attn_decay(da, s))) return rc;
  return ddecay ? sum_decay(int(d.batch) * a.pieces) : int(RNN_OK);
}

// ---------------------------------------------------------------- rotary norm

namespace {

// How a launch lies over rows and heads: the lanes of a head, and the waves of a
// row, more than one where rows alone do not fill the chip.
void rotary_lay(const rnn_rotary& p, bool vec, RotaryArgs& a) {
  const rnn_rotary_desc& d = p.d;
  const int v = vec ? 16 / p.es : 1;
  a.vec = vec;
  a.units = int(d.rotary / 2 / v + ceil_div(d.size - d.rotary, 2 * v));
  a.lph = 1;
  while (a.lph < 64 && a.lph < a.units) a.lph *= 2;
  const int64_t heads = d.q_heads + d.k_heads, rounds = ceil_div(heads, 64 / a.lph);
  a.splits = int(std::min<int64_t>(rounds, ceil_div(4 * kRotaryBlocks, std::max<int64_t>(d.rows, 1))));
  a.take = int(ceil_div(rounds, a.splits) * (64 / a.lph));
  a.splits = int(ceil_div(heads, a.take));
}

// The operands both directions read.
void rotary_inputs(const rnn_rotary& p, const rnn_rotary_operands& o, bool keys, Tensors& t, RotaryArgs& a) {
  const rnn_rotary_desc& d = p.d;
  const bool any = d.rows > 0, turned = any && d.rotary > 0;
  a.x[0] = t.rows(o.Q, p.es, d.q_heads * d.size, d.rows, "Q", any);
  a.x[1] = t.rows(o.K, p.es, d.k_heads * d.size, d.rows, "K", any && keys);
  a.scale[0] = t.tensor(o.q_scale, p.es, "q_scale", false);
  a.scale[1] = t.tensor(o.k_scale, p.es, "k_scale", false);
  a.cos = reinterpret_cast<const float*>(t.tensor(o.cos, 4, "cos", turned));
  a.sin = reinterpret_cast<const float*>(t.tensor(o.sin, 4, "sin", turned));
  a.positions = reinterpret_cast<const int32_t*>(t.tensor(o.positions, 4, "positions", turned));
  a.rows = d.rows;
  a.heads[0] = int(d.q_heads), a.heads[1] = int(d.k_heads);
  a.size = int(d.size);
  a.rotary = int(d.rotary), a.half = int(d.rotary / 2);
  a.table = int(d.table);
  a.interleaved = d.interleaved;
  a.eps = d.epsilon;
}

bool rotary_vec(const rnn_rotary& p, const RotaryArgs& a) {
  const int v = 2 * 16 / p.es;
  bool ok = p.d.size % v == 0 && p.d.rotary % v == 0 && aligned(a.cos, 16) && aligned(a.sin, 16);
  for (int k = 0; k < 2; ++k)
    ok = ok && aligned(a.x[k], 16, p.es) && aligned(a.out[k], 16, p.es) && aligned(a.dy[k], 16, p.es) && aligned(a.scale[k], 16);
  return ok;
}

}  // namespace

extern "C" int rnn_rotary_create(const rnn_rotary_desc* desc, rnn_rotary** out) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (out) *out = nullptr;
  if (!desc) return fail(RNN_ERR_ARG, kRotary, "desc: NULL");
  if (!out) return fail(RNN_ERR_ARG, kRotary, "out: NULL");
  const rnn_rotary_desc& d = *desc;
  if (d.dtype < RNN_DTYPE_F32 || d.dtype > RNN_DTYPE_BF16) return fail(RNN_ERR_ARG, kRotary, "dtype: unknown value %d", d.dtype);
  if (d.interleaved != 0 && d.interleaved != 1) return fail(RNN_ERR_ARG, kRotary, "interleaved: must be 0 or 1");
  if (!(d.epsilon >= 0.f) || std::isinf(d.epsilon)) return fail(RNN_ERR_ARG, kRotary, "epsilon: must be finite and not negative");
  if (d.rows < 0) return fail(RNN_ERR_SHAPE, kRotary, "rows: negative (%lld)", (long long)d.rows);
  if (d.q_heads < 1) return fail(RNN_ERR_SHAPE, kRotary, "q_heads: must be at least 1 (%lld)", (long long)d.q_heads);
  if (d.k_heads < 0) return fail(RNN_ERR_SHAPE, kRotary, "k_heads: negative (%lld)", (long long)d.k_heads);
  if (d.size < 1) return fail(RNN_ERR_SHAPE, kRotary, "size: must be at least 1 (%lld)", (long long)d.size);
  if (d.rotary < 0 || d.rotary > d.size || d.rotary % 2)
    return fail(RNN_ERR_SHAPE, kRotary, "rotary: even, 0 to size (%lld of %lld)", (long long)d.rotary, (long long)d.size);
  if (d.table < 0) return fail(RNN_ERR_SHAPE, kRotary, "table: negative (%lld)", (long long)d.table);
  if (d.size > kRotaryMaxSize) return fail(RNN_ERR_UNSUPPORTED, kRotary, "size: above %d", kRotaryMaxSize);
  if (d.q_heads > (int64_t(1) << 20) || d.k_heads > (int64_t(1) << 20)) return fail(RNN_ERR_UNSUPPORTED, kRotary, "heads: above 2^20");
  if (d.rows > (int64_t(1) << 30)) return fail(RNN_ERR_UNSUPPORTED, kRotary, "rows: above 2^30");
  if (d.table > (int64_t(1) << 30)) return fail(RNN_ERR_UNSUPPORTED, kRotary, "table: above 2^30");
  rnn_rotary p{};
  p.d = d;
  p.es = elem_size(d.dtype);
  if (bytes_of({d.rows, std::max(d.q_heads, d.k_heads), d.size, p.es}) < 0) return fail(RNN_ERR_SHAPE, kRotary, "Q: size overflows");
  RotaryArgs a{};
  rotary_lay(p, false, a);
  p.parts = std::max<int64_t>(1, std::min<int64_t>(kRotaryBlocks, ceil_div(d.rows * a.splits, 4)));
  Regions r;
  r.take({p.parts, 2, d.size, 4});
  p.backward_bytes = r.off;
  rnn_rotary* q = new (std::nothrow) rnn_rotary(p);
  if (!q) return fail(RNN_ERR_ARG, kRotary, "out of host memory");
  *out = q;
  return RNN_OK;
}

extern "C" void rnn_rotary_destroy(rnn_rotary* rotary) { delete rotary; }

extern "C" int rnn_rotary_scratch_size(const rnn_rotary* rotary, size_t* forward_bytes, size_t* backward_bytes) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!rotary) return fail(RNN_ERR_ARG, kRotary, "rotary: NULL");
  if (forward_bytes) *forward_bytes = 0;
  if (backward_bytes) *backward_bytes = rotary->backward_bytes;
  return RNN_OK;
}

extern "C" int rnn_rotary_encode(const rnn_rotary* rotary, const rnn_rotary_operands* operands, void* scratch, void* stream) {
  (void)scratch;
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!rotary) return fail(RNN_ERR_ARG, kRotary, "rotary: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kRotary, "operands: NULL");
  const rnn_rotary& p = *rotary;
  const rnn_rotary_desc& d = p.d;
  const rnn_rotary_operands& o = *operands;
  Tensors t(kRotary);
  RotaryArgs a{};
  rotary_inputs(p, o, o.K_out.ptr != nullptr, t, a);
  a.out[0] = t.rows(o.Q_out, p.es, d.q_heads * d.size, d.rows, "Q_out", false, true);
  a.out[1] = t.rows(o.K_out, p.es, d.k_heads * d.size, d.rows, "K_out", false, true);
  t.apart({{"Q", "Q_out"}, {"K", "K_out"}});
  if (t.status != RNN_OK) return t.status;
  for (int k = 0; k < 2; ++k)
    if (a.out[k].p && a.out[k].p == a.x[k].p && a.out[k].rs != a.x[k].rs)
      return fail(RNN_ERR_ARG, kRotary, "%s: the memory of its input at another row_stride", k ? "K_out" : "Q_out");
  if (d.rows == 0 || (!a.out[0].p && !a.out[1].p)) return RNN_OK;
  for (int k = 0; k < 2; ++k)
    if (!a.out[k].p) a.x[k].p = nullptr;
  rotary_lay(p, rotary_vec(p, a), a);
  const int64_t blocks = std::min<int64_t>(ceil_div(d.rows * a.splits, 4), kRotaryBlocks);
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_rotary(a, d.dtype, blocks, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kRotary, "launch: %s", hipGetErrorString(e));
  return RNN_OK;
}

extern "C" int rnn_rotary_encode_backward(const rnn_rotary* rotary, const rnn_rotary_operands* operands,
                                          const rnn_rotary_gradients* gradients, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!rotary) return fail(RNN_ERR_ARG, kRotary, "rotary: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kRotary, "operands: NULL");
  if (!gradients) return fail(RNN_ERR_ARG, kRotary, "gradients: NULL");
  const rnn_rotary& p = *rotary;
  const rnn_rotary_desc& d = p.d;
  const rnn_rotary_gradients& g = *gradients;
  Tensors t(kRotary);
  RotaryArgs a{};
  const bool keys = d.k_heads > 0 && (g.dK.ptr || g.dk_scale.ptr);
  const bool any = d.rows > 0;
  rotary_inputs(p, *operands, keys, t, a);
  a.dy[0] = t.rows(g.dQ_out, p.es, d.q_heads * d.size, d.rows, "dQ_out", any);
  a.dy[1] = t.rows(g.dK_out, p.es, d.k_heads * d.size, d.rows, "dK_out", any && keys);
  a.out[0] = t.rows(g.dQ, p.es, d.q_heads * d.size, d.rows, "dQ", false, true);
  a.out[1] = t.rows(g.dK, p.es, d.k_heads * d.size, d.rows, "dK", false, true);
  float* dq = reinterpret_cast<float*>(t.tensor(g.dq_scale, 4, "dq_scale", false, true));
  float* dk = reinterpret_cast<float*>(t.tensor(g.dk_scale, 4, "dk_scale", false, true));
  t.apart();
  if (t.status != RNN_OK) return t.status;
  if (!a.out[0].p && !a.out[1].p && !dq && !dk) return RNN_OK;
  if (int rc = check_scratch(kRotary, scratch, dq || dk ? p.backward_bytes : 0)) return rc;
  if (!keys) a.x[1].p = nullptr;
  if (!a.out[0].p && !dq) a.x[0].p = nullptr;
  a.part = dq || dk ? static_cast<float*>(scratch) : nullptr;
  rotary_lay(p, rotary_vec(p, a), a);
  const int64_t blocks = a.part ? p.parts : std::max<int64_t>(1, std::min<int64_t>(ceil_div(d.rows * a.splits, 4), kRotaryBlocks));
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_rotary_backward(a, d.dtype, blocks, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kRotary, "launch: %s", hipGetErrorString(e));
  if (!a.part) return RNN_OK;
  const ColSumArgs cs{a.part, int(p.parts), 2 * d.size, dq, dk, int(d.size), 1};
  if (hipError_t e = launch_colsum(cs, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kRotary, "sums launch: %s", hipGetErrorString(e));
  return RNN_OK;
}
