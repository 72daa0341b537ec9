// seq_api.cpp -- the C ABI of the state space operators (short causal
// convolution, selective scan) and of layer normalization: validation,
// scratch sizing, choice of launch shapes.  Every check runs in 64-bit checked
// arithmetic before anything is enqueued; messages name operator and argument.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>

#include "seq_check.h"

using namespace rnnhip;

struct rnn_conv {
  rnn_conv_desc d;
  int es;
  size_t backward_bytes;
  int tile, tile_b;     // steps a thread walks, forward and backward
  int64_t parts;        // partial weight gradients at most (element-wise channels: as many)
};

// How one direction of a scan lies on the chip.
struct ScanPlan {
  int nw, np;           // waves of a workgroup, states padded to their shares
  int chunk, nchunk;    // steps of a chunk of the time axis, chunks
};

struct rnn_scan {
  rnn_scan_desc d;
  int es;
  int cpg, cbg;
  bool tokens;          // forward by the kernel for a few steps
  ScanPlan f, b;
  int nseg;
  size_t forward_bytes, backward_bytes;
};

struct rnn_norm {
  rnn_norm_desc d;
  int es;
  int parts;
  size_t backward_bytes;
};

namespace {

const char kConv[] = "conv", kScan[] = "scan", kNorm[] = "layer norm";

}  // namespace

// ---------------------------------------------------------------- convolution

namespace {

// The workgroups of a launch of `v` channels a thread: `tx` threads of each
// along the channels, the others along time, `tile` steps each.
struct ConvGrid {
  int tx;
  int64_t ncb, ntb, blocks;
};
ConvGrid conv_grid_of(const rnn_conv_desc& d, int tile, int v, int tx) {
  ConvGrid g;
  g.tx = tx;
  g.ncb = ceil_div(ceil_div(d.channels, v), tx);
  g.ntb = std::max<int64_t>(ceil_div(ceil_div(d.seq, tile), 256 / tx), 1);
  g.blocks = bytes_of({d.batch, g.ncb, g.ntb});   // (-1: past any limit)
  if (g.blocks < 0) g.blocks = kMaxBytes;
  return g;
}
ConvGrid conv_grid(const rnn_conv_desc& d, int tile, int v) {
  int tx = 8;
  while (tx < 256 && tx < ceil_div(d.channels, v)) tx *= 2;
  return conv_grid_of(d, tile, v, tx);
}
ConvGrid conv_back_grid(const rnn_conv_desc& d, int tile, int v) { return conv_grid_of(d, tile, v, 64); }

int conv_launch_fits(const ConvGrid& g, ConvArgs& a) {
  if (g.blocks > kMaxThreads / 256)
    return fail(RNN_ERR_UNSUPPORTED, kConv, "seq x batch x channels: too large for one launch of tensors like these");
  a.tx = g.tx;
  a.ncb = int(g.ncb);
  a.ntb = int(g.ntb);
  return RNN_OK;
}

}  // namespace

extern "C" int rnn_conv_create(const rnn_conv_desc* desc, rnn_conv** out) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (out) *out = nullptr;
  if (!desc) return fail(RNN_ERR_ARG, kConv, "desc: NULL");
  if (!out) return fail(RNN_ERR_ARG, kConv, "out: NULL");
  const rnn_conv_desc& d = *desc;
  if (int rc = check_seq(kConv, d.dtype, d.direction, d.layout, d.seq, d.batch, d.channels)) return rc;
  if (d.silu != 0 && d.silu != 1) return fail(RNN_ERR_ARG, kConv, "silu: must be 0 or 1");
  if (d.width < 1) return fail(RNN_ERR_SHAPE, kConv, "width: must be at least 1 (%lld)", (long long)d.width);
  if (d.width < 2 || d.width > 8) return fail(RNN_ERR_UNSUPPORTED, kConv, "width: 2 to 8, got %lld", (long long)d.width);
  const int es = elem_size(d.dtype);
  if (bytes_of({d.seq, d.batch, d.channels, es}) < 0) return fail(RNN_ERR_SHAPE, kConv, "X: size overflows");
  if (bytes_of({d.batch, d.width, d.channels, es}) < 0) return fail(RNN_ERR_SHAPE, kConv, "initial_state: size overflows");
  // Steps a thread walks: long walks read the K-1 steps before them less
  // often, short ones give the chip more threads: as many steps as leave the
  // chip this many threads.  (8 x 1024 x 2048, 16 bits, the whole call.  Forward:
  // 131072 threads 16.1 us, 262144 and 524288 17.0, but with rows of unequal
  // length, as prompts have, 17.4, 16.1 and 16.1.  Backward, where a thread also
  // writes a partial sum: 65536 40.6, 131072 33.4, 262144 38.3, 524288 38.1.)
  auto tile = [&](int64_t least, int v, int64_t threads) {
    int64_t t = 64;
    while (t > least && d.batch * ceil_div(d.seq, t) * ceil_div(d.channels, v) < threads) t /= 2;
    return int(t);
  };
  const int tf = tile(8, 16 / es, 262144), tb = tile(16, 4, 131072);
  // (with the most channels a thread; the calls see to what their tensors allow)
  if (conv_grid(d, tf, d.channels % (16 / es) ? 1 : 16 / es).blocks > kMaxThreads / 256)
    return fail(RNN_ERR_UNSUPPORTED, kConv, "seq x batch x channels: too large for one launch");
  const int64_t ntb = conv_back_grid(d, tb, 1).ntb;
  Regions r;
  r.take({d.batch, ntb, d.width + 1, d.channels, 4});
  if (!r.ok) return fail(RNN_ERR_SHAPE, kConv, "scratch: size overflows");
  rnn_conv* c = new (std::nothrow) rnn_conv();
  if (!c) return fail(RNN_ERR_ARG, kConv, "out of host memory");
  c->d = d;
  c->es = es;
  c->tile = tf;
  c->tile_b = tb;
  c->parts = d.batch * ntb;
  c->backward_bytes = r.off;
  *out = c;
  return RNN_OK;
}

extern "C" void rnn_conv_destroy(rnn_conv* conv) { delete conv; }

extern "C" int rnn_conv_scratch_size(const rnn_conv* conv, size_t* forward_bytes, size_t* backward_bytes) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!conv) return fail(RNN_ERR_ARG, kConv, "conv: NULL");
  if (forward_bytes) *forward_bytes = 0;
  if (backward_bytes) *backward_bytes = conv->backward_bytes;
  return RNN_OK;
}

namespace {

// The operands both directions read.
void conv_inputs(const rnn_conv& c, const rnn_conv_operands& o, Tensors& t, ConvArgs& a) {
  const rnn_conv_desc& d = c.d;
  const int64_t rows = d.seq * d.batch;
  a.X = t.rows(o.X, c.es, d.channels, rows, "X", rows > 0);
  a.W = t.tensor(o.W, c.es, "W", true);
  a.bias = t.tensor(o.B, c.es, "B", false);
  a.geo = geometry(d.seq, d.batch, d.layout, d.direction, t.tensor(o.sequence_lens, 4, "sequence_lens", false));
  a.init = t.tensor(o.initial_state, c.es, kInitial, false);
  a.C = int(d.channels);
  a.K = int(d.width);
  a.silu = d.silu;
}

}  // namespace

extern "C" int rnn_conv_encode(const rnn_conv* conv, const rnn_conv_operands* operands, void* scratch, void* stream) {
  (void)scratch;
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!conv) return fail(RNN_ERR_ARG, kConv, "conv: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kConv, "operands: NULL");
  const rnn_conv& c = *conv;
  const rnn_conv_desc& d = c.d;
  Tensors t(kConv);
  ConvArgs a{};
  conv_inputs(c, *operands, t, a);
  a.Y = t.rows(operands->Y, c.es, d.channels, d.seq * d.batch, "Y", false, true);
  a.fin = t.tensor(operands->final_state, c.es, kFinal, false, true);
  t.apart({{kInitial, kFinal}});
  if (t.status != RNN_OK) return t.status;
  if (d.batch == 0 || (!a.Y.p && !a.fin)) return RNN_OK;
  const int v = 16 / c.es;
  const bool vec = d.channels % v == 0 && aligned(a.X, 16, c.es) && aligned(a.Y, 16, c.es) && aligned(a.W, 16) &&
                   aligned(a.bias, 16) && aligned(a.init, 16) && aligned(a.fin, 16);
  a.tile = c.tile;
  if (int rc = conv_launch_fits(conv_grid(d, a.tile, vec ? v : 1), a)) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_conv(a, d.dtype, vec ? v : 1, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kConv, "launch: %s", hipGetErrorString(e));
  return RNN_OK;
}

extern "C" int rnn_conv_encode_backward(const rnn_conv* conv, const rnn_conv_operands* operands,
                                        const rnn_conv_gradients* gradients, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!conv) return fail(RNN_ERR_ARG, kConv, "conv: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kConv, "operands: NULL");
  if (!gradients) return fail(RNN_ERR_ARG, kConv, "gradients: NULL");
  const rnn_conv& c = *conv;
  const rnn_conv_desc& d = c.d;
  const rnn_conv_gradients& g = *gradients;
  Tensors t(kConv);
  ConvArgs a{};
  const int64_t rows = d.seq * d.batch;
  conv_inputs(c, *operands, t, a);
  a.dY = t.rows(g.dY, c.es, d.channels, rows, "dY", rows > 0);
  a.dfin = t.tensor(g.d_final_state, c.es, "d_final_state", false);
  a.dX = t.rows(g.dX, c.es, d.channels, rows, "dX", false, true);
  float* dW = reinterpret_cast<float*>(t.tensor(g.dW, 4, "dW", false, true));
  float* dB = reinterpret_cast<float*>(t.tensor(g.dB, 4, "dB", false, true));
  a.dinit = t.tensor(g.d_initial_state, c.es, "d_initial_state", false, true);
  t.apart();
  if (t.status != RNN_OK) return t.status;
  if (!a.dX.p && !dW && !dB && !a.dinit) return RNN_OK;
  const size_t need = dW || dB ? c.backward_bytes : 0;
  if (int rc = check_scratch(kConv, scratch, need)) return rc;
  a.part = dW || dB ? static_cast<float*>(scratch) : nullptr;
  const size_t al = size_t(4) * c.es;   // four channels a thread
  const bool vec = d.channels % 4 == 0 && aligned(a.X, al, c.es) && aligned(a.dY, al, c.es) && aligned(a.dX, al, c.es) &&
                   aligned(a.W, al) && aligned(a.bias, al) && aligned(a.init, al) && aligned(a.dfin, al) &&
                   aligned(a.dinit, al);
  a.tile = c.tile_b;
  if (int rc = conv_launch_fits(conv_back_grid(d, a.tile, vec ? 4 : 1), a)) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_conv_backward(a, d.dtype, vec ? 4 : 1, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kConv, "launch: %s", hipGetErrorString(e));
  if (dW || dB) {
    ColSumArgs cs{a.part, int(c.parts), (d.width + 1) * d.channels, dW, dB, int(d.channels), int(d.width)};
    if (hipError_t e = launch_colsum(cs, s); e != hipSuccess)
      return fail(RNN_ERR_HIP, kConv, "sums launch: %s", hipGetErrorString(e));
  }
  return RNN_OK;
}

// ----------------------------------------------------------------------- scan

namespace {

// The split of the states and the chunks of the time axis.  `blocks`: the
// workgroups that the rows and channels give by themselves; `want`: those that
// chunks are to make of them.  A chunk has `least` steps or more, since a
// workgroup starts and joins in about the time of a tile or two of 16 steps
// (3 rows of 257 steps by 1002 channels, 24 states, forward: chunks of 64 36 us,
// of 32 48; 5 rows of 80 by 250, 10 states, backward: of 32 28 us, of 64 38),
// and there are 64 at most.
ScanPlan scan_plan(const rnn_scan_desc& d, bool backward, int64_t blocks, int64_t want) {
  const int64_t least = backward ? 32 : 64;
  ScanPlan p{};
  const int64_t n = std::min<int64_t>(std::max<int64_t>(ceil_div(want, blocks), 1), 64);
  p.chunk = int(std::max<int64_t>(ceil_div(std::max<int64_t>(ceil_div(d.seq, n), n > 1 ? least : 1), kScanTile), 1) * kScanTile);
  if (const char* e = std::getenv("RNN_SCAN_CHUNK")) {
    const int64_t c = std::atoll(e), whole = std::max<int64_t>(ceil_div(d.seq, kScanTile), 1) * kScanTile;
    if (c > 0) p.chunk = int(c >= whole ? whole : ceil_div(c, kScanTile) * kScanTile);
  }
  p.nchunk = int(std::max<int64_t>(ceil_div(d.seq, p.chunk), 1));
  scan_split(d.state, backward, &p.nw, &p.np);
  return p;
}

// Rows times channel blocks that a launch of `nw` waves a workgroup holds.
int64_t scan_most_blocks(int nchunk, int nw) { return kMaxThreads / (64 * nw) / nchunk; }

// The scratch regions of the two directions, in the order that they are taken.
struct ScanScratch {
  size_t sink, loc, sum, first, ckpt, cum, pbc, pA, pD, gloc;
};
bool scan_scratch(const rnn_scan& p, bool backward, ScanScratch* at, size_t* total) {
  const rnn_scan_desc& d = p.d;
  const ScanPlan& q = backward ? p.b : p.f;
  Regions r;
  *at = ScanScratch{};
  if (backward || !p.tokens) {
    at->sink = r.take({d.channels, 4});
    if (q.nchunk > 1) {
      at->loc = r.take({d.batch, q.nchunk, q.np, d.channels, 4});
      at->sum = r.take({d.batch, q.nchunk, d.channels, 4});
      if (!backward) at->first = r.take({d.batch, q.np, d.channels, 4});
      else at->gloc = r.take({d.batch, q.nchunk, q.np, d.channels, 4});
    }
  }
  if (backward) {
    at->ckpt = r.take({d.batch, p.nseg, q.np, d.channels, 4});
    at->cum = r.take({d.batch, p.nseg, d.channels, 4});
    at->pbc = r.take({d.groups, p.cbg, d.batch, d.seq, 2, q.np, 4});
    at->pA = r.take({d.batch, q.nchunk, q.np, d.channels, 4});
    at->pD = r.take({d.batch, q.nchunk, 2, d.channels, 4});
  }
  *total = r.off;
  return r.ok;
}

}  // namespace

extern "C" int rnn_scan_create(const rnn_scan_desc* desc, rnn_scan** out) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (out) *out = nullptr;
  if (!desc) return fail(RNN_ERR_ARG, kScan, "desc: NULL");
  if (!out) return fail(RNN_ERR_ARG, kScan, "out: NULL");
  const rnn_scan_desc& d = *desc;
  if (int rc = check_seq(kScan, d.dtype, d.direction, d.layout, d.seq, d.batch, d.channels)) return rc;
  if (d.delta_softplus != 0 && d.delta_softplus != 1) return fail(RNN_ERR_ARG, kScan, "delta_softplus: must be 0 or 1");
  if (d.state < 1) return fail(RNN_ERR_SHAPE, kScan, "state: must be at least 1 (%lld)", (long long)d.state);
  if (d.state > kScanMaxState) return fail(RNN_ERR_UNSUPPORTED, kScan, "state: above %d", kScanMaxState);
  if (d.groups < 1 || d.groups > d.channels || d.channels % d.groups)
    return fail(RNN_ERR_SHAPE, kScan, "groups: must divide channels (%lld of %lld)", (long long)d.groups, (long long)d.channels);
  rnn_scan p{};
  p.d = d;
  p.es = elem_size(d.dtype);
  p.cpg = int(d.channels / d.groups);
  p.cbg = int(ceil_div(p.cpg, 64));
  if (bytes_of({d.seq, d.batch, d.channels, p.es}) < 0) return fail(RNN_ERR_SHAPE, kScan, "X: size overflows");
  if (bytes_of({d.seq, d.batch, d.groups, d.state, p.es}) < 0) return fail(RNN_ERR_SHAPE, kScan, "B: size overflows");
  if (bytes_of({d.batch, d.channels, d.state, 4}) < 0) return fail(RNN_ERR_SHAPE, kScan, "initial_state: size overflows");
  const int64_t blocks = std::max<int64_t>(d.batch, 1) * d.groups * p.cbg;
  p.tokens = d.seq <= kScanTokens;
  // Forward, chunks cost the recurrence twice: below 160 workgroups only.  (16
  // states, 2048 channels, 1024 steps: 4 rows, 128 workgroups, in four chunks
  // 85 us, in one 113; 8 rows, 256 workgroups, in one 118.)  Backward, states
  // are computed ahead in any case.  (8 x 512 x 1024, 128 workgroups: two chunks
  // 125 us, four 133, one 215.)
  p.f = scan_plan(d, false, blocks, blocks <= 160 ? 512 : 0);
  p.b = scan_plan(d, true, blocks, 256);
  p.nseg = int(std::max<int64_t>(ceil_div(d.seq, scan_segment(p.b.np / p.b.nw)), 1));
  // (the gradient's launches are seen to by its call; its sums go in as many as
  // they need, so that what they write is the only limit)
  if (blocks > scan_most_blocks(p.f.nchunk, p.tokens ? 4 : p.f.nw))
    return fail(RNN_ERR_UNSUPPORTED, kScan, "seq x batch x channels: too large for one launch");
  if (bytes_of({d.seq, d.batch, d.groups, d.state}) >= int64_t(1) << 40)
    return fail(RNN_ERR_UNSUPPORTED, kScan, "seq x batch x groups x state: 2^40 or more");
  ScanScratch at;
  if (!scan_scratch(p, false, &at, &p.forward_bytes) || !scan_scratch(p, true, &at, &p.backward_bytes))
    return fail(RNN_ERR_SHAPE, kScan, "scratch: size overflows");
  rnn_scan* q = new (std::nothrow) rnn_scan(p);
  if (!q) return fail(RNN_ERR_ARG, kScan, "out of host memory");
  *out = q;
  return RNN_OK;
}

extern "C" void rnn_scan_destroy(rnn_scan* scan) { delete scan; }

extern "C" int rnn_scan_scratch_size(const rnn_scan* scan, size_t* forward_bytes, size_t* backward_bytes) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!scan) return fail(RNN_ERR_ARG, kScan, "scan: NULL");
  if (forward_bytes) *forward_bytes = scan->forward_bytes;
  if (backward_bytes) *backward_bytes = scan->backward_bytes;
  return RNN_OK;
}

namespace {

void scan_inputs(const rnn_scan& p, const rnn_scan_operands& o, Tensors& t, ScanArgs& a) {
  const rnn_scan_desc& d = p.d;
  const int64_t rows = d.seq * d.batch, gn = d.groups * d.state;
  const bool any = rows > 0;
  a.X = t.rows(o.X, p.es, d.channels, rows, "X", any);
  a.delta = t.rows(o.delta, p.es, d.channels, rows, "delta", any);
  a.A = reinterpret_cast<const float*>(t.tensor(o.A, 4, "A", true));
  a.Bm = t.rows(o.B, p.es, gn, rows, "B", any);
  a.Cm = t.rows(o.C, p.es, gn, rows, "C", any);
  a.D = reinterpret_cast<const float*>(t.tensor(o.D, 4, "D", false));
  a.Z = t.rows(o.Z, p.es, d.channels, rows, "Z", false);
  a.have_z = a.Z.p != nullptr;
  a.dbias = reinterpret_cast<const float*>(t.tensor(o.delta_bias, 4, "delta_bias", false));
  a.geo = geometry(d.seq, d.batch, d.layout, d.direction, t.tensor(o.sequence_lens, 4, "sequence_lens", false));
  a.init = reinterpret_cast<const float*>(t.tensor(o.initial_state, 4, kInitial, false));
  a.C = int(d.channels);
  a.N = int(d.state);
  a.G = int(d.groups);
  a.softplus = d.delta_softplus;
  a.cpg = p.cpg;
  a.cbg = p.cbg;
}

// The launch of an element type.
template <typename F>
hipError_t of_type(int dtype, F f32, F f16, F bf16, const ScanArgs& a, hipStream_t s) {
  return dtype == RNN_DTYPE_F32 ? f32(a, s) : dtype == RNN_DTYPE_F16 ? f16(a, s) : bf16(a, s);
}

// Whether every group's channels and all rows come in aligned packs of four.
bool vec_rows(const rnn_scan& p, std::initializer_list<Rows> ts) {
  const size_t n = size_t(4) * p.es;
  bool ok = p.cpg % 4 == 0;
  for (const Rows& t : ts) ok = ok && aligned(t, n, p.es);
  return ok;
}

// One direction's plan and scratch.
void scan_lay(const rnn_scan& p, bool backward, void* scratch, ScanArgs& a) {
  const ScanPlan& q = backward ? p.b : p.f;
  a.chunk = q.chunk;
  a.nchunk = q.nchunk;
  a.nw = q.nw;
  a.np = q.np;
  a.nseg = p.nseg;
  a.vec_rows = vec_rows(p, {a.X, a.delta, a.Z, a.Y, a.dY, a.dX, a.ddelta, a.dZ});
  ScanScratch at;
  size_t total;
  scan_scratch(p, backward, &at, &total);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(static_cast<char*>(scratch) + off); };
  a.sink = static_cast<char*>(scratch) + at.sink;
  a.loc = f(at.loc);
  a.sum = f(at.sum);
  a.first = f(at.first);
  a.gloc = f(at.gloc);
  a.ckpt = f(at.ckpt);
  a.cum = f(at.cum);
  a.pbc = f(at.pbc);
  a.pA = f(at.pA);
  a.pD = f(at.pD);
}

}  // namespace

extern "C" int rnn_scan_encode(const rnn_scan* scan, const rnn_scan_operands* operands, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!scan) return fail(RNN_ERR_ARG, kScan, "scan: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kScan, "operands: NULL");
  const rnn_scan& p = *scan;
  const rnn_scan_desc& d = p.d;
  Tensors t(kScan);
  ScanArgs a{};
  scan_inputs(p, *operands, t, a);
  a.Y = t.rows(operands->Y, p.es, d.channels, d.seq * d.batch, "Y", false, true);
  a.fin = reinterpret_cast<float*>(t.tensor(operands->final_state, 4, kFinal, false, true));
  t.apart({{kInitial, kFinal}});
  if (t.status != RNN_OK) return t.status;
  if (d.batch == 0 || (!a.Y.p && !a.fin)) return RNN_OK;
  if (int rc = check_scratch(kScan, scratch, p.forward_bytes)) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (p.tokens) {
    // states whole 16-byte pieces of four lanes
    const int64_t n = d.state;
    const size_t al = size_t(std::min<int64_t>(16, n));
    const size_t bc = size_t(std::min<int64_t>(n / 4, 4) * p.es);   // (a lane's piece of B and of C)
    a.vec_state = (n == 4 || n == 8 || n == 16 || n == 32 || n == 64 || n == 128) && aligned(a.A, al) && aligned(a.init, al) &&
                  aligned(a.fin, al) && aligned(a.Bm, bc, p.es) && aligned(a.Cm, bc, p.es);
    if (hipError_t e = launch_scan_tokens(a, d.dtype, s); e != hipSuccess)
      return fail(RNN_ERR_HIP, kScan, "launch: %s", hipGetErrorString(e));
    return RNN_OK;
  }
  scan_lay(p, false, scratch, a);
  if (!a.Y.p) a.Y = Rows{reinterpret_cast<char*>(a.sink), 0};   // (outputs that are not wanted)
  // more workgroups than compute units and rows of unequal length
  a.balance = a.geo.lens && a.nchunk == 1 && d.batch > 1 && d.batch <= 256 && d.batch * d.groups * p.cbg > 256;
  if (a.nchunk > 1)
    if (hipError_t e = of_type(d.dtype, launch_scan_local_f32, launch_scan_local_f16, launch_scan_local_bf16, a, s); e != hipSuccess)
      return fail(RNN_ERR_HIP, kScan, "chunk launch: %s", hipGetErrorString(e));
  if (hipError_t e = of_type(d.dtype, launch_scan_f32, launch_scan_f16, launch_scan_bf16, a, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kScan, "launch: %s", hipGetErrorString(e));
  return RNN_OK;
}

extern "C" int rnn_scan_encode_backward(const rnn_scan* scan, const rnn_scan_operands* operands,
                                        const rnn_scan_gradients* gradients, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!scan) return fail(RNN_ERR_ARG, kScan, "scan: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kScan, "operands: NULL");
  if (!gradients) return fail(RNN_ERR_ARG, kScan, "gradients: NULL");
  const rnn_scan& p = *scan;
  const rnn_scan_desc& d = p.d;
  const rnn_scan_gradients& g = *gradients;
  const int64_t rows = d.seq * d.batch, gn = d.groups * d.state;
  Tensors t(kScan);
  ScanArgs a{};
  scan_inputs(p, *operands, t, a);
  a.dY = t.rows(g.dY, p.es, d.channels, rows, "dY", rows > 0);
  a.dfin = reinterpret_cast<const float*>(t.tensor(g.d_final_state, 4, "d_final_state", false));
  a.dX = t.rows(g.dX, p.es, d.channels, rows, "dX", false, true);
  a.ddelta = t.rows(g.ddelta, p.es, d.channels, rows, "ddelta", false, true);
  a.dA = reinterpret_cast<float*>(t.tensor(g.dA, 4, "dA", false, true));
  a.dB = t.rows(g.dB, p.es, gn, rows, "dB", false, true);
  a.dC = t.rows(g.dC, p.es, gn, rows, "dC", false, true);
  a.dD = reinterpret_cast<float*>(t.tensor(g.dD, 4, "dD", false, true));
  a.dZ = t.rows(g.dZ, p.es, d.channels, rows, "dZ", false, true);
  a.ddbias = reinterpret_cast<float*>(t.tensor(g.ddelta_bias, 4, "ddelta_bias", false, true));
  a.dinit = reinterpret_cast<float*>(t.tensor(g.d_initial_state, 4, "d_initial_state", false, true));
  t.apart();
  if (t.status != RNN_OK) return t.status;
  if (a.dZ.p && !a.have_z) return fail(RNN_ERR_ARG, kScan, "dZ: there is no Z");
  if (d.batch * d.groups * p.cbg > scan_most_blocks(p.b.nchunk, p.b.nw))
    return fail(RNN_ERR_UNSUPPORTED, kScan, "seq x batch x channels: too large for one launch of the gradient");
  if (!a.dX.p && !a.ddelta.p && !a.dA && !a.dB.p && !a.dC.p && !a.dD && !a.dZ.p && !a.ddbias && !a.dinit) return RNN_OK;
  if (int rc = check_scratch(kScan, scratch, p.backward_bytes)) return rc;
  scan_lay(p, true, scratch, a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = of_type(d.dtype, launch_scan_backward_f32, launch_scan_backward_f16, launch_scan_backward_bf16, a, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kScan, "backward launch: %s", hipGetErrorString(e));
  return RNN_OK;
}

// --------------------------------------------------------- layer normalization

namespace {

// Whether a launch of `v` values a time holds all rows.  (The gradient's walks
// them with fewer workgroups, but for rows too long for registers.)
int norm_launch_fits(const rnn_norm_desc& d, int v, bool backward) {
  const NormRow r = norm_row(d.size, v, d.rows, backward);
  if ((!backward || r.shares == 0) && ceil_div(d.rows, 256 / r.threads) > kMaxThreads / 256)
    return fail(RNN_ERR_UNSUPPORTED, kNorm, "rows: too large for one launch");
  return RNN_OK;
}

}  // namespace

extern "C" int rnn_norm_create(const rnn_norm_desc* desc, rnn_norm** out) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (out) *out = nullptr;
  if (!desc) return fail(RNN_ERR_ARG, kNorm, "desc: NULL");
  if (!out) return fail(RNN_ERR_ARG, kNorm, "out: NULL");
  const rnn_norm_desc& d = *desc;
  if (d.dtype < RNN_DTYPE_F32 || d.dtype > RNN_DTYPE_BF16) return fail(RNN_ERR_ARG, kNorm, "dtype: unknown value %d", d.dtype);
  if (!(d.epsilon >= 0.f) || std::isinf(d.epsilon)) return fail(RNN_ERR_ARG, kNorm, "epsilon: must be finite and not negative");
  if (d.rows < 0) return fail(RNN_ERR_SHAPE, kNorm, "rows: negative (%lld)", (long long)d.rows);
  if (d.size < 1) return fail(RNN_ERR_SHAPE, kNorm, "size: must be at least 1 (%lld)", (long long)d.size);
  if (d.size > (int64_t(1) << 24)) return fail(RNN_ERR_UNSUPPORTED, kNorm, "size: above 16777216");
  if (d.rows > (int64_t(1) << 30)) return fail(RNN_ERR_UNSUPPORTED, kNorm, "rows: above 2^30");
  const int es = elem_size(d.dtype);
  if (bytes_of({d.rows, d.size, es}) < 0) return fail(RNN_ERR_SHAPE, kNorm, "X: size overflows");
  // (with the widest accesses; the calls see to what their tensors allow)
  if (int rc = norm_launch_fits(d, d.size % (16 / es) ? 1 : 16 / es, false)) return rc;
  rnn_norm* n = new (std::nothrow) rnn_norm();
  if (!n) return fail(RNN_ERR_ARG, kNorm, "out of host memory");
  n->d = d;
  n->es = es;
  // partial sums of dScale and dB: two workgroups a compute unit, but four
  // rows at least for each
  n->parts = int(std::max<int64_t>(1, std::min<int64_t>(512, ceil_div(d.rows, 4))));
  // rows too long for a workgroup's registers whatever their alignment: their
  // columns are summed 64 a workgroup, and 2048 of those fill the chip (1024
  // rows of 16384: 42.7 us the whole backward pass; 1024 of them 51.6, 8192
  // 45.8).  (Shorter rows go that way too, from 2049 values on, when they are
  // not whole 16-byte pieces; they keep up to 512 parts.)
  if (d.size > 8192) n->parts = int(std::max<int64_t>(1, std::min<int64_t>(n->parts, ceil_div(2048, ceil_div(d.size, 64)))));
  Regions r;
  r.take({n->parts, 2, d.size, 4});
  n->backward_bytes = r.off;
  *out = n;
  return RNN_OK;
}

extern "C" void rnn_norm_destroy(rnn_norm* norm) { delete norm; }

extern "C" int rnn_norm_scratch_size(const rnn_norm* norm, size_t* forward_bytes, size_t* backward_bytes) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!norm) return fail(RNN_ERR_ARG, kNorm, "norm: NULL");
  if (forward_bytes) *forward_bytes = 0;
  if (backward_bytes) *backward_bytes = norm->backward_bytes;
  return RNN_OK;
}

extern "C" int rnn_norm_encode(const rnn_norm* norm, const rnn_norm_operands* operands, void* scratch, void* stream) {
  (void)scratch;
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!norm) return fail(RNN_ERR_ARG, kNorm, "norm: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kNorm, "operands: NULL");
  const rnn_norm& p = *norm;
  const rnn_norm_desc& d = p.d;
  const rnn_norm_operands& o = *operands;
  Tensors t(kNorm);
  NormArgs a{};
  a.X = t.rows(o.X, p.es, d.size, d.rows, "X", d.rows > 0);
  a.scale = t.tensor(o.Scale, p.es, "Scale", true);
  a.shift = t.tensor(o.B, p.es, "B", false);
  a.Y = t.rows(o.Y, p.es, d.size, d.rows, "Y", false, true);
  a.mean = reinterpret_cast<float*>(t.tensor(o.Mean, 4, "Mean", false, true));
  a.inv = reinterpret_cast<float*>(t.tensor(o.InvStdDev, 4, "InvStdDev", false, true));
  t.apart();
  if (t.status != RNN_OK) return t.status;
  if (d.rows == 0 || (!a.Y.p && !a.mean && !a.inv)) return RNN_OK;
  a.rows = d.rows;
  a.size = int(d.size);
  a.eps = d.epsilon;
  a.vec = d.size % (16 / p.es) == 0 && aligned(a.X, 16, p.es) && aligned(a.Y, 16, p.es) && aligned(a.scale, 16) &&
          aligned(a.shift, 16);
  if (int rc = norm_launch_fits(d, a.vec ? 16 / p.es : 1, false)) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_norm(a, d.dtype, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kNorm, "launch: %s", hipGetErrorString(e));
  return RNN_OK;
}

extern "C" int rnn_norm_encode_backward(const rnn_norm* norm, const rnn_norm_operands* operands,
                                        const rnn_norm_gradients* gradients, void* scratch, void* stream) {
  set_error_of(RNN_OK, nullptr, nullptr);
  if (!norm) return fail(RNN_ERR_ARG, kNorm, "norm: NULL");
  if (!operands) return fail(RNN_ERR_ARG, kNorm, "operands: NULL");
  if (!gradients) return fail(RNN_ERR_ARG, kNorm, "gradients: NULL");
  const rnn_norm& p = *norm;
  const rnn_norm_desc& d = p.d;
  const rnn_norm_operands& o = *operands;
  const rnn_norm_gradients& g = *gradients;
  Tensors t(kNorm);
  NormArgs a{};
  const bool any = d.rows > 0;
  a.X = t.rows(o.X, p.es, d.size, d.rows, "X", any);
  a.scale = t.tensor(o.Scale, p.es, "Scale", true);
  a.mean = reinterpret_cast<float*>(t.tensor(o.Mean, 4, "Mean", any));
  a.inv = reinterpret_cast<float*>(t.tensor(o.InvStdDev, 4, "InvStdDev", any));
  a.dY = t.rows(g.dY, p.es, d.size, d.rows, "dY", any);
  a.dX = t.rows(g.dX, p.es, d.size, d.rows, "dX", false, true);
  float* dScale = reinterpret_cast<float*>(t.tensor(g.dScale, 4, "dScale", false, true));
  float* dB = reinterpret_cast<float*>(t.tensor(g.dB, 4, "dB", false, true));
  t.apart();
  if (t.status != RNN_OK) return t.status;
  if (!a.dX.p && !dScale && !dB) return RNN_OK;
  const bool sums = dScale || dB;
  if (int rc = check_scratch(kNorm, scratch, sums ? p.backward_bytes : 0)) return rc;
  a.rows = d.rows;
  a.size = int(d.size);
  a.eps = d.epsilon;
  a.parts = p.parts;
  a.part = sums ? static_cast<float*>(scratch) : nullptr;
  a.vec = d.size % (16 / p.es) == 0 && aligned(a.X, 16, p.es) && aligned(a.dY, 16, p.es) && aligned(a.dX, 16, p.es) &&
          aligned(a.scale, 16);
  if (int rc = norm_launch_fits(d, a.vec ? 16 / p.es : 1, true)) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnDevice on(s);
  if (hipError_t e = launch_norm_backward(a, d.dtype, s); e != hipSuccess)
    return fail(RNN_ERR_HIP, kNorm, "launch: %s", hipGetErrorString(e));
  if (sums) {
    ColSumArgs cs{a.part, a.parts, 2 * d.size, dScale, dB, int(d.size), 1};
    if (hipError_t e = launch_colsum(cs, s); e != hipSuccess)
      return fail(RNN_ERR_HIP, kNorm, "sums launch: %s", hipGetErrorString(e));
  }
  return RNN_OK;
}
