"""The state space operators and layer normalization on the GPU against their
64-bit plain forms, at the sizes, masks, strides and types where they can go
wrong; states carried, in place and from token to token; graphs and streams.

Tolerances count roundings (see ssm_reference.close): a convolution's sum has
width + 1 of them and its activation under a dozen; a scanned state takes one
step's (the decay's own, 6 |d A| + 8 with the step size's and A's before it) for
each step behind it; sums over n terms have n."""
import itertools

import numpy as np
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import ssm_reference as ref
from tests.gpu_harness import note

SENTINEL = -777.0
pytestmark = pytest.mark.gpu


class Bufs:
    """Device tensors for one call: inputs as given; outputs, and inputs that
    are not sequence tensors, between sentinels; sequence tensors as slices of
    wider rows where `pad` is given, the gaps holding NaN (inputs) or
    sentinels (outputs)."""

    def __init__(self, pad=0, odd=0):
        self.pad, self.odd, self.kept = pad, odd, []
        self.t = {}

    def _wide(self, shape, dtype, fill):
        n, w = int(np.prod(shape[:-1])), shape[-1] + self.pad
        flat = torch.full((n * w + 16 + self.odd,), fill, dtype=dtype, device="cuda")
        return flat, flat[8 + self.odd:8 + self.odd + n * w].view(*shape[:-1], w)[..., :shape[-1]]

    def rows(self, name, value, dtype):
        flat, view = self._wide(tuple(value.shape), dtype, float("nan"))
        view.copy_(value.to(dtype))
        self.t[name] = view

    def plain(self, name, value, dtype):
        flat = torch.full((value.numel() + 16,), float("nan") if dtype.is_floating_point else 77, dtype=dtype, device="cuda")
        view = flat[4 + self.odd:4 + self.odd + value.numel()].view(value.shape)
        view.copy_(value.to(dtype))
        self.t[name] = view

    def out(self, name, shape, dtype, row=False):
        if row:
            flat, view = self._wide(shape, dtype, SENTINEL)
        else:
            n = int(np.prod(shape))
            flat = torch.full((n + 16,), SENTINEL, dtype=dtype, device="cuda")
            view = flat[4 + self.odd:4 + self.odd + n].view(shape)
        self.kept.append((name, flat, view))
        self.t[name] = view

    def check(self):
        """Nothing but the outputs was written; every output value was."""
        torch.cuda.synchronize()
        for name, flat, view in self.kept:
            assert not (view == SENTINEL).any(), f"{name}: not written everywhere"
            view_copy = view.clone()
            view.fill_(SENTINEL)
            assert (flat == SENTINEL).all(), f"{name}: written outside"
            view.copy_(view_copy)


def lead(t, layout):
    """[batch, seq, n] <-> the layout's order of the leading dimensions."""
    return t.transpose(0, 1).contiguous() if layout == 0 else t


def rounded(t, dtype):
    return t.to(ref.TYPES[dtype]).double()


def draw(seed, **shapes):
    gen = torch.Generator().manual_seed(seed)
    return {k: torch.randn(*s, generator=gen, dtype=torch.float64) for k, s in shapes.items()}


# ------------------------------------------------------------------ convolution

def conv_case(dtype, b, s, c, k, layout=1, reverse=False, lens=None, act=True, bias=True, carried=True, pad=0, odd=0, seed=0,
              dead=0.0):
    note(f"conv {dtype} b{b} s{s} c{c} k{k} layout {layout} reverse {reverse} lens {lens} act {act} pad {pad} odd {odd}")
    dt = ref.TYPES[dtype]
    v = {n: rounded(t, dtype) for n, t in draw(seed, X=(b, s, c), W=(c, k), B=(c,), init=(b, k - 1, c), dY=(b, s, c),
                                                 dF=(b, k - 1, c)).items()}
    n = ref.lengths(lens, b, s)
    args = dict(B=v["B"] if bias else None, lens=lens, initial_state=v["init"] if carried else None, act=act, reverse=reverse)
    X, dY = v["X"].clone(), v["dY"].clone()
    for i in range(b):   # what is past a row's length is not read
        X[i, n[i]:] = dead
        dY[i, n[i]:] = dead
    op = rl.CausalConv(dtype=dtype, seq=s, batch=b, channels=c, width=k, silu=act, direction="reverse" if reverse else "forward",
                       layout=layout)

    def inputs(m):
        m.rows("X", lead(X, layout), dt)
        m.plain("W", v["W"], dt)
        if bias:
            m.plain("B", v["B"], dt)
        if carried:
            m.plain("initial_state", v["init"], dt)
        if lens is not None:
            m.plain("sequence_lens", torch.tensor(lens), torch.int32)

    shape = tuple(lead(X, layout).shape)
    m = Bufs(pad, odd)
    inputs(m)
    m.out("Y", shape, dt, row=True)
    m.out("final_state", (b, k - 1, c), dt)
    op.encode(m.t)
    m.check()
    y, h = ref.conv(v["X"], v["W"], **args)
    ym, _ = ref.conv(v["X"], v["W"], mag=True, **args)
    ref.close(lead(m.t["Y"], layout), y, ym, 2 * (k + 10), dtype, "Y")
    assert torch.equal(m.t["final_state"].cpu().double(), h), "final_state"

    g = Bufs(pad, odd)
    inputs(g)
    g.rows("dY", lead(dY, layout), dt)
    if carried:
        g.plain("d_final_state", v["dF"], dt)
    g.out("dX", shape, dt, row=True)
    g.out("dW", (c, k), torch.float32)
    g.out("dB", (c,), torch.float32)
    g.out("d_initial_state", (b, k - 1, c), dt)
    op.backward(g.t)
    g.check()
    args = dict(args, d_final=v["dF"] if carried else None)
    want, mag = ref.conv_grad(v["X"], v["W"], v["dY"], **args), ref.conv_grad(v["X"], v["W"], v["dY"], mag=True, **args)
    for name, extra, t in (("dX", 0, dtype), ("d_initial_state", 0, dtype), ("dW", b * s, "f32"), ("dB", b * s, "f32")):
        got = lead(g.t[name], layout) if name == "dX" else g.t[name]
        ref.close(got, want[name], mag[name], 3 * (k + 12) + extra, t, name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [2, 3, 4, 8])
def test_conv_widths_and_types(dtype, k):
    conv_case(dtype, 2, 37, 72, k, lens=[37, 5])


@pytest.mark.parametrize("layout,reverse,lens", [(0, False, [0, 1, 2, 50]), (1, True, [50, 3, 0, 49]), (0, True, None),
                                                 (1, False, [-4, 99, 50, 7])])
@pytest.mark.parametrize("c,pad,odd", [(64, 0, 0), (64, 8, 0), (61, 3, 1), (8, 0, 1)])
def test_conv_rows(layout, reverse, lens, c, pad, odd):
    conv_case("f16", 4, 50, c, 4, layout, reverse, lens, pad=pad, odd=odd, dead=float("nan"))


@pytest.mark.parametrize("s", [0, 1, 2, 3, 7, 8, 9, 64, 65, 200])
def test_conv_lengths(s):
    conv_case("f32", 3, s, 20, 4)
    conv_case("bf16", 2, s, 16, 8, reverse=True, carried=False, act=False, bias=False)


def test_conv_long_rows_many_tiles():
    conv_case("bf16", 2, 1200, 264, 4, lens=[1200, 700])
    conv_case("f32", 70, 33, 33, 5, layout=0)


@pytest.mark.parametrize("dtype,c", [("f16", 40), ("f32", 13)])
@pytest.mark.parametrize("reverse", [False, True])
def test_conv_pieces_and_tokens(dtype, c, reverse):
    """A prompt, then single tokens with the state updated in place, against one pass over all."""
    b, s, k, tokens = 3, 21, 4, 5
    dt = ref.TYPES[dtype]
    v = draw(5, X=(b, s + tokens, c), W=(c, k), B=(c,))
    X, W, B = (v[n].to(dt).cuda() for n in ("X", "W", "B"))

    def run(x, state):
        y = torch.empty_like(x)
        op = rl.CausalConv(dtype=dtype, seq=x.shape[1], batch=b, channels=c, width=k)
        op.encode({"X": x, "W": W, "B": B, "initial_state": state, "final_state": state, "Y": y})
        return y

    whole_state = torch.zeros(b, k - 1, c, dtype=dt, device="cuda")
    whole = run(X, whole_state)
    state = torch.zeros_like(whole_state)
    parts = [run(X[:, :s].contiguous(), state)]
    parts += [run(X[:, i:i + 1].contiguous(), state) for i in range(s, s + tokens)]
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(state, whole_state)
    assert torch.equal(state, X[:, -(k - 1):])


# ------------------------------------------------------------------------- scan

def scan_values(dtype, b, s, c, n, groups, softplus, seed=0):
    v = draw(seed, X=(b, s, c), delta=(b, s, c), A=(c, n), B=(b, s, groups * n), C=(b, s, groups * n), D=(c,), Z=(b, s, c),
             bias=(c,), init=(b, c, n), dY=(b, s, c), dF=(b, c, n))
    v["A"] = -(v["A"].abs() + 0.05)
    v["bias"] = v["bias"] * 0.5 - 1
    if not softplus:
        v["delta"], v["bias"] = v["delta"].abs() * 0.3, v["bias"].abs() * 0.1
    for k in v:
        v[k] = rounded(v[k], dtype if k in ("X", "delta", "B", "C", "Z", "dY") else "f32")
    return v


def scan_case(dtype, b, s, c, n, groups=1, gate=True, softplus=True, layout=1, reverse=False, lens=None, carried=True, skip=True,
              bias=True, pad=0, odd=0, seed=0, dead=0.0, backward=True):
    note(f"scan {dtype} b{b} s{s} c{c} n{n} groups {groups} gate {gate} softplus {softplus} layout {layout} reverse {reverse} "
         f"lens {lens} pad {pad} odd {odd}")
    dt, f32 = ref.TYPES[dtype], torch.float32
    v = scan_values(dtype, b, s, c, n, groups, softplus, seed)
    m = ref.lengths(lens, b, s)
    kw = dict(D=v["D"] if skip else None, Z=v["Z"] if gate else None, delta_bias=v["bias"] if bias else None, lens=lens,
              initial_state=v["init"] if carried else None, groups=groups, softplus=softplus, reverse=reverse)
    op = rl.SelectiveScan(dtype=dtype, seq=s, batch=b, channels=c, state=n, groups=groups, delta_softplus=softplus,
                          direction="reverse" if reverse else "forward", layout=layout)

    def cut(t):   # what is past a row's length is not read
        t = t.clone()
        for i in range(b):
            t[i, m[i]:] = dead
        return lead(t, layout)

    def inputs(bufs):
        for name in ("X", "delta", "B", "C") + (("Z",) if gate else ()):
            bufs.rows(name, cut(v[name]), dt)
        bufs.plain("A", v["A"], f32)
        if skip:
            bufs.plain("D", v["D"], f32)
        if bias:
            bufs.plain("delta_bias", v["bias"], f32)
        if carried:
            bufs.plain("initial_state", v["init"], f32)
        if lens is not None:
            bufs.plain("sequence_lens", torch.tensor(lens), torch.int32)

    row, bc = tuple(lead(v["X"], layout).shape), tuple(lead(v["B"], layout).shape)
    f = Bufs(pad, odd)
    inputs(f)
    f.out("Y", row, dt, row=True)
    f.out("final_state", (b, c, n), f32)
    op.encode(f.t)
    f.check()
    main = (v["X"], v["delta"], v["A"], v["B"], v["C"])
    y, h, kept = ref.scan(*main, **kw, keep=True)
    ym, hm = ref.scan(*main, **kw, mag=True)
    step = 8 + 6 * float((kept["d"].abs().amax((0, 1))[:, None] * v["A"].abs()).max()) if s and b else 8
    rounds = 24 + s * step + n
    ref.close(lead(f.t["Y"], layout), y, ym, rounds + 16, dtype, "Y")
    ref.close(f.t["final_state"], h, hm, rounds, "f32", "final_state")
    if not backward:
        return

    g = Bufs(pad, odd)
    inputs(g)
    g.rows("dY", cut(v["dY"]), dt)
    if carried:
        g.plain("d_final_state", v["dF"], f32)
    for name, shape in (("dX", row), ("ddelta", row), ("dB", bc), ("dC", bc)) + ((("dZ", row),) if gate else ()):
        g.out(name, shape, dt, row=True)
    for name, shape in (("dA", (c, n)), ("dD", (c,)), ("ddelta_bias", (c,)), ("d_initial_state", (b, c, n))):
        g.out(name, shape, f32)
    op.backward(g.t)
    g.check()
    kw["d_final"] = v["dF"] if carried else None
    want, mag = ref.scan_grad(*main, v["dY"], **kw), ref.scan_grad(*main, v["dY"], **kw, mag=True)
    for name, t in want.items():
        got = lead(g.t[name], layout) if g.t[name].dim() == 3 and name != "d_initial_state" else g.t[name]
        # states and their gradients meet in a product: twice a state's roundings
        terms = {"dB": c // groups, "dC": c // groups, "dA": b * s, "dD": b * s, "ddelta_bias": b * s}.get(name, 0)
        ref.close(got, t, mag[name], 2 * rounds + 40 + terms, "f32" if name in ("dA", "dD", "ddelta_bias", "d_initial_state") else dtype, name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 5, 8, 16, 24, 40, 64, 100, 128])
def test_scan_states_and_types(dtype, n):
    scan_case(dtype, 2, 21, 18, n, lens=[21, 6])


@pytest.mark.parametrize("layout,reverse,lens", [(0, False, [0, 1, 2, 50]), (1, True, [50, 3, 0, 49]), (0, True, None),
                                                 (1, False, [-4, 99, 50, 7])])
@pytest.mark.parametrize("c,groups,pad,odd", [(64, 1, 0, 0), (64, 2, 8, 0), (195, 3, 3, 1), (1, 1, 0, 1), (130, 1, 0, 0)])
def test_scan_rows(layout, reverse, lens, c, groups, pad, odd):
    scan_case("bf16", 4, 50, c, 16, groups, layout=layout, reverse=reverse, lens=lens, pad=pad, odd=odd, dead=float("nan"))


@pytest.mark.parametrize("s", [0, 1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 64, 100])
def test_scan_lengths(s):
    scan_case("f32", 3, s, 20, 16)
    scan_case("f16", 2, s, 12, 33, gate=False, carried=False, skip=False, bias=False, softplus=False, reverse=True)


@pytest.mark.parametrize("gate,softplus,skip,bias,carried", itertools.islice(itertools.product([True, False], repeat=5), 0, None, 3))
def test_scan_options(gate, softplus, skip, bias, carried):
    scan_case("f32", 2, 19, 10, 8, 2, gate=gate, softplus=softplus, skip=skip, bias=bias, carried=carried)


@pytest.mark.parametrize("n,chunk", [(2, 32), (16, 32), (16, 64), (32, 32), (64, 16), (128, 16)])
@pytest.mark.parametrize("reverse,lens", [(False, None), (True, [130, 33, 32, 1, 0, 97])])
def test_scan_chunks(monkeypatch, n, chunk, reverse, lens):
    """The time axis in chunks: joined states and gradients, ends inside and on a chunk's border."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk))
    scan_case("f32", 6, 130, 9, n, reverse=reverse, lens=lens, dead=float("inf"))


def test_scan_chunks_by_themselves():
    """Sizes whose chunks the library chooses."""
    scan_case("bf16", 1, 700, 70, 16)
    scan_case("f32", 2, 300, 33, 5, lens=[300, 129])


def scan_tensors(v, dt, lo, hi, state, **more):
    t = {n: v[n][:, lo:hi].to(dt).cuda().contiguous() for n in ("X", "delta", "B", "C", "Z")}
    t |= {"A": v["A"].float().cuda(), "D": v["D"].float().cuda(), "delta_bias": v["bias"].float().cuda()}
    return t | {"initial_state": state, "final_state": state, "Y": torch.empty_like(t["X"])} | more


@pytest.mark.parametrize("dtype,n", [("bf16", 16), ("f32", 7)])
def test_scan_pieces_and_tokens(dtype, n):
    """A prompt, then single tokens with the state updated in place: the states of one pass in one chunk, bit for bit
    (a step's operations on a state are the same in both kernels), and its outputs but for the order of a sum."""
    b, s, c, tokens = 3, 40, 70, 5
    v = scan_values(dtype, b, s + tokens, c, n, 1, True)
    dt = ref.TYPES[dtype]

    def run(lo, hi, state):
        t = scan_tensors(v, dt, lo, hi, state)
        rl.SelectiveScan(dtype=dtype, seq=hi - lo, batch=b, channels=c, state=n).encode(t)
        return t["Y"]

    whole_state = v["init"].float().cuda()
    state = whole_state.clone()
    whole = run(0, s + tokens, whole_state)
    parts = [run(0, s, state)] + [run(i, i + 1, state) for i in range(s, s + tokens)]
    assert torch.equal(state, whole_state)
    # Y sums the same n products of equal states, and the skip, each within n + 2 roundings of the terms' magnitude, and
    # is gated (six more) and rounded: two such values differ by twice that
    mag, _ = ref.scan(*(v[k] for k in ("X", "delta", "A", "B", "C", "D", "Z", "bias")), None, v["init"], mag=True)
    ref.close(torch.cat(parts, 1), whole.cpu().double(), mag, 2 * (n + 8) + 2 ** 25 * ref.EPS[dtype] * (dtype != "f32"), dtype, "Y")


@pytest.mark.parametrize("lens", [None, [200, 64, 10, 0]])
def test_scan_state_in_place_over_chunks(monkeypatch, lens):
    monkeypatch.setenv("RNN_SCAN_CHUNK", "32")
    b, s, c, n = 4, 200, 66, 16
    v = scan_values("f32", b, s, c, n, 1, True)
    op = rl.SelectiveScan(dtype="f32", seq=s, batch=b, channels=c, state=n)
    more = {} if lens is None else {"sequence_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    apart = scan_tensors(v, torch.float32, 0, s, v["init"].float().cuda(), **more)
    apart["final_state"] = torch.empty_like(apart["initial_state"])
    op.encode(apart)
    for _ in range(3):
        t = scan_tensors(v, torch.float32, 0, s, v["init"].float().cuda(), **more)
        op.encode(t)
        assert torch.equal(t["Y"], apart["Y"]) and torch.equal(t["final_state"], apart["final_state"])


def test_scan_extreme_steps():
    """Step sizes from where softplus is e^x to where it is x, decays to 0, and a NaN that stays in its own row."""
    b, s, c, n = 2, 12, 8, 4
    v = scan_values("f32", b, s, c, n, 1, True)
    v["delta"] = torch.linspace(-90, 90, s, dtype=torch.float64)[None, :, None].expand(b, s, c).float().double()
    v["bias"] = torch.zeros(c, dtype=torch.float64)
    t = scan_tensors(v, torch.float32, 0, s, v["init"].float().cuda())
    t["X"][1, 3, 2] = float("nan")
    op = rl.SelectiveScan(dtype="f32", seq=s, batch=b, channels=c, state=n)
    op.encode(t)
    main = (v["X"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["Z"], v["bias"], None, v["init"])
    y, _ = ref.scan(*main)
    ym, _ = ref.scan(*main, mag=True)
    # steps of up to 90 at |A| of a few: decays there are e^-90 and less, whose own error is nothing against
    # the step's input; where they are not, |d A| <= 20 counts (a |d A| <= 20 a, or a < 2^-28)
    ref.close(t["Y"][0], y[0], ym[0], 24 + s * 128 + n + 16, "f32", "Y")
    bad = t["Y"][1].isnan().cpu()
    assert bad[3:, 2].all() and not bad[:3].any() and bad.sum() == s - 3


@pytest.mark.parametrize("b,c,groups", [(40, 450, 1), (257, 24, 2), (256, 66, 1), (40, 448, 7)])
def test_scan_many_rows_of_unequal_length(b, c, groups):
    """More workgroups than compute units: rows in the order of their lengths (up to 256 of them), ties and empty ones
    among them."""
    lens = [(7 * i) % 23 - 1 for i in range(b)]
    scan_case("f32", b, 21, c, 3, groups, lens=lens, dead=float("nan"), backward=b == 40)


@pytest.mark.parametrize("s,lens", [(1, [0, 1, -3, 1, 7]), (2, [2, 0, 1, 1, 2]), (4, [4, 3, 0, 2, 1])])
@pytest.mark.parametrize("n,c,groups,odd,carried,reverse", [(16, 64, 1, 0, True, False), (16, 66, 2, 1, False, True),
                                                            (64, 20, 1, 0, True, True), (128, 12, 1, 0, False, False),
                                                            (3, 70, 1, 0, True, True), (100, 5, 1, 1, True, False)])
def test_scan_few_steps_of_unequal_length(s, lens, n, c, groups, odd, carried, reverse):
    """Tokens, some rows without one: whole aligned states and others."""
    for layout in (0, 1):
        scan_case("bf16", 5, s, c, n, groups, layout=layout, reverse=reverse, lens=lens, carried=carried, odd=odd,
                  dead=float("nan"), backward=layout == 0)


@pytest.mark.parametrize("k,act", [(2, True), (4, False), (5, True), (8, True)])
@pytest.mark.parametrize("lens", [None, [150, 16, 17, 0, 33]])
def test_conv_gradient_inside_tiles(k, act, lens):
    """Rows of many whole tiles, ends at and beside a tile's."""
    conv_case("f32", 5, 150, 12, k, lens=lens, act=act, dead=float("nan"))


@pytest.mark.parametrize("s", [3, 5, 17, 40])
def test_scan_infinite_last_step(s):
    """An infinite B at a row's last step makes that channel's states infinite, not NaN, wherever the step lies in a tile;
    an infinite C touches no state."""
    b, c, n = 2, 6, 4
    v = scan_values("f32", b, s, c, n, 1, True)
    lens = [s, s - 1]
    for i in range(b):
        v["B"][i, lens[i] - 1, 1] = float("inf")
        v["C"][i, lens[i] - 1, 2] = float("inf")
        v["X"][i, lens[i] - 1] = v["X"][i, lens[i] - 1].abs() + 0.1
    t = scan_tensors(v, torch.float32, 0, s, v["init"].float().cuda(), sequence_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    rl.SelectiveScan(dtype="f32", seq=s, batch=b, channels=c, state=n).encode(t)
    h = t["final_state"].cpu()
    assert (h[:, :, 1] == float("inf")).all() and h[:, :, [0, 2, 3]].isfinite().all()


# --------------------------------------------------------- layer normalization

def norm_case(dtype, rows, size, shift=True, pad=0, odd=0, seed=0, far=0.0):
    note(f"norm {dtype} rows {rows} size {size} pad {pad} odd {odd}")
    dt, f32 = ref.TYPES[dtype], torch.float32
    v = {k: rounded(t, dtype) for k, t in draw(seed, X=(rows, size), Scale=(size,), B=(size,), dY=(rows, size)).items()}
    v["X"] = rounded(v["X"] + far, dtype)
    op = rl.LayerNorm(dtype=dtype, rows=rows, size=size, epsilon=1e-5)
    m = Bufs(pad, odd)
    m.rows("X", v["X"], dt)
    m.plain("Scale", v["Scale"], dt)
    if shift:
        m.plain("B", v["B"], dt)
    m.out("Y", (rows, size), dt, row=True)
    m.out("Mean", (rows,), f32)
    m.out("InvStdDev", (rows,), f32)
    op.encode(m.t)
    m.check()
    y, mean, inv = ref.norm(v["X"], v["Scale"], v["B"] if shift else None, 1e-5)
    # sums run over at most size / 16 values in a row of additions, then a tree
    n = size // 16 + 16
    big = v["X"].abs().amax(-1)
    mag = (v["X"].abs() + big[:, None]) * inv[:, None]     # x - Mean and its error
    ref.close(m.t["Mean"], mean, big, n, "f32", "Mean")
    ref.close(m.t["InvStdDev"], inv, inv * (1 + (big * inv) ** 2 * 2 ** -24 * n), 2 * n + 8, "f32", "InvStdDev")
    most = float((mag * v["Scale"].abs()).max()) if rows else 0.0     # (InvStdDev's own error scales the value)
    ref.close(m.t["Y"], y, mag * v["Scale"].abs() * (1 + most) + v["B"].abs(), 4 * n + 16, dtype, "Y")

    mean32, inv32 = m.t["Mean"].clone(), m.t["InvStdDev"].clone()
    g = Bufs(pad, odd)
    g.rows("X", v["X"], dt)
    g.rows("dY", v["dY"], dt)
    g.plain("Scale", v["Scale"], dt)
    g.plain("Mean", mean32, f32)
    g.plain("InvStdDev", inv32, f32)
    g.out("dX", (rows, size), dt, row=True)
    g.out("dScale", (size,), f32)
    g.out("dB", (size,), f32)
    op.backward(g.t)
    g.check()
    a = (v["X"], v["Scale"], mean32.cpu().double(), inv32.cpu().double(), v["dY"])
    want, mag = ref.norm_grad(*a), ref.norm_grad(*a, mag=True)
    ref.close(g.t["dX"], want["dX"], mag["dX"], 3 * n + 16, dtype, "dX")
    ref.close(g.t["dScale"], want["dScale"], mag["dScale"], rows + 8, "f32", "dScale")
    ref.close(g.t["dB"], want["dB"], mag["dB"], rows + 8, "f32", "dB")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [1, 7, 64, 100, 128, 129, 256, 500, 512, 1000, 1024, 2048, 2056, 4096, 5001, 8192, 8200])
def test_norm_sizes(dtype, size):
    norm_case(dtype, 5, size)


@pytest.mark.parametrize("dtype,rows,size", [("bf16", 37, 16384), ("f32", 600, 9001), ("f16", 1, 70000)])
def test_norm_long_rows(dtype, rows, size):
    """Rows that a workgroup's registers do not hold."""
    norm_case(dtype, rows, size)


@pytest.mark.parametrize("dtype,rows,size", [("bf16", 4099, 2048), ("f32", 4096, 250), ("f16", 1027, 1290), ("f32", 1024, 640),
                                              ("bf16", 1025, 190)])
def test_norm_many_rows(dtype, rows, size):
    """Rows of a wave each."""
    norm_case(dtype, rows, size)


@pytest.mark.parametrize("rows", [0, 1, 3, 17, 515, 2100])
@pytest.mark.parametrize("size,pad,odd", [(64, 0, 0), (96, 32, 0), (33, 2, 1), (1032, 8, 0)])
def test_norm_rows(rows, size, pad, odd):
    norm_case("bf16", rows, size, pad=pad, odd=odd, shift=rows != 3)


def test_norm_far_from_zero():
    """Rows whose spread is small against their mean: the squares are taken of what is left of the mean."""
    norm_case("f32", 9, 1024, far=1000.0)


# ------------------------------------------------ offsets, streams, graphs, a block

def test_rows_past_32_bits():
    """Rows so far apart that their byte offsets, and element offsets, pass 32 bits."""
    far = (1 << 31) + 64
    base = torch.empty(2 * far + 4096, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(3)

    def at(c, start=0):
        return base.as_strided((1, 3, c), (3 * far, far, 1), start)

    def put(view, seed):
        x = torch.randn(*view.shape, generator=gen).to(torch.bfloat16)
        view.copy_(x)
        return x.cuda()

    c = 64
    X, Y = at(c), at(c, 512)
    near = {"X": put(X, 1), "W": torch.randn(c, 4, generator=gen).to(torch.bfloat16).cuda()}
    op = rl.CausalConv(dtype="bf16", seq=3, batch=1, channels=c, width=4)
    near["Y"] = torch.empty_like(near["X"])
    op.encode(near)
    op.encode(near | {"X": X, "Y": Y})
    assert torch.equal(Y, near["Y"])
    n = 16
    names = ("delta", "Z", "B", "C")
    wide = {k: at(c if i < 2 else n, 1024 + 256 * i) for i, k in enumerate(names)}
    near = {"X": near["X"], "A": -torch.rand(c, n, generator=gen).cuda()} | {k: put(wide[k], 2) for k in names}
    scan = rl.SelectiveScan(dtype="bf16", seq=3, batch=1, channels=c, state=n)
    near["Y"] = torch.empty_like(near["X"])
    scan.encode(near)
    scan.encode(near | wide | {"X": X, "Y": Y})
    assert torch.equal(Y, near["Y"])
    grads = {"dY": near["Y"], "dX": torch.empty_like(near["X"]), "dB": torch.empty_like(near["B"])}
    scan.backward({k: near[k] for k in near if k != "Y"} | grads)
    far_grads = {"dY": Y, "dX": at(c, 2048), "dB": at(n, 2560)}
    scan.backward({k: near[k] for k in near if k != "Y"} | wide | {"X": X} | far_grads)
    assert all(torch.equal(grads[k], far_grads[k]) for k in grads)
    norm = rl.LayerNorm(dtype="bf16", rows=3, size=c)
    scale, y = torch.ones(c, dtype=torch.bfloat16, device="cuda"), torch.empty(3, c, dtype=torch.bfloat16, device="cuda")
    norm.encode({"X": near["X"][0], "Scale": scale, "Y": y})
    norm.encode({"X": X[0], "Scale": scale, "Y": Y[0]})
    assert torch.equal(Y[0], y)


class Block:
    """Layer norm, convolution and scan one after another, as a block runs them (its products left out), and back."""

    def __init__(self, dtype, b, s, c, n, seed=0):
        self.shape, self.dtype, dt, f32 = (b, s, c, n), dtype, ref.TYPES[dtype], torch.float32
        v = scan_values(dtype, b, s, c, n, 1, True, seed)
        w = draw(seed + 1, scale=(c,), shift=(c,), W=(c, 4), cb=(c,))
        self.v = v | {k: rounded(t, dtype) for k, t in w.items()}
        g = {k: t.to(dt if k in ("X", "delta", "B", "C", "Z", "dY", "scale", "shift", "W", "cb") else f32).cuda()
             for k, t in self.v.items()}
        self.g = g

        def e(*size, to=dt):
            return torch.empty(*size, dtype=to, device="cuda")

        self.norm = rl.LayerNorm(dtype=dtype, rows=b * s, size=c)
        self.conv = rl.CausalConv(dtype=dtype, seq=s, batch=b, channels=c)
        self.scan = rl.SelectiveScan(dtype=dtype, seq=s, batch=b, channels=c, state=n)
        flat = (b * s, c)
        self.tn = {"X": g["X"].view(flat), "Scale": g["scale"], "B": g["shift"], "Y": e(flat), "Mean": e(b * s, to=f32),
                   "InvStdDev": e(b * s, to=f32)}
        self.tc = {"X": self.tn["Y"].view(b, s, c), "W": g["W"], "B": g["cb"], "Y": e(b, s, c), "final_state": e(b, 3, c)}
        self.ts = {"X": self.tc["Y"], "delta": g["delta"], "A": g["A"], "B": g["B"], "C": g["C"], "D": g["D"], "Z": g["Z"],
                   "delta_bias": g["bias"], "Y": e(b, s, c), "final_state": e(b, c, n, to=f32)}
        self.gs = {"dY": g["dY"], "dX": e(b, s, c), "ddelta": e(b, s, c), "dA": e(c, n, to=f32), "dB": e(b, s, n), "dC": e(b, s, n),
                   "dD": e(c, to=f32), "dZ": e(b, s, c), "ddelta_bias": e(c, to=f32)}
        self.gc = {"dY": self.gs["dX"], "dX": e(b, s, c), "dW": e(c, 4, to=f32), "dB": e(c, to=f32)}
        self.gn = {"dY": self.gc["dX"].view(flat), "dX": e(flat), "dScale": e(c, to=f32), "dB": e(c, to=f32)}

    def step(self):
        self.norm.encode(self.tn)
        self.conv.encode(self.tc)
        self.scan.encode(self.ts)
        self.scan.backward(self.ts | self.gs)
        self.conv.backward(self.tc | self.gc)
        self.norm.backward({k: t for k, t in self.tn.items() if k not in ("B", "Y")} | self.gn)

    def outputs(self):
        outs = [self.tn["Y"], self.tc["Y"], self.ts["Y"], self.tc["final_state"], self.ts["final_state"]]
        return outs + [t for k, t in (*self.gs.items(), *self.gc.items(), *self.gn.items()) if k != "dY"]


def test_block_gradients():
    """The block's whole step in f32 against automatic derivatives of the 64-bit forms."""
    b, s, c, n = 2, 30, 24, 8
    blk = Block("f32", b, s, c, n)
    blk.step()
    torch.cuda.synchronize()
    leaves = {k: blk.v[k].clone().requires_grad_() for k in ("X", "scale", "shift", "W", "cb", "delta", "A", "B", "C", "D", "Z", "bias")}
    x = ref.norm(leaves["X"].reshape(b * s, c), leaves["scale"], leaves["shift"])[0].view(b, s, c)
    x, _ = ref.conv(x, leaves["W"], leaves["cb"])
    y, _ = ref.scan(x, *(leaves[k] for k in ("delta", "A", "B", "C", "D", "Z", "bias")))
    want = dict(zip(leaves, torch.autograd.grad((y * blk.v["dY"]).sum(), list(leaves.values()))))
    got = {"X": blk.gn["dX"].view(b, s, c), "scale": blk.gn["dScale"], "shift": blk.gn["dB"], "W": blk.gc["dW"], "cb": blk.gc["dB"],
           "delta": blk.gs["ddelta"], "A": blk.gs["dA"], "B": blk.gs["dB"], "C": blk.gs["dC"], "D": blk.gs["dD"],
           "Z": blk.gs["dZ"], "bias": blk.gs["ddelta_bias"]}
    assert float((blk.ts["Y"].cpu().double() - y).norm() / y.norm()) < 1e-5
    for k, t in want.items():
        # f32 through some 30 steps and three operators: of the order of 100 roundings of 2^-24 in norm
        assert float((got[k].cpu().double() - t).norm() / t.norm()) < 1e-5, k


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 70, 64, 16)), ("f16", (1, 300, 40, 5))])
def test_block_runs_are_identical_and_captured(dtype, shape):
    """Two runs have the same bits; a captured step replays on new inputs, eager steps and another graph between."""
    first, other = Block(dtype, *shape, seed=1), Block(dtype, *shape, seed=2)
    first.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in first.outputs()]
    first.step()
    assert all(torch.equal(a, b) for a, b in zip(want, first.outputs()))
    other.step()
    torch.cuda.synchronize()
    want2 = [t.clone() for t in other.outputs()]
    stream = torch.cuda.Stream()
    graphs = []
    for blk in (first, other):
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            blk.step()
        graphs.append(graph)
    third = Block(dtype, *shape, seed=3)
    for turn in range(4):
        for blk, graph, w in ((first, graphs[0], want), (other, graphs[1], want2)):
            for t in blk.outputs():
                t.fill_(5)
            graph.replay()
            third.step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(w, blk.outputs())), turn
    # new values in the same tensors
    for k in ("X", "delta", "B", "C", "Z", "dY"):
        first.g[k].copy_(third.g[k])
    graphs[0].replay()
    kept = [t.clone() for t in first.outputs()]
    first.step()
    assert all(torch.equal(a, b) for a, b in zip(kept, first.outputs()))


def test_two_streams_at_once():
    """Objects of their own on two streams at once give what they give alone."""
    blocks = [Block("bf16", 2, 300, 128, 16, seed=s) for s in (4, 5)]
    for b in blocks:
        b.step()
    torch.cuda.synchronize()
    want = [[t.clone() for t in b.outputs()] for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for b, st in zip(blocks, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                b.step()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert all(torch.equal(x, y) for x, y in zip(w, b.outputs()))


def test_only_what_is_asked_for():
    """Outputs left out are not computed into others: each alone equals itself among all."""
    blk = Block("f32", 2, 20, 12, 8)
    blk.step()
    torch.cuda.synchronize()
    for op, tensors, grads in ((blk.scan, blk.ts, blk.gs), (blk.conv, blk.tc, blk.gc),
                               (blk.norm, {k: t for k, t in blk.tn.items() if k not in ("B", "Y")}, blk.gn)):
        for name in grads:
            if name == "dY":
                continue
            alone = torch.empty_like(grads[name])
            op.backward(tensors | {"dY": grads["dY"], name: alone})
            assert torch.equal(alone, grads[name]), name
    for name in ("Y", "final_state"):
        for op, t in ((blk.scan, blk.ts), (blk.conv, blk.tc)):
            alone = torch.empty_like(t[name])
            op.encode({k: x for k, x in t.items() if k not in ("Y", "final_state")} | {name: alone})
            assert torch.equal(alone, t[name]), name


def test_no_rows_give_zero_weight_gradients():
    conv = rl.CausalConv(dtype="f32", seq=0, batch=0, channels=6, width=4)
    e = torch.empty(0, 0, 6, device="cuda")
    t = {"X": e, "W": torch.ones(6, 4, device="cuda"), "dY": e, "dW": torch.ones(6, 4, device="cuda"), "dB": torch.ones(6, device="cuda")}
    conv.backward(t)
    scan = rl.SelectiveScan(dtype="f32", seq=5, batch=0, channels=6, state=4)
    r, bc = torch.empty(0, 5, 6, device="cuda"), torch.empty(0, 5, 4, device="cuda")
    u = {"X": r, "delta": r, "B": bc, "C": bc, "A": torch.ones(6, 4, device="cuda"), "dY": r, "dA": torch.ones(6, 4, device="cuda"),
         "dD": torch.ones(6, device="cuda"), "ddelta_bias": torch.ones(6, device="cuda")}
    scan.backward(u)
    norm = rl.LayerNorm(dtype="f32", rows=0, size=6)
    z = torch.empty(0, 6, device="cuda")
    m = torch.empty(0, device="cuda")
    w = {"X": z, "Scale": torch.ones(6, device="cuda"), "Mean": m, "InvStdDev": m, "dY": z, "dScale": torch.ones(6, device="cuda"),
         "dB": torch.ones(6, device="cuda")}
    norm.backward(w)
    for t in (t["dW"], t["dB"], u["dA"], u["dD"], u["ddelta_bias"], w["dScale"], w["dB"]):
        assert not t.any()
