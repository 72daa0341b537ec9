"""The state space operators on the GPU at the edges: infinite values; decays
whose product leaves f32; scratch that another stream's work may still hold."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import ssm_bounds as bounds
from tests import ssm_reference as ref
from tests.gpu_harness import note

pytestmark = pytest.mark.gpu
INF = float("inf")


def positive(b, s, c, n, groups=1, seed=0):
    """Inputs without a change of sign but A's: an infinite one makes infinite sums, and nothing that is not a number."""
    gen = torch.Generator().manual_seed(seed)
    shapes = dict(X=(b, s, c), delta=(b, s, c), A=(c, n), B=(b, s, groups * n), C=(b, s, groups * n), D=(c,), Z=(b, s, c), bias=(c,),
                  init=(b, c, n), dY=(b, s, c), dF=(b, c, n))
    v = {k: (torch.rand(*size, generator=gen, dtype=torch.float64) + 0.1).float().double() for k, size in shapes.items()}
    v["A"] = -v["A"]
    v["delta"] = (v["delta"] - 1).float().double()
    return v


def scan_both(v, groups=1, lens=None, softplus=True, gate=True, chunk=1 << 30, finite=None, backward=True):
    """Forward and backward in f32 against the 64-bit forms: infinite where those are; what is not a number there may be
    anything.  `finite`: the inputs by whose bounds finite outputs are judged (default: v)."""
    b, s, c = v["X"].shape
    n = v["A"].shape[1]
    op = rl.SelectiveScan(dtype="f32", seq=s, batch=b, channels=c, state=n, groups=groups, delta_softplus=softplus)
    t = {k: v[k].float().cuda() for k in ("X", "delta", "A", "B", "C", "D")} | {"delta_bias": v["bias"].float().cuda()}
    if gate:
        t["Z"] = v["Z"].float().cuda()
    if lens is not None:
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    t["initial_state"] = v["init"].float().cuda()
    f = {"Y": torch.empty_like(t["X"]), "final_state": torch.empty_like(t["initial_state"])}
    op.encode(t | f)
    g = {"dX": torch.empty_like(t["X"]), "ddelta": torch.empty_like(t["X"]), "dA": torch.empty_like(t["A"]), "dB": torch.empty_like(t["B"]),
         "dC": torch.empty_like(t["C"]), "dD": torch.empty_like(t["D"]), "ddelta_bias": torch.empty_like(t["D"]),
         "d_initial_state": torch.empty_like(t["initial_state"])}
    if gate:
        g["dZ"] = torch.empty_like(t["X"])
    if backward:
        op.backward(t | g | {"dY": v["dY"].float().cuda(), "d_final_state": v["dF"].float().cuda()})
    torch.cuda.synchronize()

    def args(w):
        return [w[k] for k in ("X", "delta", "A", "B", "C")], dict(D=w["D"], Z=w["Z"] if gate else None, delta_bias=w["bias"], lens=lens,
                                                                   initial_state=w["init"], groups=groups, softplus=softplus)

    # each row by itself, as long as it is: no products with steps that do not exist
    want = {}
    for i, m in enumerate(ref.lengths(lens, b, s)):
        row = {k: x if k in ("A", "D", "bias") else x[i:i + 1] if k in ("init", "dF") else x[i:i + 1, :m] for k, x in v.items()}
        main, kw = args(row)
        kw["lens"] = None
        y, h = ref.scan(*main, **kw)
        one = {"Y": y, "final_state": h} | (ref.scan_grad(*main, row["dY"], d_final=row["dF"], **kw) if backward else {})
        for k, x in one.items():
            if x.dim() == 3 and k not in ("final_state", "d_initial_state"):
                x = torch.cat([x, x.new_zeros(1, s - m, x.shape[2])], 1)
            want.setdefault(k, []).append(x)
    want = {k: sum(x) if k in ("dA", "dD", "ddelta_bias") else torch.cat(x) for k, x in want.items()}
    w = finite or v
    main, kw = args(w)
    room = bounds.scan_bounds(*main, dY=w["dY"], d_final=w["dF"], chunk=chunk, **kw)
    for name, value in want.items():
        bounds.check((f | g)[name], value, room[name], "f32", name)
    return want


@pytest.mark.parametrize("n", [1, 5, 8, 10, 16, 20, 33, 100])
@pytest.mark.parametrize("chunk", [0, 16])
@pytest.mark.parametrize("name,step", [("X", 7), ("X", 19), ("delta", 7), ("delta", 19)])
def test_scan_infinite_value(monkeypatch, n, chunk, name, step):
    """An infinite input of one channel: infinite outputs there, not NaN by states that do not exist, and nothing elsewhere."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    note(f"n {n} chunk {chunk} {name} at {step}")
    v = positive(2, 20, 6, n)
    bad = dict(v, **{name: v[name].clone()})
    bad[name][1, step, 2] = INF
    want = scan_both(bad, finite=v, chunk=chunk or 1 << 30, backward=False)
    assert want["Y"][1, step, 2] == INF


@pytest.mark.parametrize("s", [1, 2, 4])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 16, 18, 100])
def test_scan_tokens_infinite_value(s, n):
    v = positive(3, s, 6, n)
    for name in ("X", "delta"):
        bad = dict(v, **{name: v[name].clone()})
        bad[name][1, s - 1, 2] = INF
        want = scan_both(bad, finite=v, backward=False)
        assert want["Y"][1, s - 1, 2] == INF


@pytest.mark.parametrize("n", [1, 5, 8, 10, 16, 20, 33, 100])
@pytest.mark.parametrize("chunk", [0, 16])
@pytest.mark.parametrize("name,step", [("X", 7), ("delta", 7), ("dY", 7), ("dY", 31), ("Z", 3)])
def test_scan_gradient_infinite_value(monkeypatch, n, chunk, name, step):
    """The same of the gradient."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    note(f"n {n} chunk {chunk} {name} at {step}")
    v = positive(2, 32, 6, n)
    bad = dict(v, **{name: v[name].clone()})
    bad[name][1, step, 2] = INF
    want = scan_both(bad, finite=v, chunk=chunk or 1 << 30)
    assert name in ("X", "delta") or want["dX"][1, step, 2] == INF


@pytest.mark.parametrize("n,c", [(1, 6), (5, 70), (10, 64), (16, 70), (40, 6), (100, 66)])
@pytest.mark.parametrize("chunk", [0, 32])
@pytest.mark.parametrize("name", ["X", "dY", "B", "C"])
def test_scan_gradient_infinite_value_between(monkeypatch, n, c, chunk, name):
    """Infinite values with whole tiles of others before and after them, twice."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    note(f"n {n} c {c} chunk {chunk} {name}")
    v = positive(2, 96, c, n)
    bad = dict(v, **{name: v[name].clone()})
    for row, step in ((0, 24), (0, 70), (1, 40)):
        bad[name][row, step, 0] = INF
    scan_both(bad, finite=v, chunk=chunk or 1 << 30)


@pytest.mark.parametrize("n,c,groups", [(4, 6, 1), (16, 66, 1), (5, 6, 2), (64, 3, 3), (8, 64, 1)])
@pytest.mark.parametrize("name,step", [("B", 7), ("C", 7), ("B", 31), ("C", 31)])
def test_scan_infinite_weight(monkeypatch, n, c, groups, name, step):
    """An infinite B or C of one state: no NaN from the lanes that have no channel."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(1 << 20))
    note(f"n {n} c {c} {name} at {step}")
    v = positive(2, 32, c, n, groups)
    bad = dict(v, **{name: v[name].clone()})
    bad[name][1, step, 1] = INF
    want = scan_both(bad, groups, finite=v)
    assert name == "B" or want["dB"][1, step, 1] == INF


@pytest.mark.parametrize("n,c", [(1, 6), (8, 64), (16, 64), (24, 66), (64, 3), (128, 5)])
@pytest.mark.parametrize("s,lens", [(20, None), (32, [29, 1]), (40, [40, 21]), (3, None)])
@pytest.mark.parametrize("chunk", [0, 16])
def test_scan_gradient_infinite_last_step(monkeypatch, n, c, s, lens, chunk):
    """An infinite input or weight at a row's last step, inside a tile: dA, which takes the state before that step, is
    finite, whatever stands past the row's end."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    note(f"n {n} c {c} s {s} lens {lens} chunk {chunk}")
    v = positive(2, s, c, n)
    for name, at in (("X", c - 1), ("B", n - 1)):
        bad = dict(v, **{name: v[name].clone()})
        for i, m in enumerate(lens or [s, s]):
            bad[name][i, m - 1, at] = INF
        want = scan_both(bad, lens=lens, finite=v, chunk=chunk or 1 << 30)
        assert want["dA"].isfinite().all()


def growing(b, s, c, n, rate, quiet):
    """States that grow by e^rate a step, nothing happening for `quiet` steps."""
    v = positive(b, s, c, n)
    v["A"] = torch.full((c, n), float(rate), dtype=torch.float64)
    v["delta"] = torch.ones(b, s, c, dtype=torch.float64)
    v["bias"] = torch.zeros(c, dtype=torch.float64)
    v["X"][:, :quiet] = 0
    return v


@pytest.mark.parametrize("n", [3, 16, 24])
@pytest.mark.parametrize("chunk", [0, 64])
def test_scan_growing_states(monkeypatch, n, chunk):
    """Decays above 1 whose product over a chunk, e^128, passes the largest f32, on states that are zero or small."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    v = growing(2, 192, 5, n, 2.0, 170)
    for name in ("init", "dY", "dF"):
        v[name] = torch.zeros_like(v[name])
    want = scan_both(v, softplus=False, chunk=chunk or 1 << 30, backward=False)
    assert want["Y"][:, 175].abs().min() > 1
    v["delta"][:, :64], v["delta"][:, 128:] = 0, 0
    v["init"] = torch.full_like(v["init"], 1e-30).float().double()
    want = scan_both(v, softplus=False, chunk=chunk or 1 << 30, backward=False)
    assert want["final_state"].min() > 1e25


@pytest.mark.parametrize("chunk", [0, 32])
def test_scan_decay_to_nothing(monkeypatch, chunk):
    """Decays whose product over a chunk, e^-134, is below the least f32: a large state keeps what is left of it, an
    infinite one stays infinite."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    v = growing(2, 96, 5, 4, -3.0, 96)
    v["delta"][:] = 0
    v["delta"][:, 32:64] = float(torch.tensor(1.4))
    v["init"] = torch.full_like(v["init"], 1e30).float().double()
    scan_both(v, softplus=False, chunk=chunk or 1 << 30)
    bad = dict(v, init=v["init"].clone())
    bad["init"][1, 2, 1] = INF
    want = scan_both(bad, softplus=False, chunk=chunk or 1 << 30, finite=v, backward=False)
    assert want["final_state"][1, 2, 1] == INF


@pytest.mark.parametrize("n,c,groups,gate", [(3, 5, 1, True), (16, 130, 2, False), (24, 5, 1, True), (128, 3, 1, True)])
@pytest.mark.parametrize("chunk", [0, 64])
@pytest.mark.parametrize("lens", [None, [190, 129]])
def test_scan_growing_gradient(monkeypatch, n, c, groups, gate, chunk, lens):
    """The same of the gradient on its way back: of none, and of a small one to 1e22 and more."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    note(f"n {n} c {c} groups {groups} chunk {chunk} lens {lens}")
    v = growing(2, 192, c, n, 2.0, 170)
    v["B"], v["C"] = v["B"].repeat(1, 1, groups), v["C"].repeat(1, 1, groups)
    for name in ("init", "dY", "dF"):
        v[name] = torch.zeros_like(v[name])
    v["dY"][:, :20] = 1.0                   # nothing but zeros comes back to step 20, and grows from there
    v["X"][:] = 0
    more = dict(groups=groups, gate=gate, lens=lens, softplus=False, chunk=chunk or 1 << 30)
    scan_both(v, **more)
    v["delta"][:, :64], v["delta"][:, 128:] = 0, 0
    v["dY"] = torch.zeros_like(v["dY"])
    v["dF"] = torch.full_like(v["dF"], 1e-33).float().double()
    v["dY"][:, 127] = float(torch.tensor(1e-33))
    want = scan_both(v, **more)
    assert want["d_initial_state"].min() > 1e22
    v["dF"] = torch.zeros_like(v["dF"])
    want = scan_both(v, **more)
    assert want["d_initial_state"].min() > 1e20


@pytest.mark.parametrize("chunk", [0, 32])
def test_scan_steps_of_both_signs(monkeypatch, chunk):
    """A product of decays that leaves f32 downwards, by e^-120, and comes back within a chunk."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    v = growing(2, 96, 5, 4, -8.0, 96)
    for k in range(96):
        v["delta"][:, k] = 1.0 if 1 <= k % 32 <= 15 else -1.0 if 16 <= k % 32 <= 30 else 0.0
    for name in ("init", "dY", "dF"):
        v[name] = torch.zeros_like(v[name])
    v["dY"][:, 31::32] = float(torch.tensor(1e-25))
    scan_both(v, softplus=False, chunk=chunk or 1 << 30)


def test_conv_many_tokens():
    """One token of each of 16400 rows of 8200 channels: 2^24 groups of eight and more."""
    b, c, k = 16400, 8200, 3
    gen = torch.Generator("cuda").manual_seed(1)
    X, W = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16) for s in ((b, 1, c), (c, k)))
    state = torch.randn(b, k - 1, c, generator=gen, device="cuda").to(torch.bfloat16)
    Y, final = torch.empty_like(X), torch.empty_like(state)
    op = rl.CausalConv(dtype="bf16", seq=1, batch=b, channels=c, width=k, silu=False)
    op.encode({"X": X, "W": W, "initial_state": state, "Y": Y, "final_state": final})
    assert torch.equal(final[:, 0], state[:, 1]) and torch.equal(final[:, 1], X[:, 0])
    for rows in (slice(0, 100), slice(b - 100, b)):
        seen = torch.cat([state[rows], X[rows]], 1).double()
        want = (seen * W.double().t()).sum(1)
        off = (Y[rows, 0].double() - want).abs()
        room = 4 * 2.0 ** -24 * (seen * W.double().t()).abs().sum(1)     # three roundings, and that to 16 bits
        assert (off <= room + 2.0 ** -8 * (want.abs() + room)).all()


def test_norm_many_rows():
    """2^24 rows and more of a few values, forward and backward."""
    rows, size = (1 << 24) + 19, 16
    gen = torch.Generator("cuda").manual_seed(2)
    X, dY = (torch.randn(rows, size, generator=gen, device="cuda").to(torch.float16) for _ in range(2))
    scale = torch.randn(size, generator=gen, device="cuda").to(torch.float16)
    op = rl.LayerNorm(dtype="f16", rows=rows, size=size)
    t = {"X": X, "Scale": scale, "Y": torch.empty_like(X), "Mean": torch.empty(rows, device="cuda"), "InvStdDev": torch.empty(rows, device="cuda")}
    op.encode(t)
    g = {"dY": dY, "dX": torch.empty_like(X), "dB": torch.empty(size, device="cuda")}
    op.backward({k: t[k] for k in ("X", "Scale", "Mean", "InvStdDev")} | g)
    few = rl.LayerNorm(dtype="f16", rows=300, size=size)
    for at in (slice(0, 300), slice(rows - 300, rows)):        # a row does not depend on the others
        u = {"X": X[at], "Scale": scale, "Y": torch.empty_like(X[at]), "Mean": torch.empty(300, device="cuda"), "InvStdDev": torch.empty(300, device="cuda")}
        few.encode(u)
        assert all(torch.equal(u[k], t[k][at]) for k in ("Y", "Mean", "InvStdDev"))
        d = torch.empty_like(X[at])
        few.backward({k: u[k] for k in ("X", "Scale", "Mean", "InvStdDev")} | {"dY": dY[at], "dX": d})
        assert torch.equal(d, g["dX"][at])
    # 512 parts of 32768 rows, 16 of them at a time: no value goes through more than some 2200 additions
    want = dY.double().sum(0).cpu()
    assert ((g["dB"].cpu().double() - want).abs() <= 2200 * 2.0 ** -24 * dY.double().abs().sum(0).cpu()).all()


def test_scan_token_of_many_channels():
    """A token of 65536 channels by 128 states, forward and backward, by its first and last channels alone."""
    c, n = 65536, 128
    gen = torch.Generator("cuda").manual_seed(3)

    def rand(*size):
        return torch.rand(*size, generator=gen, device="cuda")

    t = {"X": rand(1, 1, c), "delta": rand(1, 1, c), "A": -rand(c, n), "B": rand(1, 1, n), "C": rand(1, 1, n), "initial_state": rand(1, c, n)}
    outs = {"Y": rand(1, 1, c), "final_state": rand(1, c, n)}
    grads = {"dX": rand(1, 1, c), "dA": rand(c, n), "d_initial_state": rand(1, c, n)}
    dY = rand(1, 1, c)
    op = rl.SelectiveScan(dtype="f32", seq=1, batch=1, channels=c, state=n)
    op.encode(t | outs)
    op.backward(t | grads | {"dY": dY})
    few = rl.SelectiveScan(dtype="f32", seq=1, batch=1, channels=64, state=n)
    for at in (slice(0, 64), slice(c - 64, c)):

        def part(name, x):
            return x[at].contiguous() if name in ("A", "dA") else x if name in ("B", "C") else x[:, at].contiguous() if name[-5:] == "state" else x[..., at].contiguous()

        u = {k: part(k, x) for k, x in t.items()}
        o = {k: torch.empty_like(part(k, x)) for k, x in outs.items()}
        g = {k: torch.empty_like(part(k, x)) for k, x in grads.items()}
        few.encode(u | o)
        few.backward(u | g | {"dY": part("dY", dY)})
        assert all(torch.equal(o[k], part(k, outs[k])) for k in o) and all(torch.equal(g[k], part(k, grads[k])) for k in g)


def test_scan_gradient_sums_in_two_launches(monkeypatch):
    """2^20 rows of B and C with 2048 weights each: 2^32 sums of dB and dC.  Rows of the batch do not depend on each other."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(1 << 20))
    b, s, g, n = 64, 16384, 16, 128
    gen = torch.Generator("cuda").manual_seed(4)

    def rand(*size):
        return torch.empty(*size, dtype=torch.bfloat16, device="cuda").uniform_(0.1, 1, generator=gen)

    t = {k: rand(b, s, g) for k in ("X", "delta")} | {k: rand(b, s, g * n) for k in ("B", "C")} | {"A": -torch.rand(g, n, generator=gen, device="cuda")}
    dY = rand(b, s, g)
    out = {k: torch.empty_like(t["B"]) for k in ("dB", "dC")} | {"dA": torch.empty_like(t["A"]), "dD": torch.empty(g, device="cuda")}
    op = rl.SelectiveScan(dtype="bf16", seq=s, batch=b, channels=g, state=n, groups=g)
    op.backward(t | out | {"dY": dY})
    half = rl.SelectiveScan(dtype="bf16", seq=s, batch=b // 2, channels=g, state=n, groups=g)
    dA, dD = torch.zeros(g, n, dtype=torch.float64, device="cuda"), torch.zeros(g, dtype=torch.float64, device="cuda")
    for at in (slice(0, b // 2), slice(b // 2, b)):
        u = {k: x if k == "A" else x[at] for k, x in t.items()}
        o = {k: torch.empty_like(u["B"]) for k in ("dB", "dC")} | {"dA": torch.empty_like(t["A"]), "dD": torch.empty(g, device="cuda")}
        half.backward(u | o | {"dY": dY[at]})
        assert torch.equal(o["dB"], out["dB"][at]) and torch.equal(o["dC"], out["dC"][at])
        dA += o["dA"]
        dD += o["dD"]
    # sums of 64 rows' sums, all of one sign: 16 additions and three more; 8 and three in each half
    for got, want in ((out["dA"], dA), (out["dD"], dD)):
        assert ((got.double() - want).abs() <= 31 * 2.0 ** -24 * want.abs()).all()


def test_first_call_captured(monkeypatch):
    """An object whose first call, the one that makes its scratch, is captured: replays among eager calls of the same and
    of another object, and eager calls once the graph is gone."""
    monkeypatch.setenv("RNN_SCAN_CHUNK", "64")
    v = positive(2, 300, 70, 16)
    t = {k: v[k].float().cuda() for k in ("X", "delta", "B", "C", "Z", "A", "D")}

    def outs():
        return {"Y": torch.zeros_like(t["X"]), "final_state": torch.zeros(2, 70, 16, device="cuda")}

    def new():
        return rl.SelectiveScan(dtype="f32", seq=300, batch=2, channels=70, state=16)

    other, want = new(), outs()
    other.encode(t | want)
    op, got, mine = new(), outs(), outs()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        op.encode(t | got)
    for turn in range(4):
        for x in got.values():
            x.fill_(7)
        graph.replay()
        other.encode(t | outs())
        op.encode(t | mine)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) and torch.equal(mine[k], want[k]) for k in want), turn
    del graph
    held = [torch.full((op.forward_bytes // 4,), 5.0, device="cuda") for _ in range(8)]
    op.encode(t | mine)
    torch.cuda.synchronize()
    assert all(torch.equal(mine[k], want[k]) for k in want) and all((h == 5).all() for h in held)


def test_scratch_while_its_memory_is_in_use():
    """The first calls of an object on one stream, while work queued on the current one still writes memory that was
    given back: the size of the scratch, many times."""
    v = positive(2, 600, 130, 16)
    t = {k: v[k].to(torch.bfloat16).cuda() for k in ("X", "delta", "B", "C", "Z")} | {k: v[k].float().cuda() for k in ("A", "D")}
    outs = {"Y": torch.empty_like(t["X"]), "final_state": torch.empty(2, 130, 16, device="cuda")}
    grads = {"dX": torch.empty_like(t["X"]), "dA": torch.empty_like(t["A"]), "dB": torch.empty_like(t["B"])}
    dY = v["dY"].to(torch.bfloat16).cuda()

    def new():
        return rl.SelectiveScan(dtype="bf16", seq=600, batch=2, channels=130, state=16)

    op = new()
    assert op.forward_bytes and op.backward_bytes
    op.encode(t | outs)
    op.backward(t | grads | {"dY": dY})
    torch.cuda.synchronize()
    want = [x.clone() for x in (*outs.values(), *grads.values())]
    busy = torch.randn(4096, 4096, device="cuda")
    other = torch.cuda.Stream()
    del op
    for _ in range(3):
        op = new()
        other.wait_stream(torch.cuda.current_stream())       # (the inputs are there)
        for x in (*outs.values(), *grads.values()):
            x.record_stream(other)
        for size in (op.forward_bytes, op.backward_bytes):
            held = torch.empty(size // 4, device="cuda")
            for _ in range(8):
                busy = busy @ busy * 0.01
                held.copy_(busy.view(-1)[:1].expand_as(held))
            del held
        op.encode(t | outs, stream=other)
        op.backward(t | grads | {"dY": dY}, stream=other)
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip((*outs.values(), *grads.values()), want))
        for x in (*outs.values(), *grads.values()):
            x.fill_(3)
        torch.cuda.synchronize()
