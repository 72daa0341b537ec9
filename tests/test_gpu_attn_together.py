"""Norms with rotations, linear attention and their gradients as a model uses
them: prompts of their own lengths, then a token at a time with the state
carried on, forward and back, captured; against the 64-bit plain form of the
whole.  And the calls that neither operator's own tests make: two at once, rows
farther apart than 32 bits reach, many rows, state in place over several pieces.

Bounds: the attention's inputs are off by what the rotation's bound allows and
by half a step of their type, each relative to the sum of their own terms'
magnitudes; an output is linear in each of them, so it moves by no more than
the same plain form of magnitudes and bounds gives."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import attn_reference as att
from tests import ssm_reference as ref
from tests import test_gpu_rotary as rot
from tests.gpu_harness import note
from tests.test_gpu_attn import SPLIT, attn_case, reference, types, values

B, S, H, GROUPS, K, V, TABLE, SCALE = 3, 90, 4, 2, 32, 24, 300, 0.3
LENS, STARTS = [90, 17, 64], [0, 100, 5]
AT = rot.pairs(K, K, False)


def model(dtype, seed=0):
    t = values(dtype, B, S, H, GROUPS, K, V, seed)
    gen = torch.Generator().manual_seed(seed + 50)
    for n in ("q_scale", "k_scale"):
        t[n] = rl_round(1 + 0.2 * torch.randn(K, generator=gen, dtype=torch.float64), dtype)
    t["cos"], t["sin"] = (x.double() for x in rot.table(TABLE, K))
    return t


def rl_round(x, dtype):
    return x.to(ref.TYPES[dtype]).double()


def positions(first, n, lens=None):
    """Of rows [batch, n]; past a row's length none."""
    p = torch.tensor(first)[:, None] + torch.arange(n)[None]
    if lens is not None:
        p = torch.where(torch.arange(n)[None] < torch.tensor(lens)[:, None], p, torch.tensor(-1))
    return p.to(torch.int32)


def turned(t, pos, which):
    """(value, bound) of a row's normed and turned heads, [batch, seq, groups * key]."""
    b, s = pos.shape
    x, live = t[which].reshape(b * s, GROUPS, K), (pos >= 0).flatten()
    at = pos.flatten().clamp(min=0).long()
    y, Y = rot.reference(x, t[which.lower() + "_scale"], t["cos"][at], t["sin"][at], live, AT, 1e-6)
    return y.reshape(b, s, -1), Y.reshape(b, s, -1)


def plain(t, pos, lens, dtype, back):
    """The whole in 64 bits: {name: (value, bound)}."""
    (q, Dq), (k, Dk) = turned(t, pos, "Q"), turned(t, pos, "K")
    eps = 0.0 if dtype == "f32" else ref.EPS[dtype]
    Dq, Dk = (1.01 * D + eps * (x.abs() + D) for D, x in ((Dq, q), (Dk, k)))
    b, s = pos.shape
    rest = dict(G=t["G"], decay=t["decay"], scale=SCALE, lens=lens, init=t["initial_state"])
    if back:
        rest.update(dY=t["dY"], d_final=t["d_final_state"])
    want = att.attn(q, k, t["V"], H, GROUPS, split=SPLIT[dtype], **rest)
    # magnitudes: how far the inputs' own errors take an output, to first and second order
    size = {n: abs(x) if n in ("init", "dY", "d_final") else x for n, x in rest.items()}
    base = att.attn(q.abs(), k.abs(), t["V"].abs(), H, GROUPS, **size)
    most = att.attn(q.abs() + Dq, k.abs() + Dk, t["V"].abs(), H, GROUPS, **size)
    return want, {n: most[n][0] - base[n][0] for n in want}, (q, k)


class Net:
    def __init__(self, dtype, s):
        self.s, self.dtype = s, dtype
        self.norm = rl.RotaryNorm(dtype=dtype, rows=B * s, q_heads=GROUPS, k_heads=GROUPS, size=K, table=TABLE)
        self.attn = rl.LinearAttention(dtype=dtype, seq=s, batch=B, heads=H, groups=GROUPS, key=K, value=V, scale=SCALE)

    def buffers(self, back=False):
        to, f32, s = types(self.dtype), torch.float32, self.s
        e = lambda *w, dt=to["Y"]: torch.full(w, float("nan"), dtype=dt, device="cuda")  # noqa: E731
        m = {"q": e(B, s, GROUPS * K), "k": e(B, s, GROUPS * K), "Y": e(B, s, H * V), "final_state": e(B, H, K, V, dt=f32)}
        if back:
            m.update(dq=e(B, s, GROUPS * K), dk=e(B, s, GROUPS * K), dV=e(B, s, H * V), dG=e(B, s, H, dt=f32), d_decay=e(H, dt=f32),
                     d_initial_state=e(B, H, K, V, dt=f32), dQ=e(B, s, GROUPS * K), dK=e(B, s, GROUPS * K), dq_scale=e(K, dt=f32),
                     dk_scale=e(K, dt=f32))
        return m

    def rows(self, t):
        return t.view(B * self.s, -1)

    def forward(self, d, m):
        shared = {n: d[n] for n in ("q_scale", "k_scale", "cos", "sin")}
        self.norm.encode({**shared, "positions": d["positions"].view(-1), "Q": self.rows(d["Q"]), "K": self.rows(d["K"]),
                          "Q_out": self.rows(m["q"]), "K_out": self.rows(m["k"])})
        self.attn.encode({**self.inputs(d, m), "Y": m["Y"], "final_state": m["final_state"]})

    def inputs(self, d, m):
        return {"Q": m["q"], "K": m["k"], **{n: d[n] for n in ("V", "G", "decay", "initial_state", "sequence_lens") if n in d}}

    def backward(self, d, m):
        self.attn.backward({**self.inputs(d, m), "dY": d["dY"], "d_final_state": d["d_final_state"], "dQ": m["dq"], "dK": m["dk"],
                            **{n: m[n] for n in ("dV", "dG", "d_decay", "d_initial_state")}})
        shared = {n: d[n] for n in ("q_scale", "k_scale", "cos", "sin")}
        self.norm.backward({**shared, "positions": d["positions"].view(-1), "Q": self.rows(d["Q"]), "K": self.rows(d["K"]),
                            "dQ_out": self.rows(m["dq"]), "dK_out": self.rows(m["dk"]), "dQ": self.rows(m["dQ"]), "dK": self.rows(m["dK"]),
                            "dq_scale": m["dq_scale"], "dk_scale": m["dk_scale"]})


def device(t, dtype, pos, lens=None):
    to = types(dtype)
    f32 = ("cos", "sin")
    d = {n: x.to(torch.float32 if n in f32 else to.get(n, ref.TYPES[dtype])).cuda() for n, x in t.items()}
    d["positions"] = pos.cuda()
    if lens is not None:
        d["sequence_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return d


def wider(pair, more, extra=1.0):
    return pair[0], pair[1] + extra * more


def test_the_whole_in_64_bits():
    """The plain form's gradients are autograd's and those of differences."""
    t, pos = model("f32"), positions(STARTS, S, LENS)
    names = ("Q", "K", "V", "G", "decay", "initial_state", "q_scale", "k_scale")
    leaves = {n: t[n].clone().requires_grad_() for n in names}

    def loss(x):
        u = {**t, **x}
        (q, _), (k, _) = turned(u, pos, "Q"), turned(u, pos, "K")
        y = att.attn(q, k, u["V"], H, GROUPS, u["G"], u["decay"], SCALE, LENS, u["initial_state"])
        return (y["Y"][0] * t["dY"]).sum() + (y["final_state"][0] * t["d_final_state"]).sum()

    loss(leaves).backward()
    want, _, _ = plain(t, pos, LENS, "f32", True)
    live = pos.flatten() >= 0
    at = pos.flatten().clamp(min=0).long()
    got = {n: want["d" + n][0] for n in ("V", "G")} | {n: want["d_" + n][0] for n in ("decay", "initial_state")}
    for n in "QK":
        (dx, _), (ds, _) = rot.reference(t[n].view(B * S, GROUPS, K), t[n.lower() + "_scale"], t["cos"][at], t["sin"][at], live, AT, 1e-6,
                                         dy=want["d" + n][0].reshape(B * S, GROUPS, K))
        got[n], got[n.lower() + "_scale"] = dx.reshape(B, S, -1), ds
    gen = torch.Generator().manual_seed(3)
    for n, x in leaves.items():
        torch.testing.assert_close(got[n], x.grad, rtol=1e-8, atol=1e-9 * float(x.grad.abs().max()), msg=n)
        way = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        step = 1e-6
        with torch.no_grad():
            slope = (loss({**leaves, n: x + step * way}) - loss({**leaves, n: x - step * way})) / (2 * step)
            want_slope = (got[n] * way).sum()
            # (a difference of 1e-6 leaves 1e-12 of the third derivative, and 1e-16 / 1e-6 of the loss)
            assert abs(slope - want_slope) <= 1e-6 * (got[n] * way).abs().sum() + 1e-8, n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
def test_prompts_then_tokens_and_back(dtype):
    note(f"together {dtype}")
    t, pos = model(dtype), positions(STARTS, S, LENS)
    d = device(t, dtype, pos, LENS)
    net, m = Net(dtype, S), None
    m = net.buffers(back=True)
    net.forward(d, m)
    net.backward(d, m)
    torch.cuda.synchronize()
    want, more, _ = plain(t, pos, LENS, dtype, True)
    fore, more_fore, _ = plain(t, pos, LENS, dtype, False)
    att.close(m["Y"], *wider(fore["Y"], more_fore["Y"]), dtype, "Y")
    att.close(m["final_state"], *wider(fore["final_state"], more_fore["final_state"]), "f32", "final_state")
    for n in ("dV", "d_initial_state"):
        att.close(m[n], *wider(want[n], more[n]), dtype if n == "dV" else "f32", n)
    # what the norm's gradient makes of the attention's, its bound and a half step of its type
    live, at = pos.flatten() >= 0, pos.flatten().clamp(min=0).long()
    eps = 0.0 if dtype == "f32" else ref.EPS[dtype]
    for n in "QK":
        dq, Dq = wider(want["d" + n], more["d" + n])
        Dq = 1.06 * Dq + eps * (dq.abs() + 1.06 * Dq)
        args = (t[n].view(B * S, GROUPS, K), t[n.lower() + "_scale"], t["cos"][at], t["sin"][at], live, AT, 1e-6)
        (dx, Dx), (ds, Ds) = rot.reference(*args, dy=dq.reshape(B * S, GROUPS, K))
        (_, Mx), (_, Ms) = rot.reference(*args, dy=Dq.reshape(B * S, GROUPS, K))
        Mx, Ms = Mx / rot.DEPTH, Ms / (rot.DEPTH + B * S * GROUPS * rot.U)
        att.close(m["d" + n], dx.reshape(B, S, -1), (Dx + Mx).reshape(B, S, -1), dtype, "d" + n)
        att.close(m[f"d{n.lower()}_scale"], ds, Ds + Ms, "f32", f"d{n.lower()}_scale")
    # tokens, the state carried on in place: as one longer prompt of each row
    one, state = Net(dtype, 1), m["final_state"].clone()
    later = model(dtype, seed=7)
    steps = 5
    outs, first = [], [a + n for a, n in zip(STARTS, LENS)]
    for i in range(steps):
        ti = {n: x[:, i:i + 1] if n in ("Q", "K", "V", "G") else x for n, x in later.items()}
        ti = {n: x for n, x in ti.items() if n not in ("dY", "d_final_state")}
        di = device(ti, dtype, positions([p + i for p in first], 1))
        di = {n: x.contiguous() for n, x in di.items()}
        di.update(initial_state=state, decay=d["decay"], q_scale=d["q_scale"], k_scale=d["k_scale"])
        mi = one.buffers()
        mi["final_state"] = state
        one.forward(di, mi)
        outs.append(mi["Y"])
    torch.cuda.synchronize()
    long = dict(t)
    for n in ("Q", "K", "V", "G"):
        x = torch.zeros(B, S + steps, t[n].shape[-1], dtype=torch.float64)
        for r, live_r in enumerate(LENS):
            x[r, :live_r] = t[n][r, :live_r]
            x[r, live_r:live_r + steps] = later[n][r, :steps]
        long[n] = x
    total = [n + steps for n in LENS]
    fore, more, _ = plain(long, positions(STARTS, S + steps, total), total, dtype, False)
    value, bound = wider(fore["Y"], more["Y"])
    pick = lambda x: torch.stack([x[r, n:n + steps] for r, n in enumerate(LENS)])  # noqa: E731
    att.close(torch.cat(outs, 1), pick(value), pick(bound), dtype, "tokens")
    att.close(state, *wider(fore["final_state"], more["final_state"]), "f32", "state")


@pytest.mark.gpu
def test_captured_and_two_at_once():
    """A captured step of both operators and their gradients, replayed between eager calls; and two nets on two streams."""
    dtype, pos = "bf16", positions(STARTS, S, LENS)
    net, eager = Net(dtype, S), Net(dtype, S)
    held, m = device(model(dtype), dtype, pos, LENS), net.buffers(back=True)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        net.forward(held, m)
        net.backward(held, m)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            net.forward(held, m)
            net.backward(held, m)
    for seed in range(1, 4):
        d = device(model(dtype, seed), dtype, pos, LENS)
        for n in held:
            held[n].copy_(d[n])
        graph.replay()
        want = eager.buffers(back=True)
        eager.forward(d, want)
        eager.backward(d, want)
        torch.cuda.synchronize()
        for n in m:
            assert torch.equal(m[n], want[n]), (seed, n)
    sides = [(Net(dtype, S), torch.cuda.Stream(), device(model(dtype, 20 + i), dtype, pos, LENS)) for i in range(2)]
    alone = []
    for one, _, d in sides:
        x = one.buffers(back=True)
        one.forward(d, x)
        one.backward(d, x)
        torch.cuda.synchronize()
        alone.append(x)
    for _ in range(5):
        both = [one.buffers(back=True) for one, _, _ in sides]
        torch.cuda.synchronize()
        for (one, side, d), x in zip(sides, both):
            with torch.cuda.stream(side):
                one.forward(d, x)
                one.backward(d, x)
        torch.cuda.synchronize()
        for x, y in zip(both, alone):
            for n in x:
                assert torch.equal(x[n], y[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("s,reverse", [(200, False), (700, True), (1500, False)])
def test_state_in_place_over_pieces(dtype, s, reverse):
    """The final state over the initial one, where pieces of the time axis each begin from it."""
    b, h, k, v = 1, 2, 64, 40
    t = values(dtype, b, s, h, h, k, v, gate=0.01, fixed=0.001)
    to = types(dtype)
    d = {n: x.to(to[n]).cuda() for n, x in t.items()}
    op = rl.LinearAttention(dtype=dtype, seq=s, batch=b, heads=h, key=k, value=v, direction="reverse" if reverse else "forward")
    state, y = d["initial_state"].clone(), torch.empty(b, s, h * v, dtype=to["Y"], device="cuda")
    op.encode({**{n: d[n] for n in ("Q", "K", "V", "G", "decay")}, "initial_state": state, "final_state": state, "Y": y})
    torch.cuda.synchronize()
    want = reference(t, dtype, h, h, 1.0, None, reverse, False, "cuda")
    att.close(y, *want["Y"], dtype, "Y")
    att.close(state, *want["final_state"], "f32", "final_state")


@pytest.mark.gpu
@pytest.mark.parametrize("s,stride", [(200, 2 ** 24), (70, 2 ** 26), (3, 2 ** 31)])
def test_rows_far_apart(s, stride):
    """Offsets past 32 bits, in a long buffer whose rows hold something else, too."""
    dtype, k = "bf16", 16
    t = values(dtype, 1, s, 1, 1, k, k)
    to = types(dtype)
    op = rl.LinearAttention(dtype=dtype, seq=s, batch=1, heads=1, key=k, value=k, scale=0.37)
    room = torch.empty(s * stride, dtype=to["Q"], device="cuda").view(1, s, stride)
    at = {n: room[..., 64 * i:64 * i + k] for i, n in enumerate(("Q", "K", "V", "dY", "Y", "dQ", "dK", "dV"))}
    for n in ("Q", "K", "V", "dY"):
        at[n].copy_(t[n].to(to[n]))
    rest = {n: t[n].float().cuda() for n in ("G", "decay", "initial_state", "d_final_state")}
    ins = {n: at[n] for n in ("Q", "K", "V")} | {n: rest[n] for n in ("G", "decay", "initial_state")}
    f = {n: torch.empty_like(x) for n, x in (("dG", rest["G"]), ("d_decay", rest["decay"]), ("d_initial_state", rest["initial_state"]))}
    op.encode({**ins, "Y": at["Y"]})
    op.backward({**ins, "dY": at["dY"], "d_final_state": rest["d_final_state"], **{n: at[n] for n in ("dQ", "dK", "dV")}, **f})
    norm = rl.RotaryNorm(dtype=dtype, rows=s, q_heads=1, k_heads=1, size=k, table=1, rotary=0)
    out = room[0][:, 1024:1024 + k]
    norm.encode({"Q": room[0][:, :k], "K": room[0][:, 64:64 + k], "Q_out": out})
    torch.cuda.synchronize()
    want = reference(t, dtype, 1, 1, 0.37, None, False, False) | reference(t, dtype, 1, 1, 0.37, None, False, True)
    for n in ("Y", "dQ", "dK", "dV"):
        att.close(at[n], *want[n], dtype, n)
    for n in f:
        att.close(f[n], *want[n], "f32", n)
    x = t["Q"].view(s, 1, k)
    one = torch.ones(s, k, dtype=torch.float64)[:, :0]
    y, Y = rot.reference(x, torch.ones(k, dtype=torch.float64), one, one, torch.ones(s, dtype=torch.bool), rot.pairs(k, 0, False), 1e-6)
    att.close(out, y.flatten(1), Y.flatten(1), dtype, "Q_out")


@pytest.mark.gpu
@pytest.mark.parametrize("b,s", [(3000, 1), (700, 6)])
def test_many_rows(b, s):
    attn_case("f16", b, s, 3, 1, 8, 12, lens=None if s == 1 else [i % (s + 1) for i in range(b)], back=True, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("b,s,groups", [(1, 130, 1), (8, 130, 4), (40, 130, 2)])
def test_gradients_side_by_side_and_one_after_another(dtype, b, s, groups):
    """One head's walks up to a chip of them, and shared heads' sums."""
    attn_case(dtype, b, s, 4, groups, 40, 24, lens=[s - i % 7 for i in range(b)], forward=False, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("k,v,pad", [(24, 20, 0), (24, 16, 3), (64, 64, 0), (128, 128, 8), (100, 70, 1), (200, 136, 0), (16, 256, 0)])
def test_walks_of_many_rows(dtype, k, v, pad):
    """More workgroups than the chip has units: each walk by itself."""
    attn_case(dtype, 90, 70, 1, 1, k, v, lens=[70 - i % 71 for i in range(90)], pad=pad, device="cuda", seed=k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("carried", [False, True])
def test_many_pieces(dtype, carried, monkeypatch):
    """Pieces' states joined by the walks (up to eight before them) and by a launch, walks side by side and one after another."""
    monkeypatch.setenv("RNN_ATTN_PIECE", "64")
    for b, s, lens, reverse in ((1, 576, None, False), (1, 640, None, True), (2, 640, [640, 577], False), (24, 200, [i * 9 for i in range(24)], True)):
        attn_case(dtype, b, s, 2, 1, 32, 48, lens=lens, reverse=reverse, device="cuda", carried=carried, seed=s, gate=0.02, fixed=0.002)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("s,h,k,v", [(2048, 32, 64, 64), (1200, 20, 40, 130)])
def test_parts_of_pieces(dtype, s, h, k, v):
    """Two pieces and more, walked for their states in parts."""
    attn_case(dtype, 2, s, h, 1, k, v, lens=[s, s - 300], back=False, device="cuda", gate=0.02, fixed=0.002)
    attn_case(dtype, 1, s, h, h, k, v, reverse=True, back=False, device="cuda", gate=0.02, fixed=0.002, carried=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("name", ["Q", "K", "V", "dY"])
@pytest.mark.parametrize("b", [2, 70])
def test_gradients_of_values_that_are_not_finite(dtype, name, b):
    """They spoil the gradients that depend on them and no other (but of K and V the decays' of the whole row and head)."""
    s, h, k, v, at = 200, 2, 32, 40, 70
    t = values(dtype, b, s, h, h, k, v)
    clean = reference(t, dtype, h, h, 1.0, None, False, True, "cuda")
    t[name][0, at, 1] = float("inf")     # of head 0
    to = types(dtype)
    d = {n: x.to(to[n]).cuda() for n, x in t.items()}
    op = rl.LinearAttention(dtype=dtype, seq=s, batch=b, heads=h, key=k, value=v)
    out = {n: torch.full(x[0].shape, float("nan"), dtype=to[n], device="cuda") for n, x in clean.items()}
    op.backward({**d, **out})
    torch.cuda.synchronize()
    want = reference(t, dtype, h, h, 1.0, None, False, True, "cuda")
    for n, (value, _) in want.items():
        if n == "d_decay":
            assert not out[n][0].isfinite() and out[n][1].isfinite()
            continue
        ok = value.isfinite()
        assert torch.equal(out[n].isfinite(), ok), n
        zero = torch.zeros_like(value)
        att.close(torch.where(ok, out[n].double(), zero), torch.where(ok, value, zero), torch.where(ok, clean[n][1], zero),
                  dtype if to[n] != torch.float32 else "f32", n)
