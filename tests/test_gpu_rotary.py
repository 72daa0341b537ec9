"""Norms of queries and keys with the position rotation on the GPU against
their 64-bit plain form: types, sizes, pairs, strides, positions that are none,
in place, graphs.

Bounds, u = 2^-24: a sum of squares adds 24 values one after another at most
(16 of a lane, six across the lanes), its root and quotient and the products by
scale, cosine or sine a dozen roundings more; a scale's gradient sums rows times
heads of them."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import attn_reference as att
from tests import ssm_reference as ref
from tests.gpu_harness import note
from tests.test_gpu_ssm import SENTINEL, Bufs, rounded

pytestmark = pytest.mark.gpu
U = att.U
DEPTH = 36 * U


def pairs(size, rotary, interleaved):
    p = torch.arange(rotary // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rotary // 2)


def turn(x, cos, sin, first, second, mag=False):
    """A rotation of [rows, heads, size], or the sum of its terms' magnitudes."""
    out = x.clone()
    a, b, c, s = x[..., first], x[..., second], cos[:, None], sin[:, None]
    if mag:
        c, s = c.abs(), s.abs()
        out[..., first], out[..., second] = a * c + b * s, b * c + a * s
    else:
        out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    return out


def reference(x, scale, cos, sin, live, at, eps, dy=None):
    """(value, bound) of the output, or of dx and dscale."""
    x = x * live[:, None, None]
    root = torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    xh = x / root
    if dy is None:
        n = xh * scale
        m = live[:, None, None].double()
        return turn(n, cos, sin, *at) * m, DEPTH * turn(n.abs(), cos, sin, *at, mag=True) * m
    dy = dy * live[:, None, None]
    g, G = turn(dy, cos, -sin, *at), turn(dy.abs(), cos, sin, *at, mag=True)
    mean, Mean = (g * scale * xh).mean(-1, keepdim=True), (G * scale.abs() * xh.abs()).mean(-1, keepdim=True)
    n = x.shape[0] * x.shape[1]
    return ((g * scale - xh * mean) / root, DEPTH * (G * scale.abs() + 2 * xh.abs() * Mean) / root), \
        ((g * xh).sum((0, 1)), (DEPTH + n * U) * (G * xh.abs()).sum((0, 1)))


def table(n, rotary):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / max(1, rotary))
    return torch.cos(a).float(), torch.sin(a).float()


def make(dtype, rows, qh, kh, size, rotary, n=100, seed=0, scales=True, none=()):
    gen = torch.Generator().manual_seed(seed)
    t = {k: rounded(torch.randn(*w, generator=gen, dtype=torch.float64), dtype) for k, w in dict(
        Q=(rows, qh * size), K=(rows, kh * size), q_scale=(size,), k_scale=(size,), dQ_out=(rows, qh * size), dK_out=(rows, kh * size)).items()}
    t["cos"], t["sin"] = (x.double() for x in table(n, rotary))
    t["positions"] = torch.randint(n, (rows,), generator=gen)
    for r in none:
        t["positions"][r] = -1 - r
    if not scales:
        del t["q_scale"], t["k_scale"]
    return t


def case(dtype, rows, qh, kh, size, rotary, interleaved=False, pad=0, odd=0, seed=0, scales=True, none=(), scale_x=1.0, eps=1e-6, n=100):
    note(f"rotary {dtype} rows {rows} heads {qh}/{kh} size {size} rotary {rotary} interleaved {interleaved} pad {pad} odd {odd} none {none}")
    t = make(dtype, rows, qh, kh, size, rotary, n, seed, scales, none)
    t["Q"], t["K"] = (rounded(t[x] * scale_x, dtype) for x in "QK")
    op = rl.RotaryNorm(dtype=dtype, rows=rows, q_heads=qh, k_heads=kh, size=size, rotary=rotary, table=n, interleaved=interleaved, epsilon=eps)
    dt, f32 = ref.TYPES[dtype], torch.float32
    live = t["positions"] >= 0
    at = pairs(size, rotary, interleaved)
    worst = {}
    for back in (False, True):
        m = Bufs(pad, odd)
        for x in ("Q", "K") + (("dQ_out", "dK_out") if back else ()):
            v = t[x].clone()
            v[~live] = float("nan")     # a row that is none is not read
            m.rows(x, v, dt)
        for x in ("q_scale", "k_scale"):
            if x in t:
                m.plain(x, t[x], dt)
        m.plain("cos", t["cos"], f32)
        m.plain("sin", t["sin"], f32)
        m.plain("positions", t["positions"], torch.int32)
        for x, h in (("Q", qh), ("K", kh)):
            m.out("d" + x if back else x + "_out", (rows, h * size), dt, row=True)
            if back:
                m.out(f"d{x.lower()}_scale", (size,), f32)
        (op.backward if back else op.encode)(m.t)
        m.check()
        cos, sin = (t[x][t["positions"].clamp(min=0)] for x in ("cos", "sin"))
        for x, h in (("Q", qh), ("K", kh)):
            scale = t.get(x.lower() + "_scale", torch.ones(size, dtype=torch.float64))
            args = (t[x].view(rows, h, size), scale, cos, sin, live, at, eps)
            if back:
                (dx, Dx), (ds, Ds) = reference(*args, dy=t[f"d{x}_out"].view(rows, h, size))
                worst["d" + x] = att.close(m.t["d" + x].view(rows, h * size), dx.flatten(1), Dx.flatten(1), dtype, "d" + x)
                worst["ds" + x] = att.close(m.t[f"d{x.lower()}_scale"], ds, Ds, "f32", f"d{x.lower()}_scale")
            else:
                y, Y = reference(*args)
                worst[x] = att.close(m.t[x + "_out"].view(rows, h * size), y.flatten(1), Y.flatten(1), dtype, x + "_out")
    note("  worst " + " ".join(f"{n} {w:.2f}" for n, w in worst.items()))


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size,rotary", [(1, 0), (2, 2), (7, 4), (16, 16), (50, 26), (64, 64), (64, 0), (80, 32), (96, 96), (128, 128), (128, 64),
                                         (129, 128), (256, 256), (511, 100), (512, 512)])
def test_sizes(dtype, interleaved, size, rotary):
    case(dtype, 5, 3, 2, size, rotary, interleaved)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("rows,qh,kh", [(1, 1, 1), (1, 33, 2), (2, 16, 16), (3, 7, 1), (64, 8, 8), (257, 6, 3), (4099, 2, 1)])
def test_rows_and_heads(dtype, rows, qh, kh):
    case(dtype, rows, qh, kh, 64, 64, none=[0] if rows == 2 else [rows // 2] if rows > 2 else [])
    case(dtype, rows, qh, kh, 48, 20, True, none=range(0, rows, 3) if rows > 1 else [])


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("pad,odd", [(0, 0), (8, 0), (16, 4), (3, 1), (0, 5)])
def test_strides(dtype, pad, odd):
    case(dtype, 9, 5, 2, 64, 32, pad=pad, odd=odd)
    case(dtype, 9, 5, 2, 64, 64, True, pad=pad, odd=odd, scales=False)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_small_and_large_values(dtype):
    case(dtype, 6, 2, 2, 32, 32, scale_x=1e-3)
    case(dtype, 6, 2, 2, 32, 32, scale_x=300.0)
    case(dtype, 6, 2, 2, 32, 32, scale_x=0.0)


def run(op, t, names, dt):
    shapes = {"Q_out": t["Q"].shape, "K_out": t["K"].shape, "dQ": t["Q"].shape, "dK": t["K"].shape}
    outs = {n: torch.full(shapes[n], SENTINEL, dtype=dt, device="cuda") if n in shapes else torch.full((op._specs[n][0]), SENTINEL, device="cuda")
            for n in names}
    (op.backward if names[0].startswith("d") else op.encode)({**{n: x for n, x in t.items() if names[0].startswith("d") or not n.startswith("d")}, **outs})
    return outs


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_in_place_chosen_outputs_and_positions_past_the_table(dtype):
    rows, qh, kh, size, rotary = 37, 6, 2, 64, 32
    dt = ref.TYPES[dtype]
    t = {n: x.to(torch.int32 if n == "positions" else torch.float32 if n in ("cos", "sin") else dt).cuda()
         for n, x in make(dtype, rows, qh, kh, size, rotary, none=[5]).items()}
    op = rl.RotaryNorm(dtype=dtype, rows=rows, q_heads=qh, k_heads=kh, size=size, rotary=rotary, table=100)
    full, back = run(op, t, ("Q_out", "K_out"), dt), run(op, t, ("dQ", "dK", "dq_scale", "dk_scale"), dt)
    torch.cuda.synchronize()
    for names, of in ((("Q_out",), full), (("K_out",), full), (("dQ",), back), (("dK",), back), (("dq_scale",), back), (("dk_scale",), back)):
        one = run(op, t, names, dt)
        torch.cuda.synchronize()
        assert torch.equal(one[names[0]], of[names[0]]), names
    q, k = t["Q"].clone(), t["K"].clone()
    op.encode({**{n: t[n] for n in ("q_scale", "k_scale", "cos", "sin", "positions")}, "Q": q, "K": k, "Q_out": q, "K_out": k})
    torch.cuda.synchronize()
    assert torch.equal(q, full["Q_out"]) and torch.equal(k, full["K_out"])
    t["positions"][7] = 100
    t["positions"][8] = 2 ** 31 - 1
    past = run(op, t, ("Q_out", "K_out"), dt)
    torch.cuda.synchronize()
    for n, h in (("Q_out", qh), ("K_out", kh)):
        x, y = past[n].view(rows, h, size), full[n].view(rows, h, size)
        assert x[7:9, :, :rotary].isnan().all() and torch.equal(x[7:9, :, rotary:], y[7:9, :, rotary:])
        assert torch.equal(x[:7], y[:7]) and torch.equal(x[9:], y[9:])


def test_empty():
    op = rl.RotaryNorm(dtype="f32", rows=0, q_heads=2, k_heads=1, size=8, table=4)
    t = {"Q": torch.empty(0, 16), "K": torch.empty(0, 8), "dQ_out": torch.empty(0, 16), "dK_out": torch.empty(0, 8),
         "cos": torch.zeros(4, 4), "sin": torch.zeros(4, 4), "positions": torch.empty(0, dtype=torch.int32)}
    back = run(op, {n: x.cuda() for n, x in t.items()}, ("dQ", "dK", "dq_scale", "dk_scale"), torch.float32)
    torch.cuda.synchronize()
    assert (back["dq_scale"] == 0).all() and (back["dk_scale"] == 0).all()
    queries = rl.RotaryNorm(dtype="f32", rows=3, q_heads=2, k_heads=0, size=8, table=4, rotary=0)
    x, y = torch.randn(3, 16, device="cuda"), torch.empty(3, 16, device="cuda")
    queries.encode({"Q": x, "Q_out": y})
    torch.cuda.synchronize()
    v = x.double().view(3, 2, 8)
    att.close(y.view(3, 2, 8), (v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6)), (DEPTH * v.abs()) / v.square().mean(-1, keepdim=True).sqrt(),
              "f32", "Q_out")


def test_graph():
    rows, qh, kh, size = 300, 4, 2, 64
    t = {n: x.to(torch.int32 if n == "positions" else torch.float32 if n in ("cos", "sin") else torch.bfloat16).cuda()
         for n, x in make("bf16", rows, qh, kh, size, size).items()}
    op = rl.RotaryNorm(dtype="bf16", rows=rows, q_heads=qh, k_heads=kh, size=size, table=100)
    names = (("Q_out", "K_out"), ("dQ", "dK", "dq_scale", "dk_scale"))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        held = [run(op, t, n, torch.bfloat16) for n in names]
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            op.encode({**{n: x for n, x in t.items() if not n.startswith("d")}, **held[0]})
            op.backward({**t, **held[1]})
    eager = rl.RotaryNorm(dtype="bf16", rows=rows, q_heads=qh, k_heads=kh, size=size, table=100)
    for seed in range(4):
        new = make("bf16", rows, qh, kh, size, size, seed=seed + 9)
        for n in t:
            t[n].copy_(new[n])
        graph.replay()
        want = [run(eager, t, n, torch.bfloat16) for n in names]
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            for n in a:
                assert torch.equal(a[n], b[n]), (seed, n)
