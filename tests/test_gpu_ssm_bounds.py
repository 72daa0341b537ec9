"""The state space operators and layer normalization on the GPU within bounds
that follow each output's own terms (tests/ssm_bounds.py), where bounds by
magnitude alone would let a lost part of a sum, or a row's mean, go unseen:
chunks of the time axis, many states, long rows and rows far from zero."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import ssm_bounds as bounds
from tests import ssm_reference as ref
from tests.gpu_harness import note
from tests.test_gpu_ssm import Bufs, conv_case, lead, rounded, scan_values

pytestmark = pytest.mark.gpu


def scan_case(monkeypatch, dtype, b, s, c, n, chunk, groups=1, lens=None, reverse=False, layout=1, gate=True, softplus=True, pad=0,
              odd=0, seed=0, signed=False):
    """Forward and backward with everything there, chunks of `chunk` steps (0: one).  `signed`: steps of both signs."""
    note(f"scan {dtype} b{b} s{s} c{c} n{n} chunk {chunk} groups {groups} lens {lens} reverse {reverse} layout {layout}")
    monkeypatch.setenv("RNN_SCAN_CHUNK", str(chunk or 1 << 20))
    dt, f32 = ref.TYPES[dtype], torch.float32
    v = scan_values(dtype, b, s, c, n, groups, softplus, seed)
    if signed:
        v["delta"] = v["delta"] * torch.where(torch.arange(s) % 3 == 0, -1.0, 1.0)[None, :, None]
    kw = dict(D=v["D"], Z=v["Z"] if gate else None, delta_bias=v["bias"], lens=lens, initial_state=v["init"], groups=groups,
              softplus=softplus, reverse=reverse)
    main = [v[k] for k in ("X", "delta", "A", "B", "C")]
    op = rl.SelectiveScan(dtype=dtype, seq=s, batch=b, channels=c, state=n, groups=groups, delta_softplus=softplus,
                          direction="reverse" if reverse else "forward", layout=layout)

    def inputs(m, names):
        for k in names:
            m.rows(k, lead(v[k], layout), dt)
        m.plain("A", v["A"], f32)
        m.plain("D", v["D"], f32)
        m.plain("delta_bias", v["bias"], f32)
        m.plain("initial_state", v["init"], f32)
        if lens is not None:
            m.plain("sequence_lens", torch.tensor(lens), torch.int32)

    rows = ("X", "delta", "B", "C") + (("Z",) if gate else ())
    row, bc = tuple(lead(v["X"], layout).shape), tuple(lead(v["B"], layout).shape)
    f = Bufs(pad, odd)
    inputs(f, rows)
    f.out("Y", row, dt, row=True)
    f.out("final_state", (b, c, n), f32)
    op.encode(f.t)
    f.check()
    g = Bufs(pad, odd)
    inputs(g, rows + ("dY",))
    g.plain("d_final_state", v["dF"], f32)
    narrow = [("dX", row), ("ddelta", row), ("dB", bc), ("dC", bc)] + ([("dZ", row)] if gate else [])
    for name, shape in narrow:
        g.out(name, shape, dt, row=True)
    for name, shape in (("dA", (c, n)), ("dD", (c,)), ("ddelta_bias", (c,)), ("d_initial_state", (b, c, n))):
        g.out(name, shape, f32)
    op.backward(g.t)
    g.check()
    y, h = ref.scan(*main, **kw)
    want = {"Y": y, "final_state": h} | ref.scan_grad(*main, v["dY"], d_final=v["dF"], **kw)
    room = bounds.scan_bounds(*main, dY=v["dY"], d_final=v["dF"], chunk=chunk or 1 << 30, **kw)
    narrow = {k for k, _ in narrow} | {"Y"}
    for name, t in want.items():
        got = (f if name in ("Y", "final_state") else g).t[name]
        bounds.check(lead(got, layout) if name in narrow else got, t, room[name], dtype if name in narrow else "f32", name)


@pytest.mark.parametrize("n,chunk", [(2, 32), (16, 32), (16, 64), (24, 32), (32, 32), (64, 16), (128, 16)])
@pytest.mark.parametrize("reverse,lens", [(False, None), (True, [130, 33, 32, 1, 0, 97])])
def test_scan_chunks(monkeypatch, n, chunk, reverse, lens):
    scan_case(monkeypatch, "f32", 6, 130, 9, n, chunk, reverse=reverse, lens=lens)


@pytest.mark.parametrize("dtype,b,s,c,n,chunk,lens", [("bf16", 1, 700, 70, 16, 64, None), ("f32", 2, 300, 33, 5, 64, [300, 129]),
                                                      ("f32", 1, 700, 70, 16, 0, None)])
def test_scan_long_rows(monkeypatch, dtype, b, s, c, n, chunk, lens):
    scan_case(monkeypatch, dtype, b, s, c, n, chunk, lens=lens)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n,groups,c", [(64, 1, 70), (64, 2, 128), (128, 1, 64), (100, 3, 195), (40, 1, 66)])
@pytest.mark.parametrize("chunk", [0, 48])
def test_scan_many_states(monkeypatch, dtype, n, groups, c, chunk):
    """64 states and more over many segments, rows of unequal length."""
    scan_case(monkeypatch, dtype, 3, 150, c, n, chunk, groups, lens=[150, 97, 46], layout=0 if groups == 2 else 1,
              reverse=groups == 3, pad=0 if n == 64 else 6)


@pytest.mark.parametrize("gate,softplus", [(False, True), (True, False), (False, False)])
def test_scan_options(monkeypatch, gate, softplus):
    scan_case(monkeypatch, "f32", 2, 70, 66, 16, 32, 2, gate=gate, softplus=softplus)


@pytest.mark.parametrize("dtype,c,n,groups,layout,reverse,lens,pad", [
    ("f32", 130, 16, 2, 0, True, [130, 64, 33, 0], 0), ("bf16", 66, 24, 1, 1, False, None, 6), ("f16", 70, 5, 1, 1, True, [97, 130, 32, 65], 3)])
def test_scan_steps_of_both_signs(monkeypatch, dtype, c, n, groups, layout, reverse, lens, pad):
    """Without softplus, every third step back: gradients at chunks' starts are walked back to, not summed forward."""
    scan_case(monkeypatch, dtype, 4, 130, c, n, 32, groups, lens, reverse, layout, softplus=False, pad=pad, signed=True)


def norm_case(dtype, rows, size, far=0.0, pad=0, odd=0):
    note(f"norm {dtype} rows {rows} size {size} far {far} pad {pad} odd {odd}")
    dt, f32 = ref.TYPES[dtype], torch.float32
    gen = torch.Generator().manual_seed(size)
    v = {k: rounded(torch.randn(*s, generator=gen, dtype=torch.float64), dtype)
         for k, s in (("X", (rows, size)), ("Scale", (size,)), ("B", (size,)), ("dY", (rows, size)))}
    v["X"] = rounded(v["X"] + far, dtype)
    op = rl.LayerNorm(dtype=dtype, rows=rows, size=size, epsilon=1e-5)
    m = Bufs(pad, odd)
    m.rows("X", v["X"], dt)
    m.plain("Scale", v["Scale"], dt)
    m.plain("B", v["B"], dt)
    m.out("Y", (rows, size), dt, row=True)
    m.out("Mean", (rows,), f32)
    m.out("InvStdDev", (rows,), f32)
    op.encode(m.t)
    m.check()
    eps = float(torch.tensor(1e-5, dtype=f32))
    y, mean, inv = ref.norm(v["X"], v["Scale"], v["B"], eps)
    room = bounds.norm_bounds(v["X"], v["Scale"], v["B"], eps)
    for name, t, kind in (("Y", y, dtype), ("Mean", mean, "f32"), ("InvStdDev", inv, "f32")):
        bounds.check(m.t[name], t, room[name], kind, name)
    g = Bufs(pad, odd)
    g.rows("X", v["X"], dt)
    g.rows("dY", v["dY"], dt)
    g.plain("Scale", v["Scale"], dt)
    g.plain("Mean", mean, f32)
    g.plain("InvStdDev", inv, f32)
    g.out("dX", (rows, size), dt, row=True)
    g.out("dScale", (size,), f32)
    g.out("dB", (size,), f32)
    op.backward(g.t)
    g.check()
    a = (v["X"], v["Scale"], mean.float().double(), inv.float().double(), v["dY"])
    want = ref.norm_grad(*a)
    # the rows' sums are in at least min(rows / 4, 15) parts of like length, joined 16 ways
    room = bounds.norm_grad_bounds(*a, -(-rows // max(1, min(-(-rows // 4), 15))) + 2 + 512 // 16 + 16)
    for name, t in want.items():
        bounds.check(g.t[name], t, room[name], dtype if name == "dX" else "f32", name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [7, 100, 129, 500, 1000, 1290, 2051, 3001, 4093, 5001, 8191, 8192, 8200])
def test_norm_sizes(dtype, size):
    """Rows that are not whole 16-byte pieces among them, with enough of them for many parts of a sum."""
    norm_case(dtype, 515, size)


@pytest.mark.parametrize("dtype,rows,size,pad,odd", [("bf16", 37, 16384, 0, 0), ("f32", 300, 9001, 3, 1), ("f16", 1, 70000, 0, 0),
                                                     ("bf16", 1030, 2050, 6, 0), ("f16", 2050, 2048, 2, 0), ("f32", 700, 4098, 0, 0)])
def test_norm_long_rows(dtype, rows, size, pad, odd):
    norm_case(dtype, rows, size, pad=pad, odd=odd)


@pytest.mark.parametrize("dtype,rows,size,far", [("f32", 9, 1024, 1000.0), ("f32", 5000, 1024, 1000.0), ("f32", 33, 1001, -300.0),
                                                 ("f32", 17, 9001, 1000.0), ("bf16", 64, 2048, 8.0), ("f16", 64, 100, 50.0)])
def test_norm_far_from_zero(dtype, rows, size, far):
    norm_case(dtype, rows, size, far=far)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [6, 7])
@pytest.mark.parametrize("c,pad,odd", [(72, 0, 0), (61, 3, 1)])
def test_conv_widths(dtype, k, c, pad, odd):
    conv_case(dtype, 3, 83, c, k, lens=[83, 16, 5], pad=pad, odd=odd, dead=float("nan"))
