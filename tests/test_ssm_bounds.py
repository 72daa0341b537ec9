"""What the bounds of tests/ssm_bounds.py let through (no GPU): outputs computed
in f32 step by step do pass, wrong ones do not.  Mistakes are planted in the
64-bit forms."""
import pytest
import torch

from tests import ssm_bounds as bounds
from tests import ssm_reference as ref


def values(b, s, c, n, groups=1, seed=0, softplus=True):
    gen = torch.Generator().manual_seed(seed)
    shapes = dict(X=(b, s, c), delta=(b, s, c), A=(c, n), B=(b, s, groups * n), C=(b, s, groups * n), D=(c,), Z=(b, s, c), bias=(c,),
                  init=(b, c, n), dY=(b, s, c), dF=(b, c, n))
    v = {k: torch.randn(*size, generator=gen, dtype=torch.float64).float().double() for k, size in shapes.items()}
    v["A"] = -(v["A"].abs() + 0.05).float().double()
    v["bias"] = (v["bias"] * 0.5 - 1).float().double()
    return v


def all_of(v, lens, f32=False, **kw):
    t = {k: x.float() for k, x in v.items()} if f32 else v
    main = [t[k] for k in ("X", "delta", "A", "B", "C")]
    opt = [t["D"], t["Z"], t["bias"], lens, t["init"]]
    y, h = ref.scan(*main, *opt, **kw)
    return {"Y": y, "final_state": h} | ref.scan_grad(*main, t["dY"], *opt, t["dF"], **kw)


def bounds_of(v, lens, chunk, **kw):
    main = [v[k] for k in ("X", "delta", "A", "B", "C", "D", "Z", "bias")]
    return bounds.scan_bounds(*main, lens, v["init"], v["dY"], v["dF"], chunk=chunk, **kw)


SHAPES = [(6, 130, 9, 64, 16, None), (6, 130, 9, 16, 32, [130, 33, 32, 1, 0, 97]), (1, 700, 70, 16, 64, None), (3, 130, 70, 128, 16, [130, 97, 40])]


@pytest.mark.parametrize("b,s,c,n,chunk,lens", SHAPES)
def test_scan_bounds(b, s, c, n, chunk, lens):
    v = values(b, s, c, n)
    want, room = all_of(v, lens), bounds_of(v, lens, chunk)
    # a step by step computation in f32 keeps to them (its dC and dB are stored in f32 too)
    # (ref's own f32 sums over channels and rows go in another order, no deeper)
    for name, t in all_of(v, lens, f32=True).items():
        bounds.check(t, want[name], room[name], "f32", name)
    # and they are narrow: zero is far outside nearly everywhere (of nine channels' sums one may lie near it)
    for name, t in want.items():
        live = t != 0
        assert float((t.abs() > 20 * room[name])[live].double().mean()) > 0.88, name


@pytest.mark.parametrize("b,s,c,n,chunk,lens", SHAPES)
def test_scan_bounds_see_a_dropped_chunk(b, s, c, n, chunk, lens):
    """The steps of one middle chunk left out of the sums over time; the state lost between two chunks."""
    v = values(b, s, c, n)
    want, room = all_of(v, lens), bounds_of(v, lens, chunk)
    at = (s // chunk // 2) * chunk
    part = slice(at, at + chunk)
    d = ref.scan(*(v[k] for k in ("X", "delta", "A", "B", "C", "D", "Z", "bias")), lens, v["init"], keep=True)[2]
    gone = {"ddelta_bias": want["ddelta"][:, part].sum((0, 1)), "dD": (v["dY"] * ref.silu(v["Z"]) * d["x"] * d["live"][..., None])[:, part].sum((0, 1))}
    for name, t in gone.items():
        assert float((t.abs() > room[name]).double().mean()) > 0.9, name
    # rows begun anew at the chunk: what the state before it gives to Y and the final state
    cut = {k: (t[:, part] if k in ("X", "delta", "B", "C", "Z", "dY") else t) for k, t in v.items()} | {"init": torch.zeros_like(v["init"])}
    anew = ref.scan(*(cut[k] for k in ("X", "delta", "A", "B", "C", "D", "Z", "bias")), None, cut["init"])[0]
    whole = torch.stack([torch.tensor(m >= at + chunk) for m in ref.lengths(lens, b, s)])
    first = (anew - want["Y"][:, part])[whole][:, 0].abs() > room["Y"][:, part][whole][:, 0]
    assert float(first.double().mean()) > 0.9


@pytest.mark.parametrize("size,far", [(1024, 1000.0), (8200, 0.0), (70000, 0.0), (2051, 3.0)])
def test_norm_bounds(size, far):
    gen = torch.Generator().manual_seed(1)
    X = (torch.randn(9, size, generator=gen, dtype=torch.float64) + far).float().double()
    scale, shift, dY = (torch.randn(*s, generator=gen, dtype=torch.float64).float().double() for s in ((size,), (size,), (9, size)))
    y, mean, inv = ref.norm(X, scale, shift)
    room = bounds.norm_bounds(X, scale, shift)
    f = [t.float() for t in ref.norm(X.float(), scale.float(), shift.float())]
    for name, got, want in zip(("Y", "Mean", "InvStdDev"), f, (y, mean, inv)):
        bounds.check(got, want, room[name], "f32", name)
    assert float(((y - shift).abs() > 5 * room["Y"]).double().mean()) > 0.9     # x left at its mean is seen
    if far >= 1000:     # and the variance as the mean of squares less the mean's square, in f32
        x = X.float()
        one_pass = 1 / ((x * x).mean(-1) - x.mean(-1) ** 2 + 1e-5).clamp(min=1e-5).sqrt()
        assert ((one_pass.double() - inv).abs() > room["InvStdDev"]).all()
    m, i = mean.float().double(), inv.float().double()
    want = ref.norm_grad(X, scale, m, i, dY)
    room = bounds.norm_grad_bounds(X, scale, m, i, dY, 9)
    for name, t in ref.norm_grad(*(t.float() for t in (X, scale, m, i, dY))).items():
        bounds.check(t, want[name], room[name], "f32", name)
        assert float((want[name].abs() > 20 * room[name]).double().mean()) > 0.9, name
    g = dY * scale
    no_mean = i[:, None] * (g - (X - m[:, None]) * i[:, None] * (g * (X - m[:, None]) * i[:, None]).mean(-1, keepdim=True))
    assert float(((no_mean - want["dX"]).abs() > room["dX"]).double().mean()) > 0.9     # a term left out
