"""The 64-bit plain form of linear attention against its definition as one sum
over pairs of steps, its gradients against automatic ones and differences."""
import pytest
import torch

from tests import attn_reference as att

CASES = [dict(s=7), dict(s=7, lens=[7, 3, 0]), dict(s=5, reverse=True, lens=[2, 5, 9]), dict(s=1), dict(s=6, groups=1), dict(s=4, carried=False)]


def make(s=7, lens=None, reverse=False, groups=2, carried=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    b, h, k, v = 3, 4, 5, 3
    t = {n: torch.randn(*w, generator=gen, dtype=torch.float64) for n, w in dict(
        Q=(b, s, groups * k), K=(b, s, groups * k), V=(b, s, h * v), G=(b, s, h), decay=(h,), init=(b, h, k, v), dY=(b, s, h * v),
        d_final=(b, h, k, v)).items()}
    t["G"], t["decay"] = -t["G"].abs() * 0.3, -t["decay"].abs() * 0.2
    if not carried:
        del t["init"], t["d_final"]
    return t, dict(heads=h, groups=groups, scale=0.7, lens=lens, reverse=reverse), (b, h, k, v)


def forward(t, kw):
    out = att.attn(t["Q"], t["K"], t["V"], G=t["G"], decay=t["decay"], init=t.get("init"), **kw)
    return out["Y"][0], out["final_state"][0]


def loss(t, kw):
    y, f = forward(t, kw)
    return (y * t["dY"]).sum() + ((f * t["d_final"]).sum() if "d_final" in t else 0.0)


@pytest.mark.parametrize("case", CASES)
def test_forward_is_the_sum_over_pairs(case):
    t, kw, (b, h, k, v) = make(**case)
    y, f = forward(t, kw)
    for i in range(b):
        n = min(kw["lens"][i], case["s"]) if kw["lens"] else case["s"]
        times = list(range(n))[::-1] if kw["reverse"] else list(range(n))
        assert (y[i, n:] == 0).all()
        for j in range(h):
            q, kk = (t[x][i].view(case["s"], kw["groups"], k)[:, j // (h // kw["groups"])] for x in "QK")
            vv, g = t["V"][i].view(case["s"], h, v)[:, j], t["G"][i, :, j] + t["decay"][j]
            init = t["init"][i, j] if "init" in t else torch.zeros(k, v, dtype=torch.float64)
            for a, ta in enumerate(times):
                want = torch.exp(sum(g[x] for x in times[:a + 1])) * (q[ta] @ init)
                for c, tc in enumerate(times[:a + 1]):
                    want = want + torch.exp(sum([g[x] for x in times[c + 1:a + 1]], torch.tensor(0.0))) * (q[ta] @ kk[tc]) * vv[tc]
                torch.testing.assert_close(y[i, ta].view(h, v)[j], kw["scale"] * want)
        if n == 0 and "init" in t:
            assert torch.equal(f[i], t["init"][i])


@pytest.mark.parametrize("case", CASES)
def test_gradients(case):
    t, kw, _ = make(**case)
    names = {"Q": "dQ", "K": "dK", "V": "dV", "G": "dG", "decay": "d_decay", "init": "d_initial_state"}
    leaves = {n: t[n].clone().requires_grad_() for n in names if n in t}
    loss({**t, **leaves}, kw).backward()
    got = att.attn(t["Q"], t["K"], t["V"], G=t["G"], decay=t["decay"], init=t.get("init"), dY=t["dY"], d_final=t.get("d_final"), **kw)
    gen = torch.Generator().manual_seed(5)
    for n, d in names.items():
        if n not in t:
            continue
        value, bound = got[d]
        want = leaves[n].grad
        want = torch.zeros_like(value) if want is None else want
        torch.testing.assert_close(value.view(want.shape), want, rtol=1e-9, atol=1e-11)
        assert (bound >= 0).all() and bound.shape == value.shape
        way = torch.randn(want.shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        slope = (loss({**t, n: t[n] + e * way}, kw) - loss({**t, n: t[n] - e * way}, kw)) / (2 * e)
        torch.testing.assert_close((value.view(want.shape) * way).sum(), slope, rtol=1e-6, atol=1e-7)


def test_decays_above_one_count_as_one():
    t, kw, _ = make(s=5)
    t["G"][:, 2] = 5.0
    flat = dict(t, G=torch.where(t["G"] + t["decay"] > 0, -t["decay"], t["G"]))
    for a, b in zip(forward(t, kw), forward(flat, kw)):
        torch.testing.assert_close(a, b)
    got = att.attn(t["Q"], t["K"], t["V"], G=t["G"], decay=t["decay"], init=t["init"], dY=t["dY"], d_final=t["d_final"], **kw)
    assert (got["dG"][0][:, 2] == 0).all()
