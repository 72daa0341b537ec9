"""The 64-bit plain forms of the state space operators and of layer
normalization (tests/ssm_reference.py) against torch's automatic derivatives
and against differences, and their magnitudes against their values."""
import pytest
import torch

from tests import ssm_reference as ref


def draw(seed, *shapes):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=gen, dtype=torch.float64) for s in shapes]


SEQ = [(False, None), (True, None), (False, [4, 0, 9, 2]), (True, [1, 5, -3, 5])]


@pytest.mark.parametrize("reverse,lens", SEQ)
@pytest.mark.parametrize("act", [True, False])
def test_conv_gradient(reverse, lens, act):
    X, W, B, init, dY, dF = draw(1, (4, 5, 3), (3, 4), (3,), (4, 3, 3), (4, 5, 3), (4, 3, 3))
    leaves = [t.requires_grad_() for t in (X, W, B, init)]
    kw = dict(act=act, reverse=reverse)

    def f(X, W, B, init):
        y, h = ref.conv(X, W, B, lens, init, **kw)
        return (y * dY).sum() + (h * dF).sum()

    auto = torch.autograd.grad(f(*leaves), leaves)
    assert torch.autograd.gradcheck(f, leaves)
    with torch.no_grad():
        got = ref.conv_grad(X, W, dY, B, lens, init, dF, **kw)
        mag = ref.conv_grad(X, W, dY, B, lens, init, dF, mag=True, **kw)
    for name, a in zip(("dX", "dW", "dB", "d_initial_state"), auto):
        assert torch.allclose(got[name], a, atol=1e-12), name
        assert (mag[name] >= got[name].abs() - 1e-12).all(), name


@pytest.mark.parametrize("reverse,lens", SEQ)
@pytest.mark.parametrize("gate,softplus,groups", [(True, True, 1), (False, True, 2), (True, False, 2)])
def test_scan_gradient(reverse, lens, gate, softplus, groups):
    b, s, c, n = 4, 5, 4, 3
    X, delta, A, B, C, D, Z, bias, init, dY, dF = draw(2, (b, s, c), (b, s, c), (c, n), (b, s, groups * n), (b, s, groups * n), (c,),
                                                        (b, s, c), (c,), (b, c, n), (b, s, c), (b, c, n))
    A = -A.abs()
    if not gate:
        Z = torch.zeros(0, dtype=torch.float64)
    leaves = [t.requires_grad_() for t in (X, delta, A, B, C, D, Z, bias, init)]
    kw = dict(groups=groups, softplus=softplus, reverse=reverse)

    def f(X, delta, A, B, C, D, Z, bias, init):
        y, h = ref.scan(X, delta, A, B, C, D, Z if gate else None, bias, lens, init, **kw)
        return (y * dY).sum() + (h * dF).sum()

    auto = torch.autograd.grad(f(*leaves), leaves, allow_unused=True)
    # The difference of two sums whose terms have the magnitude M, each off by
    # at most some 64 roundings, over a step of 2e-6: without softplus decays
    # grow, M reaches 1e5 and more, and that is above gradcheck's 1e-5.
    with torch.no_grad():
        y, h = ref.scan(X, delta, A, B, C, D, Z if gate else None, bias, lens, init, mag=True, **kw)
        M = float((y * dY.abs()).sum() + (h * dF.abs()).sum())
    assert torch.autograd.gradcheck(f, leaves, eps=1e-6, atol=1e-5 + 2 * 64 * 2.0 ** -53 * M / 2e-6)
    with torch.no_grad():
        args = (X, delta, A, B, C, dY, D, Z if gate else None, bias, lens, init, dF)
        got, mag = ref.scan_grad(*args, **kw), ref.scan_grad(*args, mag=True, **kw)
    for name, a in zip(("dX", "ddelta", "dA", "dB", "dC", "dD", "dZ", "ddelta_bias", "d_initial_state"), auto):
        if name == "dZ" and not gate:
            continue
        assert torch.allclose(got[name], a, atol=1e-12), name
        assert (mag[name] >= got[name].abs() - 1e-12).all(), name


def test_norm_gradient():
    X, scale, shift, dY = draw(3, (4, 7), (7,), (7,), (4, 7))
    leaves = [t.requires_grad_() for t in (X, scale, shift)]

    def f(X, scale, shift):
        return (ref.norm(X, scale, shift)[0] * dY).sum()

    auto = torch.autograd.grad(f(*leaves), leaves)
    assert torch.autograd.gradcheck(f, leaves)
    want = torch.nn.functional.layer_norm(X, (7,), scale, shift, 1e-5)
    assert torch.allclose(ref.norm(X, scale, shift)[0], want, atol=1e-12)
    with torch.no_grad():
        _, mean, inv = ref.norm(X, scale, shift)
        got, mag = ref.norm_grad(X, scale, mean, inv, dY), ref.norm_grad(X, scale, mean, inv, dY, mag=True)
    for name, a in zip(("dX", "dScale", "dB"), auto):
        assert torch.allclose(got[name], a, atol=1e-12), name
        assert (mag[name] >= got[name].abs() - 1e-12).all(), name


def test_conv_by_hand():
    """Two taps, no activation: y_s = 1 + 2 x_{s-1} + 3 x_s from the state 5."""
    X = torch.tensor([[[1.0], [2.0]]], dtype=torch.float64)
    W, B, init = torch.tensor([[2.0, 3.0]], dtype=torch.float64), torch.ones(1, dtype=torch.float64), torch.full((1, 1, 1), 5.0, dtype=torch.float64)
    y, h = ref.conv(X, W, B, None, init, act=False)
    assert y.flatten().tolist() == [14.0, 9.0] and h.item() == 2.0
    y, h = ref.conv(X, W, B, None, init, act=False, reverse=True)
    assert y.flatten().tolist() == [8.0, 17.0] and h.item() == 1.0


def test_scan_by_hand():
    """One channel, one state, no softplus, d = 1, a = 1/2: h = h/2 + 3 x, y = 2 h + x."""
    one = torch.ones(1, 2, 1, dtype=torch.float64)
    A = torch.log(torch.tensor([[0.5]], dtype=torch.float64))
    X = torch.tensor([[[1.0], [2.0]]], dtype=torch.float64)
    y, h = ref.scan(X, one, A, 3 * one, 2 * one, torch.ones(1, dtype=torch.float64), softplus=False,
                    initial_state=torch.full((1, 1, 1), 4.0, dtype=torch.float64))
    assert torch.allclose(y.flatten(), torch.tensor([11.0, 19.0], dtype=torch.float64)) and abs(h.item() - 8.5) < 1e-12
