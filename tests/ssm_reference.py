"""Plain 64-bit forms of the state space operators and of layer normalization,
step after step as they are defined, with the gradients' formulas, and the
magnitudes that error bounds go by.

Tensors are float64 CPU tensors, sequence tensors [batch, seq, n].  With
``mag=True`` every product and sum is taken over absolute values (the decays
exp(d A) stay as they are): the result bounds the sum of the magnitudes of all
terms that make up an output.  A computation in f32 whose longest chain of
roundings has n of them is then off by at most about n * 2^-24 times that."""
import torch

EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}     # half a step, relative
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def order(t, lens, reverse):
    """[batch, seq, n] -> its steps (zero past the length), and the way back."""
    out = torch.zeros_like(t)
    for b, n in enumerate(lens):
        out[b, :n] = t[b, :n].flip(0) if reverse else t[b, :n]
    return out


def lengths(lens, batch, seq):
    return [seq] * batch if lens is None else [min(max(int(v), 0), seq) for v in lens]


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x):
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def conv(X, W, B=None, lens=None, initial_state=None, act=True, reverse=False, mag=False):
    """Y, final_state."""
    b, s, c = X.shape
    k = W.shape[1]
    lens = lengths(lens, b, s)
    X = order(X, lens, reverse)
    init = torch.zeros(b, k - 1, c, dtype=X.dtype) if initial_state is None else initial_state
    B = torch.zeros(c, dtype=X.dtype) if B is None else B
    final = torch.stack([torch.cat([init[i], X[i, :n]])[n:n + k - 1] for i, n in enumerate(lens)]) if b else init.clone()
    if mag:
        X, W, B, init = X.abs(), W.abs(), B.abs(), init.abs()
    seen = torch.cat([init, X], 1)
    p = B + sum(seen[:, j:j + s] * W[:, j] for j in range(k))
    y = (p if mag else silu(p)) if act else p       # |silu(p)| <= |p|
    return order(y, lens, reverse), final


def conv_grad(X, W, dY, B=None, lens=None, initial_state=None, d_final=None, act=True, reverse=False, mag=False):
    b, s, c = X.shape
    k = W.shape[1]
    lens = lengths(lens, b, s)
    X, dY = order(X, lens, reverse), order(dY, lens, reverse)
    init = torch.zeros(b, k - 1, c, dtype=X.dtype) if initial_state is None else initial_state
    B = torch.zeros(c, dtype=X.dtype) if B is None else B
    seen = torch.cat([init, X], 1)
    dp = dY
    if act:
        p = B + sum(seen[:, j:j + s] * W[:, j] for j in range(k))
        if mag:   # act' and how far a rounding of p moves it: |act''| <= 1/2, by the magnitude of p's terms
            pm = B.abs() + sum(seen[:, j:j + s].abs() * W[:, j].abs() for j in range(k))
            dp = dY.abs() * (1.2 + pm)
        else:
            dp = dY * dsilu(p)
    if mag:
        W, seen, dp = W.abs(), seen.abs(), dp.abs()
    dseen = torch.zeros_like(seen)
    for j in range(k):
        dseen[:, j:j + s] += dp * W[:, j]
    if d_final is not None:
        for i, n in enumerate(lens):
            dseen[i, n:n + k - 1] += d_final[i].abs() if mag else d_final[i]
    dW = torch.stack([(dp * seen[:, j:j + s]).sum((0, 1)) for j in range(k)], 1)
    return {"dX": order(dseen[:, k - 1:], lens, reverse), "dW": dW, "dB": dp.sum((0, 1)), "d_initial_state": dseen[:, :k - 1]}


def scan(X, delta, A, B, C, D=None, Z=None, delta_bias=None, lens=None, initial_state=None, groups=1, softplus=True,
         reverse=False, mag=False, keep=False):
    """Y, final_state (with keep: all that the gradient's formulas use)."""
    b, s, c = X.shape
    n = A.shape[1]
    lens = lengths(lens, b, s)
    X, delta, B, C = (order(t, lens, reverse) for t in (X, delta, B, C))
    Z = None if Z is None else order(Z, lens, reverse)
    of = torch.arange(c) // (c // groups)
    raw = delta + (0 if delta_bias is None else delta_bias)
    d = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    Bg, Cg = B.view(b, s, groups, n)[:, :, of], C.view(b, s, groups, n)[:, :, of]
    h = torch.zeros(b, c, n, dtype=X.dtype) if initial_state is None else initial_state.clone()
    D = torch.zeros(c, dtype=X.dtype) if D is None else D
    x, dm = X, d
    if mag:
        x, dm, Bg, Cg, h, D = X.abs(), d.abs(), Bg.abs(), Cg.abs(), h.abs(), D.abs()
    live = torch.tensor([[t < m for t in range(s)] for m in lens]).view(b, s)
    hs, ys = [h], []
    for t in range(s):
        new = torch.exp(d[:, t, :, None] * A) * h + (dm[:, t] * x[:, t])[..., None] * Bg[:, t]
        h = torch.where(live[:, t, None, None], new, h)
        hs.append(h)
        ys.append((h * Cg[:, t]).sum(-1) + D * x[:, t])
    y = torch.stack(ys, 1) if s else torch.zeros_like(X)
    out = y
    if Z is not None:
        out = y * ((silu(Z)).abs() if mag else silu(Z))
    Y = order(out, lens, reverse)
    if keep:
        return Y, h, dict(x=x, raw=raw, d=d, dm=dm, Bg=Bg, Cg=Cg, D=D, hs=hs, y=y, live=live, lens=lens, Z=Z)
    return Y, h


def scan_grad(X, delta, A, B, C, dY, D=None, Z=None, delta_bias=None, lens=None, initial_state=None, d_final=None, groups=1,
              softplus=True, reverse=False, mag=False):
    b, s, c = X.shape
    n = A.shape[1]
    _, _, k = scan(X, delta, A, B, C, D, Z, delta_bias, lens, initial_state, groups, softplus, reverse, mag, keep=True)
    lens, d, dm, x = k["lens"], k["d"], k["dm"], k["x"]
    g = order(dY, lens, reverse)
    g = g.abs() if mag else g
    out = {}
    if Z is not None:
        sz, dz = silu(k["Z"]), dsilu(k["Z"])
        if mag:
            sz, dz = sz.abs(), dz.abs() + sz.abs()
        out["dZ"] = order(g * k["y"] * dz, lens, reverse)
        g = g * sz
    Am = A.abs() if mag else A
    G = torch.zeros(b, c, n, dtype=X.dtype) if d_final is None else (d_final.abs() if mag else d_final.clone())
    dB, dC = torch.zeros(b, s, groups * n, dtype=X.dtype), torch.zeros(b, s, groups * n, dtype=X.dtype)
    dx, dd = torch.zeros_like(X), torch.zeros_like(X)
    dA = torch.zeros_like(A)
    for t in reversed(range(s)):
        live = k["live"][:, t].to(X.dtype)[:, None, None]
        a = torch.exp(d[:, t, :, None] * A)
        total = G + g[:, t, :, None] * k["Cg"][:, t] * live
        dC[:, t] = (g[:, t, :, None] * k["hs"][t + 1] * live).view(b, groups, c // groups, n).sum(2).reshape(b, -1)
        dB[:, t] = (total * (dm[:, t] * x[:, t])[..., None] * live).view(b, groups, c // groups, n).sum(2).reshape(b, -1)
        q = total * a * k["hs"][t] * live
        gb = (total * k["Bg"][:, t] * live).sum(-1)
        dd[:, t] = (q * Am).sum(-1) + x[:, t] * gb
        dx[:, t] = dm[:, t] * gb + k["D"] * g[:, t]
        dA = dA + (q * dm[:, t, :, None]).sum(0)
        G = torch.where(k["live"][:, t, None, None], total * a, G)
    if softplus:
        dd = dd * torch.sigmoid(k["raw"])
    zero = k["live"][..., None].to(X.dtype)
    dd, dx = dd * zero, dx * zero
    return out | {"dX": order(dx, lens, reverse), "ddelta": order(dd, lens, reverse), "dA": dA, "dB": order(dB, lens, reverse),
                  "dC": order(dC, lens, reverse), "dD": (g * x).sum((0, 1)), "ddelta_bias": dd.sum((0, 1)), "d_initial_state": G}


def norm(X, scale, shift=None, eps=1e-5):
    mean = X.mean(-1)
    inv = 1 / torch.sqrt(((X - mean[:, None]) ** 2).mean(-1) + eps)
    y = (X - mean[:, None]) * inv[:, None] * scale
    return (y if shift is None else y + shift), mean, inv


def norm_grad(X, scale, mean, inv, dY, mag=False):
    xh = (X - mean[:, None]) * inv[:, None]
    if mag:
        xh, dY, scale = (X.abs() + mean.abs()[:, None]) * inv[:, None], dY.abs(), scale.abs()
    g = dY * scale
    s = 1 if mag else -1
    dX = inv[:, None] * (g + s * g.mean(-1, keepdim=True) + s * xh * (g * xh).mean(-1, keepdim=True))
    return {"dX": dX, "dScale": (dY * xh).sum(0), "dB": dY.sum(0)}


def close(got, ref, mag, roundings, dtype, what):
    """|got - ref| within `roundings` f32 roundings of `mag`, and half a step of the type got is stored in.
    (Values below the type's normal range are stored to half its smallest step.)"""
    got, ref = got.detach().cpu().double(), ref.detach().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tiny = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}[dtype]
    room = roundings * 2.0 ** -24 * mag
    room = room + EPS[dtype] * (ref.abs() + room) + tiny
    off = (got - ref).abs()
    bad = ~(off <= room)
    assert not bad.any(), (what, "off by %.3g where %.3g is allowed" % (off[bad][0], room.expand_as(off)[bad][0]), int(bad.sum()), tuple(got.shape))
