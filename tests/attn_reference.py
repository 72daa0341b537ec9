"""Plain 64-bit form of linear attention with a decay for each head, step after
step as it is defined, its gradients' formulas, and how far arithmetic in 32
bits may take each output.

Sequence tensors are float64 [batch, seq, n]; `walk` takes them in the order of
a row's steps and with the heads as a dimension of their own."""
import torch

from tests import ssm_reference as ref

U = 2.0 ** -24
TINY = 2.0 ** -100      # what is lost below f32's normal range


def heads_of(t, heads, per):
    """[batch, seq, groups * n] -> [batch, seq, heads, n]."""
    b, s, w = t.shape
    return t.view(b, s, heads // per, w // (heads // per)).repeat_interleave(per, 2)


def log_decays(G, decay, b, s, h, like):
    g = torch.zeros(b, s, h, dtype=like.dtype, device=like.device)
    g = g if G is None else g + G
    g = g if decay is None else g + decay
    return torch.where(g > 0, torch.zeros_like(g), g)


def walk(a, b, v, g, init, live, back=False, in_scale=1.0, out_scale=1.0, split=0.0):
    """S = e^g S + in_scale b v^T, out = out_scale a^T S, over the live steps; `back`: from the last, where the decay
    between two steps is the later one's.  {out, off, end}, off being out less the step's own v, and the same names
    with a capital: bounds of what 32-bit arithmetic may be off by.  A state's term takes at each step that it ages
    a product by a decay (its argument's rounding |g| u, its own 2 u) and a sum: 3 + 2 |g| of them (a chunk of steps
    takes one decay for many, no more than these); it enters through at most 70 others (scale, decay, sums over a
    chunk), and an output's sum over the state, or over the chunk's steps of sums over the keys, has n + 80.  `split`:
    what products by factors in halves leave, relative."""
    n, s, h, k = a.shape
    S = init.clone()
    M, N = S.abs(), torch.zeros_like(S)
    out = {name: torch.zeros(n, s, h, v.shape[-1], dtype=a.dtype, device=a.device) for name in ("out", "off", "Out", "Off")}
    depth = (k + 80) * U + split
    for i in (reversed(range(s)) if back else range(s)):
        on = live[:, i, None, None, None]
        gi = g[:, i] if not back else (torch.where(live[:, i + 1, None], g[:, i + 1], torch.zeros_like(g[:, i])) if i + 1 < s else torch.zeros_like(g[:, i]))
        dec = torch.exp(gi)[..., None, None]
        age = (3 + 2 * gi.abs().clamp(max=200))[..., None, None]
        new = in_scale * b[:, i, :, :, None] * v[:, i, :, None, :]
        S0, N0, M0 = dec * S, dec * (N + age * M), dec * M
        qa = out_scale * a[:, i, :, :, None]
        out["off"][:, i] = ((qa * S0).sum(-2) * on[..., 0])
        out["Off"][:, i] = (qa.abs() * (U * (N0 + 70 * M0) + depth * M0)).sum(-2) * on[..., 0]
        S = torch.where(on, S0 + new, S)
        N, M = torch.where(on, N0, N), torch.where(on, M0 + new.abs(), M)
        out["out"][:, i] = (qa * S).sum(-2) * on[..., 0]
        out["Out"][:, i] = (qa.abs() * (U * (N + 70 * M) + depth * M)).sum(-2) * on[..., 0]
    out["end"], out["End"] = S, U * (N + 70 * M)
    out["Mag"] = M
    return out


def attn(Q, K, V, heads, groups, G=None, decay=None, scale=1.0, lens=None, init=None, reverse=False, dY=None, d_final=None, split=0.0,
         fine=2.0 ** -22):
    """{name: (value, bound)} of Y and final_state, and with dY of every gradient.  `split`, `fine`: what products by
    factors in halves leave of outputs, and of those that the decays' gradient is made from."""
    b, s, _ = Q.shape
    per = heads // groups
    lens = ref.lengths(lens, b, s)
    live = (torch.arange(s)[None] < torch.tensor(lens).view(b, 1)).to(Q.device)
    g = ref.order(log_decays(G, decay, b, s, heads, Q), lens, reverse)
    q, k, v = (heads_of(ref.order(t, lens, reverse), heads, n) for t, n in ((Q, per), (K, per), (V, 1)))
    zero = torch.zeros(b, heads, k.shape[-1], v.shape[-1], dtype=Q.dtype, device=Q.device)
    first = zero if init is None else init

    def rows(t, of=1):
        return ref.order(t.view(b, s, heads // of, of, -1).sum(3).flatten(2), lens, reverse)

    if dY is None:
        w = walk(q, k, v, g, first, live, out_scale=scale, split=split)
        return {"Y": (rows(w["out"]), rows(w["Out"])), "final_state": (w["end"], w["End"])}
    dy = heads_of(ref.order(dY, lens, reverse), heads, 1)
    last = zero if d_final is None else d_final
    turn = lambda t: t.transpose(-1, -2)  # noqa: E731
    wq = walk(dy, v, k, g, turn(first), live, out_scale=scale, split=split)
    wk = walk(v, dy, q, g, turn(last), live, back=True, in_scale=scale, split=split)
    wv = walk(k, q, dy, g, last, live, back=True, in_scale=scale, split=split)
    fold = per * U      # the sum over a group's heads
    out = {"dQ": (rows(wq["out"], per), rows(wq["Out"] + fold * wq["out"].abs(), per)),
           "dK": (rows(wk["out"], per), rows(wk["Out"] + fold * wk["out"].abs(), per)), "dV": (rows(wv["out"]), rows(wv["Out"]))}
    r, c = (q * wq["off"]).sum(-1), (k * wk["off"]).sum(-1)
    # (the walks' own splits are finer there)
    R = (q.abs() * (wq["Off"] + (fine - split) * _mag(dy, v, k, g, turn(first), live, out_scale=scale)
                    + (key_depth(q) * U) * wq["off"].abs())).sum(-1)
    C = (k.abs() * (wk["Off"] + (fine - split) * _mag(v, dy, q, g, turn(last), live, back=True, in_scale=scale)
                    + (key_depth(q) * U) * wk["off"].abs())).sum(-1)
    ends, Ends = (wq["end"] * turn(last)).sum((-1, -2)), ((wq["End"] + 300 * U * wq["Mag"]) * turn(last).abs()).sum((-1, -2))
    x = (r - c).flip(1).cumsum(1).flip(1) + ends[:, None]
    X = (R + C).flip(1).cumsum(1).flip(1) + Ends[:, None] + U * x.abs()
    x, X = x * live[..., None], X * live[..., None]
    at = ref.order((G if G is not None else 0) + (decay if decay is not None else 0) + torch.zeros(b, s, heads, dtype=Q.dtype, device=Q.device),
                   lens, reverse)
    x = torch.where(at > 0, torch.zeros_like(x), x)
    out["dG"] = ref.order(x, lens, reverse), ref.order(X, lens, reverse)
    out["d_decay"] = x.sum((0, 1)), X.sum((0, 1)) + (b * (s // 64 + 2) + 8) * U * x.abs().sum((0, 1))
    some = (live[:, :1] if s else torch.zeros(b, 1, dtype=torch.bool, device=Q.device))[..., None, None]
    dec = torch.where(some, torch.exp(g[:, :1].sum(1))[..., None, None], torch.ones_like(zero[..., :1, :1]))
    age = (4 + 2 * g[:, :1].sum(1).abs().clamp(max=200))[..., None, None]
    out["d_initial_state"] = wv["end"] * dec, dec * (wv["End"] + age * U * wv["end"].abs())
    return out


def key_depth(q):
    return q.shape[-1] + 10


def _mag(a, b, v, *rest, **kw):
    """The sum of the magnitudes of an off output's terms."""
    kw = {n: abs(x) if n.endswith("scale") else x for n, x in kw.items()}
    g, init, live = rest
    return walk(a.abs(), b.abs(), v.abs(), g, init.abs(), live, **kw)["off"]


def close(got, want, bound, dtype, what):
    """|got - want| within the bound and half a step of the type got is stored in."""
    got, want, bound = got.detach().cpu().double(), want.detach().cpu().double(), bound.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tiny = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}[dtype] + TINY
    eps = 0.0 if dtype == "f32" else ref.EPS[dtype]
    room = 1.05 * bound + eps * (want.abs() + bound) + tiny
    off = (got - want).abs()
    bad = ~(off <= room)
    assert not bad.any(), (what, "%g where %g is right, off by %.3g, %.3g allowed" % (
        got[bad][0], want[bad][0], off[bad][0], room[bad][0]), int(bad.sum()), tuple(got.shape), "worst %.2f of the bound" % float((off / room).nan_to_num(99).max()))
    return float((off / room).max()) if off.numel() else 0.0
