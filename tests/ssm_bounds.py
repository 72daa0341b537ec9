"""How far f32 arithmetic may take the scan's and layer normalization's outputs
from their 64-bit values, term by term along the computation (tests/ssm_reference.py
bounds magnitudes alone, which for long rows and rows far from zero is loose).

u = 2^-24 is half a step.  What an operation adds, relative to its result: a
sum, product or fused multiply-add u; the hardware's 2^x and reciprocal one
unit in the last place, 2 u, and 2^x's argument, itself a rounded product by a
rounded constant, its own error times ln 2.  Errors already there go on as the
operation's derivative has them.  Products of errors are covered by SLACK."""
import torch

from tests import ssm_reference as ref

U = 2.0 ** -24
SLACK = 1.05
TINY = 2.0 ** -110     # results of 2^x below the normal range are zero


def scan_bounds(X, delta, A, B, C, D=None, Z=None, delta_bias=None, lens=None, initial_state=None, dY=None, d_final=None,
                groups=1, softplus=True, reverse=False, chunk=1 << 30):
    """Bounds of Y, final_state and, with dY, of every gradient, before their rounding to a narrower type.
    `chunk`: steps of a chunk of the time axis."""
    b, s, c = X.shape
    n = A.shape[1]
    _, _, k = ref.scan(X, delta, A, B, C, D, Z, delta_bias, lens, initial_state, groups, softplus, reverse, keep=True)
    x, raw, d, Bg, Cg, hs, y, live = (k[i] for i in ("x", "raw", "d", "Bg", "Cg", "hs", "y", "live"))
    lens, Dk, Zk = k["lens"], k["D"], k["Z"]
    # the step size: softplus is taken of a rounded sum (derivative x sigma / softplus <= 1 + |x|), its 2^x has
    # 1.5 |x| of the argument, and a dozen operations follow
    rd = (17 + 2.5 * raw.abs()) * U if softplus else torch.full_like(raw, U)
    aA = A.abs()

    def rel_decay(t):      # of 2^(d A'), A' = A log2 e rounded twice
        return (d[:, t].abs() * (rd[:, t] + 3 * U))[..., None] * aA + 4 * U

    def far(at, steps_abs):   # the same of 2^(A' sum of step sizes), a sum of up to `chunk` of them
        return (steps_abs * (rd.amax(1) + (min(chunk, s) + 3) * U))[..., None] * aA + 8 * U

    zero = torch.zeros(b, c, n, dtype=torch.float64)
    E, h_start, E_start = zero, hs[0], zero
    hl, El, cum, cum_abs = hs[0], zero, torch.zeros(b, c, dtype=torch.float64), torch.zeros(b, c, dtype=torch.float64)
    Eb = zero                 # of a state that the gradient starts from any segment on
    Ehs, Ebs, Ey, ends = [zero], [zero], [], []
    for t in range(s):
        on = live[:, t, None, None]
        if t and t % chunk == 0:
            P = torch.exp(A * cum[..., None])
            if t == chunk:
                joined = El
            else:
                joined = P * E_start + P * h_start.abs() * far(t, cum_abs) + El + U * hs[t].abs()
            ends.append((P, cum_abs))
            h_start, E_start = hs[t], joined
            E = torch.where(on, joined, E)
            Eb = torch.where(on, joined, Eb)
            Ehs[-1], Ebs[-1] = torch.maximum(Ehs[-1], E), torch.maximum(Ebs[-1], Eb)
            hl, El, cum, cum_abs = zero, zero, torch.zeros_like(cum), torch.zeros_like(cum)
        a, ra = torch.exp(d[:, t, :, None] * A), rel_decay(t)
        inp = (d[:, t] * x[:, t])[..., None] * Bg[:, t]
        new = inp.abs() * (rd[:, t, :, None] + 3 * U)
        E = torch.where(on, a * E + a * hs[t].abs() * ra + new + U * hs[t + 1].abs(), E)
        nl = a * hl + inp
        El = torch.where(on, a * El + a * hl.abs() * ra + new + U * nl.abs(), El)
        hl = torch.where(on, nl, hl)
        cum, cum_abs = (torch.where(on[..., 0], v + w, v) for v, w in ((cum, d[:, t]), (cum_abs, d[:, t].abs())))
        direct = El
        if t >= chunk:
            P = torch.exp(A * cum[..., None])
            direct = El + P * E_start + P * h_start.abs() * far(t, cum_abs) + U * hs[t + 1].abs()
        step = a * Eb + a * hs[t].abs() * ra + new + U * hs[t + 1].abs()
        Eb = torch.where(on, torch.maximum(direct, step), Eb)
        Ehs.append(E)
        Ebs.append(Eb)
        Ey.append((Cg[:, t].abs() * E).sum(-1) + (n + 12) * U * ((Cg[:, t] * hs[t + 1]).abs().sum(-1) + (Dk * x[:, t]).abs()))
    ends.append((torch.exp(A * cum[..., None]), cum_abs))
    Ey = torch.stack(Ey, 1) if s else torch.zeros_like(X)
    out = {"final_state": E}
    Eo = Ey
    rg = torch.zeros_like(X)
    if Zk is not None:
        rg = (1.5 * Zk.abs() + 8) * U
        Eo = Ey * ref.silu(Zk).abs() + (y * ref.silu(Zk)).abs() * (rg + U)
    out["Y"] = ref.order(Eo, lens, reverse)
    if dY is not None:
        g = ref.order(dY, lens, reverse)
        out |= _scan_grad_bounds(A, g, Zk, Cg, Bg, Dk, hs, Ebs, x, d, raw, y, live, lens, rd, rg, rel_decay, far, ends, chunk, d_final,
                                 groups, softplus, reverse)
    return {name: SLACK * t + TINY for name, t in out.items()}


def _scan_grad_bounds(A, g, Z, Cg, Bg, D, hs, Ebs, x, d, raw, y, live, lens, rd, rg, rel_decay, far, ends, chunk, d_final, groups,
                      softplus, reverse):
    b, s, c = x.shape
    n, aA = A.shape[1], A.abs()
    out = {}
    depth_y = (n + 12) * U
    if Z is not None:
        sg, dz = torch.sigmoid(Z), ref.dsilu(Z)
        e_dz = dz.abs() * (1.5 * Z.abs() + 10) * U + sg * (Z.abs() * (sg * (1.5 * Z.abs() + 5) + 2) + 2) * U
        Eyb = [(Cg[:, t].abs() * Ebs[t + 1]).sum(-1) + depth_y * ((Cg[:, t] * hs[t + 1]).abs().sum(-1) + (D * x[:, t]).abs())
               for t in range(s)]
        Eyb = torch.stack(Eyb, 1) if s else torch.zeros_like(x)
        out["dZ"] = ref.order((g * dz).abs() * Eyb + (g * y).abs() * e_dz, lens, reverse)
        g = g * ref.silu(Z)
    zero = torch.zeros(b, c, n, dtype=torch.float64)
    # the gradient at each chunk's start from a zero one at its end, as it is summed forward
    locs = []
    for first in range(0, s, chunk):
        Q, rq, mag, err = torch.ones_like(zero), zero, zero, zero
        for t in range(first, min(first + chunk, s)):
            on = live[:, t, None, None]
            Q, rq = torch.where(on, Q * torch.exp(d[:, t, :, None] * A), Q), torch.where(on, rq + rel_decay(t) + U, rq)
            term = torch.where(on, (Q * Cg[:, t] * g[:, t, :, None]).abs(), zero)
            mag, err = mag + term, err + term * (rq + rg[:, t, :, None] + 2 * U)
        locs.append(err + min(chunk, s) * U * mag)
    G = zero if d_final is None else d_final
    EG, G_end, E_end = zero, G, zero
    dB, dC = torch.zeros(b, s, groups * n, dtype=torch.float64), torch.zeros(b, s, groups * n, dtype=torch.float64)
    dx, dd = torch.zeros_like(x), torch.zeros_like(x)
    dA, magA = torch.zeros_like(A), torch.zeros_like(A)
    dD, magD = torch.zeros(c, dtype=torch.float64), torch.zeros(c, dtype=torch.float64)
    magb = torch.zeros_like(magD)
    fold = (6 + -(-(c // groups) // 64) + 2) * U

    def of_groups(t):
        return t.view(b, groups, c // groups, n).sum(2).reshape(b, -1)

    for t in reversed(range(s)):
        on = live[:, t, None, None]
        one = on.double()
        if (t + 1) % chunk == 0 and t + 1 < s:
            later = live[:, t + 1, None, None]     # the chunk after this one has steps
            j = (t + 1) // chunk
            P, steps_abs = ends[j]
            joined = P * E_end + P * G_end.abs() * far(t, steps_abs) + locs[j] + U * G.abs()
            EG = torch.where(later, joined, EG)
            G_end, E_end = torch.where(later, G, G_end), torch.where(later, EG, E_end)
        a, ra = torch.exp(d[:, t, :, None] * A), rel_decay(t)
        term = g[:, t, :, None] * Cg[:, t]
        tot = G + term * one
        Et = EG + (term.abs() * rg[:, t, :, None] + U * tot.abs()) * one
        u = (d[:, t] * x[:, t])[..., None]
        gy = g[:, t, :, None]
        dB[:, t] = of_groups((Et * u.abs() + (tot * u).abs() * (rd[:, t, :, None] + 3 * U)) * one) + fold * of_groups((tot * u).abs() * one)
        dC[:, t] = of_groups((gy.abs() * Ebs[t + 1] + (gy * hs[t + 1]).abs() * (rg[:, t, :, None] + U)) * one) \
            + fold * of_groups((gy * hs[t + 1]).abs() * one)
        sb = (tot * Bg[:, t]).sum(-1)
        Esb = (Et * Bg[:, t].abs()).sum(-1) + depth_y * (tot * Bg[:, t]).abs().sum(-1)
        Ga = tot * a
        EGa = a * Et + Ga.abs() * (ra + U)
        q = Ga * hs[t]
        Eq = EGa * hs[t].abs() + Ga.abs() * Ebs[t] + U * q.abs()
        sq = (q * A).sum(-1)
        Esq = (Eq * aA).sum(-1) + (depth_y + 6 * U) * (q * A).abs().sum(-1)
        dr = x[:, t] * sb + sq
        Edr = x[:, t].abs() * Esb + Esq + U * dr.abs()
        if softplus:
            sig = torch.sigmoid(raw[:, t])
            Edr = Edr * sig + (dr * sig).abs() * (2.5 * raw[:, t].abs() + 8) * U
            dr = dr * sig
        row = one[..., 0]
        dx[:, t] = (d[:, t].abs() * Esb + (d[:, t] * sb).abs() * rd[:, t] + (D * g[:, t]).abs() * (rg[:, t] + U)
                    + U * (d[:, t] * sb + D * g[:, t]).abs()) * row
        dd[:, t] = Edr * row
        magb = magb + (dr.abs() * row).sum(0)
        dA = dA + ((Eq * d[:, t, :, None].abs() + (q * d[:, t, :, None]).abs() * (rd[:, t, :, None] + U)) * one).sum(0)
        magA = magA + ((q * d[:, t, :, None]).abs() * one).sum(0)
        gx = (g[:, t] * x[:, t]).abs() * row
        dD, magD = dD + (gx * rg[:, t]).sum(0), magD + gx.sum(0)
        EG = torch.where(on, EGa, EG)
        G = torch.where(on, Ga, G)
    long = (min(chunk, max(s, 1)) + b * (-(-s // chunk)) + 8) * U      # a sum's longest way
    return out | {"dX": ref.order(dx, lens, reverse), "ddelta": ref.order(dd, lens, reverse), "dB": ref.order(dB, lens, reverse),
                  "dC": ref.order(dC, lens, reverse), "dA": dA + long * magA, "dD": dD + long * magD,
                  "ddelta_bias": dd.sum((0, 1)) + long * magb, "d_initial_state": EG}


def norm_bounds(X, scale, shift, eps=1e-5):
    """Bounds of Y, Mean and InvStdDev before their rounding to a narrower type."""
    size = X.shape[-1]
    y, mean, inv = ref.norm(X, scale, shift, eps)
    depth = sum_depth(size)
    d = X - mean[:, None]
    var = d.square().mean(-1)
    dm = (depth + 2) * U * X.abs().mean(-1)            # of Mean: a sum, 1 / size, a product
    # squares are taken of x - Mean', whose sum over a row is off by that of Mean alone: the cross term vanishes
    dvar = (depth + 3) * U * (var + dm ** 2) + dm ** 2 + 2 * U * (var + dm * d.abs().mean(-1))
    rel = 0.5 * dvar * inv ** 2 + 4 * U                # a fused multiply-add, a root, a quotient
    dd = dm[:, None] + U * (d.abs() + dm[:, None])
    Y = scale.abs() * inv[:, None] * (dd + d.abs() * (rel[:, None] + 2 * U)) + U * y.abs()
    return {"Y": SLACK * Y + TINY, "Mean": SLACK * dm + TINY, "InvStdDev": SLACK * rel * inv + TINY}


def sum_depth(size):
    """Additions one after another in a row's sum, at most: a thread's values (up to 32 in registers, else a 256th of
    the row), a wave's six, four waves."""
    return max(32, size // 256 + 8) + 6 + 4


def norm_grad_bounds(X, scale, mean, inv, dY, rows_deep):
    """The same of dX, dScale and dB.  `rows_deep`: additions one after another in a sum over rows, at most."""
    size = X.shape[-1]
    n = (sum_depth(size) + 2) * U
    xh = (X - mean[:, None]) * inv[:, None]            # off by 2 u: a difference and a product
    g = dY * scale
    m0, m1 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    e0 = (n + U) * g.abs().mean(-1, keepdim=True)
    e1 = (n + 4 * U) * (g * xh).abs().mean(-1, keepdim=True)
    sub = m0 + xh * m1
    esub = e0 + xh.abs() * e1 + (xh * m1).abs() * 2 * U + U * sub.abs()
    dX = inv[:, None] * (esub + U * g.abs() + 2 * U * (g - sub).abs())
    return {"dX": SLACK * dX + TINY, "dScale": SLACK * (rows_deep + 3) * U * (dY * xh).abs().sum(0) + TINY,
            "dB": SLACK * rows_deep * U * dY.abs().sum(0) + TINY}


def check(got, want, bound, dtype, what):
    """|got - want| within the bound and half a step of the type got is stored in.  Where the 64-bit value is infinite got
    is that; where it is not a number got may be anything."""
    got, want = got.detach().cpu().double(), want.detach().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tiny = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}[dtype]
    eps = 0.0 if dtype == "f32" else ref.EPS[dtype]
    room = bound + eps * (want.abs() + bound) + tiny
    off = (got - want).abs()
    bad = torch.where(want.isfinite(), ~(off <= room), torch.where(want.isnan(), torch.zeros_like(off, dtype=torch.bool), got != want))
    assert not bad.any(), (what, "%g where %g is right, off by %.3g, %.3g allowed" % (
        got[bad][0], want[bad][0], off[bad][0], room.expand_as(off)[bad][0]), int(bad.sum()), tuple(got.shape))
