"""The operators of a linear attention block, as measured: linear attention with a decay for each head, and the norm of queries and
keys for each head with the position rotation; forward, backward and for single tokens.

`own = False` computes them from elementary torch operations in 32 bits; `own = True` calls this framework."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 64  # steps that the plain form takes together


def _attn(name, mode, dtype, batch, seq, heads, groups, key, value, gate=True, reverse=False, layout=1, ragged=False, carried=True):
    return dict(name=name, op="attn", mode=mode, dtype=dtype, batch=batch, seq=seq, heads=heads, groups=groups, key=key, value=value,
                gate=gate, reverse=reverse, layout=layout, ragged=ragged, carried=carried)


def _rotary(name, mode, dtype, rows, q_heads, k_heads, size, rotary, interleaved=False, table=4096):
    return dict(name=name, op="rotary", mode=mode, dtype=dtype, rows=rows, q_heads=q_heads, k_heads=k_heads, size=size, rotary=rotary,
                interleaved=interleaved, table=table)


def listed():
    return [
        # one token of one request on a small model: nothing but latency
        _attn("attn_token_one_f16", "forward", "f16", 1, 1, 8, 8, 64, 64, gate=False),
        # one token of each of 64 running requests: the state is read and written
        _attn("attn_tokens_bf16", "forward", "bf16", 64, 1, 16, 16, 128, 128),
        # a batch of prompts of unequal length, following an earlier piece of each text
        _attn("attn_prompts_bf16", "forward", "bf16", 8, 1024, 16, 16, 128, 128, ragged=True),
        # one long prompt, alone on the GPU, a fixed decay for each head: little work side by side
        _attn("attn_long_prompt_f16", "forward", "f16", 1, 4096, 16, 16, 128, 128, gate=False),
        # the matrix-valued form of a state space block: queries and keys shared by all heads
        _attn("attn_shared_bf16", "forward", "bf16", 4, 2048, 32, 1, 128, 64),
        # the reverse half of a two-way layer, time first, with sizes that fill no tile
        _attn("attn_reverse_f32", "forward", "f32", 3, 257, 6, 2, 50, 42, reverse=True, layout=0, ragged=True),
        # a training step
        _attn("attn_grad_bf16", "backward", "bf16", 8, 1024, 16, 16, 128, 128, carried=False),
        # a small two-way tagger's training step: short sentences of unequal length
        _attn("attn_grad_small_f32", "backward", "f32", 5, 80, 4, 2, 24, 30, reverse=True, layout=0, ragged=True),
        # queries and keys of one token of each of 64 requests: latency
        _rotary("rotary_tokens_bf16", "forward", "bf16", 64, 16, 16, 128, 128),
        # the same for a batch of prompts
        _rotary("rotary_prompts_f16", "forward", "f16", 8192, 16, 16, 128, 128),
        # a training step's, the weights' gradients among it
        _rotary("rotary_grad_bf16", "backward", "bf16", 8192, 16, 16, 128, 128),
        # part of each head rotated, pairs side by side, few key heads, sizes that fill no tile
        _rotary("rotary_partial_f32", "forward", "f32", 771, 6, 2, 50, 26, interleaved=True),
    ]


def draw(rng):
    def size(lo, hi):
        return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))

    dtype, mode = rng.choice(["f32", "f16", "bf16"]), rng.choice(["forward", "forward", "backward"])
    if rng.random() < 0.35:
        width = rng.choice([16, 50, 64, 64, 96, 128, 128, 128, 256, size(2, 256)])
        q_heads = size(1, 32)
        k_heads = rng.choice([q_heads, max(1, q_heads // 4), 1])
        rows = size(1, max(1, min(16384, (1 << 25) // ((q_heads + k_heads) * width))))
        rotary = rng.choice([width // 2 * 2, width // 2 * 2, width // 4 * 2])
        case = _rotary("", mode, dtype, rows, q_heads, k_heads, width, rotary, rng.random() < 0.4, rng.choice([512, 4096, 32768]))
    else:
        dims = [16, 32, 50, 64, 64, 64, 96, 128, 128, 128, 256, size(1, 256)]
        key, value = rng.choice(dims), rng.choice(dims)
        heads = size(1, 32)
        groups = rng.choice([heads, heads, heads, 1] + [g for g in range(1, heads + 1) if heads % g == 0])
        batch = size(1, 64)
        seq = 1 if mode == "forward" and rng.random() < 0.3 else size(2, 4096)
        if seq == 1:
            batch = max(1, min(batch, (1 << 24) // (heads * key * value)))
        else:
            most = (1 << 23) // (heads * (key + value))
            batch = max(1, min(batch, most // 64))
            seq = max(2, min(seq, most // batch))
        case = _attn("", mode, dtype, batch, seq, heads, groups, key, value, rng.random() < 0.6, rng.random() < 0.3, rng.choice([0, 1, 1]),
                     rng.random() < 0.5, rng.random() < 0.5)
    del case["name"]
    return case


def _lens(case):
    """Lengths from a quarter of the longest to the longest, in no order; None where all are equal."""
    if not case.get("ragged"):
        return None
    n, s = case["batch"], case["seq"]
    return [s - (3 * s // 4) * ((5 * b) % n) // max(1, n - 1) if n > 1 else s for b in range(n)]


def _positions(case):
    lens = _lens(case)
    return case["batch"] * case["seq"] if lens is None else sum(lens)


def work(case):
    e, back = BYTES[case["dtype"]], case["mode"] == "backward"
    if case["op"] == "rotary":
        n, c, r = case["rows"], (case["q_heads"] + case["k_heads"]) * case["size"], case["rotary"]
        table = 4 * r * min(n, case["table"]) + 4 * n
        if back:
            return {"bytes": 3 * e * n * c + table + (4 + e) * 2 * case["size"], "flops": 17 * n * c}
        return {"bytes": 2 * e * n * c + table + e * 2 * case["size"], "flops": 9 * n * c}
    b, h, g, k, v, live = case["batch"], case["heads"], case["groups"], case["key"], case["value"], _positions(case)
    rows = b * case["seq"]  # outputs are written past a row's length too (zeros)
    state = 4 * b * h * k * v
    own_decay = 4 * h * (live if case["gate"] else 1)
    # a position and head: the state's update and its product with the query, or both within a chunk of c steps, where that is less
    form = min(4 * k * v, min(case["seq"], CHUNK) * (k + v) + 4 * k * v * (case["carried"] or case["seq"] > CHUNK))
    if back:
        decay = own_decay + 4 * h * (rows if case["gate"] else 1)
        moved = e * live * (2 * g * k + 2 * h * v) + e * rows * (2 * g * k + h * v)
        return {"bytes": moved + decay + 3 * state * case["carried"], "flops": 3 * live * h * form}
    return {"bytes": e * live * (2 * g * k + h * v) + e * rows * h * v + own_decay + state * (1 + case["carried"]), "flops": live * h * form}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, f32 = DTYPES[case["dtype"]], torch.float32

    def normal(*shape, to=dt, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(to)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def empty(*shape, to=dt):
        return torch.empty(*shape, dtype=to, device="cuda")

    back = case["mode"] == "backward"
    if case["op"] == "rotary":
        n, d, r = case["rows"], case["size"], case["rotary"]
        q, k = case["q_heads"] * d, case["k_heads"] * d
        both = normal(n, q + k, by=1.5)  # the projection's two parts
        turn = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(r // 2, device="cuda", dtype=torch.float64) * 2 / max(1, r))
        t = {"Q": both[:, :q], "K": both[:, q:], "q_scale": (1 + normal(d, to=f32, by=0.2)).to(dt), "k_scale": (1 + normal(d, to=f32, by=0.2)).to(dt),
             "cos": torch.cos(turn).float(), "sin": torch.sin(turn).float(),
             "positions": torch.randint(case["table"], (n,), generator=gen, device="cuda", dtype=torch.int32)}
        if back:
            t |= {"dQ_out": normal(n, q), "dK_out": normal(n, k)}
            out = {"dQ": empty(n, q), "dK": empty(n, k), "dq_scale": empty(d, to=f32), "dk_scale": empty(d, to=f32)}
        else:
            out = {"Q_out": empty(n, q), "K_out": empty(n, k)}
        state = {"case": case, "in": t, "out": out}
        if own:
            import onnx_recurrent_layers_amd as rl
            state["op"] = rl.RotaryNorm(dtype=case["dtype"], rows=n, q_heads=case["q_heads"], k_heads=case["k_heads"], size=d, rotary=r,
                                        table=case["table"], interleaved=case["interleaved"], epsilon=1e-6)
        return state

    b, s, h, g, k, v = (case[n] for n in ("batch", "seq", "heads", "groups", "key", "value"))
    lead = (s, b) if case["layout"] == 0 else (b, s)
    rows = normal(*lead, 2 * g * k + h * v)  # the projection's three parts
    t = {"Q": rows[..., :g * k], "K": rows[..., g * k:2 * g * k], "V": rows[..., 2 * g * k:]}
    if case["gate"]:  # steps that forget between a thousandth and a third, a head by its own measure
        t["G"] = -torch.exp(uniform(math.log(0.003), math.log(0.1), h)) * torch.exp(normal(*lead, h, to=f32, by=0.5))
    else:
        t["decay"] = torch.log1p(-torch.exp2(-5 - 4 * torch.arange(h, device="cuda") / max(1, h - 1)))
    lens = _lens(case)
    if lens is not None:
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["carried"]:
        t["initial_state"] = normal(b, h, k, v, to=f32, by=3.0)
    if back:
        t["dY"] = normal(*lead, h * v)
        out = {"dQ": empty(*lead, g * k), "dK": empty(*lead, g * k), "dV": empty(*lead, h * v)}
        out |= {"dG": empty(*lead, h, to=f32)} if case["gate"] else {"d_decay": empty(h, to=f32)}
        if case["carried"]:
            t["d_final_state"] = normal(b, h, k, v, to=f32, by=0.1)
            out["d_initial_state"] = empty(b, h, k, v, to=f32)
    else:
        out = {"Y": empty(*lead, h * v), "final_state": empty(b, h, k, v, to=f32)}
    state = {"case": case, "in": t, "out": out}
    if own:
        import onnx_recurrent_layers_amd as rl
        state["op"] = rl.LinearAttention(dtype=case["dtype"], seq=s, batch=b, heads=h, groups=g, key=k, value=v, scale=k ** -0.5,
                                         direction="reverse" if case["reverse"] else "forward", layout=case["layout"])
    return state


def run(state):
    case, t = state["case"], state["in"]
    if own:
        getattr(state["op"], "backward" if case["mode"] == "backward" else "encode")({**t, **state["out"]})
        return state["out"]
    return {"attn": _plain_attn, "rotary": _plain_rotary}[case["op"]](case, t)


# ---- the plain forms: 32 bits, rounded once at the end

def _order(case, t):
    """Which steps a row takes, and the time of each, as [batch, seq]; None where every row takes every step in its own order."""
    s = torch.arange(case["seq"], device="cuda")
    if "sequence_lens" in t:
        n = t["sequence_lens"].long()[:, None]
    elif case["reverse"]:
        n = torch.full((case["batch"], 1), case["seq"], device="cuda")
    else:
        return None, None
    live = s < n
    return live, torch.where(live, n - 1 - s, s) if case["reverse"] else None


def _steps(case, x, live, at):
    """A tensor of rows as [batch, steps, ...] in 32 bits, zero past a row's length."""
    x = x.float()
    x = x.transpose(0, 1) if case["layout"] == 0 else x
    if at is not None:
        x = x.gather(1, at[..., None].expand(-1, -1, x.shape[-1]))
    return x if live is None else x.masked_fill(~live[..., None], 0.0)


def _rows(case, x, live, at, to):
    """The way back, rounded to the tensors' type."""
    x = _steps(dict(case, layout=1), x, live, None)
    if at is not None:
        x = x.gather(1, at[..., None].expand(-1, -1, x.shape[-1]))
    return (x.transpose(0, 1) if case["layout"] == 0 else x).to(to).contiguous()


def _apply(a, b, v, first, within, since, left, between):
    """Linear attention over chunks, [batch, heads, chunks, steps, size]: outputs, and the state after the last step. `within`: the decay
    from step j to i of a chunk (zero for j > i), `since`: from a chunk's start to after a step, `left`: from after a step to a chunk's
    end, `between`: from after chunk m to before chunk n."""
    local = (b * left[..., None]).transpose(-1, -2) @ v  # what a chunk adds to the state
    shape = local.shape
    flat = torch.cat([first[:, :, None], local], 2).flatten(3)  # the first state stands for a chunk before all
    starts = (between @ flat).view(shape[0], shape[1], -1, *shape[3:])
    y = ((a @ b.transpose(-1, -2)) * within) @ v + (a * since[..., None]) @ starts[:, :, :-1]
    return y, starts[:, :, -1]


def _decays(g):
    """The decays that _apply takes, from log decays [batch, heads, chunks, steps]; differences of sums in 64 bits."""
    n, c = g.shape[2], g.shape[3]
    d = g.double()
    sums = d.cumsum(-1)
    lower = torch.ones(c, c, dtype=torch.bool, device="cuda").tril()
    within = torch.exp((sums[..., :, None] - sums[..., None, :]).masked_fill(~lower, -math.inf).float())
    ends = torch.cat([torch.zeros_like(d[:, :, :1, 0]), sums[..., -1].cumsum(2)], 2)  # after the first state, after chunk 0, ...
    lower = torch.ones(n + 1, n + 1, dtype=torch.bool, device="cuda").tril()
    between = torch.exp((ends[..., :, None] - ends[..., None, :]).masked_fill(~lower, -math.inf).float())
    return within, torch.exp(sums.float()), torch.exp((sums[..., -1:] - sums).float()), between


def _chunks(case, x, heads):
    """[batch, steps, heads * size] -> [batch, all heads, chunks, steps, size], groups repeated for their heads."""
    b, s, _ = x.shape
    c = min(CHUNK, s)
    x = torch.nn.functional.pad(x, (0, 0, 0, -s % c))
    x = x.view(b, -1, c, heads, x.shape[-1] // heads).permute(0, 3, 1, 2, 4)
    return x.repeat_interleave(case["heads"] // heads, 1) if heads < case["heads"] else x


def _flat(case, x, heads):
    """The way back, heads of a group summed."""
    b, h, n, c, d = x.shape
    x = x.view(b, heads, h // heads, n, c, d).sum(2).permute(0, 2, 3, 1, 4).reshape(b, n * c, heads * d)
    return x[:, :case["seq"]]


def _plain_attn(case, t):
    b, s, h, g, k, v = (case[n] for n in ("batch", "seq", "heads", "groups", "key", "value"))
    dt, scale = DTYPES[case["dtype"]], k ** -0.5
    live, at = _order(case, t)
    q, kk, vv = (_chunks(case, _steps(case, t[n], live, at), m) for n, m in (("Q", g), ("K", g), ("V", h)))
    if "G" in t:
        log = _steps(case, t["G"], live, at)
    else:
        log = t["decay"].expand(b, s, h)
        log = log if live is None else log.masked_fill(~live[..., None], 0.0)
    zero = q.new_zeros(b, h, k, v)
    first = t["initial_state"] if "initial_state" in t else zero
    decays = _decays(_chunks(case, log, h)[..., 0])
    if case["mode"] == "forward":
        y, last = _apply(q * scale, kk, vv, first, *decays)
        return {"Y": _rows(case, _flat(case, y, h), live, at, dt), "final_state": last.contiguous()}
    dy = _chunks(case, _steps(case, t["dY"], live, at), h)
    dlast = t["d_final_state"] if "d_final_state" in t else zero
    # the same operator with the roles changed: forward in time for dQ, back for dK and dV, where a step's decay is the one after it
    dq, last = _apply(dy * scale, vv, kk, first.transpose(-1, -2), *decays)
    nexts = torch.cat([_chunks(case, log, h)[..., 0].flatten(2)[:, :, 1:], log.new_zeros(b, h, 1)], -1).flip(-1).view(b, h, *q.shape[2:4])
    back = _decays(nexts)
    turn = lambda x: x.flip(2, 3)  # noqa: E731
    dk, _ = _apply(turn(vv), turn(dy * scale), turn(q), dlast.transpose(-1, -2), *back)
    dv, dstart = _apply(turn(kk), turn(q * scale), turn(dy), dlast, *back)
    out = {"dQ": _rows(case, _flat(case, dq, g), live, at, dt), "dK": _rows(case, _flat(case, turn(dk), g), live, at, dt),
           "dV": _rows(case, _flat(case, turn(dv), h), live, at, dt)}
    # pairs of steps on both sides of a decay: what goes to later steps less what earlier ones give, summed in 64 bits
    pairs = (q.double() * dq.double()).sum(-1) - (kk.double() * turn(dk).double()).sum(-1)
    pairs = pairs.flatten(2)
    ends = (last.double() * dlast.double().transpose(-1, -2)).sum((-1, -2))
    dlog = (pairs.flip(-1).cumsum(-1).flip(-1) + ends[..., None]).transpose(1, 2)[:, :s]
    dlog = dlog if live is None else dlog.masked_fill(~live[..., None], 0.0)
    if "G" in t:
        out["dG"] = _rows(case, dlog, live, at, torch.float32)
    else:
        out["d_decay"] = dlog.sum((0, 1)).float()
    if "initial_state" in t:
        out["d_initial_state"] = dstart * torch.exp(log[:, 0])[..., None, None]
    return out


def _split(case, x):
    """A head's rotated elements as pairs, and the rest."""
    r = case["rotary"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _join(case, a, b, rest):
    both = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _plain_rotary(case, t):
    n, d, dt = case["rows"], case["size"], DTYPES[case["dtype"]]
    at = t["positions"].long()
    cos, sin = t["cos"][at][:, None], t["sin"][at][:, None]
    out = {}
    for x, w, heads in (("Q", "q_scale", case["q_heads"]), ("K", "k_scale", case["k_heads"])):
        v, scale = t[x].float().view(n, heads, d), t[w].float()
        inv = torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
        if case["mode"] == "forward":
            a, b, rest = _split(case, v * inv * scale)
            out[x + "_out"] = _join(case, a * cos - b * sin, b * cos + a * sin, rest).to(dt).view(n, heads * d)
        else:
            a, b, rest = _split(case, t["d" + x + "_out"].float().view(n, heads, d))
            g = _join(case, a * cos + b * sin, b * cos - a * sin, rest)
            xh = v * inv
            out["d" + w] = (g * xh).sum((0, 1))
            g = g * scale
            out["d" + x] = (inv * (g - xh * (g * xh).mean(-1, keepdim=True))).to(dt).view(n, heads * d)
    return out


# ---- the definitions in 64 bits, one row after another: all pairs of steps, each by its own decay

def exact(case, seed):
    t = {k: v.double() if v.is_floating_point() else v for k, v in prepare(case, seed)["in"].items()}
    return _exact_rotary(case, t) if case["op"] == "rotary" else _exact_attn(case, t)


def _exact_attn(case, t):
    b, s, h, g, k, v = (case[n] for n in ("batch", "seq", "heads", "groups", "key", "value"))
    scale, of = k ** -0.5, torch.arange(h, device="cuda") // (h // g)
    lens = t["sequence_lens"].tolist() if "sequence_lens" in t else [s] * b
    back = case["mode"] == "backward"
    f64 = dict(dtype=torch.float64, device="cuda")
    shape = (s, b) if case["layout"] == 0 else (b, s)
    names = {"dQ": g * k, "dK": g * k, "dV": h * v, "dG": h} if back else {"Y": h * v}
    out = {n: torch.zeros(*shape, w, **f64) for n, w in names.items()}
    ends = torch.zeros(b, h, k, v, **f64)
    ddecay = torch.zeros(h, **f64)
    for i in range(b):
        at = torch.arange(lens[i], device="cuda")
        at = at.flip(0) if case["reverse"] else at
        where = (at, i) if case["layout"] == 0 else (i, at)

        def get(name, heads):
            return t[name][where].view(lens[i], heads, -1).transpose(0, 1)

        q, kk, vv = get("Q", g)[of], get("K", g)[of], get("V", h)
        log = get("G", h)[..., 0] if "G" in t else t["decay"][:, None].expand(h, lens[i])
        c = log.cumsum(-1)
        first = t["initial_state"][i] if "initial_state" in t else torch.zeros(h, k, v, **f64)
        last = torch.zeros(h, k, v, **f64)
        if back and "d_final_state" in t:
            last = t["d_final_state"][i]
        dy = get("dY", h) if back else None
        res = {n: torch.zeros(lens[i], w // (k if n in ("dQ", "dK") else v if n != "dG" else 1), k if n in ("dQ", "dK") else v if n != "dG" else 1, **f64)
               for n, w in names.items()}
        for j in range(h):  # one head's matrix of pairs at a time
            decay = torch.exp((c[j][:, None] - c[j][None, :]).masked_fill(~torch.ones(lens[i], lens[i], dtype=torch.bool, device="cuda").tril(), -math.inf))
            since, left = torch.exp(c[j]), torch.exp(c[j][-1] - c[j])
            score = scale * (q[j] @ kk[j].t())
            if not back:
                res["Y"][:, j] = (score * decay) @ vv[j] + scale * since[:, None] * (q[j] @ first[j])
                ends[i, j] = (kk[j] * left[:, None]).t() @ vv[j] + since[-1] * first[j]
                continue
            grad = scale * (dy[j] @ vv[j].t()) * decay
            res["dQ"][:, of[j]] += grad @ kk[j] + scale * since[:, None] * (dy[j] @ first[j].t())
            res["dK"][:, of[j]] += grad.t() @ q[j] + left[:, None] * (vv[j] @ last[j].t())
            res["dV"][:, j] = (score * decay).t() @ dy[j] + left[:, None] * (kk[j] @ last[j])
            ends[i, j] = scale * (q[j] * since[:, None]).t() @ dy[j] + since[-1] * last[j]
            # a decay's gradient: all pairs that it lies between, the states at both ends among them
            pair = torch.zeros(lens[i] + 1, lens[i] + 1, **f64)  # [later step or the end, the start or earlier step]
            pair[:-1, 1:] = grad * (q[j] @ kk[j].t())
            pair[:-1, 0] = scale * since * ((q[j] @ first[j]) * dy[j]).sum(-1)
            pair[-1, 1:] = left * ((kk[j] @ last[j]) * vv[j]).sum(-1)
            pair[-1, 0] = since[-1] * (first[j] * last[j]).sum()
            before = pair.cumsum(1)[:, :-1]  # [later, t]: from the start and steps before t
            res["dG"][:, j, 0] = before.tril().sum(0)
        for n in names:
            out[n][where] = res[n].flatten(1)
        if back:
            ddecay += res["dG"][..., 0].sum(0)
    if not back:
        return {"Y": out["Y"], "final_state": ends}
    if "G" not in t:
        del out["dG"]
        out["d_decay"] = ddecay
    return out | ({"d_initial_state": ends} if "initial_state" in t else {})


def _exact_rotary(case, t):
    n, d, r = case["rows"], case["size"], case["rotary"]
    first = torch.arange(r // 2, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else r // 2)
    turn = torch.eye(d, dtype=torch.float64, device="cuda").repeat(n, 1, 1)  # a row's rotation as a matrix
    at = t["positions"].long()
    turn[:, first, first] = turn[:, second, second] = t["cos"][at]
    turn[:, first, second], turn[:, second, first] = -t["sin"][at], t["sin"][at]
    out = {}
    for x, w, heads in (("Q", "q_scale", case["q_heads"]), ("K", "k_scale", case["k_heads"])):
        v = t[x].reshape(n, heads, d)
        root = torch.sqrt((v * v).sum(-1, keepdim=True) / d + 1e-6)
        if case["mode"] == "forward":
            out[x + "_out"] = (v / root * t[w]) @ turn.transpose(1, 2)
        else:
            g = t["d" + x + "_out"].reshape(n, heads, d) @ turn
            out["d" + w] = (g * v / root).sum((0, 1))
            g = g * t[w]
            out["d" + x] = g / root - v * (g * v).sum(-1, keepdim=True) / (d * root ** 3)
        for name in (x + "_out", "d" + x):
            if name in out:
                out[name] = out[name].reshape(n, heads * d)
    return out
