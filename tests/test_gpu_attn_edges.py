"""Linear attention on the GPU where values, sizes or what is asked for are far
from usual."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import ssm_reference as ref
from tests.gpu_harness import SENTINEL
from tests.test_gpu_attn import types, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("seq", [16, 3000])
def test_empty_batch(dtype, layout, seq):
    """A batch of no rows: the decays' gradient is zero, the others have no elements."""
    h, k, v = 4, 64, 64
    op = rl.LinearAttention(dtype=dtype, seq=seq, batch=0, heads=h, groups=2, key=k, value=v, layout=layout)
    lead = (seq, 0) if layout == 0 else (0, seq)
    e = {n: torch.empty(*lead, w, dtype=ref.TYPES[dtype], device="cuda") for n, w in (("Q", 2 * k), ("K", 2 * k), ("V", h * v), ("dY", h * v))}
    dd = torch.full((h,), SENTINEL, device="cuda")
    op.backward({**e, "d_decay": dd})
    torch.cuda.synchronize()
    assert (dd == 0).all()
    op.backward({**e, "dQ": torch.empty_like(e["Q"]), "dV": torch.empty_like(e["V"]), "d_decay": dd.fill_(SENTINEL)})
    torch.cuda.synchronize()
    assert (dd == 0).all()


@pytest.mark.parametrize("dtype,k,v", [("f32", 32, 128), ("f32", 128, 32), ("f32", 64, 128), ("f32", 200, 128), ("f16", 64, 200), ("f16", 200, 64),
                                       ("bf16", 64, 200), ("bf16", 200, 128)])
@pytest.mark.parametrize("s", [100, 600])
def test_each_gradient_alone(dtype, k, v, s):
    """Walks side by side of keys and values so unlike that each by itself would have chunks of its own length: each
    output alone is bit for bit that of all together, and of all with one that lies off any alignment."""
    b, h = 2, 4
    to = types(dtype)
    d = {n: x.to(to[n]).cuda() for n, x in values(dtype, b, s, h, 2, k, v).items()}
    op = rl.LinearAttention(dtype=dtype, seq=s, batch=b, heads=h, groups=2, key=k, value=v)
    shapes = {"dV": (b, s, h * v), "dQ": (b, s, 2 * k), "dK": (b, s, 2 * k), "dG": (b, s, h), "d_decay": (h,), "d_initial_state": (b, h, k, v)}
    for names in (("dQ", "dK", "dV", "d_initial_state"), ("dV", "dG", "d_decay", "d_initial_state")):
        full = {n: torch.empty(shapes[n], dtype=to[n], device="cuda") for n in names}
        op.backward({**d, **full})
        odd = {n: torch.empty_like(x) for n, x in full.items()}
        last = "dQ" if "dQ" in full else "dV"
        flat = torch.empty(odd[last].numel() + 1, dtype=to[last], device="cuda")
        odd[last] = flat[1:].view(shapes[last])
        op.backward({**d, **odd})
        for n in names:
            one = torch.empty_like(full[n])
            op.backward({**d, n: one})
            torch.cuda.synchronize()
            assert torch.equal(one, full[n]), n
            assert torch.equal(odd[n], full[n]), n


def test_tokens_of_many_rows():
    """A token of each of 16384 rows, 16 heads of 128 x 128: 2^32 elements of state, 16 GiB, updated in place; rows here and there."""
    b, h, k, v = 16384, 16, 128, 128
    gen = torch.Generator("cuda").manual_seed(3)

    def new(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    q, key, val = new(b, 1, h * k), new(b, 1, h * k), new(b, 1, h * v)
    decay = -torch.rand(h, generator=gen, device="cuda")
    state = torch.empty(b, h, k, v, device="cuda")
    state.normal_(generator=gen)
    at = [0, 1, 8191, 8192, 12345, b - 1]
    before = state[at].double()
    y = torch.empty_like(val)
    op = rl.LinearAttention(dtype="bf16", seq=1, batch=b, heads=h, key=k, value=v, scale=0.1)
    op.encode({"Q": q, "K": key, "V": val, "decay": decay, "initial_state": state, "final_state": state, "Y": y})
    torch.cuda.synchronize()
    qs, ks, vs = (t[at].double().view(len(at), h, -1) for t in (q, key, val))
    new_state = before * decay.double().exp()[:, None, None] + ks[..., None] * vs[..., None, :]
    out = 0.1 * (qs[..., None] * new_state).sum(-2)
    # (a product by a decay, its two roundings and its argument's, one by a value and a sum; sums of 128 and a scale)
    terms = before.abs() + ks.abs()[..., None] * vs.abs()[..., None, :]
    assert ((state[at].double() - new_state).abs() <= 6 * 2.0 ** -24 * terms).all()
    room = 2.0 ** -8 * out.abs() + 140 * 2.0 ** -24 * 0.1 * (qs.abs()[..., None] * terms).sum(-2)
    assert ((y[at].double().view(len(at), h, v) - out).abs() <= room).all()
