"""Norms of queries and keys on the GPU where a call has less than the usual
operands."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl
from tests import ssm_reference as ref
from tests.test_gpu_rotary import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("names", [("dQ",), ("dq_scale",), ("dQ", "dq_scale")])
def test_queries_gradients_without_the_keys(dtype, names):
    """K is required with a gradient of the keys only, also where the gradient of their outputs is at hand."""
    rows, qh, kh, size = 70, 3, 2, 48
    dt = ref.TYPES[dtype]
    t = make(dtype, rows, qh, kh, size, size)
    d = {n: x.to({"cos": torch.float32, "sin": torch.float32, "positions": torch.int32}.get(n, dt)).cuda() for n, x in t.items()}
    op = rl.RotaryNorm(dtype=dtype, rows=rows, q_heads=qh, k_heads=kh, size=size, table=100)

    def new(n):
        return torch.empty(size, device="cuda") if n.endswith("scale") else torch.empty(rows, (qh if n == "dQ" else kh) * size, dtype=dt, device="cuda")

    whole = {n: new(n) for n in ("dQ", "dK", "dq_scale", "dk_scale")}
    op.backward({**d, **whole})
    out = {n: new(n) for n in names}
    op.backward({**{n: x for n, x in d.items() if n not in ("K", "k_scale")}, **out})
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(out[n], whole[n]), n
