"""The state space operators on the GPU at the edges: scratch that another
stream's work may still hold."""
import pytest
import torch

import onnx_recurrent_layers_amd as rl

pytestmark = pytest.mark.gpu


def positive(b, s, c, n, groups=1, seed=0):
    """Inputs without a change of sign but A's: an infinite one makes infinite sums, and nothing that is not a number."""
    gen = torch.Generator().manual_seed(seed)
    shapes = dict(X=(b, s, c), delta=(b, s, c), A=(c, n), B=(b, s, groups * n), C=(b, s, groups * n), D=(c,), Z=(b, s, c), bias=(c,),
                  init=(b, c, n), dY=(b, s, c), dF=(b, c, n))
    v = {k: (torch.rand(*size, generator=gen, dtype=torch.float64) + 0.1).float().double() for k, size in shapes.items()}
    v["A"] = -v["A"]
    v["delta"] = (v["delta"] - 1).float().double()
    return v


def test_scratch_while_its_memory_is_in_use():
    """The first calls of an object on one stream, while work queued on the current one still writes memory that was
    given back: the size of the scratch, many times."""
    v = positive(2, 600, 130, 16)
    t = {k: v[k].to(torch.bfloat16).cuda() for k in ("X", "delta", "B", "C", "Z")} | {k: v[k].float().cuda() for k in ("A", "D")}
    outs = {"Y": torch.empty_like(t["X"]), "final_state": torch.empty(2, 130, 16, device="cuda")}
    grads = {"dX": torch.empty_like(t["X"]), "dA": torch.empty_like(t["A"]), "dB": torch.empty_like(t["B"])}
    dY = v["dY"].to(torch.bfloat16).cuda()

    def new():
        return rl.SelectiveScan(dtype="bf16", seq=600, batch=2, channels=130, state=16)

    op = new()
    assert op.forward_bytes and op.backward_bytes
    op.encode(t | outs)
    op.backward(t | grads | {"dY": dY})
    torch.cuda.synchronize()
    want = [x.clone() for x in (*outs.values(), *grads.values())]
    busy = torch.randn(4096, 4096, device="cuda")
    other = torch.cuda.Stream()
    del op
    for _ in range(3):
        op = new()
        other.wait_stream(torch.cuda.current_stream())       # (the inputs are there)
        for x in (*outs.values(), *grads.values()):
            x.record_stream(other)
        for size in (op.forward_bytes, op.backward_bytes):
            held = torch.empty(size // 4, device="cuda")
            for _ in range(8):
                busy = busy @ busy * 0.01
                held.copy_(busy.view(-1)[:1].expand_as(held))
            del held
        op.encode(t | outs, stream=other)
        op.backward(t | grads | {"dY": dY}, stream=other)
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip((*outs.values(), *grads.values()), want))
        for x in (*outs.values(), *grads.values()):
            x.fill_(3)
        torch.cuda.synchronize()
