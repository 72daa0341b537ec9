"""The largest sizes that the state space operators and layer normalization
take, just below and at each limit (no GPU: nothing that is accepted is run)."""
import pytest

import onnx_recurrent_layers_amd as rl
from tests.test_ssm_host import FAKE, OPS, UNSUPPORTED, filled, refused


def created(op, fields):
    """Created and destroyed; with backward also its scratch sizes."""
    create, destroy, desc, _ = OPS[op]
    h = create(desc(**fields))
    destroy(h)


def at_call(op, fields, backward=False, **odd):
    """The call is refused, though the description is not: tensors named in `odd` are moved by so many bytes."""
    create, destroy, desc, start = OPS[op]
    h = create(desc(**fields))
    try:
        ops, grads = filled(op, "operands"), filled(op, "gradients")
        for name, by in odd.items():
            getattr(ops, name).ptr += by
        if backward:
            refused(lambda: getattr(rl, f"rnn_{op}_encode_backward")(h, ops, grads, FAKE << 8), UNSUPPORTED, start, "too large for one launch")
        else:
            refused(lambda: getattr(rl, f"rnn_{op}_encode")(h, ops, FAKE << 8), UNSUPPORTED, start, "too large for one launch")
    finally:
        destroy(h)


BF16 = dict(dtype=2)
# 8 channels a thread, 256 threads a workgroup: 4 workgroups for a row of 8192 channels; one thread a channel: 32
CONV = BF16 | dict(seq=1, channels=8192, width=4)


def test_conv_limits():
    created("conv", BF16 | dict(seq=65536, batch=16, channels=8192))
    created("conv", BF16 | dict(seq=65536, batch=16, channels=8190))
    created("conv", CONV | dict(batch=(1 << 22) - 1))
    refused(lambda: created("conv", CONV | dict(batch=1 << 22)), UNSUPPORTED, "conv: ", "too large for one launch")
    at_call("conv", CONV | dict(batch=1 << 19), X=2)
    at_call("conv", CONV | dict(batch=1 << 19), backward=True)      # four channels a thread, 64 such threads a workgroup
    created("conv", CONV | dict(channels=8191, batch=(1 << 19) - 1))
    refused(lambda: created("conv", CONV | dict(channels=8191, batch=1 << 19)), UNSUPPORTED, "conv: ", "too large for one launch")


def test_norm_limits():
    created("norm", BF16 | dict(rows=1 << 24, size=64))             # 16 threads a row
    created("norm", BF16 | dict(rows=(1 << 28) - 16, size=128))
    created("norm", BF16 | dict(rows=(1 << 28) - 16, size=1))
    refused(lambda: created("norm", BF16 | dict(rows=1 << 28, size=128)), UNSUPPORTED, "layer norm: ", "too large for one launch")
    created("norm", BF16 | dict(rows=(1 << 27) - 8, size=256))      # 32
    refused(lambda: created("norm", BF16 | dict(rows=1 << 27, size=256)), UNSUPPORTED, "layer norm: ", "too large for one launch")
    created("norm", BF16 | dict(rows=(1 << 26) - 4, size=512))      # a wave
    created("norm", BF16 | dict(rows=(1 << 26) - 4, size=2048))
    created("norm", BF16 | dict(rows=(1 << 24) - 1, size=2056))     # a workgroup
    refused(lambda: created("norm", BF16 | dict(rows=1 << 24, size=2056)), UNSUPPORTED, "layer norm: ", "too large for one launch")
    at_call("norm", BF16 | dict(rows=1 << 26, size=128), X=2)       # 128 values of one access each: a wave a row
    at_call("norm", BF16 | dict(rows=1 << 24, size=2048), X=2)
    at_call("norm", dict(dtype=0, rows=1 << 24, size=1024), X=4)    # (f32: a wave a row in whole pieces)
    h = OPS["norm"][0](OPS["norm"][2](**BF16, rows=1 << 24, size=64))
    parts = 512     # of sums over the rows, whatever their number
    assert rl.rnn_norm_scratch_size(h) == (0, parts * 2 * 64 * 4)
    rl.rnn_norm_destroy(h)


def test_scan_limits(monkeypatch):
    monkeypatch.delenv("RNN_SCAN_CHUNK", raising=False)
    scan = BF16 | dict(groups=1, state=128)
    created("scan", scan | dict(seq=131072, batch=64, channels=2048))
    created("scan", scan | dict(seq=16384, batch=64, channels=2048, groups=8))
    created("scan", scan | dict(seq=1, batch=1, channels=65536))
    created("scan", scan | dict(seq=1 << 20, batch=1 << 10, channels=2048, state=16, groups=32))     # B of 2^39 elements
    refused(lambda: created("scan", scan | dict(seq=1 << 20, batch=1 << 10, channels=2048, state=16, groups=64)), UNSUPPORTED, "scan: ", "2^40")
    # a token: workgroups of 256 threads, 64 channels each; the gradient of 128 states takes 512
    token = scan | dict(seq=1, channels=2048)
    created("scan", token | dict(batch=(1 << 19) - 1))
    refused(lambda: created("scan", token | dict(batch=1 << 19)), UNSUPPORTED, "scan: ", "too large for one launch")
    at_call("scan", token | dict(batch=1 << 18), backward=True)
    many = scan | dict(seq=5, channels=2048)
    created("scan", many | dict(batch=(1 << 18) - 1))
    refused(lambda: created("scan", many | dict(batch=1 << 18)), UNSUPPORTED, "scan: ", "too large for one launch")
